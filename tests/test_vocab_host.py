"""Refusals of the vocabulary operators: decided on the host, before anything
touches a device.  The addresses are never read."""
import ctypes

import pytest
import torch

OK, INVALID = 0, 1
F32, I32, BF16, I64 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from cluster_reductions_gb300 import build
    build.build()
    import cluster_reductions_gb300 as rr
    return rr.load()


A, B, C, D, E, G = (k << 32 for k in range(1, 7))     # far apart, aligned
f = ctypes.c_float


def test_embedding(lib):
    def call(w=A, V=10, D_=8, dt=BF16, tok=B, tdt=I32, n=4, scale=1.0, out=C):
        return lib.rr_embedding(w, V, D_, dt, tok, tdt, n, f(scale), out, None)
    assert call(n=0) == OK and call(D_=0) == OK
    for bad in (dict(V=-1), dict(V=2**31 - 1), dict(D_=-1), dict(D_=2**24 + 1), dict(n=-1),
                dict(n=2**30 + 1), dict(dt=I32), dict(dt=I64), dict(tdt=F32), dict(tdt=9),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(w=None), dict(tok=None),
                dict(out=None), dict(w=A + 1), dict(out=C + 1), dict(tok=B + 2), dict(tok=B + 4, tdt=I64),
                dict(dt=F32, w=A + 2), dict(out=A + 2), dict(out=B), dict(out=B - 16)):
        assert call(**bad) == INVALID, bad


def test_embedding_grad(lib):
    need = ctypes.c_size_t()
    assert lib.rr_embedding_grad_workspace_size(4, 8, ctypes.byref(need)) == OK
    assert lib.rr_embedding_grad_workspace_size(0, 8, ctypes.byref(ctypes.c_size_t())) == OK
    assert lib.rr_embedding_grad_workspace_size(-1, 8, ctypes.byref(need)) == INVALID
    assert lib.rr_embedding_grad_workspace_size(4, 8, None) == INVALID

    def call(dy=A, n=4, D_=8, dt=BF16, tok=B, tdt=I32, V=10, scale=1.0, dw=C, gdt=BF16, add=0, ws=D,
             nws=need.value):
        return lib.rr_embedding_grad(dy, n, D_, dt, tok, tdt, V, f(scale), dw, gdt, add, ws, nws, None)
    assert call(V=0) == OK and call(D_=0) == OK and call(n=0, add=1) == OK
    for bad in (dict(V=-1), dict(V=2**31 - 1), dict(D_=2**24 + 1), dict(n=2**30 + 1), dict(n=-2),
                dict(dt=I32), dict(gdt=I32), dict(dt=F32, gdt=BF16), dict(tdt=BF16),
                dict(scale=float("inf")), dict(dy=None), dict(tok=None), dict(dw=None), dict(ws=None),
                dict(ws=D + 8), dict(nws=need.value - 1), dict(dy=A + 1), dict(dw=C + 1),
                dict(gdt=F32, dw=C + 2), dict(tok=B + 1), dict(dw=A), dict(dw=B), dict(ws=C), dict(ws=A),
                dict(ws=B), dict(dw=D + 16)):
        assert call(**bad) == INVALID, bad


def test_embedding_grad_beyond_a_grid(lib):
    # (chunks of the list) x (column tiles) past 2^31 - 1 is refused before the
    # first launch, which would clear dw
    n, D_ = 2**30, 2**24
    need = ctypes.c_size_t()
    assert lib.rr_embedding_grad_workspace_size(n, D_, ctypes.byref(need)) == OK
    for add in (0, 1):
        st = lib.rr_embedding_grad(1 << 60, n, D_, BF16, 1 << 57, I32, 10, f(1.0), 1 << 56, BF16, add, 1 << 58,
                                   need.value, None)
        assert st == INVALID


def test_distill(lib):
    def loss(x=A, rows=3, V=100, ld=100, dt=BF16, idx=B, idt=I32, t=C, tdt=F32, K=5, T=1.0, lo=D, ls=E):
        return lib.rr_distill_loss(x, rows, V, ld, dt, idx, idt, t, tdt, K, f(T), lo, ls, None)

    def both(x=A, rows=3, V=100, ld=100, dt=BF16, idx=B, idt=I32, t=C, tdt=F32, K=5, T=1.0, g=G, lo=D,
             ls=E, dx=G << 1, ldx=100):
        return lib.rr_distill_loss_grad(x, rows, V, ld, dt, idx, idt, t, tdt, K, f(T), g, lo, ls, dx, ldx,
                                        None)

    def grad(x=A, rows=3, V=100, ld=100, dt=BF16, idx=B, idt=I32, t=C, tdt=F32, K=5, T=1.0, ls=E, g=G,
             dx=G << 1, ldx=100):
        return lib.rr_distill_grad(x, rows, V, ld, dt, idx, idt, t, tdt, K, f(T), ls, g, dx, ldx, None)
    for call in (loss, both, grad):
        assert call(rows=0) == OK
        for bad in (dict(rows=-1), dict(V=0), dict(V=2**31 - 1), dict(ld=99), dict(dt=I32), dict(idt=F32),
                    dict(tdt=I32), dict(K=0), dict(K=1025), dict(T=0.0), dict(T=-1.0),
                    dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-45), dict(x=None),
                    dict(idx=None), dict(t=None), dict(ls=None), dict(x=A + 1), dict(idx=B + 2),
                    dict(idx=B + 4, idt=I64), dict(t=C + 2), dict(ls=E + 2),
                    dict(rows=2**31, V=2**30, ld=2**31)):
            assert call(**bad) == INVALID, (call, bad)
    for call in (loss, both):
        for bad in (dict(lo=None), dict(lo=E), dict(lo=A), dict(ls=B), dict(ls=C), dict(lo=A + 500)):
            assert call(**bad) == INVALID, (call, bad)
    for call in (both, grad):
        for bad in (dict(g=None), dict(g=G + 1), dict(dx=None), dict(dx=A + 2), dict(dx=A, ldx=101),
                    dict(ldx=99), dict(dx=B), dict(dx=C), dict(dx=G), dict(dx=E), dict(dx=(G << 1) + 1)):
            assert call(**bad) == INVALID, (call, bad)


def test_sample(lib):
    from cluster_reductions_gb300._lib import rr_sample_params

    def call(x=A, rows=3, V=100, ld=100, dt=BF16, u=B, out=C, lp=D, **kw):
        p = rr_sample_params(1.0, 1.0, 0.0, 0, kw.get("T"), kw.get("p"), kw.get("q"), kw.get("k"))
        return lib.rr_sample(x, rows, V, ld, dt, u, ctypes.byref(p), out, lp, None)
    assert call(rows=0) == OK
    for bad in (dict(rows=-1), dict(V=0), dict(V=2**20 + 1), dict(ld=99), dict(dt=I32), dict(dt=I64),
                dict(x=None), dict(u=None), dict(out=None), dict(x=A + 1), dict(u=B + 2), dict(out=C + 1),
                dict(lp=D + 2), dict(out=A), dict(lp=A + 16), dict(out=B), dict(lp=C), dict(T=C),
                dict(p=D), dict(q=C + 4), dict(k=D), dict(T=E + 1), dict(k=E + 2)):
        assert call(**bad) == INVALID, bad


def test_binding_refuses():
    import cluster_reductions_gb300 as rr
    x = torch.zeros((3, 8))
    i, t, g = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2)), torch.zeros(3)
    z = torch.zeros(3, dtype=torch.int32)
    calls = [
        (ValueError, lambda: rr.embedding(x[0], z)),
        (TypeError, lambda: rr.embedding(x.half(), z)),
        (TypeError, lambda: rr.embedding(x, z.float())),
        (ValueError, lambda: rr.embedding_grad(x, z[:2], 5)),
        (TypeError, lambda: rr.embedding_grad(x, z.short(), 5)),
        (ValueError, lambda: rr.embedding_grad(x, z, 5, accumulate=True)),
        (TypeError, lambda: rr.embedding_grad(x, z, 5, dtype=torch.bfloat16)),
        (ValueError, lambda: rr.sample(x[None], g)),
        (ValueError, lambda: rr.sample(x.t(), g)),
        (ValueError, lambda: rr.sample(x[:1].expand(3, 8), g)),
        (ValueError, lambda: rr.distill_loss(x.t(), i, t)),
        (ValueError, lambda: rr.distill_loss(x[None], i, t)),
    ]
    for kind, call in calls:
        with pytest.raises(kind):
            call()


def test_first_argument_by_name():
    # every binding call takes its arguments by the names it documents: what
    # follows are refusals of values, which a call that lost its first argument
    # does not reach
    import cluster_reductions_gb300 as rr
    x, z = torch.zeros((3, 8)), torch.zeros(3, dtype=torch.int32)
    calls = [
        (ValueError, "weight must be", lambda: rr.embedding(weight=x[0], tokens=z)),
        (ValueError, "dy must be", lambda: rr.embedding_grad(dy=x, tokens=z[:2], num_embeddings=5)),
        (ValueError, "contiguous", lambda: rr.sample(x=x.t(), u=x[0])),
        (ValueError, "contiguous", lambda: rr.distill_loss(x=x.t(), idx=z, teacher=z)),
        (ValueError, "contiguous", lambda: rr.distill_grad(x=x.t(), idx=z, teacher=z, lse=z, grad_out=z)),
        (ValueError, "contiguous", lambda: rr.distill_loss_grad(x=x.t(), idx=z, teacher=z, grad_out=z)),
        (ValueError, "O must be", lambda: rr.splitk_combine(O=x, m=x, l=x, scale_log2e=1.0)),
        (ValueError, "vals must be", lambda: rr.cluster_allreduce(vals=x)),
        (ValueError, "contiguous", lambda: rr.softmax(x=x.t())),
    ]
    for kind, words, call in calls:
        with pytest.raises(kind, match=words):
            call()
    with pytest.raises(TypeError, match="missing"):
        rr.embedding(tokens=z)
