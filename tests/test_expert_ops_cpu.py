"""CPU checks of the norm and the expert-major operators: argument validation through the C
ABI (nothing is enqueued, no GPU is touched: every call here fails validation or has no
tokens to work on), the binding's shape checks, and the 64-bit plain forms the GPU tests
compare with (their gradients against autograd and against differences)."""
import ctypes
import os

import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_ops as PL
from combine_ep_get_03_amd import _binding

P = ctypes.c_void_p
A16 = P(0x10000)   # an aligned, non-NULL stand-in (never dereferenced)
B16 = P(0x20000)
A8 = P(0x10008)
A4 = P(0x10004)
MIS = P(0x10001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_binding.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return ep.load()


def norm(lib, x=A16, res=A16, w=A16, f32=0, eps=1e-6, T=4, H=256, ro=A16, y=B16, c=A16, s=A16):
    return lib.ep_rmsnorm(x, res, w, f32, eps, T, H, ro, y, c, s, None)


def test_norm_refusals(lib):
    for bad in (dict(T=-1), dict(H=0), dict(H=-8), dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF),
                dict(T=2**31), dict(H=2**30), dict(x=None), dict(w=None), dict(res=None),
                dict(c=None), dict(s=None), dict(ro=None, y=None, c=None, s=None),
                dict(y=A16)):  # y and residual_out in one place
        assert norm(lib, **bad) == ep.EP_ERR_ARG, bad
    for bad in (dict(H=252), dict(H=264), dict(x=A8), dict(res=A8), dict(w=A8), dict(ro=A8),
                dict(y=A8), dict(c=A4), dict(s=MIS)):
        assert norm(lib, **bad) == ep.EP_ERR_ALIGN, bad
    assert norm(lib, T=0) == ep.EP_OK
    assert norm(lib, T=0, H=264, c=None, s=None) == ep.EP_OK  # multiples of 8 without e4m3


def norm_grad(lib, dy=A16, dr=A16, h=A16, w=A16, f32=0, eps=1e-6, T=4, H=256, dx=A16, dw=A16,
              ws=A16, wsb=1 << 30):
    return lib.ep_rmsnorm_grad(dy, dr, h, w, f32, eps, T, H, dx, dw, ws, wsb, None)


def test_norm_grad_refusals(lib):
    for bad in (dict(T=-1), dict(H=0), dict(eps=-1.0), dict(eps=NAN), dict(dy=None), dict(h=None),
                dict(w=None), dict(dx=None), dict(T=2**31), dict(H=2**30)):
        assert norm_grad(lib, **bad) == ep.EP_ERR_ARG, bad
    for bad in (dict(H=252), dict(dy=A8), dict(dr=A8), dict(h=A8), dict(w=A8), dict(dx=A8),
                dict(dw=MIS), dict(ws=A8)):
        assert norm_grad(lib, **bad) == ep.EP_ERR_ALIGN, bad
    need = ep.ep_rmsnorm_grad_workspace_bytes(4, 256)
    assert need > 0
    assert norm_grad(lib, wsb=need - 1) == ep.EP_ERR_CAPACITY
    assert norm_grad(lib, ws=None) == ep.EP_ERR_CAPACITY
    assert norm_grad(lib, T=0, dw=None, ws=None, wsb=0) == ep.EP_OK


def test_norm_grad_workspace_query(lib):
    assert ep.ep_rmsnorm_grad_workspace_bytes(0, 256) == 0
    for T, H in [(-1, 256), (4, 0), (4, 252), (4, 2**30), (2**31, 256)]:
        assert ep.ep_rmsnorm_grad_workspace_bytes(T, H) == 0
    for H in (8, 512, 1024, 2056, 7168, 16384, 40960):  # enough for a larger batch is enough
        sizes = [ep.ep_rmsnorm_grad_workspace_bytes(T, H) for T in
                 [*range(1, 1100), 2047, 2048, 2049, 4096, 4099, 100000]]
        assert sizes == sorted(sizes), H
    for T in (1, 100, 4096, 100000):
        assert 0 < ep.ep_rmsnorm_grad_workspace_bytes(T, 7168) < 64 << 20


def perm8(lib, x=A16, sc=A16, w=A16, T=4, H=256, k=2, slot=A16, px=A16, ps=A16, pw=A16, pi=A16,
          cap=8, err=A16):
    return lib.ep_dispatch_permute_fp8(x, sc, w, T, H, k, slot, px, ps, pw, pi, cap, err, None)


def unperm(lib, rows=A16, n=8, w=A16, T=4, H=256, k=2, slot=A16, add=A16, out=A16, err=A16):
    return lib.ep_combine_unpermute(rows, n, w, T, H, k, slot, add, out, err, None)


def unperm_grad(lib, go=A16, rows=A16, n=8, w=A16, T=4, H=256, k=2, slot=A16, gr=A16, gw=A16,
                err=A16):
    return lib.ep_combine_unpermute_grad(go, rows, n, w, T, H, k, slot, gr, gw, err, None)


def perm_grad(lib, gp=A16, gpw=A16, n=8, T=4, H=256, k=2, slot=A16, gx=A16, gw=A16, err=A16):
    return lib.ep_dispatch_permute_grad(gp, gpw, n, T, H, k, slot, gx, gw, err, None)


def test_expert_rows_size_refusals(lib):
    for f, rows in ((perm8, "cap"), (unperm, "n"), (unperm_grad, "n"), (perm_grad, "n")):
        for bad in (dict(T=-1), dict(H=0), dict(k=0), dict(k=-1), dict(k=8193), {rows: -1},
                    dict(T=2**30, k=4),
                    dict(H=2**30)):
            assert f(lib, **bad) == ep.EP_ERR_ARG, (f.__name__, bad)
        assert f(lib, H=252) == ep.EP_ERR_ALIGN
        assert f(lib, T=0) == ep.EP_OK
    assert perm8(lib, H=264) == ep.EP_ERR_ALIGN


def test_expert_rows_pointer_refusals(lib):
    for name in ("x", "sc", "slot", "px", "ps", "w"):  # w: needed by perm_weights
        assert perm8(lib, **{name: None}) == ep.EP_ERR_ARG, name
    for name in ("rows", "slot", "out"):
        assert unperm(lib, **{name: None}) == ep.EP_ERR_ARG, name
    for name in ("go", "rows", "slot", "gr"):  # rows: needed by grad_topk_weights
        assert unperm_grad(lib, **{name: None}) == ep.EP_ERR_ARG, name
    for name in ("gp", "gpw", "slot", "gx"):  # gpw: needed by grad_topk_weights
        assert perm_grad(lib, **{name: None}) == ep.EP_ERR_ARG, name
    for f, rows, words in ((perm8, ("x", "px"), ("sc", "w", "slot", "ps", "pw", "pi", "err")),
                           (unperm, ("rows", "add", "out"), ("w", "slot", "err")),
                           (unperm_grad, ("go", "rows", "gr"), ("w", "slot", "gw", "err")),
                           (perm_grad, ("gp", "gx"), ("gpw", "slot", "gw", "err"))):
        for name in rows:
            assert f(lib, **{name: A8}) == ep.EP_ERR_ALIGN, (f.__name__, name)
        for name in words:
            assert f(lib, **{name: MIS}) == ep.EP_ERR_ALIGN, (f.__name__, name)


@pytest.mark.skipif(torch.cuda.is_available() or os.path.exists("/dev/kfd"),
                    reason="the stand-in pointers are only safe where no kernel can start")
def test_a_launch_that_fails_is_reported(lib):
    """Without a GPU every launch fails: each call that gets past its checks says so, in each
    of its forms."""
    big = 1 << 40
    for kw in (dict(), dict(H=64, c=None, s=None), dict(H=1024), dict(H=2048), dict(H=32768),
               dict(H=40960), dict(T=5_000_000, H=1024)):
        assert norm(lib, **kw) == ep.EP_ERR_HIP, kw
    for kw in (dict(), dict(dw=None), dict(T=5000, H=8192), dict(H=40960), dict(H=40960, dw=None),
               dict(T=1, H=64), dict(T=0)):
        assert norm_grad(lib, wsb=big, **kw) == ep.EP_ERR_HIP, kw
    for kw in (dict(), dict(H=2048), dict(H=8192), dict(H=40960), dict(T=100000, k=8, H=7168),
               dict(T=2**24, k=8)):
        assert perm8(lib, cap=2**40, **kw) == ep.EP_ERR_HIP, kw
    for kw in (dict(), dict(k=1), dict(k=3), dict(k=8), dict(T=2**24 + 1, k=1)):
        assert unperm(lib, n=2**40, **kw) == ep.EP_ERR_HIP, kw
        assert perm_grad(lib, n=2**40, **kw) == ep.EP_ERR_HIP, kw
    for kw in (dict(), dict(gw=None), dict(T=5000, k=8, H=7168), dict(T=3000, k=2),
               dict(T=2**22, k=8)):
        assert unperm_grad(lib, n=2**40, **kw) == ep.EP_ERR_HIP, kw


def test_binding_refuses_shapes_types_and_host_tensors():
    T, H, k = 4, 256, 2
    x = torch.zeros((T, H), dtype=torch.bfloat16)
    w = torch.ones(H)
    slot = torch.zeros((T, k), dtype=torch.int32)
    gate = torch.ones((T, k))
    rows = torch.zeros((T * k, H), dtype=torch.bfloat16)
    c8, s8 = torch.zeros((T, H), dtype=torch.uint8), torch.ones((T, H // 128))
    p8, ps = torch.zeros((T * k, H), dtype=torch.uint8), torch.ones((T * k, H // 128))
    bad_shapes = [
        lambda: ep.ep_rmsnorm(x, w, y=x[:3]),
        lambda: ep.ep_rmsnorm(x, w[:8], y=x),
        lambda: ep.ep_rmsnorm(x, w, residual=x[:, :8], y=x),
        lambda: ep.ep_rmsnorm(x, w, y_fp8=c8, y_scales=s8[:, :1]),
        lambda: ep.ep_rmsnorm(x.view(2, 2, H), w, y=x),
        lambda: ep.ep_rmsnorm_grad(x, x, w, grad_x=x[:2]),
        lambda: ep.ep_rmsnorm_grad(x, x, w, grad_x=x, grad_weight=w[:8]),
        lambda: ep.ep_dispatch_permute_fp8(c8, s8[:2], None, slot, perm_x_fp8=p8, perm_scales=ps),
        lambda: ep.ep_dispatch_permute_fp8(c8, s8, gate[:1], slot, perm_x_fp8=p8, perm_scales=ps),
        lambda: ep.ep_dispatch_permute_fp8(c8, s8, None, slot[:1], perm_x_fp8=p8, perm_scales=ps),
        lambda: ep.ep_dispatch_permute_fp8(c8, s8, None, slot, perm_x_fp8=p8, perm_scales=ps[:2]),
        lambda: ep.ep_combine_unpermute(rows, gate[:, :1], slot, out=x),
        lambda: ep.ep_combine_unpermute(rows, gate, slot, out=x[:, :8]),
        lambda: ep.ep_combine_unpermute(rows, gate, slot, out=x, addend=x[:1]),
        lambda: ep.ep_combine_unpermute_grad(x, rows[:3], gate, slot, grad_expert_out=rows),
        lambda: ep.ep_combine_unpermute_grad(x, rows, gate, slot[:2], grad_expert_out=rows),
        lambda: ep.ep_combine_unpermute_grad(x, rows, gate, slot, grad_expert_out=rows,
                                             grad_topk_weights=gate[:1]),
        lambda: ep.ep_dispatch_permute_grad(rows, slot, grad_x=x[:1]),
        lambda: ep.ep_dispatch_permute_grad(rows, slot, grad_x=x, grad_perm_weights=gate),
    ]
    for i, f in enumerate(bad_shapes):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError, match="weight"):
        ep.ep_rmsnorm(x, w.double(), y=x)
    with pytest.raises(TypeError):
        ep.ep_combine_unpermute(rows.float(), gate, slot, out=x)
    for f in (lambda: ep.ep_rmsnorm(x, w, y=x),
              lambda: ep.ep_combine_unpermute(rows, gate, slot, out=x)):
        with pytest.raises(ValueError, match="device tensor"):
            f()


# ---- the plain forms: gradients against autograd and against differences

def leaf(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float64).requires_grad_()


def by_differences(f, t, d, step=1e-5):
    """The derivative of f() along d at the leaf t, by central differences."""
    with torch.no_grad():
        t += step * d
        up = f()
        t -= 2 * step * d
        down = f()
        t += step * d
    return (up - down) / (2 * step)


def check_gradient(f, grads, g):
    """grads: {leaf: gradient}; f's own autograd and central differences give the same."""
    f().backward()
    for t, got in grads:
        assert torch.allclose(t.grad, got, rtol=1e-10, atol=1e-12)
        d = torch.randn(t.shape, generator=g, dtype=torch.float64)
        want = by_differences(lambda: f().detach(), t, d)
        assert abs(want - (got * d).sum()) <= 1e-7 * (1 + (got * d).abs().sum())


def test_plain_norm_gradient():
    g = torch.Generator().manual_seed(0)
    x, res, w = leaf(g, 5, 24), leaf(g, 5, 24), leaf(g, 24)
    dy, ds = torch.randn((2, 5, 24), generator=g, dtype=torch.float64)

    def f():
        s, y = PL.rmsnorm(x, res, w, 1e-3)
        return (s * ds).sum() + (y * dy).sum()

    with torch.no_grad():
        dx, dw = PL.rmsnorm_grad(dy, ds, x + res, w, 1e-3)
    check_gradient(f, [(x, dx), (res, dx), (w, dw)], g)


def test_plain_unpermute_gradients():
    g = torch.Generator().manual_seed(1)
    T, k, H, cap = 6, 3, 10, 20
    slot = torch.randperm(cap, generator=g)[:T * k].reshape(T, k)
    slot[0] = -1
    slot[3, 1] = -1
    rows, w, add = leaf(g, cap, H), leaf(g, T, k), leaf(g, T, H)
    do = torch.randn((T, H), generator=g, dtype=torch.float64)
    with torch.no_grad():
        by_pair, dw = PL.unpermute_grad(do, rows, w, slot)
        drows = torch.zeros((cap, H), dtype=torch.float64)
        drows[slot[slot >= 0]] = by_pair[slot >= 0]
    check_gradient(lambda: (PL.unpermute(rows, w, slot, add) * do).sum(),
                   [(rows, drows), (w, dw), (add, do)], g)


def test_plain_permute_gradient():
    g = torch.Generator().manual_seed(2)
    T, k, H, cap = 5, 4, 7, 20
    slot = torch.randperm(cap, generator=g)[:T * k].reshape(T, k)
    slot[2, :2] = -1
    x = leaf(g, T, H)
    dp = torch.randn((cap, H), generator=g, dtype=torch.float64)
    t, j = torch.nonzero(slot >= 0, as_tuple=True)
    with torch.no_grad():
        dx = PL.unpermute(dp, None, slot, None)
    check_gradient(lambda: (x[t] * dp[slot[t, j]]).sum(), [(x, dx)], g)


def test_bounds_reject_a_planted_mistake():
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn((4, 256), generator=g, dtype=torch.float64), torch.ones(256, dtype=torch.float64)
    _, y = PL.rmsnorm(x, None, w, 1e-6)
    PL.assert_within(y.to(torch.bfloat16), y, PL.y_bound(y), "y")
    wrong = x / torch.sqrt(x.square().sum(dim=1, keepdim=True) / 248 + 1e-6)  # a width off by 8
    with pytest.raises(AssertionError):
        PL.assert_within(wrong.to(torch.bfloat16), y, PL.y_bound(y), "y")
    slot = torch.arange(8).reshape(4, 2)
    rows = torch.randn((8, 256), generator=g, dtype=torch.float64)
    gate = torch.rand((4, 2), generator=g, dtype=torch.float64)
    out = PL.unpermute(rows, gate, slot, None)
    with pytest.raises(AssertionError):  # two slots of a token swapped
        PL.assert_within(PL.unpermute(rows, gate, slot.flip(1), None), out,
                         PL.unpermute_bound(out, rows, gate, slot, None), "out")
