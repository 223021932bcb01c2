"""Plain 64-bit forms of the norm and of the expert-major operators, and the bounds their
fp32 kernels have to keep, for the tests. CPU float64 tensors in and out.

Bounds. u = 2^-24 is half a step of fp32, 2^-8 half a step of bf16 (relative to the value),
2^-4 of e4m3 (2^-10 below its smallest normal, 2^-6). A sum of n fp32 terms in any order is
off by at most (n - 1) u times the sum of the terms' magnitudes, to first order; the kernels'
row sums of H terms join per-lane chains of at most H / 64 terms with a tree, so n is at
most H / 64 + 16 there, and H / 64 + 16 <= 1024 for every width tested.
"""
import torch

BF16 = 2.0**-8
U = 2.0**-24
TINY_BF16 = 2.0**-133  # a bf16 subnormal's step
GROUP = 128


def f64(t):
    return t.detach().cpu().to(torch.float64)


def rmsnorm(x, residual, weight, eps):
    s = x if residual is None else x + residual
    r = 1.0 / torch.sqrt(s.square().mean(dim=1, keepdim=True) + eps)
    return s, s * r * weight


def fp8_scales(y):
    a = y.view(y.shape[0], -1, GROUP).abs().amax(dim=2)
    a = torch.where(a > 0, a.clamp(min=2.0**-100), torch.full_like(a, 448.0))
    return a / 448.0


def rmsnorm_grad(dy, dres, h, weight, eps):
    r = 1.0 / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps)
    n, g = h * r, dy * weight
    dx = r * (g - n * (g * n).mean(dim=1, keepdim=True))
    if dres is not None:
        dx = dx + dres
    return dx, (dy * n).sum(dim=0)


def gather(rows, slot):
    """[T][k][H]: the row of every pair, zeros where the pair is not routed."""
    got = rows[slot.clamp(min=0).long()]
    return torch.where((slot >= 0).unsqueeze(2), got, torch.zeros((), dtype=rows.dtype))


def unpermute(rows, w, slot, addend):
    got = gather(rows, slot)
    if w is not None:
        got = got * w.unsqueeze(2)
    out = got.sum(dim=1)
    return out if addend is None else out + addend


def unpermute_grad(dout, rows, w, slot):
    """(rows' gradient [T][k][H] by pair, the weights' gradient [T][k])."""
    wt = torch.ones(slot.shape, dtype=torch.float64) if w is None else w
    drows = torch.where((slot >= 0).unsqueeze(2), dout.unsqueeze(1) * wt.unsqueeze(2),
                        torch.zeros((), dtype=torch.float64))
    return drows, (gather(rows, slot) * dout.unsqueeze(1)).sum(dim=2)


# ---- bounds

def y_bound(y):
    # the row sum's relative error (at most 1024 u) is halved by the square root; mean, eps,
    # root, reciprocal and the two products add under 16 u: 2^-15 covers them; then one
    # rounding to bf16
    return (BF16 + 2.0**-15) * y.abs() + TINY_BF16


def sum_bound(s):
    return (BF16 + 2 * U) * s.abs() + TINY_BF16


def fp8_bound(y, scale):
    step = scale.repeat_interleave(GROUP, dim=1)
    code = torch.maximum(2.0**-4 * (y / step).abs(), torch.full_like(y, 2.0**-10))
    return step * code * (1 + 2.0**-12) + 2.0**-13 * y.abs()


def dx_bound(dx, dy, dres, h, weight, eps):
    # before the rounding, each term's error is under 2^-14 of its own magnitude: 1024 u
    # through the two sums, 1.5 times that through r^3, and a few u for the products
    r = 1.0 / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps)
    n, g = (h * r).abs(), (dy * weight).abs()
    a = r * (g + n * (g * n).mean(dim=1, keepdim=True))
    if dres is not None:
        a = a + dres.abs()
    return BF16 * dx.abs() + 2.0**-13 * a + TINY_BF16


def dw_bound(dy, h, eps):
    # T terms in some order, each with n = h r off by 2^-15 at most
    r = 1.0 / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps)
    mag = (dy * h * r).abs().sum(dim=0)
    return (h.shape[0] * U + 2.0**-15) * mag


def unpermute_bound(out, rows, w, slot, addend):
    mag = unpermute(rows.abs(), None if w is None else w.abs(), slot,
                    None if addend is None else addend.abs())
    return BF16 * out.abs() + (slot.shape[1] + 3) * U * mag + TINY_BF16


def dot_bound(dout, rows, slot):
    mag = (gather(rows, slot).abs() * dout.abs().unsqueeze(1)).sum(dim=2)
    return 1024 * U * mag


def assert_within(got, want, bound, what):
    """got (any float tensor) against want (64 bits); NaNs have to be in the same places."""
    g = f64(got)
    assert g.shape == want.shape, what
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaNs differ"
    off = torch.where(nan | (g == want), torch.zeros((), dtype=torch.float64), (g - want).abs() - bound)
    worst = off.flatten().argmax() if off.numel() else None
    assert worst is None or off.flatten()[worst] <= 0, (
        f"{what}: {g.flatten()[worst].item()} against {want.flatten()[worst].item()} at "
        f"{int(worst)}, bound {bound.flatten()[worst].item()}")
