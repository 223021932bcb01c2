"""The experts' products on the GPU against their 64-bit plain forms: ep_expert_gate_up,
ep_expert_down (bf16 and e4m3), ep_expert_down_grad, ep_expert_gate_up_grad and
ep_expert_weight_grad. Experts with no row, one, a few and many; widths from the smallest on,
odd ones; rows that belong to no expert; offsets past the buffer; streams and graphs."""
import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_experts as X
import plain_ops as P

pytestmark = pytest.mark.gpu

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
SENT = 0x7FC3  # a bf16 NaN pattern


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def sentinel(*shape):
    return torch.full(shape, SENT, dtype=torch.int16, device="cuda").view(BF16)


def flag():
    return torch.zeros(1, dtype=I32, device="cuda")


def rows_of(g, counts, lead, tail, W, scale=1.0):
    """bf16 rows, NaN before the first and behind the last expert's."""
    n = sum(counts)
    x = sentinel(lead + n + tail, W)
    x[lead:lead + n] = (torch.randn((n, W), generator=g, device="cuda") * scale).to(BF16)
    return x


def offsets(counts, lead):
    off = [lead]
    for c in counts:
        off.append(off[-1] + c)
    return off, torch.tensor(off, dtype=I32, device="cuda")


def weights(g, E, N, K):
    return (torch.randn((E, N, K), generator=g, device="cuda") * K**-0.5).to(BF16)


def codes(g, *shape):
    return (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(
        torch.float8_e4m3fn).view(U8)


def fp8_rows(g, counts, lead, tail, W):
    n = lead + sum(counts) + tail
    c, s = codes(g, n, W), torch.rand((n, W // 128), generator=g, device="cuda") * 0.01 + 0.001
    for part in (slice(0, lead), slice(lead + sum(counts), n)):
        c[part], s[part] = 0x7F, float("nan")
    return c, s


def fp8_weights(g, E, N, K):
    s = torch.rand((E, N // 128, K // 128), generator=g, device="cuda") + 0.5
    return codes(g, E, N, K), s * (0.01 * K**-0.5)


def finite(t, lo, hi):
    """The rows in use as 64-bit numbers, zeros elsewhere."""
    out = torch.zeros(t.shape, dtype=torch.float64)
    out[lo:hi] = P.f64(t[lo:hi])
    return out


def check(got, want, bound, lo, hi, what):
    """Rows lo .. hi - 1 within the bound; the others as they were."""
    X.assert_within(got[lo:hi], want[lo:hi], bound[lo:hi], what)
    for part in (got[:lo], got[hi:]):
        assert bool((part.contiguous().view(torch.int16) == SENT).all()), f"{what}: other rows"


# counts per expert, rows before the first and behind the last, H, I
SHAPES = [
    ([1], 0, 0, 8, 8),
    ([0, 1, 0], 3, 2, 64, 8),
    ([5, 0, 17, 1], 0, 7, 72, 24),
    ([16, 15, 33, 2], 1, 0, 128, 128),
    ([64, 31], 0, 5, 200, 136),
    ([256], 0, 0, 512, 256),
    ([257, 255, 0, 1], 2, 2, 256, 264),
    ([700, 3], 0, 9, 136, 520),
    ([40] * 9, 5, 5, 1024, 128),
    ([513, 100], 0, 1, 2056, 72),
    ([3] * 130, 0, 11, 64, 64),
    ([0, 0, 0], 2, 2, 64, 64),
    ([300, 20], 0, 0, 96, 1000),
]
FP8_SHAPES = [
    ([1], 0, 0, 128, 128),
    ([0, 1, 0], 3, 2, 256, 128),
    ([5, 0, 17, 1], 0, 7, 128, 384),
    ([16, 33, 2], 1, 0, 640, 256),
    ([257, 255, 0, 1], 2, 2, 384, 640),
    ([700, 3], 0, 9, 1024, 128),
    ([3] * 130, 0, 11, 128, 128),
    ([0, 0], 2, 2, 128, 128),
]


def ids(shapes):
    return [f"{sum(c)}rows{len(c)}e-{H}x{I}" for c, _, _, H, I in shapes]


@pytest.mark.parametrize("counts,lead,tail,H,I", SHAPES, ids=ids(SHAPES))
def test_gate_up(counts, lead, tail, H, I):
    g = gen(1 + H + I)
    off, offset = offsets(counts, lead)
    E, lo, hi = len(counts), off[0], off[-1]
    x, w = rows_of(g, counts, lead, tail, H), weights(g, E, 2 * I, H)
    n = x.shape[0]
    gu, err, act, act_err = X.gate_up(finite(x, lo, hi), P.f64(w), off)
    for kept in ["none", "bf16"] + (["fp8", "both"] if I % 128 == 0 else []):
        out, fl = sentinel(n, I), flag()
        kw = {}
        if kept in ("bf16", "both"):
            kw["gate_up"] = sentinel(n, 2 * I)
        if kept in ("fp8", "both"):
            kw["gate_up_fp8"] = torch.full((n, 2 * I), 0x5A, dtype=U8, device="cuda")
            kw["gate_up_scales"] = torch.full((n, 2 * I // 128), -3.0, device="cuda")
        ep.ep_expert_gate_up(x, w, offset, act=out, error_flag=fl, **kw)
        assert fl.item() == 0
        check(out, act, X.rounded(act, act_err), lo, hi, f"act, kept {kept}")
        if "gate_up" in kw:
            check(kw["gate_up"], gu, X.rounded(gu, err), lo, hi, "gate_up")
        if "gate_up_fp8" in kw:
            c, s = kw["gate_up_fp8"], kw["gate_up_scales"]
            check_codes(c, s, gu, err, lo, hi, "gate_up")


def check_codes(c, s, value, err, lo, hi, what):
    want = P.fp8_scales(value[lo:hi]) if hi > lo else torch.zeros((0, s.shape[1]), dtype=torch.float64)
    X.assert_within(s[lo:hi], want, X.scale_bound(value[lo:hi], err[lo:hi], want), f"{what} scales")
    X.assert_within(X.fp8_rows(c[lo:hi], s[lo:hi]), value[lo:hi],
                    X.codes_bound(value[lo:hi], err[lo:hi], want), f"{what} codes")
    for part in (slice(0, lo), slice(hi, None)):
        assert bool((c[part] == 0x5A).all()) and bool((s[part] == -3.0).all())


@pytest.mark.parametrize("counts,lead,tail,H,I", FP8_SHAPES, ids=ids(FP8_SHAPES))
def test_gate_up_fp8(counts, lead, tail, H, I):
    g = gen(2 + H + I)
    off, offset = offsets(counts, lead)
    E, lo, hi = len(counts), off[0], off[-1]
    (x, xs), (w, ws) = fp8_rows(g, counts, lead, tail, H), fp8_weights(g, E, 2 * I, H)
    n = x.shape[0]
    xv = torch.zeros((n, H), dtype=torch.float64)
    xv[lo:hi] = X.fp8_rows(x[lo:hi], xs[lo:hi])
    _, _, act, err = X.gate_up(xv, X.fp8_weights(w, ws), off, fp8=True)
    c = torch.full((n, I), 0x5A, dtype=U8, device="cuda")
    s, fl = torch.full((n, I // 128), -3.0, device="cuda"), flag()
    ep.ep_expert_gate_up_fp8(x, xs, w, ws, offset, act_fp8=c, act_scales=s, error_flag=fl)
    assert fl.item() == 0
    check_codes(c, s, act, err, lo, hi, "act")


@pytest.mark.parametrize("counts,lead,tail,H,I", SHAPES, ids=ids(SHAPES))
def test_down_and_gradients(counts, lead, tail, H, I):
    g = gen(3 + H + I)
    off, offset = offsets(counts, lead)
    E, lo, hi = len(counts), off[0], off[-1]
    act, w_down = rows_of(g, counts, lead, tail, I), weights(g, E, H, I)
    n = act.shape[0]
    out, fl = sentinel(n, H), flag()
    ep.ep_expert_down(act, w_down, offset, expert_out=out, error_flag=fl)
    want, mag = X.nt(finite(act, lo, hi), P.f64(w_down), off)
    check(out, want, X.rounded(want, X.product_error(I) * mag), lo, hi, "expert_out")

    # through the second product and the activation
    dout = rows_of(g, counts, lead, tail, H)
    for kept in ["bf16", "in place"] + (["fp8"] if I % 128 == 0 else []):
        dgu, a2, kw = sentinel(n, 2 * I), sentinel(n, I), {}
        if kept == "fp8":
            kw["gate_up_fp8"], kw["gate_up_scales"] = fp8_rows(g, counts, lead, tail, 2 * I)
            gu = torch.zeros((n, 2 * I), dtype=torch.float64)
            gu[lo:hi] = X.fp8_rows(kw["gate_up_fp8"][lo:hi], kw["gate_up_scales"][lo:hi])
        else:
            kw["gate_up"] = rows_of(g, counts, lead, tail, 2 * I, 3.0)
            gu = finite(kw["gate_up"], lo, hi)
            if kept == "in place":
                dgu, a2 = kw["gate_up"], None
        ep.ep_expert_down_grad(dout, w_down, offset, grad_gate_up=dgu, act=a2, error_flag=fl, **kw)
        grad, bound, again, again_bound = X.down_grad(finite(dout, lo, hi), P.f64(w_down), gu, off)
        check(dgu, grad, bound, lo, hi, f"grad_gate_up, kept {kept}")
        if a2 is not None:
            check(a2, again, again_bound, lo, hi, f"act again, kept {kept}")

    # through the first products
    w = weights(g, E, 2 * I, H)
    dgu = rows_of(g, counts, lead, tail, 2 * I)
    dx = sentinel(n, H)
    ep.ep_expert_gate_up_grad(dgu, w, offset, grad_x=dx, error_flag=fl)
    want, mag = X.nn(finite(dgu, lo, hi), P.f64(w), off)
    check(dx, want, X.rounded(want, X.product_error(2 * I) * mag), lo, hi, "grad_x")
    assert fl.item() == 0


@pytest.mark.parametrize("counts,lead,tail,H,I", FP8_SHAPES, ids=ids(FP8_SHAPES))
def test_down_fp8(counts, lead, tail, H, I):
    g = gen(4 + H + I)
    off, offset = offsets(counts, lead)
    E, lo, hi = len(counts), off[0], off[-1]
    (a, s), (w, ws) = fp8_rows(g, counts, lead, tail, I), fp8_weights(g, E, H, I)
    n = a.shape[0]
    av = torch.zeros((n, I), dtype=torch.float64)
    av[lo:hi] = X.fp8_rows(a[lo:hi], s[lo:hi])
    out, fl = sentinel(n, H), flag()
    ep.ep_expert_down_fp8(a.view(torch.float8_e4m3fn), s, w, ws, offset, expert_out=out,
                          error_flag=fl)
    want, mag = X.nt(av, X.fp8_weights(w, ws), off)
    check(out, want, X.rounded(want, X.product_error(I, True) * mag), lo, hi, "expert_out")
    assert fl.item() == 0


@pytest.mark.parametrize("counts,lead,tail,M,N", SHAPES, ids=ids(SHAPES))
def test_weight_grad(counts, lead, tail, M, N):
    g = gen(5 + M + N)
    off, offset = offsets(counts, lead)
    E, lo, hi = len(counts), off[0], off[-1]
    grad, inp = rows_of(g, counts, lead, tail, M), rows_of(g, counts, lead, tail, N)
    want, err = X.weight_grad(finite(grad, lo, hi), finite(inp, lo, hi), off)
    before = torch.randn((E, M, N), generator=g, device="cuda")
    fl = flag()
    for dtype in (F32, BF16):
        for accumulate in (False, True):
            out = before.to(dtype) if accumulate else torch.full((E, M, N), float("nan"),
                                                                 dtype=dtype, device="cuda")
            full = want + P.f64(out) if accumulate else want
            ep.ep_expert_weight_grad(grad, inp, offset, grad_weight=out, accumulate=accumulate,
                                     error_flag=fl)
            bound = X.rounded(full, err) if dtype is BF16 else err + 2 * P.U * full.abs()
            X.assert_within(out, full, bound, f"{dtype} accumulate={accumulate}")
    assert fl.item() == 0
