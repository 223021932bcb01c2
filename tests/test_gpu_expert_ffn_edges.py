"""The experts' products at the edges of their contract: sums that do not depend on the other
experts' rows; pieces of tiles that get no row; arrays of no rows;
sums whose largest products cancel."""
import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_experts as X
import plain_ops as P
from test_gpu_expert_ffn import (BF16, I32, U8, check, check_codes, finite, flag, fp8_rows, fp8_weights, gen,
                                 offsets, rows_of, sentinel, weights)

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8)


# The first expert's rows beside others of the same number in all, whose tiles fill the last round
# more or less, so that the first expert's are whole in one call and cut in two or four in the
# other; of 128 and of 256 rows.
BESIDE = [([128, 128, 128, 128], [128, 129, 129, 126], 4096), ([100, 156, 128, 128], [100, 154, 129, 129], 4096),
          ([70, 186, 128, 128], [70, 130, 130, 182], 4096), ([256, 256, 256, 256], [256, 257, 257, 254], 4096),
          ([200, 256, 256, 256, 0], [200, 257, 257, 254, 0], 4096),
          ([128, 128, 128, 128], [128, 129, 129, 126], 8192),
          ([256, 256, 256, 256], [256, 257, 257, 254], 8192),
          ([200, 256, 256, 256, 0], [200, 257, 257, 254, 0], 8192)]


@pytest.mark.parametrize("counts,others,I", BESIDE, ids=lambda v: str(v))
def test_a_row_is_the_same_beside_other_rows(counts, others, I):
    """Sums in an order fixed by the sizes and the expert's own rows."""
    print(f"\ncase: {counts} {others} {I}", flush=True)
    H, E, n, mine = 256, len(counts), sum(counts), counts[0]
    assert sum(others) == n and others[0] == mine
    g = gen(50 + mine)
    x, dout = rows_of(g, counts, 0, 0, H), rows_of(g, counts, 0, 0, H)
    wide, act = rows_of(g, counts, 0, 0, 2 * I), rows_of(g, counts, 0, 0, I)
    w, wd, wb = weights(g, E, 2 * I, H), weights(g, E, H, I), weights(g, E, I, H)
    (x8, xs), (w8, ws) = fp8_rows(g, counts, 0, 0, H), fp8_weights(g, E, 2 * I, H)
    wd8, wds = fp8_weights(g, E, I, H)  # the second product with as many output channels
    got = []
    for c in (counts, others):
        _, offset = offsets(c, 0)
        fl = flag()
        o = dict(act=torch.zeros((n, I), dtype=BF16), gu=torch.zeros((n, 2 * I), dtype=BF16),
                 codes=torch.zeros((n, 2 * I), dtype=U8), scales=torch.zeros((n, 2 * I // 128)),
                 act8=torch.zeros((n, I), dtype=U8), act8s=torch.zeros((n, I // 128)),
                 down=torch.zeros((n, I), dtype=BF16), down8=torch.zeros((n, I), dtype=BF16),
                 dgu=torch.zeros((n, 2 * I), dtype=BF16), dx=torch.zeros((n, I), dtype=BF16))
        o = {k: v.cuda() for k, v in o.items()}
        ep.ep_expert_gate_up(x, w, offset, act=o["act"], gate_up=o["gu"], gate_up_fp8=o["codes"],
                             gate_up_scales=o["scales"], error_flag=fl)
        ep.ep_expert_gate_up_fp8(x8, xs, w8, ws, offset, act_fp8=o["act8"], act_scales=o["act8s"],
                                 error_flag=fl)
        ep.ep_expert_down(x, wb, offset, expert_out=o["down"], error_flag=fl)
        ep.ep_expert_down_fp8(x8, xs, wd8, wds, offset, expert_out=o["down8"], error_flag=fl)
        ep.ep_expert_down_grad(dout, wd, offset, grad_gate_up=o["dgu"], gate_up=wide, error_flag=fl)
        ep.ep_expert_gate_up_grad(x, w[:, :H].contiguous().view(E, H, H).repeat(1, 1, I // H), offset,
                                  grad_x=o["dx"], error_flag=fl)
        assert fl.item() == 0
        got.append(o)
    for name in got[0]:
        a, b = (o[name][:mine] for o in got)
        assert bool(a.any()), name
        same = torch.equal(bits(a), bits(b))
        assert same, name


# One row of the last expert, in tiles that are cut in two or four because the last round has room:
# the pieces behind the first get no row, and would begin in the rows of no expert. Of the lowest,
# the middle and the highest tiles.
ONE_ROW = [([30, 0, 0, 1], 49, 4096), ([70, 0, 0, 1], 310, 5504), ([200, 1], 399, 8192), ([200, 1], 1399, 4096)]


@pytest.mark.parametrize("counts,tail,I", ONE_ROW, ids=lambda v: str(v))
def test_a_piece_without_rows_writes_nothing(counts, tail, I):
    print(f"\ncase: {counts} {tail} {I}", flush=True)
    g, H = gen(60 + I), 64
    off, offset = offsets(counts, 0)
    x, w = rows_of(g, counts, 0, tail, H), weights(g, len(counts), 2 * I, H)
    n, hi, fl = x.shape[0], off[-1], flag()
    act, gu = sentinel(n, I), sentinel(n, 2 * I)
    c = torch.full((n, 2 * I), 0x5A, dtype=U8, device="cuda")
    s = torch.full((n, 2 * I // 128), -3.0, device="cuda")
    ep.ep_expert_gate_up(x, w, offset, act=act, gate_up=gu, gate_up_fp8=c, gate_up_scales=s, error_flag=fl)
    want, err, wact, act_err = X.gate_up(finite(x, 0, hi), P.f64(w), off)
    check(act, wact, X.rounded(wact, act_err), 0, hi, "act")
    check(gu, want, X.rounded(want, err), 0, hi, "gate_up")
    check_codes(c, s, want, err, 0, hi, "gate_up")
    assert fl.item() == 0


@pytest.mark.parametrize("off,sets", [([0, 0, 0], False), ([0, 5, 9], True), ([0, 3, 1], True),
                                      ([-1, 0, 0], True)], ids=str)
def test_arrays_of_no_rows(off, sets):
    """Nothing to compute: the row-wise calls launch nothing and leave the flag, whatever the
    offsets; the weights' gradients write their zeros and look at them."""
    E, H, I = 2, 128, 128
    offset = torch.tensor(off, dtype=I32, device="cuda")
    b = lambda *s: torch.empty(s, dtype=BF16, device="cuda")
    u = lambda *s: torch.empty(s, dtype=U8, device="cuda")
    f = lambda *s: torch.ones(s, device="cuda")
    fl = flag()
    ep.ep_expert_gate_up(b(0, H), b(E, 2 * I, H), offset, act=b(0, I), gate_up=b(0, 2 * I), error_flag=fl)
    ep.ep_expert_gate_up_fp8(u(0, H), f(0, 1), u(E, 2 * I, H), f(E, 2, 1), offset, act_fp8=u(0, I),
                             act_scales=f(0, 1), error_flag=fl)
    ep.ep_expert_down(b(0, I), b(E, H, I), offset, expert_out=b(0, H), error_flag=fl)
    ep.ep_expert_down_fp8(u(0, I), f(0, 1), u(E, H, I), f(E, 1, 1), offset, expert_out=b(0, H), error_flag=fl)
    ep.ep_expert_down_grad(b(0, H), b(E, H, I), offset, grad_gate_up=b(0, 2 * I), gate_up=b(0, 2 * I),
                           act=b(0, I), error_flag=fl)
    ep.ep_expert_gate_up_grad(b(0, 2 * I), b(E, 2 * I, H), offset, grad_x=b(0, H), error_flag=fl)
    assert fl.item() == 0
    dw = f(E, H, I)
    ep.ep_expert_weight_grad(b(0, H), b(0, I), offset, grad_weight=dw, error_flag=fl)
    assert (fl.item() == ep.EP_DEVERR_SLOT_RANGE) == sets
    ascending = off[0] >= 0 and all(x <= y for x, y in zip(off, off[1:]))
    assert bool((dw == (0.0 if ascending else 1.0)).all())


# A block's largest products, of +448^2 and -448^2, cancel beside others of these sizes; or one
# product of 2^16 stands beside 127 that lie just below 14 bits under it.
CANCEL = [400.0, 100.0, 10.0, 1.0, 0.1, "beside"]


def cancelling(g, size, n, N, K):
    """Codes of n rows and N channels of the weights."""
    if size == "beside":
        a, b = torch.full((n, K), 1.875, device="cuda"), torch.full((1, N, K), 1.875, device="cuda")
        at = torch.randint(0, 128, (K // 128,), generator=g, device="cuda")
        for block, place in enumerate(at.tolist()):
            a[:, 128 * block + place] = 256
            b[:, :, 128 * block + place] = 256
    else:
        a = (torch.randn((n, K), generator=g, device="cuda") * size).clamp(-448, 448)
        b = (torch.randn((1, N, K), generator=g, device="cuda") * size).clamp(-448, 448)
        a[:, ::128], a[:, 64::128], b[:, :, ::128], b[:, :, 64::128] = 448, 448, 448, -448
    return (t.to(torch.float8_e4m3fn).view(U8) for t in (a, b))


@pytest.mark.parametrize("n,N,K", [(40, 256, 128), (600, 16384, 512)])
@pytest.mark.parametrize("size", CANCEL)
def test_sums_whose_largest_products_cancel(size, n, N, K):
    """ep_expert_down_fp8 within 2^-11 of its products' magnitudes, ep_expert_gate_up_fp8 within what
    sums in fp32 keep; scales 1 and 2^-16, so that the activation does not overflow."""
    print(f"\ncase: {size} {n} {N} {K}", flush=True)
    g = gen(70 + K)
    a, b = cancelling(g, size, n, N, K)
    offset, fl = torch.tensor([0, n], dtype=I32, device="cuda"), flag()
    s, ws = torch.ones((n, K // 128), device="cuda"), torch.ones((1, N // 128, K // 128), device="cuda")
    out = sentinel(n, N)
    ep.ep_expert_down_fp8(a, s, b, ws, offset, expert_out=out, error_flag=fl)
    want, mag = X.nt(X.fp8_rows(a, s), X.fp8_weights(b, ws), [0, n])
    # 7 of 8 products lose at most 2^-14 of the largest, less than 2^-11; the blocks' sums in fp32
    X.assert_within(out, want, X.rounded(want, (2.0**-11 + (K / 128 + 4) * 2.0**-23) * mag), "expert_out")
    ws = ws * 2.0**-16
    c = torch.full((n, N // 2), 0x5A, dtype=U8, device="cuda")
    cs = torch.full((n, N // 256), -3.0, device="cuda")
    ep.ep_expert_gate_up_fp8(a, s, b, ws, offset, act_fp8=c, act_scales=cs, error_flag=fl)
    _, _, act, err = X.gate_up(X.fp8_rows(a, s), X.fp8_weights(b, ws), [0, n], fp8=True)
    check_codes(c, cs, act, err, 0, n, "act")
    assert fl.item() == 0


# Gate and up kept in e4m3, and the gradient written over gate_up, in each of the three tiles (rows
# per expert and outputs decide): 32, 128 and 256 rows; a last expert of one row, rows of no expert.
KEPT = [([5, 0, 17, 1], 3, 2, 72, 384), ([70, 0, 60, 1], 1, 130, 40, 11008), ([200, 140, 1], 2, 130, 72, 11008),
        ([300, 257, 0, 129, 1], 3, 30, 40, 8192)]


@pytest.mark.parametrize("counts,lead,tail,H,I", KEPT, ids=lambda v: str(v))
def test_down_gradient_of_every_kept_form_in_every_tile(counts, lead, tail, H, I):
    print(f"\ncase: {counts} {H} {I}", flush=True)
    g = gen(80 + I)
    off, offset = offsets(counts, lead)
    lo, hi = off[0], off[-1]
    wd, dout = weights(g, len(counts), H, I), rows_of(g, counts, lead, tail, H)
    n, fl = dout.shape[0], flag()
    kept = rows_of(g, counts, lead, tail, 2 * I, 3.0)
    c, s = fp8_rows(g, counts, lead, tail, 2 * I)
    values = torch.zeros((n, 2 * I), dtype=torch.float64)
    values[lo:hi] = X.fp8_rows(c[lo:hi], s[lo:hi])
    for form, gu, kw in (("fp8", values, dict(gate_up_fp8=c, gate_up_scales=s)),
                         ("bf16", finite(kept, lo, hi), dict(gate_up=kept))):
        grad, bound, again, again_bound = X.down_grad(finite(dout, lo, hi), P.f64(wd), gu, off)
        outs = []
        for made in (True, False):  # act again, or not
            dgu, act = sentinel(n, 2 * I), sentinel(n, I) if made else None
            ep.ep_expert_down_grad(dout, wd, offset, grad_gate_up=dgu, act=act, error_flag=fl, **kw)
            check(dgu, grad, bound, lo, hi, f"grad_gate_up, {form}")
            if made:
                check(act, again, again_bound, lo, hi, f"act again, {form}")
            outs.append(dgu)
        same = torch.equal(bits(outs[0]), bits(outs[1]))
        assert same, form
    act = sentinel(n, I)
    ep.ep_expert_down_grad(dout, wd, offset, grad_gate_up=kept, gate_up=kept, act=act, error_flag=fl)
    same = torch.equal(bits(kept), bits(outs[0]))  # in place: the same bits as beside it
    assert same
    check(act, again, again_bound, lo, hi, "act again, in place")
    assert fl.item() == 0
