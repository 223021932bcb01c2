"""The experts' products as a program uses them: every tile that the sizes can take, long inner
sizes, capacities smaller than the routing, offsets that make no sense, more experts than fit
the kernels' tables, arrays past 4 GiB, streams, graphs, repeated calls; and ExpertPath's block
with its experts, forwards and backwards, in bf16 and e4m3."""
import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_experts as X
import plain_ops as P
from combine_ep_get_03_amd.pipeline import ExpertPath
from test_gpu_expert_ffn import (BF16, F32, I32, SENT, U8, check, check_codes, codes, finite, flag,
                                 fp8_rows, fp8_weights, gen, ids, offsets, rows_of, sentinel, weights)

pytestmark = pytest.mark.gpu

EIGHT = [300, 20, 0, 257, 129, 1, 64, 140]     # about 114 rows per expert
SIXTEEN = [70, 0, 33, 129, 5, 64, 40, 31, 32, 1, 0, 96, 65, 20, 17, 128]  # about 45
# wide enough outputs for more tiles than CUs, so that every tile height and several rounds of
# tiles per block are met; short inner sizes keep the 64-bit form quick
TALL = [(EIGHT, 3, 4, 72, 4872), (EIGHT, 0, 1, 64, 4864), (SIXTEEN, 1, 2, 40, 3400),
        (SIXTEEN, 0, 3, 128, 3456)]
WIDE = [(EIGHT, 3, 4, 9728, 72), (SIXTEEN, 1, 2, 6800, 40), ([150, 250], 0, 0, 20480, 24)]
LONG = [([40, 3, 0, 21], 2, 2, 7176, 128), ([33] * 3, 0, 0, 4096, 2056)]


def all_bf16(counts, lead, tail, H, I, seed, grads=True):
    """gate_up, down, down_grad, gate_up_grad and the weights' gradients of one set of shapes."""
    g = gen(seed)
    off, offset = offsets(counts, lead)
    E, lo, hi = len(counts), off[0], off[-1]
    x, w, wd = rows_of(g, counts, lead, tail, H), weights(g, E, 2 * I, H), weights(g, E, H, I)
    n = x.shape[0]
    fl = flag()
    act, gu = sentinel(n, I), sentinel(n, 2 * I)
    ep.ep_expert_gate_up(x, w, offset, act=act, gate_up=gu, error_flag=fl)
    wgu, err, wact, act_err = X.gate_up(finite(x, lo, hi), P.f64(w), off)
    check(act, wact, X.rounded(wact, act_err), lo, hi, "act")
    check(gu, wgu, X.rounded(wgu, err), lo, hi, "gate_up")
    if I % 128 == 0:
        c = torch.full((n, 2 * I), 0x5A, dtype=U8, device="cuda")
        s = torch.full((n, 2 * I // 128), -3.0, device="cuda")
        act8 = sentinel(n, I)
        ep.ep_expert_gate_up(x, w, offset, act=act8, gate_up_fp8=c, gate_up_scales=s, error_flag=fl)
        check(act8, wact, X.rounded(wact, act_err), lo, hi, "act beside codes")
        check_codes(c, s, wgu, err, lo, hi, "gate_up")
    out = sentinel(n, H)
    ep.ep_expert_down(act, wd, offset, expert_out=out, error_flag=fl)
    want, mag = X.nt(finite(act, lo, hi), P.f64(wd), off)
    check(out, want, X.rounded(want, X.product_error(I) * mag), lo, hi, "expert_out")
    if not grads:
        assert fl.item() == 0
        return
    dout = rows_of(g, counts, lead, tail, H)
    dgu, again = sentinel(n, 2 * I), sentinel(n, I)
    ep.ep_expert_down_grad(dout, wd, offset, grad_gate_up=dgu, gate_up=gu, act=again, error_flag=fl)
    grad, bound, wagain, again_bound = X.down_grad(finite(dout, lo, hi), P.f64(wd),
                                                   finite(gu, lo, hi), off)
    check(dgu, grad, bound, lo, hi, "grad_gate_up")
    check(again, wagain, again_bound, lo, hi, "act again")
    dx = sentinel(n, H)
    ep.ep_expert_gate_up_grad(dgu, w, offset, grad_x=dx, error_flag=fl)
    want, mag = X.nn(finite(dgu, lo, hi), P.f64(w), off)
    check(dx, want, X.rounded(want, X.product_error(2 * I) * mag), lo, hi, "grad_x")
    dw = torch.empty((E, H, I), device="cuda")
    ep.ep_expert_weight_grad(dout, act, offset, grad_weight=dw, error_flag=fl)
    want, err = X.weight_grad(finite(dout, lo, hi), finite(act, lo, hi), off)
    X.assert_within(dw, want, err, "grad_w_down")
    assert fl.item() == 0


@pytest.mark.parametrize("counts,lead,tail,H,I", TALL + WIDE, ids=ids(TALL + WIDE))
def test_every_tile(counts, lead, tail, H, I):
    print(f"\ncase: {counts} H={H} I={I}", flush=True)
    all_bf16(counts, lead, tail, H, I, 11 + H + I)


@pytest.mark.parametrize("counts,lead,tail,H,I", LONG, ids=ids(LONG))
def test_long_inner_sizes(counts, lead, tail, H, I):
    print(f"\ncase: {counts} H={H} I={I}", flush=True)
    all_bf16(counts, lead, tail, H, I, 12 + H + I, grads=H < 7000)


FP8 = [(EIGHT, 3, 4, 128, 4864), (SIXTEEN, 0, 3, 256, 2304), ([150, 250], 0, 0, 128, 20480),
       ([9, 40, 0, 2], 0, 1, 7168, 256), ([3] * 40, 1, 0, 256, 2048)]


@pytest.mark.parametrize("counts,lead,tail,H,I", FP8, ids=ids(FP8))
def test_every_tile_fp8(counts, lead, tail, H, I):
    print(f"\ncase: e4m3 {counts} H={H} I={I}", flush=True)
    g = gen(13 + H + I)
    off, offset = offsets(counts, lead)
    E, lo, hi = len(counts), off[0], off[-1]
    (x, xs), (w, ws) = fp8_rows(g, counts, lead, tail, H), fp8_weights(g, E, 2 * I, H)
    n, fl = x.shape[0], flag()
    xv = torch.zeros((n, H), dtype=torch.float64)
    xv[lo:hi] = X.fp8_rows(x[lo:hi], xs[lo:hi])
    _, _, act, err = X.gate_up(xv, X.fp8_weights(w, ws), off, fp8=True)
    c = torch.full((n, I), 0x5A, dtype=U8, device="cuda")
    s = torch.full((n, I // 128), -3.0, device="cuda")
    ep.ep_expert_gate_up_fp8(x, xs, w, ws, offset, act_fp8=c, act_scales=s, error_flag=fl)
    check_codes(c, s, act, err, lo, hi, "act")
    # the second product the other way round: outputs of I channels, so as many tiles
    (wd, wds), out = fp8_weights(g, E, I, H), sentinel(n, I)
    ep.ep_expert_down_fp8(x, xs, wd, wds, offset, expert_out=out, error_flag=fl)
    want, mag = X.nt(xv, X.fp8_weights(wd, wds), off)
    check(out, want, X.rounded(want, X.product_error(H, True) * mag), lo, hi, "expert_out")
    assert fl.item() == 0


@pytest.mark.parametrize("M,N", [(520, 264), (4104, 520)])
@pytest.mark.parametrize("counts", [[0, 700, 3, 0, 900], [40, 0, 5, 64, 65, 1] * 6, [0] * 7],
                         ids=["many", "few", "none"])
def test_weight_gradients_of_many_and_few_rows(counts, M, N):
    print(f"\ncase: weight gradient {M}x{N} {counts[:6]}", flush=True)
    g = gen(14 + M)
    off, offset = offsets(counts, 2)
    E, lo, hi = len(counts), off[0], off[-1]
    grad, inp = rows_of(g, counts, 2, 3, M), rows_of(g, counts, 2, 3, N)
    want, err = X.weight_grad(finite(grad, lo, hi), finite(inp, lo, hi), off)
    for dtype in (F32, BF16):
        for accumulate in (False, True):
            out = torch.randn((E, M, N), generator=g, device="cuda").to(dtype)
            full = want + P.f64(out) if accumulate else want
            ep.ep_expert_weight_grad(grad, inp, offset, grad_weight=out, accumulate=accumulate)
            bound = X.rounded(full, err) if dtype is BF16 else err + 2 * P.U * full.abs()
            X.assert_within(out, full, bound, f"{dtype} accumulate={accumulate}")


def small(seed=0, counts=(5, 0, 40, 3), H=256, I=128, tail=4):
    g = gen(seed)
    counts = list(counts)
    off, offset = offsets(counts, 0)
    E = len(counts)
    return dict(off=off, offset=offset, x=rows_of(g, counts, 0, tail, H), w=weights(g, E, 2 * I, H),
                wd=weights(g, E, H, I), dout=rows_of(g, counts, 0, tail, H), H=H, I=I, E=E,
                n=off[-1] + tail)


def run_all(d, offset, fl, n=None):
    """All bf16 calls on the first n rows; every output, prefilled."""
    n = d["n"] if n is None else n
    x, dout, H, I, E = d["x"][:n], d["dout"][:n], d["H"], d["I"], d["E"]
    o = dict(act=sentinel(n, I), gu=sentinel(n, 2 * I), out=sentinel(n, H), dgu=sentinel(n, 2 * I),
             dx=sentinel(n, H), dw=torch.full((E, 2 * I, H), 7.0, device="cuda"))
    ep.ep_expert_gate_up(x, d["w"], offset, act=o["act"], gate_up=o["gu"], error_flag=fl)
    ep.ep_expert_down(o["act"], d["wd"], offset, expert_out=o["out"], error_flag=fl)
    ep.ep_expert_down_grad(dout, d["wd"], offset, grad_gate_up=o["dgu"], gate_up=o["gu"],
                           error_flag=fl)
    ep.ep_expert_gate_up_grad(o["dgu"], d["w"], offset, grad_x=o["dx"], error_flag=fl)
    ep.ep_expert_weight_grad(o["dgu"], x, offset, grad_weight=o["dw"], error_flag=fl)
    return o


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_rows_past_the_capacity_are_skipped():
    d = small()
    for cut in (46, 45, 44, 20, 5, 3, 1):
        print(f"\ncase: {cut} rows of {d['off'][-1]}", flush=True)
        fl, ref_fl = flag(), flag()
        got = run_all(d, d["offset"], fl, cut)
        clamped = d["offset"].clamp(max=cut)
        want = run_all(d, clamped, ref_fl, cut)
        assert fl.item() == ep.EP_DEVERR_SLOT_RANGE and ref_fl.item() == 0
        for name in got:
            assert same(got[name], want[name]), name


@pytest.mark.parametrize("bad", [[-1, 5, 5, 45, 48], [0, 5, 4, 45, 48], [0, 5, 5, 45, 44],
                                 [-5, -4, -3, -2, -1], [48, 45, 45, 5, 0]])
def test_offsets_that_make_no_sense_compute_nothing(bad):
    d, fl = small(), flag()
    o = run_all(d, torch.tensor(bad, dtype=I32, device="cuda"), fl)
    assert fl.item() == ep.EP_DEVERR_SLOT_RANGE
    assert bool((o["dw"] == 7.0).all())
    for name in ("act", "gu", "out", "dgu", "dx"):
        assert bool((o[name].view(torch.int16) == SENT).all()), name
    run_all(d, torch.tensor(bad, dtype=I32, device="cuda"), None)  # a flag may be missing


def test_more_experts_than_the_table_holds():
    """2000 experts, most without rows: bf16, e4m3 and weights' gradients."""
    g = gen(21)
    counts = [0] * 2000
    for e, c in ((0, 3), (1, 1), (777, 40), (1024, 2), (1025, 33), (1999, 5)):
        counts[e] = c
    all_bf16(counts, 1, 1, 64, 64, 22)
    off, offset = offsets(counts, 0)
    (x, xs), (w, ws) = fp8_rows(g, counts, 0, 2, 128), fp8_weights(g, 2000, 128, 128)
    out, n = sentinel(off[-1] + 2, 128), off[-1]
    ep.ep_expert_down_fp8(x, xs, w, ws, offset, expert_out=out)
    xv = torch.zeros((n + 2, 128), dtype=torch.float64)
    xv[:n] = X.fp8_rows(x[:n], xs[:n])
    want, mag = X.nt(xv, X.fp8_weights(w, ws), off)
    check(out, want, X.rounded(want, X.product_error(128, True) * mag), 0, n, "expert_out")


def test_rows_and_weights_past_4_gib():
    """The last expert's rows lie past 4 GiB of every rows' array, and its weights too."""
    print("\ncase: past 4 GiB", flush=True)
    H, I, E, lead, mine = 4096, 512, 600, 600_000, 70
    n = lead + mine
    g = gen(23)
    off = torch.zeros(E + 1, dtype=I32, device="cuda")
    off[:] = lead
    off[E] = n
    x = torch.empty((n, H), dtype=BF16, device="cuda")
    w = torch.empty((E, 2 * I, H), dtype=BF16, device="cuda")
    wd = torch.empty((E, H, I), dtype=BF16, device="cuda")
    assert w.numel() * 2 > 2**32 and x.numel() * 2 > 2**32
    x[lead:] = torch.randn((mine, H), generator=g, device="cuda").to(BF16)
    w[-1], wd[-1] = weights(g, 1, 2 * I, H)[0], weights(g, 1, H, I)[0]
    act, gu = torch.empty((n, I), dtype=BF16, device="cuda"), torch.empty((n, 2 * I), dtype=BF16, device="cuda")
    out, fl = torch.empty((n, H), dtype=BF16, device="cuda"), flag()
    ep.ep_expert_gate_up(x, w, off, act=act, gate_up=gu, error_flag=fl)
    ep.ep_expert_down(act, wd, off, expert_out=out, error_flag=fl)
    one = [0, mine]
    xv, wv, wdv = P.f64(x[lead:]), P.f64(w[-1:]), P.f64(wd[-1:])
    _, _, wact, err = X.gate_up(xv, wv, one)
    X.assert_within(act[lead:], wact, X.rounded(wact, err), "act")
    want, mag = X.nt(P.f64(act[lead:]), wdv, one)
    X.assert_within(out[lead:], want, X.rounded(want, X.product_error(I) * mag), "expert_out")
    dgu = torch.empty((n, 2 * I), dtype=BF16, device="cuda")
    ep.ep_expert_down_grad(x, wd, off, grad_gate_up=dgu, gate_up=gu, error_flag=fl)
    grad, bound, _, _ = X.down_grad(xv, wdv, P.f64(gu[lead:]), one)
    X.assert_within(dgu[lead:], grad, bound, "grad_gate_up")
    ep.ep_expert_gate_up_grad(dgu, w, off, grad_x=out, error_flag=fl)
    want, mag = X.nn(P.f64(dgu[lead:]), wv, one)
    X.assert_within(out[lead:], want, X.rounded(want, X.product_error(2 * I) * mag), "grad_x")
    del out
    dw = w  # a weight's gradient past 4 GiB, in the place of weights no longer needed
    ep.ep_expert_weight_grad(dgu, x, off, grad_weight=dw, error_flag=fl)
    want, err = X.weight_grad(P.f64(dgu[lead:]), xv, one)
    X.assert_within(dw[-1:], want, X.rounded(want, err), "grad_w_gate_up")
    assert not bool(dw[:-1].any())
    assert fl.item() == 0


def test_a_row_that_is_not_finite_stays_alone():
    """NaN and infinities in one row reach that row's outputs and, of the weights' gradients,
    the expert's own, and no other; a group with an infinity has scale infinity, codes NaN for
    its infinities and 0 for the rest."""
    d, fl = small(31), flag()
    clean = run_all(d, d["offset"], fl)
    x = d["x"].clone()
    x[2, 7], x[30, 3] = float("nan"), float("inf")
    hit = run_all({**d, "x": x}, d["offset"], fl)
    rows = [r for r in range(d["n"]) if r not in (2, 30)]
    for name in ("act", "gu", "out", "dgu", "dx"):
        assert same(clean[name][rows], hit[name][rows]), name
    assert bool(torch.isnan(hit["act"][2]).all()) and bool(torch.isnan(hit["out"][2]).all())
    assert not bool(torch.isfinite(hit["gu"][30]).any())
    assert bool((hit["dw"][1] == 0).all()) and same(clean["dw"][3], hit["dw"][3])
    # the e4m3 form kept: row 5 has one infinite gate (its weights' row is infinite there)
    H, I, n = d["H"], d["I"], d["n"]
    w = d["w"].clone()
    w[2, 9] = 0
    w[2, 9, 0] = float("inf")
    x = d["x"].clone()
    x[5:45, 0] = x[5:45, 0].abs() + 0.5
    c, s = torch.zeros((n, 2 * I), dtype=U8, device="cuda"), torch.zeros((n, 2 * I // 128), device="cuda")
    ep.ep_expert_gate_up(x, w, d["offset"], act=sentinel(n, I), gate_up_fp8=c, gate_up_scales=s)
    assert bool(torch.isinf(s[5:45, 0]).all()) and bool(torch.isfinite(s[5:45, 1]).all())
    assert bool(((c[5:45, 9] & 0x7F) == 0x7F).all())
    assert bool(((c[5:45, [k for k in range(128) if k != 9]] & 0x7F) == 0).all())
    assert fl.item() == 0


def test_zero_rows_and_zero_groups():
    d = small(32)
    x = torch.zeros_like(d["x"])
    n, I = d["n"], d["I"]
    c, s = torch.full((n, 2 * I), 9, dtype=U8, device="cuda"), torch.zeros((n, 2 * I // 128), device="cuda")
    act = sentinel(n, I)
    ep.ep_expert_gate_up(x, d["w"], d["offset"], act=act, gate_up_fp8=c, gate_up_scales=s)
    hi = d["off"][-1]
    assert bool((act[:hi] == 0).all()) and bool(((c[:hi] & 0x7F) == 0).all()) and bool((s[:hi] == 1).all())
    for E in (1, 4):  # no rows at all
        off = torch.zeros(E + 1, dtype=I32, device="cuda")
        ep.ep_expert_gate_up(d["x"][:0], d["w"][:E], off, act=act[:0])
        ep.ep_expert_down(act[:0], d["wd"][:E], off, expert_out=d["x"][:0])
        dw = torch.ones((E, 256, 128), device="cuda")
        ep.ep_expert_weight_grad(d["x"][:0], act[:0], off, grad_weight=dw)
        assert not bool(dw.any())


def test_the_same_call_gives_the_same_bits_on_any_stream():
    """Repeated, on other streams and two at once: the same bits."""
    d, other = small(33, counts=(300, 0, 129, 64), H=520, I=1032), small(34)
    first, second = run_all(d, d["offset"], None), run_all(other, other["offset"], None)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(a):
            again = run_all(d, d["offset"], None)
        with torch.cuda.stream(b):
            beside = run_all(other, other["offset"], None)
        torch.cuda.synchronize()
        for name in first:
            assert same(first[name], again[name]), name
            assert same(second[name], beside[name]), name
    out = sentinel(*first["act"].shape)
    ep.ep_expert_gate_up(d["x"], d["w"], d["offset"], act=out, stream=a)
    a.synchronize()
    assert same(out, first["act"])


def test_replays_follow_the_offsets():
    """One captured call serves every routing of its capacity: the counts are read on the GPU."""
    counts = [[64, 0, 10, 22], [0, 96, 0, 0], [1, 2, 3, 4], [0, 0, 0, 0], [24, 24, 24, 24]]
    d = small(35, counts=counts[0], tail=0)
    d["x"] = torch.randn((96, d["H"]), generator=gen(36), device="cuda").to(BF16)
    d["dout"] = torch.randn((96, d["H"]), generator=gen(37), device="cuda").to(BF16)
    offset, fl = d["offset"].clone(), flag()
    run_all(d, offset, fl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = run_all(d, offset, fl)
    for rep, c in enumerate(counts + counts[:1]):
        off, _ = offsets(c, 0)
        offset.copy_(torch.tensor(off, dtype=I32))
        want = run_all(d, offset, fl)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in o:
            assert same(o[name], want[name]), (rep, name)
        assert fl.item() == 0


# ------------------------------------------------------------------------ ExpertPath

def block_inputs(seed, T, H, E, k, I):
    g = gen(seed)

    def r(*s, scale=1.0):
        return (torch.randn(s, generator=g, device="cuda") * scale).to(BF16)

    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices
    idx = torch.where(torch.rand((T, k), generator=g, device="cuda") < 0.1, -1, idx)
    return dict(x=r(T, H), residual=r(T, H), weight=r(H) * 0.1 + 1, idx=idx,
                gate=torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1),
                shared=r(T, H), grad_out=r(T, H), grad_res=r(T, H), w=weights(g, E, 2 * I, H),
                wd=weights(g, E, H, I))


def train(p, d, gg, gd, accumulate=False):
    p.norm(d["x"], d["weight"], d["residual"])
    p.dispatch(d["idx"])
    p.experts(d["w"], d["wd"])
    p.combine(p.expert_out, d["gate"], addend=d["shared"])
    p.combine_grad(d["grad_out"], p.expert_out, d["gate"])
    p.experts_grad(d["w"], d["wd"], grad_w_gate_up=gg, grad_w_down=gd, accumulate=accumulate)
    p.dispatch_grad(p.grad_perm_x)
    p.norm_grad(d["weight"], d["grad_res"])


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,E,k,I", [(1, 1024, 16, 4, 128), (257, 512, 16, 4, 256),
                                       (700, 256, 4, 2, 384)])
def test_block_with_its_experts(T, H, E, k, I, checkpoint):
    """Each step of the block against the 64-bit form of what the step before it left."""
    print(f"\ncase: block T={T} H={H} E={E} k={k} I={I} {checkpoint}", flush=True)
    d = block_inputs(T + H, T, H, E, k, I)
    p = ExpertPath(T, H, E, k, training=True, inter=I, checkpoint=checkpoint)
    gg = torch.zeros((E, 2 * I, H), device="cuda")
    gd = torch.zeros((E, H, I), dtype=BF16, device="cuda")
    train(p, d, gg, gd)
    assert int(p.error_flag) == 0
    off = p.expert_offset.cpu().tolist()
    M = off[-1]
    w, wd = P.f64(d["w"]), P.f64(d["wd"])
    px = finite(p.perm_x, 0, M)
    gu, err, act, act_err = X.gate_up(px, w, off)
    if checkpoint == "bf16":
        kept = finite(p.gate_up, 0, M)
        X.assert_within(p.gate_up[:M], gu[:M], X.rounded(gu, err)[:M], "gate_up")
        X.assert_within(p.act[:M], act[:M], X.rounded(act, act_err)[:M], "act")
    else:
        kept = torch.zeros((T * k, 2 * I), dtype=torch.float64)
        kept[:M] = X.fp8_rows(p.gate_up_fp8[:M], p.gate_up_scales[:M])
        X.assert_within(kept[:M], gu[:M], X.codes_bound(gu[:M], err[:M], P.fp8_scales(gu[:M])), "kept")
    dout = finite(p.grad_expert_out, 0, M)
    grad, bound, again, again_bound = X.down_grad(dout, wd, kept, off)
    X.assert_within(p.grad_gate_up[:M], grad[:M], bound[:M], "grad_gate_up")
    if checkpoint == "fp8":
        X.assert_within(p.act[:M], again[:M], again_bound[:M], "act again")
    # expert_out came of the forward's act, whose bound reaches it through |Wd|
    want, mag = X.nt(act, wd, off)
    _, reach = X.nt(X.rounded(act, act_err), wd, off)
    X.assert_within(p.expert_out[:M], want[:M],
                    X.rounded(want, reach + 2 * X.product_error(I) * mag)[:M], "expert_out")
    want, err = X.weight_grad(dout, finite(p.act, 0, M), off)
    X.assert_within(gd, want, X.rounded(want, err), "grad_w_down")
    dgu = finite(p.grad_gate_up, 0, M)
    want, err = X.weight_grad(dgu, px, off)
    X.assert_within(gg, want, err, "grad_w_gate_up")
    want, mag = X.nn(dgu, w, off)
    X.assert_within(p.grad_perm_x[:M], want[:M], X.rounded(want, X.product_error(2 * I) * mag)[:M],
                    "grad_perm_x")
    # a second micro-batch added to the first
    before = gg.clone()
    train(p, d, gg, gd, accumulate=True)
    X.assert_within(gg, 2 * P.f64(before), 4 * P.U * P.f64(before).abs(), "accumulated")


@pytest.mark.parametrize("T,H,E,k,I", [(1, 1024, 16, 4, 128), (129, 512, 16, 4, 256)])
def test_serving_block_in_e4m3(T, H, E, k, I):
    print(f"\ncase: e4m3 block T={T} H={H} E={E} I={I}", flush=True)
    d, g = block_inputs(T + I, T, H, E, k, I), gen(41)
    (w, ws), (wd, wds) = fp8_weights(g, E, 2 * I, H), fp8_weights(g, E, H, I)
    p = ExpertPath(T, H, E, k, fp8=True, inter=I)
    p.norm(d["x"], d["weight"], d["residual"])
    p.dispatch(d["idx"])
    p.experts((w, ws), (wd, wds))
    p.combine(p.expert_out, d["gate"])
    assert int(p.error_flag) == 0
    off = p.expert_offset.cpu().tolist()
    M = off[-1]
    px = torch.zeros((T * k, H), dtype=torch.float64)
    px[:M] = X.fp8_rows(p.perm_x_fp8[:M], p.perm_scales[:M])
    _, _, act, err = X.gate_up(px, X.fp8_weights(w, ws), off, fp8=True)
    want = P.fp8_scales(act[:M])
    X.assert_within(p.act_scales[:M], want, X.scale_bound(act[:M], err[:M], want), "act scales")
    av = torch.zeros((T * k, I), dtype=torch.float64)
    av[:M] = X.fp8_rows(p.act_fp8[:M], p.act_scales[:M])
    X.assert_within(av[:M], act[:M], X.codes_bound(act[:M], err[:M], want), "act codes")
    want, mag = X.nt(av, X.fp8_weights(wd, wds), off)
    X.assert_within(p.expert_out[:M], want[:M], X.rounded(want, X.product_error(I, True) * mag)[:M],
                    "expert_out")


def test_training_step_with_experts_in_a_graph():
    """The step captured and replayed on new batches (new routings), the same step run eagerly on
    a second path between the replays; both give the same bits."""
    T, H, E, k, I = 200, 512, 16, 4, 256
    d = block_inputs(51, T, H, E, k, I)
    a, b = (ExpertPath(T, H, E, k, training=True, inter=I, checkpoint="fp8") for _ in range(2))
    grads = [(torch.zeros((E, 2 * I, H), device="cuda"), torch.zeros((E, H, I), device="cuda"))
             for _ in range(2)]
    names = ["out", "grad_topk_weights", "grad_y", "grad_x", "grad_weight"]
    train(a, d, *grads[0])
    train(b, d, *grads[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train(a, d, *grads[0])
    for rep in range(3):
        new = block_inputs(60 + rep, T, H, E, k, I)
        for n in d:
            d[n].copy_(new[n])
        graph.replay()
        train(b, d, *grads[1])
        torch.cuda.synchronize()
        for n in names:
            assert same(getattr(a, n), getattr(b, n)), (rep, n)
        for u, v in zip(*grads):
            assert same(u, v), rep
        assert int(a.error_flag) == 0 and int(b.error_flag) == 0


def test_an_empty_batch_through_the_experts():
    p = ExpertPath(0, 256, 4, 2, training=True, inter=128)
    d = block_inputs(71, 1, 256, 4, 2, 128)
    d = {n: t[:0] if n in ("x", "residual", "idx", "gate", "shared", "grad_out", "grad_res") else t
         for n, t in d.items()}
    gg, gd = torch.ones((4, 256, 256), device="cuda"), torch.ones((4, 256, 128), device="cuda")
    train(p, d, gg, gd)
    assert not bool(gg.any()) and not bool(gd.any()) and int(p.error_flag) == 0


def test_as_many_rows_as_32_bits_number():
    """One expert of INT32_MAX rows of eight channels (34 GB): the first and the last ones."""
    n, H, I, some = 2**31 - 1, 8, 8, 1000
    print(f"\ncase: {n} rows of {H}", flush=True)
    g = gen(29)
    off = torch.tensor([0, n], dtype=I32, device="cuda")
    x = torch.zeros((n, H), dtype=BF16, device="cuda")
    for r in (slice(0, some), slice(n - some, n)):
        x[r] = torch.randn((some, H), generator=g, device="cuda").to(BF16)
    w, wd = weights(g, 1, 2 * I, H), weights(g, 1, H, I)
    act, fl = torch.empty((n, I), dtype=BF16, device="cuda"), flag()
    ep.ep_expert_gate_up(x, w, off, act=act, error_flag=fl)
    for r in (slice(0, some), slice(n - some, n)):
        _, _, wact, err = X.gate_up(P.f64(x[r]), P.f64(w), [0, some])
        X.assert_within(act[r], wact, X.rounded(wact, err), "act")
    ep.ep_expert_down(act, wd, off, expert_out=x, error_flag=fl)
    for r in (slice(0, some), slice(n - some, n)):
        want, mag = X.nt(P.f64(act[r]), P.f64(wd), [0, some])
        X.assert_within(x[r], want, X.rounded(want, X.product_error(I) * mag), "expert_out")
    assert fl.item() == 0
