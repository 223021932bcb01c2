"""The operators over expert-major rows on the GPU against their 64-bit plain forms:
ep_dispatch_permute_fp8, ep_combine_unpermute, ep_combine_unpermute_grad and
ep_dispatch_permute_grad. Widths and top-k from the smallest on, dropped pairs and tokens
with none, rows that no pair names, rows out of range, outputs in the place of inputs,
buffers past 4 GiB, graphs and streams."""
import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_ops as P

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
SENT = 0x7FC3  # a bf16 NaN pattern


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def sentinel(*shape):
    return torch.full(shape, SENT, dtype=torch.int16, device="cuda").view(BF16)


def flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def slots(g, T, k, cap, dropped=0.2, empty_tokens=True):
    """Distinct rows below cap in a random order, some pairs dropped, every seventh token
    without any."""
    s = torch.randperm(cap, generator=g, device="cuda")[:T * k].to(torch.int32).reshape(T, k)
    s = torch.where(torch.rand((T, k), generator=g, device="cuda") < dropped, -1, s)
    if empty_tokens:
        s[::7] = -1
    return s.contiguous()


def case(seed, T, H, k, extra=5, dropped=0.2, empty_tokens=True):
    """Inputs of the bf16 calls; rows that no pair names hold NaN."""
    g = gen(seed)
    cap = T * k + extra
    slot = slots(g, T, k, cap, dropped, empty_tokens)
    rows = sentinel(cap, H)
    used = slot[slot >= 0].long()
    rows[used] = rand(g, used.numel(), H)
    w = torch.rand((T, k), generator=g, device="cuda")
    w[slot < 0] = float("nan")  # the weight of a pair that is not routed is not used
    return g, cap, slot, rows, w


SHAPES = [(1, 8, 1), (1, 7168, 8), (2, 16, 3), (7, 128, 1), (13, 520, 2), (64, 1000, 5),
          (65, 1024, 4), (129, 2056, 6), (33, 4096, 16), (40, 7168, 8), (21, 8192, 9),
          (6, 8200, 7), (5, 16384, 8), (3, 40960, 4), (9, 64, 17), (4, 256, 40), (3, 8, 300),
          (1000, 64, 8), (301, 512, 8)]


def wsafe(w, slot):
    return torch.where(slot >= 0, P.f64(w), torch.zeros((), dtype=torch.float64))


@pytest.mark.parametrize("T,H,k", SHAPES)
def test_unpermute(T, H, k):
    print(f"\ncase: unpermute T={T} H={H} k={k}", flush=True)
    g, cap, slot, rows, w = case(T + H + k, T, H, k)
    s, r, wd = slot.cpu(), P.f64(rows), wsafe(w, slot.cpu())
    for weights in (w, None):
        for addend in (None, rand(g, T, H)):
            out, err = sentinel(T, H), flag()
            ep.ep_combine_unpermute(rows, weights, slot, out=out, addend=addend, error_flag=err)
            a = (r, None if weights is None else wd, s, None if addend is None else P.f64(addend))
            want = P.unpermute(*a)
            r0 = torch.where(torch.isnan(r), torch.zeros((), dtype=torch.float64), r)
            P.assert_within(out, want, P.unpermute_bound(want, r0, *a[1:]), "out")
            assert int(err) == 0
            if addend is None:
                none = (s < 0).all(dim=1)
                assert torch.all(out.cpu()[none].view(torch.int16) == 0)  # +0.0


@pytest.mark.parametrize("T,H,k", SHAPES)
def test_unpermute_grad(T, H, k):
    print(f"\ncase: unpermute_grad T={T} H={H} k={k}", flush=True)
    g, cap, slot, rows, w = case(T * 3 + H + k, T, H, k)
    s, r, wd = slot.cpu(), P.f64(rows), wsafe(w, slot.cpu())
    go = rand(g, T, H)
    hit = s >= 0
    for weights in (w, None):
        want, want_w = P.unpermute_grad(P.f64(go), r, None if weights is None else wd, s)
        for form in ("both", "rows only", "in place"):
            y = rows.clone()
            gr = y if form == "in place" else sentinel(cap, H)
            gw = None if form == "rows only" else torch.full((T, k), -9.0, device="cuda")
            err = flag()
            ep.ep_combine_unpermute_grad(go, None if form == "rows only" else y, weights, slot,
                                         grad_expert_out=gr, grad_topk_weights=gw, error_flag=err)
            got = gr.cpu()
            P.assert_within(got[s[hit].long()], want[hit],
                            (P.BF16 + 4 * P.U) * want[hit].abs() + P.TINY_BF16, "grad_expert_out")
            left = torch.ones(cap, dtype=torch.bool)
            left[s[hit].long()] = False  # rows of no pair keep what they held
            assert torch.all(got[left].view(torch.int16) == SENT)
            if gw is not None:
                r0 = torch.where(torch.isnan(r), torch.zeros((), dtype=torch.float64), r)
                P.assert_within(gw, want_w, P.dot_bound(P.f64(go), r0, s), "grad_topk_weights")
                assert torch.all(gw.cpu()[~hit].view(torch.int32) == 0)
            assert int(err) == 0


@pytest.mark.parametrize("T,H,k", SHAPES)
def test_permute_grad(T, H, k):
    print(f"\ncase: permute_grad T={T} H={H} k={k}", flush=True)
    g, cap, slot, rows, _ = case(T * 5 + H + k, T, H, k)
    s, r = slot.cpu(), P.f64(rows)
    gp = torch.randn(cap, generator=g, device="cuda")
    for with_w in (True, False):
        gx, err = sentinel(T, H), flag()
        gw = torch.full((T, k), -9.0, device="cuda") if with_w else None
        ep.ep_dispatch_permute_grad(rows, slot, grad_x=gx, grad_perm_weights=gp if with_w else None,
                                    grad_topk_weights=gw, error_flag=err)
        want = P.unpermute(r, None, s, None)
        r0 = torch.where(torch.isnan(r), torch.zeros((), dtype=torch.float64), r)
        P.assert_within(gx, want, P.unpermute_bound(want, r0, None, s, None), "grad_x")
        if with_w:
            ref = torch.where(s >= 0, gp.cpu()[s.clamp(min=0).long()], torch.zeros(()))
            assert torch.equal(gw.cpu().view(torch.int32), ref.view(torch.int32))
        assert int(err) == 0


FP8_SHAPES = [(1, 128, 1), (1, 7168, 8), (2, 256, 3), (7, 384, 2), (64, 1024, 4), (129, 2048, 6),
              (33, 4096, 16), (40, 7168, 8), (21, 8192, 9), (6, 8320, 7), (5, 16384, 8),
              (3, 40960, 4), (9, 128, 17), (4, 256, 300), (1000, 128, 8)]


@pytest.mark.parametrize("T,H,k", FP8_SHAPES)
def test_permute_fp8(T, H, k):
    print(f"\ncase: permute_fp8 T={T} H={H} k={k}", flush=True)
    g = gen(T + H * 3 + k)
    cap = T * k + 5
    slot = slots(g, T, k, cap)
    x = torch.randint(0, 256, (T, H), generator=g, device="cuda").to(torch.uint8)
    sc = torch.randint(-2**31, 2**31 - 1, (T, H // 128), generator=g, device="cuda").to(
        torch.int32).view(torch.float32)  # any bits travel unchanged
    w = torch.rand((T, k), generator=g, device="cuda")
    s = slot.cpu()
    t, j = torch.nonzero(s >= 0, as_tuple=True)
    q = s[t, j].long()
    for extras in (True, False):
        px = torch.full((cap, H), 0x5A, dtype=torch.uint8, device="cuda")
        ps = torch.full((cap, H // 128), 0x5A5A5A5A, dtype=torch.int32, device="cuda").view(torch.float32)
        pw = torch.full((cap,), -5.0, device="cuda") if extras else None
        pi = torch.full((cap,), -5, dtype=torch.int32, device="cuda") if extras else None
        err = flag()
        ep.ep_dispatch_permute_fp8(x.view(torch.float8_e4m3fn) if extras else x, sc,
                                   w if extras else None, slot,
                                   perm_x_fp8=px.view(torch.float8_e4m3fn) if extras else px,
                                   perm_scales=ps, perm_weights=pw, perm_src_idx=pi, error_flag=err)
        rx = torch.full((cap, H), 0x5A, dtype=torch.uint8)
        rs = torch.full((cap, H // 128), 0x5A5A5A5A, dtype=torch.int32)
        rx[q], rs[q] = x.cpu()[t], sc.cpu().view(torch.int32)[t]
        assert torch.equal(px.cpu(), rx) and torch.equal(ps.cpu().view(torch.int32), rs)
        if extras:
            rw, ri = torch.full((cap,), -5.0), torch.full((cap,), -5, dtype=torch.int32)
            rw[q], ri[q] = w.cpu()[t, j], t.to(torch.int32)
            assert torch.equal(pw.cpu(), rw) and torch.equal(pi.cpu(), ri)
        assert int(err) == 0


@pytest.mark.parametrize("T,H,k", [(601, 7168, 8), (8300, 1024, 4), (1200, 8200, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_unpermute_grad_in_two_launches(T, H, k, in_place):
    """More than 64 MB of rows: the dots and the rows are separate launches."""
    print(f"\ncase: unpermute_grad in two launches T={T} H={H} k={k}", flush=True)
    assert T * k * H * 2 > 64 << 20
    g, cap, slot, rows, w = case(T, T, H, k)
    go = rand(g, T, H)
    y = rows.clone()
    gr = y if in_place else sentinel(cap, H)
    gw, err = torch.full((T, k), -9.0, device="cuda"), flag()
    ep.ep_combine_unpermute_grad(go, y, w, slot, grad_expert_out=gr, grad_topk_weights=gw,
                                 error_flag=err)
    s, r, wd = slot.cpu(), P.f64(rows), wsafe(w, slot.cpu())
    hit = s >= 0
    want, want_w = P.unpermute_grad(P.f64(go), r, wd, s)
    got = gr.cpu()
    P.assert_within(got[s[hit].long()], want[hit], (P.BF16 + 4 * P.U) * want[hit].abs()
                    + P.TINY_BF16, "grad_expert_out")
    left = torch.ones(cap, dtype=torch.bool)
    left[s[hit].long()] = False
    assert torch.all(got[left].view(torch.int16) == SENT)
    r0 = torch.where(torch.isnan(r), torch.zeros((), dtype=torch.float64), r)
    P.assert_within(gw, want_w, P.dot_bound(P.f64(go), r0, s), "grad_topk_weights")
    assert torch.all(gw.cpu()[~hit].view(torch.int32) == 0) and int(err) == 0


@pytest.mark.parametrize("T,H,k", [(10_000, 7168, 8), (70_001, 512, 16)])
def test_permute_fp8_of_many_scales(T, H, k):
    """More than 16 MB of scales, which leave with another store."""
    print(f"\ncase: permute_fp8 T={T} H={H} k={k}", flush=True)
    assert T * k * (H // 128) * 4 > 16 << 20
    g = gen(T)
    slot = slots(g, T, k, T * k + 3)
    x = torch.randint(1, 256, (T, H), generator=g, device="cuda").to(torch.uint8)
    sc = torch.rand((T, H // 128), generator=g, device="cuda") + 1
    px = torch.zeros((T * k + 3, H), dtype=torch.uint8, device="cuda")
    ps = torch.zeros((T * k + 3, H // 128), device="cuda")
    pi = torch.full((T * k + 3,), -1, dtype=torch.int32, device="cuda")
    ep.ep_dispatch_permute_fp8(x, sc, None, slot, perm_x_fp8=px, perm_scales=ps, perm_src_idx=pi)
    t, j = torch.nonzero(slot >= 0, as_tuple=True)
    q = slot[t, j].long()
    assert torch.equal(px[q], x[t]) and torch.equal(ps[q], sc[t]) and torch.equal(pi[q].long(), t)
    left = torch.ones(T * k + 3, dtype=torch.bool, device="cuda")
    left[q] = False
    assert not px[left].any() and not ps[left].any() and torch.all(pi[left] == -1)


def test_calls_of_several_launches():
    """More than 2^24 waves: each call runs over several token ranges. Small integers and
    weights that are powers of two, so that every result is exact."""
    print("\ncase: several launches per call", flush=True)
    g = gen(31)

    def ints(*shape):
        return torch.randint(-8, 9, shape, generator=g, device="cuda").to(BF16)

    def pow2(*shape):
        return torch.randint(-1, 2, shape, generator=g, device="cuda").float().exp2()

    T, H = 17_000_001, 8  # one wave per token
    slot = torch.randperm(T, generator=g, device="cuda").to(torch.int32).reshape(T, 1)
    slot[5::11] = -1
    rows, w, hit = ints(T, H), pow2(T, 1), slot[:, 0] >= 0
    want = torch.where(hit[:, None], rows[slot[:, 0].clamp(min=0).long()].float() * w, 0.0).to(BF16)
    out = sentinel(T, H)
    ep.ep_combine_unpermute(rows, w, slot, out=out)
    assert torch.equal(out, want)
    del out, want, rows, slot, w, hit

    T, k, H = 2_100_001, 8, 8  # eight waves per token
    slot = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).reshape(T, k)
    slot[3::7, 2] = -1
    rows, go, w = ints(T * k, H), ints(T, H), pow2(T, k)
    gr, gw = torch.zeros((T * k, H), dtype=BF16, device="cuda"), torch.full((T, k), 99.0, device="cuda")
    ep.ep_combine_unpermute_grad(go, rows, w, slot, grad_expert_out=gr, grad_topk_weights=gw)
    for j in range(k):
        t = torch.nonzero(slot[:, j] >= 0).squeeze(1)
        q = slot[t, j].long()
        assert torch.equal(gr[q], (go[t].float() * w[t, j, None]).to(BF16))
        assert torch.equal(gw[t, j], (go[t].float() * rows[q].float()).sum(dim=1))
    assert torch.all(gw[slot < 0] == 0)
    del rows, go, gr, gw

    H = 128
    x = torch.randint(0, 256, (T, H), generator=g, device="cuda").to(torch.uint8)
    sc = torch.rand((T, 1), generator=g, device="cuda")
    px = torch.zeros((T * k, H), dtype=torch.uint8, device="cuda")
    ps = torch.zeros((T * k, 1), device="cuda")
    pi = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    ep.ep_dispatch_permute_fp8(x, sc, None, slot, perm_x_fp8=px, perm_scales=ps, perm_src_idx=pi)
    for j in range(k):
        t = torch.nonzero(slot[:, j] >= 0).squeeze(1)
        q = slot[t, j].long()
        assert torch.equal(px[q], x[t]) and torch.equal(ps[q], sc[t]) and torch.equal(pi[q].long(), t)


def test_rows_out_of_range_are_skipped_and_reported():
    T, H, k = 50, 256, 4
    print("\ncase: rows out of range", flush=True)
    g, cap, slot, rows, w = case(11, T, H, k, dropped=0.0, empty_tokens=False)
    slot[3, 1], slot[20, 0], slot[49, 3] = cap, cap + 1000, 2**31 - 1
    slot[5, 2] = -(2**31)
    kept = torch.where(slot >= cap, -1, slot)
    sk = kept.cpu()
    w = torch.rand((T, k), generator=g, device="cuda")
    r = P.f64(rows)
    r0 = torch.where(torch.isnan(r), torch.zeros((), dtype=torch.float64), r)
    out, err = sentinel(T, H), flag()
    ep.ep_combine_unpermute(rows, w, slot, out=out, error_flag=err)
    want = P.unpermute(r, P.f64(w), sk, None)
    P.assert_within(out, want, P.unpermute_bound(want, r0, P.f64(w), sk, None), "out")
    assert int(err) == ep.EP_DEVERR_SLOT_RANGE

    go, err = rand(g, T, H), flag()
    gr, gw = sentinel(cap, H), torch.full((T, k), -9.0, device="cuda")
    ep.ep_combine_unpermute_grad(go, rows, w, slot, grad_expert_out=gr, grad_topk_weights=gw,
                                 error_flag=err)
    want, want_w = P.unpermute_grad(P.f64(go), r, P.f64(w), sk)
    hit = sk >= 0
    P.assert_within(gr.cpu()[sk[hit].long()], want[hit], (P.BF16 + 4 * P.U) * want[hit].abs()
                    + P.TINY_BF16, "grad rows")
    P.assert_within(gw, want_w, P.dot_bound(P.f64(go), r0, sk), "grad weights")
    assert torch.all(gw.cpu()[~hit] == 0) and int(err) == ep.EP_DEVERR_SLOT_RANGE

    gx, gp, err = sentinel(T, H), torch.randn(cap, generator=g, device="cuda"), flag()
    gw.fill_(-9.0)
    ep.ep_dispatch_permute_grad(rows, slot, grad_x=gx, grad_perm_weights=gp, grad_topk_weights=gw,
                                error_flag=err)
    want = P.unpermute(r, None, sk, None)
    P.assert_within(gx, want, P.unpermute_bound(want, r0, None, sk, None), "grad_x")
    assert torch.all(gw.cpu()[~hit] == 0) and int(err) == ep.EP_DEVERR_SLOT_RANGE

    x = torch.randint(0, 256, (T, H), generator=g, device="cuda").to(torch.uint8)
    sc = torch.rand((T, H // 128), generator=g, device="cuda")
    px = torch.full((cap, H), 0x5A, dtype=torch.uint8, device="cuda")
    ps = torch.full((cap, H // 128), -1.0, device="cuda")
    err = flag()
    ep.ep_dispatch_permute_fp8(x, sc, None, slot, perm_x_fp8=px, perm_scales=ps, error_flag=err)
    t, j = torch.nonzero(hit, as_tuple=True)
    rx = torch.full((cap, H), 0x5A, dtype=torch.uint8)
    rx[sk[t, j].long()] = x.cpu()[t]
    assert torch.equal(px.cpu(), rx) and int(err) == ep.EP_DEVERR_RECV_OVERFLOW
    # without an error flag the same rows are skipped
    ep.ep_combine_unpermute(rows, w, slot, out=out)
    ep.ep_combine_unpermute_grad(go, rows, w, slot, grad_expert_out=gr, grad_topk_weights=gw)
    torch.cuda.synchronize()


def test_error_bits_are_added_to_the_flag():
    g, cap, slot, rows, w = case(12, 4, 64, 2)
    err = torch.full((1,), ep.EP_DEVERR_TOPK_RANGE, dtype=torch.int32, device="cuda")
    out = sentinel(4, 64)
    ep.ep_combine_unpermute(rows, w, slot, out=out, error_flag=err)
    assert int(err) == ep.EP_DEVERR_TOPK_RANGE
    slot[1, 0] = cap
    ep.ep_combine_unpermute(rows, w, slot, out=out, error_flag=err)
    assert int(err) == ep.EP_DEVERR_TOPK_RANGE | ep.EP_DEVERR_SLOT_RANGE


def test_refusals_of_the_binding():
    T, H, k = 4, 64, 2
    g, cap, slot, rows, w = case(33, T, H, k, dropped=0.0, empty_tokens=False)
    out = sentinel(T, H)
    for kw, exc in ((dict(error_flag=torch.zeros(1, device="cuda")), TypeError),
                    (dict(error_flag=torch.zeros(0, dtype=torch.int32, device="cuda")), ValueError),
                    (dict(error_flag=torch.zeros(1, dtype=torch.int32)), ValueError),
                    (dict(addend=out[:2]), ValueError), (dict(addend=out.float()), TypeError)):
        with pytest.raises(exc):
            ep.ep_combine_unpermute(rows, w, slot, out=out, **kw)
    for args in ((rows, w.t().contiguous().t(), slot), (rows, w, slot.long()), (rows, w.cpu(), slot),
                 (rows[:, ::2], w, slot), (rows.view(-1), w, slot), (None, w, slot), (rows, w, 3)):
        with pytest.raises((ValueError, TypeError)):
            ep.ep_combine_unpermute(*args, out=out)
    torch.cuda.synchronize()
    assert torch.all(out.view(torch.int16) == SENT)  # nothing ran
    ep.ep_combine_unpermute(rows, torch.nn.Parameter(w.clone()), slot, out=out,
                            error_flag=torch.zeros(3, dtype=torch.int32, device="cuda"))
    s, r = slot.cpu(), P.f64(rows)
    r0 = torch.where(torch.isnan(r), torch.zeros((), dtype=torch.float64), r)
    want = P.unpermute(r, P.f64(w), s, None)
    P.assert_within(out, want, P.unpermute_bound(want, r0, P.f64(w), s, None), "out")


def test_no_rows_and_no_tokens():
    T, H, k = 5, 128, 3
    slot = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    rows = torch.empty((0, H), dtype=BF16, device="cuda")
    add = rand(gen(1), T, H)
    out, w = sentinel(T, H), torch.ones((T, k), device="cuda")
    ep.ep_combine_unpermute(rows, w, slot, out=out, addend=add)
    assert torch.equal(out, add)
    gw = torch.full((T, k), 3.0, device="cuda")
    ep.ep_combine_unpermute_grad(add, rows, w, slot, grad_expert_out=rows, grad_topk_weights=gw)
    assert torch.all(gw == 0)
    gx = sentinel(T, H)
    ep.ep_dispatch_permute_grad(rows, slot, grad_x=gx)
    assert torch.all(gx.view(torch.int16) == 0)
    none = torch.empty((0, k), dtype=torch.int32, device="cuda")
    ep.ep_combine_unpermute(rand(gen(2), 4, H), None, none, out=rows)
    ep.ep_dispatch_permute_grad(rand(gen(2), 4, H), none, grad_x=rows)
    torch.cuda.synchronize()


def test_sums_take_a_row_that_several_pairs_name():
    T, H, k = 30, 256, 4
    g = gen(21)
    rows = rand(g, 10, H)
    slot = torch.randint(-1, 10, (T, k), generator=g, device="cuda").to(torch.int32)
    w = torch.rand((T, k), generator=g, device="cuda")
    out, gx = sentinel(T, H), sentinel(T, H)
    ep.ep_combine_unpermute(rows, w, slot, out=out)
    ep.ep_dispatch_permute_grad(rows, slot, grad_x=gx)
    s, r = slot.cpu(), P.f64(rows)
    want = P.unpermute(r, P.f64(w), s, None)
    P.assert_within(out, want, P.unpermute_bound(want, r, P.f64(w), s, None), "out")
    want = P.unpermute(r, None, s, None)
    P.assert_within(gx, want, P.unpermute_bound(want, r, None, s, None), "grad_x")


def test_the_same_bits_twice():
    T, H, k = 700, 7168, 8
    print("\ncase: the same bits twice", flush=True)
    g, cap, slot, rows, w = case(22, T, H, k)
    go = rand(g, T, H)
    got = []
    for _ in range(2):
        out, gr, gw = sentinel(T, H), sentinel(cap, H), torch.zeros((T, k), device="cuda")
        ep.ep_combine_unpermute(rows, w, slot, out=out)
        ep.ep_combine_unpermute_grad(go, rows, w, slot, grad_expert_out=gr, grad_topk_weights=gw)
        got.append((out.view(torch.int16), gr.view(torch.int16), gw.view(torch.int32)))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_unpermute_out_in_the_addends_place():
    for T, H, k in [(64, 7168, 8), (33, 520, 3)]:
        g, cap, slot, rows, w = case(14, T, H, k)
        add = rand(g, T, H)
        apart, here = sentinel(T, H), add.clone()
        ep.ep_combine_unpermute(rows, w, slot, out=apart, addend=add)
        ep.ep_combine_unpermute(rows, w, slot, out=here, addend=here)
        assert torch.equal(apart.view(torch.int16), here.view(torch.int16))


def test_infinite_rows_reach_their_own_token_alone():
    T, H, k = 20, 512, 4
    g, cap, slot, rows, w = case(15, T, H, k, dropped=0.0, empty_tokens=False)
    rows[slot[3, 1].long(), 100] = float("inf")
    rows[slot[4, 0].long(), 7] = float("nan")
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    out = sentinel(T, H)
    ep.ep_combine_unpermute(rows, w, slot, out=out)
    bad = ~torch.isfinite(out)
    assert int(bad.sum()) == 2 and bool(torch.isinf(out[3, 100])) and bool(torch.isnan(out[4, 7]))
    gw = torch.zeros((T, k), device="cuda")
    go = rand(g, T, H)
    ep.ep_combine_unpermute_grad(go, rows, w, slot, grad_expert_out=sentinel(cap, H),
                                 grad_topk_weights=gw)
    bad = ~torch.isfinite(gw)
    assert int(bad.sum()) == 2 and bool(bad[3, 1]) and bool(bad[4, 0])


def test_rows_past_4_gib():
    """330000 rows of 7168 bf16 channels (4.7 GB): every row of a few hundred tokens, the
    last ones of the buffer among them."""
    cap, H, k, T = 330_000, 7168, 8, 301
    print(f"\ncase: rows past 4 GiB cap={cap}", flush=True)
    g = gen(16)
    rows = torch.zeros((cap, H), dtype=BF16, device="cuda")
    slot = (cap - 1 - torch.randperm(cap, generator=g, device="cuda")[:T * k]).to(torch.int32)
    slot[:3] = torch.tensor([cap - 1, 0, 299_594])  # the last: its first byte is past 2^32
    slot = torch.unique(slot)[:T * k]
    slot = torch.cat([slot, torch.full((T * k - slot.numel(),), -1, dtype=torch.int32, device="cuda")])
    slot = slot[torch.randperm(T * k, generator=g, device="cuda")].reshape(T, k).contiguous()
    hit = slot >= 0
    vals = rand(g, int(hit.sum()), H)
    rows[slot[hit].long()] = vals
    w = torch.rand((T, k), generator=g, device="cuda")
    s = slot.cpu()
    small = torch.zeros(s.shape, dtype=torch.int64)
    small[s >= 0] = torch.arange(int((s >= 0).sum()))
    small[s < 0] = -1
    r = P.f64(vals)
    out = sentinel(T, H)
    ep.ep_combine_unpermute(rows, w, slot, out=out)
    want = P.unpermute(r, P.f64(w), small, None)
    P.assert_within(out, want, P.unpermute_bound(want, r, P.f64(w), small, None), "out")
    go, gw = rand(g, T, H), torch.zeros((T, k), device="cuda")
    ep.ep_combine_unpermute_grad(go, rows, w, slot, grad_expert_out=rows, grad_topk_weights=gw)
    want, want_w = P.unpermute_grad(P.f64(go), r, P.f64(w), small)
    P.assert_within(rows[slot[hit].long()], want[s >= 0],
                    (P.BF16 + 4 * P.U) * want[s >= 0].abs() + P.TINY_BF16, "grad rows")
    P.assert_within(gw, want_w, P.dot_bound(P.f64(go), r, small), "grad weights")
    rest = torch.ones(cap, dtype=torch.bool, device="cuda")
    rest[slot[hit].long()] = False
    for c in range(0, cap, 65536):  # the rows of no pair are still zero
        assert not rows[c:c + 65536][rest[c:c + 65536]].any()
    del rows
    px = torch.zeros((660_000, H), dtype=torch.uint8, device="cuda")
    ps = torch.zeros((660_000, H // 128), device="cuda")
    x = torch.randint(1, 256, (T, H), generator=g, device="cuda").to(torch.uint8)
    sc = torch.rand((T, H // 128), generator=g, device="cuda") + 1
    slot = torch.where(hit, slot + 330_000, -1).to(torch.int32).contiguous()
    ep.ep_dispatch_permute_fp8(x, sc, None, slot, perm_x_fp8=px, perm_scales=ps)
    t, j = torch.nonzero(hit, as_tuple=True)
    q = slot[t, j].long()
    assert torch.equal(px[q], x[t]) and torch.equal(ps[q], sc[t])
    assert int((ps[:, 0] != 0).sum()) == q.numel()


def test_calls_replay_in_a_graph():
    T, H, k = 200, 1024, 6
    print("\ncase: expert rows graph", flush=True)
    g, cap, slot, rows, w = case(17, T, H, k)
    w = torch.rand((T, k), generator=g, device="cuda")
    go, add, gp = rand(g, T, H), rand(g, T, H), torch.randn(cap, generator=g, device="cuda")
    x = torch.randint(0, 256, (T, H), generator=g, device="cuda").to(torch.uint8)
    sc = torch.rand((T, H // 128), generator=g, device="cuda")
    o = dict(out=sentinel(T, H), gr=sentinel(cap, H), gw=torch.zeros((T, k), device="cuda"),
             gx=sentinel(T, H), gw2=torch.zeros((T, k), device="cuda"),
             px=torch.zeros((cap, H), dtype=torch.uint8, device="cuda"),
             ps=torch.zeros((cap, H // 128), device="cuda"))
    err = flag()

    def calls():
        ep.ep_dispatch_permute_fp8(x, sc, None, slot, perm_x_fp8=o["px"], perm_scales=o["ps"],
                                   error_flag=err)
        ep.ep_combine_unpermute(rows, w, slot, out=o["out"], addend=add, error_flag=err)
        ep.ep_combine_unpermute_grad(go, rows, w, slot, grad_expert_out=o["gr"],
                                     grad_topk_weights=o["gw"], error_flag=err)
        ep.ep_dispatch_permute_grad(rows, slot, grad_x=o["gx"], grad_perm_weights=gp,
                                    grad_topk_weights=o["gw2"], error_flag=err)

    graph = torch.cuda.CUDAGraph()
    calls()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls()
    for rep in range(3):
        go.copy_(rand(gen(50 + rep), T, H))
        w.copy_(torch.rand((T, k), generator=gen(60 + rep), device="cuda"))
        for t in o.values():
            t.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in o.items()}
        for t in o.values():
            t.view(torch.uint8).fill_(0x5A)
        calls()
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(got[n].view(torch.uint8), o[n].view(torch.uint8)), (rep, n)
    assert int(err) == 0


def test_two_streams_at_once():
    print("\ncase: expert rows on two streams", flush=True)
    sets = []
    for seed, (T, H, k) in enumerate([(700, 2048, 8), (900, 1024, 4)]):
        g, cap, slot, rows, w = case(30 + seed, T, H, k)
        sets.append((slot, rows, w, rand(g, T, H), sentinel(T, H), sentinel(cap, H),
                     torch.zeros((T, k), device="cuda")))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for (slot, rows, w, go, out, gr, gw), st in zip(sets, streams):
            ep.ep_combine_unpermute(rows, w, slot, out=out, stream=st)
            ep.ep_combine_unpermute_grad(go, rows, w, slot, grad_expert_out=gr,
                                         grad_topk_weights=gw, stream=st)
    torch.cuda.synchronize()
    for slot, rows, w, go, out, gr, gw in sets:
        s, r = slot.cpu(), P.f64(rows)
        r0 = torch.where(torch.isnan(r), torch.zeros((), dtype=torch.float64), r)
        wd = wsafe(w, s)
        want = P.unpermute(r, wd, s, None)
        P.assert_within(out, want, P.unpermute_bound(want, r0, wd, s, None), "out")
        _, want_w = P.unpermute_grad(P.f64(go), r, wd, s)
        P.assert_within(gw, want_w, P.dot_bound(P.f64(go), r0, s), "grad weights")


@pytest.mark.parametrize("k", [1, 2, 3, 4, 8, 9, 20])
@pytest.mark.parametrize("H", [8, 520, 7168])
def test_an_addend_comes_back_bit_for_bit(H, k):
    """A token with no pair (not routed, or its row out of range) gets addend[t] itself, its
    negative zeros, subnormals and infinities too; and zeros of both signs under pairs: the
    sum of negative zeros alone is a negative zero, any other sum of zeros a positive one."""
    print(f"\ncase: addend bits H={H} k={k}", flush=True)
    T = 12
    g = gen(H + k)
    values = torch.tensor([-0.0, 0.0, 1.0, -2.0**-133, 2.0**-130, float("inf"), float("-inf"), -3.5],
                          device="cuda", dtype=BF16)
    add = values[torch.randint(0, 8, (T, H), generator=g, device="cuda")]
    add[0], add[1], add[6:] = -0.0, 0.0, -0.0
    rows = torch.zeros((20, H), dtype=BF16, device="cuda")
    rows[10:] = -0.0
    slot = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    slot[5] = 20                       # out of range
    slot[6, 0], slot[7, -1] = 10, 3    # one pair of -0.0, one of +0.0
    slot[8], slot[9] = 11, 4           # all pairs of -0.0, all of +0.0
    slot[10, 0], slot[11, 0] = 12, 5   # a weight below zero turns the sign
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    w[10:] = -1.0
    w[0] = float("nan")
    out, fl = sentinel(T, H), flag()
    ep.ep_combine_unpermute(rows, w, slot, out=out, addend=add, error_flag=fl)
    assert int(fl) == ep.EP_DEVERR_SLOT_RANGE
    bits = out.view(torch.int16)
    assert torch.equal(bits[:6], add[:6].view(torch.int16))
    for t, negative in ((6, True), (7, False), (8, True), (9, False), (10, False), (11, True)):
        assert torch.all(bits[t] == (-0x8000 if negative else 0)), t
    # every weight 1, and in the addend's own place
    here = add.clone()
    ep.ep_combine_unpermute(rows, None, slot, out=here, addend=here)
    bits = here.view(torch.int16)
    assert torch.equal(bits[:6], add[:6].view(torch.int16))
    for t, negative in ((6, True), (7, False), (8, True), (9, False), (10, True), (11, False)):
        assert torch.all(bits[t] == (-0x8000 if negative else 0)), t
    # without an addend a sum of zeros is +0.0, as it is for a token with no pair
    ep.ep_combine_unpermute(rows, w, slot, out=out)
    assert torch.all(out.view(torch.int16) == 0)
