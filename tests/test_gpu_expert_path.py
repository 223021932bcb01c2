"""The operators together, as a mixture-of-experts block uses them: norm, layout, expert-major
dispatch, experts, weighted way back, and the gradients from the block's output to its
inputs, through ExpertPath and against the whole block in 64 bits on the CPU (the routing
taken as given). Also a decode loop of single tokens and a training step in a graph."""
import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_ops as P
from combine_ep_get_03_amd.pipeline import ExpertPath

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def inputs(seed, T, H, E, k, dropped=0.1):
    g = gen(seed)
    d = dict(x=torch.randn((T, H), generator=g, device="cuda").to(BF16),
             residual=(2 * torch.randn((T, H), generator=g, device="cuda")).to(BF16),
             weight=(1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16),
             shared=torch.randn((T, H), generator=g, device="cuda").to(BF16),
             grad_out=torch.randn((T, H), generator=g, device="cuda").to(BF16),
             grad_res=torch.randn((T, H), generator=g, device="cuda").to(BF16),
             gate=torch.rand((T, k), generator=g, device="cuda") + 0.1,
             scale=0.5 + torch.rand((E, H), generator=g, device="cuda"))
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices
    drop = torch.rand((T, k), generator=g, device="cuda") < dropped
    d["idx"] = torch.where(drop, -1, idx).contiguous()
    return d


def expert_rows(offset, T, k, E):
    """Expert of every routed row, from the layout's offsets."""
    o = offset.long()
    row = torch.arange(int(o[-1]), device=o.device)
    return torch.bucketize(row, o[1:], right=True)


def experts(rows, e, scale):
    """Each expert scales its channels: bf16(row * scale[e])."""
    return (rows.float() * scale[e]).to(BF16)


def block_64(d, eps):
    """The block in 64 bits, with autograd: (residual_out, y, out, leaves)."""
    leaf = {n: P.f64(d[n]).requires_grad_() for n in ("x", "residual", "weight", "gate", "shared")}
    s, y = P.rmsnorm(leaf["x"], leaf["residual"], leaf["weight"], eps)
    idx = d["idx"].cpu()
    hit = (idx >= 0).unsqueeze(2)
    zero = torch.zeros((), dtype=torch.float64)
    per = y.unsqueeze(1) * P.f64(d["scale"])[idx.clamp(min=0)]
    out = (torch.where(hit, per, zero) * leaf["gate"].unsqueeze(2)).sum(dim=1) + leaf["shared"]
    return s, y, out, leaf


@pytest.mark.parametrize("T,H,E,k,R,N", [(1, 7168, 256, 8, 32, 4), (257, 1024, 16, 4, 4, 2),
                                         (130, 512, 64, 6, 1, 1), (1000, 128, 16, 2, 2, 1)])
def test_block_forward_and_backward(T, H, E, k, R, N):
    print(f"\ncase: block T={T} H={H} E={E} k={k}", flush=True)
    d = inputs(T + H, T, H, E, k)
    p = ExpertPath(T, H, E, k, R=R, N=N, training=True)
    p.norm(d["x"], d["weight"], d["residual"])
    p.dispatch(d["idx"])
    M = int(p.expert_offset[-1])
    assert M == int((d["idx"] >= 0).sum())
    e = expert_rows(p.expert_offset, T, k, E)
    expert_out = torch.full((T * k, H), float("nan"), dtype=BF16, device="cuda")
    expert_out[:M] = experts(p.perm_x[:M], e, d["scale"])
    p.combine(expert_out, d["gate"], addend=d["shared"])
    # backwards
    p.combine_grad(d["grad_out"], expert_out, d["gate"])
    grad_perm = torch.full((T * k, H), float("nan"), dtype=BF16, device="cuda")
    grad_perm[:M] = experts(p.grad_expert_out[:M], e, d["scale"])
    p.dispatch_grad(grad_perm)
    p.norm_grad(d["weight"], d["grad_res"])
    assert int(p.error_flag) == 0

    s, y, out, leaf = block_64(d, p.eps)
    (out * P.f64(d["grad_out"])).sum().add((s * P.f64(d["grad_res"])).sum()).backward()
    with torch.no_grad():
        gate, scale, idx = P.f64(d["gate"]), P.f64(d["scale"]), d["idx"].cpu()
        P.assert_within(p.residual_out, s, P.sum_bound(s), "residual_out")
        P.assert_within(p.y, y, P.y_bound(y), "y")
        hit = (idx >= 0).unsqueeze(2)
        zero = torch.zeros((), dtype=torch.float64)
        # out: each pair's row was rounded to bf16 twice (the norm's output, the expert's), the
        # sum once more
        mag = (torch.where(hit, (y.unsqueeze(1) * scale[idx.clamp(min=0)]).abs(), zero)
               * gate.unsqueeze(2)).sum(dim=1)
        P.assert_within(p.out, out, 2.2 * P.BF16 * mag + P.BF16 * 1.01 * out.abs() + 1e-6 * leaf["shared"].abs(),
                        "out")
        # the gate's gradient: rows twice rounded, under a dot product with grad_out
        go = P.f64(d["grad_out"])
        dot = torch.where(hit, (y.unsqueeze(1) * scale[idx.clamp(min=0)] * go.unsqueeze(1)).abs(), zero).sum(dim=2)
        P.assert_within(p.grad_topk_weights, leaf["gate"].grad, 2.2 * P.BF16 * dot, "gate's gradient")
        # the norm's incoming gradient: three roundings on the way (the row's gradient, the
        # expert's, the sum over a token's rows)
        dy = (torch.where(hit, scale[idx.clamp(min=0)] * go.unsqueeze(1), zero) * gate.unsqueeze(2))
        gy, gy_mag = dy.sum(dim=1), dy.abs().sum(dim=1)
        gy_off = 2.2 * P.BF16 * gy_mag + 1.01 * P.BF16 * gy.abs()
        P.assert_within(p.grad_y, gy, gy_off, "grad_y")
        # the norm's own gradient, with grad_y off by gy_off and h rounded to bf16: n is off by
        # BF16 |n| and r by BF16 relative at most, so each term of dx = r (g - n mean(g n))
        # by at most 3 BF16 (four factors that hold h: r, n, r and n) plus its share of gy_off
        w = P.f64(d["weight"]).abs()
        r = 1 / torch.sqrt(s.square().mean(dim=1, keepdim=True) + p.eps)
        n, g, g_off = (s * r).abs(), gy.abs() * w, gy_off * w
        first, second = r * g, r * n * (g * n).mean(dim=1, keepdim=True)
        off = r * (g_off + n * (g_off * n).mean(dim=1, keepdim=True)) + P.BF16 * 1.1 * first + 5 * P.BF16 * second
        P.assert_within(p.grad_x, leaf["x"].grad, 1.05 * off + P.BF16 * 1.01 * leaf["x"].grad.abs(), "grad_x")
        assert torch.equal(leaf["x"].grad, leaf["residual"].grad)
        woff = ((gy_off + 2.2 * P.BF16 * gy.abs()) * n).sum(dim=0)
        P.assert_within(p.grad_weight, leaf["weight"].grad, 1.05 * woff, "grad_weight")


@pytest.mark.parametrize("T,H,E,k", [(1, 7168, 256, 8), (100, 1024, 16, 4)])
def test_block_with_e4m3_rows(T, H, E, k):
    print(f"\ncase: fp8 block T={T} H={H}", flush=True)
    d = inputs(T + H + 1, T, H, E, k)
    p = ExpertPath(T, H, E, k, fp8=True)
    p.norm(d["x"], d["weight"], d["residual"])
    p.dispatch(d["idx"])
    M = int(p.expert_offset[-1])
    e = expert_rows(p.expert_offset, T, k, E)
    rows = p.perm_x_fp8[:M].view(torch.float8_e4m3fn).float() * p.perm_scales[:M].repeat_interleave(128, dim=1)
    expert_out = torch.full((T * k, H), float("nan"), dtype=BF16, device="cuda")
    expert_out[:M] = experts(rows, e, d["scale"])
    p.combine(expert_out, d["gate"], addend=d["shared"])
    assert int(p.error_flag) == 0
    src = p.perm_src_idx[:M].cpu().long()
    assert torch.equal(p.perm_x_fp8[:M].cpu(), p.y_fp8.cpu()[src])
    s, y, out, _ = block_64(d, p.eps)
    with torch.no_grad():
        idx, hit = d["idx"].cpu(), (d["idx"].cpu() >= 0).unsqueeze(2)
        zero = torch.zeros((), dtype=torch.float64)
        scale = P.f64(d["scale"])[idx.clamp(min=0)]
        per_off = P.fp8_bound(y, P.fp8_scales(y)).unsqueeze(1) * scale * (1 + P.BF16) \
            + P.BF16 * (y.unsqueeze(1) * scale).abs()
        off = (torch.where(hit, per_off, zero) * P.f64(d["gate"]).unsqueeze(2)).sum(dim=1)
        P.assert_within(p.out, out, 1.02 * off + P.BF16 * 1.02 * out.abs() + 1e-5, "out")


def test_decode_loop_of_single_tokens():
    """Ten steps of one token through one ExpertPath, the residual stream kept in place."""
    H, E, k, T = 2048, 64, 8, 1
    print("\ncase: decode loop", flush=True)
    p = ExpertPath(T, H, E, k)
    d = inputs(77, T, H, E, k, dropped=0.0)
    res, x = d["residual"], d["x"]
    for step in range(10):
        p.norm(x, d["weight"], res)
        s, y = P.rmsnorm(P.f64(x), P.f64(res), P.f64(d["weight"]), p.eps)
        P.assert_within(p.y, y, P.y_bound(y), f"y of step {step}")
        idx = torch.rand((T, E), generator=gen(step), device="cuda").topk(k, dim=1).indices
        p.dispatch(idx)
        e = expert_rows(p.expert_offset, T, k, E)
        expert_out = experts(p.perm_x, e, d["scale"])
        p.combine(expert_out, d["gate"])
        slot = p.layout_buf.expert_slot.cpu()
        want = P.unpermute(P.f64(expert_out), P.f64(d["gate"]), slot, None)
        P.assert_within(p.out, want, P.unpermute_bound(want, P.f64(expert_out), P.f64(d["gate"]), slot, None),
                        f"out of step {step}")
        x, res = p.out.clone(), p.residual_out.clone()


def test_training_step_replays_in_a_graph_beside_an_eager_one():
    """The whole step captured, replayed on new inputs, with the same step run eagerly on a
    second ExpertPath between the replays; both give the same bits."""
    T, H, E, k = 200, 1024, 16, 4
    print("\ncase: training step in a graph", flush=True)
    d = inputs(5, T, H, E, k)
    a, b = (ExpertPath(T, H, E, k, training=True) for _ in range(2))

    def step(p):
        p.norm(d["x"], d["weight"], d["residual"])
        p.dispatch(d["idx"])
        p.combine(p.perm_x, d["gate"], addend=d["shared"])
        p.combine_grad(d["grad_out"], p.perm_x, d["gate"])
        p.dispatch_grad(p.grad_expert_out)
        p.norm_grad(d["weight"], d["grad_res"])

    names = ["residual_out", "y", "out", "grad_expert_out", "grad_topk_weights", "grad_y", "grad_x",
             "grad_weight"]
    for p in (a, b):
        p.grad_expert_out.zero_()
    step(a)
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for rep in range(3):
        new = inputs(200 + rep, T, H, E, k)
        for n in d:
            d[n].copy_(new[n])
        for p in (a, b):
            for n in names:
                getattr(p, n).zero_()
        torch.cuda.synchronize()
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        for n in names:
            u, v = getattr(a, n), getattr(b, n)
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)), (rep, n)
        assert int(a.error_flag) == 0 and int(b.error_flag) == 0


def test_an_empty_batch():
    p = ExpertPath(0, 256, 16, 2, training=True)
    x = torch.empty((0, 256), dtype=BF16, device="cuda")
    w = torch.ones(256, device="cuda")
    gate = torch.empty((0, 2), device="cuda")
    p.grad_weight.fill_(4.0)
    p.norm(x, w, x)
    p.dispatch(torch.empty((0, 2), dtype=torch.int64, device="cuda"))
    assert int(p.expert_offset[-1]) == 0
    p.combine(p.perm_x, gate)
    p.combine_grad(x, p.perm_x, gate)
    p.dispatch_grad(p.grad_expert_out)
    p.norm_grad(w)
    assert torch.all(p.grad_weight == 0) and int(p.error_flag) == 0


def test_duplicate_and_bad_expert_ids():
    """A token that names an expert twice has two rows of it; ids out of range are dropped and
    reported, and their gate's gradient is zero."""
    T, H, E, k = 60, 256, 8, 4
    print("\ncase: duplicate and bad ids", flush=True)
    d = inputs(9, T, H, E, k, dropped=0.0)
    d["idx"][3] = 5
    d["idx"][10, 1] = E + 2
    d["idx"][11, 0] = -7
    p = ExpertPath(T, H, E, k, training=True)
    p.norm(d["x"], d["weight"])
    assert p.h is d["x"]
    p.dispatch(d["idx"])
    M = int(p.expert_offset[-1])
    assert M == T * k - 2 and int(p.error_flag) == ep.EP_DEVERR_TOPK_RANGE
    p.combine(p.perm_x, d["gate"])
    _, y = P.rmsnorm(P.f64(d["x"]), None, P.f64(d["weight"]), p.eps)
    routed = (d["idx"].cpu() >= 0) & (d["idx"].cpu() < E)
    gate = torch.where(routed, P.f64(d["gate"]), torch.zeros((), dtype=torch.float64))
    want = y * gate.sum(dim=1, keepdim=True)
    # every row of a token is its y, rounded once; the sum once more
    P.assert_within(p.out, want, 2.1 * P.BF16 * want.abs() + 1e-30, "out")
    p.combine_grad(d["grad_out"], p.perm_x, d["gate"])
    gw = p.grad_topk_weights.cpu()
    assert torch.all(gw[~routed] == 0) and torch.all(gw[routed] != 0)
    assert torch.equal(gw[3], gw[3, :1].expand(k))


def test_gradients_need_a_training_path():
    p = ExpertPath(4, 128, 16, 2)
    x = torch.zeros((4, 128), dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="training"):
        p.dispatch_grad(x)
    q = ExpertPath(4, 128, 16, 2, training=True)
    with pytest.raises(ValueError, match="norm"):
        q.norm_grad(torch.ones(128, device="cuda"))
    assert ep.EP_OK == 0


def whole_block_64(d, eps):
    """The block whose gate and shared expert are functions of y, in 64 bits with autograd:
    gate[t][j] = <y[t], router[:, idx[t][j]]>, shared = y * shared_scale."""
    leaf = {n: P.f64(d[n]).requires_grad_() for n in ("x", "residual", "weight")}
    s, y = P.rmsnorm(leaf["x"], leaf["residual"], leaf["weight"], eps)
    idx = d["idx"].cpu()
    hit = (idx >= 0).unsqueeze(2)
    zero = torch.zeros((), dtype=torch.float64)
    gate = (y @ P.f64(d["router"])).gather(1, idx.clamp(min=0))
    per = y.unsqueeze(1) * P.f64(d["scale"])[idx.clamp(min=0)]
    out = torch.where(hit, per * gate.unsqueeze(2), zero).sum(dim=1) + y * P.f64(d["shared_scale"])
    return s, y, gate, out, leaf


@pytest.mark.parametrize("T,H,E,k,apart", [(1, 7168, 256, 8, True), (130, 512, 64, 6, True),
                                           (257, 1024, 16, 4, True), (257, 1024, 16, 4, False),
                                           (1000, 128, 16, 2, True)])
def test_block_whose_gate_and_shared_expert_come_from_the_norm(T, H, E, k, apart):
    """All three ways of y's gradient: expert rows, router, shared expert. The addend is a
    tensor of its own, or what grad_y holds."""
    print(f"\ncase: whole block T={T} H={H} E={E} k={k} own addend {apart}", flush=True)
    d = inputs(T + H + 3, T, H, E, k)
    g = gen(T + H + 4)
    d["router"] = torch.randn((H, E), generator=g, device="cuda") / H**0.5
    d["shared_scale"] = torch.rand(H, generator=g, device="cuda") + 0.5
    idx = d["idx"].clamp(min=0)
    hit = d["idx"] >= 0
    p = ExpertPath(T, H, E, k, training=True)
    p.norm(d["x"], d["weight"], d["residual"])
    gate = (p.y.double() @ d["router"].double()).gather(1, idx).float().contiguous()
    p.dispatch(d["idx"])
    M = int(p.expert_offset[-1])
    e = expert_rows(p.expert_offset, T, k, E)
    expert_out = torch.full((T * k, H), float("nan"), dtype=BF16, device="cuda")
    expert_out[:M] = experts(p.perm_x[:M], e, d["scale"])
    p.combine(expert_out, gate, addend=(p.y.float() * d["shared_scale"]).to(BF16))
    # backwards
    p.combine_grad(d["grad_out"], expert_out, gate)
    to_router = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    to_router.scatter_add_(1, idx, torch.where(hit, p.grad_topk_weights.double(), 0.0))
    rest = (to_router @ d["router"].double().t().contiguous()
            + d["grad_out"].double() * d["shared_scale"].double()).to(BF16)
    grad_perm = torch.full((T * k, H), float("nan"), dtype=BF16, device="cuda")
    grad_perm[:M] = experts(p.grad_expert_out[:M], e, d["scale"])
    if apart:
        p.dispatch_grad(grad_perm, addend=rest)
    else:
        p.grad_y.copy_(rest)
        p.dispatch_grad(grad_perm, addend=p.grad_y)
    slot = p.layout_buf.expert_slot.cpu()
    want = P.unpermute(P.f64(grad_perm), None, slot, P.f64(rest))
    P.assert_within(p.grad_y, want, P.unpermute_bound(want, P.f64(grad_perm), None, slot, P.f64(rest)),
                    "grad_y of its inputs")
    p.norm_grad(d["weight"], d["grad_res"])
    assert int(p.error_flag) == 0

    s, y, gate64, out, leaf = whole_block_64(d, p.eps)
    y.retain_grad()
    (out * P.f64(d["grad_out"])).sum().add((s * P.f64(d["grad_res"])).sum()).backward()
    with torch.no_grad():
        idx, hit = idx.cpu(), hit.cpu().unsqueeze(2)
        zero = torch.zeros((), dtype=torch.float64)
        go, scale = P.f64(d["grad_out"]), P.f64(d["scale"])[idx]
        router = P.f64(d["router"])
        # Roundings, each BF16 relative. y was rounded once, so a gate weight is off by
        # BF16 gm at most, gm the sum of its terms' magnitudes. On the expert rows' way:
        # the gate weight, its product with grad_out, the expert's product. On the router's:
        # y and the expert's row under the dot product, the addend's. On the shared expert's:
        # the addend's. At last grad_y's own. 0.2 BF16 more for fp32 and second-order terms.
        gm = (y.abs() @ router.abs()).gather(1, idx)
        rows = torch.where(hit, (scale * go.abs().unsqueeze(1)) * gm.unsqueeze(2), zero).sum(dim=1)
        dot = torch.where(hit, (y.unsqueeze(1) * scale * go.unsqueeze(1)).abs(), zero).sum(dim=2)
        way = torch.zeros((T, E), dtype=torch.float64).scatter_add_(1, idx, dot) @ router.abs().t()
        gy = y.grad
        gy_off = P.BF16 * (3.2 * rows + 3.2 * way + 1.2 * P.f64(d["shared_scale"]) * go.abs() + 1.01 * gy.abs())
        P.assert_within(p.grad_y, gy, gy_off, "grad_y")
        # The same gradient at the values that the forward pass held (its roundings apart): what
        # is left are the backward pass's own roundings, two on the expert rows' way (row and
        # expert), one of the addend, grad_y's; and the dot product's in fp32 on the router's.
        # This bound sees each of the two further ways: grad_y without it fails.
        by_expert = torch.where(hit, P.gather(P.f64(expert_out), slot) * go.unsqueeze(1), zero)
        to_e = torch.zeros((T, E), dtype=torch.float64)
        by_router = to_e.scatter_add(1, idx, by_expert.sum(dim=2)) @ router.t()
        way = to_e.scatter_add(1, idx, by_expert.abs().sum(dim=2)) @ router.abs().t()
        by_shared = go * P.f64(d["shared_scale"])
        by_rows = torch.where(hit, scale * P.f64(gate).unsqueeze(2) * go.unsqueeze(1), zero)
        held = by_rows.sum(dim=1) + by_router + by_shared
        off = P.BF16 * (2.1 * by_rows.abs().sum(dim=1) + 1.1 * (by_router + by_shared).abs()
                        + 1.01 * held.abs()) + 2.0**-13 * way
        P.assert_within(p.grad_y, held, off, "grad_y at the values held")
        for part in (by_router, by_shared):
            with pytest.raises(AssertionError):
                P.assert_within(held - part, held, off, "grad_y without a part")
        # the norm's gradient of it, as in the block above
        w = P.f64(d["weight"]).abs()
        r = 1 / torch.sqrt(s.square().mean(dim=1, keepdim=True) + p.eps)
        n, g_, g_off = (s * r).abs(), gy.abs() * w, gy_off * w
        first, second = r * g_, r * n * (g_ * n).mean(dim=1, keepdim=True)
        off = r * (g_off + n * (g_off * n).mean(dim=1, keepdim=True)) + P.BF16 * 1.1 * first + 5 * P.BF16 * second
        P.assert_within(p.grad_x, leaf["x"].grad, 1.05 * off + P.BF16 * 1.01 * leaf["x"].grad.abs(), "grad_x")
        woff = ((gy_off + 2.2 * P.BF16 * gy.abs()) * n).sum(dim=0)
        P.assert_within(p.grad_weight, leaf["weight"].grad, 1.05 * woff, "grad_weight")
