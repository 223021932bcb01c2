"""ep_rmsnorm and ep_rmsnorm_grad on the GPU against their 64-bit plain forms: widths from 8
channels to past what a block holds in registers, one token to many, both weight types, every
choice of outputs, outputs in the place of inputs, rows of zeros, infinities and NaN, graphs
and streams."""
import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_ops as P

pytestmark = pytest.mark.gpu

EPS = 1e-6
BF16 = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def weight_of(g, H, dtype):
    return (1 + 0.25 * torch.randn(H, generator=g, device="cuda")).to(dtype)


def e4m3(t):
    return P.f64(t.view(torch.float8_e4m3fn).float())


def check_norm(x, residual, w, residual_out=None, y=None, y_fp8=None, y_scales=None, eps=EPS):
    s, want = P.rmsnorm(P.f64(x), None if residual is None else P.f64(residual), P.f64(w), eps)
    if residual_out is not None:
        P.assert_within(residual_out, s, P.sum_bound(s), "residual_out")
    if y is not None:
        P.assert_within(y, want, P.y_bound(want), "y")
    if y_fp8 is not None:
        scale = P.fp8_scales(want)
        P.assert_within(y_scales, scale, 2.0**-14 * scale, "y_scales")
        step = P.f64(y_scales).repeat_interleave(P.GROUP, dim=1)
        P.assert_within(e4m3(y_fp8) * step, want, P.fp8_bound(want, scale), "y_fp8")


WIDTHS = [8, 16, 64, 128, 136, 384, 512, 520, 1000, 1024, 2056, 4096, 6144, 7168, 8192, 8200,
          16384, 16392, 32768, 40960]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T", [1, 5, 130])
def test_norm_widths(T, H):
    print(f"\ncase: rmsnorm T={T} H={H}", flush=True)
    g = gen(T * 100003 + H)
    for dtype in (BF16, torch.float32):
        for with_res in (False, True):
            x, w = rand(g, T, H), weight_of(g, H, dtype)
            res = rand(g, T, H, scale=3.0) if with_res else None
            o = dict(y=torch.full((T, H), 7.0, dtype=BF16, device="cuda"))
            if with_res:
                o["residual_out"] = torch.full((T, H), 7.0, dtype=BF16, device="cuda")
            if H % 128 == 0:
                o["y_fp8"] = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda")
                o["y_scales"] = torch.full((T, H // 128), -1.0, device="cuda")
            ep.ep_rmsnorm(x, w, residual=res, eps=EPS, **o)
            check_norm(x, res, w, **o)


@pytest.mark.parametrize("T,H", [(4096, 7168), (2049, 2048), (8193, 256), (20000, 64), (70000, 8),
                                 (60000, 264), (30001, 1032), (2_100_000, 8)])
def test_norm_many_rows(T, H):
    print(f"\ncase: rmsnorm T={T} H={H}", flush=True)
    g = gen(T)
    x, res, w = rand(g, T, H), rand(g, T, H), weight_of(g, H, BF16)
    y, ro = torch.zeros_like(x), torch.zeros_like(x)
    ep.ep_rmsnorm(x, w, residual=res, residual_out=ro, y=y, eps=EPS)
    pick = torch.randperm(T, generator=gen(1), device="cuda")[:512]
    pick[:2] = torch.tensor([0, T - 1])
    check_norm(x[pick], res[pick], w, residual_out=ro[pick], y=y[pick])


@pytest.mark.parametrize("outs", ["residual_out", "y", "fp8", "residual_out+fp8"])
def test_norm_each_choice_of_outputs_alone(outs):
    T, H = 33, 1280
    print(f"\ncase: rmsnorm outputs {outs}", flush=True)
    g = gen(5)
    x, res, w = rand(g, T, H), rand(g, T, H), weight_of(g, H, torch.float32)
    o = {}
    if "residual_out" in outs:
        o["residual_out"] = torch.zeros_like(x)
    if outs == "y":
        o["y"] = torch.zeros_like(x)
    if "fp8" in outs:
        o["y_fp8"] = torch.zeros((T, H), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        o["y_scales"] = torch.zeros((T, H // 128), device="cuda")
    ep.ep_rmsnorm(x, w, residual=res, eps=EPS, **o)
    check_norm(x, res, w, **o)


@pytest.mark.parametrize("H", [256, 7168, 40960])
def test_norm_in_place(H):
    T = 37
    print(f"\ncase: rmsnorm in place H={H}", flush=True)
    g = gen(H)
    x, res, w = rand(g, T, H), rand(g, T, H), weight_of(g, H, BF16)
    for swap in (False, True):
        a, b = x.clone(), res.clone()
        ro, y = (a, b) if swap else (b, a)
        ep.ep_rmsnorm(a, w, residual=b, residual_out=ro, y=y, eps=EPS)
        check_norm(x, res, w, residual_out=ro, y=y)


def test_norm_rows_of_zeros_infinities_and_nan():
    T, H = 12, 512
    print("\ncase: rmsnorm special rows", flush=True)
    g = gen(9)
    x, w = rand(g, T, H), weight_of(g, H, BF16)
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 130] = float("inf")
    x[4] = 1e-30          # squares below fp32: eps alone is left
    x[5] = 2.0**-133      # bf16 subnormals
    x[6, :128] = 0        # one group of zeros
    x[7, 5:] = 0
    x[8] = 1e17
    y = torch.zeros_like(x)
    codes = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((T, H // 128), device="cuda")
    ep.ep_rmsnorm(x, w, y=y, y_fp8=codes, y_scales=scales, eps=EPS)
    fine = [0, 1, 4, 5, 6, 7, 8, 9, 10, 11]
    check_norm(x[fine], None, w, y=y[fine], y_fp8=codes[fine], y_scales=scales[fine])
    assert torch.all(y[1] == 0) and torch.all(codes[1] == 0) and torch.all(scales[1] == 1)
    assert torch.all(codes[6, :128] == 0) and scales[6, 0] == 1
    assert torch.isnan(y[2]).all() and torch.isnan(codes[2].view(torch.float8_e4m3fn).float()).all()
    # 1 / sqrt(inf) = 0: the infinite channel is NaN, the others 0
    assert torch.isnan(y[3, 130]) and torch.all(y[3, :130] == 0) and torch.all(y[3, 131:] == 0)
    assert torch.isnan(codes[3].view(torch.float8_e4m3fn).float()).sum() == 1


@pytest.mark.parametrize("H", [128, 1024, 7168, 40960])
def test_codes_are_those_of_the_fp8_dispatch(H):
    """Rows of +-1 with eps 0 have r = 1 and y = +-weight, exact in bf16: the norm's codes and
    scales are then, bit for bit, what ep_dispatch_fp8 makes of y."""
    T = 9
    print(f"\ncase: codes against ep_dispatch_fp8 H={H}", flush=True)
    g = gen(H + 3)
    x = (torch.randint(0, 2, (T, H), generator=g, device="cuda") * 2 - 1).to(BF16)
    w = (torch.randn(H, generator=g, device="cuda") * torch.randn(H, generator=g, device="cuda").exp()).to(BF16)
    w[:128] = 0 if H > 128 else w[:128]
    y = torch.zeros_like(x)
    codes = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((T, H // 128), device="cuda")
    ep.ep_rmsnorm(x, w, y=y, y_fp8=codes, y_scales=scales, eps=0.0)
    assert torch.equal(y.float(), x.float() * w.float())
    slot = torch.arange(T, dtype=torch.int32, device="cuda").reshape(T, 1)
    idx = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    want, want_scales = torch.zeros_like(codes), torch.zeros_like(scales)
    ep.ep_dispatch_fp8(y, idx, None, 1, 1, slot, recv_x_fp8=want, recv_scales=want_scales)
    assert torch.equal(codes, want)
    assert torch.equal(scales.view(torch.int32), want_scales.view(torch.int32))


def test_norm_nan_weight_poisons_its_channel_alone():
    T, H = 3, 256
    g = gen(4)
    x, w = rand(g, T, H), weight_of(g, H, torch.float32)
    w[9] = float("nan")
    y = torch.zeros_like(x)
    codes = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((T, H // 128), device="cuda")
    ep.ep_rmsnorm(x, w, y=y, y_fp8=codes, y_scales=scales, eps=EPS)
    bad = torch.isnan(codes.view(torch.float8_e4m3fn).float())
    assert torch.equal(bad, torch.isnan(y)) and bad.sum() == T and bad[:, 9].all()
    w0 = w.clone()
    w0[9] = 0.0
    keep = [c for c in range(H) if c != 9]
    s, want = P.rmsnorm(P.f64(x), None, P.f64(w0), EPS)
    step = P.f64(scales).repeat_interleave(P.GROUP, dim=1)
    P.assert_within((e4m3(codes) * step)[:, keep], want[:, keep],
                    P.fp8_bound(want, P.fp8_scales(want))[:, keep], "codes beside a NaN")


def test_norm_infinite_weight_takes_its_group():
    """An infinity in a group of 128: scale infinity, the NaN code for itself, 0 for the rest;
    the other groups are as they would be."""
    T, H = 3, 384
    g = gen(14)
    x, w = rand(g, T, H), weight_of(g, H, torch.float32)
    x[:, 200] = 2.0
    w[200] = float("inf")
    y = torch.zeros_like(x)
    codes = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.zeros((T, H // 128), device="cuda")
    ep.ep_rmsnorm(x, w, y=y, y_fp8=codes, y_scales=scales, eps=EPS)
    v = codes.view(torch.float8_e4m3fn).float()
    assert torch.isinf(y[:, 200]).all() and torch.isinf(scales[:, 1]).all()
    assert torch.isnan(v[:, 200]).all()
    rest = [c for c in range(128, 256) if c != 200]
    assert torch.all(v[:, rest] == 0)
    keep = list(range(128)) + list(range(256, 384))
    w[200] = 0.0
    _, want = P.rmsnorm(P.f64(x), None, P.f64(w), EPS)
    step = P.f64(scales)[:, [0, 2]].repeat_interleave(128, dim=1)
    P.assert_within(e4m3(codes)[:, keep] * step, want[:, keep],
                    P.fp8_bound(want, P.fp8_scales(want))[:, keep], "the other groups")


def test_norm_of_squares_past_fp32_is_zero():
    x = torch.full((2, 256), 1e25, dtype=BF16, device="cuda")
    x[1] = 1.0
    y = torch.ones_like(x)
    ep.ep_rmsnorm(x, torch.ones(256, device="cuda"), y=y, eps=EPS)
    assert torch.all(y[0] == 0) and torch.all((y[1].float() - 1).abs() <= P.BF16)


def test_strided_host_and_wrongly_typed_tensors_are_refused():
    T, H = 8, 256
    x, w = torch.zeros((T, H), dtype=BF16, device="cuda"), torch.ones(H, device="cuda")
    wide = torch.zeros((T, 2 * H), dtype=BF16, device="cuda")
    y = torch.full_like(x, 3.0)
    for bad, exc in ((dict(residual=wide[:, ::2]), ValueError), (dict(residual=wide[:, :H]), ValueError),
                     (dict(residual=x.cpu()), ValueError), (dict(residual=x.half()), TypeError),
                     (dict(residual=x.float()), TypeError)):
        with pytest.raises(exc):
            ep.ep_rmsnorm(x, w, y=y, **bad)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x, w.cpu(), y=y)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x, torch.ones(2 * H, device="cuda")[::2], y=y)
    with pytest.raises(ep.EPError) as e:  # rows off the 16-byte grid
        off = torch.zeros(T * H + 4, dtype=BF16, device="cuda")[4:].view(T, H)
        ep.ep_rmsnorm(off, w, y=y)
    assert e.value.status == ep.EP_ERR_ALIGN
    torch.cuda.synchronize()
    assert torch.all(y == 3.0)  # nothing ran


def test_norm_tiny_weights_keep_finite_codes():
    T, H = 2, 128
    g = gen(6)
    x = rand(g, T, H)
    w = torch.full((H,), 2.0**-120, device="cuda")
    codes = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((T, 1), device="cuda")
    ep.ep_rmsnorm(x, w, y_fp8=codes, y_scales=scales, eps=EPS)
    assert torch.all(scales == 2.0**-100 / 448)
    assert torch.all(codes.view(torch.float8_e4m3fn).float().abs() < 1)


# ------------------------------------------------------------------------------- gradient

def check_grad(dy, dres, h, w, dx, dw, eps=EPS):
    a = [None if t is None else P.f64(t) for t in (dy, dres, h, w)]
    want, want_w = P.rmsnorm_grad(*a, eps)
    P.assert_within(dx, want, P.dx_bound(want, *a, eps), "grad_x")
    if dw is not None:
        P.assert_within(dw, want_w, P.dw_bound(a[0], a[2], eps), "grad_weight")


def workspace(T, H):
    return torch.full((max(16, ep.ep_rmsnorm_grad_workspace_bytes(T, H)),), 0xA5, dtype=torch.uint8,
                      device="cuda")


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T", [1, 3, 130])
def test_grad_widths(T, H):
    print(f"\ncase: rmsnorm_grad T={T} H={H}", flush=True)
    g = gen(T * 1000 + H)
    for dtype in (BF16, torch.float32):
        for with_res in (False, True):
            dy, h, w = rand(g, T, H), rand(g, T, H, scale=2.0), weight_of(g, H, dtype)
            dres = rand(g, T, H) if with_res else None
            dx = torch.full_like(h, 9.0)
            dw = torch.full((H,), -3.0, device="cuda")
            ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_residual_out=dres, grad_weight=dw,
                               workspace=workspace(T, H), eps=EPS)
            check_grad(dy, dres, h, w, dx, dw)


@pytest.mark.parametrize("T,H", [(2000, 1024), (4099, 256), (1021, 2056), (9001, 40), (600, 7168),
                                 (3001, 7168), (2600, 8200), (257, 520), (1300, 16384)])
def test_grad_many_rows_and_the_same_bits_twice(T, H):
    print(f"\ncase: rmsnorm_grad T={T} H={H}", flush=True)
    g = gen(T + H)
    dy, dres, h, w = rand(g, T, H), rand(g, T, H), rand(g, T, H), weight_of(g, H, torch.float32)
    dx, dw = torch.zeros_like(h), torch.zeros(H, device="cuda")
    ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_residual_out=dres, grad_weight=dw,
                       workspace=workspace(T, H), eps=EPS)
    check_grad(dy, dres, h, w, dx, dw)
    dx2, dw2 = torch.zeros_like(h), torch.zeros(H, device="cuda")
    ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx2, grad_residual_out=dres, grad_weight=dw2,
                       workspace=workspace(T, H), eps=EPS)
    assert torch.equal(dx.view(torch.int16), dx2.view(torch.int16))
    assert torch.equal(dw.view(torch.int32), dw2.view(torch.int32))


@pytest.mark.parametrize("H", [136, 7168, 40960])
@pytest.mark.parametrize("place", ["grad_y", "grad_residual_out", "h"])
def test_grad_in_place_and_without_the_weights_gradient(place, H):
    T = 70
    print(f"\ncase: rmsnorm_grad in place of {place} H={H}", flush=True)
    g = gen(H)
    t = dict(grad_y=rand(g, T, H), grad_residual_out=rand(g, T, H), h=rand(g, T, H))
    w = weight_of(g, H, BF16)
    for with_w in (True, False):
        c = {k: v.clone() for k, v in t.items()}
        dw = torch.zeros(H, device="cuda") if with_w else None
        ep.ep_rmsnorm_grad(c["grad_y"], c["h"], w, grad_x=c[place],
                           grad_residual_out=c["grad_residual_out"], grad_weight=dw,
                           workspace=workspace(T, H) if with_w else None, eps=EPS)
        check_grad(t["grad_y"], t["grad_residual_out"], t["h"], w, c[place], dw)


def test_grad_of_a_row_of_zeros_and_a_nan_row():
    T, H = 6, 256
    g = gen(2)
    dy, h, w = rand(g, T, H), rand(g, T, H), weight_of(g, H, BF16)
    h[1] = 0
    dx, dw = torch.zeros_like(h), torch.zeros(H, device="cuda")
    ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_weight=dw, workspace=workspace(T, H), eps=EPS)
    check_grad(dy, None, h, w, dx, dw)
    h[2, 3] = float("nan")
    ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_weight=dw, workspace=workspace(T, H), eps=EPS)
    assert torch.isnan(dx[2]).all() and torch.isnan(dw).all()
    rest = [0, 1, 3, 4, 5]
    check_grad(dy[rest], None, h[rest], w, dx[rest], None)


@pytest.mark.parametrize("H", [64, 1024, 7168])
def test_grad_of_shorter_batches_in_the_longest_ones_workspace(H):
    print(f"\ncase: rmsnorm_grad H={H}, one workspace for many lengths", flush=True)
    g = gen(H)
    w = weight_of(g, H, BF16)
    ws = workspace(700, H)
    for T in (700, 255, 256, 257, 1, 699, 512, 3, 513):
        dy, h = rand(g, T, H), rand(g, T, H)
        dx, dw = torch.zeros_like(h), torch.zeros(H, device="cuda")
        ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_weight=dw, workspace=ws, eps=EPS)
        check_grad(dy, None, h, w, dx, dw)


def test_grad_weight_off_the_16_byte_grid():
    """grad_weight needs 4-byte alignment only; one block's sum leaves in wide words where it
    may."""
    for T, H in ((1, 1024), (2, 7168), (300, 512)):
        print(f"\ncase: rmsnorm_grad T={T} H={H}, grad_weight at 4 bytes", flush=True)
        g = gen(T)
        dy, h, w = rand(g, T, H), rand(g, T, H), weight_of(g, H, BF16)
        room = torch.full((H + 2,), 7.0, device="cuda")
        dx = torch.zeros_like(h)
        ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_weight=room[1:H + 1], workspace=workspace(T, H),
                           eps=EPS)
        check_grad(dy, None, h, w, dx, room[1:H + 1])
        assert float(room[0]) == 7.0 and float(room[H + 1]) == 7.0


def test_grad_with_eps_zero_and_a_last_block_half_empty():
    """Rows that are not there (a block holds several) leave no 0 / 0 in the sums."""
    T, H = 5, 64
    g = gen(1)
    dy, h, w = rand(g, T, H), rand(g, T, H), weight_of(g, H, BF16)
    dx, dw = torch.zeros_like(h), torch.zeros(H, device="cuda")
    ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_weight=dw, workspace=workspace(T, H), eps=0.0)
    check_grad(dy, None, h, w, dx, dw, eps=0.0)
    for T, H in ((259, 64), (1021, 2056)):
        dy, h, w = rand(g, T, H), rand(g, T, H), weight_of(g, H, BF16)
        dx, dw = torch.zeros_like(h), torch.zeros(H, device="cuda")
        ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_weight=dw, workspace=workspace(T, H), eps=0.0)
        check_grad(dy, None, h, w, dx, dw, eps=0.0)


def test_no_tokens():
    H = 256
    w = torch.ones(H, device="cuda")
    x = torch.empty((0, H), dtype=BF16, device="cuda")
    ep.ep_rmsnorm(x, w, y=torch.empty_like(x))
    dw = torch.full((H,), 5.0, device="cuda")
    ep.ep_rmsnorm_grad(x, x, w, grad_x=torch.empty_like(x), grad_weight=dw)
    assert torch.all(dw == 0)
    dw.fill_(5.0)
    ep.ep_rmsnorm_grad(x, x, w, grad_x=torch.empty_like(x), grad_weight=dw,
                       workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert torch.all(dw == 0)
    assert ep.ep_rmsnorm_grad_workspace_bytes(0, H) == 0


def test_norm_and_grad_replay_in_a_graph():
    T, H = 300, 1024
    print("\ncase: rmsnorm graph", flush=True)
    g = gen(8)
    x, res, dy = rand(g, T, H), rand(g, T, H), rand(g, T, H)
    w = weight_of(g, H, BF16)
    ro, y, dx = (torch.zeros_like(x) for _ in range(3))
    codes = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((T, H // 128), device="cuda")
    dw, ws = torch.zeros(H, device="cuda"), workspace(T, H)

    def calls():
        ep.ep_rmsnorm(x, w, residual=res, residual_out=ro, y=y, y_fp8=codes, y_scales=scales)
        ep.ep_rmsnorm_grad(dy, ro, w, grad_x=dx, grad_residual_out=y, grad_weight=dw, workspace=ws)

    outs = [ro, y, dx, codes, scales, dw]
    graph = torch.cuda.CUDAGraph()
    calls()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls()
    for rep in range(3):
        x.copy_(rand(gen(100 + rep), T, H))
        for t in outs:
            t.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        calls()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), rep


def test_norm_on_two_streams():
    print("\ncase: rmsnorm on two streams", flush=True)
    H = 2048
    g = gen(3)
    w = weight_of(g, H, BF16)
    sets = []
    for T in (900, 1100):
        h, dy = rand(g, T, H), rand(g, T, H)
        sets.append((h, dy, torch.zeros_like(h), torch.zeros_like(h), torch.zeros(H, device="cuda"),
                     workspace(T, H)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for (h, dy, y, dx, dw, ws), s in zip(sets, streams):
            ep.ep_rmsnorm(h, w, y=y, stream=s)
            ep.ep_rmsnorm_grad(dy, h, w, grad_x=dx, grad_weight=dw, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for h, dy, y, dx, dw, _ in sets:
        check_norm(h, None, w, y=y)
        check_grad(dy, None, h, w, dx, dw)


def test_grad_workspace_too_small_is_refused():
    T, H = 64, 128
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    w = torch.ones(H, device="cuda")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for ws in (small, None):
        with pytest.raises(ep.EPError) as e:
            ep.ep_rmsnorm_grad(x, x, w, grad_x=torch.empty_like(x),
                               grad_weight=torch.zeros(H, device="cuda"), workspace=ws)
        assert e.value.status == ep.EP_ERR_CAPACITY


def repeats_of(base, times):
    """[times * n][H]: the base's n rows over and over."""
    return base.unsqueeze(0).expand(times, *base.shape).reshape(times * base.shape[0], -1).contiguous()


def assert_repeats(got, base, times, what):
    """Every repeat of the base's rows holds the base's bits."""
    got = got.view(times, *base.shape)
    for i in range(times):
        assert torch.equal(got[i].view(torch.uint8), base.view(torch.uint8)), f"{what}: repeat {i} of {times}"


@pytest.mark.parametrize("H", [8, 128, 512, 1024, 2048, 2176])
def test_norm_in_two_launches_on_every_row(H):
    """2^21 + 4096 rows, past what one launch takes, in each form of the kernel: all rows of all
    outputs, the codes and scales of the second launch among them."""
    n, times = 4096, 513
    print(f"\ncase: rmsnorm in two launches H={H}", flush=True)
    g = gen(H)
    x, res, w = rand(g, n, H), rand(g, n, H, scale=3.0), weight_of(g, H, BF16)

    def outputs(T):
        o = dict(y=torch.full((T, H), 7.0, dtype=BF16, device="cuda"),
                 residual_out=torch.full((T, H), 7.0, dtype=BF16, device="cuda"))
        if H % 128 == 0:
            o["y_fp8"] = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda")
            o["y_scales"] = torch.full((T, H // 128), -1.0, device="cuda")
        return o

    base, many = outputs(n), outputs(n * times)
    ep.ep_rmsnorm(x, w, residual=res, eps=EPS, **base)
    check_norm(x, res, w, **base)
    ep.ep_rmsnorm(repeats_of(x, times), w, residual=repeats_of(res, times), eps=EPS, **many)
    for name in base:
        assert_repeats(many[name], base[name], times, name)


@pytest.mark.parametrize("H,n,times", [(8, 4096, 270), (64, 4096, 270), (264, 4096, 270),
                                       (7168, 4096, 17), (40960, 512, 9)])
@pytest.mark.parametrize("with_res", [False, True])
def test_grad_without_the_weights_gradient_on_every_row(H, n, times, with_res):
    """More rows than the blocks of one launch hold at once: blocks walk on to further rows.
    (Rows past 16384 channels take a block each.)"""
    print(f"\ncase: rmsnorm_grad without grad_weight T={n * times} H={H} res={with_res}", flush=True)
    g = gen(H + 1)
    dy, h, w = rand(g, n, H), rand(g, n, H, scale=4.0), weight_of(g, H, torch.float32)
    dres = rand(g, n, H) if with_res else None
    base = torch.full((n, H), 7.0, dtype=BF16, device="cuda")
    many = torch.full((n * times, H), 7.0, dtype=BF16, device="cuda")
    ep.ep_rmsnorm_grad(dy, h, w, grad_x=base, grad_residual_out=dres, eps=EPS)
    d = (P.f64(dy), P.f64(dres) if with_res else None, P.f64(h), P.f64(w), EPS)
    dx, _ = P.rmsnorm_grad(*d)
    P.assert_within(base, dx, P.dx_bound(dx, *d), "grad_x")
    ep.ep_rmsnorm_grad(repeats_of(dy, times), repeats_of(h, times), w, grad_x=many,
                       grad_residual_out=repeats_of(dres, times) if with_res else None, eps=EPS)
    assert_repeats(many, base, times, "grad_x")
