"""Small weights' gradients over many rows, whose rows are cut into pieces: against 64 bits, with
experts of no row, one, a piece's rows and one more; both types, added to or not; rows past the
capacity, offsets that make no sense, another stream, a graph; and through ExpertPath."""
import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_experts as X
import plain_ops as P
from test_gpu_expert_ffn import BF16, F32, I32, U8, finite, flag, gen, offsets, rows_of

pytestmark = pytest.mark.gpu

# (rows per expert, rows before and behind them, M, N)
CASES = [([5000], 0, 0, 72, 8), ([1024], 0, 0, 8, 264), ([4099], 700, 3, 136, 520),
         ([1], 2000, 0, 128, 256), ([0], 3000, 0, 8, 8), ([0, 1025, 0, 0, 6000, 1, 256, 257, 0], 5, 0, 200, 72),
         ([256, 512, 0, 8000], 256, 0, 64, 384), ([2048] * 3 + [0] * 2, 0, 300, 1032, 1000),
         ([2048, 1, 2047], 0, 300, 1032, 1000),
         ([300] * 100 + [90000], 0, 0, 24, 40)]


def given(E, n, M, N):
    return torch.full((ep.ep_expert_weight_grad_workspace_bytes(E, n, M, N),), 0xA5, dtype=U8,
                      device="cuda")


@pytest.mark.parametrize("counts,lead,tail,M,N", CASES, ids=lambda v: str(v)[:24])
def test_pieces_against_64_bits(counts, lead, tail, M, N):
    print(f"\ncase: {counts[:9]} {lead} {tail} {M}x{N}", flush=True)
    g = gen(31 + M)
    off, offset = offsets(counts, lead)
    E, lo, hi = len(counts), off[0], off[-1]
    grad, inp = rows_of(g, counts, lead, tail, M), rows_of(g, counts, lead, tail, N)
    ws = given(E, grad.shape[0], M, N)
    tiles = E * -(-M // 128) * -(-N // 256)
    assert (ws.numel() > 0) == (tiles <= 128) and ws.numel() <= 64 << 20
    want, err = X.weight_grad(finite(grad, lo, hi), finite(inp, lo, hi), off)
    fl = flag()
    for dtype in (F32, BF16):
        for accumulate in (False, True):
            old = torch.randn((E, M, N), generator=g, device="cuda").to(dtype)
            full = want + P.f64(old) if accumulate else want
            outs = []
            for workspace in (ws, None):
                out = old.clone()
                ep.ep_expert_weight_grad(grad, inp, offset, grad_weight=out, accumulate=accumulate,
                                         workspace=workspace, error_flag=fl)
                outs.append(out)
            assert torch.equal(outs[0], outs[1])
            bound = X.rounded(full, err) if dtype is BF16 else err + 2 * P.U * full.abs()
            X.assert_within(outs[0], full, bound, f"{dtype} accumulate={accumulate}")
    assert fl.item() == 0


def inputs(seed=3, counts=(1500, 0, 3000), M=136, N=72):
    g = gen(seed)
    off, offset = offsets(list(counts), 0)
    return off, offset, rows_of(g, list(counts), 0, 0, M), rows_of(g, list(counts), 0, 0, N)


def test_rows_past_the_capacity_are_skipped():
    off, offset, grad, inp = inputs()
    n = 3700
    fl = flag()
    out = torch.empty((3, 136, 72), device="cuda")
    ep.ep_expert_weight_grad(grad[:n], inp[:n], offset, grad_weight=out, error_flag=fl)
    want, err = X.weight_grad(P.f64(grad[:n]), P.f64(inp[:n]), [0, 1500, 1500, n])
    X.assert_within(out, want, err + 2 * P.U * want.abs(), "grad_weight")
    assert fl.item() != 0


@pytest.mark.parametrize("bad", [[-1, 5, 5, 4500], [0, 5, 4, 4500], [0, 5, 5, 3], [7, 5, 9, 4500]])
def test_offsets_that_make_no_sense_compute_nothing(bad):
    _, _, grad, inp = inputs()
    fl = flag()
    out = torch.full((3, 136, 72), 7.0, device="cuda")
    ep.ep_expert_weight_grad(grad, inp, torch.tensor(bad, dtype=I32, device="cuda"),
                             grad_weight=out, error_flag=fl)
    assert bool((out == 7.0).all()) and fl.item() != 0


def test_a_workspace_that_is_too_small_is_refused():
    _, offset, grad, inp = inputs()
    ws = given(3, grad.shape[0], 136, 72)
    out = torch.full((3, 136, 72), 7.0, device="cuda")
    with pytest.raises(ep.EPError, match="EP_ERR_CAPACITY"):
        ep.ep_expert_weight_grad(grad, inp, offset, grad_weight=out, workspace=ws[:-16])
    with pytest.raises(ep.EPError, match="EP_ERR_ALIGN"):
        ep.ep_expert_weight_grad(grad, inp, offset, grad_weight=out,
                                 workspace=torch.empty(ws.numel() + 16, dtype=U8, device="cuda")[8:])
    assert bool((out == 7.0).all())


def test_streams_and_replays():
    _, offset, grad, inp = inputs()
    other = torch.tensor([0, 10, 2000, 4400], dtype=I32, device="cuda")
    want = []
    for o in (offset, other):
        out = torch.empty((3, 136, 72), device="cuda")
        ep.ep_expert_weight_grad(grad, inp, o, grad_weight=out)
        want.append(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):  # allocated for the call on the call's stream
        outs = [torch.empty((3, 136, 72), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for out in outs:
            ep.ep_expert_weight_grad(grad, inp, offset, grad_weight=out, stream=s)
        side.synchronize()
        assert all(torch.equal(out, want[0]) for out in outs)
    off = offset.clone()
    out = torch.empty((3, 136, 72), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_weight_grad(grad, inp, off, grad_weight=out)
    for i in range(4):
        off.copy_((offset, other)[i % 2])
        out.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i % 2])
