"""What ExpertPath keeps from experts() for experts_grad(), on the CPU: the library's calls are
stand-ins that do nothing."""
import pytest
import torch

from combine_ep_get_03_amd import pipeline

T, H, E, K, I = 4, 128, 2, 1, 128
CALLS = ("ep_get_layout", "ep_dispatch_permute", "ep_dispatch_permute_fp8", "ep_combine_unpermute",
         "ep_combine_unpermute_grad", "ep_expert_gate_up", "ep_expert_down", "ep_expert_down_grad",
         "ep_expert_gate_up_grad", "ep_expert_weight_grad", "ep_expert_gate_up_fp8", "ep_expert_down_fp8")
IDX = torch.zeros((T, K), dtype=torch.int64)
GATE = torch.ones((T, K))
ROWS = torch.zeros((T, H), dtype=torch.bfloat16)
W = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16), torch.zeros((E, H, I), dtype=torch.bfloat16)


@pytest.fixture
def seen(monkeypatch):
    names = []
    for name in CALLS:
        monkeypatch.setattr(pipeline.B, name, lambda *a, _n=name, **kw: names.append(_n))
    return names


def path(**kw):
    return pipeline.ExpertPath(T, H, E, K, device="cpu", **{"training": True, "inter": I, **kw})


def step(p):
    p.dispatch(IDX)
    p.experts(*W)
    p.combine(p.expert_out, GATE)
    p.combine_grad(ROWS, p.expert_out, GATE)


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
def test_what_another_batch_has_kept_is_not_used(seen, checkpoint):
    """dispatch() brings new offsets and rows: gate, up and act of the batch before do not go with
    them, and the caller's own products keep nothing."""
    p = path(checkpoint=checkpoint)
    for _ in range(2):
        step(p)
        p.experts_grad(*W)
        p.experts_grad(*W, accumulate=True)  # what is kept of a batch stays until the next one
        p.dispatch(IDX)
        p.combine_grad(ROWS, ROWS, GATE)
        before = len(seen)
        with pytest.raises(ValueError, match="experts\\(\\) first"):
            p.experts_grad(*W)
        assert len(seen) == before


def test_act_is_shared_only_where_it_is_made_again(seen):
    """With checkpoint="fp8" the backward makes act again, and without training nothing reads it
    later; with checkpoint="bf16" it is what w_down's gradient is taken of."""
    for kw in (dict(checkpoint="fp8"), dict(training=False), dict(training=False, checkpoint="fp8")):
        p, q = path(**kw), path(**kw)
        p.act = q.act
        assert p.act is q.act
        step(p) if p.training else p.experts(*W)
    p, q = path(), path()
    mine = p.act
    with pytest.raises(ValueError, match="act"):
        p.act = q.act
    assert p.act is mine and p.act.shape == (T * K, I)
    step(p)
    p.experts_grad(*W)
