"""What ExpertPath keeps from norm() for norm_grad(), on the CPU: the library's calls are
stand-ins that do nothing."""
import pytest
import torch

from combine_ep_get_03_amd import pipeline

T, H, E, K = 4, 256, 16, 2
CALLS = ("ep_rmsnorm", "ep_rmsnorm_grad", "ep_get_layout", "ep_dispatch_permute",
         "ep_dispatch_permute_grad", "ep_combine_unpermute", "ep_combine_unpermute_grad")


@pytest.fixture
def made(monkeypatch):
    seen = []
    for name in CALLS:
        monkeypatch.setattr(pipeline.B, name, lambda *a, _n=name, **kw: seen.append((_n, a)))
    return seen


def path(**kw):
    return pipeline.ExpertPath(T, H, E, K, device="cpu", **{"training": True, **kw})


W = torch.ones(H)
GATE = torch.ones((T, K))
IDX = torch.zeros((T, K), dtype=torch.int64)


def rows(n=T):
    return torch.zeros((n, H), dtype=torch.bfloat16)


# which of the path's own buffers is x, and the call that writes it
@pytest.mark.parametrize("own,call,by", [
    (lambda p: p.y, lambda p: None, "norm"),
    (lambda p: p.perm_x[:T], lambda p: p.dispatch(IDX), "dispatch"),
    (lambda p: p.perm_x[T:], lambda p: p.dispatch(IDX), "dispatch"),
    (lambda p: p.out, lambda p: p.combine(rows(T * K), GATE), "combine"),
    (lambda p: p.grad_expert_out[1:T + 1], lambda p: p.combine_grad(rows(), rows(T * K), GATE),
     "combine_grad"),
    (lambda p: p.grad_y, lambda p: p.dispatch_grad(rows(T * K)), "dispatch_grad"),
    (lambda p: p.grad_y, lambda p: p.dispatch_grad(rows(T * K), addend=rows()), "dispatch_grad"),
    (lambda p: p.grad_x, lambda p: p.norm_grad(W), "norm_grad"),
])
def test_rows_that_a_call_has_written_over_are_not_used(made, own, call, by):
    p = path()
    x = own(p)
    p.norm(x, W)
    call(p)
    before = len(made)
    with pytest.raises(ValueError, match=rf"{by}\(\) has written over them"):
        p.norm_grad(W)
    assert len(made) == before
    p.norm(rows(), W)  # a new forward pass puts it right
    p.norm_grad(W)


def test_rows_that_nothing_writes_are_used(made):
    """x apart from the path's buffers, the sum with a residual whatever x and the residual are,
    and a buffer that is written only after norm_grad() has read it."""
    p = path()
    x = rows()

    def block():
        p.dispatch(IDX)
        p.combine(p.perm_x, GATE)
        p.combine_grad(rows(), p.perm_x, GATE)
        p.dispatch_grad(p.grad_expert_out)

    for y, res, h in ((x, None, x), (p.out, x, p.residual_out), (p.y, p.residual_out, p.residual_out),
                      (p.grad_x, None, p.grad_x), (p.residual_out, None, p.residual_out)):
        p.norm(y, W, res)
        assert p.h is h
        block()
        p.norm_grad(W)
        assert made[-1][0] == "ep_rmsnorm_grad" and made[-1][1][1] is h
    p.norm(p.out, W)
    p.norm_grad(W)  # out is as it was
    with pytest.raises(ValueError, match="norm\\(\\) first"):
        path().norm_grad(W)


def test_a_path_without_gradients_chains_on_its_own_output(made):
    for p in (path(training=False), path()):
        for _ in range(3):
            p.norm(p.out, W)
            p.dispatch(IDX)
            p.combine(p.perm_x, GATE)
