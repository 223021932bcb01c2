"""One batch through the whole path on the GPU, on one stream, in three forms with the same
outputs:
- the counts path (R <= EP_COUNTS_MAX_RANKS): ep_layout_counts (counts, offsets and the
  restripe in one launch), ep_dispatch_layout (the dispatch computing the receive rows and
  writing the slot table), ep_combine; for a batch of at most
  EP_LAYOUT_DISPATCH_MAX_TOKENS tokens the first two are one call, ep_layout_dispatch;
- the preprocess path: ep_dispatch_preprocess (layout and restripe in one call),
  ep_dispatch, ep_combine;
- one call per step: ep_get_layout, ep_dispatch, ep_restripe_prob, ep_combine.
`step()` takes the one-call layout + dispatch or the counts path where they apply. Also the two-phase ("hook") form of
dispatch and combine, whose send phase returns a callable that enqueues the receive phase
later, and ExpertPath, the expert-major block with the norm in front of it and its gradients.

Device buffers are allocated once per shape (torch, memory plumbing only); the step
functions enqueue their calls and return without synchronising.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import torch

from . import _binding as B
from .buffers import DispatchBuffers, LayoutBuffers, StageBuffers


@dataclasses.dataclass
class DeviceBatch:
    topk_idx: torch.Tensor                 # int64 [T][k]
    topk_weights: torch.Tensor             # fp32 [T][k]
    x: torch.Tensor                        # bf16 [T][H]
    prob: torch.Tensor                     # fp32 [T][N][P]
    partials: Optional[torch.Tensor]       # bf16 [rows][H]; None = combine the dispatched rows

    @classmethod
    def from_host(cls, topk_idx, topk_weights, x_bits, prob, partial_bits=None,
                  device="cuda") -> "DeviceBatch":
        """numpy inputs (bf16 as uint16 bit patterns) copied to the device."""
        import numpy as np

        def bf16(a):
            return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(
                torch.bfloat16).to(device)

        return cls(torch.from_numpy(np.ascontiguousarray(topk_idx)).to(device),
                   torch.from_numpy(np.ascontiguousarray(topk_weights)).to(device),
                   bf16(x_bits), torch.from_numpy(np.ascontiguousarray(prob)).to(device),
                   None if partial_bits is None else bf16(partial_bits))


class Path:
    """Buffers and calls for one shape: T tokens, hidden H, E experts, top-k, R ranks,
    N nodes, P prob floats per (token, node), Tmax rows per node block."""

    def __init__(self, T: int, H: int, E: int, k: int, R: int, N: int, P: int, Tmax: int,
                 device="cuda", recv_capacity: Optional[int] = None, node_slots: bool = False):
        self.T, self.H, self.E, self.k, self.R, self.N, self.P, self.Tmax = T, H, E, k, R, N, P, Tmax
        self.cap = T * min(k, R) if recv_capacity is None else recv_capacity
        self.layout_buf = LayoutBuffers.alloc(T, E, R, N, device, node_slots=node_slots)
        self.recv = DispatchBuffers.alloc(self.cap, H, k, device)
        self.prob_dest_major = torch.empty((N, Tmax, P), dtype=torch.float32, device=device)
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.stage: Optional[StageBuffers] = None
        self._dispatch_pending = False  # a dispatch send whose receive hook has not run
        # The counts path writes no node slots, so a Path that keeps them for the two-phase
        # calls steps on the preprocess path.
        self.counts_path = R <= B.EP_COUNTS_MAX_RANKS and not node_slots
        self.counts_ws: Optional[torch.Tensor] = None  # workspace of the counts path
        if self.counts_path:
            self._counts_workspace()

    @property
    def error_flag(self) -> torch.Tensor:
        return self.layout_buf.error_flag

    def layout(self, b: DeviceBatch, stream=None) -> None:
        self.layout_buf.compute(b.topk_idx, self.E, self.R, self.N, stream=stream)

    def dispatch(self, b: DeviceBatch, stream=None) -> None:
        r = self.recv
        B.ep_dispatch(b.x, b.topk_idx, b.topk_weights, self.E, self.R,
                      self.layout_buf.token_slot, recv_x=r.recv_x, recv_topk_idx=r.recv_topk_idx,
                      recv_topk_weights=r.recv_topk_weights, recv_src_idx=r.recv_src_idx,
                      error_flag=self.error_flag, stream=stream)

    def restripe(self, b: DeviceBatch, stream=None) -> None:
        B.ep_restripe_prob(b.prob, self.prob_dest_major, stream=stream)

    def combine(self, b: DeviceBatch, stream=None) -> None:
        partial = self.recv.recv_x if b.partials is None else b.partials
        B.ep_combine(partial, self.layout_buf.token_slot, out=self.out,
                     error_flag=self.error_flag, stream=stream)

    def preprocess(self, b: DeviceBatch, stream=None) -> None:
        """layout() and restripe() in one call: the restripe's blocks run in the layout's
        first launch (ep_dispatch_preprocess)."""
        self.layout_buf.compute_with_restripe(b.topk_idx, self.E, self.R, self.N, b.prob,
                                              self.prob_dest_major, stream=stream)

    def step(self, b: DeviceBatch, stream=None) -> None:
        """The whole path on one batch: where R allows it and the Path keeps no node slots,
        step_small() for a batch of at most EP_LAYOUT_DISPATCH_MAX_TOKENS tokens and
        step_counts() for a larger one; else step_preprocess()."""
        if self.counts_path and 0 < self.T <= B.EP_LAYOUT_DISPATCH_MAX_TOKENS:
            self.step_small(b, stream)
        elif self.counts_path:
            self.step_counts(b, stream)
        else:
            self.step_preprocess(b, stream)

    def step_small(self, b: DeviceBatch, stream=None) -> None:
        """The same outputs as step_counts() in two launches: ep_layout_dispatch (layout,
        dispatch and restripe), ep_combine. Needs T <= EP_LAYOUT_DISPATCH_MAX_TOKENS and
        R <= EP_COUNTS_MAX_RANKS."""
        self.layout_dispatch(b, stream)
        self.combine(b, stream)

    def layout_dispatch(self, b: DeviceBatch, stream=None) -> None:
        """Layout, dispatch and restripe of a batch of at most EP_LAYOUT_DISPATCH_MAX_TOKENS
        tokens in one launch."""
        lb, r = self.layout_buf, self.recv
        B.ep_layout_dispatch(b.x, b.topk_idx, b.topk_weights, self.E, self.R, self.N,
                             token_slot=lb.token_slot, recv_x=r.recv_x,
                             num_tokens_per_rank=lb.num_tokens_per_rank,
                             rank_offset=lb.rank_offset, error_flag=self.error_flag,
                             is_token_in_rank=lb.is_token_in_rank,
                             num_tokens_per_node=lb.num_tokens_per_node,
                             num_tokens_per_expert=lb.num_tokens_per_expert,
                             expert_offset=lb.expert_offset, recv_topk_idx=r.recv_topk_idx,
                             recv_topk_weights=r.recv_topk_weights,
                             recv_src_idx=r.recv_src_idx, prob=b.prob,
                             prob_dest_major=self.prob_dest_major, stream=stream)

    def step_preprocess(self, b: DeviceBatch, stream=None) -> None:
        """Layout and restripe (one call), dispatch, combine."""
        self.preprocess(b, stream)
        self.dispatch(b, stream)
        self.combine(b, stream)

    def _counts_workspace(self) -> torch.Tensor:
        if self.counts_ws is None:
            if self.R > B.EP_COUNTS_MAX_RANKS:
                raise ValueError(f"the counts path needs num_ranks <= {B.EP_COUNTS_MAX_RANKS}")
            n = B.ep_layout_counts_workspace_bytes(self.T, self.E, self.R, self.N)
            # zero-filled once: every call leaves the ticket at the start zero again
            self.counts_ws = torch.zeros(max(16, n), dtype=torch.uint8, device=self.out.device)
        return self.counts_ws

    def step_counts(self, b: DeviceBatch, stream=None) -> None:
        """The same outputs as step_preprocess() in one launch less: ep_layout_counts
        (counts, and the restripe in the same launch), ep_dispatch_layout (the dispatch
        computing every receive row itself, writing token_slot and the bitmap),
        ep_combine. Needs R <= EP_COUNTS_MAX_RANKS."""
        self.layout_counts(b, stream)
        self.dispatch_layout(b, stream)
        self.combine(b, stream)

    def layout_counts(self, b: DeviceBatch, stream=None) -> None:
        """The counts path's first call: the per-block tables in the workspace, and the
        restripe in the same launch."""
        B.ep_layout_counts(b.topk_idx, self.E, self.R, self.N, error_flag=self.error_flag,
                           workspace=self._counts_workspace(), prob=b.prob,
                           prob_dest_major=self.prob_dest_major, stream=stream)

    def dispatch_layout(self, b: DeviceBatch, stream=None) -> None:
        """The counts path's dispatch, after layout_counts() on the same batch."""
        ws, lb, r = self._counts_workspace(), self.layout_buf, self.recv
        B.ep_dispatch_layout(b.x, b.topk_idx, b.topk_weights, self.E, self.R, self.N,
                             token_slot=lb.token_slot, is_token_in_rank=lb.is_token_in_rank,
                             num_tokens_per_rank=lb.num_tokens_per_rank,
                             rank_offset=lb.rank_offset,
                             num_tokens_per_node=lb.num_tokens_per_node,
                             num_tokens_per_expert=lb.num_tokens_per_expert,
                             expert_offset=lb.expert_offset,
                             recv_x=r.recv_x, recv_topk_idx=r.recv_topk_idx,
                             recv_topk_weights=r.recv_topk_weights, recv_src_idx=r.recv_src_idx,
                             error_flag=self.error_flag, workspace=ws, stream=stream)

    def step_separate(self, b: DeviceBatch, stream=None) -> None:
        """The same outputs as step_preprocess(), one call per step of the path."""
        self.layout(b, stream)
        self.dispatch(b, stream)
        self.restripe(b, stream)
        self.combine(b, stream)

    # --- two-phase ("hook") dispatch and combine -----------------------------------------

    def _hook_buffers(self) -> StageBuffers:
        if self.stage is None:
            self.stage = StageBuffers.alloc(self.N, self.Tmax, self.H, self.k,
                                            self.out.device)
        if self.layout_buf.node_slot is None:
            raise ValueError("the two-phase calls need node slots: build the Path with "
                             "node_slots=True and run layout() first")
        return self.stage

    def dispatch_send(self, b: DeviceBatch, stream=None, num_workgroups: int = 0):
        """Enqueue the send phase; returns the receive hook, a callable(stream=None) that
        enqueues the receive phase (on a stream ordered after this one). num_workgroups > 0
        bounds the workgroups the send occupies (room for compute on another queue)."""
        st, lb = self._hook_buffers(), self.layout_buf
        B.ep_dispatch_send(b.x, b.topk_idx, b.topk_weights, lb.node_slot, stage_x=st.stage_x,
                           stage_topk_idx=st.stage_topk_idx,
                           stage_topk_weights=st.stage_topk_weights, stage_src=st.stage_src,
                           error_flag=self.error_flag, num_workgroups=num_workgroups,
                           stream=stream)

        self._dispatch_pending = True

        def recv_hook(stream=None) -> None:
            self._dispatch_pending = False
            r = self.recv
            B.ep_dispatch_recv(st.stage_x, st.stage_topk_idx, st.stage_topk_weights,
                               st.stage_src, lb.num_tokens_per_node, self.E, self.R,
                               lb.token_slot, recv_x=r.recv_x, recv_topk_idx=r.recv_topk_idx,
                               recv_topk_weights=r.recv_topk_weights,
                               recv_src_idx=r.recv_src_idx, error_flag=self.error_flag,
                               stream=stream)
        return recv_hook

    def combine_send(self, b: DeviceBatch, stream=None, num_workgroups: int = 0):
        """Enqueue the combine's send phase (per-node sums); returns its receive hook.
        The sums reuse the dispatch's staging rows, so a pending dispatch receive hook
        must have been enqueued first."""
        if self._dispatch_pending:
            raise RuntimeError("combine_send would overwrite the staged dispatch rows: run the "
                               "dispatch receive hook first")
        st, lb = self._hook_buffers(), self.layout_buf
        partial = self.recv.recv_x if b.partials is None else b.partials
        B.ep_combine_send(partial, lb.token_slot, lb.node_slot, stage=st.stage_x,
                          error_flag=self.error_flag, num_workgroups=num_workgroups,
                          stream=stream)

        def recv_hook(stream=None) -> None:
            B.ep_combine_recv(st.stage_x, lb.node_slot, out=self.out, error_flag=self.error_flag,
                              stream=stream)
        return recv_hook


class ExpertPath:
    """The expert-major block on one GPU: buffers and calls for T tokens of H channels over E
    experts, top-k (k <= EP_EXPERT_SLOT_MAX_K; H a multiple of 128 with fp8=True).

        norm(x, weight, residual)        ep_rmsnorm: residual_out, y (and e4m3 with fp8=True)
        dispatch(topk_idx)               ep_get_layout with expert slots, then
                                         ep_dispatch_permute, or with fp8=True
                                         ep_dispatch_permute_fp8, of the norm's output
        ... the caller's experts on rows expert_offset[e] .. expert_offset[e + 1] - 1 of
            perm_x (perm_x_fp8 and perm_scales with fp8=True) ...
        combine(expert_out, topk_weights, addend)   ep_combine_unpermute: out

    and with training=True, in reverse,

        combine_grad(grad_out, expert_out, topk_weights)  grad_expert_out, grad_topk_weights
        dispatch_grad(grad_perm_x, addend=...)            grad_y
        norm_grad(weight, grad_residual_out)              grad_x, grad_weight

    The gate weights are applied once, by combine(), so their gradient is combine_grad()'s.
    y feeds more than the dispatch: the router that the gate weights come from, and a shared
    expert where there is one. The caller takes grad_topk_weights back through the router and
    grad_out (combine()'s addend's gradient) back through the shared expert, and gives
    dispatch_grad() the sum of both as its addend; without them grad_y, and with it grad_x and
    grad_weight, is the expert rows' share alone.
    h is what the norm was taken of as the backward reads it: residual_out, or x itself without
    a residual. That x has to keep its rows until norm_grad(); where it is one of the path's
    own buffers (p.norm(p.out, ...) in a chain) and a call has written over it, norm_grad()
    refuses. Rows of perm_x behind the last routed pair are left as they were."""

    def __init__(self, T: int, H: int, E: int, k: int, *, R: int = 1, N: int = 1,
                 eps: float = 1e-6, fp8: bool = False, training: bool = False, device="cuda"):
        self.T, self.H, self.E, self.k, self.R, self.N, self.eps = T, H, E, k, R, N, eps
        self.fp8, self.training = fp8, training
        bf16 = dict(dtype=torch.bfloat16, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        u8 = dict(dtype=torch.uint8, device=device)
        cap = T * k
        self.layout_buf = LayoutBuffers.alloc(T, E, R, N, device, k_expert_slots=k)
        self.residual_out = torch.empty((T, H), **bf16)
        self.y = torch.empty((T, H), **bf16)
        self.out = torch.empty((T, H), **bf16)
        self.perm_src_idx = torch.empty(cap, dtype=torch.int32, device=device)
        self.h: Optional[torch.Tensor] = None  # set by norm()
        self._h_overwritten_by = ""
        if fp8:
            self.y_fp8 = torch.empty((T, H), **u8)
            self.y_scales = torch.empty((T, H // 128), **f32)
            self.perm_x_fp8 = torch.empty((cap, H), **u8)
            self.perm_scales = torch.empty((cap, H // 128), **f32)
        else:
            self.perm_x = torch.empty((cap, H), **bf16)
        if training:
            self.grad_expert_out = torch.empty((cap, H), **bf16)
            self.grad_topk_weights = torch.empty((T, k), **f32)
            self.grad_y = torch.empty((T, H), **bf16)
            self.grad_x = torch.empty((T, H), **bf16)
            self.grad_weight = torch.empty(H, **f32)
            ws = max(16, B.ep_rmsnorm_grad_workspace_bytes(T, H))
            self.norm_workspace = torch.empty(ws, **u8)

    @property
    def error_flag(self) -> torch.Tensor:
        return self.layout_buf.error_flag

    @property
    def expert_offset(self) -> torch.Tensor:
        return self.layout_buf.expert_offset

    def norm(self, x, weight, residual=None, stream=None) -> None:
        with_sum = residual is not None
        B.ep_rmsnorm(x, weight, residual=residual,
                     residual_out=self.residual_out if with_sum else None, y=self.y,
                     y_fp8=self.y_fp8 if self.fp8 else None,
                     y_scales=self.y_scales if self.fp8 else None, eps=self.eps, stream=stream)
        self.h = self.residual_out if with_sum else x
        self._wrote(self.y, "norm")

    def _wrote(self, buffer, call: str) -> None:
        """A call has written `buffer`: h is gone if it lies there."""
        h = self.h
        if not self.training or h is None or h is self.residual_out:
            return
        at, by = h.data_ptr(), buffer.data_ptr()
        if at < by + buffer.numel() * buffer.element_size() and by < at + h.numel() * h.element_size():
            self.h, self._h_overwritten_by = None, call

    def dispatch(self, topk_idx, stream=None) -> None:
        """The layout of the batch and the norm's rows in expert-major order."""
        lb = self.layout_buf
        lb.compute(topk_idx, self.E, self.R, self.N, stream=stream)
        if self.fp8:
            B.ep_dispatch_permute_fp8(self.y_fp8, self.y_scales, None, lb.expert_slot,
                                      perm_x_fp8=self.perm_x_fp8, perm_scales=self.perm_scales,
                                      perm_src_idx=self.perm_src_idx,
                                      error_flag=self.error_flag, stream=stream)
        else:
            B.ep_dispatch_permute(self.y, None, lb.expert_slot, perm_x=self.perm_x,
                                  perm_src_idx=self.perm_src_idx, error_flag=self.error_flag,
                                  stream=stream)
            self._wrote(self.perm_x, "dispatch")

    def combine(self, expert_out, topk_weights, addend=None, stream=None) -> None:
        B.ep_combine_unpermute(expert_out, topk_weights, self.layout_buf.expert_slot,
                               out=self.out, addend=addend, error_flag=self.error_flag,
                               stream=stream)
        self._wrote(self.out, "combine")

    def _needs_training(self) -> None:
        if not self.training:
            raise ValueError("the gradients need an ExpertPath built with training=True")

    def combine_grad(self, grad_out, expert_out, topk_weights, stream=None) -> None:
        self._needs_training()
        B.ep_combine_unpermute_grad(grad_out, expert_out, topk_weights,
                                    self.layout_buf.expert_slot,
                                    grad_expert_out=self.grad_expert_out,
                                    grad_topk_weights=self.grad_topk_weights,
                                    error_flag=self.error_flag, stream=stream)
        self._wrote(self.grad_expert_out, "combine_grad")

    def dispatch_grad(self, grad_perm_x, stream=None, *, addend=None) -> None:
        """grad_y = the sum of each token's routed rows of grad_perm_x, + addend (bf16 [T][H]:
        what reaches y through the router and a shared expert; may be grad_y itself), in fp32
        and rounded once. It is the sum that ep_combine_unpermute makes with every weight 1."""
        self._needs_training()
        if addend is not None:
            B.ep_combine_unpermute(grad_perm_x, None, self.layout_buf.expert_slot,
                                   out=self.grad_y, addend=addend, error_flag=self.error_flag,
                                   stream=stream)
        else:
            B.ep_dispatch_permute_grad(grad_perm_x, self.layout_buf.expert_slot,
                                       grad_x=self.grad_y, error_flag=self.error_flag,
                                       stream=stream)
        self._wrote(self.grad_y, "dispatch_grad")

    def norm_grad(self, weight, grad_residual_out=None, stream=None) -> None:
        self._needs_training()
        if self.h is None and self._h_overwritten_by:
            raise ValueError(f"norm_grad needs the rows that norm() was taken of, and "
                             f"{self._h_overwritten_by}() has written over them: give norm() a copy")
        if self.h is None:
            raise ValueError("norm_grad needs norm() first")
        B.ep_rmsnorm_grad(self.grad_y, self.h, weight, grad_x=self.grad_x,
                          grad_residual_out=grad_residual_out, grad_weight=self.grad_weight,
                          workspace=self.norm_workspace, eps=self.eps, stream=stream)
        self._wrote(self.grad_x, "norm_grad")
