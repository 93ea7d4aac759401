"""Convenience wrappers: plan once, upload once, run many times."""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import _lib


class SplitKVAttention:
    """Split-KV attention for one batch layout.

    Builds the plan (``splitkv_plan``), allocates and fills the workspace
    (``splitkv_plan_upload``) and then runs the fused path (``splitkv_decode``)
    or the two-stage path (``splitkv_partial`` + ``merge_states``).  The plan
    and workspace are reusable for every layer that shares the batch lengths.
    """

    def __init__(self, problem: _lib.AttentionProblem, params: Optional[_lib.PlanParams] = None,
                 stream=None):
        self.problem = problem
        self.plan = _lib.splitkv_plan(problem, params)
        dev = problem.q.device
        self.workspace = _lib.alloc_workspace(self.plan, dev)
        self.state_indptr = torch.from_numpy(self.plan.state_indptr()).to(dev)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=dev)
        _lib.splitkv_plan_upload(self.plan, self.workspace, stream)

    def out_like(self):
        p = self.problem
        dt = torch.bfloat16 if p.dtype == _lib.BF16 else torch.float32
        out = torch.empty(p.total_q, p.num_q_heads, p.head_dim_v, dtype=dt, device=p.q.device)
        lse = torch.empty(p.total_q, p.num_q_heads, dtype=torch.float32, device=p.q.device)
        return out, lse

    def decode(self, out=None, lse=None, stream=None):
        if out is None:
            out, lse = self.out_like()
        _lib.splitkv_decode(self.problem, self.plan, self.workspace, out, lse, self.error_word, stream)
        return out, lse

    def partial(self, stream=None):
        dev = self.problem.q.device
        o_part = torch.empty(max(1, self.plan.num_states), self.problem.head_dim_v, dtype=self.plan.partial_dtype,
                             device=dev)
        lse_part = torch.empty(max(1, self.plan.num_states), dtype=torch.float32, device=dev)
        _lib.splitkv_partial(self.problem, self.plan, self.workspace, o_part, lse_part, self.error_word, stream)
        return o_part, lse_part

    def two_stage(self, out=None, lse=None, stream=None):
        o_part, lse_part = self.partial(stream)
        if out is None:
            out, lse = self.out_like()
        _lib.merge_states(o_part, lse_part, self.state_indptr, out.view(-1, self.problem.head_dim_v),
                          lse.view(-1) if lse is not None else None, stream)
        return out, lse

    def check_device_error(self, clear: bool = True):
        st, raw = _lib.read_device_error(self.error_word, None, clear)
        if st != _lib.OK:
            raise _lib.SplitKVError(st, f"device error word 0x{raw:x}")


class LatentAttention:
    """Latent (MLA) attention from the model's own queries, for one batch layout.

    ``k_cache`` [num_pages, P, 576] holds the latent rows (bfloat16, or uint8 E4M3
    codes with ``k_scale``), ``w_kv_b`` [H, 256, 512] each head's key and value
    up-projections.  Calling it with q [total_q, H, 192] gives out [total_q, H,
    128]: row i of a request attends keys 0 .. seq_len - q_len + i.

    ``form``: "expanded" computes every head's keys and values first (prompts,
    chunks), "absorbed" attends the latent rows themselves (decode), "auto" takes
    the one that the lengths make cheaper: one form for the whole batch, so prompts and
    decoding requests go into batches of their own.  ``params`` plans the absorbed form.
    The plan and workspace are reusable for every layer that shares the lengths;
    ``w_kv_b`` may be replaced between calls (attribute of the same name).  Calls
    of one object share its buffers: order them on one stream.
    """

    def __init__(self, *, k_cache: torch.Tensor, w_kv_b: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                 qo_indptr: torch.Tensor, scale: float, form: str = "auto", seq_lens_host: Optional[Sequence[int]] = None,
                 qo_indptr_host: Optional[Sequence[int]] = None, k_scale: Optional[float] = None,
                 params: Optional[_lib.PlanParams] = None, stream=None):
        if form not in ("auto", "expanded", "absorbed"):
            raise ValueError(f"form {form!r} is not auto, expanded or absorbed")
        if k_cache.dim() != 3 or k_cache.shape[2] != 576:
            raise TypeError("k_cache must be [num_pages, page_size, 576]")
        if k_cache.dtype not in (torch.bfloat16, torch.uint8):
            raise TypeError(f"unsupported cache dtype {k_cache.dtype}")
        heads, dev = int(w_kv_b.shape[0]), k_cache.device
        if qo_indptr_host is None:
            qo_indptr_host = qo_indptr.cpu().numpy()
        total = int(qo_indptr_host[-1])
        self.w_kv_b = w_kv_b
        make = lambda q: _lib.AttentionProblem(  # noqa: E731
            q=q, k_cache=k_cache, v_cache=None, page_table=page_table, seq_lens=seq_lens, qo_indptr=qo_indptr,
            num_q_heads=heads, num_kv_heads=1, head_dim_qk=576, head_dim_v=512, page_size=int(k_cache.shape[1]), scale=scale,
            kind="mla", seq_lens_host=seq_lens_host, qo_indptr_host=qo_indptr_host, k_scale=k_scale,
            v_scale=None if k_scale is None else 1.0)
        self.problem = make(torch.empty(0, dtype=torch.bfloat16, device=dev))
        if form == "auto":
            form = "expanded" if _lib.latent_prefers_expanded(self.problem) else "absorbed"
        self.form = form
        if form == "expanded":
            self.plan = _lib.LatentPlan(self.problem)
            self.workspace = _lib.alloc_workspace(self.plan, dev)
            self.error_word = torch.zeros(1, dtype=torch.int32, device=dev)
            _lib.latent_upload(self.plan, self.workspace, stream)
        else:
            self.q_abs = torch.empty(total, heads, 576, dtype=torch.bfloat16, device=dev)
            self.problem = make(self.q_abs)
            if params is None:
                # the kernel attends 128 keys (two pages) at a time: splits of less waste its products
                units = -(-int(self.problem.seq_lens_host.max()) // 128)
                params = _lib.plan_params(max_splits=max(1, min(64, units)))
            base = SplitKVAttention(self.problem, params, stream)
            self.plan, self.workspace, self.error_word = base.plan, base.workspace, base.error_word
            self.state_indptr = base.state_indptr
            states = max(1, self.plan.num_states)
            self.o_part = torch.empty(states, 512, dtype=self.plan.partial_dtype, device=dev)
            self.lse_part = torch.empty(states, dtype=torch.float32, device=dev)

    def __call__(self, q: torch.Tensor, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None):
        """out [total_q, H, 128] bfloat16 (allocated when None); lse [total_q, H] float32, written when given."""
        p = self.problem
        if out is None:
            out = torch.empty(p.total_q, p.num_q_heads, 128, dtype=torch.bfloat16, device=p.k_cache.device)
        layer = _lib.latent_layer(p, q, self.w_kv_b, out, lse)
        if p.total_q == 0:
            return out
        if self.form == "expanded":
            _lib.latent_expanded(p, self.plan, layer, self.workspace, self.error_word, stream)
        else:
            _lib.latent_absorb_query(p, layer, self.q_abs, self.error_word, stream)
            _lib.splitkv_partial(p, self.plan, self.workspace, self.o_part, self.lse_part, self.error_word, stream)
            _lib.latent_project(p, layer, self.o_part, self.lse_part, self.state_indptr, self.error_word, stream)
        return out

    def check_device_error(self, clear: bool = True):
        st, raw = _lib.read_device_error(self.error_word, None, clear)
        if st != _lib.OK:
            raise _lib.SplitKVError(st, f"device error word 0x{raw:x}")
