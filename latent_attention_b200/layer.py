"""Convenience holders that keep device buffers for repeated calls.

``MlaPrefill`` and ``MlaDecode`` own the device copies of the weights, the
RoPE tables and the workspace (torch allocations), ``MlaPagedCache`` owns the
paged latent cache and its tables; they call the C ABI and do no arithmetic of
their own.
"""
import torch

from . import (MlaError, make_config, mla_build_rope_tables, mla_prefill_workspace_size,
               mla_prefill_forward, mla_decode_workspace_size,
               mla_decode_absorbed, mla_check_device_status,
               mla_paged_workspace_size, mla_paged_plan, mla_paged_append,
               mla_paged_gather, mla_decode_paged_workspace_size,
               mla_decode_paged)

_WEIGHT_KEYS = ("w_q_a", "g_q_a", "w_q_b", "w_q", "w_kv_a", "g_kv_a", "w_kv_b",
                "w_o")
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class MlaPrefill:
    def __init__(self, cfg, weights, B, T, device="cuda", max_pos=None):
        self.cfg, self.B, self.T = cfg, B, T
        self.c = make_config(cfg)
        self.dtype = _DT[cfg.dtype]
        self.device = torch.device(device)
        self.w = {}
        for k in _WEIGHT_KEYS:
            t = weights.get(k) if isinstance(weights, dict) else getattr(weights, k)
            self.w[k] = None if t is None else t.to(self.device).contiguous()
        d = cfg.qk_rope_head_dim
        mp = max_pos or T
        self.cos = torch.empty(mp, d, dtype=torch.float32, device=self.device)
        self.sin = torch.empty_like(self.cos)
        mla_build_rope_tables(self.c, mp, self.cos, self.sin)
        n, self.layout = mla_prefill_workspace_size(self.c, B, T)
        self.ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        self.out = torch.empty(B, T, cfg.hidden_size, dtype=self.dtype,
                               device=self.device)

    def __call__(self, x, out=None, latent_cache_out=None, stream=None):
        out = self.out if out is None else out
        mla_prefill_forward(self.c, self.w, x, self.B, self.T, self.cos,
                            self.sin, out, self.ws, latent_cache_out, stream)
        return out

    def view(self, name, shape, dtype=None):
        """A tensor view of a workspace intermediate (see mla_prefill_layout)."""
        off = self.layout[name]
        if off < 0:
            return None
        dt = dtype or self.dtype
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        return self.ws[off:off + nbytes].view(dt).view(*shape)

    def check_status(self, stream=None):
        mla_check_device_status(self.ws, stream)


class MlaDecode:
    def __init__(self, cfg, B, max_ctx, device="cuda"):
        self.cfg, self.B, self.max_ctx = cfg, B, max_ctx
        self.c = make_config(cfg)
        self.dtype = _DT[cfg.dtype]
        self.device = torch.device(device)
        n, self.layout = mla_decode_workspace_size(self.c, B, max_ctx)
        self.ws = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, q_nope, q_pe, w_kv_b, cache, cu_ctx, out, w_o=None,
                 stream=None):
        mla_decode_absorbed(self.c, q_nope, q_pe, w_kv_b, cache, cu_ctx,
                            self.B, self.max_ctx, w_o, out, self.ws, stream)
        return out

    def check_status(self, stream=None):
        mla_check_device_status(self.ws, stream)


class MlaPagedCache:
    """The paged 8-bit latent cache of up to ``max_requests`` requests of
    ``max_blocks`` blocks each: the pool, the block tables, the free ring and
    the lengths, all on the device.  One serving step is ``plan`` (blocks and
    slots of the new tokens), ``append`` (their latent rows) and ``decode`` or
    ``gather``; nothing in it waits for the device, so a step can be captured
    into a CUDA graph.  Each of the four has a workspace of its own, because a
    call starts its workspace's status afresh: what a plan reported is still
    there when ``check_status`` reads it at the step's end."""

    def __init__(self, cfg, max_requests, max_blocks, n_blocks, block_size=64, capacity=None,
                 device="cuda"):
        self.cfg, self.B, self.max_blocks = cfg, max_requests, max_blocks
        self.n_blocks, self.block_size = n_blocks, block_size
        self.capacity = max_requests if capacity is None else capacity
        self.c = make_config(cfg)
        self.dtype = _DT[cfg.dtype]
        self.device = torch.device(device)
        self.width = cfg.kv_lora_rank + cfg.qk_rope_head_dim
        i32 = dict(dtype=torch.int32, device=self.device)
        self.cache = torch.zeros(n_blocks, block_size, self.width, dtype=torch.float8_e4m3fn,
                                 device=self.device)
        self.scales = torch.ones(n_blocks, dtype=torch.float32, device=self.device)
        self.table = torch.full((max_requests, max_blocks), -1, **i32)
        self.ring = torch.arange(n_blocks, **i32)
        self.state = torch.tensor([0, n_blocks], **i32)
        self.ctx = torch.zeros(max_requests, **i32)
        self.slots = torch.empty(self.capacity, **i32)
        self.positions = torch.empty(self.capacity, **i32)
        self.cu_new = torch.empty(max_requests + 1, **i32)
        n = mla_paged_workspace_size(n_blocks)
        self.plan_ws, self.ws, self.gather_ws = (
            torch.empty(n, dtype=torch.uint8, device=self.device) for _ in range(3))
        n, self.layout = mla_decode_paged_workspace_size(self.c, max_requests, max_blocks,
                                                         block_size)
        self.decode_ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        for ws in (self.plan_ws, self.ws, self.gather_ws, self.decode_ws):
            ws[:256].zero_()           # MLA_OK until a call leaves its own status

    def plan(self, new_len, stream=None):
        """Blocks and slots of ``new_len`` [B] tokens (int32; -1: the request
        leaves).  Returns the slot map, the positions and their prefix sums."""
        mla_paged_plan(self.ctx, new_len, self.table, self.ring, self.state, self.ctx, self.state,
                       self.slots, self.positions, self.cu_new, self.B, self.max_blocks,
                       self.n_blocks, self.block_size, self.capacity, self.plan_ws,
                       stream)
        return self.slots, self.positions, self.cu_new

    def append(self, rows, slots=None, stream=None):
        """Quantise ``rows`` [n, W] into the planned slots."""
        mla_paged_append(self.c, rows, self.slots if slots is None else slots, self.cache,
                         self.scales, rows.shape[0], self.n_blocks, self.block_size, self.ws,
                         stream)

    def gather(self, rows_out, cu_ctx, stream=None):
        mla_paged_gather(self.c, self.cache, self.scales, self.table, self.ctx, rows_out, cu_ctx,
                         self.B, self.max_blocks, self.n_blocks, self.block_size,
                         rows_out.shape[0], self.gather_ws, stream)
        return rows_out, cu_ctx

    def decode(self, q_nope, q_pe, w_kv_b, out, w_o=None, stream=None):
        mla_decode_paged(self.c, q_nope, q_pe, w_kv_b, self.cache, self.scales, self.table,
                         self.ctx, self.B, self.max_blocks, self.n_blocks, self.block_size, w_o,
                         out, self.decode_ws, stream)
        return out

    def check_status(self, stream=None):
        """The statuses of the last plan, append, gather and decode: all are read
        and cleared, and the first of them that is not MLA_OK is raised.  A plan
        that failed has done nothing, so the append behind it wrote no row and the
        decode saw the old lengths."""
        failed = None
        for ws in (self.plan_ws, self.ws, self.gather_ws, self.decode_ws):
            try:
                mla_check_device_status(ws, stream)
            except MlaError as e:
                failed = failed or e
        if failed:
            raise failed
