"""The paged cache between prefills on a B200: packed prompts into blocks, their
rows gathered again as the history of a chunked prefill (one request at a time:
``mla_prefill_chunked`` takes one length of history), the chunk's rows appended
behind them; and the plan's positions as rows of the RoPE tables."""
import copy

import numpy as np
import pytest
import torch

import latent_attention_b200 as L
import oracle
from gpu_helpers import TOL, f64
from latent_attention_b200.layer import MlaPagedCache
from mla_inputs import WORKLOADS, make_prefill_inputs
from oracle import paged as O
from test_gpu_guards import _tables, _weights, small_bf16
from test_gpu_paged import i32

pytestmark = pytest.mark.gpu

CONFIGS = {"f32": WORKLOADS["tiny_f32"].cfg, "bf16_yarn": small_bf16(),
           "bf16_direct_q": small_bf16(q_lora_rank=0, rope_type="plain", num_heads=2)}
PROMPTS, CHUNKS = [37, 5, 130, 64], [20, 1, 33, 17]


def part(inp, x):
    """The inputs with the packed rows ``x`` [n, hidden] as one sequence."""
    p = copy.copy(inp)
    p.x, p.B, p.T = x[None], 1, x.shape[0]
    return p


@pytest.mark.parametrize("name", list(CONFIGS))
def test_history_from_blocks_for_a_chunked_prefill(cuda, name):
    cfg = CONFIGS[name]
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    B, bs, H = len(PROMPTS), 16, cfg.hidden_size
    W, r = cfg.kv_lora_rank + cfg.qk_rope_head_dim, cfg.kv_lora_rank
    total, fresh = sum(PROMPTS), sum(CHUNKS)
    inp = make_prefill_inputs(cfg, 1, total + fresh, seed=81)
    x, w = inp.x[0], _weights(inp, cuda)
    cos, sin = _tables(cfg, max(p + c for p, c in zip(PROMPTS, CHUNKS)), cuda)
    pc = MlaPagedCache(cfg, B, max_blocks=12, n_blocks=40, block_size=bs, capacity=total)

    # the prompts, packed; their rows in the order of the plan's slots
    slots, positions, cu = pc.plan(i32(PROMPTS))
    n, _ = L.mla_prefill_varlen_workspace_size(cfg, B, total, max(PROMPTS))
    ws = torch.empty(n, dtype=torch.uint8, device=cuda)
    out = torch.empty(total, H, dtype=dt, device=cuda)
    rows = torch.empty(total, W, dtype=dt, device=cuda)
    L.mla_prefill_varlen(cfg, w, x[:total].to(cuda), cu, B, total, max(PROMPTS), cos, sin, out,
                         ws, latent_cache_out=rows)
    pc.append(rows)
    pc.check_status()
    L.mla_check_device_status(ws)
    assert positions.tolist() == [p for n_ in PROMPTS for p in range(n_)]
    host = (f64(rows), slots.tolist())

    # their rows again, and one chunk each behind them
    history = torch.empty(total, W, dtype=dt, device=cuda)
    past_at = torch.empty(B + 1, dtype=torch.int32, device=cuda)
    pc.gather(history, past_at)
    slots, positions, cu = pc.plan(i32(CHUNKS))
    pc.check_status()
    past_at, cu = past_at.tolist(), cu.tolist()
    cache, scales = O.append(host[0], host[1], np.zeros((40, bs, W), np.uint8), np.ones(40), bs)
    table = pc.table.cpu().numpy()
    for b in range(B):
        assert np.array_equal(f64(history[past_at[b]:past_at[b + 1]]),
                              O.rows_of(cache, scales, table, PROMPTS, b, bs))
    new_rows = torch.empty(fresh, W, dtype=dt, device=cuda)
    for b, (past, new) in enumerate(zip(PROMPTS, CHUNKS)):
        xb = x[total + cu[b]:total + cu[b + 1]]
        hist = history[past_at[b]:past_at[b + 1]]
        n, _ = L.mla_prefill_chunked_workspace_size(cfg, 1, new, past)
        ws = torch.empty(n, dtype=torch.uint8, device=cuda)
        out = torch.empty(1, new, H, dtype=dt, device=cuda)
        L.mla_prefill_chunked(cfg, w, xb[None].to(cuda), 1, new, hist, past, cos, sin, out, ws,
                              latent_cache_out=new_rows[cu[b]:cu[b + 1]])
        L.mla_check_device_status(ws)
        want = oracle.prefill_chunked(cfg, part(inp, xb), hist[None].cpu(), past)
        assert oracle.max_rel_err(out, want) <= TOL[cfg.dtype]
    pc.append(new_rows, slots[:fresh])
    everything = torch.empty(total + fresh, W, dtype=dt, device=cuda)
    at = torch.empty(B + 1, dtype=torch.int32, device=cuda)
    pc.gather(everything, at)
    pc.check_status()
    cache, scales = O.append(f64(new_rows), slots.tolist()[:fresh], cache, scales, bs)
    ctx = [p + c for p, c in zip(PROMPTS, CHUNKS)]
    assert pc.ctx.tolist() == ctx
    want = np.concatenate([O.rows_of(cache, scales, table, ctx, b, bs) for b in range(B)])
    assert np.array_equal(f64(everything), want)

    # a key roped at the plan's positions is the key that the prefill cached
    pos = positions[:fresh].long()
    k = torch.from_numpy(f64(x[total:]) @ f64(inp.w_kv_a).T[:, r:]).to(cuda)
    half = k.shape[1] // 2
    turned = torch.cat([-k[:, half:], k[:, :half]], 1)
    if cfg.rope_type != "none":
        k = k * cos[pos].double() + turned * sin[pos].double()
    assert oracle.max_rel_err(new_rows[:, r:], k.cpu().numpy()) <= TOL[cfg.dtype]
