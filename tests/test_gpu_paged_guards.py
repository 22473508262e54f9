"""Out-of-bounds writes of the paged operators, caught without a sanitizer: every
buffer that a call may write lies between guard regions that must hold their
pattern bit for bit afterwards, at sizes with ragged tails; and none of the calls
allocates device memory."""
import numpy as np
import pytest
import torch

import latent_attention_b200 as L
import oracle
from gpu_helpers import TOL, f64
from oracle import paged as O
from test_gpu_guards import Guarded
from test_gpu_paged import (F32, bf16, check_plan, decode_inputs, dirty_pool, i32, make_tables,
                            pool_state, random_rows, slots_for, want_decode, width)

pytestmark = pytest.mark.gpu


def guarded(values, dtype, dev):
    """A guarded copy of ``values``."""
    v = torch.as_tensor(np.asarray(values)).to(dtype)
    g = Guarded(tuple(v.shape), dtype, dev, 0x5A if dtype != torch.float32 else 7.25)
    g.t.copy_(v)
    return g


def blank(shape, dtype, dev):
    return Guarded(shape, dtype, dev, float("nan") if dtype.is_floating_point else 0x5A)


def all_intact(*gs):
    torch.cuda.synchronize()
    return all(g.guards_intact() for g in gs)


def paged_ws(n_blocks, dev):
    return Guarded((L.mla_paged_workspace_size(n_blocks),), torch.uint8, dev, 0xA5)


@pytest.mark.parametrize("B,bs,hi_ctx,hi_new,leave", [
    (1, 16, 0, 1, 0), (31, 32, 900, 40, .3), (33, 16, 100, 300, .1), (257, 64, 3000, 1, .05),
    (8192, 16, 40, 2, .1)])
def test_plan(cuda, B, bs, hi_ctx, hi_new, leave):
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, hi_ctx + 1, B)
    new = np.where(rng.random(B) < leave, -1, rng.integers(0, hi_new + 1, B))
    cap = int(np.maximum(new, 0).sum()) + 1
    width_ = -(-(hi_ctx + hi_new) // bs) + 1
    take = int((-(-(ctx + np.maximum(new, 0)) // bs) - -(-ctx // bs)).sum())
    table, ring, state, n = pool_state(rng, ctx, bs, take + 1, width_)
    # one that happens, one that does not
    for st in (state, [state[0], max(0, take - 1)]):
        want = O.plan(ctx, new, table, ring, st, bs, cap)
        t, r = guarded(table, torch.int32, cuda), guarded(ring, torch.int32, cuda)
        co, so = (blank((k,), torch.int32, cuda) for k in (B, 2))
        sl, po, cu = (blank((k,), torch.int32, cuda) for k in (cap, cap, B + 1))
        ws = paged_ws(n, cuda)
        L.mla_paged_plan(i32(ctx), i32(new), t.t, r.t, i32(st), co.t, so.t, sl.t, po.t, cu.t, B,
                         width_, n, bs, cap, ws.t)
        assert all_intact(t, r, co, so, sl, po, cu, ws)
        for g, k in ((t, "table"), (r, "ring"), (co, "ctx"), (so, "state"), (sl, "slots"),
                     (po, "pos"), (cu, "cu")):
            assert np.array_equal(g.t.cpu().numpy(), want[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs,runs", [
    (16, [(0, 16), (15, 1), (0, 16)]), (128, [(0, 128), (127, 1), (1, 2), (64, 64)] * 3),
    (16, [(0, 16)] * 700 + [(2, 14)])])
def test_append(cuda, dtype, bs, runs):
    """The first and the last block of the pool are among those written."""
    cfg = bf16(2) if dtype == "bf16" else F32
    n_blocks = len(runs)
    slots = slots_for(np.random.default_rng(bs), n_blocks, bs, runs)
    rows = random_rows(len(slots), width(cfg), torch.bfloat16 if dtype == "bf16"
                       else torch.float32, bs)
    cache, scales = dirty_pool(n_blocks, bs, width(cfg), 5)
    c, s = guarded(cache, torch.uint8, cuda), guarded(scales, torch.float32, cuda)
    ws = paged_ws(n_blocks, cuda)
    L.mla_paged_append(cfg, rows.cuda(), i32(slots), c.t, s.t, len(slots), n_blocks, bs, ws.t)
    assert all_intact(c, s, ws)
    L.mla_check_device_status(ws.t)
    want, wsc = O.append(rows, slots, cache.numpy(), scales.numpy(), bs)
    assert np.array_equal(s.t.cpu().numpy(), wsc)
    assert np.array_equal(O.E4M3[c.t.cpu().numpy()], O.E4M3[want])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs,ctx", [(16, [1]), (64, [63, 64, 65, 0, 1, 128]), (32, list(range(70)))])
def test_gather(cuda, dtype, bs, ctx):
    cfg = bf16(2) if dtype == "bf16" else F32
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    table, n = make_tables(np.random.default_rng(len(ctx)), ctx, bs, spare=0, extra_width=0)
    cache, scales = dirty_pool(n, bs, width(cfg), 7)
    want = np.concatenate([O.rows_of(cache, scales, table, ctx, b, bs) for b in range(len(ctx))])
    for cap in (sum(ctx), max(1, sum(ctx) // 2)):     # whole, and cut off
        rows, cu = blank((cap, width(cfg)), dt, cuda), blank((len(ctx) + 1,), torch.int32, cuda)
        ws = paged_ws(n, cuda)
        L.mla_paged_gather(cfg, cache.cuda(), scales.cuda(), i32(table), i32(ctx), rows.t, cu.t,
                           len(ctx), table.shape[1], n, bs, cap, ws.t)
        assert all_intact(rows, cu, ws)
        assert np.array_equal(f64(rows.t), want[:cap])


@pytest.mark.parametrize("with_o", [False, True])
@pytest.mark.parametrize("cfg", [
    F32, bf16(1), bf16(20), bf16(65, hidden_size=136), bf16(128),
    bf16(3, kv_lora_rank=96, qk_rope_head_dim=32, qk_nope_head_dim=24, v_head_dim=40),
    bf16(3, qk_nope_head_dim=200, v_head_dim=72)],
    ids=["f32", "h1", "h20", "h65", "h128", "other", "wide"])
@pytest.mark.parametrize("bs,ctx", [(16, [1, 17, 0, 500, 33]), (64, [3000, 1, 129]),
                                    (32, [40 * b % 97 for b in range(40)])])
def test_decode(cuda, cfg, bs, ctx, with_o):
    d = decode_inputs(cfg, ctx, bs, len(ctx))
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    B, mb = len(ctx), d["table"].shape[1]
    n, _ = L.mla_decode_paged_workspace_size(cfg, B, mb, bs)
    ws = Guarded((n,), torch.uint8, cuda, 0xA5)
    out = blank((B, cfg.hidden_size if with_o else cfg.num_heads * cfg.v_head_dim), dt, cuda)
    cache, scales = guarded(d["cache"], torch.uint8, cuda), guarded(d["scales"], torch.float32, cuda)
    L.mla_decode_paged(cfg, d["q_nope"].cuda(), d["q_pe"].cuda(), d["w"].cuda(), cache.t, scales.t,
                       i32(d["table"]), i32(ctx), B, mb, d["n_blocks"], bs,
                       d["w_o"].cuda() if with_o else None, out.t, ws.t)
    assert all_intact(ws, out, cache, scales)
    L.mla_check_device_status(ws.t)
    assert torch.equal(cache.t.cpu(), d["cache"])
    assert oracle.max_rel_err(out.t, want_decode(cfg, d, bs, with_o)) <= TOL[cfg.dtype]


@pytest.mark.parametrize("cfg", [F32, bf16(16), bf16(128)], ids=["f32", "h16", "h128"])
def test_no_call_allocates_device_memory(cuda, cfg):
    from latent_attention_b200.layer import MlaPagedCache
    B, h = 5, cfg.num_heads
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    pc = MlaPagedCache(cfg, B, max_blocks=40, n_blocks=200, block_size=16, capacity=3000)
    new = i32([600, 1, 0, 300, 40])
    rows = torch.randn(3000, width(cfg), device=cuda).to(dt)
    q = [torch.randn(B, h, k, device=cuda).to(dt)
         for k in (cfg.qk_nope_head_dim, cfg.qk_rope_head_dim)]
    w = torch.randn(h * (cfg.qk_nope_head_dim + cfg.v_head_dim), cfg.kv_lora_rank,
                    device=cuda).to(dt)
    w_o = torch.randn(cfg.hidden_size, h * cfg.v_head_dim, device=cuda).to(dt)
    out = torch.empty(B, cfg.hidden_size, dtype=dt, device=cuda)
    got = torch.empty(3000, width(cfg), dtype=dt, device=cuda)
    cu = torch.empty(B + 1, dtype=torch.int32, device=cuda)

    def step():
        pc.plan(new)
        pc.append(rows)
        pc.decode(*q, w, out, w_o)
        pc.gather(got, cu)
        torch.cuda.synchronize()

    step()                                          # loads the kernels
    pc.check_status()
    new.copy_(i32([1, 1, 1, 1, -1]))
    free, made = torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        step()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == made
    assert torch.cuda.mem_get_info()[0] == free
    pc.check_status()
