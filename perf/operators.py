"""The paged 8-bit latent cache and the operators around it: what is measured.

A serving step with this library keeps the compressed latent rows
``[RMSNorm(c) | roped k_pe]`` of all requests in one pool of blocks, 8 bits
(e4m3) a value and one power-of-two scale a block.  Four operators:

* ``plan``    block tables and slot maps from request lengths,
* ``append``  latent rows into the blocks that a slot map names,
* ``gather``  the rows of whole requests back in the model's type,
* ``decode``  weight-absorbed attention of one query token per request over
  the blocks of its table.

``run`` computes each in plain torch operations, or, with ``own``, through the
library's entry points.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
MIN_EXP = -64            # smallest exponent of a block's scale
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Head dimensions: the DeepSeek-V3 / Kimi latent, and the small fp32 layer.
WIDE = {"dn": 128, "dr": 64, "dv": 128, "r": 512}
SMALL = {"dn": 32, "dr": 16, "dv": 32, "r": 32}
# (nope + rope)^-0.5 times the YaRN factor (0.1 ln 40 + 1)^2, and without it.
YARN_SCALE = (0.1 * math.log(40.0) + 1.0) ** 2 / math.sqrt(192.0)


def dims_of(case):
    return WIDE if case["dtype"] == "bf16" else SMALL


def scale_of(case):
    d = dims_of(case)
    return YARN_SCALE if case["dtype"] == "bf16" else (d["dn"] + d["dr"]) ** -0.5


def listed():
    return [
        # One decode step of a full server: 256 requests, one new token each
        # but for a few that finished.
        {"name": "plan_step", "op": "plan", "requests": 256, "ctx_min": 1, "ctx_max": 32768,
         "new_min": 1, "new_max": 1, "leave": 0.03, "block_size": 64},
        # A batch of prompts admitted at once, small blocks.
        {"name": "plan_prompts", "op": "plan", "requests": 61, "ctx_min": 0, "ctx_max": 512,
         "new_min": 100, "new_max": 8192, "leave": 0.0, "block_size": 16},
        # The new rows of one decode step, one per request, into part-filled blocks.
        {"name": "append_step", "op": "append", "requests": 128, "new_min": 1, "new_max": 1,
         "fill": 1, "block_size": 64, "dtype": "bf16"},
        # One prompt of 4096 tokens into fresh blocks.
        {"name": "append_prompt", "op": "append", "requests": 1, "new_min": 4096, "new_max": 4096,
         "fill": 0, "block_size": 64, "dtype": "bf16"},
        # Chunks of many prompts of odd lengths, first blocks part-filled.
        {"name": "append_chunks", "op": "append", "requests": 37, "new_min": 129,
         "new_max": 2500, "fill": 1, "block_size": 32, "dtype": "bf16"},
        # The shared prefix of four requests, for a chunked prefill after it.
        {"name": "gather_prefix", "op": "gather", "requests": 4, "ctx_min": 2048,
         "ctx_max": 2048, "block_size": 64, "dtype": "bf16"},
        # The whole cache of a mixed batch.
        {"name": "gather_mixed", "op": "gather", "requests": 64, "ctx_min": 1000,
         "ctx_max": 16384, "block_size": 64, "dtype": "bf16"},
        # A lightly loaded server: few requests with short contexts, latency counts.
        {"name": "decode_short", "op": "decode", "requests": 4, "heads": 128, "ctx_min": 90,
         "ctx_max": 700, "block_size": 64, "dtype": "bf16", "hidden": 0},
        # One request with a very long context, all 128 heads on one GPU.
        {"name": "decode_long", "op": "decode", "requests": 1, "heads": 128, "ctx_min": 131000,
         "ctx_max": 131000, "block_size": 64, "dtype": "bf16", "hidden": 0},
        # The serving batch: 64 requests of mixed lengths, 128 heads.
        {"name": "decode_batch", "op": "decode", "requests": 64, "heads": 128, "ctx_min": 1024,
         "ctx_max": 32768, "block_size": 64, "dtype": "bf16", "hidden": 0},
        # An eighth of the heads (they are split over GPUs), a larger batch,
        # small blocks, the output projection of the layer's width.
        {"name": "decode_heads16", "op": "decode", "requests": 96, "heads": 16, "ctx_min": 1,
         "ctx_max": 12000, "block_size": 16, "dtype": "bf16", "hidden": 4096},
        # The fp32 layer.
        {"name": "decode_f32", "op": "decode", "requests": 8, "heads": 4, "ctx_min": 1,
         "ctx_max": 2000, "block_size": 32, "dtype": "f32", "hidden": 0},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "gather", "decode", "decode"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _spread(rng, 1, 1024)
        hi = _spread(rng, 1, max(1, min(8192, 250000 // B)))
        return {"op": op, "requests": B, "ctx_min": 0, "ctx_max": _spread(rng, 1, 32768),
                "new_min": rng.choice([0, 1, max(1, hi // 8)]) if hi > 1 else 1, "new_max": hi,
                "leave": rng.choice([0.0, 0.05, 0.3]), "block_size": bs}
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        B = _spread(rng, 1, 256)
        hi = _spread(rng, 1, max(1, min(8192, 48000 // B)))
        return {"op": op, "requests": B, "new_min": max(1, hi // rng.choice([1, 2, 16])),
                "new_max": hi, "fill": rng.choice([0, 1]), "block_size": bs, "dtype": dtype}
    if op == "gather":
        B = _spread(rng, 1, 256)
        hi = _spread(rng, 1, max(1, min(16384, 500000 // B)))
        return {"op": op, "requests": B, "ctx_min": rng.choice([0, 1, max(1, hi // 4)]),
                "ctx_max": hi, "block_size": bs, "dtype": dtype}
    if dtype == "f32":
        B = _spread(rng, 1, 16)
        hi = _spread(rng, 1, 4000)
        return {"op": op, "requests": B, "heads": rng.randint(1, 6), "ctx_min": rng.choice([0, 1]),
                "ctx_max": hi, "block_size": bs, "dtype": dtype, "hidden": rng.choice([0, 256])}
    B = _spread(rng, 1, 128)
    hi = _spread(rng, 1, max(1, min(65536, 1000000 // B)))
    return {"op": op, "requests": B, "heads": rng.choice([1, 5, 8, 16, 31, 32, 48, 64, 96, 128]),
            "ctx_min": rng.choice([0, 1, max(1, hi // 4)]), "ctx_max": hi, "block_size": bs,
            "dtype": dtype, "hidden": rng.choice([0, 0, 1024, 4096])}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _lengths(case, lo, hi, which):
    """The case's lengths, uniform on [lo, hi]: the case alone sets them, so
    that all seeds give outputs of the same sizes."""
    g = torch.Generator().manual_seed(1000 * which + case["requests"])
    return torch.randint(lo, hi + 1, (case["requests"],), generator=g)


def _blocks(lens, bs):
    return (lens + bs - 1) // bs


def _pool(n_blocks, bs, W, g):
    """A pool of filled blocks: latent rows of a normalised layer, some blocks
    with rows a few times larger, quantised with their block's scale."""
    x = torch.randn(n_blocks, bs, W, device="cuda", generator=g)
    x *= 2.0 ** (2.0 * torch.rand(n_blocks, 1, 1, device="cuda", generator=g))
    scales = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 2)) / FP8_MAX)))
    return (x / scales[:, None, None]).to(FP8), scales


def _tables(counts, n_blocks, width, g):
    """Tables of distinct blocks in random order; entries past a request's
    blocks are -1."""
    order = torch.randperm(n_blocks, device="cuda", generator=g).to(torch.int32)
    counts = counts.cuda()
    first = torch.cumsum(counts, 0) - counts
    j = torch.arange(width, device="cuda")
    idx = (first[:, None] + j).clamp_(max=n_blocks - 1)
    return torch.where(j < counts[:, None], order[idx], -1).to(torch.int32).contiguous(), order


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, bs, op = case["requests"], case["block_size"], case["op"]
    s = {"case": case}
    # the requests come in another order with every seed
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed))
    if op == "plan":
        ctx = _lengths(case, case["ctx_min"], case["ctx_max"], 1)[order]
        new = _lengths(case, case["new_min"], case["new_max"], 2)
        new[_lengths(case, 0, 999, 3) < 1000 * case["leave"]] = -1
        new = new[order]
        held = _blocks(ctx, bs)
        after = _blocks(ctx + new.clamp(min=0), bs)
        n_blocks = int((held + after).sum()) + 7
        s["max_blocks"] = int(max(int(after.max()), int(held.max()), 1)) + 1
        s["table"], ids = _tables(held, n_blocks, s["max_blocks"], g)
        # the free ring: every block that no request holds, from `head` on
        used = int(held.sum())
        head = (seed * 7919) % n_blocks
        s["ring"] = torch.roll(torch.cat([ids[used:], ids[:used]]), head).contiguous()
        s["state"] = torch.tensor([head, n_blocks - used], dtype=torch.int32, device="cuda")
        s["ctx"], s["new"] = ctx.to(torch.int32).cuda(), new.to(torch.int32).cuda()
        s["n_blocks"] = n_blocks
        s["capacity"] = int(new.clamp(min=0).sum()) + 5
        i32 = dict(dtype=torch.int32, device="cuda")
        s["ctx_out"], s["state_out"] = torch.empty(B, **i32), torch.empty(2, **i32)
        s["slots"], s["pos"] = torch.empty(s["capacity"], **i32), torch.empty(s["capacity"], **i32)
        s["cu"] = torch.empty(B + 1, **i32)
        return s
    d = dims_of(case)
    W, dt = d["r"] + d["dr"], DTYPES[case["dtype"]]
    if op == "append":
        new = _lengths(case, case["new_min"], case["new_max"], 1)[order]
        filled = _lengths(case, 0, case["fill"] * (bs - 1), 2)[order]
        counts = _blocks(filled + new, bs)
        n_blocks = int(counts.sum()) + 9
        s["cache"], s["scales"] = _pool(n_blocks, bs, W, g)
        table, _ = _tables(counts, n_blocks, int(counts.max()), g)
        n = int(new.sum())
        seq = torch.repeat_interleave(torch.arange(B), new).cuda()
        at = (torch.arange(n) - torch.repeat_interleave(torch.cumsum(new, 0) - new, new)
              + torch.repeat_interleave(filled, new)).cuda()
        s["slots"] = (table[seq, at // bs].long() * bs + at % bs).to(torch.int32)
        rows = torch.randn(n, W, device="cuda", generator=g)
        rows *= 2.0 ** (2.0 * torch.rand(n, 1, device="cuda", generator=g))
        s["rows"], s["n"], s["n_blocks"] = rows.to(dt), n, n_blocks
        return s
    ctx = _lengths(case, case["ctx_min"], case["ctx_max"], 1)[order]
    counts = _blocks(ctx, bs)
    s["max_blocks"] = max(1, int(counts.max()))
    s["n_blocks"] = n_blocks = int(counts.sum()) + 5
    s["cache"], s["scales"] = _pool(n_blocks, bs, W, g)
    s["table"], _ = _tables(counts, n_blocks, s["max_blocks"], g)
    s["ctx"] = ctx.to(torch.int32).cuda()
    if op == "gather":
        s["capacity"] = max(1, int(ctx.sum()))
        s["rows"] = torch.zeros(s["capacity"], W, dtype=dt, device="cuda")
        s["cu"] = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        return s
    h, hidden = case["heads"], case["hidden"]
    s["q_nope"] = torch.randn(B, h, d["dn"], device="cuda", generator=g).to(dt)
    s["q_pe"] = torch.randn(B, h, d["dr"], device="cuda", generator=g).to(dt)
    s["w_kv_b"] = (0.02 * torch.randn(h * (d["dn"] + d["dv"]), d["r"], device="cuda",
                                      generator=g)).to(dt)
    s["w_o"] = (0.02 * torch.randn(hidden, h * d["dv"], device="cuda", generator=g)).to(dt) \
        if hidden else None
    s["out"] = torch.empty(B, hidden or h * d["dv"], dtype=dt, device="cuda")
    return s


# --------------------------------------------------------------------------
# The plain forms
# --------------------------------------------------------------------------
def _plan(s):
    case = s["case"]
    bs, n_blocks, cap = case["block_size"], s["n_blocks"], s["capacity"]
    table, ring = s["table"], s["ring"]
    width = s["max_blocks"]
    ctx, new = s["ctx"].long(), s["new"].long()
    leave = new < 0
    grow = new.clamp(min=0)
    held = (ctx + bs - 1) // bs
    want = torch.where(leave, held, (ctx + grow + bs - 1) // bs)
    add = want - held
    give = torch.where(leave, held, 0)
    head, count = s["state"][0].long(), s["state"][1].long()
    ok = ((ctx >= 0) & (new >= -1) & (want <= width)).all() & (add.sum() <= count) \
        & (grow.sum() <= cap)
    j = torch.arange(width, device="cuda")
    # released blocks go behind the free ones, in table order
    back = torch.where((j < give[:, None]) & ok,
                       (head + count + (torch.cumsum(give, 0) - give)[:, None] + j) % n_blocks,
                       n_blocks)
    fresh = (j >= held[:, None]) & (j < want[:, None]) & ok
    take = (head + (torch.cumsum(add, 0) - add - held)[:, None] + j) % n_blocks
    taken = torch.where(fresh, ring[take], table)
    wide = torch.cat([ring, ring[:1]])
    wide.scatter_(0, back.reshape(-1), table.reshape(-1))
    ring.copy_(wide[:n_blocks])
    table.copy_(taken)
    ends = torch.cumsum(grow, 0)
    i = torch.arange(cap, device="cuda")
    b = torch.searchsorted(ends, i, right=True).clamp_(max=len(ctx) - 1)
    at = ctx[b] + i - (ends - grow)[b]
    live = (i < ends[-1]) & ok
    page = table[b, (at // bs).clamp_(0, width - 1)].long()
    s["slots"].copy_(torch.where(live, page * bs + at % bs, -1))
    s["pos"].copy_(torch.where(live, at, 0))
    s["cu"][:1].zero_()
    s["cu"][1:].copy_(torch.where(ok, ends, 0))
    s["ctx_out"].copy_(torch.where(ok, torch.where(leave, 0, ctx + grow), ctx))
    s["state_out"].copy_(torch.where(ok, torch.stack([(head + add.sum()) % n_blocks,
                                                      count - add.sum() + give.sum()]),
                                     s["state"].long()))


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, at least MIN_EXP."""
    m, k = torch.frexp(amax)
    e = k - 9 + (m > 0.875).to(k.dtype)
    return torch.where(amax > 0, e, MIN_EXP).clamp_(min=MIN_EXP)


def _append(s):
    case, cache, scales = s["case"], s["cache"], s["scales"]
    bs = case["block_size"]
    slots = s["slots"].long()
    rows = s["rows"].float()
    block, at = slots // bs, slots % bs
    touched, run = torch.unique(block, return_inverse=True)
    n = len(touched)
    amax = torch.zeros(n, device="cuda").scatter_reduce_(0, run, rows.abs().amax(1), "amax")
    first = torch.full((n,), bs, device="cuda").scatter_reduce_(0, run, at, "amin")
    old = torch.frexp(scales[touched])[1] - 1
    e = _exponent(amax)
    e = torch.where(first > 0, torch.maximum(e, old), e)
    # rows in front of the new ones move to the block's new scale
    kept = cache.view(torch.uint8)[touched].view(FP8)
    moved = torch.ldexp(kept.float(), (old - e)[:, None, None]).to(FP8)
    front = torch.arange(bs, device="cuda") < first[:, None]
    cache.view(torch.uint8)[touched] = torch.where(front[..., None], moved.view(torch.uint8),
                                                   kept.view(torch.uint8))
    scales[touched] = torch.exp2(e.float())
    q = torch.ldexp(rows, -e[run][:, None]).to(FP8)
    cache.view(torch.uint8)[block, at] = q.view(torch.uint8)


def _rows_of(s):
    """Dequantised rows of every request, [B, max_blocks * bs, W], fp32."""
    t = s["table"].long().clamp(min=0)
    c = s["cache"].view(torch.uint8)[t].view(FP8).float()
    c *= s["scales"][t][..., None, None]
    return c.flatten(1, 2)


def _gather(s):
    bs = s["case"]["block_size"]
    ctx = s["ctx"].long()
    ends = torch.cumsum(ctx, 0)
    i = torch.arange(s["capacity"], device="cuda")
    b = torch.searchsorted(ends, i, right=True).clamp_(max=len(ctx) - 1)
    at = i - (ends - ctx)[b]
    live = i < ends[-1]
    page = s["table"][b, (at // bs).clamp_(0, s["max_blocks"] - 1)].long().clamp_(min=0)
    rows = s["cache"].view(torch.uint8)[page, at.clamp(min=0) % bs].view(FP8).float()
    rows *= s["scales"][page][:, None]
    s["rows"].copy_(torch.where(live[:, None], rows, s["rows"].float()))
    s["cu"][:1].zero_()
    s["cu"][1:].copy_(ends)


def _decode(s):
    case = s["case"]
    d, h, B = dims_of(case), case["heads"], case["requests"]
    r, dn, dv = d["r"], d["dn"], d["dv"]
    w = s["w_kv_b"].float().view(h, dn + dv, r)
    q = torch.cat([torch.einsum("bhd,hdr->bhr", s["q_nope"].float(), w[:, :dn]),
                   s["q_pe"].float()], -1)
    c = _rows_of(s)
    score = torch.matmul(q, c.transpose(1, 2)) * scale_of(case)
    seen = torch.arange(c.shape[1], device="cuda") < s["ctx"].long()[:, None, None]
    score.masked_fill_(~seen, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -torch.inf, 0, top))
    p /= p.sum(-1, keepdim=True).clamp_(min=1e-30)
    c.masked_fill_(~seen.transpose(1, 2), 0.0)
    o = torch.einsum("bhr,hvr->bhv", torch.matmul(p, c[..., :r]), w[:, dn:]).flatten(1)
    s["out"].copy_(o if s["w_o"] is None else o @ s["w_o"].float().T)


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------
def _config(case):
    import types
    d = dims_of(case)
    return types.SimpleNamespace(
        hidden_size=case.get("hidden") or 256, num_heads=case.get("heads", 1), q_lora_rank=0,
        kv_lora_rank=d["r"], qk_nope_head_dim=d["dn"], qk_rope_head_dim=d["dr"],
        v_head_dim=d["dv"], rope_type="none", rope_theta=1e4, rope_factor=1.0, rope_mscale=1.0,
        rope_mscale_all_dim=0.0, beta_fast=32.0, beta_slow=1.0,
        original_max_position_embeddings=4096, rms_eps=1e-6, softmax_scale=scale_of(case),
        dtype=case["dtype"])


def _handle(s):
    """The configuration and the workspace that a program keeps between calls."""
    if "ws" not in s:
        import latent_attention_b200 as mla
        case = s["case"]
        s["cfg"] = mla.make_config(_config(case)) if case["op"] != "plan" else None
        if case["op"] == "decode":
            n, _ = mla.mla_decode_paged_workspace_size(s["cfg"], case["requests"],
                                                       s["max_blocks"], case["block_size"])
        else:
            n = mla.mla_paged_workspace_size(s["n_blocks"])
        s["mla"], s["ws"] = mla, torch.empty(n, dtype=torch.uint8, device="cuda")
    return s["mla"]


def _call(s):
    case, op = s["case"], s["case"]["op"]
    B, bs = case["requests"], case["block_size"]
    mla = _handle(s)
    if op == "plan":
        mla.mla_paged_plan(s["ctx"], s["new"], s["table"], s["ring"], s["state"], s["ctx_out"],
                           s["state_out"], s["slots"], s["pos"], s["cu"], B, s["max_blocks"],
                           s["n_blocks"], bs, s["capacity"], s["ws"])
    elif op == "append":
        mla.mla_paged_append(s["cfg"], s["rows"], s["slots"], s["cache"], s["scales"], s["n"],
                             s["n_blocks"], bs, s["ws"])
    elif op == "gather":
        mla.mla_paged_gather(s["cfg"], s["cache"], s["scales"], s["table"], s["ctx"], s["rows"],
                             s["cu"], B, s["max_blocks"], s["n_blocks"], bs, s["capacity"],
                             s["ws"])
    else:
        mla.mla_decode_paged(s["cfg"], s["q_nope"], s["q_pe"], s["w_kv_b"], s["cache"],
                             s["scales"], s["table"], s["ctx"], B, s["max_blocks"],
                             s["n_blocks"], bs, s["w_o"], s["out"], s["ws"])


def run(state):
    op = state["case"]["op"]
    if own:
        _call(state)
    else:
        {"plan": _plan, "append": _append, "gather": _gather, "decode": _decode}[op](state)
    keys = {"plan": ("table", "ring", "state_out", "ctx_out", "slots", "pos", "cu"),
            "append": ("cache", "scales"), "gather": ("rows", "cu"), "decode": ("out",)}[op]
    return {k: state[k] for k in keys}


# --------------------------------------------------------------------------
# Work, and the definition in 64 bits
# --------------------------------------------------------------------------
def work(case):
    B, bs, op = case["requests"], case["block_size"], case["op"]
    if op == "plan":
        new = (case["new_min"] + case["new_max"]) / 2 * (1 - case["leave"]) * B
        held = (case["ctx_min"] + case["ctx_max"]) / 2 / bs * case["leave"] * B
        # lengths in and out, cu; a slot and a position per new token; a ring
        # and a table entry per block that changes hands
        return {"bytes": 16 * B + 8 * new + 8 * (new / bs + held), "flops": 0}
    d = dims_of(case)
    W, es = d["r"] + d["dr"], 2 if case["dtype"] == "bf16" else 4
    if op == "append":
        n = (case["new_min"] + case["new_max"]) / 2 * B
        return {"bytes": n * (W * es + W + 4) + 8 * (n / bs + B), "flops": 2 * n * W}
    n = (case["ctx_min"] + case["ctx_max"]) / 2 * B
    if op == "gather":
        return {"bytes": n * (W + W * es) + 8 * n / bs + 8 * B, "flops": n * W}
    h, hidden, v = case["heads"], case["hidden"], case["heads"] * d["dv"]
    weights = h * (d["dn"] + d["dv"]) * d["r"] + hidden * v
    return {"bytes": n * W + 8 * n / bs + es * (weights + B * h * (d["dn"] + d["dr"])
                                                + B * (hidden or v)),
            "flops": 2 * n * h * (W + d["r"]) + 2 * B * weights}


def _e4m3_64(x):
    """The nearest e4m3 value (ties to even) of float64 values within +-448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    bs = case["block_size"]
    if case["op"] == "append":
        val, sc = s["cache"].double(), s["scales"].double()
        slots, rows = s["slots"].tolist(), s["rows"].double()
        i = 0
        while i < len(slots):
            blk, first, k = slots[i] // bs, slots[i] % bs, i + 1
            while k < len(slots) and slots[k] // bs == blk:
                k += 1
            big = float(rows[i:k].abs().max())
            e = max(MIN_EXP, math.ceil(math.log2(big / FP8_MAX))) if big else MIN_EXP
            new = max(2.0 ** e, float(sc[blk])) if first else 2.0 ** e
            val[blk, :first] = _e4m3_64(val[blk, :first] * (float(sc[blk]) / new))
            val[blk, first:first + k - i] = _e4m3_64(rows[i:k] / new)
            sc[blk] = new
            i = k
        return {"cache": val, "scales": sc}
    ctx, table = s["ctx"].tolist(), s["table"].long()

    def rows_of(b):
        t = table[b, :(ctx[b] + bs - 1) // bs]
        c = s["cache"].view(torch.uint8)[t].view(FP8).double() * s["scales"].double()[t][:, None, None]
        return c.flatten(0, 1)[:ctx[b]]

    if case["op"] == "gather":
        got = torch.cat([rows_of(b) for b in range(len(ctx))]
                        + [torch.zeros(max(0, s["capacity"] - sum(ctx)), s["rows"].shape[1],
                                       dtype=torch.float64, device="cuda")])
        return {"rows": got, "cu": None}
    d, h = dims_of(case), case["heads"]
    w = s["w_kv_b"].double().view(h, d["dn"] + d["dv"], d["r"])
    out = []
    for b, n in enumerate(ctx):
        o = torch.zeros(h, d["dv"], dtype=torch.float64, device="cuda")
        if n:
            c = rows_of(b)
            k = torch.einsum("hd,hdr->hr", s["q_nope"][b].double(), w[:, :d["dn"]])
            score = k @ c[:, :d["r"]].T + s["q_pe"][b].double() @ c[:, d["r"]:].T
            p = torch.softmax(score * scale_of(case), -1)
            o = torch.einsum("hr,hvr->hv", p @ c[:, :d["r"]], w[:, d["dn"]:])
        o = o.flatten()
        out.append(o if s["w_o"] is None else s["w_o"].double() @ o)
    return {"out": torch.stack(out)}
