"""The paged 8-bit latent cache on a B200 against the fp64 oracle.

plan, append and gather have exact answers (whole numbers, e4m3 bytes, powers
of two; a gathered value e4m3 * 2^e has 4 significant bits), so they are
compared bit for bit.  The decode is held to the tolerances of the other
decode paths: 1e-5 (fp32) and 2e-2 (bf16) of the largest output."""
import numpy as np
import pytest
import torch

import latent_attention_b200 as L
import oracle
from gpu_helpers import TOL, f64
from latent_attention_b200.layer import MlaDecode, MlaPagedCache
from mla_inputs import WORKLOADS, MlaConfig
from oracle import paged as O

pytestmark = pytest.mark.gpu

F32 = WORKLOADS["tiny_f32"].cfg
DSV3 = WORKLOADS["dsv3_decode"].cfg
FP8 = torch.float8_e4m3fn


def bf16(heads, **kw):
    base = dict(hidden_size=256, num_heads=heads, q_lora_rank=0, kv_lora_rank=512,
                qk_nope_head_dim=128, qk_rope_head_dim=64, v_head_dim=128, rope_type="none",
                dtype="bf16")
    base.update(kw)
    return MlaConfig(**base)


def i32(x, dev="cuda"):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev).contiguous()


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def paged_ws(n_blocks):
    return torch.empty(L.mla_paged_workspace_size(n_blocks), dtype=torch.uint8, device="cuda")


# -------------------------------------------------------------------- plan
def run_plan(ctx, new, table, ring, state, bs, cap, in_place=False, pos=True):
    B, width = table.shape
    d = dict(ctx=i32(ctx), new=i32(new), table=i32(table), ring=i32(ring), state=i32(state))
    d["ctx_out"] = d["ctx"] if in_place else torch.full_like(d["ctx"], 77)
    d["state_out"] = d["state"] if in_place else torch.full_like(d["state"], 77)
    d["slots"] = torch.full((cap + 3,), 77, dtype=torch.int32, device="cuda")
    d["pos"] = torch.full((cap + 3,), 77, dtype=torch.int32, device="cuda") if pos else None
    d["cu"] = torch.full((B + 4,), 77, dtype=torch.int32, device="cuda")
    ws = paged_ws(len(ring))
    L.mla_paged_plan(d["ctx"], d["new"], d["table"], d["ring"], d["state"], d["ctx_out"],
                     d["state_out"], d["slots"] if cap else None, d["pos"], d["cu"], B, width,
                     len(ring), bs, cap, ws)
    try:
        L.mla_check_device_status(ws)
        status = "ok"
    except L.MlaError as e:
        status = {"MLA_ERR_SHAPE": "shape", "MLA_ERR_NO_BLOCKS": "blocks"}[e.name]
    return d, status


def check_plan(ctx, new, table, ring, state, bs, cap, **kw):
    want = O.plan(ctx, new, table, ring, state, bs, cap)
    d, status = run_plan(ctx, new, table, ring, state, bs, cap, **kw)
    assert status == want["status"]
    B = len(ctx)
    for k, w in (("table", want["table"]), ("ring", want["ring"]), ("ctx_out", want["ctx"]),
                 ("state_out", want["state"])):
        assert np.array_equal(d[k].cpu().numpy(), w), k
    assert np.array_equal(d["cu"].cpu().numpy(), np.concatenate([want["cu"], [77] * 3]))
    assert np.array_equal(d["slots"].cpu().numpy(), np.concatenate([want["slots"], [77] * 3]))
    if d["pos"] is not None:
        assert np.array_equal(d["pos"].cpu().numpy(), np.concatenate([want["pos"], [77] * 3]))
    return want


def pool_state(rng, ctx, bs, extra, width):
    """Tables of distinct blocks for `ctx`, and the ring of the others."""
    held = [-(-int(c) // bs) for c in ctx]
    n_blocks = sum(held) + extra
    ids = rng.permutation(n_blocks)
    table, at = np.full((len(ctx), width), -1), 0
    for b, k in enumerate(held):
        table[b, :k] = ids[at:at + k]
        at += k
    head = int(rng.integers(0, n_blocks))
    ring = np.roll(np.concatenate([ids[at:], ids[:at]]), head)
    return table, ring, [head, extra], n_blocks


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,bs,hi_ctx,hi_new,leave", [
    (1, 16, 0, 1, 0), (1, 128, 5, 700, 0), (3, 64, 300, 0, 0), (31, 32, 900, 40, .3),
    (33, 16, 100, 300, .1), (256, 64, 5000, 1, .05), (1024, 16, 60, 3, .2),
    (1025, 32, 400, 20, .5), (8192, 16, 40, 2, .1)])
def test_plan_matches_the_oracle(cuda, B, bs, hi_ctx, hi_new, leave, in_place):
    rng = np.random.default_rng(B + bs)
    ctx = rng.integers(0, hi_ctx + 1, B)
    new = np.where(rng.random(B) < leave, -1, rng.integers(0, hi_new + 1, B))
    width = -(-(hi_ctx + hi_new) // bs) + 1
    want_new = int(np.maximum(new, 0).sum())
    take = int((-(-(ctx + np.maximum(new, 0)) // bs) - -(-ctx // bs)).sum())
    table, ring, state, _ = pool_state(rng, ctx, bs, take + 3, width)
    want = check_plan(ctx, new, table, ring, state, bs, want_new + 2, in_place=in_place)
    assert want["status"] == "ok"
    check_plan(ctx, new, table, ring, state, bs, want_new, in_place=in_place, pos=False)


def test_plan_is_all_or_nothing(cuda):
    rng = np.random.default_rng(0)
    ctx, new = np.array([10, 0, 33, 64]), np.array([7, 20, -1, 1])
    table, ring, state, n = pool_state(rng, ctx, 16, 4, 6)
    ok = (ctx, new, table, ring, state, 16, 28)
    assert check_plan(*ok)["status"] == "ok"
    assert check_plan(*ok[:6], 27)["status"] == "blocks"              # one slot short
    assert check_plan(*ok[:4], [state[0], 3], *ok[5:])["status"] == "blocks"
    assert check_plan(*ok[:4], [n, 4], *ok[5:])["status"] == "shape"   # head out of range
    assert check_plan(*ok[:4], [state[0], -1], *ok[5:])["status"] == "shape"
    assert check_plan(*ok[:4], [state[0], n - 1], *ok[5:])["status"] == "shape"
    assert check_plan([10, -1, 33, 64], *ok[1:])["status"] == "shape"
    assert check_plan(ctx, [7, 20, -2, 1], *ok[2:])["status"] == "shape"
    assert check_plan(ctx, [7, 97, -1, 1], *ok[2:])["status"] == "shape"   # table too narrow
    big = 2 ** 31 - 1
    assert check_plan([big, big, 33, 64], [big, 1, 0, 1], *ok[2:])["status"] == "shape"


def test_plan_without_new_tokens(cuda):
    rng = np.random.default_rng(1)
    ctx = np.array([5, 0, 40])
    table, ring, state, _ = pool_state(rng, ctx, 16, 2, 4)
    check_plan(ctx, [0, 0, 0], table, ring, state, 16, 0, pos=False)
    check_plan(ctx, [-1, -1, -1], table, ring, state, 16, 4)


# ------------------------------------------------------------------ append
def dirty_pool(n_blocks, bs, W, seed):
    g = torch.Generator().manual_seed(seed)
    b = torch.randint(0, 256, (n_blocks, bs, W), generator=g, dtype=torch.uint8)
    b = torch.where((b & 127) == 127, b - 1, b)                   # no NaN
    s = torch.exp2(torch.randint(-9, 4, (n_blocks,), generator=g).float())
    return b, s


def run_append(cfg, rows, slots, cache, scales, bs):
    c, s = cache.cuda().contiguous(), scales.cuda()
    ws = paged_ws(c.shape[0])
    L.mla_paged_append(cfg, rows.cuda().contiguous(), i32(slots), c, s, len(slots), c.shape[0],
                       bs, ws)
    torch.cuda.synchronize()
    return c.cpu().numpy(), s.cpu().numpy(), ws


def check_append(cfg, rows, slots, cache, scales, bs):
    got, sc, ws = run_append(cfg, rows, slots, cache, scales, bs)
    L.mla_check_device_status(ws)
    want, wsc = O.append(rows, slots, cache.numpy(), scales.numpy(), bs)
    assert np.array_equal(sc, wsc)
    assert (np.isnan(O.E4M3[got]) == np.isnan(O.E4M3[want])).all()
    same = (got == want) | np.isnan(O.E4M3[want])
    # a zero may carry either sign
    same |= (O.E4M3[got] == 0) & (O.E4M3[want] == 0)
    assert same.all(), np.argwhere(~same)[:5]


def width(cfg):
    return cfg.kv_lora_rank + cfg.qk_rope_head_dim


def random_rows(n, W, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, W, generator=g) * torch.exp2(6 * torch.rand(n, 1, generator=g) - 3)
    return x.to(dtype)


def slots_for(rng, n_blocks, bs, runs):
    """Slots of (first row, count) runs in distinct blocks of random order."""
    ids = rng.permutation(n_blocks)[:len(runs)]
    return [int(b) * bs + o + i for b, (o, k) in zip(ids, runs) for i in range(k)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs,runs", [
    (16, [(0, 1)]), (16, [(15, 1), (0, 16), (3, 13)]), (32, [(31, 1)] * 7 + [(0, 5)]),
    (64, [(0, 64)] * 5 + [(0, 17)]), (64, [(i, 1) for i in range(64)]),
    (128, [(0, 128), (127, 1), (1, 2), (64, 64)] * 3), (16, [(0, 16)] * 300 + [(2, 9)])])
def test_append_matches_the_oracle(cuda, dtype, bs, runs):
    cfg = bf16(2) if dtype == "bf16" else F32
    rng = np.random.default_rng(len(runs) + bs)
    n_blocks = len(runs) + 3
    slots = slots_for(rng, n_blocks, bs, runs)
    rows = random_rows(len(slots), width(cfg), torch.bfloat16 if dtype == "bf16"
                       else torch.float32, bs)
    check_append(cfg, rows, slots, *dirty_pool(n_blocks, bs, width(cfg), 5), bs)


def test_append_skips_minus_one(cuda):
    W = width(F32)
    rows = random_rows(9, W, torch.float32, 1)
    slots = [-1, 16, 17, -1, 18, -1, 3, 4, -1]       # 18 starts a second run in block 1
    cache, scales = dirty_pool(4, 16, W, 1)
    got, sc, ws = run_append(F32, rows, [-1] * 9, cache, scales, 16)
    L.mla_check_device_status(ws)
    assert np.array_equal(got, cache.numpy()) and np.array_equal(sc, scales.numpy())
    check_append(F32, rows, [-1, 16, 17, -1, -1, -1, 3, 4, -1], cache, scales, 16)
    _, _, ws = run_append(F32, rows, slots, cache, scales, 16)
    with pytest.raises(L.MlaError, match="SHAPE"):
        L.mla_check_device_status(ws)


def test_append_values_at_the_ends(cuda):
    """Zeros, rows whose maximum meets the scale's border, ties, subnormals,
    infinities and NaN; one block each."""
    W, inf, nan = width(F32), float("inf"), float("nan")
    rows = torch.zeros(10, W)
    rows[1, 0] = 448.0
    rows[2, 0] = float(np.nextafter(np.float32(448), np.float32(1e9)))
    rows[3] = torch.linspace(-448, 448, W)
    rows[4, :4] = torch.tensor([448.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -9])
    rows[5, :3] = torch.tensor([1.0, inf, -inf])
    rows[6, :3] = torch.tensor([1.0, nan, -3.0])
    rows[7, :2] = torch.tensor([3e38, -1e-30])
    rows[8, 0] = 1e-38
    rows[9] = nan
    check_append(F32, rows, [16 * i for i in range(10)], *dirty_pool(11, 16, W, 2), 16)


def test_append_moves_kept_rows_to_a_larger_scale_only(cuda):
    W = width(F32)
    cache, _ = dirty_pool(4, 32, W, 3)
    rows = torch.full((4, W), 10.0)
    scales = torch.tensor([2.0 ** -9, 2.0 ** -4, 1.0, 2.0 ** 6])
    check_append(F32, rows, [20, 52, 84, 116], cache, scales, 32)


@pytest.mark.parametrize("slots", [[64, 1], [-2, 1], [2 ** 31 - 1, 1], [5, 5], [5, 4],
                                   [5, 7], [3, 20, 8], [7, 7]])
def test_append_refuses_bad_slots_and_writes_the_rest(cuda, slots):
    """Pool of 4 blocks of 16: what is out of order or range is reported and
    skipped, the other blocks stay as they were."""
    W = width(F32)
    cache, scales = dirty_pool(4, 16, W, 4)
    rows = random_rows(len(slots), W, torch.float32, 2)
    got, sc, ws = run_append(F32, rows, slots, cache, scales, 16)
    with pytest.raises(L.MlaError, match="SHAPE"):
        L.mla_check_device_status(ws)
    touched = {s // 16 for s in slots if 0 <= s < 64}
    for b in set(range(4)) - touched:
        assert np.array_equal(got[b], cache.numpy()[b]) and sc[b] == scales[b]


def test_append_reports_a_broken_scale(cuda):
    W = width(F32)
    for bad in (float("nan"), 0.0, 3.0, -1.0, float("inf"), 2.0 ** -70):
        cache, scales = dirty_pool(2, 16, W, 6)
        scales[1] = bad
        rows = random_rows(1, W, torch.float32, 3)
        check_append(F32, rows, [16], cache, scales, 16)        # row 0: the old one is not used
        _, sc, ws = run_append(F32, rows, [20], cache, scales, 16)
        with pytest.raises(L.MlaError, match="SHAPE"):
            L.mla_check_device_status(ws)
        assert np.isfinite(sc[1]) and sc[1] > 0


# ------------------------------------------------------------------ gather
def run_gather(cfg, cache, scales, table, ctx, bs, cap):
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    rows = torch.full((cap + 2, width(cfg)), 5.0, dtype=dt, device="cuda")
    cu = torch.full((len(ctx) + 1,), -9, dtype=torch.int32, device="cuda")
    ws = paged_ws(cache.shape[0])
    L.mla_paged_gather(cfg, cache.cuda(), scales.cuda(), i32(table), i32(ctx),
                       rows if cap else None, cu, len(ctx), np.shape(table)[1], cache.shape[0],
                       bs, cap, ws)
    torch.cuda.synchronize()
    return f64(rows), cu.cpu().numpy(), ws


def make_tables(rng, ctx, bs, spare=2, extra_width=1):
    held = [-(-int(c) // bs) for c in ctx]
    ids, at = rng.permutation(sum(held) + spare), 0
    table = np.full((len(ctx), max(held + [1]) + extra_width), -1)
    for b, k in enumerate(held):
        table[b, :k] = ids[at:at + k]
        at += k
    return table, len(ids)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs,ctx", [
    (16, [0]), (16, [1]), (64, [63, 64, 65, 0, 1, 128]), (128, [300, 0, 0, 5]),
    (32, list(range(70))), (16, [0, 0, 0]), (16, [1] * 2000), (64, [5000, 3])])
def test_gather_matches_the_oracle(cuda, dtype, bs, ctx):
    cfg = bf16(2) if dtype == "bf16" else F32
    rng = np.random.default_rng(len(ctx))
    table, n_blocks = make_tables(rng, ctx, bs)
    cache, scales = dirty_pool(n_blocks, bs, width(cfg), 7)
    total = sum(ctx)
    rows, cu, ws = run_gather(cfg, cache, scales, table, ctx, bs, total)
    L.mla_check_device_status(ws)
    want = np.concatenate([O.rows_of(cache, scales, table, ctx, b, bs) for b in range(len(ctx))])
    assert np.array_equal(rows[:total], want)
    assert (rows[total:] == 5).all()
    assert np.array_equal(cu, np.concatenate([[0], np.cumsum(ctx)]))
    # a larger buffer: rows behind the last are left alone
    rows, _, ws = run_gather(cfg, cache, scales, table, ctx, bs, total + 100)
    L.mla_check_device_status(ws)
    assert np.array_equal(rows[:total], want) and (rows[total:] == 5).all()


def test_gather_reports_what_is_out_of_range(cuda):
    ctx, bs = [40, 20], 16
    table, n = make_tables(np.random.default_rng(0), ctx, bs, extra_width=0)
    cache, scales = dirty_pool(n, bs, width(F32), 8)
    want = np.concatenate([O.rows_of(cache, scales, table, ctx, b, bs) for b in range(2)])
    rows, cu, ws = run_gather(F32, cache, scales, table, ctx, bs, 50)   # too small
    with pytest.raises(L.MlaError, match="SHAPE"):
        L.mla_check_device_status(ws)
    assert np.array_equal(rows[:50], want[:50]) and (rows[50:] == 5).all()
    for bad in (-1, n, 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[0, 1] = bad
        rows, _, ws = run_gather(F32, cache, scales, t, ctx, bs, 60)
        with pytest.raises(L.MlaError, match="SHAPE"):
            L.mla_check_device_status(ws)
        w = want.copy()
        w[16:32] = 0
        assert np.array_equal(rows[:60], w)
    for bad, n_rows in (([-5, 20], 20), ([49, 20], 68)):      # the table holds 48 tokens
        rows, cu, ws = run_gather(F32, cache, scales, table, bad, bs, 70)
        with pytest.raises(L.MlaError, match="SHAPE"):
            L.mla_check_device_status(ws)
        assert cu[-1] == n_rows


BAD_SCALES = [float("nan"), float("inf"), 0.0, -1.0, 3.0, 2.0 ** -65, 2.0 ** 121]


@pytest.mark.parametrize("bad", BAD_SCALES)
def test_gather_reads_a_broken_scale_as_one(cuda, bad):
    ctx, bs = [40, 20], 16
    table, n = make_tables(np.random.default_rng(0), ctx, bs, extra_width=0)
    cache, scales = dirty_pool(n, bs, width(F32), 8)
    broken, as_one = scales.clone(), scales.clone()
    broken[table[0, 1]], as_one[table[0, 1]] = bad, 1.0
    want = np.concatenate([O.rows_of(cache, as_one, table, ctx, b, bs) for b in range(2)])
    rows, _, ws = run_gather(F32, cache, broken, table, ctx, bs, 60)
    with pytest.raises(L.MlaError, match="SHAPE"):
        L.mla_check_device_status(ws)
    assert np.array_equal(rows[:60], want, equal_nan=True)


# ------------------------------------------------------------------ decode
def decode_inputs(cfg, ctx, bs, seed, spread=2.0, poison=True):
    """Blocks of normalised rows; everything that no token owns (blocks of no
    request, rows behind the last token, their scales) holds NaN."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    table, n_blocks = make_tables(rng, ctx, bs)
    W, h, B = width(cfg), cfg.num_heads, len(ctx)
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    x = torch.randn(n_blocks, bs, W, generator=g)
    x *= torch.exp2(spread * torch.rand(n_blocks, 1, 1, generator=g))
    e = torch.ceil(torch.log2(x.abs().amax((1, 2)) / 448))
    cache = (x / torch.exp2(e)[:, None, None]).to(FP8).view(torch.uint8)
    scales = torch.exp2(e)
    if poison:
        live = torch.zeros(n_blocks, bs, dtype=torch.bool)
        for b, n in enumerate(ctx):
            for j in range(-(-n // bs)):
                live[table[b, j], :min(bs, n - j * bs)] = True
        cache[~live] = 0x7f
        scales[~live.any(1)] = float("nan")
    q_nope = torch.randn(B, h, cfg.qk_nope_head_dim, generator=g).to(dt)
    q_pe = torch.randn(B, h, cfg.qk_rope_head_dim, generator=g).to(dt)
    w = (torch.randn(h * (cfg.qk_nope_head_dim + cfg.v_head_dim), cfg.kv_lora_rank, generator=g)
         * 0.02).to(dt)
    w_o = (torch.randn(cfg.hidden_size, h * cfg.v_head_dim, generator=g) * 0.02).to(dt)
    return dict(q_nope=q_nope, q_pe=q_pe, w=w, w_o=w_o, cache=cache, scales=scales, table=table,
                ctx=ctx, n_blocks=n_blocks)


def run_decode_paged(cfg, d, bs, with_o=False, check=True, stream=None):
    B, mb = len(d["ctx"]), np.shape(d["table"])[1]
    n, _ = L.mla_decode_paged_workspace_size(cfg, B, mb, bs)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")      # NaN everywhere
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    H = cfg.hidden_size if with_o else cfg.num_heads * cfg.v_head_dim
    out = torch.full((B + 1, H), 9.0, dtype=dt, device="cuda")
    L.mla_decode_paged(cfg, d["q_nope"].cuda(), d["q_pe"].cuda(), d["w"].cuda(),
                       d["cache"].cuda(), d["scales"].cuda(), i32(d["table"]), i32(d["ctx"]), B,
                       mb, d["n_blocks"], bs, d["w_o"].cuda() if with_o else None, out, ws,
                       stream)
    torch.cuda.synchronize()
    if check:
        L.mla_check_device_status(ws)
    assert (out[B] == 9).all()
    return out[:B], ws


def want_decode(cfg, d, bs, with_o=False):
    return O.decode(cfg, d["q_nope"], d["q_pe"], d["w"], d["cache"].numpy(), d["scales"].numpy(),
                    d["table"], d["ctx"], bs, d["w_o"] if with_o else None)


def check_decode(cfg, ctx, bs, seed, with_o=False, **kw):
    d = decode_inputs(cfg, ctx, bs, seed, **kw)
    out, _ = run_decode_paged(cfg, d, bs, with_o)
    want = want_decode(cfg, d, bs, with_o)
    for b, n in enumerate(ctx):
        if n == 0:
            assert (out[b] == 0).all()
    assert oracle.max_rel_err(out, want) <= TOL[cfg.dtype]


@pytest.mark.parametrize("with_o", [False, True])
@pytest.mark.parametrize("bs,ctx", [
    (16, [1]), (16, [0]), (32, [5, 0, 33, 1]), (64, [63, 64, 65, 127, 128, 129]),
    (128, [1000, 0, 2050, 1]), (16, [1024, 1025, 3000])])
def test_decode_f32(cuda, bs, ctx, with_o):
    check_decode(F32, ctx, bs, seed=len(ctx), with_o=with_o)


@pytest.mark.parametrize("B", [1, 7, 8, 9, 128, 129])
def test_decode_f32_output_projection_rows(cuda, B):
    check_decode(F32.with_(hidden_size=40), [(3 * b) % 50 for b in range(B)], 16, seed=B,
                 with_o=True)


@pytest.mark.parametrize("heads", [1, 5, 16, 31, 48, 64, 96, 128])
@pytest.mark.parametrize("bs,ctx", [
    (16, [1, 17, 0, 500]), (64, [127, 128, 129, 64, 1]), (128, [700, 1, 0, 1300])])
def test_decode_bf16(cuda, heads, bs, ctx):
    check_decode(bf16(heads), ctx, bs, seed=heads + bs)


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_decode_bf16_long_and_mixed(cuda, bs):
    check_decode(bf16(128), [20000, 1, 4097, 300], bs, seed=bs)
    check_decode(bf16(16), [30011], bs, seed=bs + 1, with_o=True)


@pytest.mark.parametrize("heads,chunks", [(16, 12), (128, 6)])
def test_decode_bf16_requests_of_one_to_many_partials(cuda, heads, chunks):
    # slices of some `chunks` chunks: request k is cut into about k pieces
    check_decode(bf16(heads), [128 * chunks * k + 5 for k in range(13)] + [1], 64, seed=heads)


@pytest.mark.parametrize("heads", [16, 128])
def test_decode_bf16_many_requests(cuda, heads):
    rng = np.random.default_rng(heads)
    ctx = [int(x) for x in rng.integers(0, 400, 300)]
    check_decode(bf16(heads), ctx, 32, seed=heads)


@pytest.mark.parametrize("cfg", [F32, bf16(16), bf16(65)], ids=["f32", "h16", "h65"])
def test_decode_of_the_most_requests(cuda, cfg):
    rng = np.random.default_rng(3)
    B, bs = 8192, 16
    ctx = [int(x) for x in rng.integers(0, 41, B)]
    d = decode_inputs(cfg, ctx, bs, 3)
    out, _ = run_decode_paged(cfg, d, bs)
    some = sorted(set(rng.integers(0, B, 60).tolist()) | {0, 31, 32, 127, 128, B - 1})
    part = dict(d, q_nope=d["q_nope"][some], q_pe=d["q_pe"][some], table=d["table"][some],
                ctx=[ctx[b] for b in some])
    assert oracle.max_rel_err(out[some], want_decode(cfg, part, bs)) <= TOL[cfg.dtype]
    for b, n in enumerate(ctx):
        assert n or (out[b] == 0).all()


def test_decode_bf16_other_widths_run_on_cuda_cores(cuda):
    cfg = bf16(3, kv_lora_rank=96, qk_rope_head_dim=32, qk_nope_head_dim=24, v_head_dim=40)
    check_decode(cfg, [0, 1, 1500, 64], 32, seed=9)


def test_decode_dsv3_with_output_projection(cuda):
    check_decode(DSV3, [3, 300, 1025], 64, seed=4, with_o=True)


def test_decode_no_tokens_at_all(cuda):
    for cfg in (F32, bf16(128), bf16(4)):
        d = decode_inputs(cfg, [0, 0, 0], 16, 1)
        for with_o in (False, True):
            out, _ = run_decode_paged(cfg, d, 16, with_o)
            assert (out == 0).all()


@pytest.mark.parametrize("heads", [4, 40, 128])
def test_decode_one_dominant_token_over_a_flat_background(cuda, heads):
    """Scores that put half of the weight on one token and spread the other
    half over thousands that all point the same way: small weights count.

    The two halves nearly cancel (0.39 of a row of -1 against 0.61 of rows
    around 0.6), so the error is held against what is summed, not only
    against what is left: a weight rounded to 8 significant bits is off by up
    to 2^-8 of itself, and all equal weights alike, which moves the output by
    up to 2^-8 sum_j p_j |W_UV c_j|."""
    cfg, bs, n = bf16(heads), 64, 9000
    d = decode_inputs(cfg, [n], bs, 3, spread=0.0)
    d["q_nope"].zero_()
    d["q_pe"].zero_()
    d["q_pe"][..., 0] = 8.0
    scale = oracle.softmax_scale(cfg)
    # the key's first rope column decides; e4m3 holds 60 and 0 exactly
    x = torch.randn(d["n_blocks"], bs, width(cfg)) * 0.2 + 0.6
    x[..., 512:] = 0
    blk, row = d["table"][0, 0], 5
    x[blk, row] = -1.0
    x[blk, row, 512] = 15.0                        # score 120 * scale
    assert 8.0 < 120 * scale < np.log(n) + 1
    d["cache"] = (x / 0.125).to(FP8).view(torch.uint8)
    d["scales"] = torch.full((d["n_blocks"],), 0.125)
    out, _ = run_decode_paged(cfg, d, bs)
    want = want_decode(cfg, d, bs)
    rows = O.rows_of(d["cache"].numpy(), d["scales"].numpy(), d["table"], d["ctx"], 0, bs)
    e = np.exp(8.0 * scale * (rows[:, 512] - rows[:, 512].max()))
    w_uv = f64(d["w"]).reshape(heads, 256, 512)[:, 128:]
    summed = max((np.abs(rows[:, :512] @ w_uv[h].T) * (e / e.sum())[:, None]).sum(0).max()
                 for h in range(heads))
    err = np.abs(f64(out) - want).max()
    assert err <= TOL["bf16"] * np.abs(want).max() + 2.0 ** -8 * summed


@pytest.mark.parametrize("cfg", [F32, bf16(24), bf16(128)], ids=["f32", "h24", "h128"])
def test_decode_scores_that_climb(cuda, cfg):
    """The running maximum rises by far more than any fixed margin, in both
    directions of time.

    A score of magnitude S is rounded to fp32 up to 8 times (five additions
    across the lanes, the last of the dot product, the two scalings), S 2^-24 each, and an
    error d of the scores moves a weight by at most 2 d relative to it (its
    own exponential and the normaliser); the few tokens that share the weight
    have rows up to twice as large as their mean.  That is 32 S 2^-24 on top
    of the tolerance for scores near one: 3e-3 at S = 4 * 3000 * 48^-0.5, where
    neighbouring fp32 numbers are 1.2e-4 apart."""
    bs, n = 32, 3000
    tol = TOL[cfg.dtype] + 32 * 4 * n * oracle.softmax_scale(cfg) * 2.0 ** -24
    for sign in (1, -1):
        d = decode_inputs(cfg, [n, 700], bs, 5, spread=0.0)
        r = cfg.kv_lora_rank
        x = torch.randn(d["n_blocks"], bs, width(cfg)) * 0.5
        for b, m in enumerate(d["ctx"]):
            for j in range(m):
                t = j if sign > 0 else m - 1 - j
                x[d["table"][b, j // bs], j % bs, r] = float(t)
        e = torch.ceil(torch.log2(x.abs().amax((1, 2)) / 448))
        d["cache"] = (x / torch.exp2(e)[:, None, None]).to(FP8).view(torch.uint8)
        d["scales"] = torch.exp2(e)
        d["q_pe"][..., 0] = 4.0
        out, _ = run_decode_paged(cfg, d, bs)
        assert oracle.max_rel_err(out, want_decode(cfg, d, bs)) <= tol


@pytest.mark.parametrize("cfg", [F32, bf16(24), bf16(128)], ids=["f32", "h24", "h128"])
def test_decode_block_scales_far_apart(cuda, cfg):
    """Blocks of zeros (scale 2^-64) and of very different magnitudes."""
    bs = 16
    d = decode_inputs(cfg, [400, 130], bs, 6)
    ids = d["table"][0]
    d["cache"][ids[3]] = 0
    d["scales"][ids[3]] = 2.0 ** -64
    d["scales"][ids[7]] = 2.0 ** -30
    d["scales"][ids[9]] = 2.0 ** -2
    d["q_nope"] *= 0.25
    d["q_pe"] *= 0.25
    out, _ = run_decode_paged(cfg, d, bs)
    assert oracle.max_rel_err(out, want_decode(cfg, d, bs)) <= TOL[cfg.dtype]


@pytest.mark.parametrize("cfg", [F32, bf16(24), bf16(128)], ids=["f32", "h24", "h128"])
def test_decode_keeps_nan_in_its_request(cuda, cfg):
    bs = 32
    d = decode_inputs(cfg, [200, 150, 90], bs, 7)
    d["cache"][d["table"][1, 2], 5, 3] = 0x7f
    out, _ = run_decode_paged(cfg, d, bs)
    want = want_decode(cfg, d, bs)
    assert torch.isnan(out[1].float()).all()
    keep = [0, 2]
    assert oracle.max_rel_err(out[keep], want[keep]) <= TOL[cfg.dtype]


@pytest.mark.parametrize("cfg", [F32, bf16(24), bf16(128)], ids=["f32", "h24", "h128"])
def test_decode_reports_what_is_out_of_range(cuda, cfg):
    bs = 16
    good = decode_inputs(cfg, [100, 50, 64], bs, 8, poison=False)
    want = want_decode(cfg, good, bs)
    for kind in ("block", "length", "negative"):
        d = dict(good, table=good["table"].copy(), ctx=list(good["ctx"]))
        if kind == "block":
            d["table"][1, 1] = d["n_blocks"]
        elif kind == "length":
            d["ctx"][1] = d["table"].shape[1] * bs + 1
        else:
            d["ctx"][1] = -4
        out, ws = run_decode_paged(cfg, d, bs, check=False)
        with pytest.raises(L.MlaError, match="SHAPE"):
            L.mla_check_device_status(ws)
        keep = [0, 2]
        assert oracle.max_rel_err(out[keep], want[keep]) <= TOL[cfg.dtype]


@pytest.mark.parametrize("bad", BAD_SCALES)
@pytest.mark.parametrize("cfg", [F32, bf16(24)], ids=["f32", "h24"])
def test_decode_reads_a_broken_scale_as_one(cuda, cfg, bad):
    bs = 16
    d = decode_inputs(cfg, [100, 50, 64], bs, 8, poison=False)
    at = int(d["table"][1, 1])
    g = torch.Generator().manual_seed(9)
    d["cache"][at] = torch.randn(bs, width(cfg), generator=g).to(FP8).view(torch.uint8)
    scales = d["scales"].clone()
    scales[at] = 1.0
    want = want_decode(cfg, dict(d, scales=scales), bs)
    scales = scales.clone()
    scales[at] = bad
    out, ws = run_decode_paged(cfg, dict(d, scales=scales), bs, check=False)
    with pytest.raises(L.MlaError, match="SHAPE"):
        L.mla_check_device_status(ws)
    assert oracle.max_rel_err(out, want) <= TOL[cfg.dtype]


def test_decode_shares_blocks_between_requests(cuda):
    """Two requests whose tables name the same prefix blocks."""
    cfg, bs = bf16(16), 32
    d = decode_inputs(cfg, [320, 300], bs, 10, poison=False)
    d["table"][1, :5] = d["table"][0, :5]
    out, _ = run_decode_paged(cfg, d, bs)
    assert oracle.max_rel_err(out, want_decode(cfg, d, bs)) <= TOL["bf16"]


def test_decode_is_deterministic(cuda):
    cfg = bf16(128)
    d = decode_inputs(cfg, [5000, 77, 1200], 64, 11)
    a, _ = run_decode_paged(cfg, d, 64)
    b, _ = run_decode_paged(cfg, d, 64)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_offsets_beyond_32_bits(cuda):
    """Block ids whose byte offset passes 2^32 (a pool of 4.8 GB)."""
    cfg, bs = bf16(16), 64
    W, n_blocks = width(cfg), 130000
    assert n_blocks * bs * W > 2 ** 32
    cache = torch.zeros(n_blocks, bs, W, dtype=torch.uint8, device="cuda")
    scales = torch.ones(n_blocks, device="cuda")
    ids = [n_blocks - 1, 3, n_blocks - 2, 116600, 58300]
    n = 5 * bs - 7
    rows = random_rows(n, W, torch.bfloat16, 12)
    slots = [ids[j // bs] * bs + j % bs for j in range(n)]
    ws = paged_ws(n_blocks)
    L.mla_paged_append(cfg, rows.cuda(), i32(slots), cache, scales, n, n_blocks, bs, ws)
    L.mla_check_device_status(ws)
    small = cache[torch.tensor(ids).cuda()].cpu().numpy()
    ssc = scales[torch.tensor(ids).cuda()].cpu().numpy()
    want, wsc = O.append(rows, list(range(n)), np.zeros((5, bs, W), np.uint8), np.ones(5), bs)
    assert np.array_equal(ssc, wsc) and np.array_equal(O.E4M3[small], O.E4M3[want])
    got = torch.empty(n, W, dtype=torch.bfloat16, device="cuda")
    cu = torch.empty(2, dtype=torch.int32, device="cuda")
    L.mla_paged_gather(cfg, cache, scales, i32([ids]), i32([n]), got, cu, 1, 5, n_blocks, bs, n,
                       ws)
    L.mla_check_device_status(ws)
    assert np.array_equal(f64(got), O.rows_of(small, ssc, [list(range(5))], [n], 0, bs))
    d = decode_inputs(cfg, [n], bs, 13)
    d.update(table=np.array([ids]), n_blocks=n_blocks, cache=cache, scales=scales)
    out, _ = run_decode_paged(cfg, d, bs)
    d.update(table=np.array([list(range(5))]), cache=torch.from_numpy(small),
             scales=torch.from_numpy(ssc))
    assert oracle.max_rel_err(out, want_decode(cfg, d, bs)) <= TOL["bf16"]


# ------------------------------------------------------------- all together
def serve(cfg, steps, B, bs, n_blocks, seed, stream=None):
    """Requests that come, grow and leave: plan, append, decode and gather of
    every step against the oracle's own state."""
    rng = np.random.default_rng(seed)
    W, h = width(cfg), cfg.num_heads
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    pc = MlaPagedCache(cfg, B, max_blocks=24, n_blocks=n_blocks, block_size=bs, capacity=600)
    pc.cache.view(torch.uint8).fill_(0x7f)
    table, ring = pc.table.cpu().numpy(), pc.ring.cpu().numpy()
    ctx, state = np.zeros(B, int), np.array([0, n_blocks])
    cache = pc.cache.view(torch.uint8).cpu().numpy()
    scales = np.ones(n_blocks)
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(h * (cfg.qk_nope_head_dim + cfg.v_head_dim), cfg.kv_lora_rank, generator=g)
         * 0.02).to(dt)
    for step in range(steps):
        new = np.where(rng.random(B) < 0.15, -1, np.where(ctx == 0, rng.integers(0, 90, B), 1))
        want = O.plan(ctx, new, table, ring, state, bs, 600)
        assert want["status"] == "ok"
        total = int(want["cu"][-1])
        rows = random_rows(600, W, dt, seed + step)
        q_nope = torch.randn(B, h, cfg.qk_nope_head_dim, generator=g).to(dt)
        q_pe = torch.randn(B, h, cfg.qk_rope_head_dim, generator=g).to(dt)
        dev = [i32(new), rows.cuda(), q_nope.cuda(), q_pe.cuda(), w.cuda()]
        out = torch.empty(B, h * cfg.v_head_dim, dtype=dt, device="cuda")
        got = torch.zeros(4096, W, dtype=dt, device="cuda")
        cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(stream) if stream else torch.cuda.stream(None):
            pc.plan(dev[0])
            pc.append(dev[1])                     # rows behind the last token have slot -1
            pc.decode(*dev[2:], out)
            pc.gather(got, cu)
        torch.cuda.synchronize()
        pc.check_status()
        table, ring, state, ctx = want["table"], want["ring"], want["state"], want["ctx"]
        cache, scales = O.append(rows, want["slots"], cache, scales, bs)
        assert np.array_equal(pc.table.cpu().numpy(), table)
        assert np.array_equal(pc.ctx.cpu().numpy(), ctx)
        assert np.array_equal(pc.scales.cpu().numpy(), scales)
        want_rows = np.concatenate([O.rows_of(cache, scales, table, ctx, b, bs)
                                    for b in range(B)])
        assert np.array_equal(f64(got)[:len(want_rows)], want_rows)
        assert total <= 600
        ref = O.decode(cfg, q_nope, q_pe, w, cache, scales, table, ctx, bs)
        assert oracle.max_rel_err(out, ref) <= TOL[cfg.dtype]


@pytest.mark.parametrize("cfg", [F32, bf16(16), bf16(128)], ids=["f32", "h16", "h128"])
def test_serving_steps(cuda, cfg):
    serve(cfg, steps=6, B=7, bs=16, n_blocks=150, seed=21)


def test_serving_steps_on_another_stream(cuda):
    serve(bf16(16), steps=3, B=5, bs=32, n_blocks=80, seed=22, stream=torch.cuda.Stream())


@pytest.mark.parametrize("cfg", [F32, bf16(16), bf16(128)], ids=["f32", "h16", "h128"])
def test_a_captured_step_follows_its_inputs(cuda, cfg):
    """plan + append + decode captured once and replayed: lengths, rows and
    queries of every replay are read from the device."""
    B, bs, W, h = 4, 16, width(cfg), cfg.num_heads
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32

    def fresh():
        return MlaPagedCache(cfg, B, max_blocks=12, n_blocks=60, block_size=bs, capacity=64)
    g = torch.Generator().manual_seed(31)
    w = (torch.randn(h * (cfg.qk_nope_head_dim + cfg.v_head_dim), cfg.kv_lora_rank, generator=g)
         * 0.02).to(dt).cuda()
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = torch.zeros(64, W, dtype=dt, device="cuda")
    qn = torch.zeros(B, h, cfg.qk_nope_head_dim, dtype=dt, device="cuda")
    qp = torch.zeros(B, h, cfg.qk_rope_head_dim, dtype=dt, device="cuda")
    out = torch.zeros(B, h * cfg.v_head_dim, dtype=dt, device="cuda")

    def step(pc):
        pc.plan(new)
        pc.append(rows)
        pc.decode(qn, qp, w, out)

    warm = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    graphed, eager = fresh(), fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for i, lens in enumerate(([20, 0, 3, 33], [1, 5, 1, 1], [1, 1, -1, 1], [1, 1, 30, -1])):
        new.copy_(i32(lens))
        rows.copy_(random_rows(64, W, dt, 40 + i))
        qn.copy_(torch.randn(qn.shape, generator=g))
        qp.copy_(torch.randn(qp.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        graphed.check_status()
        first = out.clone()
        step(eager)
        torch.cuda.synchronize()
        eager.check_status()
        assert torch.equal(first, out)
        assert torch.equal(graphed.ctx, eager.ctx) and torch.equal(graphed.table, eager.table)
        live = O.rows_of  # the two pools hold the same live rows
        for b in range(B):
            a = live(u8(graphed.cache), graphed.scales.cpu().numpy(),
                     graphed.table.cpu().numpy(), graphed.ctx.cpu().numpy(), b, bs)
            e = live(u8(eager.cache), eager.scales.cpu().numpy(), eager.table.cpu().numpy(),
                     eager.ctx.cpu().numpy(), b, bs)
            assert np.array_equal(a, e)
    del graph


def test_gathered_rows_feed_the_contiguous_paths(cuda):
    """gather -> mla_decode_absorbed gives what mla_decode_paged gives."""
    cfg, bs, ctx = bf16(128), 64, [100, 700, 1, 64]
    d = decode_inputs(cfg, ctx, bs, 14)
    paged, _ = run_decode_paged(cfg, d, bs)
    n = sum(ctx)
    rows = torch.empty(n, width(cfg), dtype=torch.bfloat16, device="cuda")
    cu = torch.empty(len(ctx) + 1, dtype=torch.int32, device="cuda")
    ws = paged_ws(d["n_blocks"])
    L.mla_paged_gather(cfg, d["cache"].cuda(), d["scales"].cuda(), i32(d["table"]), i32(ctx),
                       rows, cu, len(ctx), d["table"].shape[1], d["n_blocks"], bs, n, ws)
    dec = MlaDecode(cfg, len(ctx), 1024)
    out = torch.empty_like(paged)
    dec(d["q_nope"].cuda(), d["q_pe"].cuda(), d["w"].cuda(), rows, cu, out)
    torch.cuda.synchronize()
    dec.check_status()
    assert oracle.max_rel_err(paged, out) <= TOL["bf16"]


def test_two_calls_at_once_on_workspaces_of_their_own(cuda):
    cfg, bs = bf16(16), 32
    ds = [decode_inputs(cfg, c, bs, 50 + i) for i, c in enumerate(([900, 40], [333, 2000]))]
    alone = [run_decode_paged(cfg, d, bs)[0] for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    outs, keep = [], []
    for d, st in zip(ds, streams):
        B, mb = len(d["ctx"]), d["table"].shape[1]
        n, _ = L.mla_decode_paged_workspace_size(cfg, B, mb, bs)
        a = [d["q_nope"].cuda(), d["q_pe"].cuda(), d["w"].cuda(), d["cache"].cuda(),
             d["scales"].cuda(), i32(d["table"]), i32(d["ctx"])]
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        out = torch.empty(B, cfg.num_heads * cfg.v_head_dim, dtype=torch.bfloat16, device="cuda")
        outs.append(out)
        keep.append((a, ws, B, mb, d["n_blocks"]))
    torch.cuda.synchronize()
    for (a, ws, B, mb, nb), out, st in zip(keep, outs, streams):
        L.mla_decode_paged(cfg, *a, B, mb, nb, bs, None, out, ws, st)
    torch.cuda.synchronize()
    for out, ref in zip(outs, alone):
        assert torch.equal(out, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_aligned_to_16_bytes_only(cuda, dtype):
    cfg = bf16(2) if dtype == "bf16" else F32
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    W, bs, n = width(cfg), 32, 100
    off = 16 // dt.itemsize
    buf = torch.empty(n * W + off, dtype=dt, device="cuda")
    rows = buf[off:].view(n, W)
    assert rows.data_ptr() % 32 == 16
    host = random_rows(n, W, dt, 3)
    rows.copy_(host)
    cache, scales = dirty_pool(6, bs, W, 9)
    c, s, ws = cache.cuda(), scales.cuda(), paged_ws(6)
    slots = list(range(5, 5 + n))
    L.mla_paged_append(cfg, rows, i32(slots), c, s, n, 6, bs, ws)
    L.mla_check_device_status(ws)
    want, wsc = O.append(host, slots, cache.numpy(), scales.numpy(), bs)
    assert np.array_equal(s.cpu().numpy(), wsc)
    assert np.array_equal(O.E4M3[c.cpu().numpy()], O.E4M3[want])
    cu = torch.empty(2, dtype=torch.int32, device="cuda")
    L.mla_paged_gather(cfg, c, s, i32([[0, 1, 2, 3, 4, 5]]), i32([n]), rows, cu, 1, 6, 6, bs, n, ws)
    L.mla_check_device_status(ws)
    assert np.array_equal(f64(rows), O.rows_of(want, wsc, [[0, 1, 2, 3, 4, 5]], [n], 0, bs))


@pytest.mark.parametrize("capacity", [2048, 2049, 30000])
def test_plan_on_either_side_of_one_block(cuda, capacity):
    rng = np.random.default_rng(capacity)
    ctx = rng.integers(0, 700, 9)
    new = np.array([capacity // 9] * 8 + [-1])
    table, ring, state, _ = pool_state(rng, ctx, 16, capacity // 16 + 20, 300)
    assert check_plan(ctx, new, table, ring, state, 16, capacity, in_place=True)["status"] == "ok"
    check_plan(ctx, new, table, ring, [state[0], 3], 16, capacity, in_place=True)


@pytest.mark.parametrize("dn,dv,B", [(128, 128, 33), (64, 192, 5), (200, 72, 130), (8, 8, 300),
                                     (264, 264, 40)])
def test_decode_head_widths_and_batches(cuda, dn, dv, B):
    """Nope and value widths either side of 128, batches either side of a
    round and of a block of the projections."""
    cfg = bf16(3, qk_nope_head_dim=dn, v_head_dim=dv, softmax_scale=0.07)
    rng = np.random.default_rng(B)
    check_decode(cfg, [int(x) for x in rng.integers(0, 300, B)], 16, seed=dn + dv)


def test_decode_zero_and_huge_queries(cuda):
    cfg = bf16(20)
    d = decode_inputs(cfg, [300, 200, 100], 32, 15)
    d["q_nope"][0] = 0
    d["q_pe"][0] = 0
    d["q_nope"][1] *= 2.0 ** 40
    d["q_pe"][1] *= 2.0 ** 40
    d["q_nope"][2, 3, 5] = float("inf")
    out, _ = run_decode_paged(cfg, d, 32)
    want = want_decode(cfg, d, 32)
    assert torch.isnan(out[2].view(20, 128)[3].float()).all()
    keep = [0, 2]
    w = np.nan_to_num(want.reshape(3, 20, 128)[keep])
    o = torch.nan_to_num(out.view(3, 20, 128)[keep].float())
    w[1, 3] = 0
    o[1, 3] = 0
    assert oracle.max_rel_err(o, w) <= TOL["bf16"]
    # at 2^40 one token takes all of the weight: a row of the cache, through W_UV
    assert torch.isfinite(out[1].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_runs,rows_max", [(700, 1), (1500, 5), (4500, 1), (300, 9)])
def test_append_of_many_short_runs(cuda, dtype, n_runs, rows_max):
    """The new tokens of many requests: runs of a few rows, several a window,
    with and without kept rows, some windows with a long one among them."""
    cfg = bf16(2) if dtype == "bf16" else F32
    rng = np.random.default_rng(n_runs)
    bs = 16
    runs = [(int(rng.integers(0, bs - rows_max + 1)), int(rng.integers(1, rows_max + 1)))
            for _ in range(n_runs)]
    runs[5] = (0, bs)
    slots = slots_for(rng, n_runs + 3, bs, runs)
    slots[-1] = -1
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    check_append(cfg, random_rows(len(slots), width(cfg), dt, n_runs), slots,
                 *dirty_pool(n_runs + 3, bs, width(cfg), 11), bs)


def test_append_refuses_a_second_run_among_many(cuda):
    """Below and above the count from which blocks are claimed by a bit."""
    for n in (300, 4600):
        slots = [16 * i for i in range(n)]
        slots[n - 2] = 16 * 7 + 3
        cache, scales = dirty_pool(n, 16, width(F32), 12)
        rows = random_rows(n, width(F32), torch.float32, 13)
        got, sc, ws = run_append(F32, rows, slots, cache, scales, 16)
        with pytest.raises(L.MlaError, match="SHAPE"):
            L.mla_check_device_status(ws)
        L.mla_check_device_status(ws)               # read once
        ok = [i for i in range(n) if i not in (7, n - 2)]
        want, wsc = O.append(rows[ok], [slots[i] for i in ok], cache.numpy(), scales.numpy(), 16)
        idx = [slots[i] // 16 for i in ok]
        assert np.array_equal(sc[idx], wsc[idx])
        assert np.array_equal(O.E4M3[got[idx]], O.E4M3[want[idx]])


@pytest.mark.parametrize("heads,hidden,B", [(1, 8, 1), (3, 136, 17), (16, 1000, 130), (128, 264, 5),
                                            (5, 4096, 96), (40, 512, 300)])
def test_decode_output_projection_shapes(cuda, heads, hidden, B):
    """Tiles, pieces of K and batches that end inside a block."""
    cfg = bf16(heads, hidden_size=hidden)
    rng = np.random.default_rng(B)
    check_decode(cfg, [int(x) for x in rng.integers(0, 60, B)], 16, seed=heads, with_o=True)


def test_decode_other_widths_with_output_projection(cuda):
    cfg = bf16(3, kv_lora_rank=96, qk_rope_head_dim=32, qk_nope_head_dim=24, v_head_dim=40,
               hidden_size=120)
    check_decode(cfg, [0, 70, 300], 32, seed=9, with_o=True)


@pytest.mark.parametrize("cfg", [F32, bf16(16)], ids=["f32", "h16"])
def test_two_captured_graphs_share_a_workspace(cuda, cfg):
    bs = 16
    ds = [decode_inputs(cfg, ctx, bs, i) for i, ctx in enumerate(([700, 3, 0], [90] * 40))]
    dev = [{k: v.cuda() for k, v in d.items() if torch.is_tensor(v)} for d in ds]
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    size = max(L.mla_decode_paged_workspace_size(cfg, len(d["ctx"]), d["table"].shape[1], bs)[0]
               for d in ds)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for d, g in zip(ds, dev):
        B, tb, cx = len(d["ctx"]), i32(d["table"]), i32(d["ctx"])
        out = torch.zeros(B, cfg.num_heads * cfg.v_head_dim, dtype=dt, device="cuda")
        call = lambda: L.mla_decode_paged(cfg, g["q_nope"], g["q_pe"], g["w"], g["cache"],
                                          g["scales"], tb, cx, B, tb.shape[1], d["n_blocks"], bs,
                                          None, out, ws)
        call()
        torch.cuda.synchronize()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, tb, cx))
        outs.append((out, want))
    for i in (0, 1, 1, 0, 1, 0):
        outs[i][0].zero_()
        graphs[i][0].replay()
        torch.cuda.synchronize()
        L.mla_check_device_status(ws)
        assert torch.equal(outs[i][0], outs[i][1])
