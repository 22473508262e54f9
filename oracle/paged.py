"""fp64 oracle of the paged 8-bit latent cache: plan, append, gather, decode.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Blocks hold e4m3
bytes and one power-of-two scale; a request's token j lies in row
j % block_size of block table[b][j // block_size].  Pinned by
tests/test_paged_cpu.py: the e4m3 table against the format's definition, the
rounding against exhaustive nearest values, the plan against conservation of
blocks.
"""
import numpy as np

from .mla_oracle import _f64, decode_absorbed

MIN_EXP = -64


def _e4m3_table():
    t = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        t[b] = np.nan if (b & 127) == 127 else (-v if s else v)
    return t


E4M3 = _e4m3_table()


def to_e4m3(x):
    """Bytes of the nearest e4m3 values (ties to even) of |x| <= 464; NaN gives
    0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isnan(x), 0.0, np.abs(x))
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    q = np.rint(a / 2.0 ** (e - 3))                # rint: ties to even
    e, q = np.where(q == 16, e + 1, e), np.where(q == 16, 8, q)
    byte = np.where(q < 8, q, (e + 7) * 8 + (q - 8)).astype(np.int64)
    assert (byte <= 0x7e).all()
    byte = byte + np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7f, byte).astype(np.uint8)


def scale_exp(amax):
    """Smallest e >= MIN_EXP with amax <= 448 * 2^e."""
    e = MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def plan(ctx, new, table, ring, state, block_size, capacity):
    """One step on copies of the inputs.  Returns a dict of every output and
    ``ok``, or None in ``ok``'s place of a step that did not happen."""
    ctx, new = [int(x) for x in ctx], [int(x) for x in new]
    table, ring = np.array(table), np.array(ring)
    head, count = int(state[0]), int(state[1])
    n_blocks, width = len(ring), table.shape[1]
    blocks = lambda n: -(-n // block_size)
    broken = not (0 <= head < n_blocks and 0 <= count <= n_blocks)
    take, give, total = 0, 0, 0
    bad_id = lambda v: not 0 <= int(v) < n_blocks
    ids = []                                       # of blocks given back or filled further
    for b, (c, n) in enumerate(zip(ctx, new)):
        if c < 0 or n < -1 or blocks(c + max(n, 0)) > width:
            broken = True
            continue
        take += 0 if n < 0 else blocks(c + n) - blocks(c)
        give += blocks(c) if n < 0 else 0
        total += max(n, 0)
        ids += list(table[b, :blocks(c)]) if n < 0 else \
            [table[b, c // block_size]] if n > 0 and c % block_size else []
    broken = broken or count + give > n_blocks
    short = take > count or total > capacity
    if not broken and not short:
        ids += [ring[(head + i) % n_blocks] for i in range(take)]
        broken = any(bad_id(v) for v in ids)
    res = dict(table=table, ring=ring, ctx=np.array(ctx), state=np.array([head, count]),
               cu=np.zeros(len(ctx) + 1, np.int64), slots=np.full(capacity, -1, np.int64),
               pos=np.zeros(capacity, np.int64),
               status="shape" if broken else "blocks" if short else "ok")
    if broken or short:
        return res
    taken, back = head, head + count
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        if n < 0:
            for j in range(blocks(c)):
                ring[back % n_blocks] = table[b, j]
                back += 1
            res["ctx"][b] = 0
        else:
            for j in range(blocks(c), blocks(c + n)):
                table[b, j] = ring[taken % n_blocks]
                taken += 1
            for p in range(c, c + n):
                res["slots"][at] = table[b, p // block_size] * block_size + p % block_size
                res["pos"][at] = p
                at += 1
            res["ctx"][b] = c + n
        res["cu"][b + 1] = at
    res["state"] = np.array([taken % n_blocks, count - take + give])
    return res


def append(rows, slots, cache, scales, block_size):
    """Bytes and scales after the append (valid slot maps only)."""
    rows, slots = _f64(rows), [int(s) for s in slots]
    cache, scales = np.array(cache), np.array(scales, dtype=np.float64)
    i = 0
    while i < len(slots):
        if slots[i] < 0:
            i += 1
            continue
        blk, off, k = slots[i] // block_size, slots[i] % block_size, i + 1
        while k < len(slots) and slots[k] == slots[k - 1] + 1 and slots[k] // block_size == blk:
            k += 1
        run = rows[i:k]
        fin = np.abs(run[np.isfinite(run)])
        e = scale_exp(fin.max() if fin.size else 0.0)
        if off:
            old = int(np.log2(scales[blk]))
            e = max(e, old)
            if e != old:
                cache[blk, :off] = to_e4m3(E4M3[cache[blk, :off]] * 2.0 ** (old - e))
        v = np.where(np.isfinite(run), run, np.nan)
        cache[blk, off:off + k - i] = to_e4m3(v * 2.0 ** -e)
        scales[blk] = 2.0 ** e
        i = k
    return cache, scales


def rows_of(cache, scales, table, ctx, b, block_size):
    """Latent rows of request b, [ctx_b, W]."""
    n = int(ctx[b])
    ids = np.asarray(table)[b, :-(-n // block_size)].astype(np.int64)
    v = E4M3[np.asarray(cache)[ids]] * np.asarray(scales, dtype=np.float64)[ids][:, None, None]
    return v.reshape(-1, v.shape[-1])[:n] if n else np.zeros((0, np.asarray(cache).shape[-1]))


def decode(cfg, q_nope, q_pe, w_kv_b, cache, scales, table, ctx, block_size, w_o=None):
    """Weight-absorbed decode over the blocks; a request without tokens gives
    a zero row."""
    out = []
    width = cfg.hidden_size if w_o is not None else cfg.num_heads * cfg.v_head_dim
    qn, qp = _f64(q_nope), _f64(q_pe)
    for b in range(len(ctx)):
        rows = rows_of(cache, scales, table, ctx, b, block_size)
        if not len(rows):
            out.append(np.zeros(width))
            continue
        out.append(decode_absorbed(cfg, qn[b:b + 1], qp[b:b + 1], w_kv_b, rows, [0, len(rows)],
                                   w_o)[0])
    return np.stack(out)
