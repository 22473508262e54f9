"""The precision that ``mla.h`` states for the tensor-core paged decode, held
elementwise where it shows: neighbouring blocks whose scales lie far apart.

With t_j = p_j 2^e_j (weight times block scale, relative to any common factor)
and M the largest t of the 32 tokens that j stands with, what multiplies the
bytes b_j is off by at most (2^-8 + 2^-11) t_j + 2^-17 M, so

  |d o_lat| <= sum_j ((2^-8 + 2^-11) t_j + 2^-17 M_j) |b_j|  / sum_j p_j.

On top: o_lat as two bf16 terms, each rounded to nearest (2^-8 of what it
rounds): 2^-16; fp32 scores and exponentials below 2^-18 of a weight (scores up to 4,
a handful of roundings of 2^-24 each, and ex2's 2^-22); sums of up to 1024 fp32
terms, 2^-24 each at most: 2^-14.  All relative to sum_j p_j |c_j|, through
|W_UV|.  The output is rounded to bf16, 2^-8 of it."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import f64
from oracle import paged as O
from test_gpu_paged import FP8, bf16, decode_inputs, run_decode_paged, want_decode, width

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gap", [0, 4, 9, 12, 16, 20, 30])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("heads", [4, 24, 40, 128])
def test_blocks_of_scales_far_apart(cuda, heads, bs, gap):
    """Every other block is 2^-gap of its neighbours and alone fills the upper
    half of the latent dims, which the upper half of W_UV reads."""
    cfg, n = bf16(heads, softmax_scale=0.05), 400
    d = decode_inputs(cfg, [n], bs, gap, poison=False)
    g = torch.Generator().manual_seed(gap + heads)
    nb = d["n_blocks"]
    x = (torch.rand(nb, bs, width(cfg), generator=g) + 0.5) * 100
    x = x.to(FP8).float()
    small = torch.zeros(nb, dtype=torch.bool)
    small[torch.from_numpy(d["table"][0, 1:-(-n // bs):2])] = True
    x[small, :, :256] = 0
    x[~small, :, 256:512] = 0
    # scores: 10 q k with k in [0, 8) steps of 1 (x 2^gap where the scale is 2^-gap)
    k = torch.randint(0, 8, (nb, bs), generator=g).float()
    x[..., 512:] = 0
    x[~small, :, 512] = k[~small]
    x[small, :, 513] = k[small]
    d["cache"] = x.to(FP8).view(torch.uint8)
    d["scales"] = torch.where(small, 2.0 ** -gap, 1.0)
    d["q_nope"].zero_()
    d["q_pe"].zero_()
    d["q_pe"][..., 0] = 10.0
    d["q_pe"][..., 1] = 10.0
    w = d["w"].view(heads, 256, 512)
    w[:, 128:192, 256:] = 0
    w[:, 192:, :256] = 0
    out, _ = run_decode_paged(cfg, d, bs)
    want = want_decode(cfg, d, bs).reshape(heads, 128)

    rows = O.rows_of(d["cache"].numpy(), d["scales"].numpy(), d["table"], [n], 0, bs)
    s = 10.0 * oracle.softmax_scale(cfg) * (rows[:, 512] + rows[:, 513])
    p = np.exp(s - s.max())
    e = d["scales"].numpy()[d["table"][0, np.arange(n) // bs]]
    t = p * e
    most = np.array([t[32 * (j // 32):32 * (j // 32) + 32].max() for j in range(n)])
    b = np.abs(rows[:, :512]) / e[:, None]
    eps = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16 + 2.0 ** -18 + 2.0 ** -14
    d_lat = ((eps * t + 2.0 ** -17 * most) @ b) / p.sum()
    w_uv = np.abs(f64(w)[:, 128:])
    bound = w_uv @ d_lat + 2.0 ** -8 * np.abs(want)
    err = np.abs(f64(out).reshape(heads, 128) - want)
    assert (err <= bound).all(), (err / bound).max()


def eight_bits(q):
    """A vector as two e4m3 terms and a power of two."""
    e = np.ceil(np.log2(np.abs(q).max() / 448))
    s = q / 2.0 ** e
    hi = O.E4M3[O.to_e4m3(s)]
    return (hi + O.E4M3[O.to_e4m3(s - hi)]) * 2.0 ** e


@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("heads,dn,dv", [(3, 128, 128), (17, 64, 72), (5, 200, 136)])
def test_scores_of_hundreds(cuda, heads, dn, dv, bs):
    """Where scores reach hundreds the query's 8 significant bits decide what the
    weights are: the output is that of the stated query, to the tolerance of the
    other bf16 decodes (the weights' rounding 2^-8, the output's 2^-8, and fp32
    scores: 400 2^-24 a rounding)."""
    cfg = bf16(heads, qk_nope_head_dim=dn, v_head_dim=dv, softmax_scale=0.15)
    ctx = [700, 1, 90, 333]
    d = decode_inputs(cfg, ctx, bs, heads, spread=5.0)
    d["q_nope"] *= 4
    d["q_pe"] *= 4
    out, _ = run_decode_paged(cfg, d, bs)
    w = f64(d["w"]).reshape(heads, dn + dv, 512)
    want, top = np.zeros((len(ctx), heads, dv)), 0.0
    for b in range(len(ctx)):
        c = O.rows_of(d["cache"].numpy(), d["scales"].numpy(), d["table"], ctx, b, bs)
        for h in range(heads):
            q = np.concatenate([f64(d["q_nope"])[b, h] @ w[h, :dn], f64(d["q_pe"])[b, h]])
            s = cfg.softmax_scale * (c @ eight_bits(q))
            top = max(top, np.abs(s).max())
            p = np.exp(s - s.max())
            want[b, h] = w[h, dn:] @ ((p / p.sum()) @ c[:, :512])
    assert top > 100
    assert oracle.max_rel_err(out, want.reshape(len(ctx), -1)) <= 2e-2
