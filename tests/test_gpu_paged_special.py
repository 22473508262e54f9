"""Infinities and NaN in the paged decode's weights and queries: they reach what
the formula multiplies them with, and nothing else."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import TOL, f64
from test_gpu_paged import F32, bf16, decode_inputs, run_decode_paged, want_decode

pytestmark = pytest.mark.gpu


def head_rows(cfg, head, up):
    """Rows of w_kv_b of a head's W_UK (up: W_UV)."""
    a = head * (cfg.qk_nope_head_dim + cfg.v_head_dim)
    b = a + cfg.qk_nope_head_dim
    return (b, b + cfg.v_head_dim) if up else (a, b)


CASES = [F32] + [bf16(3, qk_nope_head_dim=dn, v_head_dim=dv, softmax_scale=0.07)
                 for dn, dv in ((128, 128), (64, 192), (8, 8), (200, 72), (136, 40))]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cfg", CASES, ids=lambda c: f"{c.dtype}-{c.qk_nope_head_dim}-{c.v_head_dim}")
def test_a_weight_that_is_no_number_stays_in_its_column(cuda, cfg, bad):
    """A W_UV value spoils the output column that it belongs to (of a request
    without tokens too: 0 times it); a W_UK value its head."""
    ctx = [70, 0, 300, 5]
    live = [b for b, n in enumerate(ctx) if n]
    h, dv = cfg.num_heads, cfg.v_head_dim
    for up in (True, False):
        d = decode_inputs(cfg, ctx, 32, 3)
        clean = want_decode(cfg, d, 32).reshape(len(ctx), h, dv)
        first, last = head_rows(cfg, 1, up)
        for row in (first, last - 1):
            e = dict(d, w=d["w"].clone())
            e["w"][row, 7] = bad
            out, _ = run_decode_paged(cfg, e, 32)
            got = f64(out).reshape(len(ctx), h, dv)
            spoilt = np.zeros(got.shape, bool)
            if up:
                spoilt[:, 1, row - first] = True
            else:
                spoilt[live, 1] = True
            assert not np.isfinite(got[spoilt]).any()
            assert oracle.max_rel_err(np.where(spoilt, 0, got), np.where(spoilt, 0, clean)) \
                <= TOL[cfg.dtype]
            assert (got[1][~spoilt[1]] == 0).all()
