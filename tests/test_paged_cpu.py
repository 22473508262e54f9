"""The paged 8-bit latent cache without a GPU: the oracle's pins, the entry
points' refusals (nothing is launched) and the binding's checks."""
import ctypes as C

import numpy as np
import pytest
import torch

import latent_attention_b200 as P
from latent_attention_b200._lib import mla_paged_layout
from mla_inputs import WORKLOADS, MlaConfig
from oracle import paged as O

BF16 = WORKLOADS["dsv3_decode"].cfg
F32 = WORKLOADS["tiny_f32"].cfg


# ------------------------------------------------------------------ oracle
def test_e4m3_table_is_the_format():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(O.E4M3))
    assert np.array_equal(np.nan_to_num(t), np.nan_to_num(O.E4M3))


def test_rounding_takes_the_nearest_value_ties_to_even():
    vals = np.unique(np.nan_to_num(O.E4M3[:127]))
    mids = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([vals, mids, mids * (1 + 2.0 ** -40), mids * (1 - 2.0 ** -40)])
    x = np.concatenate([x, -x])
    got = O.E4M3[O.to_e4m3(x)]
    near = np.abs(x[:, None] - np.concatenate([vals, -vals])[None]).min(1)
    assert np.array_equal(np.abs(got - x), near)
    bytes_ = O.to_e4m3(mids)
    assert (bytes_ % 2 == 0).all()                  # a tie goes to the even mantissa
    assert O.to_e4m3(np.nan) == 0x7f


def test_scale_exponent_is_the_smallest():
    for a in (0.0, 1.0, 448.0, 448.5, 447.0, 1e-30, 2.0 ** 100, 1.75, 1.7500001):
        e = O.scale_exp(a)
        assert a <= 448 * 2.0 ** e and (e == O.MIN_EXP or a > 448 * 2.0 ** (e - 1))


def test_plan_conserves_blocks():
    rng = np.random.default_rng(3)
    n_blocks, width, bs, B = 40, 9, 16, 6
    table, ring, ctx = np.full((B, width), -1), rng.permutation(n_blocks), np.zeros(B, int)
    state = np.array([5, n_blocks])
    for _ in range(60):
        new = np.array([-1 if rng.random() < 0.2 else rng.integers(0, 40) for _ in range(B)])
        r = O.plan(ctx, new, table, ring, state, bs, 1000)
        if r["status"] != "ok":
            assert np.array_equal(r["table"], table) and np.array_equal(r["ring"], ring)
            new = np.full(B, -1)
            r = O.plan(ctx, new, table, ring, state, bs, 1000)
        ctx, table, ring, state = r["ctx"], r["table"], r["ring"], r["state"]
        held = [table[b, j] for b in range(B) for j in range(-(-ctx[b] // bs))]
        free = [ring[(state[0] + i) % n_blocks] for i in range(state[1])]
        assert sorted(held + free) == list(range(n_blocks))
        slots = r["slots"][:r["cu"][-1]]
        assert len(set(slots.tolist())) == len(slots)


# ------------------------------------------------------- refusals, C ABI
@pytest.fixture(scope="module")
def lib():
    import os
    from latent_attention_b200 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def _p(a):
    return C.c_void_p(a)


A = 0x100000
BIG = C.c_size_t(1 << 40)


def plan_args(**kw):
    a = dict(ctx=_p(A), new=_p(A), table=_p(A), ring=_p(A), state=_p(A), ctx_out=_p(A),
             state_out=_p(A), slots=_p(A), pos=_p(A), cu=_p(A), B=4, max_blocks=8, n_blocks=32,
             bs=16, capacity=64, ws=_p(A), ws_bytes=BIG, stream=_p(0))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=_p(0)), 1), (dict(slots=_p(0)), 1), (dict(ws=_p(0)), 1), (dict(cu=_p(0)), 1),
    (dict(bs=48), 2), (dict(bs=0), 2), (dict(B=0), 2), (dict(B=8193), 2),
    (dict(max_blocks=0), 2), (dict(max_blocks=1 << 28), 2), (dict(n_blocks=0), 2),
    (dict(n_blocks=1 << 27), 2), (dict(capacity=-1), 2), (dict(capacity=(1 << 30) + 1), 2),
    (dict(capacity=(1 << 31) - 1), 2), (dict(table=_p(A + 2)), 3),
    (dict(ws=_p(A + 16)), 3), (dict(ws_bytes=C.c_size_t(255)), 5)])
def test_plan_refuses(lib, kw, status):
    assert lib.mla_paged_plan(*plan_args(**kw)) == status


def append_args(config=BF16, **kw):
    c = P.make_config(config)
    a = dict(cfg=C.byref(c), rows=_p(A), slots=_p(A), cache=_p(A), scales=_p(A), n=4,
             n_blocks=32, bs=16, ws=_p(A), ws_bytes=BIG, stream=_p(0))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(cfg=None), 1), (dict(rows=_p(0)), 1), (dict(scales=_p(0)), 1), (dict(n=0), 2),
    (dict(n=(1 << 30) + 1), 2), (dict(n=(1 << 31) - 1), 2),
    (dict(bs=20), 2), (dict(n_blocks=-1), 2), (dict(rows=_p(A + 8)), 3),
    (dict(cache=_p(A + 4)), 3), (dict(slots=_p(A + 1)), 3), (dict(ws=_p(A + 128)), 3),
    (dict(ws_bytes=C.c_size_t(256)), 5)])
def test_append_refuses(lib, kw, status):
    assert lib.mla_paged_append(*append_args(**kw)) == status


def test_row_width_must_be_a_multiple_of_16(lib):
    odd = F32.with_(kv_lora_rank=40)
    assert lib.mla_paged_append(*append_args(odd)) == 6
    assert b"multiple of 16" in lib.mla_last_error_detail()
    n = lib.mla_decode_paged_workspace_size(C.byref(P.make_config(odd)), 2, 4, 16, None)
    assert n == 0


def gather_args(config=BF16, **kw):
    c = P.make_config(config)
    a = dict(cfg=C.byref(c), cache=_p(A), scales=_p(A), table=_p(A), ctx=_p(A), rows=_p(A),
             cu=_p(A), B=4, max_blocks=8, n_blocks=32, bs=16, capacity=64, ws=_p(A),
             ws_bytes=BIG, stream=_p(0))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(cache=_p(0)), 1), (dict(rows=_p(0)), 1), (dict(cu=_p(0)), 1), (dict(B=-1), 2),
    (dict(max_blocks=0), 2), (dict(bs=17), 2), (dict(capacity=-2), 2), (dict(rows=_p(A + 2)), 3),
    (dict(capacity=(1 << 30) + 1), 2), (dict(capacity=(1 << 31) - 1), 2),
    (dict(ctx=_p(A + 2)), 3), (dict(ws_bytes=C.c_size_t(0)), 5)])
def test_gather_refuses(lib, kw, status):
    assert lib.mla_paged_gather(*gather_args(**kw)) == status


def decode_args(config=BF16, **kw):
    c = P.make_config(config)
    a = dict(cfg=C.byref(c), qn=_p(A), qp=_p(A), w=_p(A), cache=_p(A), scales=_p(A), table=_p(A),
             ctx=_p(A), B=4, max_blocks=8, n_blocks=32, bs=16, w_o=_p(0), out=_p(A), ws=_p(A),
             ws_bytes=BIG, stream=_p(0))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(qn=_p(0)), 1), (dict(ctx=_p(0)), 1), (dict(out=_p(0)), 1), (dict(ws=_p(0)), 1),
    (dict(B=0), 2), (dict(B=8193), 2), (dict(bs=8), 2), (dict(n_blocks=0), 2),
    (dict(max_blocks=-3), 2), (dict(qn=_p(A + 2)), 3), (dict(w_o=_p(A + 2)), 3),
    (dict(table=_p(A + 1)), 3), (dict(ws=_p(A + 64)), 3), (dict(ws_bytes=C.c_size_t(4096)), 5)])
def test_decode_refuses(lib, kw, status):
    assert lib.mla_decode_paged(*decode_args(**kw)) == status


def test_workspace_sizes(lib):
    assert P.mla_paged_workspace_size(1) >= 256 + 4
    assert P.mla_paged_workspace_size(1000) >= 256 + 125
    with pytest.raises(P.MlaError):
        P.mla_paged_workspace_size(0)
    n, lay = P.mla_decode_paged_workspace_size(F32, 3, 100, 32)
    assert n == lay["total_bytes"] and lay["split_tokens"] % 64 == 0
    assert lay["max_splits"] == -(-3200 // lay["split_tokens"])
    with pytest.raises(P.MlaError):
        P.mla_decode_paged_workspace_size(F32, 3, 100, 33)


def test_layout_struct_matches_the_header(tmp_path):
    import os
    import subprocess
    from conftest import ROOT
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mla.h"\nint main(void) {'
                   'printf("%zu %zu", sizeof(mla_paged_layout),'
                   'offsetof(mla_paged_layout, max_splits)); return 0; }')
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    size, off = map(int, subprocess.run([str(exe)], capture_output=True, text=True,
                                        check=True).stdout.split())
    assert C.sizeof(mla_paged_layout) == size and mla_paged_layout.max_splits.offset == off


# ----------------------------------------------------------------- binding
class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    f = FakeLib()
    monkeypatch.setattr(P._lib, "load", lambda: f)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    return f


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def binding_args(cfg=BF16):
    W, dt = cfg.kv_lora_rank + cfg.qk_rope_head_dim, \
        torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    B, nb, bs, mb = 2, 3, 16, 2
    pool = dict(cache=torch.zeros(nb, bs, W, dtype=torch.uint8).view(torch.float8_e4m3fn),
                scales=torch.ones(nb))
    ws = torch.zeros(512, dtype=torch.uint8)
    h = cfg.num_heads
    return dict(
        plan=dict(ctx_len=i32(B), new_len=i32(B), block_table=i32(B, mb), free_ring=i32(nb),
                  free_state=i32(2), ctx_out=i32(B), free_state_out=i32(2), slot_map=i32(7),
                  positions=i32(7), cu_new=i32(B + 1), B=B, max_blocks=mb, n_blocks=nb,
                  block_size=bs, capacity=7, workspace=ws, stream=0),
        append=dict(cfg=cfg, rows=torch.zeros(5, W, dtype=dt), slot_map=i32(5), **pool, n_rows=5,
                    n_blocks=nb, block_size=bs, workspace=ws, stream=0),
        gather=dict(cfg=cfg, **pool, block_table=i32(B, mb), ctx_len=i32(B),
                    rows_out=torch.zeros(9, W, dtype=dt), cu_ctx=i32(B + 1), B=B, max_blocks=mb,
                    n_blocks=nb, block_size=bs, capacity=9, workspace=ws, stream=0),
        decode=dict(cfg=cfg, q_nope=torch.zeros(B, h, cfg.qk_nope_head_dim, dtype=dt),
                    q_pe=torch.zeros(B, h, cfg.qk_rope_head_dim, dtype=dt),
                    w_kv_b=torch.zeros(h * (cfg.qk_nope_head_dim + cfg.v_head_dim),
                                       cfg.kv_lora_rank, dtype=dt),
                    **pool, block_table=i32(B, mb), ctx_len=i32(B), B=B, max_blocks=mb,
                    n_blocks=nb, block_size=bs, w_o=None,
                    out=torch.zeros(B, h * cfg.v_head_dim, dtype=dt), workspace=ws, stream=0))


CALLS = dict(plan="mla_paged_plan", append="mla_paged_append", gather="mla_paged_gather",
             decode="mla_decode_paged")


@pytest.mark.parametrize("op", list(CALLS))
@pytest.mark.parametrize("cfg", [BF16, F32], ids=["bf16", "f32"])
def test_binding_passes_declared_shapes_and_refuses_others(fake, op, cfg):
    f = getattr(P, CALLS[op])
    good = binding_args(cfg)[op]
    f(**good)
    assert fake.calls[-1][0] == CALLS[op]
    assert good["workspace"].data_ptr() in [getattr(a, "value", a) for a in fake.calls[-1][1]]
    n = len(fake.calls)
    for k, t in good.items():
        if not isinstance(t, torch.Tensor) or k == "workspace":
            continue
        bad = dict(good)
        bad[k] = t.flatten()[:-1].contiguous()             # too short
        with pytest.raises(ValueError, match=k):
            f(**bad)
        bad[k] = t.to(torch.float64) if t.dtype != torch.float8_e4m3fn else t.float()
        with pytest.raises(ValueError, match=k):
            f(**bad)
        bad[k] = torch.stack([t.view(torch.uint8)] * 2, -1)[..., 0] \
            if t.dtype == torch.float8_e4m3fn else torch.stack([t, t], -1)[..., 0]
        with pytest.raises(ValueError, match=k):           # not contiguous
            f(**bad)
        if k not in ("positions", "w_o"):
            bad[k] = None
            with pytest.raises(ValueError, match=k):
                f(**bad)
    assert len(fake.calls) == n


def test_binding_takes_bytes_and_optional_outputs(fake):
    a = binding_args()
    d = a["append"]
    d["cache"] = d["cache"].view(torch.uint8)
    P.mla_paged_append(**d)
    p = a["plan"]
    p.update(positions=None)
    P.mla_paged_plan(**p)
    p.update(slot_map=None, capacity=0)
    P.mla_paged_plan(**p)
    g = a["gather"]
    g.update(rows_out=None, capacity=0)
    P.mla_paged_gather(**g)
    assert len(fake.calls) == 4


def test_binding_needs_a_gpu():
    with pytest.raises(ValueError, match="CUDA"):
        P.mla_paged_append(**binding_args()["append"])


@pytest.mark.parametrize("op", list(CALLS))
def test_binding_refuses_tensors_of_two_devices(fake, op):
    good = binding_args()[op]
    k = {"plan": "free_ring", "append": "rows", "gather": "ctx_len", "decode": "q_pe"}[op]
    good[k] = good[k].to("meta")
    with pytest.raises(ValueError, match="different devices"):
        getattr(P, CALLS[op])(**good)
