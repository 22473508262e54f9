"""Workspace sizes of the paged decode: what the call needs, and that a
workspace of the largest batch serves every smaller one."""
import pytest

import latent_attention_b200 as P
from latent_attention_b200._lib import LIB_PATH
from mla_inputs import WORKLOADS, MlaConfig

F32 = WORKLOADS["tiny_f32"].cfg
WIDE = dict(hidden_size=256, q_lora_rank=0, qk_nope_head_dim=128, v_head_dim=128,
            rope_type="none", dtype="bf16")
CONFIGS = {
    "f32": F32, "f32_h1": F32.with_(num_heads=1), "f32_r512": F32.with_(kv_lora_rank=512),
    "bf16_other_width": MlaConfig(num_heads=7, kv_lora_rank=96, qk_rope_head_dim=32, **WIDE),
    "bf16_many_heads": MlaConfig(num_heads=200, kv_lora_rank=96, qk_rope_head_dim=32, **WIDE),
    "bf16_tensor_cores": MlaConfig(num_heads=128, kv_lora_rank=512, qk_rope_head_dim=64, **WIDE)}


@pytest.fixture(scope="module", autouse=True)
def built():
    import os
    from latent_attention_b200 import build
    if not os.path.exists(LIB_PATH):
        build.build()


@pytest.mark.parametrize("name", list(CONFIGS))
def test_size_never_falls_with_the_batch_or_the_table(name):
    c = P.make_config(CONFIGS[name])
    batches = list(range(1, 70)) + [100, 127, 128, 129, 300, 1000, 8191, 8192]
    tables = [1, 2, 3, 7, 16, 31, 32, 62, 63, 64, 65, 127, 128, 500, 511, 512, 2000]
    for bs in (16, 32, 128):
        size = {(B, mb): P.mla_decode_paged_workspace_size(c, B, mb, bs)[0]
                for B in batches for mb in tables}
        for a, b in zip(batches, batches[1:]):
            for mb in tables:
                assert size[a, mb] <= size[b, mb], (a, b, mb, bs)
        for a, b in zip(tables, tables[1:]):
            for B in batches:
                assert size[B, a] <= size[B, b], (B, a, b, bs)


@pytest.mark.parametrize("name", [n for n in CONFIGS if n != "bf16_tensor_cores"])
def test_partials_of_every_split_fit(name):
    cfg = CONFIGS[name]
    c, h, r = P.make_config(cfg), cfg.num_heads, cfg.kv_lora_rank
    for B in list(range(1, 41)) + [500, 8192]:
        for mb in (1, 5, 63, 64, 200, 1000, 40000):
            for bs in (16, 128):
                _, lay = P.mla_decode_paged_workspace_size(c, B, mb, bs)
                assert lay["max_splits"] == -(-mb * bs // lay["split_tokens"])
                parts = B * lay["max_splits"] * h
                assert lay["part_lse"] - lay["part_o"] >= parts * r * 4
                assert lay["o_lat"] - lay["part_lse"] >= parts * 4
