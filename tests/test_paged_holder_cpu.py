"""``MlaPagedCache`` without a GPU: a stand-in for the library writes and reads
the status words in the (CPU) workspaces as the kernels do, so what
``check_status`` can still see after a whole step shows here."""
import ctypes as C

import pytest
import torch

import latent_attention_b200 as P
from latent_attention_b200.layer import MlaPagedCache
from mla_inputs import WORKLOADS

F32 = WORKLOADS["tiny_f32"].cfg
SHAPE, NO_BLOCKS = 2, 9
# position of the workspace among the C arguments
WS_AT = {"mla_paged_plan": 15, "mla_paged_append": 8, "mla_paged_gather": 12,
         "mla_decode_paged": 14}


class StatusLib:
    """Every call starts its workspace's status afresh and leaves there what
    ``outcome`` says; reading a status clears it."""

    def __init__(self):
        self.outcome, self.seen = {}, {}

    def _word(self, ws):
        return C.cast(ws if isinstance(ws, int) else ws.value, C.POINTER(C.c_uint32))

    def mla_paged_workspace_size(self, n_blocks):
        return 4096

    def mla_decode_paged_workspace_size(self, *a):
        return 4096

    def mla_last_error_detail(self):
        return b""

    def mla_status_string(self, s):
        return {SHAPE: b"MLA_ERR_SHAPE", NO_BLOCKS: b"MLA_ERR_NO_BLOCKS"}[s]

    def mla_check_device_status(self, ws, stream):
        word = self._word(ws)
        s, word[0] = word[0], 0
        return s

    def __getattr__(self, name):
        def call(*args):
            ws = args[WS_AT[name]]
            self.seen[name] = ws
            self._word(ws)[0] = self.outcome.get(name, 0)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    f = StatusLib()
    monkeypatch.setattr(P._lib, "load", lambda: f)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    return f


def cache():
    return MlaPagedCache(F32, 2, max_blocks=4, n_blocks=8, block_size=16, capacity=8, device="cpu")


def step(pc):
    W, h = pc.width, F32.num_heads
    pc.plan(torch.zeros(2, dtype=torch.int32), stream=0)
    pc.append(torch.zeros(8, W), stream=0)
    pc.decode(torch.zeros(2, h, F32.qk_nope_head_dim), torch.zeros(2, h, F32.qk_rope_head_dim),
              torch.zeros(h * (F32.qk_nope_head_dim + F32.v_head_dim), F32.kv_lora_rank),
              torch.zeros(2, h * F32.v_head_dim), stream=0)
    pc.gather(torch.zeros(8, W), torch.zeros(3, dtype=torch.int32), stream=0)


def test_status_before_the_first_call_of_a_kind(lib, monkeypatch):
    """A step of prompts appends and never decodes: what the memory behind the
    decode's workspace held before is no status."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(255))
    pc = cache()
    pc.check_status(stream=0)
    pc.plan(torch.zeros(2, dtype=torch.int32), stream=0)
    pc.append(torch.zeros(8, pc.width), stream=0)
    pc.check_status(stream=0)


@pytest.mark.parametrize("op,status,name", [
    ("mla_paged_plan", NO_BLOCKS, "NO_BLOCKS"), ("mla_paged_append", SHAPE, "SHAPE"),
    ("mla_paged_gather", SHAPE, "SHAPE"), ("mla_decode_paged", SHAPE, "SHAPE")])
def test_a_failure_in_mid_step_is_seen_at_its_end(lib, op, status, name):
    pc = cache()
    lib.outcome[op] = status
    step(pc)
    with pytest.raises(P.MlaError, match=name):
        pc.check_status(stream=0)
    pc.check_status(stream=0)                     # read once
    lib.outcome.clear()
    step(pc)
    pc.check_status(stream=0)


def test_all_statuses_are_read_when_several_failed(lib):
    pc = cache()
    lib.outcome.update(mla_paged_plan=NO_BLOCKS, mla_decode_paged=SHAPE)
    step(pc)
    with pytest.raises(P.MlaError, match="NO_BLOCKS"):
        pc.check_status(stream=0)
    pc.check_status(stream=0)
