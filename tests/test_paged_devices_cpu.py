"""The paged calls refuse tensors that are not on the current device (the kernels
launch there), and tensors of two devices: shown on tensors that claim to be on
some GPU."""
import pytest
import torch

import latent_attention_b200 as P
from test_paged_cpu import CALLS, binding_args, fake  # noqa: F401


@pytest.fixture
def on_gpu_1(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    P._torch()
    monkeypatch.setattr(P, "_raw_stream", lambda device: 0)


@pytest.mark.parametrize("op", list(CALLS))
def test_the_current_device_is_another(fake, on_gpu_1, monkeypatch, op):  # noqa: F811
    monkeypatch.setattr(P, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        getattr(P, CALLS[op])(**binding_args()[op])
    assert not fake.calls
    monkeypatch.setattr(P, "_current_device", lambda: 1)
    getattr(P, CALLS[op])(**binding_args()[op])
    assert len(fake.calls) == 1


@pytest.mark.parametrize("op,name", [("plan", "free_ring"), ("append", "slot_map"),
                                     ("gather", "block_table"), ("decode", "w_kv_b")])
def test_one_tensor_on_another_device(fake, monkeypatch, op, name):  # noqa: F811
    args = binding_args()[op]
    there = args[name].data_ptr()
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 2 if self.data_ptr() == there else 1)
    monkeypatch.setattr(torch.Tensor, "device", property(
        lambda self: torch.device("cuda", 2 if self.data_ptr() == there else 1)))
    P._torch()
    monkeypatch.setattr(P, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match=f"different devices: {name}"):
        getattr(P, CALLS[op])(**args)
    assert not fake.calls
