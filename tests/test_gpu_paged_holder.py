"""``MlaPagedCache`` on a B200: what a step reports at its end, eager and
captured."""
import pytest
import torch

from latent_attention_b200 import MlaError
from latent_attention_b200.layer import MlaPagedCache
from mla_inputs import WORKLOADS

pytestmark = pytest.mark.gpu

F32 = WORKLOADS["tiny_f32"].cfg


class Step:
    """plan + append + decode + gather on buffers that a replay reads again."""

    def __init__(self, B=3, n_blocks=6, capacity=40):
        h = F32.num_heads
        self.pc = MlaPagedCache(F32, B, max_blocks=5, n_blocks=n_blocks, block_size=16,
                                capacity=capacity)
        self.new = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.rows = torch.randn(capacity, self.pc.width, device="cuda")
        self.q = [torch.randn(B, h, d, device="cuda")
                  for d in (F32.qk_nope_head_dim, F32.qk_rope_head_dim)]
        self.w = 0.1 * torch.randn(h * (F32.qk_nope_head_dim + F32.v_head_dim), F32.kv_lora_rank,
                                   device="cuda")
        self.out = torch.zeros(B, h * F32.v_head_dim, device="cuda")
        self.got = torch.zeros(B * 80, self.pc.width, device="cuda")
        self.cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")

    def __call__(self):
        self.pc.plan(self.new)
        self.pc.append(self.rows)
        self.pc.decode(*self.q, self.w, self.out)
        self.pc.gather(self.got, self.cu)

    def state(self):
        pc = self.pc
        return [t.clone() for t in (pc.table, pc.ring, pc.state, pc.ctx, pc.cache.view(torch.uint8),
                                    pc.scales)]


@pytest.mark.parametrize("captured", [False, True])
def test_a_plan_that_fails_in_mid_step_is_reported(cuda, captured):
    step = Step()
    run = step
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            Step()()                              # loads the kernels
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    for lens, fails in (([20, 1, 7], False),      # 4 of the 6 blocks
                        ([29, 1, 10], True),      # 3 blocks more: two are left
                        ([1, 1, 1], False),
                        ([20, 20, 1], True),      # 41 tokens, 40 slots
                        ([-1, -1, -1], False),
                        ([16, 16, 8], False)):
        step.new.copy_(torch.tensor(lens, dtype=torch.int32))
        before = step.state()
        run()
        torch.cuda.synchronize()
        if fails:
            with pytest.raises(MlaError, match="NO_BLOCKS"):
                step.pc.check_status()
            for a, b in zip(before, step.state()):
                assert torch.equal(a, b)
        step.pc.check_status()
    assert step.pc.ctx.tolist() == [16, 16, 8]


@pytest.mark.parametrize("B", [1, 19, 20])
def test_a_workspace_of_the_largest_batch_serves_smaller_ones(cuda, B):
    """63 blocks of 32: 20 requests run in splits of 128 tokens, 19 in splits
    of 64, which leave more partial results."""
    import latent_attention_b200 as L
    h, bs, mb, n_blocks = F32.num_heads, 32, 63, 64
    g = torch.Generator().manual_seed(B)
    cache = torch.randn(n_blocks, bs, F32.kv_lora_rank + F32.qk_rope_head_dim, generator=g)
    cache = cache.to(torch.float8_e4m3fn).cuda()
    scales = torch.ones(n_blocks, device="cuda")
    table = torch.randint(0, n_blocks, (B, mb), dtype=torch.int32, generator=g).cuda()
    ctx = torch.randint(0, mb * bs + 1, (B,), dtype=torch.int32, generator=g).cuda()
    qn = torch.randn(B, h, F32.qk_nope_head_dim, generator=g).cuda()
    qp = torch.randn(B, h, F32.qk_rope_head_dim, generator=g).cuda()
    w = (0.1 * torch.randn(h * (F32.qk_nope_head_dim + F32.v_head_dim), F32.kv_lora_rank,
                           generator=g)).cuda()
    outs = []
    for sized_for in (20, B):
        n, _ = L.mla_decode_paged_workspace_size(F32, sized_for, mb, bs)
        ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
        out = torch.full((B, h * F32.v_head_dim), 9.0, device="cuda")
        L.mla_decode_paged(F32, qn, qp, w, cache, scales, table, ctx, B, mb, n_blocks, bs, None,
                           out, ws)
        L.mla_check_device_status(ws)
        outs.append(out)
    assert torch.equal(*outs) and not torch.isnan(outs[0]).any()
