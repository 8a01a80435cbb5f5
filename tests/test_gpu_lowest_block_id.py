"""A block-table entry of -2^31 is flagged like any other out of range by the prefill and the
shared-prefix kernels."""

import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from synth import make_decode_step, make_prefill_step
from synth.device import decode_to_device, prefill_to_device

pytestmark = pytest.mark.gpu

LOWEST = -(1 << 31)


@pytest.mark.parametrize("value", [-1, LOWEST])
def test_prefill(cuda_device, value):
    step = make_prefill_step(5, [300, 140], cached_blocks=[1, 0], num_q_heads=4, num_kv_heads=2,
                             head_dim=64, block_size=16)
    t = prefill_to_device(step, cuda_device)
    nvpa.store_kvcache(t["k_new"], t["v_new"], t["k_cache"], t["v_cache"], t["slot_mapping"])
    t["block_tables"][0, 3] = value
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = nvpa.varlen_prefill_attention(t["q"], t["k_cache"], t["v_cache"], t["block_tables"], t["cu_seqlens_q"],
                                        t["cu_seqlens_k"], step.max_seqlen_q, step.max_seqlen_k, step.scale,
                                        err_flag=err)
    assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("value", [-1, LOWEST])
def test_shared_prefix(cuda_device, value):
    step = make_decode_step(7, [300] * 12, num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=16)
    step.block_tables[:, :8] = step.block_tables[0, :8]
    t = decode_to_device(step, cuda_device)
    nvpa.store_kvcache(t["k_new"], t["v_new"], t["k_cache"], t["v_cache"], t["slot_mapping"])
    t["block_tables"][:, 3] = value
    ws = torch.empty(nvpa.decode_shared_prefix_workspace_size(12, 4, 2, 64, 300, 16, 0, 4), dtype=torch.uint8,
                     device=cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = nvpa.decode_step_shared_prefix(t["q"], None, None, t["k_cache"], t["v_cache"], None, t["block_tables"],
                                         t["context_lens"], 300, step.scale, workspace=ws, min_group_size=4,
                                         err_flag=err)
    assert ws[:20].view(torch.int32).cpu().tolist()[2:4] == [1, 12]       # one group of all twelve
    assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
    assert torch.isfinite(out.float()).all()
