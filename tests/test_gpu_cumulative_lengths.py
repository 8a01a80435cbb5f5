"""Cumulative lengths at the ends of int32: flagged, in bounds, and nothing written."""

import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from synth.device import i32

pytestmark = pytest.mark.gpu

LOW, HIGH = -(1 << 31), (1 << 31) - 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cu", [[LOW, 100, 120], [LOW, LOW, 120], [-5, 3, 7], [LOW, HIGH, HIGH], [HIGH, LOW, 0]])
def test_gather(cuda_device, fp8, cu):
    dev = cuda_device
    cache = torch.ones((4, 16, 2, 64), dtype=torch.bfloat16, device=dev)
    tables = i32([[1, 2], [3, 0]], dev)
    out = torch.full((7, 2, 64), 5.0, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    if fp8:
        scales = torch.full((4, 2, 16), 127, dtype=torch.uint8, device=dev)
        nvpa.gather_kv_fp8(cache.to(torch.float8_e4m3fn), scales, tables, i32(cu, dev), 7, out=out, err_flag=err)
    else:
        nvpa.gather_kv(cache, tables, i32(cu, dev), 7, out=out, err_flag=err)
    assert err.item() == nvpa.NVPA_FLAG_BAD_LENGTH
    # rows of a sequence that starts at a row are as they should be, the others as they were
    want = torch.full_like(out, 5.0)
    if cu == [-5, 3, 7]:
        want[3:] = 1.0
    assert torch.equal(out, want)


@pytest.mark.parametrize("cu_q,cu_k", [([HIGH, LOW], [0, 4]), ([0, 2], [HIGH, LOW]), ([HIGH, LOW], [HIGH, LOW]),
                                       ([LOW, HIGH], [LOW, HIGH]), ([0, 2], [LOW, HIGH])])
def test_prefill(cuda_device, cu_q, cu_k):
    dev = cuda_device
    cache = torch.ones((4, 16, 2, 64), dtype=torch.bfloat16, device=dev)
    q = torch.ones((2, 4, 64), dtype=torch.bfloat16, device=dev)
    out, lse = torch.full_like(q, 5.0), torch.full((2, 4), 5.0, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    nvpa.varlen_prefill_attention(q, cache, cache, i32([[1, 2]], dev), i32(cu_q, dev), i32(cu_k, dev), 2, 20, 0.1, out=out,
                                  lse=lse, err_flag=err)
    assert err.item() == nvpa.NVPA_FLAG_BAD_LENGTH
    assert bool((out == 5.0).all()) and bool((lse == 5.0).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("max_q", [2, 40])
@pytest.mark.parametrize("cu", [[HIGH, LOW, 2], [LOW, HIGH, 2], [0, LOW, HIGH], [LOW, LOW, LOW], [HIGH, HIGH, LOW]])
def test_chunks(cuda_device, fp8, max_q, cu):
    dev = cuda_device
    cache = torch.ones((4, 16, 2, 64), dtype=torch.bfloat16, device=dev)
    sc = {}
    if fp8:
        cache = cache.to(torch.float8_e4m3fn)
        sc = {x: torch.full((4, 2, 16), 127, dtype=torch.uint8, device=dev) for x in ("k_scales", "v_scales")}
    q = torch.ones((2, 4, 64), dtype=torch.bfloat16, device=dev)
    out, lse = torch.full_like(q, 5.0), torch.full((2, 4), 5.0, device=dev)
    for lens in ([20, 20], [HIGH, LOW]):
        for num_splits in (0, 1, 2):
            err = torch.zeros(1, dtype=torch.int32, device=dev)
            nvpa.chunk_attention(q, cache, cache, i32([[1, 2], [3, 0]], dev), i32(cu, dev), i32(lens, dev), max_q, 20, 0.1,
                                 num_splits=num_splits, out=out, lse=lse, err_flag=err, **sc)
            assert err.item() == nvpa.NVPA_FLAG_BAD_LENGTH
            assert bool((out == 5.0).all()) and bool((lse == 5.0).all())
