"""A visible block whose table entry is out of range is flagged and absent: the sequence attends its
other keys, whichever kernel the call takes."""

import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from tests.window_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 5, 12, 40, 150])
@pytest.mark.parametrize("value", [-1, -2, -(1 << 31), (1 << 31) - 1])
def test_every_id_out_of_range_is_flagged(cuda_device, fp8, new, value):
    dev = cuda_device
    case = Case(90, [300], [new], 4, 2, 64, 16, fp8)
    t = case.device(dev)
    for num_splits in (0, 1, 3):
        for j in (0, 7, 18):
            tables = t["tables"].clone()
            tables[0, j] = value
            err = torch.zeros(1, dtype=torch.int32, device=dev)
            out, lse = nvpa.chunk_attention(
                t["q"], t["k_cache"], t["v_cache"], tables, t["cu"], t["lens"], new, 300, case.scale,
                k_scales=t["k_scales"], v_scales=t["v_scales"], num_splits=num_splits, err_flag=err, return_lse=True)
            assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
            assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
