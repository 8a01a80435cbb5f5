"""Infinite values in a bf16 cache: a query that sees one gets an infinity in that channel, as in
the sum of the definition, and its other channels are unharmed."""

import math

import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from tests.window_helpers import ROW_BITS, TILE_BITS, Case, check_answers

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 2, 4, 8, 20, 70])
@pytest.mark.parametrize("num_splits", [0, 1, 3])
def test_infinite_values(cuda_device, d, new, num_splits):
    case = Case(81 + d + new, [300], [new], 8, 4, d, 16, False)
    t = case.device(cuda_device)
    want = {}
    for i, (key, head, dim, value) in enumerate([(3, 0, 5, math.inf), (77, 1, 0, -math.inf), (200, 2, d - 1, math.inf),
                                                 (201, 2, d - 1, math.inf), (9, 3, 7, math.inf), (99, 3, 7, -math.inf)]):
        t["v_cache"][int(t["tables"][0, key // 16]), key % 16, head, dim] = value
        want.setdefault((head, dim), []).append(value)
    out, lse = nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], new, 300,
                                    case.scale, num_splits=num_splits, return_lse=True)
    if new == 1:
        again, again_lse = nvpa.paged_decode_attention_window(
            t["q"], t["k_cache"], t["v_cache"], t["tables"], t["lens"], 300, case.scale, num_splits=num_splits,
            return_lse=True)
        assert torch.equal(lse, again_lse) and torch.equal(out.nan_to_num(nan=9.0), again.nan_to_num(nan=9.0))
    clean = torch.from_numpy(case.answers()[0]).to(out)
    for (head, dim), values in want.items():
        got = out[:, 2 * head:2 * head + 2, dim].float()
        total = sum(values)                       # inf, -inf, or nan for one of each
        if math.isnan(total):
            assert bool(got.isnan().all())
        else:
            assert bool((got == total).all()), (head, dim, got)
        out[:, 2 * head:2 * head + 2, dim] = clean[:, 2 * head:2 * head + 2, dim]
    check_answers(case, out, lse, TILE_BITS if 2 * new > 16 else ROW_BITS[False], "the other channels")
