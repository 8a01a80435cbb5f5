"""Queries and visible keys that are not numbers show in the rows that they reach, whole or in
partitions, and in no other; scales and bounds at their ends."""

import math

import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from tests.window_helpers import ROW_BITS, TILE_BITS, Case, check_answers

pytestmark = pytest.mark.gpu

NEWS = [1, 5, 40, 150]          # the row kernel's one and several rows, one query tile, a pair


def _bits(fp8, new):     # 2 query heads per KV head: chunks of more than 16 rows (24 of e4m3) on tiles
    return TILE_BITS if 2 * new > (24 if fp8 else 16) else ROW_BITS[fp8]


def _call(case, t, num_splits=0, **kw):
    args = dict(window=case.window, num_sinks=case.sinks, k_scales=t["k_scales"], v_scales=t["v_scales"])
    args.update(kw)
    return nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], max(case.news),
                                max(case.lens), case.scale, num_splits=num_splits, return_lse=True, **args)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", NEWS)
@pytest.mark.parametrize("num_splits", [0, 1, 4])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_query_that_is_not_a_number(cuda_device, fp8, new, num_splits, value):
    case = Case(31, [200, 170], [new, max(1, new // 2)], 4, 2, 64, 16, fp8)
    t = case.device(cuda_device)
    want, want_lse = _call(case, t, num_splits)
    # inf times keys of either sign: scores of +inf among them, and inf - inf in the softmax
    t["q"][new, 1, 3] = value
    out, lse = _call(case, t, num_splits)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device=cuda_device)
    hit[new, 1] = True
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(out[:new], want[:new]) and torch.equal(lse[:new], want_lse[:new])   # the other sequence
    out, lse = torch.where(hit[..., None], want, out), torch.where(hit, want_lse, lse)
    check_answers(case, out, lse, _bits(fp8, new), "the other rows")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", NEWS)
@pytest.mark.parametrize("num_splits", [0, 1, 4])
def test_a_key_that_is_not_a_number(cuda_device, fp8, new, num_splits):
    n, at = 200, 53
    case = Case(32, [n], [new], 4, 2, 64, 16, fp8)
    t = case.device(cuda_device)
    blk = int(t["tables"][0, at // 16])
    if fp8:
        t["k_cache"].view(torch.uint8)[blk, at % 16, 1, 7] = 0x7F
    else:
        t["k_cache"][blk, at % 16, 1, 7] = math.nan
    out, lse = _call(case, t, num_splits)
    pos = torch.arange(n - new, n, device=cuda_device)
    hit = (pos >= at)[:, None] & (torch.arange(4, device=cuda_device) >= 2)[None]
    assert torch.equal(lse.isnan(), hit)
    assert torch.equal(out.isnan(), hit[..., None].expand_as(out))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("num_splits", [0, 1, 4])
def test_decode_of_a_query_that_is_not_a_number(cuda_device, fp8, num_splits):
    case = Case(33, [300, 41, 200], [1, 1, 1], 4, 2, 128, 32, fp8)
    t = case.device(cuda_device)
    t["q"][0, 2] = math.nan
    out, lse = nvpa.paged_decode_attention_window(
        t["q"], t["k_cache"], t["v_cache"], t["tables"], t["lens"], 300, case.scale, k_scales=t["k_scales"],
        v_scales=t["v_scales"], num_splits=num_splits, return_lse=True)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device=cuda_device)
    hit[0, 2] = True
    assert torch.equal(lse.isnan(), hit) and torch.equal(out.isnan(), hit[..., None].expand_as(out))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", NEWS)
@pytest.mark.parametrize("scale", [0.0, 1e-30])
def test_a_scale_of_zero_weighs_all_keys_alike(cuda_device, fp8, new, scale):
    case = Case(34, [200, 170], [new, max(1, new // 2)], 4, 2, 64, 16, fp8, scale=scale)
    t = case.device(cuda_device)
    for num_splits in (0, 1, 4):
        out, lse = _call(case, t, num_splits)
        check_answers(case, out, lse, _bits(fp8, new), f"{num_splits} splits")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", NEWS)
def test_bounds_at_their_ends(cuda_device, fp8, new):
    case = Case(35, [200, 170], [new, max(1, new // 2)], 4, 2, 64, 16, fp8)
    t = case.device(cuda_device)
    big = 2 ** 31 - 1
    for window, sinks in ((big, 0), (big, big), (1, big)):       # every key is visible
        out, lse = _call(case, t, window=window, num_sinks=sinks)
        check_answers(case, out, lse, _bits(fp8, new), f"window {window}, {sinks} sinks")
    # no row fits a bound of zero: all are flagged and none is written
    for max_q, max_ctx in ((0, 200), (new, 0)):
        out = torch.full_like(t["q"], 7)
        err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], max_q, max_ctx,
                             case.scale, k_scales=t["k_scales"], v_scales=t["v_scales"], out=out, err_flag=err)
        assert err.item() != 0 and bool((out == 7).all())
    # sequences without new tokens
    out = torch.full_like(t["q"], 7)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], torch.zeros_like(t["cu"]), t["lens"], new,
                         200, case.scale, k_scales=t["k_scales"], v_scales=t["v_scales"], out=out, err_flag=err)
    assert err.item() == 0 and bool((out == 7).all())
