"""A visible block whose table entry is out of range is flagged and absent: the sequence attends its
other keys, whichever kernel the call takes."""

import numpy as np
import pytest
import torch

import oracle.window_attention
import paged_kv_cache_422_b200 as nvpa
from tests.window_helpers import ROW_BITS, TILE_BITS, Case, check_answers

pytestmark = pytest.mark.gpu


def _check(dev, monkeypatch, case, bad, num_splits, value):
    """Table entries `bad` of the only sequence replaced by `value`."""
    n, new = case.lens[0], case.news[0]
    absent = np.isin(np.arange(n) // case.bs, bad)
    t = case.device(dev)
    for j in bad:
        t["tables"][0, j] = value
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = nvpa.chunk_attention(
        t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], new, n, case.scale, window=case.window,
        num_sinks=case.sinks, k_scales=t["k_scales"], v_scales=t["v_scales"], num_splits=num_splits, err_flag=err,
        return_lse=True)
    assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
    seen = oracle.window_attention.seen
    rows = new * (case.hq // case.hkv)
    with monkeypatch.context() as m:
        m.setattr(oracle.window_attention, "seen", lambda *a: seen(*a) & ~absent)
        check_answers(case, out, lse, TILE_BITS if rows > (24 if case.fp8 else 16) else ROW_BITS[case.fp8],
                      f"blocks {bad} absent, splits {num_splits}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 64), (64, 256)])
@pytest.mark.parametrize("new", [1, 5, 12, 40, 150, 300])
def test_absent_blocks(cuda_device, monkeypatch, fp8, d, bs, new):
    n = 700
    case = Case(91 + d + bs + new, [n], [new], 4, 2, d, bs, fp8)
    last = (n - 1) // bs
    for bad, value in (([0], -1), ([1], case.num_blocks), ([0, last], 1 << 30), ([last], -(1 << 31))):
        for num_splits in (0, 1, 3):
            _check(cuda_device, monkeypatch, case, bad, num_splits, value)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 5, 40, 150])
@pytest.mark.parametrize("window,sinks", [(50, 0), (130, 4), (300, 40)])
def test_absent_blocks_in_a_window(cuda_device, monkeypatch, fp8, new, window, sinks):
    n, bs = 700, 16
    case = Case(95 + new, [n], [new], 4, 2, 64, bs, fp8, window=window, sinks=sinks)
    first = (n - new - window + 1) // bs          # the block with the first row's first key
    choices = [[first], [first + 1, (n - 1) // bs]] + ([[0], [0, first + 2]] if sinks else [])
    for bad in choices:
        for num_splits in (0, 2):
            _check(cuda_device, monkeypatch, case, bad, num_splits, case.num_blocks + 3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("new", [5, 40, 150])
def test_absent_blocks_of_long_contexts(cuda_device, monkeypatch, fp8, bs, new):
    """Tens of key tiles: what was absent in one tile is there again in later ones."""
    n = 3500
    case = Case(99 + bs, [n], [new], 2, 1, 64, bs, fp8)
    last = (n - 1) // bs
    for bad in ([0], [1, last // 2], list(range(3, 9)) + [last - 1]):
        for num_splits in (1, 2):
            _check(cuda_device, monkeypatch, case, bad, num_splits, -3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,window", [(40, 0), (40, 100), (150, 0)])
def test_an_absent_block_harms_no_other_sequence(cuda_device, fp8, new, window):
    """More (sequence, KV head) pairs than SMs, so that a block of threads goes on from a damaged
    sequence to others; a damaged one comes out as in a call of its own."""
    dev = cuda_device
    lens = [200 + 9 * (i % 13) for i in range(60)]
    case = Case(101, lens, [new] * 60, 8, 4, 64, 16, fp8, window=window, sinks=3)
    t = case.device(dev)

    def call(tables, cu, lens, q):
        return nvpa.chunk_attention(q, t["k_cache"], t["v_cache"], tables, cu, lens, new, 400, case.scale,
                                    window=window, num_sinks=3, k_scales=t["k_scales"], v_scales=t["v_scales"],
                                    num_splits=1, return_lse=True)

    good, good_lse = call(t["tables"], t["cu"], t["lens"], t["q"])
    tables = t["tables"].clone()
    for b in (0, 7, 31, 32, 50):
        tables[b, (lens[b] - 1) // 16 - b % 3] = -9
    out, lse = call(tables, t["cu"], t["lens"], t["q"])
    for b in range(60):
        rows = slice(b * new, (b + 1) * new)
        if b in (0, 7, 31, 32, 50):
            want, want_lse = call(tables[b:b + 1].contiguous(), t["cu"][:2], t["lens"][b:b + 1], t["q"][rows])
            assert not torch.equal(out[rows], good[rows])
        else:
            want, want_lse = good[rows], good_lse[rows]
        assert torch.equal(out[rows], want) and torch.equal(lse[rows], want_lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 5, 40, 150])
def test_every_block_absent(cuda_device, fp8, new):
    dev = cuda_device
    case = Case(97, [200, 170], [new, max(1, new // 2)], 4, 2, 64, 16, fp8)
    t = case.device(dev)
    good, good_lse = nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], new, 200,
                                          case.scale, k_scales=t["k_scales"], v_scales=t["v_scales"], return_lse=True)
    t["tables"][1] = -1
    for num_splits in (0, 1, 3):
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        out, lse = nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], new, 200,
                                        case.scale, k_scales=t["k_scales"], v_scales=t["v_scales"],
                                        num_splits=num_splits, err_flag=err, return_lse=True)
        assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
        assert bool((out[new:] == 0).all()) and bool(torch.isneginf(lse[new:]).all())
        if num_splits == 0:
            assert torch.equal(out[:new], good[:new]) and torch.equal(lse[:new], good_lse[:new])


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
