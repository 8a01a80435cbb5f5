"""Values far apart: what a small weight, a small query element or a small row adds shows in the
channels that nothing larger reaches, wherever its key lies."""

import numpy as np
import pytest

import paged_kv_cache_422_b200 as nvpa
from oracle.paged_attention import bf16_to_f64
from oracle.window_attention import dequantise_rows, gather, quantise_rows
from synth.workloads import bf16_bits_from_f32
from tests.window_helpers import ROW_BITS, TILE_BITS, Case, check_answers

pytestmark = pytest.mark.gpu


def bits_of(case):
    """Significant bits of the weights in the kernel that a call with these chunks takes."""
    rows = max(case.news) * (case.hq // case.hkv)
    return TILE_BITS if rows > (24 if case.fp8 else 16) else ROW_BITS[case.fp8]


def run(case, dev, num_splits=0):
    t = case.device(dev)
    return nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], max(case.news),
                                max(case.lens), case.scale, window=case.window, num_sinks=case.sinks,
                                k_scales=t["k_scales"], v_scales=t["v_scales"], num_splits=num_splits, return_lse=True)


def set_rows(case, which, x):
    """Cache rows x [num_blocks, bs, Hkv, D] for K (0) or V (1)."""
    case.kv_bits[which] = bf16_bits_from_f32(x.astype(np.float32)).reshape(x.shape)
    assert case.fp8
    case.codes[which], case.scales[which] = quantise_rows(case.kv_bits[which])
    case.values[which] = dequantise_rows(case.codes[which], case.scales[which])


# new tokens: 8, 16 and 24 rows per KV head, and a 128-row tile (4 query heads per KV head)
NEWS = [1, 2, 4, 5, 6, 20]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", NEWS)
@pytest.mark.parametrize("spread", [12, 20, 28])
def test_value_rows_of_very_different_size_in_channels_of_their_own(cuda_device, d, new, spread):
    """Key j has one value, in channel j mod D, of a size between 1 and 2^spread: a channel's
    result hangs on few keys, most of them far below the largest.  Scores within 2^8 of one
    another: every weight times its value's scale is above 2^-36 of the largest."""
    case = Case(51 + d + new, [300, 77], [new, max(1, new // 2)], 4, 1, d, 16, True, q_mult=0.5)
    rng = np.random.default_rng(spread)
    nb, bs, hkv, _ = case.kv_bits[1].shape
    v = np.zeros((nb, bs, hkv, d))
    size = np.exp2(rng.integers(0, spread + 1, size=(nb, bs, hkv))) * rng.uniform(1, 2, size=(nb, bs, hkv))
    channel = rng.integers(0, d, size=(nb, bs, hkv))
    np.put_along_axis(v, channel[..., None], size[..., None], -1)
    set_rows(case, 1, v)
    for num_splits in (0, 1, 3):
        out, lse = run(case, cuda_device, num_splits)
        check_answers(case, out, lse, bits_of(case), f"{num_splits} splits")


class AlikeScales(Case):
    """Bounds for values whose scales lie within 2 of one another: an fp16 weight of the e4m3 cache
    is 2^6 or more for a row's largest and off by at most 2^-25, half of fp16's smallest step, so a
    softmax weight is off by at most 2^-31 of the largest."""

    def answers(self):
        out, lse, ob, mass, lb = super().answers()
        for b, (n, m) in enumerate(zip(self.lens, self.news)):
            size = np.abs(gather(self.values[1], self.tables[b], n, self.bs)).sum(0)          # [Hkv, D]
            ob[self.cu[b]:self.cu[b + 1]] += 2.0 ** -31 * np.repeat(size, self.hq // self.hkv, 0)
        return out, lse, ob, mass, lb


@pytest.mark.parametrize("new", NEWS)
@pytest.mark.parametrize("first", [0, 5, 290])
def test_many_small_weights_beside_a_large_one(cuda_device, new, first):
    """One key scores 18 above the others (their weights are 2^-26 of its) and has no value but in
    channel 0; the others' values, in the other channels, still come out."""
    d = 64
    case = AlikeScales(61, [300], [new], 4, 1, d, 16, True, scale=1.0)
    first = min(first, 300 - new)
    q = np.zeros((new, 4, d), np.float32)
    q[..., 0] = 1
    case.q = bf16_bits_from_f32(q).reshape(q.shape)
    nb, bs = case.kv_bits[1].shape[:2]
    k = np.zeros((nb, bs, 1, d))
    blk, row = case.tables[0, first // 16], first % 16
    k[blk, row, 0, 0] = 18
    v = np.random.default_rng(7).standard_normal((nb, bs, 1, d))
    v[..., 0] = 0
    v[blk, row, 0] = 0
    v[blk, row, 0, 0] = 1
    set_rows(case, 0, k)
    set_rows(case, 1, v)
    for num_splits in (0, 1, 3):
        out, lse = run(case, cuda_device, num_splits)
        check_answers(case, out, lse, bits_of(case), f"{num_splits} splits")


class FineQuery(Case):
    """The share of the query's rounding in the bounds at 2^-39 of its largest element (top
    elements are scaled to [2^14, 2^16) and fp16 steps are 2^-24) instead of 2^-25."""

    def answers(self):
        out, lse, ob, mass, lb = super().answers()
        q = bf16_to_f64(self.q)
        for b, (n, m) in enumerate(zip(self.lens, self.news)):
            rows = slice(self.cu[b], self.cu[b + 1])
            kabs = np.abs(gather(self.values[0], self.tables[b], n, self.bs)).sum(-1).max(0)
            share = 2.0 ** -25 * abs(self.scale) * np.abs(q[rows]).max(-1) * \
                np.repeat(kabs, self.hq // self.hkv)[None, :]
            ob[rows] -= (2 * share * (1 - 2.0 ** -14))[..., None] * mass[rows]
            lb[rows] -= share * (1 - 2.0 ** -14)
        return out, lse, ob, mass, lb


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", NEWS)
@pytest.mark.parametrize("gap", [12, 20, 26])
def test_query_elements_of_very_different_size(cuda_device, d, new, gap):
    """A query's largest element meets keys that are zero there; the scores come from elements
    2^-gap of it."""
    case = FineQuery(71 + d, [150, 40], [new, 1], 4, 1, d, 16, True, scale=1.0)
    rng = np.random.default_rng(gap)
    q = (rng.standard_normal(case.q.shape) * 2.0 ** -gap).astype(np.float32)
    q[..., 3] = 1.5
    case.q = bf16_bits_from_f32(q).reshape(q.shape)
    k = rng.standard_normal(case.kv_bits[0].shape) * 2.0 ** (gap - 3)
    k[..., 3] = 0
    set_rows(case, 0, k)
    for num_splits in (0, 2):
        out, lse = run(case, cuda_device, num_splits)
        check_answers(case, out, lse, bits_of(case), f"{num_splits} splits")
