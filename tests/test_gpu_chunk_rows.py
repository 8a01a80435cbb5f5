"""Chunks of few rows, which run as the decode does: held to the weights' bits of that kernel, with and
without a plan kernel ahead of it, in batches as an engine has them."""

import itertools

import numpy as np
import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from tests.window_helpers import ROW_BITS, Case, check_answers

pytestmark = pytest.mark.gpu


class Once(Case):
    """A case whose answers are computed once."""

    def answers(self):
        if not hasattr(self, "known"):
            self.known = super().answers()
        return self.known


def _run(case, t, num_splits=0, **kw):
    assert max(case.news) * (case.hq // case.hkv) <= (24 if case.fp8 else 16)      # the row kernel's
    return nvpa.chunk_attention(
        t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], max(case.news), max(case.lens), case.scale,
        window=case.window, num_sinks=case.sinks, k_scales=t["k_scales"], v_scales=t["v_scales"],
        num_splits=num_splits, return_lse=True, **kw)


def _check(dev, case, num_splits, what):
    t = case.device(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _run(case, t, num_splits, err_flag=err)
    assert err.item() == 0, what
    check_answers(case, out, lse, ROW_BITS[case.fp8], what)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3), (300, 17)])
@pytest.mark.parametrize("lens,news,hq,hkv,d,bs", [
    ([5, 9, 300], [2, 1, 2], 8, 2, 128, 16),
    ([40, 0, 77], [2, 0, 1], 7, 1, 64, 32),
    ([257, 128, 12], [16, 9, 12], 4, 4, 128, 256),
    ([700, 16], [5, 3], 12, 4, 64, 64),
    ([1100, 1030], [2, 1], 16, 2, 128, 128),
    ([513, 31], [8, 8], 2, 1, 64, 16),
])
def test_shapes(cuda_device, fp8, window, sinks, lens, news, hq, hkv, d, bs):
    case = Once(sum(lens) + window, lens, news, hq, hkv, d, bs, fp8, window, sinks)
    for ns in (0, 1, 3):
        _check(cuda_device, case, ns, f"splits {ns}")


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 4)])
@pytest.mark.parametrize("lens,news,hq,hkv,d", [
    ([1300, 257, 31], [24, 24, 24], 2, 2, 128), ([900, 333], [6, 5], 4, 1, 64), ([2000, 40], [3, 3], 16, 2, 128),
    ([600, 77], [12, 11], 4, 2, 64), ([515], [20], 1, 1, 128),
])
def test_24_rows(cuda_device, window, sinks, lens, news, hq, hkv, d):
    case = Once(sum(lens) + 1, lens, news, hq, hkv, d, 16, True, window, sinks)
    for ns in (0, 1, 4):
        _check(cuda_device, case, ns, f"splits {ns}")


# batches of more than 128 sequences, and more items than the GPU holds warps: both have a plan kernel
BATCHES = [
    (129, 300, 5, 4, 2, 64, 16),
    (200, 500, 5, 8, 2, 64, 32),
    (64, 1500, 5, 16, 8, 64, 16),
    (150, 400, 2, 16, 4, 128, 64),
    (40, 2600, 1, 8, 8, 64, 256),
]


def _batch(fp8, batch, longest, most, hq, hkv, d, bs, window, sinks):
    rng = np.random.default_rng(batch + most)
    news = rng.integers(0, most + 1, size=batch)
    news[:2] = most, 0
    lens = [int(max(m, rng.integers(0, longest + 1))) for m in news]
    lens[0] = longest
    return Once(batch + d, lens, [int(m) for m in news], hq, hkv, d, bs, fp8, window, sinks, extra_rows=3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
@pytest.mark.parametrize("batch", BATCHES)
def test_large_batches(cuda_device, fp8, window, sinks, batch):
    dev = cuda_device
    if not fp8 and batch[2] * (batch[3] // batch[4]) > 16:
        batch = batch[:2] + (4,) + batch[3:]
    case = _batch(fp8, *batch, window, sinks)
    t = case.device(dev)
    for ns in (0, 1, 4):
        out, lse = torch.full_like(t["q"], 3.0), torch.full(t["q"].shape[:2], 9.0, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        _run(case, t, ns, out=out, lse=lse, err_flag=err)
        assert err.item() == 0
        check_answers(case, out, lse, ROW_BITS[fp8], f"splits {ns}")
        assert bool((out[case.total:] == 3.0).all()) and bool((lse[case.total:] == 9.0).all())
        again, again_lse = _run(case, t, ns)
        assert torch.equal(out[:case.total], again[:case.total]) and torch.equal(lse[:case.total], again_lse[:case.total])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", BATCHES[:3])
def test_a_bad_length_in_a_large_batch(cuda_device, fp8, batch):
    """The sequence is flagged and its rows stay as they were; the others do not notice."""
    dev = cuda_device
    if not fp8:
        batch = batch[:2] + (4,) + batch[3:]
    case = _batch(fp8, *batch, 0, 0)
    t = case.device(dev)
    lens = t["lens"].clone()
    for num_splits, value in itertools.product((0, 1, 4), (-1, case.news[0] - 1, max(case.lens) + 1)):
        t["lens"].copy_(lens)
        good, good_lse = _run(case, t, num_splits)
        t["lens"][0] = value
        out, lse = torch.full_like(t["q"], 3.0), torch.full(t["q"].shape[:2], 9.0, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        _run(case, t, num_splits, out=out, lse=lse, err_flag=err)
        assert err.item() == nvpa.NVPA_FLAG_BAD_LENGTH
        rows = case.news[0]
        assert bool((out[:rows] == 3.0).all()) and bool((lse[:rows] == 9.0).all())
        assert torch.equal(out[rows:case.total], good[rows:case.total])
        assert torch.equal(lse[rows:case.total], good_lse[rows:case.total])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_large_batch_captured_and_replayed(cuda_device, fp8):
    dev = cuda_device
    case = _batch(fp8, 150, 400, 4, 8, 2, 64, 16, 90, 4)
    t = case.device(dev)
    size = nvpa.chunk_attention_workspace_size(150, len(t["q"]), 8, 2, 64, max(case.news), max(case.lens), 16, 90, 4)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    out, lse = torch.full_like(t["q"], 3.0), torch.full(t["q"].shape[:2], 9.0, device=dev)
    _run(case, t, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(case, t, out=out, lse=lse, workspace=ws)
    for _ in range(2):
        ws.fill_(0xFF)
        out.zero_()
        graph.replay()
        check_answers(case, out, lse, ROW_BITS[fp8], "replay")
