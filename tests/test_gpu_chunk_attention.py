"""Chunk attention over bf16 and e4m3 caches on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from tests.window_helpers import TILE_BITS, Case, check_answers

pytestmark = pytest.mark.gpu


def _run(case, t, num_splits=0, err=None, **kw):
    return nvpa.chunk_attention(
        t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], max(case.news), max(case.lens),
        case.scale, window=case.window, num_sinks=case.sinks, k_scales=t["k_scales"], v_scales=t["v_scales"],
        num_splits=num_splits, err_flag=err, return_lse=True, **kw)


def _check(dev, case, num_splits=0, what="", **kw):
    t = case.device(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _run(case, t, num_splits, err, **kw)
    assert err.item() == 0, what
    check_answers(case, out, lse, TILE_BITS, what)
    return t, out, lse


CHUNKS = [
    # (context lens, new tokens, Hq, Hkv, D, block size)
    ([1], [1], 4, 2, 64, 16),
    ([5, 9, 300], [5, 2, 3], 8, 2, 128, 16),
    ([40, 0, 77], [7, 0, 1], 7, 1, 64, 32),
    ([257, 128, 129], [130, 128, 1], 4, 4, 128, 256),
    ([700], [33], 12, 4, 64, 64),
    ([513, 300, 31], [257, 12, 31], 6, 2, 128, 128),
    ([1100, 1030], [5, 4], 16, 2, 128, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,news,hq,hkv,d,bs", CHUNKS)
def test_chunks_without_a_window(cuda_device, fp8, lens, news, hq, hkv, d, bs):
    case = Case(sum(lens), lens, news, hq, hkv, d, bs, fp8)
    for ns in (0, 1, 3):
        _check(cuda_device, case, ns, f"{lens} {news} splits {ns}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (128, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (7, 4), (33, 0), (64, 16), (128, 1), (200, 140), (300, 4)])
def test_chunks_with_windows_and_sinks(cuda_device, fp8, d, bs, window, sinks):
    lens, news = [600, 129, 3, 420], [140, 129, 1, 6]
    case = Case(window + sinks + d, lens, news, 4, 2, d, bs, fp8, window, sinks)
    for ns in (0, 2):
        _check(cuda_device, case, ns, f"window {window} sinks {sinks} splits {ns}")


@pytest.mark.parametrize("fp8", [False, True])
def test_long_context_short_chunk(cuda_device, fp8):
    case = Case(77, [4100, 3333], [4, 2], 4, 1, 128, 16, fp8)
    _check(cuda_device, case, 0, "long")
    case = Case(78, [4100], [20], 2, 1, 64, 256, fp8, window=3000, sinks=200)
    _check(cuda_device, case, 0, "long, window")


def test_large_scores(cuda_device):
    for fp8 in (False, True):
        case = Case(5, [400, 90], [70, 90], 8, 2, 128, 16, fp8, q_mult=12.0, spread_scales=True)
        _check(cuda_device, case, 0, f"fp8 {fp8}")
        case = Case(6, [300], [40], 4, 2, 64, 16, fp8, scale=-0.5)
        _check(cuda_device, case, 0, f"negative scale, fp8 {fp8}")


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_behind_the_last_sequence_stay(cuda_device, fp8):
    case = Case(9, [50, 300], [20, 40], 4, 2, 64, 16, fp8, extra_rows=5)
    t = case.device(cuda_device)
    for ns in (0, 1):
        out = torch.full_like(t["q"], 3.0)
        lse = torch.full(t["q"].shape[:2], 9.0, device=cuda_device)
        _run(case, t, ns, out=out, lse=lse)
        check_answers(case, out, lse, TILE_BITS, "extra rows")
        assert (out[60:] == 3.0).all() and (lse[60:] == 9.0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lengths_leave_the_rows_unwritten(cuda_device, fp8):
    dev = cuda_device
    case = Case(10, [50, 300, 70], [20, 40, 7], 4, 2, 64, 16, fp8)
    t = case.device(dev)
    good, glse = _run(case, t)
    for name, value in (("lens", [50, 301, 70]), ("lens", [50, 39, 70]), ("lens", [50, -1, 70])):
        u = dict(t)
        u[name] = torch.tensor(value, dtype=torch.int32, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        out = torch.full_like(t["q"], 3.0)
        out, lse = _run(case, u, err=err, out=out)
        assert err.item() == nvpa.NVPA_FLAG_BAD_LENGTH
        assert torch.equal(out[:20], good[:20]) and torch.equal(out[60:], good[60:])
        assert (out[20:60] == 3.0).all()
    # cumulative lengths that run backwards or past the rows: flagged, in bounds
    for cu in ([0, 60, 30, 67], [0, 20, 60, 80], [-3, 20, 60, 67]):
        u = dict(t, cu=torch.tensor(cu, dtype=torch.int32, device=dev))
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        _run(case, u, err=err)
        assert err.item() & nvpa.NVPA_FLAG_BAD_LENGTH
    # a visible block with an impossible id: flagged, the other sequences unharmed
    u = dict(t, tables=t["tables"].clone())
    u["tables"][1, 3] = case.num_blocks + 5
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, _ = _run(case, u, err=err)
    assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
    assert torch.equal(out[:20], good[:20]) and torch.equal(out[60:], good[60:])
    assert torch.isfinite(out.float()).all()


def test_chunk_by_chunk_equals_the_whole_prompt(cuda_device):
    """A prompt written and attended in three chunks: each row within the bounds of the same
    answer as when the whole prompt is one chunk."""
    dev = cuda_device
    n = 300
    case = Case(12, [n], [n], 8, 2, 128, 16, True, window=90, sinks=4)
    t, out, lse = _check(dev, case, 0, "whole")
    parts = []
    for a, b in ((0, 7), (7, 160), (160, 300)):
        parts.append(nvpa.chunk_attention(
            t["q"][a:b].contiguous(), t["k_cache"], t["v_cache"], t["tables"],
            torch.tensor([0, b - a], dtype=torch.int32, device=dev),
            torch.tensor([b], dtype=torch.int32, device=dev), b - a, b, case.scale, window=90, num_sinks=4,
            k_scales=t["k_scales"], v_scales=t["v_scales"], return_lse=True))
    check_answers(case, torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts]), TILE_BITS, "parts")


def test_store_chunk_decode_as_served(cuda_device):
    """A prompt stored in the 8-bit cache and attended as a chunk, then single tokens stored
    and decoded, each against the oracle's attention over what the cache holds."""
    dev = cuda_device
    lens = [100, 37]
    case = Case(40, [n + 3 for n in lens], [n + 3 for n in lens], 4, 2, 64, 16, True, window=50, sinks=4)
    t = case.device(dev)
    for x in "kv":
        t[x + "_cache"].view(torch.uint8).fill_(0x7F)
        t[x + "_scales"].fill_(255)
    bits = case.kv_bits
    full = np.concatenate([case.tables[b, j // 16] * 16 + j % 16 + 0 * np.arange(1)
                           for b, n in enumerate(case.lens) for j in range(n)])
    rows = bits.reshape(2, -1, 2, 64)[:, full]
    order = [[case.cu[b] + j for j in range(n)] for b, n in enumerate(case.lens)]

    from synth.device import bf16_tensor, i32

    def store(idx):
        nvpa.store_kvcache_fp8(bf16_tensor(rows[0][idx], dev), bf16_tensor(rows[1][idx], dev), t["k_cache"],
                               t["v_cache"], t["k_scales"], t["v_scales"], i32(full[idx], dev))

    tables = i32(case.tables, dev)
    sc = dict(window=50, num_sinks=4, k_scales=t["k_scales"], v_scales=t["v_scales"], return_lse=True)
    out, lse = torch.empty_like(t["q"]), torch.empty(t["q"].shape[:2], device=dev)
    first = np.concatenate([o[:n] for o, n in zip(order, lens)])
    store(first)
    o, l = nvpa.chunk_attention(t["q"][torch.from_numpy(first).to(dev)].contiguous(), t["k_cache"], t["v_cache"], tables,
                                i32([0, lens[0], sum(lens)], dev), i32(lens, dev), max(lens), max(lens),
                                case.scale, **sc)
    out[torch.from_numpy(first).to(dev)] = o
    lse[torch.from_numpy(first).to(dev)] = l
    for s in range(3):
        idx = np.array([o[n + s] for o, n in zip(order, lens)])
        store(idx)
        at = torch.from_numpy(idx).to(dev)
        o, l = nvpa.paged_decode_attention_window(t["q"][at].contiguous(), t["k_cache"], t["v_cache"], tables,
                                                  i32([n + s + 1 for n in lens], dev), max(lens) + s + 1,
                                                  case.scale, **sc)
        out[at] = o
        lse[at] = l
    check_answers(case, out, lse, TILE_BITS, "served")


def test_captured_and_replayed(cuda_device):
    dev = cuda_device
    for fp8 in (False, True):
        case = Case(50, [200, 333], [70, 5], 4, 2, 128, 16, fp8, window=100, sinks=4)
        t = case.device(dev)
        ws = torch.empty(nvpa.chunk_attention_workspace_size(2, 75, 4, 2, 128, 70, 333, 16, 100, 4), dtype=torch.uint8,
                         device=dev)
        out, lse = torch.empty_like(t["q"]), torch.empty((75, 4), device=dev)
        _run(case, t, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _run(case, t, out=out, lse=lse, workspace=ws)
        for _ in range(2):
            ws.fill_(0xFF)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            check_answers(case, out, lse, TILE_BITS, "replay")


def test_two_streams_with_workspaces_of_their_own(cuda_device):
    dev = cuda_device
    cases = [Case(60 + i, [900, 40], [33, 2], 4, 2, 64, 16, bool(i)) for i in range(2)]
    ts = [c.device(dev) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [_run(c, t, stream=s) for c, t, s in zip(cases, ts, streams)]
    torch.cuda.synchronize()
    for c, (out, lse) in zip(cases, got):
        check_answers(c, out, lse, TILE_BITS, "two streams")
