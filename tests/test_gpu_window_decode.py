"""Windowed decode over bf16 and e4m3 caches on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from tests.window_helpers import ROW_BITS, Case, check_answers

pytestmark = pytest.mark.gpu


def _run(case, t, num_splits=0, err=None, max_ctx=None, **kw):
    return nvpa.paged_decode_attention_window(
        t["q"], t["k_cache"], t["v_cache"], t["tables"], t["lens"], max_ctx or max(1, max(case.lens)), case.scale,
        window=case.window, num_sinks=case.sinks, k_scales=t["k_scales"], v_scales=t["v_scales"],
        num_splits=num_splits, err_flag=err, return_lse=True, **kw)


def _check(dev, case, num_splits=0, what="", **kw):
    t = case.device(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _run(case, t, num_splits, err, **kw)
    assert err.item() == 0, what
    check_answers(case, out, lse, ROW_BITS[case.fp8], what)
    return t, out, lse


def _ones(lens):
    return [1] * len(lens)


SHAPES = [
    # (context lens, Hq, Hkv, D, block size)
    ([1, 2, 15, 16, 17], 4, 4, 64, 16),
    ([0, 1, 300, 33], 8, 4, 64, 32),
    ([64, 65, 127, 128, 129], 6, 2, 128, 64),
    ([1000, 5, 257], 8, 1, 128, 128),
    ([511, 512, 513, 1], 16, 2, 128, 256),
    ([77, 300], 7, 1, 64, 16),
    ([2000, 31], 12, 4, 128, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d,bs", SHAPES)
def test_shapes_without_a_window(cuda_device, fp8, lens, hq, hkv, d, bs):
    case = Case(sum(lens) + hq, lens, _ones(lens), hq, hkv, d, bs, fp8)
    for ns in (0, 1, 3):
        _check(cuda_device, case, ns, f"{lens} splits={ns}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 32), (128, 256)])
@pytest.mark.parametrize("window,sinks", [
    (1, 0), (1, 1), (7, 4), (16, 0), (17, 3), (64, 16), (100, 130), (250, 17), (257, 4), (4096, 4), (2**31 - 1, 2**31 - 1),
])
def test_windows_and_sinks(cuda_device, fp8, d, bs, window, sinks):
    lens = [1, 16, 97, 256, 257, 700, 0]
    case = Case(window % 1000 + sinks % 1000 + d, lens, _ones(lens), 8, 2, d, bs, fp8, window, sinks)
    for ns in (0, 2):
        _check(cuda_device, case, ns, f"window {window} sinks {sinks} splits {ns}")


@pytest.mark.parametrize("fp8", [False, True])
def test_many_sequences_long_and_short(cuda_device, fp8):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 1500, size=70)]
    case = Case(8, lens, _ones(lens), 4, 2, 128, 16, fp8)
    t, a, la = _check(cuda_device, case, 0, "70 sequences")
    # the same call again gives the same bits
    b, lb = _run(case, t)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("spread", [False, True])
def test_large_scores_and_rows_of_very_different_size(cuda_device, spread):
    lens = [300, 41, 513]
    for fp8 in (False, True):
        case = Case(21, lens, _ones(lens), 8, 2, 128, 16, fp8, q_mult=16.0, spread_scales=spread)
        _check(cuda_device, case, 0, f"fp8 {fp8}")
        case = Case(22, lens, _ones(lens), 8, 2, 64, 32, fp8, q_mult=1e-3, scale=-3.0, spread_scales=spread)
        _check(cuda_device, case, 2, f"negative scale, fp8 {fp8}")


def test_agrees_with_the_unwindowed_decode(cuda_device):
    """bf16 cache, no window: the same attention as paged_decode_attention.  Both are within
    the bounds of the same answer, so they differ by at most twice that."""
    lens = [700, 33, 1]
    case = Case(3, lens, _ones(lens), 8, 4, 128, 16, False)
    t, out, lse = _check(cuda_device, case)
    ref, rlse = nvpa.paged_decode_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["lens"], 700,
                                            case.scale, return_lse=True)
    _, _, ob, mass, lb = case.answers()
    assert ((out.double() - ref.double()).abs().cpu().numpy() <= 2 * (ob + 2.0 ** -16 * mass)).all()
    assert ((lse.double() - rlse.double()).abs().cpu().numpy() <= 2 * lb).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lengths_and_blocks_are_flagged(cuda_device, fp8):
    dev = cuda_device
    lens = [40, 40, 40]
    case = Case(4, lens, _ones(lens), 4, 2, 64, 16, fp8, window=20)
    t = case.device(dev)
    good, _ = _run(case, t)
    # a length above the bound is clamped to it, a negative one is empty
    t["lens"] = torch.tensor([41, -5, 40], dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _run(case, t, err=err)
    assert err.item() == nvpa.NVPA_FLAG_BAD_LENGTH
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    # a visible block with an impossible id: its rows are absent, other sequences unharmed
    t = case.device(dev)
    t["tables"][1, 2] = case.num_blocks
    err.zero_()
    out, lse = _run(case, t, err=err)
    assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
    assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.isfinite(out.float()).all()


def test_captured_and_replayed_with_new_lengths(cuda_device):
    dev = cuda_device
    lens = [64, 200, 9, 1]
    cases = [Case(30 + i, x, _ones(x), 8, 2, 128, 16, True, window=50, sinks=3)
             for i, x in enumerate((lens, [130, 7, 200, 0]))]
    width = max(c.tables.shape[1] for c in cases)
    nb = max(c.num_blocks for c in cases)
    t = cases[0].device(dev)
    buf = dict(q=t["q"].clone(), lens=t["lens"].clone(),
               tables=torch.full((4, width), -1, dtype=torch.int32, device=dev))
    for x in "kv":
        buf[x + "_cache"] = torch.zeros((nb,) + t[x + "_cache"].shape[1:], dtype=torch.uint8, device=dev)
        buf[x + "_scales"] = torch.zeros((nb,) + t[x + "_scales"].shape[1:], dtype=torch.uint8, device=dev)

    def load(c):
        d = c.device(dev)
        buf["q"].copy_(d["q"])
        buf["lens"].copy_(d["lens"])
        buf["tables"][:, :c.tables.shape[1]] = d["tables"]
        for x in "kv":
            buf[x + "_cache"][:c.num_blocks] = d[x + "_cache"].view(torch.uint8)
            buf[x + "_scales"][:c.num_blocks] = d[x + "_scales"]

    load(cases[0])
    ws = torch.empty(nvpa.paged_decode_window_workspace_size(4, 8, 2, 128, 256, 16, 50, 3), dtype=torch.uint8,
                     device=dev)
    out, lse = torch.empty_like(buf["q"]), torch.empty((4, 8), dtype=torch.float32, device=dev)

    def call():
        nvpa.paged_decode_attention_window(
            buf["q"], buf["k_cache"].view(torch.float8_e4m3fn), buf["v_cache"].view(torch.float8_e4m3fn),
            buf["tables"], buf["lens"], 256, cases[0].scale, window=50, num_sinks=3, k_scales=buf["k_scales"],
            v_scales=buf["v_scales"], out=out, lse=lse, workspace=ws, return_lse=True)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in (cases[1], cases[0], cases[1]):
        load(c)
        ws.fill_(0xFF)       # nothing in the workspace has to survive
        graph.replay()
        torch.cuda.synchronize()
        check_answers(c, out, lse, ROW_BITS[True], "replay")


def test_refusals_of_the_binding(cuda_device):
    dev = cuda_device
    case = Case(1, [20, 20], [1, 1], 4, 2, 64, 16, True)
    t = case.device(dev)
    args = (t["q"], t["k_cache"], t["v_cache"], t["tables"], t["lens"], 20, 0.125)
    sc = dict(k_scales=t["k_scales"], v_scales=t["v_scales"])
    f = nvpa.paged_decode_attention_window
    with pytest.raises(TypeError):
        f(*args)                                                  # e4m3 without scales
    with pytest.raises(ValueError):
        f(*args, k_scales=t["k_scales"])
    with pytest.raises(ValueError):
        f(*args, k_scales=t["k_scales"][:1].contiguous(), v_scales=t["v_scales"])
    with pytest.raises(ValueError):
        f(*args, **sc, out=t["q"][:1].clone())
    with pytest.raises(ValueError):
        f(*args, **sc, lse=torch.empty((2, 3), device=dev))
    with pytest.raises(ValueError):
        f(*args[:4], t["lens"][:1], 20, 0.125, **sc)
    with pytest.raises(ValueError):
        f(*args, **sc, err_flag=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(nvpa.NvpaError):
        f(*args, **sc, window=-1)
    with pytest.raises(nvpa.NvpaError):
        f(*args, **sc, workspace=torch.empty(256, dtype=torch.uint8, device=dev))


def test_empty_batch(cuda_device):
    case = Case(1, [20], [1], 4, 2, 64, 16, True)
    t = case.device(cuda_device)
    out = nvpa.paged_decode_attention_window(t["q"][:0], t["k_cache"], t["v_cache"], t["tables"][:0], t["lens"][:0], 20,
                                             0.1, k_scales=t["k_scales"], v_scales=t["v_scales"])
    assert out.shape == (0, 4, 64)
