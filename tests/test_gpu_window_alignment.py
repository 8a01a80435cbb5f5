"""Tensors that start 16 bytes into their storage (4 bytes for int32 ones), as slices of larger buffers
do: the same bits as from tensors of their own."""

import numpy as np
import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from synth.device import i32
from tests.window_helpers import Case

pytestmark = pytest.mark.gpu


def _shifted(t):
    """t's values in memory that starts one 16-byte step (one element of 4 bytes) into a buffer."""
    by = 1 if t.element_size() == 4 else 16 // t.element_size()
    flat = t.contiguous().view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.contiguous()
    buf = torch.zeros(flat.numel() + by, dtype=flat.dtype, device=t.device)
    buf[by:] = flat.flatten()
    out = buf[by:].view(flat.shape)
    out = out.view(t.dtype) if t.dtype == torch.float8_e4m3fn else out
    assert out.data_ptr() % 32 == (4 if by == 1 else 16) and out.is_contiguous()
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 4, 30, 140])
def test_attention(cuda_device, fp8, d, new):
    case = Case(11 + d + new, [300, 200], [new, max(1, new // 3)], 4, 2, d, 16, fp8, window=150, sinks=3)
    t = case.device(cuda_device)
    s = {k: v if v is None else _shifted(v) for k, v in t.items()}

    def run(t, **kw):
        return nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], new, 300,
                                    case.scale, window=150, num_sinks=3, k_scales=t["k_scales"], v_scales=t["v_scales"],
                                    return_lse=True, **kw)

    for num_splits in (0, 1):
        want, want_lse = run(t, num_splits=num_splits)
        out, lse = run(s, num_splits=num_splits, out=_shifted(torch.zeros_like(want)),
                       lse=_shifted(torch.zeros_like(want_lse)))
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        if new == 1:
            out, lse = nvpa.paged_decode_attention_window(
                s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], 300, case.scale, window=150, num_sinks=3,
                k_scales=s["k_scales"], v_scales=s["v_scales"], num_splits=num_splits, return_lse=True,
                out=_shifted(torch.zeros_like(want)), lse=_shifted(torch.zeros_like(want_lse)))
            assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("d,hkv", [(64, 1), (64, 3), (128, 8)])
def test_store_and_read_back(cuda_device, d, hkv):
    dev, n, bs = cuda_device, 77, 32
    g = torch.Generator(device=dev).manual_seed(2)
    k, v = (torch.randn((n, hkv, d), generator=g, device=dev).to(torch.bfloat16) for _ in "kv")
    slots = torch.randperm(4 * bs, generator=g, device=dev)[:n].to(torch.int32)
    pools = []
    for shift in (lambda t: t, _shifted):
        p = [shift(torch.zeros((4, bs, hkv, d), dtype=torch.float8_e4m3fn, device=dev)) for _ in "kv"]
        p += [shift(torch.zeros((4, hkv, bs), dtype=torch.uint8, device=dev)) for _ in "kv"]
        nvpa.store_kvcache_fp8(shift(k), shift(v), *p, shift(slots))
        pools.append(p)
    for a, b in zip(*pools):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    tables, cu = i32(np.array([[3, 1, 0], [2, 0, 1]]), dev), i32(np.array([0, 90, 131]), dev)
    want = nvpa.gather_kv_fp8(pools[0][0], pools[0][2], tables, cu, 131)
    out = _shifted(torch.zeros_like(want))
    nvpa.gather_kv_fp8(pools[1][0], pools[1][2], _shifted(tables), _shifted(cu), 131, out=out)
    assert torch.equal(out, want)


def test_smaller_steps_are_refused(cuda_device):
    case = Case(3, [40], [3], 4, 2, 64, 16, True)
    t = case.device(cuda_device)

    def odd(t):
        return torch.zeros(t.numel() + 4, dtype=t.dtype, device=t.device)[4:].view(t.shape)

    for name in ("q", "k_scales", "v_scales"):
        with pytest.raises(nvpa.NvpaError, match="align"):
            s = dict(t, **{name: odd(t[name])})
            nvpa.chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["cu"], s["lens"], 3, 40, 0.1,
                                 k_scales=s["k_scales"], v_scales=s["v_scales"])
