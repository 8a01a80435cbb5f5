"""The 8-bit cache, the windowed decode and the chunk attention without a GPU: the oracle's
own pins, and what the entry points refuse before they touch the device."""

import math

import numpy as np
import pytest
import torch

from oracle.paged_attention import bf16_to_f64
from oracle.window_attention import (attend, dequantise_rows, e4m3_to_f64, f64_to_e4m3, quantise_rows,
                                     seen)
import paged_kv_cache_422_b200 as nvpa
from paged_kv_cache_422_b200 import _lib
from synth.workloads import bf16_bits_from_f32

FAKE = 0x10000  # 256-byte aligned fake device address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_422_b200.build import build
    build()
    return _lib.lib()


# ---------------------------------------------------------------- the oracle's pins

def test_e4m3_table_agrees_with_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3_to_f64(codes), want, equal_nan=True)


def test_rounding_agrees_with_torch_at_every_bf16_value_in_range():
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    x = bf16_to_f64(bits)
    ok = np.isfinite(x) & (np.abs(x) <= 448)
    want = torch.from_numpy(x[ok]).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f64_to_e4m3(x[ok]), want)


def test_every_finite_row_maximum_fits_and_reads_back_within_half_a_step():
    """Rows of one value: |code| <= 448 uses the top binade but for the smallest rows, and the
    value read back is off by at most u(e4m3) = 2^-4 relative (2^-128 at the smallest)."""
    bits = np.arange(1, 0x7F80, dtype=np.uint32).astype(np.uint16)[:, None]
    codes, scales = quantise_rows(bits)
    x = bf16_to_f64(bits)
    mag = np.abs(e4m3_to_f64(codes))
    assert (mag <= 448).all() and (mag[x >= 2.0 ** -109] >= 224).all()
    assert scales.min() == 9 and scales.max() == 247
    err = np.abs(dequantise_rows(codes, scales) - x)
    assert (err <= np.maximum(2.0 ** -4 * x, 2.0 ** -128)).all()


def test_reading_back_is_exact_in_bf16():
    codes = np.arange(256, dtype=np.uint8)
    for b in (9, 10, 100, 127, 200, 246):
        v = dequantise_rows(codes, np.asarray(b))
        v = v[np.isfinite(v)]
        assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def test_non_finite_values_become_nan_codes_and_do_not_scale_the_row():
    row = bf16_bits_from_f32(np.array([1.0, -2.0, 0.0, 0.5], np.float32))
    row[2] = 0x7F80
    c, s = quantise_rows(row[None])
    assert c[0, 2] == 0x7F and dequantise_rows(c, s)[0, [0, 1, 3]].tolist() == [1.0, -2.0, 0.5]
    row[1] = 0xFFC0
    c, s = quantise_rows(row[None])
    assert c[0, 1] == 0x7F and dequantise_rows(c, s)[0, 0] == 1.0


def test_window_and_sinks_by_hand():
    assert seen(8, 5, 3, 0).tolist() == [0, 0, 0, 1, 1, 1, 0, 0]
    assert seen(8, 5, 3, 2).tolist() == [1, 1, 0, 1, 1, 1, 0, 0]
    assert seen(8, 5, 0, 2).tolist() == [1] * 6 + [0] * 2
    assert seen(8, 1, 4, 6).tolist() == [1, 1] + [0] * 6      # sinks do not see the future


def test_attend_agrees_with_torch_sdpa():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    pos = np.arange(4, 9)
    out, lse, _, _ = attend(q, k, v, pos, 3, 1, 0.3)
    mask = np.stack([seen(9, p, 3, 1) for p in pos])
    tq = torch.from_numpy(q).transpose(0, 1)
    tk, tv = (torch.from_numpy(np.repeat(x, 2, 1)).transpose(0, 1) for x in (k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, torch.from_numpy(mask), scale=0.3)
    assert np.allclose(out, ref.transpose(0, 1).numpy(), atol=1e-12)
    s = torch.einsum("hld,hnd->hln", tq, tk) * 0.3
    s = s.masked_fill(~torch.from_numpy(mask), -math.inf)
    assert np.allclose(lse, torch.logsumexp(s, -1).T.numpy(), atol=1e-12)


# ---------------------------------------------------------------- refusals of the C ABI

def _store(lib, **kw):
    a = dict(k=FAKE, v=FAKE, ks=256, vs=256, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, slots=FAKE, n=4, hkv=2,
             d=128, nb=8, bs=16)
    a.update(kw)
    return lib.nvpa_store_kvcache_fp8(a["k"], a["v"], a["ks"], a["vs"], a["kc"], a["vc"], a["ksc"], a["vsc"],
                                      a["slots"], a["n"], a["hkv"], a["d"], a["nb"], a["bs"], None, None)


INVALID, UNSUPPORTED, OK = _lib.NVPA_ERR_INVALID_ARG, _lib.NVPA_ERR_UNSUPPORTED, _lib.NVPA_OK


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(n=0, k=None), OK), (dict(ks=255), INVALID), (dict(vs=128), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(hkv=0), INVALID),
    (dict(ksc=None), INVALID), (dict(vsc=FAKE + 8), INVALID), (dict(kc=FAKE + 2), INVALID),
    (dict(slots=None), INVALID), (dict(nb=1 << 24, bs=256), UNSUPPORTED), (dict(nb=0), INVALID),
])
def test_store_fp8_refuses(lib, kw, status):
    assert _store(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(total=-1), INVALID), (dict(total=0, dst=None), OK), (dict(bs=24), UNSUPPORTED),
    (dict(d=32), UNSUPPORTED), (dict(dst=None), INVALID), (dict(sc=None), INVALID), (dict(sc=FAKE + 4), INVALID),
    (dict(width=0), INVALID), (dict(batch=-1), INVALID),
])
def test_gather_fp8_refuses(lib, kw, status):
    a = dict(dst=FAKE, sc=FAKE, width=4, batch=2, total=10, d=64, bs=16)
    a.update(kw)
    assert lib.nvpa_gather_kv_fp8(a["dst"], FAKE, a["sc"], FAKE, a["width"], FAKE, a["batch"], a["total"], 2,
                                  a["d"], 8, a["bs"], None, None) == status


WINDOW_REFUSALS = [
    (dict(d=96), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(hq=6, hkv=4), INVALID),
    (dict(hq=18, hkv=2), UNSUPPORTED), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(ws=FAKE + 16), INVALID), (dict(ws=None), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(batch=-1), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(kind=2), INVALID), (dict(kind=0), INVALID),       # scales, bf16
    (dict(ksc=None), INVALID), (dict(vsc=FAKE + 8), INVALID), (dict(maxctx=-1), INVALID), (dict(ns=-1), INVALID),
    (dict(maxctx=100000, wsb=16), _lib.NVPA_ERR_WORKSPACE_TOO_SMALL), (dict(maxblk=0), INVALID),
    (dict(nb=1 << 28, bs=16), UNSUPPORTED), (dict(batch=0), OK),
]


def _args(kw):
    a = dict(out=FAKE, lse=None, q=FAKE, k=FAKE, v=FAKE, kind=1, ksc=FAKE, vsc=FAKE, bt=FAKE, maxblk=4, cu=FAKE,
             ctx=FAKE, batch=2, total=6, maxq=4, hq=8, hkv=2, d=128, nb=16, bs=16, maxctx=64, scale=0.1, window=0,
             sinks=0, ns=0, ws=FAKE, wsb=1 << 24)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", WINDOW_REFUSALS)
def test_window_decode_refuses(lib, kw, status):
    a = _args(kw)
    assert lib.nvpa_paged_decode_attention_window(
        a["out"], a["lse"], a["q"], a["k"], a["v"], a["kind"], a["ksc"], a["vsc"], a["bt"], a["maxblk"], a["ctx"],
        a["batch"], a["hq"], a["hkv"], a["d"], a["nb"], a["bs"], a["maxctx"], a["scale"], a["window"], a["sinks"],
        a["ns"], a["ws"], a["wsb"], None, None) == status


@pytest.mark.parametrize("kw,status", WINDOW_REFUSALS + [
    (dict(total=-1), INVALID), (dict(total=0, q=None), OK), (dict(maxq=-1), INVALID), (dict(cu=None), INVALID),
    (dict(total=1 << 30), UNSUPPORTED),
])
def test_chunk_attention_refuses(lib, kw, status):
    a = _args(kw)
    assert lib.nvpa_chunk_attention(
        a["out"], a["lse"], a["q"], a["k"], a["v"], a["kind"], a["ksc"], a["vsc"], a["bt"], a["maxblk"], a["cu"],
        a["ctx"], a["batch"], a["total"], a["maxq"], a["maxctx"], a["hq"], a["hkv"], a["d"], a["nb"], a["bs"],
        a["scale"], a["window"], a["sinks"], a["ns"], a["ws"], a["wsb"], None, None) == status


def test_workspace_sizes_are_host_only(lib):
    f = lib.nvpa_paged_decode_window_workspace_size
    assert 0 < f(64, 16, 8, 128, 4096, 256, 512, 4, 0) < f(64, 16, 8, 128, 65536, 256, 0, 0, 0)
    assert f(64, 16, 8, 128, 1 << 20, 256, 512, 4, 0) == f(64, 16, 8, 128, 1 << 24, 256, 512, 4, 0)
    assert f(-1, 16, 8, 128, 4096, 256, 0, 0, 0) == 0 and f(4, 15, 8, 128, 4096, 256, 0, 0, 0) == 0
    assert f(4, 16, 8, 128, 4096, 24, 0, 0, 0) == 0 and f(4, 16, 8, 128, 4096, 256, -1, 0, 0) == 0
    # windows and sinks of any size do not overflow
    big = (1 << 31) - 1
    assert f(1, 16, 8, 128, 4096, 256, big, big, 0) == f(1, 16, 8, 128, 4096, 256, 0, 0, 0)
    g = lib.nvpa_chunk_attention_workspace_size
    assert 0 < g(2, 600, 16, 8, 128, 512, 8192, 256, 0, 0, 0)
    assert g(2, -1, 16, 8, 128, 512, 8192, 256, 0, 0, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    kc = torch.zeros((2, 16, 2, 64), dtype=torch.float8_e4m3fn)
    sc = torch.zeros((2, 2, 16), dtype=torch.uint8)
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nvpa.store_kvcache_fp8(x, x, kc, kc, sc, sc, slots)
    with pytest.raises(TypeError):
        nvpa.store_kvcache_fp8(x, x, kc.view(torch.uint8), kc, sc, sc, slots)
    with pytest.raises(ValueError, match="CUDA"):
        nvpa.gather_kv_fp8(kc, sc, slots[None], slots, 1)
    with pytest.raises(ValueError, match="together"):
        nvpa.paged_decode_attention_window(x, kc, kc, slots[None], slots, 1, 1.0, k_scales=sc)
