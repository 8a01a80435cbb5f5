"""The 8-bit store takes rows of any token stride: of a dimension of size 1 the stride says nothing."""

import pytest
import torch

import paged_kv_cache_422_b200 as nvpa

pytestmark = pytest.mark.gpu


def _rows(kind, n, hkv, d, dev):
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((n, hkv, d), generator=g, device=dev).to(torch.bfloat16)
    if kind == "heads first":                 # [Hkv, N, D] transposed, as attention layers hold it
        return x, x.transpose(0, 1).contiguous().transpose(0, 1)
    if kind == "expanded":
        return x, x.as_strided(x.shape, (0 if n == 1 else hkv * d, d, 1))
    if kind == "odd stride":
        return x, x.as_strided(x.shape, (hkv * d + 3 if n == 1 else hkv * d, d if hkv > 1 else 5, 1))
    wide = torch.zeros((n, hkv * d + 8), dtype=torch.bfloat16, device=dev)     # one head of a wider row
    wide[:, 8:] = x.flatten(1)
    return x, wide[:, 8:].unflatten(1, (hkv, d))


@pytest.mark.parametrize("kind", ["heads first", "expanded", "odd stride", "wide"])
@pytest.mark.parametrize("n,hkv", [(1, 4), (1, 1), (7, 1)])
def test_strides(cuda_device, kind, n, hkv):
    dev, d, bs = cuda_device, 64, 16
    x, view = _rows(kind, n, hkv, d, dev)
    assert torch.equal(x, view)
    got = []
    for k in (x, view):
        pools = [torch.zeros((2, bs, hkv, d), dtype=torch.float8_e4m3fn, device=dev) for _ in "kv"]
        scales = [torch.zeros((2, hkv, bs), dtype=torch.uint8, device=dev) for _ in "kv"]
        nvpa.store_kvcache_fp8(k, k, *pools, *scales, torch.arange(3, 3 + n, dtype=torch.int32, device=dev))
        got.append([p.view(torch.uint8) for p in pools] + scales)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert bool(got[0][0].any())


def test_rows_that_are_not_contiguous_are_refused(cuda_device):
    dev = cuda_device
    x = torch.zeros((4, 3, 128), dtype=torch.bfloat16, device=dev)
    pools = [torch.zeros((2, 16, 3, 64), dtype=torch.float8_e4m3fn, device=dev) for _ in "kv"]
    scales = [torch.zeros((2, 3, 16), dtype=torch.uint8, device=dev) for _ in "kv"]
    slots = torch.arange(4, dtype=torch.int32, device=dev)
    for bad in (x[..., :64], x[..., ::2], x.view(3, 4, 128).transpose(0, 1)[..., :64]):
        with pytest.raises(ValueError, match="contiguous"):
            nvpa.store_kvcache_fp8(bad, bad, *pools, *scales, slots)
    y = torch.zeros((4, 3 * 64 + 4), dtype=torch.bfloat16, device=dev)[:, :192].unflatten(1, (3, 64))
    with pytest.raises(nvpa.NvpaError):       # a token stride that is not a multiple of 16 bytes
        nvpa.store_kvcache_fp8(y, y, *pools, *scales, slots)
