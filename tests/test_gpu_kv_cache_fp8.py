"""The 8-bit cache on the GPU: rows quantised as they are stored, and read back, bit for bit
against the float64 oracle."""

import numpy as np
import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from oracle.window_attention import dequantise_rows, quantise_rows
from synth.device import bf16_tensor, bits_of, i32
from synth.workloads import bf16_bits_from_f32

pytestmark = pytest.mark.gpu

FILL = 0xA5


def _pools(nb, bs, hkv, d, dev):
    code = lambda: torch.full((nb, bs, hkv, d), FILL, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)  # noqa: E731
    scale = lambda: torch.full((nb, hkv, bs), FILL, dtype=torch.uint8, device=dev)  # noqa: E731
    return code(), code(), scale(), scale()


def _expect(bits, slots, nb, bs, hkv, d):
    codes = np.full((nb, bs, hkv, d), FILL, np.uint8)
    scales = np.full((nb, bs, hkv), FILL, np.uint8)
    c, s = quantise_rows(bits)
    for t, slot in enumerate(slots):
        if 0 <= slot < nb * bs:
            codes[slot // bs, slot % bs] = c[t]
            scales[slot // bs, slot % bs] = s[t]
    return codes, scales.transpose(0, 2, 1)


def _check(dev, kb, vb, slots, nb, bs, pad=0, flags=0):
    n, hkv, d = kb.shape
    kc, vc, ks, vs = _pools(nb, bs, hkv, d, dev)

    def strided(bits):   # token stride hkv * d + pad
        full = np.zeros((n, hkv * d + pad), np.uint16)
        full[:, :hkv * d] = bits.reshape(n, -1)
        return bf16_tensor(full, dev)[:, :hkv * d].unflatten(1, (hkv, d))

    err = torch.zeros(1, dtype=torch.int32, device=dev)
    nvpa.store_kvcache_fp8(strided(kb), strided(vb), kc, vc, ks, vs, i32(slots, dev), err_flag=err)
    assert err.item() == flags
    for got_c, got_s, bits in ((kc, ks, kb), (vc, vs, vb)):
        codes, scales = _expect(bits, slots, nb, bs, hkv, d)
        assert np.array_equal(got_c.view(torch.uint8).cpu().numpy(), codes)
        assert np.array_equal(got_s.cpu().numpy(), scales)


@pytest.mark.parametrize("n,hkv,d,bs,pad", [
    (1, 1, 64, 16, 0), (5, 2, 64, 16, 8), (33, 8, 128, 256, 0), (7, 3, 128, 32, 24), (600, 5, 64, 64, 0),
    (2500, 8, 128, 128, 8),
])
def test_store_matches_oracle(cuda_device, n, hkv, d, bs, pad):
    rng = np.random.default_rng(n)
    x = rng.standard_normal((2, n, hkv, d)) * np.exp2(rng.integers(-40, 40, size=(2, n, hkv, 1)))
    x[:, :, :, ::17] = 0
    kb, vb = bf16_bits_from_f32(x.astype(np.float32)).reshape(x.shape)
    nb = -(-n // bs) + 2
    slots = rng.permutation(nb * bs)[:n]
    flags = 0
    if n > 3:
        slots[1] = -1                                   # padding
        slots[2], slots[3] = nb * bs, -2                # bad slots: flagged, not written
        flags = nvpa.NVPA_FLAG_BAD_SLOT
    _check(cuda_device, kb, vb, slots, nb, bs, pad, flags)


def test_store_every_bf16_pattern_and_every_row_size(cuda_device):
    """Rows made of all 65536 bit patterns (infinities, NaN and subnormals among them), and
    rows whose maximum takes every finite positive value."""
    d = 128
    every = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    rng = np.random.default_rng(0)
    a = rng.permutation(every).reshape(-1, 2, d)
    top = np.zeros((0x7F80, d), np.uint16)
    top[:, 5] = np.arange(0x7F80)
    for k in range(1, 9):                                # smaller values beside the maximum
        top[:, 5 + 9 * k] = np.maximum(np.arange(0x7F80) - 61 * k, 0) | 0x8000 * (k % 2)
    b = top.reshape(-1, 2, d)
    bits = np.concatenate([a, b])
    n = len(bits)
    bs = 256
    _check(cuda_device, bits, bits[::-1].copy(), np.arange(n), -(-n // bs), bs)


def test_store_nothing(cuda_device):
    kc, vc, ks, vs = _pools(2, 16, 2, 64, cuda_device)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=cuda_device)
    nvpa.store_kvcache_fp8(e, e, kc, vc, ks, vs, torch.empty(0, dtype=torch.int32, device=cuda_device))
    assert (kc.view(torch.uint8) == FILL).all()


@pytest.mark.parametrize("lens,hkv,d,bs", [
    ([1], 1, 64, 16), ([17, 0, 256, 300, 700], 2, 64, 256), ([33, 1, 90], 8, 128, 16), ([129, 128], 3, 128, 64),
])
def test_gather_reads_back_exactly(cuda_device, lens, hkv, d, bs):
    rng = np.random.default_rng(sum(lens))
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 2
    order = rng.permutation(nb)
    tables = np.full((len(lens), max(need)), -7, np.int64)
    at = 0
    for b, k in enumerate(need):
        tables[b, :k] = order[at:at + k]
        at += k
    x = rng.standard_normal((nb, bs, hkv, d)) * np.exp2(rng.integers(-60, 60, size=(nb, bs, hkv, 1)))
    codes, scales = quantise_rows(bf16_bits_from_f32(x.astype(np.float32)).reshape(x.shape))
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1])
    out = torch.full((total + 3, hkv, d), 7.0, dtype=torch.bfloat16, device=cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    nvpa.gather_kv_fp8(torch.from_numpy(codes).to(cuda_device).view(torch.float8_e4m3fn),
                       torch.from_numpy(np.ascontiguousarray(scales.transpose(0, 2, 1))).to(cuda_device),
                       i32(tables, cuda_device), i32(cu, cuda_device), total, out=out[:total], err_flag=err)
    assert err.item() == 0
    values = dequantise_rows(codes, scales)
    want = np.stack([values[tables[b, j // bs], j % bs] for b, n in enumerate(lens) for j in range(n)])
    assert np.array_equal(out[:total].double().cpu().numpy(), want)
    assert (out[total:] == 7.0).all()


def test_gather_bad_block_ids_are_zeroed_and_flagged(cuda_device):
    dev = cuda_device
    codes = torch.full((4, 16, 2, 64), 0x38, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)   # 1.0
    scales = torch.full((4, 2, 16), 128, dtype=torch.uint8, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = nvpa.gather_kv_fp8(codes, scales, i32([[1, 4], [-1, 2]], dev), i32([0, 20, 37], dev), 37, err_flag=err)
    assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
    o = out.float().cpu().numpy()
    assert (o[:16] == 2).all() and (o[16:36] == 0).all() and (o[36:] == 2).all()
    # rows behind the last sequence: flagged, left as they were
    err.zero_()
    out.fill_(5)
    nvpa.gather_kv_fp8(codes, scales, i32([[1], [2]], dev), i32([0, 3, 5], dev), 7, out=out[:7], err_flag=err)
    assert err.item() == nvpa.NVPA_FLAG_BAD_LENGTH
    assert (out[:5] == 2).all() and (out[5:] == 5).all()


def test_store_then_gather_round_trip_within_half_a_step(cuda_device):
    """|read back - x| <= 2^-4 |x|, or half the smallest step of the row's scale."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(3)
    k = torch.randn((300, 4, 128), generator=g, device=dev).to(torch.bfloat16)
    kc, vc, ks, vs = _pools(2, 256, 4, 128, dev)
    slots = torch.arange(300, dtype=torch.int32, device=dev)
    nvpa.store_kvcache_fp8(k, k, kc, vc, ks, vs, slots)
    back = nvpa.gather_kv_fp8(kc, ks, i32([[0, 1]], dev), i32([0, 300], dev), 300)
    step = torch.exp2(ks.double() - 127 - 10).transpose(1, 2).reshape(512, 4)[:300, :, None]
    assert ((back.double() - k.double()).abs() <= torch.maximum(2.0 ** -4 * k.double().abs(), step)).all()


def test_store_on_another_stream_and_in_a_graph(cuda_device):
    dev = cuda_device
    rng = np.random.default_rng(9)
    bits = bf16_bits_from_f32(rng.standard_normal((40, 2, 64)).astype(np.float32)).reshape(40, 2, 64)
    kc, vc, ks, vs = _pools(4, 16, 2, 64, dev)
    k, slots = bf16_tensor(np.zeros_like(bits), dev), i32(np.arange(40), dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        nvpa.store_kvcache_fp8(k, k, kc, vc, ks, vs, slots)
    k.copy_(bf16_tensor(bits, dev))
    graph.replay()
    torch.cuda.synchronize()
    codes, scales = _expect(bits, np.arange(40), 4, 16, 2, 64)
    assert np.array_equal(kc.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(ks.cpu().numpy(), scales)
    assert np.array_equal(bits_of(k), bits)


@pytest.mark.parametrize("lens,hkv,d,bs", [
    ([300, 0, 41], 160, 64, 16),          # a row of more chunks than a block takes at once
    ([5, 9], 128, 128, 16),
    ([1] * 700, 1, 64, 16),               # many short sequences
    ([20000], 1, 128, 256),
])
def test_gather_of_wide_rows_and_many_sequences(cuda_device, lens, hkv, d, bs):
    dev = cuda_device
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 1
    g = torch.Generator(device=dev).manual_seed(5)
    codes = torch.randint(0, 127, (nb, bs, hkv, d), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.randint(100, 140, (nb, hkv, bs), generator=g, device=dev, dtype=torch.uint8)
    order = torch.randperm(nb, generator=g, device=dev).int()
    tables = torch.full((len(lens), max(need)), -3, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        tables[b, :k] = order[at:at + k]
        at += k
    cu = i32(np.concatenate([[0], np.cumsum(lens)]), dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = nvpa.gather_kv_fp8(codes.view(torch.float8_e4m3fn), scales, tables, cu, sum(lens), err_flag=err)
    assert err.item() == 0
    full = codes.view(torch.float8_e4m3fn).float() * torch.exp2(scales.float() - 127).transpose(1, 2)[..., None]
    want = torch.cat([full[tables[b, :need[b]].long()].flatten(0, 1)[:n] for b, n in enumerate(lens) if n])
    assert torch.equal(out.float(), want)      # a code times a power of two is a bf16 value


def test_read_back_of_very_wide_rows(cuda_device):
    # 66536 chunks of 16 codes in a row: more than 2^16
    dev, hkv, d, bs, nb = cuda_device, 8317, 128, 16, 3
    g = torch.Generator(device=dev).manual_seed(3)
    codes = torch.randint(0, 127, (nb, bs, hkv, d), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.randint(100, 140, (nb, hkv, bs), generator=g, device=dev, dtype=torch.uint8)
    tables = i32(np.array([[2, 0]]), dev)
    out = nvpa.gather_kv_fp8(codes.view(torch.float8_e4m3fn), scales, tables, i32(np.array([0, 19]), dev), 19)
    full = codes.view(torch.float8_e4m3fn).float() * torch.exp2(scales.float() - 127).transpose(1, 2)[..., None]
    assert torch.equal(out.float(), torch.cat([full[2], full[0, :3]]))
