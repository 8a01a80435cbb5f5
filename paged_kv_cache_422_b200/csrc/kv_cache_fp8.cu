// store_kvcache_fp8: quantise new K/V rows to e4m3 codes with a power-of-two scale per
// (slot, KV head) while scattering them through slot_mapping; gather_kv_fp8 reads a
// sequence's rows back as bf16 (exactly: see fp8.cuh).
//
// Both are bound by HBM bandwidth (3 bytes per value: 2 of bf16, 1 of e4m3), so each value
// is loaded once with 16-byte loads and the row's maximum never leaves the registers: D / 16
// lanes hold one row (16 values each), log2(D / 16) shuffles give its largest magnitude.
#include <algorithm>

#include <cuda_fp16.h>

#include "fp8.cuh"
#include "nvpa_internal.h"

namespace nvpa {

namespace {

// Largest finite magnitude (bf16 bits) among the 16 values of a lane; `odd` is set when some
// value is not finite.
__device__ __forceinline__ uint32_t lane_amax(const uint32_t (&w)[8], bool& odd) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    odd = m >= 0x7f80u;
    if (odd) {   // rare: leave infinities and NaN out
        m = 0;
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
            if (a < 0x7f80u) m = max(m, a);
            if (b < 0x7f80u) m = max(m, b);
        }
    }
    return m;
}

// The 16 values of a lane as e4m3 codes, multiplied by inv = 2^-e (exact) first.
__device__ __forceinline__ uint4 lane_codes(const uint32_t (&w)[8], float inv, bool odd) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = pack_e4m3x2(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
    if (odd) {   // an infinity has no code: it is stored as NaN, like a NaN
        for (int i = 0; i < 8; ++i) {
            if ((w[i] & 0x7fffu) >= 0x7f80u) h[i] = (h[i] & 0xff00u) | kE4m3Nan;
            if (((w[i] >> 16) & 0x7fffu) >= 0x7f80u) h[i] = (h[i] & 0x00ffu) | (kE4m3Nan << 8);
        }
    }
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

struct StoreFp8Params {
    const uint16_t* k;
    const uint16_t* v;
    long long k_stride, v_stride;
    uint8_t* k_cache;
    uint8_t* v_cache;
    uint8_t* k_scales;
    uint8_t* v_scales;
    const int32_t* slots;
    int num_tokens, hkv, block_size;
    long long capacity;
    int32_t* err;
};

// LPR = D / 16 lanes per (token, KV head) row pair; consecutive lane groups take
// consecutive heads, so that a warp reads and writes contiguous memory.
template <int D>
__global__ void __launch_bounds__(256) store_fp8_kernel(const StoreFp8Params p) {
    constexpr int LPR = D / 16;
    const int sub = threadIdx.x % LPR;
    const long long rows = (long long)p.num_tokens * p.hkv;
    const long long step = (long long)gridDim.x * (256 / LPR);
    // the loop bound is that of the warp's first row: every lane takes part in the shuffles
    const long long first = (long long)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const long long warp_first = first - (threadIdx.x % 32) / LPR;
    for (long long d = 0; warp_first + d < rows; d += step) {
        const long long row = first + d;
        int slot = -1, h = 0;
        long long t = 0;
        if (row < rows) {
            t = row / p.hkv;
            h = (int)(row - t * p.hkv);
            slot = __ldg(p.slots + t);
            if (slot != -1 && (slot < 0 || (long long)slot >= p.capacity)) {
                if (sub == 0 && h == 0) flag_error(p.err, NVPA_FLAG_BAD_SLOT);
                slot = -1;
            }
        }
        uint32_t kw[8] = {}, vw[8] = {};
        if (slot >= 0) {
            const uint4* ks = reinterpret_cast<const uint4*>(p.k + t * p.k_stride + (long long)h * D + sub * 16);
            const uint4* vs = reinterpret_cast<const uint4*>(p.v + t * p.v_stride + (long long)h * D + sub * 16);
            const uint4 a = __ldcs(ks), b = __ldcs(ks + 1), c = __ldcs(vs), e = __ldcs(vs + 1);
            kw[0] = a.x; kw[1] = a.y; kw[2] = a.z; kw[3] = a.w; kw[4] = b.x; kw[5] = b.y; kw[6] = b.z; kw[7] = b.w;
            vw[0] = c.x; vw[1] = c.y; vw[2] = c.z; vw[3] = c.w; vw[4] = e.x; vw[5] = e.y; vw[6] = e.z; vw[7] = e.w;
        }
        bool kodd, vodd;
        // both maxima in one word: K's in the high half
        uint32_t km = lane_amax(kw, kodd), vm = lane_amax(vw, vodd);
        uint32_t m = km << 16 | vm;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (slot < 0) continue;
        const int kb = scale_byte(m >> 16), vb = scale_byte(m & 0xffffu);
        const size_t at = ((size_t)slot * p.hkv + h) * D + sub * 16;
        *reinterpret_cast<uint4*>(p.k_cache + at) = lane_codes(kw, scale_value(254 - kb), kodd);
        *reinterpret_cast<uint4*>(p.v_cache + at) = lane_codes(vw, scale_value(254 - vb), vodd);
        if (sub == 0) {
            const int blk = slot / p.block_size;
            const size_t sat = ((size_t)blk * p.hkv + h) * p.block_size + (slot - blk * p.block_size);
            p.k_scales[sat] = (uint8_t)kb;
            p.v_scales[sat] = (uint8_t)vb;
        }
    }
}

// One warp per destination row; 16 codes (32 bytes of bf16) per lane and step.
template <int D>
__global__ void __launch_bounds__(256) gather_fp8_kernel(
    uint16_t* __restrict__ dst, const uint8_t* __restrict__ cache, const uint8_t* __restrict__ scales,
    const int32_t* __restrict__ block_tables, int max_blocks, const int32_t* __restrict__ cu, int batch,
    int total_k, int hkv, int num_blocks, int block_size, int block_shift, int32_t* err) {
    constexpr int CPH = D / 16;   // chunks per head
    const int lane = threadIdx.x & 31;
    for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < total_k;
         row += (long long)gridDim.x * 8) {
        int lo = 0, hi = batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(cu + mid) <= row) lo = mid; else hi = mid - 1;
        }
        const int k0 = __ldg(cu + lo), k1 = __ldg(cu + lo + 1);
        const int pos = (int)(row - k0);
        uint16_t* d = dst + (size_t)row * hkv * D;
        if (row < k0 || row >= k1 || (long long)pos >= (long long)max_blocks * block_size) {
            if (lane == 0) flag_error(err, NVPA_FLAG_BAD_LENGTH);
            continue;
        }
        const int blk = checked_block(block_tables + (size_t)lo * max_blocks, pos, block_shift, num_blocks,
                                      lane == 0 ? err : nullptr);
        const int r = pos & (block_size - 1);
        const uint8_t* s = cache + ((size_t)max(blk, 0) * block_size + r) * hkv * D;
        const uint8_t* sc = scales + (size_t)max(blk, 0) * hkv * block_size + r;
        for (int c = lane; c < hkv * CPH; c += 32) {
            uint32_t w[8] = {};
            if (blk >= 0) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(s) + c);
                const float f = scale_value(__ldg(sc + (size_t)(c / CPH) * block_size));
                const uint32_t in[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a, b;
                    e4m3x4_to_half2(in[i], a, b);
                    const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a));
                    const float2 y = __half22float2(*reinterpret_cast<__half2*>(&b));
                    w[2 * i] = pack_bf16x2(x.x * f, x.y * f);
                    w[2 * i + 1] = pack_bf16x2(y.x * f, y.y * f);
                }
            }
            uint4* o = reinterpret_cast<uint4*>(d) + 2 * c;
            o[0] = make_uint4(w[0], w[1], w[2], w[3]);
            o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

}  // namespace

nvpa_status_t run_store_kvcache_fp8(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                                    void* k_cache, void* v_cache, uint8_t* k_scales, uint8_t* v_scales,
                                    const int32_t* slot_mapping, int num_tokens, int hkv, int head_dim,
                                    int num_blocks, int block_size, int32_t* err_flag, cudaStream_t stream) {
    if (num_tokens == 0) return NVPA_OK;
    StoreFp8Params p{};
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.k_cache = static_cast<uint8_t*>(k_cache);
    p.v_cache = static_cast<uint8_t*>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.slots = slot_mapping;
    p.num_tokens = num_tokens;
    p.hkv = hkv;
    p.block_size = block_size;
    p.capacity = (long long)num_blocks * block_size;
    p.err = err_flag;
    const long long per = 256 / (head_dim / 16);
    const long long need = ((long long)num_tokens * hkv + per - 1) / per;
    const int grid = (int)std::max(1LL, std::min<long long>(need, (long long)device_sm_count() * 8));
    if (head_dim == 128) store_fp8_kernel<128><<<grid, 256, 0, stream>>>(p);
    else store_fp8_kernel<64><<<grid, 256, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failure(e, "store_kvcache_fp8 launch");
    count_launches(1);
    return NVPA_OK;
}

nvpa_status_t run_gather_kv_fp8(void* dst, const void* cache, const uint8_t* scales,
                                const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* cu_seqlens_k, int batch, int total_k, int hkv, int head_dim,
                                int num_blocks, int block_size, int32_t* err_flag, cudaStream_t stream) {
    if (total_k == 0 || batch == 0) return NVPA_OK;
    const int grid = (int)std::min<long long>(((long long)total_k + 7) / 8, (long long)device_sm_count() * 16);
    const int shift = __builtin_ctz((unsigned)block_size);
    auto* d = static_cast<uint16_t*>(dst);
    auto* c = static_cast<const uint8_t*>(cache);
    if (head_dim == 128)
        gather_fp8_kernel<128><<<grid, 256, 0, stream>>>(d, c, scales, block_tables, max_blocks_per_seq, cu_seqlens_k,
                                                         batch, total_k, hkv, num_blocks, block_size, shift, err_flag);
    else
        gather_fp8_kernel<64><<<grid, 256, 0, stream>>>(d, c, scales, block_tables, max_blocks_per_seq, cu_seqlens_k,
                                                        batch, total_k, hkv, num_blocks, block_size, shift, err_flag);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failure(e, "gather_kv_fp8 launch");
    count_launches(1);
    return NVPA_OK;
}

}  // namespace nvpa
