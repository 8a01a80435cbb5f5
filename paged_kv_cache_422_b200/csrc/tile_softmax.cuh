// The softmax of one 128-row tensor-core tile, one thread per query row: masking, row
// maximum, exponentials and the P store, shared by the prefill, shared-prefix and chunk
// attention kernels; and the host side's tensor maps.
#pragma once

#include <cuda.h>
#include <mutex>

#include "attn_warp.cuh"
#include "sm100.cuh"

namespace nvpa {

using namespace sm100;

// Bit k set for the first n of 32 columns (n clamped to [0, 32]).
__device__ __forceinline__ uint32_t visible_mask(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : ((1u << n) - 1u);
}

// bits as a float when bit k of vm is set, else `fill` (shift/and/or, no predicate).
__device__ __forceinline__ float keep_or(uint32_t bits, uint32_t vm, int k, float fill) {
    const uint32_t keep = (uint32_t)((int32_t)(vm << (31 - k)) >> 31);
    return __uint_as_float((bits & keep) | (__float_as_uint(fill) & ~keep));
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The softmax of one S row (one thread per row, the whole 128-column row in registers) is a
// single code path for every tile and either sign of the scale, kept small on purpose: the
// warps that issue the MMAs and the copies share each SM sub-partition's instruction
// cache with two softmax warps, and the fully unrolled row loops are most of the kernel's
// code.

// Columns at or past lim - key0 (keys the row does not see, including rows past the
// sequence) become -inf by bit mask, whatever they held.
template <int N>
__device__ __forceinline__ void mask_row(uint32_t (&sv)[N], int key0, int lim) {
#pragma unroll
    for (int c = 0; c < N / 32; ++c) {
        const uint32_t vm = visible_mask(lim - key0 - c * 32);
#pragma unroll
        for (int k = 0; k < 32; ++k) sv[c * 32 + k] = __float_as_uint(keep_or(sv[c * 32 + k], vm, k, -INFINITY));
    }
}

// Largest value of the row: two independent accumulators, two new values per three-input
// instruction.
template <int N>
__device__ __forceinline__ float row_max(const uint32_t (&sv)[N]) {
    float e0 = -INFINITY, e1 = -INFINITY;
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        e0 = max3(e0, __uint_as_float(sv[k]), __uint_as_float(sv[k + 1]));
        e1 = max3(e1, __uint_as_float(sv[k + 2]), __uint_as_float(sv[k + 3]));
    }
    return fmaxf(e0, e1);
}

// P = exp2(s * c + nm) of N raw scores of a row (c > 0: the scale in log2 units; one
// packed FMA per pair of scores), packed to bf16 pairs and written to TMEM from column
// p_col on (32 S columns become 16 P columns); returns the sum of the fp32 values.  A -inf
// score or offset gives 0.
template <int N>
__device__ __forceinline__ float exp_row(const uint32_t (&sv)[N], uint32_t p_col, float c, float nm) {
    const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(nm, nm);
    uint64_t l0 = f2_pack(0.f, 0.f), l1 = l0;
#pragma unroll
    for (int cc = 0; cc < N / 32; ++cc) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[cc * 32 + k]), __uint_as_float(sv[cc * 32 + k + 1])), c2, nm2),
                      a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            const uint64_t p2 = f2_pack(a, b);
            if ((k / 2) & 1)
                l1 = f2_add(l1, p2);
            else
                l0 = f2_add(l0, p2);
            pk[k / 2] = pack_bf16x2(a, b);
        }
        tmem_st16(p_col + cc * 16, pk);
    }
    float a0, b0, a1, b1;
    f2_unpack(l0, a0, b0);
    f2_unpack(l1, a1, b1);
    return (a0 + b0) + (a1 + b1);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// 3-D view (dim, heads, rows) of a [rows, heads, dim] bf16 array; box = 64 x box_heads x
// box_rows, 128-byte swizzle.
inline bool make_map(CUtensorMap* map, const void* base, int dim, int heads, long long rows, int box_heads,
                     int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t gdim[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t gstride[2] = {(cuuint64_t)dim * 2, (cuuint64_t)dim * heads * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    const cuuint32_t estride[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace nvpa
