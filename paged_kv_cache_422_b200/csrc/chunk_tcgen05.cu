// Attention of long chunks of new tokens over a bf16 or e4m3 paged cache on the
// 5th-generation tensor cores (tcgen05 + TMEM), with an optional sliding window and first
// tokens that stay visible.  (Chunks of a few rows per KV head go to row_attention.cu.)
//
// Mathematics.  As in row_attention.cu: query at position p sees key j iff j <= p and (no
// window, or j > p - window, or j < sinks); per query row s_j = scale <q, k_j>, out =
// sum_j softmax(s)_j v_j, lse = log sum_j exp(s_j), in one pass over the keys with a running
// maximum and sum per row (float32).  4 D flops per (query row, visible key); with hundreds
// of rows per key the products bound it, so both run as tcgen05 MMAs with bf16 operands and
// float32 accumulators in TMEM.  Weights are rounded to bf16 (2^-9 of each weight) for the
// second product; scores, sums and outputs stay float32 up to the final bf16 store.
//
// The e4m3 cache is widened on chip: code * 2^e is exact in bf16 (fp8.cuh), so everything
// behind the widening is the bf16 kernel.  Feeding the codes to the MMAs themselves would
// need 8-bit queries and weights.
//
// Tiles.  A query tile is 128 MMA rows: floor(128 / G) tokens times the G query heads of one
// KV head.  A work unit is a pair of adjacent query tiles A, B of one sequence and KV head
// and a range of 128-key tiles: both read the same K/V tiles, so each is fetched (and
// widened) once for up to 256 rows, and one tile's MMAs run while the other's softmax does.
// When the call has fewer units than SMs, the key ranges are cut into partitions whose
// results are merged by the decode combine.
//
// Keys.  The keys that a unit sees are one virtual range: the sinks (rounded up to 16), then
// the window from its first row's first key (rounded down to 16) on; virtual key v is key v
// or, past the sinks, v + skip.  128-key tiles are cut from that range, so a few sinks cost a
// few rows of one tile instead of a tile of their own.  With a window, tiles are copied in
// pieces of 16 rows (a tile may start anywhere); without, in pieces of min(block, 128) rows.
// Rows that nobody in the unit sees are masked by -inf scores and zeroed values (never by
// arithmetic that would keep a NaN), and so are those of blocks whose ids are out of range; blocks
// without a visible key are not looked up.
//
// Warp roles (one persistent CTA per SM, units claimed longest first):
//   warps 0 2 3  copy Q and K/V tiles by TMA (e4m3: codes and scales into a staging ring);
//   warp 1       issues the MMAs: S_A0 S_B0 | O_A += P_A0 V_0, S_A1, O_B += P_B0 V_0, ...;
//   warps 4..11  softmax of tiles A and B, one thread per row;
//   warps 12..15 (e4m3 only) widen staged codes into the K/V ring, one thread per key row.
// TMEM: tile A S/P [0, 128), O [128, 256); tile B S/P [256, 384), O [384, 512).
//
// Chunks of one query tile (a few dozen rows over a long context) have no tile B, so their
// units split: A and B are two key ranges of the same query tile, each with its own stream of
// K/V tiles, and their results are two partitions for the merge.
//
// Measured (32 / 8 heads of 128, 512-token chunks over 4 to 8 k keys): bf16 cache 414 us, 980
// TFLOP/s (0.60 of the measured bf16 burst), e4m3 cache 500 us, 810 TFLOP/s.  A pair advances one
// key tile in about 3900 cycles (e4m3 4600), against 2048 of tensor work: the softmax of two
// tiles, back to back on each sub-partition, sets the pace, as in the prefill kernel; the
// widening takes 900 of the warp instructions that share its issue slots.  A unit's fill and
// drain take 5 us (e4m3 8).
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>

#include <cuda_fp16.h>

#include "decode_params.cuh"
#include "fp8.cuh"
#include "nvpa_internal.h"
#include "tile_softmax.cuh"

namespace nvpa {

namespace {

constexpr int kRows = 128;        // query rows per tile (MMA M)
constexpr int kKeys = 128;        // keys per tile
constexpr int kProducers = 3;     // warps that may issue copies: 0, 2 and 3
constexpr int kUnits = 4;         // claimed units handed from the producer to the others
constexpr int kBuckets = 4096;    // plan: key-tile counts sorted exactly
constexpr int kGran = 16;         // granularity of the virtual key range
constexpr int kKeeps = 8;         // K tiles whose masks of present keys are held: the copies run at most 4
                                  // ahead of the softmax (half of the slots of the rings)

// Registers per thread after setmaxnreg: the shares of the warpgroups add up to the launch's.
template <bool FP8>
struct Roles {
    static constexpr int WARPS = FP8 ? 16 : 12;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int LAUNCH_REGS = FP8 ? 128 : 168;
    static constexpr int SMALL_REGS = FP8 ? 80 : 104;      // warps 0..3 and 12..15
    static constexpr int SOFTMAX_REGS = FP8 ? 176 : 200;   // warps 4..11
    static constexpr int READERS = 1 + 8 + (FP8 ? 4 : 0);  // of the unit ring, and producers but the first
    // shared memory at head_dim 128: Q tiles and K/V tiles (bf16, ready for the MMAs) of 32 KB,
    // staged e4m3 tiles of 16 KB.  A tile takes 2 us from its copy's issue to its arrival, so
    // the e4m3 cache's copies run four tiles ahead of the widening.
    static constexpr int QBUFS = FP8 ? 2 : 3;
    static constexpr int RING = FP8 ? 3 : 4;
    static constexpr int STAGES = FP8 ? 4 : 1;
    static_assert((WARPS - 8) * SMALL_REGS + 8 * SOFTMAX_REGS == WARPS * LAUNCH_REGS, "register split");
    static_assert(((WARPS - 8) / 4 * SMALL_REGS + 2 * SOFTMAX_REGS) * 32 <= 16384, "sub-partition registers");
};

struct ChunkParams {
    const int32_t* block_tables;
    const int32_t* cu_q;
    const int32_t* context_lens;
    const uint8_t* k_scales;     // [num_blocks, hkv, block_size] (e4m3 cache)
    const uint8_t* v_scales;
    uint16_t* out;
    float* lse_out;
    float* o_part;               // [total_q * hq, s_max, D] partial outputs, normalised
    float* lse_part;
    int4* entries;               // plan: (sequence, pair, unit of the pair's keys, -)
    int32_t* counter;            // [0] units claimed, [1] entries
    int32_t* nsplit;             // [total_q] partitions of each query token, 0: none
    int32_t* err;
    int batch, total_q, max_q, max_ctx, hq, hkv, group;
    int tq;                      // tokens per query tile
    int row_pairs;               // pairs of the longest chunk
    int max_blocks, num_blocks, block_size, block_shift;
    int piece;                   // rows per K/V copy
    int window, sinks;           // window 0: none
    int chunk;                   // key tiles per partition
    int split;                   // chunks of one query tile: tiles A and B are two partitions of it
    int b_step;                  // tokens between tiles A and B: tq, split: 0
    int unit_tiles;              // key tiles per unit: chunk, split: 2 chunk
    int s_max, max_entries;
    float scale_log2;            // > 0
    int negate_qk;               // scale < 0: S = -Q K^T
    int out_v8;                  // out is 32-byte aligned
};

// The virtual keys of a pair of query tiles (see the top): key v is v below `head`, v + skip
// from there on.
struct Keys {
    int p_first, p_last;   // positions of the pair's first and last query token
    int head, skip;
    __device__ __forceinline__ int real(int v) const { return v < head ? v : v + skip; }
    // virtual keys up to position pos
    __device__ __forceinline__ int upto(int pos) const { return pos + 1 - skip; }
    __device__ __forceinline__ int tiles(int pos) const { return (pos - skip) / kKeys + 1; }
};
__device__ __forceinline__ Keys pair_keys(const ChunkParams& p, int lq, int ctx, int pair) {
    Keys k;
    k.p_first = ctx - lq + 2 * pair * p.tq;
    k.p_last = ctx - lq + min(lq, (2 * pair + 2) * p.tq) - 1;
    k.head = k.skip = 0;
    if (p.window > 0) {
        const int lo = max(0, k.p_first - p.window + 1) / kGran * kGran;
        k.head = (int)min((long long)lo, ((long long)p.sinks + kGran - 1) / kGran * kGran);
        k.skip = lo - k.head;
    }
    return k;
}
// Key tiles that tile x of the pair sees (0: no such tile).
__device__ __forceinline__ int tile_count(const ChunkParams& p, const Keys& k, int ntok, int x) {
    return ntok > 0 ? k.tiles(k.p_first + x * p.tq + ntok - 1) : 0;
}
__device__ __forceinline__ int tile_tokens(const ChunkParams& p, int lq, int pair, int x) {
    return min(p.tq, lq - (2 * pair + x) * p.tq);
}

// The order in which a unit's K/V tiles pass through the rings, walked by every role: K_0 of
// each stream, then for each key tile j and stream x: V_xj, K_x(j+1).
struct TileWalk {
    int x = 0, kv = 0, j = 0;
    __device__ __forceinline__ void next(int sn0, int sn1) {
        if (kv == 1 && j + 1 < (x ? sn1 : sn0)) {   // V_xj -> K_x(j+1)
            kv = 0;
            ++j;
            return;
        }
        if (kv == 0 && j == 0) {                    // the K_0s -> V_00
            if (x == 0 && sn1 > 0) x = 1;
            else x = 0, kv = 1;
            return;
        }
        const int round = kv ? j : j - 1;           // stream x is done with it
        kv = 1;
        if (x == 0 && round < sn1) {
            x = 1;
            j = round;
        } else {
            x = 0;
            j = round + 1;
        }
    }
};

// A work unit: a pair of query tiles A, B of a sequence, one KV head and one partition of the
// keys, worked out by the first producer warp for all the others.  seq < 0 ends the loop.
struct __align__(16) ChunkUnit {
    int seq, hk, row0, part;   // row0: the first query row; part: partition of A (B: + split)
    int nk[2];                 // key tiles of their partition that A and B see
    int ntok[2];               // their tokens
    int ns[2];                 // their partitions
    int sn[2];                 // K/V tiles that the unit reads: one stream of the longer tile's
                               // key tiles; split: a stream for A and one for B
    Keys keys;
    __device__ __forceinline__ int first_key(const ChunkParams& p, int x) const {   // virtual, of stream x
        return (part * p.chunk + (x && p.split ? p.chunk : 0)) * kKeys;
    }
};
static_assert(sizeof(ChunkUnit) == 64, "unit size");

template <int D, bool FP8>
struct ChunkLayout {
    using R = Roles<FP8>;
    static constexpr int REGIONS = D / 64;                  // 64 bf16 = one 128-byte swizzle row
    static constexpr int REGION_BYTES = 128 * 128;
    static constexpr int TILE_BYTES = REGIONS * REGION_BYTES;
    static constexpr int Q_OFF = 0;
    static constexpr int RING_OFF = R::QBUFS * TILE_BYTES;
    static constexpr int STAGE_OFF = RING_OFF + R::RING * TILE_BYTES;      // codes [128 rows][D]
    static constexpr int STAGE_BYTES = FP8 ? kKeys * D : 0;
    static constexpr int SCALE_OFF = STAGE_OFF + R::STAGES * STAGE_BYTES;   // 128 scale bytes each
    static constexpr int BAR_OFF = SCALE_OFF + (FP8 ? R::STAGES * kKeys : 0);
    // barriers (per query tile in pairs: + 0 for A, + 1 for B)
    static constexpr int B_QFULL = 0, B_QEMPTY = R::QBUFS, B_KVFULL = 2 * R::QBUFS, B_KVEMPTY = B_KVFULL + R::RING;
    static constexpr int B_SFULL = B_KVEMPTY + R::RING, B_PFULL = B_SFULL + 2, B_ODONE = B_PFULL + 2;
    static constexpr int B_OFINAL = B_ODONE + 2, B_OFREE = B_OFINAL + 2, B_DRAIN = B_OFREE + 2;
    static constexpr int B_UFULL = B_DRAIN + 1, B_UEMPTY = B_UFULL + kUnits;
    static constexpr int B_STFULL = B_UEMPTY + kUnits, B_STEMPTY = B_STFULL + R::STAGES;
    static constexpr int NBARS = B_STEMPTY + R::STAGES;
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;     // tmem base, abort flag, bad block seen, staged piece masks
    static constexpr int UNIT_OFF = (MISC_OFF + 12 + 4 * kProducers * R::STAGES + 15) / 16 * 16;
    static constexpr int KEEP_OFF = UNIT_OFF + (int)sizeof(ChunkUnit) * kUnits;
    static constexpr int BYTES = KEEP_OFF + kKeeps * (kKeys / 8);
    static constexpr int ALLOC = BYTES + 1024;               // room to align the base to 1024
};
static_assert(ChunkLayout<128, false>::ALLOC <= 227 * 1024 && ChunkLayout<128, true>::ALLOC <= 227 * 1024,
              "shared memory per CTA");

// ------------------------------------------------------------------------------------
// plan: the units, those with the most key tiles first
// ------------------------------------------------------------------------------------
// A counting sort over the units' key-tile counts; the order inside one count is whatever the
// atomics give, which decides only which CTA runs a unit, never a result.
__global__ void __launch_bounds__(1024) chunk_plan_kernel(const ChunkParams p) {
    __shared__ int s_hist[kBuckets];
    __shared__ int warp_tot[32];
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int lim = (int)min((long long)p.max_ctx, (long long)p.max_blocks * p.block_size);
    for (int b = tid; b < kBuckets; b += blockDim.x) s_hist[b] = 0;
    if (p.s_max > 1)
        for (int i = tid; i < p.total_q; i += blockDim.x) p.nsplit[i] = 0;
    __syncthreads();
    // pair i of the call: (sequence, pair); tiles = 0 when there is none
    struct Pair {
        int b, w, q0, lq, ctx, tiles;
    };
    auto pair = [&](int i, bool flag) {
        Pair r;
        r.b = i / p.row_pairs;
        r.w = i - r.b * p.row_pairs;
        r.q0 = __ldg(p.cu_q + r.b);
        const int q1 = __ldg(p.cu_q + r.b + 1);
        r.lq = q1 - r.q0;
        r.ctx = __ldg(p.context_lens + r.b);
        // (a negative start with a huge end overflows: the order of the tests keeps it out)
        const bool ok = r.q0 >= 0 && q1 >= r.q0 && q1 <= p.total_q && r.lq <= p.max_q && r.ctx >= r.lq &&
                        r.ctx <= lim;
        if (!ok && flag && r.w == 0) flag_error(p.err, NVPA_FLAG_BAD_LENGTH);
        r.tiles = 0;
        if (ok && 2 * r.w * p.tq < r.lq) {
            const Keys k = pair_keys(p, r.lq, r.ctx, r.w);
            r.tiles = k.tiles(k.p_last);
        }
        return r;
    };
    // descending order: bucket of a unit with n key tiles
    auto bucket = [](int n) { return kBuckets - 1 - min(n, kBuckets - 1); };
    const int n = p.batch * p.row_pairs;
    for (int i = tid; i < n; i += blockDim.x) {
        const Pair r = pair(i, true);
        if (r.tiles == 0) continue;
        const int full = r.tiles / p.unit_tiles, rest = r.tiles - full * p.unit_tiles;
        if (full > 0) atomicAdd(&s_hist[bucket(p.unit_tiles)], full);
        if (rest > 0) atomicAdd(&s_hist[bucket(rest)], 1);
    }
    __syncthreads();
    constexpr int kPer = kBuckets / 1024;
    int v[kPer], sum = 0, total = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        v[k] = s_hist[kPer * tid + k];
        sum += v[k];
    }
    int at = block_exclusive_scan(sum, warp_tot, total);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        s_hist[kPer * tid + k] = at;
        at += v[k];
    }
    __syncthreads();
    for (int i = tid; i < n; i += blockDim.x) {
        const Pair r = pair(i, false);
        if (r.tiles == 0) continue;
        const int full = r.tiles / p.unit_tiles, rest = r.tiles - full * p.unit_tiles;
        // (cumulative lengths that run backwards can claim rows twice, and so more entries
        // than the table holds: what does not fit is dropped and flagged below)
        auto put = [&](int pos, int s) {
            if (pos < p.max_entries) p.entries[pos] = make_int4(r.b, r.w, s, 0);
        };
        if (full > 0) {
            const int pos = atomicAdd(&s_hist[bucket(p.unit_tiles)], full);
            for (int s = 0; s < full; ++s) put(pos + s, s);
        }
        if (rest > 0) put(atomicAdd(&s_hist[bucket(rest)], 1), full);
        if (p.s_max > 1) {
            const Keys k = pair_keys(p, r.lq, r.ctx, r.w);
            for (int x = 0; x < 2; ++x) {
                const int ntok = tile_tokens(p, r.lq, r.w, x);
                const int parts = (tile_count(p, k, ntok, x) + p.chunk - 1) / p.chunk;
                for (int j = 0; j < ntok; ++j) p.nsplit[r.q0 + (2 * r.w + x) * p.tq + j] = parts;
            }
        }
    }
    if (tid == 0) {
        if (total > p.max_entries) flag_error(p.err, NVPA_FLAG_BAD_LENGTH);
        p.counter[0] = 0;
        p.counter[1] = min(total, p.max_entries);
    }
}

// ------------------------------------------------------------------------------------
// the attention kernel
// ------------------------------------------------------------------------------------

// Columns of S (virtual keys base ..) that a row does not see become -inf; it sees virtual
// keys [0, a) and [b, c) but those without a bit in `keep`.
__device__ __forceinline__ void mask_columns(uint32_t (&sv)[kKeys], int base, int a, int b, int c,
                                             const volatile uint32_t* keep) {
#pragma unroll
    for (int i = 0; i < kKeys / 32; ++i) {
        const int at = base + 32 * i;
        const uint32_t vm = (visible_mask(a - at) | ~visible_mask(b - at)) & visible_mask(c - at) & keep[i];
#pragma unroll
        for (int k = 0; k < 32; ++k)
            sv[i * 32 + k] = __float_as_uint(keep_or(sv[i * 32 + k], vm, k, -INFINITY));
    }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Roles<FP8>::THREADS, 1)
chunk_tcgen05_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const ChunkParams p) {
    using L = ChunkLayout<D, FP8>;
    using R = Roles<FP8>;
    constexpr int QBUFS = R::QBUFS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(smem);

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
    volatile int* bad_seen = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 8);   // a block id out of range so far
    uint32_t* stage_mask = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF + 12);   // [stage][producer] its pieces present
    ChunkUnit* unit_ring = reinterpret_cast<ChunkUnit*>(smem + L::UNIT_OFF);
    // [K tile, modulo kKeeps] a bit per key: 0 where its block id is out of range
    volatile uint32_t* keeps = reinterpret_cast<volatile uint32_t*>(smem + L::KEEP_OFF);
    constexpr int KEEP = kKeys / 32;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int producers = min(kProducers, kKeys / p.piece);   // at most one per piece of a tile

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(bars + L::B_SFULL + x, 1);
            mbar_init(bars + L::B_PFULL + x, 4);
            mbar_init(bars + L::B_ODONE + x, 1);
            mbar_init(bars + L::B_OFINAL + x, 1);
            mbar_init(bars + L::B_OFREE + x, 4);
        }
        for (int q = 0; q < QBUFS; ++q) {
            mbar_init(bars + L::B_QFULL + q, 1);
            mbar_init(bars + L::B_QEMPTY + q, 1);
        }
        for (int s = 0; s < R::RING; ++s) {
            mbar_init(bars + L::B_KVFULL + s, FP8 ? 4 : producers);
            mbar_init(bars + L::B_KVEMPTY + s, 1);
        }
        for (int s = 0; s < R::STAGES; ++s) {
            mbar_init(bars + L::B_STFULL + s, producers);
            mbar_init(bars + L::B_STEMPTY + s, 4);
        }
        mbar_init(bars + L::B_DRAIN, 1);
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(bars + L::B_UFULL + i, 1);
            mbar_init(bars + L::B_UEMPTY + i, R::READERS + producers - 1);
        }
        *abort_flag = 0;
        *bad_seen = 0;
        fence_mbar_init();
        tma_prefetch_desc(&q_map);
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    if (threadIdx.x < kKeeps * KEEP) keeps[threadIdx.x] = 0xffffffffu;
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (broadcast, so that the compiler keeps what is derived from it warp-uniform)
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_wait();   // nothing the plan writes is read before this

    const int total = __ldcg(p.counter + 1) * p.hkv;
    // The n-th unit of this CTA, for a reader; seq is -1 at the end, -2 if a wait timed out.
    auto claim = [&](int n) -> ChunkUnit {
        const int slot = n % kUnits;
        ChunkUnit u;
        if (!mbar_wait(bars + L::B_UFULL + slot, (n / kUnits) & 1, abort_flag, p.err)) {
            u = ChunkUnit{};
            u.seq = -2;
            return u;
        }
        u = unit_ring[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::B_UEMPTY + slot);
        return u;
    };

    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::SMALL_REGS));
      if (warp == 0 || (warp >= 2 && warp - 1 < producers)) {
        // ============================ producers ============================
        // Up to three warps copy every tile together, a share of its pieces each: with 16-row pieces
        // one issuing thread needs 200 cycles per piece and 64 columns, 6600 for the 32 of a K
        // and V tile, where the MMAs and softmaxes of a pair need half of that.
        const int pw = warp == 0 ? 0 : warp - 1;
        const int pc = pw + producers * lane;      // this lane's piece of every tile
        uint32_t fill = 0, qfill = 0;
        uint32_t kfill = 0;                        // K tiles so far
        bool was_bad = false;                      // this lane has met a block id out of range
        const int piece = p.piece;
        const bool has_piece = pc * piece < kKeys;
        // Warp 0 claims units, one ahead of the one whose copies are issued.
        auto claim_next = [&]() -> int { return lane == 0 ? atomicAdd(p.counter, 1) : 0; };
        auto describe = [&](int pending) -> ChunkUnit {
            const int i = __shfl_sync(0xffffffffu, pending, 0);
            ChunkUnit u{};
            u.seq = -1;
            if (i < total) {
                const int4 e = __ldcg(p.entries + i / p.hkv);
                const int q0 = __ldg(p.cu_q + e.x), lq = __ldg(p.cu_q + e.x + 1) - q0;
                u.seq = e.x;
                u.hk = i % p.hkv;
                u.row0 = q0 + 2 * e.y * p.tq;
                u.part = p.split ? 2 * e.z : e.z;
                u.keys = pair_keys(p, lq, __ldg(p.context_lens + e.x), e.y);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    u.ntok[x] = tile_tokens(p, lq, e.y, p.split ? 0 : x);
                    const int n = tile_count(p, u.keys, u.ntok[x], p.split ? 0 : x);
                    u.nk[x] = max(0, min(p.chunk, n - u.first_key(p, x) / kKeys));
                    u.ns[x] = (n + p.chunk - 1) / p.chunk;
                }
                u.sn[0] = p.split ? u.nk[0] : max(u.nk[0], u.nk[1]);
                u.sn[1] = p.split ? u.nk[1] : 0;
            }
            return u;
        };
        ChunkUnit cur, nxt;
        int pending = total;
        if (warp == 0) {
            nxt = describe(claim_next());
            pending = nxt.seq >= 0 ? claim_next() : total;
        }
        bool ok = true;
        for (int n = 0; ok; ++n) {
            if (warp == 0) {
                cur = nxt;
                const int uslot = n % kUnits;
                if (!mbar_wait(bars + L::B_UEMPTY + uslot, ((n / kUnits) & 1) ^ 1, abort_flag, p.err)) break;
                if (lane == 0) {
                    unit_ring[uslot] = cur;
                    mbar_arrive(bars + L::B_UFULL + uslot);
                }
            } else {
                cur = claim(n);
            }
            if (cur.seq < 0) break;
            const Keys keys = cur.keys;
            const int sn0 = cur.sn[0], sn1 = cur.sn[1];
            const int va0 = cur.first_key(p, 0) + pc * piece, vb0 = cur.first_key(p, 1) + pc * piece;
            const int vend = keys.upto(keys.p_last);        // virtual keys of the unit's rows
            const int32_t* bt = p.block_tables + (size_t)cur.seq * p.max_blocks;
            // The first key of this lane's piece of key tile j of stream x, whether there is one (pieces
            // past the last visible key are not looked up), and its block id (range-checked where it is
            // used).
            auto piece_key = [&](int x, int j) { return (x ? vb0 : va0) + j * kKeys; };
            auto is_piece = [&](int v) { return has_piece && v < vend; };
            auto load_piece = [&](int x, int j) {
                const int v = piece_key(x, j);
                return j < (x ? sn1 : sn0) && is_piece(v) ? __ldg(bt + (keys.real(v) >> p.block_shift)) : -1;
            };
            // of each stream's current key tile and the next
            int blk_a = load_piece(0, 0), next_a = load_piece(0, 1);
            int blk_b = load_piece(1, 0), next_b = load_piece(1, 1);
            if (warp == 0) {
                nxt = describe(pending);
                pending = nxt.seq >= 0 ? claim_next() : total;
            }
            auto load_q = [&](int x) -> bool {
                if ((x ? p.split || cur.nk[1] == 0 : cur.nk[0] == 0) || warp != 0) return true;
                const uint32_t qs = qfill % QBUFS;
                if (!mbar_wait(bars + L::B_QEMPTY + qs, ((qfill / QBUFS) & 1) ^ 1, abort_flag, p.err)) return false;
                uint8_t* qdst = smem + L::Q_OFF + qs * L::TILE_BYTES;
                if (lane == 0) {
                    // (tq * group rows of 128 bytes: the tile's rows behind them stay as they were)
                    mbar_arrive_expect_tx(bars + L::B_QFULL + qs, (uint32_t)(p.tq * p.group * 128 * L::REGIONS));
                    for (int r = 0; r < L::REGIONS; ++r)
                        tma_load_3d(qdst + r * L::REGION_BYTES, &q_map, bars + L::B_QFULL + qs, r * 64,
                                    cur.hk * p.group, cur.row0 + x * p.tq);
                }
                ++qfill;
                return true;
            };
            // This warp's share of K (kv = 0) or V of key tile j.  A block id out of range is
            // flagged (once, with K), its rows are zero and its keys are absent: their bits in `keeps` are
            // cleared ahead of K's arrival and so of S.  A lane writes the bits of its piece from the first
            // such id that it meets on; nothing else clears them.
            auto load_kv = [&](int x, int kv, int j, int blk) -> bool {
                constexpr int RING = FP8 ? R::STAGES : R::RING;
                const int slot = fill % RING;
                uint64_t* full = bars + (FP8 ? L::B_STFULL : L::B_KVFULL) + slot;
                if (!mbar_wait(bars + (FP8 ? L::B_STEMPTY : L::B_KVEMPTY) + slot, ((fill / RING) & 1) ^ 1,
                               abort_flag, p.err))
                    return false;
                ++fill;
                const int v = piece_key(x, j);
                const bool good = blk >= 0 && blk < p.num_blocks;
                const bool in_range = is_piece(v) && good, bad = is_piece(v) && !good;
                was_bad = was_bad || bad;
                if (kv == 0 && was_bad) {
                    if (bad) {
                        flag_error(p.err, NVPA_FLAG_BAD_BLOCK_ID);
                        *bad_seen = 1;
                    }
                    volatile uint16_t* keep = reinterpret_cast<volatile uint16_t*>(
                        keeps + kfill % kKeeps * KEEP) + pc * piece / 16;
                    for (int i = 0; i < piece / 16; ++i) keep[i] = bad ? 0 : 0xffff;
                    __threadfence_block();   // (lane 0 arrives below)
                }
                kfill += 1 - kv;
                const uint32_t valid = __ballot_sync(0xffffffffu, in_range);
                uint8_t* tile = smem + (FP8 ? L::STAGE_OFF + slot * L::STAGE_BYTES : L::RING_OFF + slot * L::TILE_BYTES);
                if constexpr (!FP8) {
                    for (uint32_t m = __ballot_sync(0xffffffffu, bad); m != 0; m &= m - 1) {
                        const int c = pw + producers * (__ffs(m) - 1);
                        for (int r = 0; r < L::REGIONS; ++r) {
                            uint4* rows = reinterpret_cast<uint4*>(tile + r * L::REGION_BYTES + c * piece * 128);
                            for (int k = lane; k < piece * 8; k += 32) rows[k] = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    if constexpr (FP8) stage_mask[slot * kProducers + pw] = valid;
                    mbar_arrive_expect_tx(full, (uint32_t)__popc(valid) *
                                                    (uint32_t)(FP8 ? piece * (D + 1) : piece * 128 * L::REGIONS));
                }
                __syncwarp();
                if (in_range) {
                    const CUtensorMap* map = kv ? &v_map : &k_map;
                    const int row = keys.real(v) & (p.block_size - 1);
                    const int z = blk * p.block_size + row;
                    if constexpr (FP8) {
                        tma_load_3d(tile + pc * piece * D, map, full, 0, cur.hk, z);
                        const uint8_t* sc = (kv ? p.v_scales : p.k_scales) +
                                            ((size_t)blk * p.hkv + cur.hk) * p.block_size + row;
                        bulk_load(smem + L::SCALE_OFF + slot * kKeys + pc * piece, sc, (uint32_t)piece, full);
                    } else {
#pragma unroll
                        for (int r = 0; r < L::REGIONS; ++r)
                            tma_load_3d(tile + r * L::REGION_BYTES + pc * piece * 128, map, full, r * 64, cur.hk, z);
                    }
                }
                __syncwarp();
                return true;
            };
            // K_0 first (its ring slot frees early), then Q_A, ..., V_0, Q_B, and the rest
            TileWalk w;
            for (int i = 0; i < 2 * (sn0 + sn1) && ok; ++i, w.next(sn0, sn1)) {
                if (w.kv == 0 && w.j > 0) {   // on to the stream's next key tile
                    if (w.x) {
                        blk_b = next_b;
                        next_b = load_piece(1, w.j + 1);
                    } else {
                        blk_a = next_a;
                        next_a = load_piece(0, w.j + 1);
                    }
                }
                ok = load_kv(w.x, w.kv, w.j, w.x ? blk_b : blk_a);
                if (w.j == 0 && w.x == 0 && ok) ok = load_q(w.kv);
            }
        }
        // let every copy this warp started land before the CTA can exit
        if (lane == 0) {
            auto drain = [&](uint64_t* full, uint32_t used, uint32_t ring) {
                for (uint32_t s = 0; s < ring; ++s) {
                    if (used <= s) continue;
                    const uint32_t last = used - 1 - (used - 1 - s) % ring;   // last fill of slot s
                    const uint64_t t0 = global_ns();
                    while (!mbar_try_wait(full + s, (last / ring) & 1) && global_ns() - t0 < 100000000ull) {
                    }
                }
            };
            drain(bars + (FP8 ? L::B_STFULL : L::B_KVFULL), fill, FP8 ? R::STAGES : R::RING);
            drain(bars + L::B_QFULL, qfill, QBUFS);
        }
      } else if (warp == 1) {
        // ============================ MMA issuer ============================
        const uint32_t IDESC_QK = idesc_bf16_f32(kRows, kKeys, false) | (p.negate_qk ? (1u << 13) : 0u);
        constexpr uint32_t IDESC_PV = idesc_bf16_f32(kRows, D, true);
        uint32_t f = 0;                        // ring position
        uint32_t qcons = 0;                    // Q tiles consumed
        uint32_t puse[2] = {0, 0};             // P_j waits per tile
        int units[2] = {0, 0};                 // units in which the tile had work
        bool ok = true;
        constexpr uint32_t DESC_HI = sdesc_sw128_hi(1024);
        constexpr uint32_t TILE16 = L::TILE_BYTES >> 4, REGION16 = L::REGION_BYTES >> 4;
        const uint32_t q_lo = sdesc_sw128_lo(sbase + L::Q_OFF, 16);
        const uint32_t k_lo = sdesc_sw128_lo(sbase + L::RING_OFF, 16);
        const uint32_t v_lo = sdesc_sw128_lo(sbase + L::RING_OFF, L::REGION_BYTES);
        auto issue_qk = [&](int x, int kslot, uint32_t qs) {
            const uint32_t a = q_lo + qs * TILE16, b = k_lo + (uint32_t)kslot * TILE16;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = (kk / 4) * REGION16 + (kk % 4) * 2;   // 64-column region, 32 bytes of K
                umma_ss(tmem + x * 256, sdesc_join(a + o, DESC_HI), sdesc_join(b + o, DESC_HI), IDESC_QK,
                        kk > 0 ? 1u : 0u);
            }
            umma_commit(bars + L::B_SFULL + x);
        };
        auto issue_pv = [&](int x, int vslot, bool accumulate) {
            const uint32_t b = v_lo + (uint32_t)vslot * TILE16;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)   // 16 keys = 16 rows of 128 bytes per MMA
                umma_ts(tmem + x * 256 + kKeys, tmem + x * 256 + kk * 8, sdesc_join(b + kk * 128, DESC_HI), IDESC_PV,
                        (accumulate || kk > 0) ? 1u : 0u);
            umma_commit(bars + L::B_ODONE + x);
        };
        for (int n = 0; ok; ++n) {
            const ChunkUnit u = claim(n);
            if (__shfl_sync(0xffffffffu, u.seq, 0) < 0) break;
            const int nk[2] = {__shfl_sync(0xffffffffu, u.nk[0], 0), __shfl_sync(0xffffffffu, u.nk[1], 0)};
            const int nkv = max(nk[0], nk[1]);
            // the key tile after whose S tile x's Q buffer is free (split: A and B share one Q, which
            // the later of their last S's releases)
            const bool b_last = nk[1] == nk[0];
            const int q_free[2] = {p.split && b_last ? -1 : nk[0] - 1, p.split ? (b_last ? nk[0] - 1 : -1) : nk[1] - 1};
            // S of key tile 0: tile A as soon as Q_A and K_0 are in, then tile B
            uint32_t qsl[2] = {0, 0};
            bool have = false;
            for (int x = 0; x < 2; ++x) {
                if (nk[x] == 0) continue;
                if (!have && !mbar_wait(bars + L::B_KVFULL + f % R::RING, (f / R::RING) & 1, abort_flag, p.err)) {
                    ok = false;
                    break;
                }
                have = true;
                if (x == 1 && p.split) {
                    qsl[1] = qsl[0];
                } else {
                    qsl[x] = qcons % QBUFS;
                    if (!mbar_wait(bars + L::B_QFULL + qsl[x], (qcons / QBUFS) & 1, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    ++qcons;
                }
                tc_fence_after();
                const bool done = p.split || x == 1 || nk[1] == 0;   // with this K tile
                if (lane == 0) {
                    issue_qk(x, f % R::RING, qsl[x]);
                    if (q_free[x] == 0) umma_commit(bars + L::B_QEMPTY + qsl[x]);
                    if (done) umma_commit(bars + L::B_KVEMPTY + f % R::RING);
                }
                __syncwarp();
                if (done) {
                    ++f;
                    have = false;
                }
            }
            for (int j = 0; j < nkv && ok; ++j) {
                bool v_here = false, k_here = false;
                for (int x = 0; x < 2; ++x) {
                    if (j >= nk[x]) continue;
                    const uint32_t fv = f, fk = f + 1;   // V_j and K_{j+1}
                    if (!v_here && !mbar_wait(bars + L::B_KVFULL + fv % R::RING, (fv / R::RING) & 1, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    v_here = true;
                    if (!mbar_wait(bars + L::B_PFULL + x, puse[x] & 1, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    ++puse[x];
                    if (j == 0 && units[x] > 0 &&
                        !mbar_wait(bars + L::B_OFREE + x, (units[x] - 1) & 1, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // P V first: it does not need K_{j+1}, which may still be in flight
                    if (lane == 0) {
                        issue_pv(x, fv % R::RING, j > 0);
                        if (j == nk[x] - 1) umma_commit(bars + L::B_OFINAL + x);
                    }
                    __syncwarp();
                    if (j + 1 < nk[x]) {
                        if (!k_here) {
                            if (!mbar_wait(bars + L::B_KVFULL + fk % R::RING, (fk / R::RING) & 1, abort_flag, p.err)) {
                                ok = false;
                                break;
                            }
                            k_here = true;
                            tc_fence_after();
                        }
                        if (lane == 0) {
                            issue_qk(x, fk % R::RING, qsl[x]);
                            if (j + 1 == q_free[x]) umma_commit(bars + L::B_QEMPTY + qsl[x]);
                        }
                        __syncwarp();
                    }
                    if (p.split || x == 1 || j >= nk[1]) {   // done with these tiles
                        if (lane == 0) {
                            umma_commit(bars + L::B_KVEMPTY + fv % R::RING);
                            if (k_here) umma_commit(bars + L::B_KVEMPTY + fk % R::RING);
                        }
                        __syncwarp();
                        f += k_here ? 2 : 1;
                        v_here = k_here = false;
                    }
                }
            }
            for (int x = 0; x < 2; ++x) {
                if (nk[x] > 0) ++units[x];
            }
        }
        // every MMA this thread issued completes before TMEM is released
        if (lane == 0) umma_commit(bars + L::B_DRAIN);
        __syncwarp();
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(bars + L::B_DRAIN, 0) && global_ns() - t0 < 100000000ull) {
        }
      }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::SOFTMAX_REGS));
        // ============================ softmax warps ============================
        // warps 4..7: tile A, warps 8..11: tile B
        const int x = (warp - 4) >> 2;
        const int quarter = warp & 3;                 // TMEM lanes 32*quarter .. +31
        const int r = quarter * 32 + lane;            // row of the tile: token r / G, head r % G
        const int rtok = r / p.group;
        const int rhead = r - rtok * p.group;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_col = tmem + lane_base + x * 256;
        const uint32_t o_col = s_col + kKeys;
        uint64_t* b_sfull = bars + L::B_SFULL + x;
        uint64_t* b_pfull = bars + L::B_PFULL + x;
        uint64_t* b_odone = bars + L::B_ODONE + x;
        uint64_t* b_ofinal = bars + L::B_OFINAL + x;
        uint64_t* b_ofree = bars + L::B_OFREE + x;
        uint32_t s_use = 0, fbase = 0;
        int tcount = 0;
        uint32_t pv_before = 0;                       // PVs issued for this tile slot before
        for (int n = 0;; ++n) {
            const ChunkUnit u = claim(n);
            if (u.seq < 0) break;
            const uint32_t unit_base = fbase;
            fbase += 2 * (uint32_t)(u.sn[0] + u.sn[1]);
            const int nk = x ? u.nk[1] : u.nk[0], ntok = x ? u.ntok[1] : u.ntok[0];   // (no indexed copy)
            if (nk == 0) continue;
            const Keys& keys = u.keys;
            // a warp whose rows are all behind the tile's last one only keeps the protocol
            const bool idle = quarter * 32 >= ntok * p.group;
            const int pos = keys.p_first + x * p.b_step + min(rtok, ntok - 1);
            // virtual keys that the row sees: [0, va) and [vb, vc)
            const int va = p.window > 0 ? min(p.sinks, pos + 1) : 0;
            const int vb = p.window > 0 ? max(0, pos - p.window + 1) - keys.skip : 0;
            const int vc = keys.upto(pos);
            // and that some row of the pair sees: [0, pa) and [pb, pc)
            const int pa = p.window > 0 ? min(p.sinks, keys.p_first + 1) : 0;
            const int pb = p.window > 0 ? max(0, keys.p_first - p.window + 1) - keys.skip : 0;
            const int pc = keys.upto(keys.p_last);
            const int v0 = u.first_key(p, x);
            const int a_min = __reduce_min_sync(0xffffffffu, va);
            const int b_max = __reduce_max_sync(0xffffffffu, vb);
            const int c_min = __reduce_min_sync(0xffffffffu, vc);
            // key tiles without a mask anywhere in the warp: [open_lo, open_hi), and the whole tiles
            // of long sinks, [0, open_sinks)
            const int open_lo = max(0, (b_max - v0 + kKeys - 1) / kKeys), open_hi = (c_min - v0) / kKeys;
            const int open_sinks = (a_min - v0) / kKeys;
            // which of the unit's K tiles is key tile j of this tile's stream, in the order of the walk: K_0, K_1,
            // ... or, split, A's K_0, B's K_0, A's K_1, ... until B has no more
            const int sn1 = u.sn[1];
            auto k_order = [&](int j) { return p.split && x ? 2 * j + 1 : j + min(j, sn1); };
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < nk; ++j) {
                if (!mbar_wait(b_sfull, s_use & 1, abort_flag, p.err)) {
                    ok = false;
                    break;
                }
                ++s_use;
                tc_fence_after();
                const bool open = (j >= open_lo && j < open_hi) || j < open_sinks;
                if (!idle) {
                    uint32_t sv[kKeys];
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c)
                        tmem_ld32(s_col + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + c * 32));
                    // (behind S, and so behind K's arrival.  Masks in shared memory that are all ones but for
                    // bad blocks: whole prompts 267 -> 271 us, 512-token chunks as before; looking the
                    // blocks up here, in line or in a function, costs calls without any 2 to 5 %.)
                    const bool bad = *bad_seen != 0;
                    tmem_wait_ld();
                    if (!open || bad)
                        mask_columns(sv, v0 + j * kKeys, va, vb, vc, keeps + (unit_base / 2 + k_order(j)) % kKeeps * KEEP);
                    const float mt = row_max<kKeys>(sv) * p.scale_log2;
                    const bool over = mt > m + kRescaleSlack;
                    const bool rescale = __any_sync(0xffffffffu, over);
                    float alpha = 1.f;
                    if (rescale) {
                        const float m_new = over ? mt : m;
                        alpha = over ? (m == -INFINITY ? 0.f : fast_exp2(m - m_new)) : 1.f;
                        l *= alpha;
                        m = m_new;
                    }
                    // a row with no visible key yet (m = -inf) gets exp2(-inf) = 0 through its offset
                    l += exp_row<kKeys>(sv, s_col, p.scale_log2, m > -INFINITY ? -m : -INFINITY);
                    if (rescale && j > 0) {
                        // O holds P_0..P_{j-1} V (all complete once S_j is): rescale it before
                        // P_j is released to the MMA
                        if (!mbar_wait(b_odone, (pv_before + j - 1) & 1, abort_flag, p.err)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(o_col + c * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                            tmem_st32(o_col + c * 32, o);
                        }
                    }
                    tmem_wait_st();
                }
                if constexpr (!FP8) {
                    // V rows that nobody in the pair sees hold stale values, or what the ring
                    // held before: zeroed here, a row per thread, by the warps of the first tile
                    // whose P V reads them (the widening does it for the e4m3 cache)
                    const int base = v0 + j * kKeys;
                    if (!open && (base + kKeys > pc || (base < pb && base + kKeys > pa)) &&
                        (p.split || x == 0 || j >= u.nk[0])) {
                        // ring position of V_j: behind the K_0s and 2 j tiles of this stream, and
                        // what the other stream has passed
                        uint32_t fv = unit_base + 1 + 2 * j + (sn1 > 0 ? 1 + min(j, sn1) + min(j, sn1 - 1) : 0);
                        if (p.split && x == 1) fv += j + 1 < u.sn[0] ? 2 : 1;
                        if (!mbar_wait(bars + L::B_KVFULL + fv % R::RING, (fv / R::RING) & 1, abort_flag, p.err)) {
                            ok = false;
                            break;
                        }
                        const int v = base + r;
                        if (!(v < pc && (v >= pb || v < pa))) {
                            uint8_t* row = smem + L::RING_OFF + (fv % R::RING) * L::TILE_BYTES + r * 128;
#pragma unroll
                            for (int c = 0; c < 8 * L::REGIONS; ++c)   // (r & 7: a warp's stores spread over the banks)
                                *reinterpret_cast<uint4*>(row + (c >> 3) * L::REGION_BYTES + (((c ^ r) & 7) << 4)) =
                                    make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_pfull);
            }
            if (!ok) break;
            if (!mbar_wait(b_ofinal, tcount & 1, abort_flag, p.err)) break;
            tc_fence_after();
            const bool row_ok = rtok < ntok;
            // (a sum that is not a number keeps the row from looking empty)
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            const size_t orow = (size_t)(u.row0 + x * p.b_step + rtok) * p.hq + u.hk * p.group + rhead;
            const bool partial = (x ? u.ns[1] : u.ns[0]) > 1;
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D);
            const size_t prow = orow * p.s_max + u.part + (x && p.split ? 1 : 0);
            float* pdst = p.o_part + prow * D;
            // (loops stay rolled where they can: the warps of a sub-partition share its instruction
            // cache, and a unit's boundary is code that runs once in many key tiles)
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(o_col + c * 32, o);
                tmem_wait_ld();
                if (c == D / 32 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_ofree);
                }
                // (every lane takes part in the loads above: no early exit)
                if (row_ok) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[k]) * inv);
                    if (partial) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            __stcg(reinterpret_cast<uint4*>(pdst + c * 32 + 4 * q),
                                   make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]));
                    } else {
                        uint32_t w[2][8];
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            w[k / 8][k % 8] = pack_bf16x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (p.out_v8) {
                                st_global_v8(dst + c * 4 + 2 * q, w[q]);
                            } else {
                                dst[c * 4 + 2 * q] = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
                                dst[c * 4 + 2 * q + 1] = make_uint4(w[q][4], w[q][5], w[q][6], w[q][7]);
                            }
                        }
                    }
                }
            }
            if (row_ok) {
                if (partial) __stcg(p.lse_part + prow, lse == lse ? lse : INFINITY);   // (NaN: as in the row kernel)
                else if (p.lse_out != nullptr) p.lse_out[orow] = lse;
            }
            pv_before += (uint32_t)nk;
            ++tcount;
        }
    } else {
        // ============================ widening warps (e4m3) ============================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::SMALL_REGS));
        if constexpr (FP8) {
            const int r = (warp - 12) * 32 + lane;    // key row of the tile
            const int prow = r / p.piece;             // its piece: number prow / producers of a producer
            const int of = prow % producers, bit = prow / producers;
            uint32_t fill = 0;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                const ChunkUnit u = claim(n);
                if (u.seq < 0) break;
                const Keys keys = u.keys;
                const int sn0 = u.sn[0], sn1 = u.sn[1];
                TileWalk w;
                for (int i = 0; i < 2 * (sn0 + sn1) && ok; ++i, ++fill, w.next(sn0, sn1)) {
                    const int slot = fill % R::STAGES, ring = fill % R::RING;
                    if (!mbar_wait(bars + L::B_STFULL + slot, (fill / R::STAGES) & 1, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    // rows that nobody in the pair sees, or whose block id is bad, become zero
                    const int key = keys.real(u.first_key(p, w.x) + w.j * kKeys + r);
                    const uint32_t present = stage_mask[slot * kProducers + of] >> bit;
                    const bool seen = (present & 1) && key <= keys.p_last &&
                                      (p.window == 0 || key > keys.p_first - p.window || key < p.sinks);
                    const RowScale f = row_scale(smem[L::SCALE_OFF + slot * kKeys + r]);
                    const uint8_t* src = smem + L::STAGE_OFF + slot * L::STAGE_BYTES + r * D;
                    // 128-byte rows: chunk c lies at c ^ (r % 8); 64-byte rows: at c ^ (r / 2 % 4)
                    const int sx = D == 128 ? r & 7 : (r >> 1) & 3;
                    if (!mbar_wait(bars + L::B_KVEMPTY + ring, ((fill / R::RING) & 1) ^ 1, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    uint8_t* dst = smem + L::RING_OFF + ring * L::TILE_BYTES + r * 128;
                    auto put = [&](int c, const uint4& lo, const uint4& hi) {
                        uint8_t* d = dst + (c / 4) * L::REGION_BYTES;
                        *reinterpret_cast<uint4*>(d + ((((c % 4) * 2) ^ (r & 7)) << 4)) = lo;
                        *reinterpret_cast<uint4*>(d + ((((c % 4) * 2 + 1) ^ (r & 7)) << 4)) = hi;
                    };
                    if (__all_sync(0xffffffffu, seen && f.half != 0)) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D / 16; c0 += 4) {
                            uint4 code[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                code[i] = *reinterpret_cast<const uint4*>(src + (((c0 + i) ^ sx) << 4));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint4 lo, hi;
                                widen16(code[i], f.half, lo, hi);
                                put(c0 + i, lo, hi);
                            }
                        }
                    } else {   // a warp with a special row
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint4 lo, hi;
                            widen16_any(*reinterpret_cast<const uint4*>(src + ((c ^ sx) << 4)), f.value, lo, hi);
                            if (!seen) lo = hi = make_uint4(0, 0, 0, 0);
                            put(c, lo, hi);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bars + L::B_STEMPTY + slot);
                        mbar_arrive(bars + L::B_KVFULL + ring);
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------

// 3-D view (dim, heads, rows) of an e4m3 pool [rows, heads, dim]; box = dim x 1 x box_rows,
// swizzled over its whole row (128 or 64 bytes).
bool make_code_map(CUtensorMap* map, const void* base, int dim, int heads, long long rows, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t gdim[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t gstride[2] = {(cuuint64_t)dim, (cuuint64_t)dim * heads};
    const cuuint32_t box[3] = {(cuuint32_t)dim, 1, (cuuint32_t)box_rows};
    const cuuint32_t estride[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), gdim, gstride, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE, dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FP8>
cudaError_t launch_chunk(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const ChunkParams& p,
                         int grid, cudaStream_t stream) {
    static std::once_flag once[64];
    static int launch_regs[64];
    constexpr int smem = ChunkLayout<D, FP8>::ALLOC;
    auto kern = chunk_tcgen05_kernel<D, FP8>;
    int dev = 0;
    cudaGetDevice(&dev);
    dev &= 63;
    std::call_once(once[dev], [&] {
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        cudaFuncAttributes fa{};
        launch_regs[dev] = cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
    });
    // The warpgroups' setmaxnreg shares add up to LAUNCH_REGS per thread: with fewer registers
    // at launch the raising warpgroups could never get their share, so do not launch.
    if (launch_regs[dev] != Roles<FP8>::LAUNCH_REGS) {
        set_error("chunk kernel compiled with %d registers per thread, %d expected", launch_regs[dev],
                  Roles<FP8>::LAUNCH_REGS);
        return cudaErrorInvalidConfiguration;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Roles<FP8>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, qm, km, vm, p);
}

struct ChunkGeometry {
    int tq, row_pairs, chunk, split, s_max;
    long long pairs;     // bound on the call's pairs
    size_t nsplit, entries, lse_part, o_part, total;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Depends on host-side values only, so that a captured call's launches and workspace are fixed.
ChunkGeometry chunk_geometry(int batch, int total_q, int max_q, int hq, int hkv, int head_dim, int max_ctx,
                             int window, int sinks, int num_splits) {
    ChunkGeometry g{};
    const int group = std::max(1, hq / hkv);
    g.tq = kRows / group;
    const int two = 2 * g.tq;
    g.row_pairs = std::max(1, (int)(((long long)max_q + two - 1) / two));
    g.pairs = std::min((long long)batch * g.row_pairs, (long long)batch + total_q / two);
    // key tiles that a pair can see
    long long keys = std::max(1, max_ctx);
    if (window > 0) keys = std::min(keys, (long long)window + two + (long long)sinks + 2 * kGran);
    const long long tiles = (keys + kKeys - 1) / kKeys;
    g.split = max_q <= g.tq;
    const long long units = std::max(1LL, g.pairs * hkv);
    long long chunk;
    if (num_splits > 0) {
        chunk = std::max(1LL, (tiles + num_splits - 1) / num_splits);
    } else {
        // Units per pair: the number n that gives the least time in key tiles of a pair (2.2 us):
        // rounds of units on 148 SMs, each with about 4 tiles to fill and drain its pipeline;
        // more than one unit also writes and reads a float32 partial per row and partition
        // (14 MB per tile) and launches the merge.  (A split unit works on two partitions at
        // once, so it has partials anyway.  16 windowed chunks of 256 tokens, 256 units: whole
        // 72 us, two parts each 140; 512-token chunks over 8 k tokens, 512 units: 513 and 616;
        // 32-row chunks over 8 k tokens, 64 split units of 64 tiles: 127 us as they are, 72 cut
        // in two.)
        const int lanes = g.split ? 2 : 1;
        const long long row_bytes = (long long)total_q * hq * head_dim * 8;
        long long best = 0, parts = 1;
        for (long long n = 1; n <= std::min(tiles, 64LL); ++n) {
            const long long rounds = (units * n + 147) / 148;
            const long long merge = n > 1 || g.split ? 3 + n * lanes * row_bytes / 14000000 : 0;
            const long long cost = rounds * ((tiles + n * lanes - 1) / (n * lanes) + 4) + merge;
            if (n == 1 || cost < best) {
                best = cost;
                parts = n;
            }
        }
        chunk = std::max(1LL, (tiles + parts * lanes - 1) / (parts * lanes));
    }
    // the partition index stays in 15 bits
    chunk = std::max(chunk, (tiles + 32766) / 32767);
    g.chunk = (int)chunk;
    g.s_max = (int)((tiles + chunk - 1) / chunk);
    size_t off = 256;
    g.nsplit = off; off = align256(off + (g.s_max > 1 ? sizeof(int32_t) * (size_t)total_q : 0));
    g.entries = off; off = align256(off + sizeof(int4) * (size_t)g.pairs * g.s_max);
    g.lse_part = off; off = align256(off + (g.s_max > 1 ? sizeof(float) * (size_t)total_q * hq * g.s_max : 0));
    g.o_part = off; off = align256(off + (g.s_max > 1 ? sizeof(float) * (size_t)total_q * hq * g.s_max * head_dim : 0));
    g.total = off;
    return g;
}

}  // namespace

size_t chunk_tiles_workspace_bytes(int batch, int total_q, int max_q, int hq, int hkv, int head_dim, int max_ctx,
                                   int window, int sinks, int num_splits) {
    return chunk_geometry(batch, total_q, max_q, hq, hkv, head_dim, max_ctx, window, sinks, num_splits).total;
}

nvpa_status_t run_chunk_tiles(const WindowCall& c, cudaStream_t stream) {
    const ChunkGeometry g = chunk_geometry(c.batch, c.total_q, c.max_seqlen_q, c.hq, c.hkv, c.head_dim,
                                           c.max_context_len, c.window, c.num_sinks, c.num_splits);
    if (c.workspace_bytes < g.total) {
        set_error("workspace too small: %zu bytes given, %zu needed", c.workspace_bytes, g.total);
        return NVPA_ERR_WORKSPACE_TOO_SMALL;
    }
    if (g.pairs * g.s_max * c.hkv > 0x7fffffffLL / 2 || (long long)c.batch * g.row_pairs > 0x7fffffffLL / 2) {
        set_error("more than 2^30 work items");
        return NVPA_ERR_UNSUPPORTED;
    }
    const bool fp8 = c.k_scales != nullptr;
    ChunkParams p{};
    // (a window as long as the longest context hides nothing)
    p.window = c.window >= c.max_context_len ? 0 : c.window;
    p.sinks = std::min(c.num_sinks, c.max_context_len);
    p.piece = p.window > 0 ? kGran : std::min(c.block_size, kKeys);
    p.tq = g.tq;
    p.group = c.hq / c.hkv;
    CUtensorMap qm, km, vm;
    const long long rows = (long long)c.num_blocks * c.block_size;
    bool mapped = make_map(&qm, c.q, c.head_dim, c.hq, c.total_q, p.group, p.tq);
    if (fp8)
        mapped = mapped && make_code_map(&km, c.k_cache, c.head_dim, c.hkv, rows, p.piece) &&
                 make_code_map(&vm, c.v_cache, c.head_dim, c.hkv, rows, p.piece);
    else
        mapped = mapped && make_map(&km, c.k_cache, c.head_dim, c.hkv, rows, 1, p.piece) &&
                 make_map(&vm, c.v_cache, c.head_dim, c.hkv, rows, 1, p.piece);
    if (!mapped) {
        set_error("cuTensorMapEncodeTiled failed (driver entry point missing or bad layout)");
        return NVPA_ERR_CUDA;
    }
    uint8_t* ws = static_cast<uint8_t*>(c.workspace);
    p.block_tables = c.block_tables;
    p.cu_q = c.cu_seqlens_q;
    p.context_lens = c.context_lens;
    p.k_scales = c.k_scales;
    p.v_scales = c.v_scales;
    p.out = static_cast<uint16_t*>(c.out);
    p.lse_out = c.lse_out;
    p.counter = reinterpret_cast<int32_t*>(ws);
    p.nsplit = reinterpret_cast<int32_t*>(ws + g.nsplit);
    p.entries = reinterpret_cast<int4*>(ws + g.entries);
    p.lse_part = reinterpret_cast<float*>(ws + g.lse_part);
    p.o_part = reinterpret_cast<float*>(ws + g.o_part);
    p.err = c.err_flag;
    p.batch = c.batch;
    p.total_q = c.total_q;
    p.max_q = c.max_seqlen_q;
    p.max_ctx = c.max_context_len;
    p.hq = c.hq;
    p.hkv = c.hkv;
    p.row_pairs = g.row_pairs;
    p.max_blocks = c.max_blocks_per_seq;
    p.num_blocks = c.num_blocks;
    p.block_size = c.block_size;
    p.block_shift = __builtin_ctz((unsigned)c.block_size);
    p.chunk = g.chunk;
    p.split = g.split;
    p.b_step = g.split ? 0 : g.tq;
    p.unit_tiles = g.split ? 2 * g.chunk : g.chunk;
    p.s_max = g.s_max;
    p.max_entries = (int)(g.pairs * g.s_max);
    // the scale multiplies raw scores as a positive factor; a negative one flips the sign of
    // Q K^T in the MMA, and zero becomes the smallest normal float (uniform weights)
    const float a = std::fabs(c.scale) * kLog2e;
    p.scale_log2 = a > 0.f ? a : FLT_MIN;
    p.negate_qk = c.scale < 0.f;
    p.out_v8 = (reinterpret_cast<uintptr_t>(c.out) & 31u) == 0;

    chunk_plan_kernel<<<1, 1024, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failure(e, "chunk attention plan launch");
    count_launches(1);
    const long long max_units = g.pairs * g.s_max * c.hkv;
    const int grid = (int)std::max(1LL, std::min<long long>((long long)device_sm_count(), max_units));
    if (c.head_dim == 128)
        e = fp8 ? launch_chunk<128, true>(qm, km, vm, p, grid, stream)
                : launch_chunk<128, false>(qm, km, vm, p, grid, stream);
    else
        e = fp8 ? launch_chunk<64, true>(qm, km, vm, p, grid, stream)
                : launch_chunk<64, false>(qm, km, vm, p, grid, stream);
    if (e != cudaSuccess) return cuda_failure(e, "chunk attention launch");
    count_launches(1);
    if (g.s_max > 1) {
        AttnParams cp{};
        cp.out = p.out;
        cp.lse_out = p.lse_out;
        cp.o_part = p.o_part;
        cp.lse_part = p.lse_part;
        cp.nsplit = p.nsplit;
        cp.batch = c.total_q;
        cp.hq = c.hq;
        cp.s_max = g.s_max;
        e = launch_decode_combine(cp, c.head_dim, stream);
        if (e != cudaSuccess) return cuda_failure(e, "chunk attention combine launch");
        count_launches(1);
    }
    return NVPA_OK;
}

}  // namespace nvpa
