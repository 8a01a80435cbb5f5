// Attention of a few query rows per KV head over a bf16 or e4m3 paged cache, with an
// optional sliding window and first tokens that stay visible: the decode step (one token
// per sequence) and short chunks of new tokens.
//
// Mathematics.  Query token at position p sees key j iff j <= p and (no window, or
// j > p - window, or j < sinks).  Per query row: s_j = scale <q, k_j> over its visible
// keys, out = sum_j softmax(s)_j v_j, lse = log sum_j exp(s_j), in one pass with a running
// maximum and sum.  An e4m3 row is c * 2^e (fp8.cuh): the key's 2^e multiplies its score
// in float32, the value's 2^e its weight.
//
// Bound by the bytes of the visible keys and values (2 G flop per bf16 byte, 4 G per e4m3
// byte for G query heads per KV head).  The products are small matrix products over the G
// heads, so they go to warp-level MMAs with the keys as the M dimension and the query rows
// as N = 8: S^T[16 keys, 8 rows] = K Q^T and O^T[D, 8 rows] += V^T P^T.  With CUDA-core
// products the e4m3 cache's instructions per byte would bound the kernel; with MMAs 32 keys of
// it take about 670 warp instructions for any G up to 8, a third of them the conversion of its
// codes.  (tcgen05 needs M = 64 or 128 rows of accumulators in TMEM per product, a single
// warp's stream of keys has no use for it.)
// Measured: 8 contexts of 32 k keys, 32 / 8 heads of 128, e4m3 cache: 105 us, 5.1 TB/s (0.79 of
// the copy bandwidth; the marginal rate of more contexts is 6.3 TB/s, the rest is the start of
// the streams, the merge and the launches); 256 contexts in a window of 1024 keys, bf16 cache:
// 194 us, 5.5 TB/s; a context of 4 k keys alone 15 us.
//
// Layout.  Every warp is an independent worker: it takes items (KV head, range of
// 16-key tiles of one sequence) and streams their K and V through its own ring of two shared
// memory stages (of two tiles, e4m3) with 16-byte cp.async copies.  Chunks of up to 24 rows per
// KV head (16 over a bf16 cache) take 2 or 3 such N = 8 row groups in one pass over the keys.  Rows that no query row of the item sees are
// zero-filled and never read, and neither are the block-table entries of blocks without a
// visible key: blocks that fell out of the window may be freed.  A row's 16-byte chunks are
// XOR-swizzled by its key so that the fragment loads below hit all banks.
//   K fragment (A of S^T, keys x dims): the MMA's k index may be any order of the dims as
//     long as Q's fragment has the same, so lane (g, t) = (lane / 4, lane % 4) reads whole
//     16-byte chunks of keys g and g + 8.
//   V fragment (A of O^T, dims x keys): bf16 through ldmatrix.trans; e4m3 by loading 16
//     (D = 128) or 8 dims of the lane's four keys and interleaving pairs of keys with prmt.
//   P^T (B of O^T): the scores lie with keys in rows; movmatrix transposes 8 x 8 tiles.
// Rounding: an e4m3 code is exact in fp16; q is scaled by a power of two per row to [2^14, 2^15)
// for its largest element and rounded to fp16 (bf16 has 8 significant bits: exact for elements
// down to 2^-31 of the largest, and off by 2^-39 of it at most).  Weights are fp16 for the e4m3
// cache (2^-11 relative) and a sum of two bf16 for the bf16 cache, whose values are used as they
// are: its upper half cut off (2^-7) and the rest rounded (2^-9 of it), 2^-16 in all.
// The fp16 weight includes the value's 2^e and is taken relative to 2^-7 of the largest such
// weight (a running maximum of its own beside the softmax's), so a scale of any size does not
// overflow.  fp16 holds w = p 2^(e - gap) only to 2^-25 (p: the softmax weight relative to its
// own reference, gap: the difference of the two references), which is 2^(gap - e - 25) of p: for
// e >= gap at most 2^-25, as an fp16 softmax weight alone would have it, and 2^-32 where the
// values' scales are alike.  A stage with a key of a smaller scale (rows 2^7 below the one that
// counts most) takes float32 weights and CUDA-core products instead, which cost it about five
// times as much.  (A second product for the weights below 2^-14 of every stage, with the values
// scaled by 2^-15, costs 3 % of a decode and 17 to 26 % of the 16- and 24-row passes.)
#include <algorithm>
#include <cuda_fp16.h>
#include <mutex>

#include "decode_params.cuh"
#include "fp8.cuh"

namespace nvpa {

namespace {

constexpr int kRowWarps = 4;
constexpr float kWeightTop = 7.f;   // log2 of the largest fp16 weight when its reference is set: with
                                    // kRescaleSlack above it 2^15

struct RowParams {
    const uint16_t* q;           // [total_q, hq, D]
    const void* k_cache;
    const void* v_cache;
    const uint8_t* k_scales;     // [num_blocks, hkv, block_size] (e4m3 cache)
    const uint8_t* v_scales;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* cu_q;         // null: one query token per sequence
    uint16_t* out;
    float* lse_out;
    float* o_part;
    float* lse_part;
    int4* items;                 // two int4 per item
    int32_t* nsplit;             // [total_q] partitions of each query token, 0: none
    int32_t* counter;            // [0] items claimed after the first round, [1] items
    int32_t* err;
    int batch, total_q, max_q, hq, hkv, group;
    int max_blocks, num_blocks, block_size, block_shift;
    int max_ctx;
    int window, sinks;           // window 0: none
    int planned;                 // items come from the plan kernel
    int chunk;                   // 16-key tiles per partition
    int s_max;
    int max_entries;             // entries that the item table holds
    float scale_log2;
};

// The 16-key tiles that the queries at positions [p0, p1] see, as one virtual range: `head`
// tiles from key 0 on (the sinks), then those from key 16 * (head + skip) on.
struct TileRange {
    int head, skip, count;
};
__device__ __forceinline__ TileRange tile_range(int p0, int p1, int window, int sinks) {
    TileRange r;
    const int lo = window > 0 ? max(0, p0 - window + 1) : 0;
    const int first = lo / kTileKeys;
    r.head = min(first, (int)(((long long)min(sinks, p0) + kTileKeys - 1) / kTileKeys));
    r.skip = first - r.head;
    r.count = r.head + p1 / kTileKeys + 1 - first;
    return r;
}

// Bit i set for the first n of 16 keys.
__device__ __forceinline__ uint32_t first_keys(int n) {
    return n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1u;
}
// Keys key0 .. key0 + 15 that a query at position p sees (p < 0: none).
__device__ __forceinline__ uint32_t seen_keys(int key0, int p, int window, int sinks) {
    uint32_t m = first_keys(p + 1 - key0);
    if (window > 0) m &= ~first_keys(p - window + 1 - key0) | first_keys(sinks - key0);
    return m;
}

// The query tokens of sequence b, which are one item per KV head and partition; ntok = 0 when there
// are none.
struct RowSeq {
    int b, q0, ntok, p0;
    int tiles, ns;       // 16-key tiles that it sees, partitions
};
__device__ __forceinline__ RowSeq row_seq(const RowParams& p, int b, bool flag) {
    const int lim = (int)min((long long)p.max_ctx, (long long)p.max_blocks * p.block_size);
    RowSeq t;
    t.b = b;
    int ctx = __ldg(p.context_lens + b);
    t.ntok = 1;
    t.q0 = b;
    bool ok = ctx >= 0 && ctx <= lim;
    if (p.cu_q != nullptr) {
        t.q0 = __ldg(p.cu_q + b);
        const int q1 = __ldg(p.cu_q + b + 1);
        ok = ok && t.q0 >= 0 && q1 >= t.q0 && q1 <= p.total_q && q1 - t.q0 <= p.max_q && q1 - t.q0 <= ctx;
        t.ntok = ok ? q1 - t.q0 : 0;   // a bad sequence's rows are left unwritten
    } else {
        ctx = min(max(ctx, 0), lim);
    }
    if (!ok && flag) flag_error(p.err, NVPA_FLAG_BAD_LENGTH);
    t.p0 = ctx - t.ntok;
    t.tiles = t.ntok > 0 && t.p0 >= 0 ? tile_range(t.p0, t.p0 + t.ntok - 1, p.window, p.sinks).count : 0;
    t.ns = t.ntok > 0 ? max(1, (t.tiles + p.chunk - 1) / p.chunk) : 0;
    return t;
}
// Its partitions of the full size; the last one is shorter when there is one more.
__device__ __forceinline__ int full_parts(const RowParams& p, const RowSeq& t) {
    return t.ns - (t.tiles < t.ns * p.chunk ? 1 : 0);
}

// ------------------------------------------------------------------------------------
// plan: context lengths -> items, full partitions first, then the shorter ones, longest
// first (as the decode plan orders them)
// ------------------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) row_plan_kernel(const RowParams p) {
    __shared__ int warp_tot[32];
    __shared__ int s_cls[kLengthClasses];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    for (int i = tid; i < kLengthClasses; i += blockDim.x) s_cls[i] = 0;
    if (p.cu_q != nullptr)
        for (int i = tid; i < p.total_q; i += blockDim.x) p.nsplit[i] = 0;
    __syncthreads();
    // (cumulative lengths that run backwards can claim rows twice, and so more entries than
    // the table has room for: what does not fit is dropped and flagged)
    auto put = [&](int at, const RowSeq& t, int s) {
        if (at >= p.max_entries) return;
        p.items[2 * at] = make_int4(t.b, s | (t.ns << 16), t.q0, t.ntok);
        p.items[2 * at + 1] = make_int4(t.p0, s * p.chunk, min(t.tiles, (s + 1) * p.chunk), 0);
    };
    int carry = 0;
    const int n = p.batch;
    for (int base = 0; base < n; base += blockDim.x) {
        const int i = base + tid;
        RowSeq t{};
        int nfull = 0;
        if (i < n) {
            t = row_seq(p, i, true);
            if (t.ns > 0) {
                for (int k = 0; k < t.ntok; ++k) p.nsplit[t.q0 + k] = t.ns;
                const int last = t.tiles - (t.ns - 1) * p.chunk;
                nfull = last == p.chunk ? t.ns : t.ns - 1;
                if (last < p.chunk) atomicAdd(s_cls + length_class(last, p.chunk), 1);
            }
        }
        int block_tot = 0;
        const int e = carry + block_exclusive_scan(nfull, warp_tot, block_tot);
        for (int s = 0; s < nfull; ++s) put(e + s, t, s);
        carry += block_tot;
    }
    __syncthreads();
    const int cls = kLengthClasses - 1 - tid;
    const int v = tid < kLengthClasses ? s_cls[cls] : 0;
    int tot_short = 0;
    const int e = block_exclusive_scan(v, warp_tot, tot_short);
    if (tid < kLengthClasses) s_cls[cls] = carry + e;
    __syncthreads();
    for (int i = tid; i < n; i += blockDim.x) {
        const RowSeq t = row_seq(p, i, false);
        if (t.ns == 0) continue;
        const int last = t.tiles - (t.ns - 1) * p.chunk;
        if (last == p.chunk) continue;
        put(atomicAdd(s_cls + length_class(last, p.chunk), 1), t, t.ns - 1);
    }
    if (tid == 0) {
        const int total = carry + tot_short;
        if (total > p.max_entries) flag_error(p.err, NVPA_FLAG_BAD_LENGTH);
        p.counter[0] = 0;
        p.counter[1] = min(total, p.max_entries) * p.hkv;
    }
}

// ------------------------------------------------------------------------------------
// the worker kernel
// ------------------------------------------------------------------------------------
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&a)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float max_over_keys(float v) {   // lanes with the same lane % 4
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A stage of a warp's ring: TILES 16-key tiles that are worked on together.
template <int D, bool FP8, int NT>
struct RowStage {
    static constexpr int TILES = FP8 ? 2 : 1;
    // The Q fragments of 24 rows live in shared memory: beside 48 registers of them only one tile
    // at a time would fit the register file, and two independent tiles hide the latency of 8
    // warps per SM (5 draft tokens, 4 heads per group, 30 contexts of 8 k: 157 us, one tile 193;
    // 16 rows one tile at a time in 12 warps per SM: 179 us against 136).
    static constexpr bool Q_SMEM = NT > 2;
    static constexpr int Q_BYTES = Q_SMEM ? NT * (D / 16) * 32 * 8 : 0;
    static constexpr int ROW = FP8 ? D : 2 * D;             // bytes of a key's row
    static constexpr int CHUNKS = ROW / 16;
    static constexpr int KV = kTileKeys * ROW;              // K of a tile, then its V
    static constexpr int SCALES = TILES * 2 * KV;           // per tile 16 K scales, 16 V scales
    static constexpr int META = SCALES + (FP8 ? TILES * 32 : 0);
    static constexpr int BYTES = META + 16;
    // byte offset of chunk c of key row r
    __device__ static __forceinline__ int at(int r, int c) {
        return r * ROW + ((CHUNKS >= 8 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3))) << 4);
    }
};

// Ring depth: a warp loads one stage while it works on the other.
constexpr int kRowStages = 2;

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kRowWarps * 32, D == 128 && FP8 && NT == 1 ? 3 : 0)
row_attention_kernel(const RowParams p) {
    using Stage = RowStage<D, FP8, NT>;
    constexpr int STAGES = kRowStages;
    constexpr int TILES = Stage::TILES;
    constexpr uint32_t ALL = TILES == 2 ? 0xffffffffu : 0xffffu;   // every key of a stage
    constexpr int KK = D / 16;    // MMAs along D
    constexpr int MT = D / 16;    // 16-dim tiles of O^T
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t* wsm = smem + (size_t)warp * STAGES * Stage::BYTES;
    const uint32_t wbase = smem_u32(wsm);
    const size_t row_bytes = (size_t)p.hkv * Stage::ROW;   // bytes between cache rows (slots)
    const int tile_shift = p.block_shift - 4;              // 16-key tiles per block, log2

    // ---------------- issue side ----------------
    bool it_valid = false;
    int4 it_a = make_int4(0, 0, 0, 0), it_b = it_a;
    int it_hk = 0, it_v = 0, it_end = 0, it_plast = 0;
    int it_blk[TILES] = {};
    TileRange it_r{};
    const int32_t* it_bt = nullptr;

    const int nwarps = gridDim.x * kRowWarps;
    int nx_item = blockIdx.x * kRowWarps + warp;
    // A call whose items fit one round has no plan kernel, which would cost 5 us of its 15 to 100:
    // every CTA counts the sequences' partitions itself, a sequence per thread.  Items are the
    // full partitions of all sequences, then the shorter last ones, each for every KV head.  (With
    // several rounds the plan's order and dynamic claims are worth more than its time: 64 contexts
    // of 0.5 to 4 k keys 72 us with it, 78 without.)
    __shared__ int s_full[kRowWarps * 32], s_rest[kRowWarps * 32], s_scan[32];
    int total_items = 0, total_full = 0;
    if (p.planned) {
        pdl_wait();
        total_items = __ldcg(p.counter + 1);
    } else {
        int full = 0, rest = 0, total_rest = 0;
        if ((int)threadIdx.x < p.batch) {
            const RowSeq r = row_seq(p, threadIdx.x, blockIdx.x == 0);
            full = full_parts(p, r);
            rest = r.ns - full;
        }
        s_full[threadIdx.x] = block_exclusive_scan(full, s_scan, total_full);
        s_rest[threadIdx.x] = block_exclusive_scan(rest, s_scan, total_rest);
        __syncthreads();
        total_items = (total_full + total_rest) * p.hkv;
    }
    // item c (of one KV head) without a plan: its sequence is the last one with at most c
    // partitions before it
    auto find = [&](int c) {
        const bool rest = c >= total_full;
        const int k = rest ? c - total_full : c;
        const int* before = rest ? s_rest : s_full;
        int i = -1;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) i += __popc(__ballot_sync(0xffffffffu, before[32 * w + lane] <= k));
        const RowSeq r = row_seq(p, i, false);
        const int s = rest ? r.ns - 1 : k - before[i];
        it_a = make_int4(r.b, s | (r.ns << 16), r.q0, r.ntok);
        it_b = make_int4(r.p0, s * p.chunk, min(r.tiles, (s + 1) * p.chunk), 0);
    };
    auto real_tile = [&](int v) { return v < it_r.head ? v : v + it_r.skip; };
    auto load_block = [&]() {   // the table entries of the stage to be issued next (checked there)
#pragma unroll
        for (int u = 0; u < TILES; ++u)
            it_blk[u] = it_v + u < it_end ? __ldg(it_bt + (real_tile(it_v + u) >> tile_shift)) : 0;
    };
    auto fetch = [&]() {
        const int idx = __shfl_sync(0xffffffffu, nx_item, 0);
        if (idx >= total_items) {
            it_valid = false;
            return;
        }
        it_valid = true;
        const int e = idx / p.hkv;
        it_hk = idx - e * p.hkv;
        if (p.planned) {
            if (lane == 0) nx_item = nwarps + atomicAdd(p.counter, 1);
            it_a = __ldcg(reinterpret_cast<const int4*>(p.items) + 2 * e);
            it_b = __ldcg(reinterpret_cast<const int4*>(p.items) + 2 * e + 1);
        } else {
            nx_item += nwarps;
            find(e);
        }
        it_bt = p.block_tables + (size_t)it_a.x * p.max_blocks;
        it_plast = it_b.x + it_a.w - 1;
        it_r = tile_range(max(it_b.x, 0), max(it_plast, 0), p.window, p.sinks);
        it_v = it_b.y;
        it_end = it_b.z;
        load_block();
    };
    // this lane's chunk of rows lane / CHUNKS + i * (32 / CHUNKS)
    constexpr int COPIES = Stage::CHUNKS / 2, STEP = 32 / Stage::CHUNKS;
    const size_t lane_off = (size_t)(lane / Stage::CHUNKS) * row_bytes + (lane % Stage::CHUNKS) * 16;
    const size_t row_step = (size_t)STEP * row_bytes;
    const uint32_t lane_row = wbase + Stage::at(lane / Stage::CHUNKS, lane % Stage::CHUNKS);
    const uint32_t lane_row2 = wbase + Stage::at(lane / Stage::CHUNKS + STEP, lane % Stage::CHUNKS);
    // The swizzle repeats every 8 rows (4 rows of 64 bytes: every 8 too), so copy i goes to
    // copy i - 2's place plus 2 STEP rows when STEP is 4; otherwise it is computed.
    auto dst_of = [&](int i) -> uint32_t {
        if constexpr (STEP == 4) return ((i & 1) ? lane_row2 : lane_row) + (i >> 1) * 8 * Stage::ROW;
        else return wbase + Stage::at(lane / Stage::CHUNKS + i * STEP, lane % Stage::CHUNKS);
    };
    // meta: (real tile, first | last << 1 | open << 2, seen keys, real second tile); tile -1
    // ends the loop, -2 is an item without keys; an open stage is seen whole by every row
    auto issue = [&](int st) {
        uint8_t* sb = wsm + st * Stage::BYTES;
        int4* meta = reinterpret_cast<int4*>(sb + Stage::META);
        if (!it_valid) {
            if (lane == 0) *meta = make_int4(-1, 0, 0, 0);
            cp_async_commit();
            return;
        }
        const bool first = it_v == it_b.y, last = it_v + TILES >= it_end;
        if (it_v < it_end) {
            int tile[2] = {0, 0};
            bool open = it_v + TILES <= it_end;
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                tile[u] = real_tile(it_v + (u > 0 && it_v + u < it_end ? u : 0));
                const int key0 = tile[u] * kTileKeys;
                open = open && key0 + kTileKeys - 1 <= it_b.x && it_blk[u] >= 0 && it_blk[u] < p.num_blocks &&
                       (p.window == 0 || key0 > it_plast - p.window || key0 + kTileKeys <= p.sinks);
            }
            uint32_t seen = ALL;
            if (!open) {
                seen = 0;
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    const bool have = it_v + u < it_end;
                    const int key0 = tile[u] * kTileKeys;
                    // keys that the item's first or any later query token sees
                    uint32_t m = have ? first_keys(it_plast + 1 - key0) : 0;
                    if (p.window > 0) m &= ~first_keys(it_b.x - p.window + 1 - key0) | first_keys(p.sinks - key0);
                    if (have && (it_blk[u] < 0 || it_blk[u] >= p.num_blocks)) {
                        if (lane == 0) flag_error(p.err, NVPA_FLAG_BAD_BLOCK_ID);
                        m = 0;   // its rows are absent
                    }
                    if (m == 0) it_blk[u] = 0;   // nothing is read
                    seen |= m << (16 * u);
                }
            }
            const uint32_t sd = (uint32_t)(st * Stage::BYTES);
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                const size_t slot = (size_t)it_blk[u] * p.block_size + (tile[u] * kTileKeys & (p.block_size - 1));
                const size_t off = slot * row_bytes + (size_t)it_hk * Stage::ROW + lane_off;
                const uint8_t* kg = static_cast<const uint8_t*>(p.k_cache) + off;
                const uint8_t* vg = static_cast<const uint8_t*>(p.v_cache) + off;
                const uint32_t kd = sd + u * 2 * Stage::KV;
                if (open) {
#pragma unroll
                    for (int i = 0; i < COPIES; ++i, kg += row_step, vg += row_step) {
                        cp_async16_to(dst_of(i) + kd, kg, 16);
                        cp_async16_to(dst_of(i) + kd + Stage::KV, vg, 16);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < COPIES; ++i, kg += row_step, vg += row_step) {
                        // 0: zero-filled, not read
                        const int nb = (seen >> (16 * u + lane / Stage::CHUNKS + i * STEP)) & 1 ? 16 : 0;
                        cp_async16_to(dst_of(i) + kd, kg, nb);
                        cp_async16_to(dst_of(i) + kd + Stage::KV, vg, nb);
                    }
                }
            }
            if constexpr (FP8) {
                // lane 2 u + v: the K (v = 0) or V scales of tile u
                if (lane < 2 * TILES) {
                    const int u = lane >> 1;
                    const size_t so = ((size_t)(u ? it_blk[TILES - 1] : it_blk[0]) * p.hkv + it_hk) * p.block_size +
                                      ((u ? tile[1] : tile[0]) * kTileKeys & (p.block_size - 1));
                    cp_async16_to(wbase + sd + Stage::SCALES + lane * 16,
                                  ((lane & 1) ? p.v_scales : p.k_scales) + so, 16);
                }
            }
            if (lane == 0)
                *meta = make_int4(tile[0], (first ? 1 : 0) | (last ? 2 : 0) | (open ? 4 : 0), (int)seen, tile[1]);
        } else if (lane == 0) {
            *meta = make_int4(-2, 3, 0, 0);
        }
        cp_async_commit();
        it_v += TILES;
        if (last) fetch(); else load_block();
    };

    // ---------------- consume side ----------------
    int4 a = make_int4(0, 0, 0, 0), b = a;
    int hk = 0;                    // item being consumed
    uint32_t qf[Stage::Q_SMEM ? 1 : NT][Stage::Q_SMEM ? 1 : KK][2] = {};
    uint2* const qs_mem = reinterpret_cast<uint2*>(smem + (size_t)kRowWarps * STAGES * (Stage::BYTES + 48) +
                                                   warp * Stage::Q_BYTES) + lane;
    auto q_frag = [&](int j, int k) {
        if constexpr (Stage::Q_SMEM) return qs_mem[(j * KK + k) * 32];
        else return make_uint2(qf[j][k][0], qf[j][k][1]);
    };
    auto set_q = [&](int j, int k, uint32_t x, uint32_t y) {
        if constexpr (Stage::Q_SMEM) qs_mem[(j * KK + k) * 32] = make_uint2(x, y);
        else qf[j][k][0] = x, qf[j][k][1] = y;
    };
    float qs[NT][2];               // score factor of rows 8 j + 2 t + {0, 1}
    int pos[NT][2];                // their positions (-1: no such row)
    float o[NT][MT][4];
    float m[NT][2], mv[NT][2], l[NT][2];
    float gap = 0.f;               // largest mv - m of this lane's rows
    uint32_t unset = 0;            // rows (bit 2 j + x) that have seen no key: their m and mv mean nothing yet

    auto start = [&](const int4& na, const int4& nb, int nhk) {
        a = na;
        b = nb;
        hk = nhk;
        unset = 0;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            // Q^T fragment: row n = 8 j + g, the dims that this lane's K chunks hold
            const int n = 8 * j + g;
            const int tk = n / p.group, hd = n - tk * p.group;
            const bool ok = tk < a.w;
            const uint16_t* src = p.q + ((size_t)(a.z + (ok ? tk : 0)) * p.hq + hk * p.group + hd) * D;
            float fac = p.scale_log2;
            if constexpr (FP8) {
                uint32_t w[KK][2];
#pragma unroll
                for (int i = 0; i < KK / 4; ++i) {   // 16 dims per 16-byte chunk of codes
                    const uint4* from = reinterpret_cast<const uint4*>(src + ((KK / 4) * t + i) * 16);
                    const uint4 u = ok ? __ldg(from) : make_uint4(0, 0, 0, 0);
                    const uint4 v = ok ? __ldg(from + 1) : make_uint4(0, 0, 0, 0);
                    w[4 * i][0] = u.x; w[4 * i][1] = u.y; w[4 * i + 1][0] = u.z; w[4 * i + 1][1] = u.w;
                    w[4 * i + 2][0] = v.x; w[4 * i + 2][1] = v.y; w[4 * i + 3][0] = v.z; w[4 * i + 3][1] = v.w;
                }
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < KK; ++i) mx = __vmaxu2(mx, __vmaxu2(w[i][0] & 0x7fff7fffu, w[i][1] & 0x7fff7fffu));
                mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                // the largest element to [2^14, 2^15), near the top of fp16's range (a largest one of
                // 2^127 or more to 2^15 at most times 1.9922, still below 65504); rows too small or
                // not finite stay in range
                const int eq = min(max((int)(mx >> 7), 15), 253);
                const float inv = scale_value(254 + 14 - eq);
                fac *= scale_value(eq - 14);
#pragma unroll
                for (int i = 0; i < KK; ++i)
                    set_q(j, i, pack_half2(bf16_lo(w[i][0]) * inv, bf16_hi(w[i][0]) * inv),
                          pack_half2(bf16_lo(w[i][1]) * inv, bf16_hi(w[i][1]) * inv));
            } else {
#pragma unroll
                for (int i = 0; i < KK / 2; ++i) {   // 8 dims per chunk
                    const int c = 2 * t + (i & 1) + 8 * (i >> 1);
                    const uint4 u = ok ? __ldg(reinterpret_cast<const uint4*>(src + c * 8)) : make_uint4(0, 0, 0, 0);
                    set_q(j, 2 * i, u.x, u.y);
                    set_q(j, 2 * i + 1, u.z, u.w);
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                qs[j][x] = __shfl_sync(0xffffffffu, fac, (2 * t + x) * 4);
                const int r = 8 * j + 2 * t + x, rt = r / p.group;
                pos[j][x] = rt < a.w ? b.x + rt : -1;
                m[j][x] = mv[j][x] = l[j][x] = 0.f;
                if (pos[j][x] >= 0) unset |= 1u << (2 * j + x);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[j][i][x] = 0.f;
        }
    };

    auto epilogue = [&]() {
        const int s = a.y & 0xffff, ns = a.y >> 16;
        if (!p.planned && s == 0 && hk == 0 && lane < a.w) p.nsplit[a.z + lane] = ns;   // for the combine
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float sum = l[j][x];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                const int r = 8 * j + 2 * t + x, tk = r / p.group;
                if (tk >= a.w) continue;
                const size_t row = (size_t)(a.z + tk) * p.hq + hk * p.group + (r - tk * p.group);
                float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
                if constexpr (FP8) inv = sum == 0.f ? 0.f : inv * exp2f(mv[j][x] - m[j][x]);
                const float lse = sum == 0.f ? -INFINITY : (m[j][x] + log2f(sum)) * kLn2;
                if (g == 0) {
                    // (NaN as +inf: the combine drops a NaN from its maximum, and a row that
                    // is not a number would come out as one without keys)
                    if (ns > 1) __stcg(p.lse_part + row * p.s_max + s, lse == lse ? lse : INFINITY);
                    else if (p.lse_out != nullptr) p.lse_out[row] = lse;
                }
                if constexpr (FP8) {
                    // this lane's dims: g * (D / 8) .. + D / 8
                    constexpr int N = D / 8;
                    float v[N];
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        v[2 * i] = o[j][i][x] * inv;
                        v[2 * i + 1] = o[j][i][2 + x] * inv;
                    }
                    if (ns > 1) {
                        float* dst = p.o_part + (row * p.s_max + s) * D + g * N;
#pragma unroll
                        for (int i = 0; i < N; i += 4)
                            __stcg(reinterpret_cast<float4*>(dst + i), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
                    } else {
                        uint16_t* dst = p.out + row * D + g * N;
#pragma unroll
                        for (int i = 0; i < N; i += 8)
                            *reinterpret_cast<uint4*>(dst + i) =
                                make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                                           pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float v = o[j][i][2 * y + x] * inv;
                            const int dim = 16 * i + 8 * y + g;
                            if (ns > 1) __stcg(p.o_part + (row * p.s_max + s) * D + dim, v);
                            else reinterpret_cast<__nv_bfloat16*>(p.out)[row * D + dim] = __float2bfloat16_rn(v);
                        }
                }
            }
    };

    // Sums and O^T += V^T P^T of an e4m3 stage with float32 weights, key by key on the CUDA cores.
    auto add_float32 = [&](const uint8_t* sb, const float (&sc)[TILES][NT][4], const float (&ew)[TILES][NT][4]) {
        constexpr int N = D / 8;   // dims of this lane: g * N ..
#pragma unroll
        for (int u = 0; u < TILES; ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float w[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        l[j][x] += fast_exp2(sc[u][j][2 * y + x]);
                        w[j][x] = fast_exp2(ew[u][j][2 * y + x]);
                    }
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {   // key k + 8 y of tile u, its weights from the lanes that have it
                    float wk[NT][2];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int x = 0; x < 2; ++x) wk[j][x] = __shfl_sync(0xffffffffu, w[j][x], 4 * k + t);
                    const uint8_t* vs = sb + u * 2 * Stage::KV + Stage::KV;
#pragma unroll
                    for (int i = 0; i < MT; i += 2) {   // four dims
                        const int dim = g * N + 2 * i;
                        uint32_t h[2];
                        e4m3x4_to_half2(*reinterpret_cast<const uint32_t*>(
                            vs + Stage::at(k + 8 * y, dim >> 4) + (dim & 15)), h[0], h[1]);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h[z]));
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    o[j][i + z][x] = fmaf(wk[j][x], c.x, o[j][i + z][x]);
                                    o[j][i + z][2 + x] = fmaf(wk[j][x], c.y, o[j][i + z][2 + x]);
                                }
                        }
                    }
                }
            }
    };

    auto consume = [&](int st, const int4& meta) {
        const uint8_t* sb = wsm + st * Stage::BYTES;
        const uint32_t sa = wbase + st * Stage::BYTES;
        const int key0[2] = {meta.x * kTileKeys, meta.w * kTileKeys};
        // ---- S^T = K Q^T ----
        float sc[TILES][NT][4];
#pragma unroll
        for (int u = 0; u < TILES; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) sc[u][j][x] = 0.f;
        if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < KK / 4; ++i) {
                const int c = (KK / 4) * t + i;
                uint32_t lo[TILES][4], hi[TILES][4];
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    const uint8_t* ks = sb + u * 2 * Stage::KV;
                    const uint4 a0 = *reinterpret_cast<const uint4*>(ks + Stage::at(g, c));
                    const uint4 a1 = *reinterpret_cast<const uint4*>(ks + Stage::at(g + 8, c));
                    lo[u][0] = a0.x; lo[u][1] = a0.y; lo[u][2] = a0.z; lo[u][3] = a0.w;
                    hi[u][0] = a1.x; hi[u][1] = a1.y; hi[u][2] = a1.z; hi[u][3] = a1.w;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    uint32_t f[TILES][4];
#pragma unroll
                    for (int u = 0; u < TILES; ++u) {
                        e4m3x4_to_half2(lo[u][y], f[u][0], f[u][2]);
                        e4m3x4_to_half2(hi[u][y], f[u][1], f[u][3]);
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint2 q = q_frag(j, 4 * i + y);
#pragma unroll
                        for (int u = 0; u < TILES; ++u) mma_f16(sc[u][j], f[u], q.x, q.y);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < KK / 2; ++i) {
                const int c = 2 * t + (i & 1) + 8 * (i >> 1);
                const uint4 a0 = *reinterpret_cast<const uint4*>(sb + Stage::at(g, c));
                const uint4 a1 = *reinterpret_cast<const uint4*>(sb + Stage::at(g + 8, c));
                const uint32_t f0[4] = {a0.x, a1.x, a0.y, a1.y}, f1[4] = {a0.z, a1.z, a0.w, a1.w};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint2 q0 = q_frag(j, 2 * i), q1 = q_frag(j, 2 * i + 1);
                    mma_bf16(sc[0][j], f0, q0.x, q0.y);
                    mma_bf16(sc[0][j], f1, q1.x, q1.y);
                }
            }
        }
        // ---- softmax: this lane has keys g (x = 0, 1) and g + 8 (x = 2, 3) of rows 2t, 2t + 1 ----
        float kf[TILES][2], ve[TILES][2];
#pragma unroll
        for (int u = 0; u < TILES; ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                kf[u][y] = 1.f;
                ve[u][y] = 0.f;
                if constexpr (FP8) {
                    const uint8_t* ss = sb + Stage::SCALES + u * 32 + g + 8 * y;
                    kf[u][y] = scale_value(ss[0]);
                    ve[u][y] = (float)((int)ss[16] - 127);
                }
            }
        // Exponents against the rows' references: sc - m for the sum, and for the e4m3 weights
        // (which carry the value's 2^ve) sc + ve - mv.  `arg` turns raw scores into them.
        float ew[TILES][NT][4];
        (void)ew;
        auto arg = [&](int j) {
#pragma unroll
            for (int u = 0; u < TILES; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if constexpr (FP8) {
                        const float f = qs[j][x & 1] * kf[u][x >> 1];
                        ew[u][j][x] = fmaf(sc[u][j][x], f, ve[u][x >> 1] - mv[j][x & 1]);
                        sc[u][j][x] = fmaf(sc[u][j][x], f, -m[j][x & 1]);
                    } else {
                        sc[u][j][x] = fmaf(sc[u][j][x], qs[j][x & 1], -m[j][x & 1]);
                    }
                }
        };
        float top = -INFINITY, topv = -INFINITY;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            arg(j);
            // keys that a row does not see weigh 0 (rows that do not exist may see them)
            if (!(meta.y & 4)) {
#pragma unroll
                for (int u = 0; u < TILES; ++u)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t seen = seen_keys(key0[u], pos[j][x], p.window, p.sinks) &
                                              ((uint32_t)meta.z >> (16 * u));
                        if (!((seen >> g) & 1)) sc[u][j][x] = ew[u][j][x] = -INFINITY;
                        if (!((seen >> (g + 8)) & 1)) sc[u][j][2 + x] = ew[u][j][2 + x] = -INFINITY;
                    }
            }
#pragma unroll
            for (int u = 0; u < TILES; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    top = fmaxf(top, sc[u][j][x]);
                    if constexpr (FP8) topv = fmaxf(topv, ew[u][j][x]);
                }
        }
        // lazy rescaling, as in attn_warp.cuh: the references move only when some exponent is
        // more than kRescaleSlack above them, and when a row sees its first keys
        if (__any_sync(0xffffffffu, top > kRescaleSlack || topv > kWeightTop + kRescaleSlack || unset != 0)) {
            gap = -INFINITY;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float up = -INFINITY, upv = -INFINITY;   // how far the references move
#pragma unroll
                    for (int u = 0; u < TILES; ++u) {
                        up = fmaxf(up, fmaxf(sc[u][j][x], sc[u][j][2 + x]));
                        if constexpr (FP8) upv = fmaxf(upv, fmaxf(ew[u][j][x], ew[u][j][2 + x]));
                    }
                    up = max_over_keys(up);
                    upv = FP8 ? max_over_keys(upv) - kWeightTop : up;
                    const uint32_t bit = 1u << (2 * j + x);
                    const bool fresh = (unset & bit) != 0, some = up > -INFINITY;
                    if (!fresh) {
                        up = fmaxf(up, 0.f);
                        upv = fmaxf(upv, 0.f);
                    }
                    if (!some) up = upv = 0.f;
                    else unset &= ~bit;
                    m[j][x] += up;
                    mv[j][x] += upv;
                    if (pos[j][x] >= 0 && !(unset & bit)) gap = fmaxf(gap, mv[j][x] - m[j][x]);
                    const float al = fresh ? 1.f : fast_exp2(-up), ao = fresh ? 1.f : fast_exp2(-upv);
                    l[j][x] *= al;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[j][i][x] *= ao;
                        o[j][i][2 + x] *= ao;
                    }
#pragma unroll
                    for (int u = 0; u < TILES; ++u)
#pragma unroll
                        for (int y = 0; y < 4; y += 2) {
                            sc[u][j][x + y] -= up;
                            if constexpr (FP8) ew[u][j][x + y] -= upv;
                        }
                }
        }
        uint32_t ph[TILES][NT][2], pl[TILES][NT][2];
        (void)pl;
        if constexpr (FP8) {
            // keys whose scale lies so far below the rows' that fp16 weights would lose them (see the top)
            bool small = false;
#pragma unroll
            for (int u = 0; u < TILES; ++u) small = small || fminf(ve[u][0], ve[u][1]) < gap;
            if (__any_sync(0xffffffffu, small)) {
                // (a key that no row sees, or whose weight is 0, does not count)
                float most = -INFINITY;
#pragma unroll
                for (int u = 0; u < TILES; ++u)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (ve[u][x >> 1] < gap) most = fmaxf(most, sc[u][j][x]);
                if (__any_sync(0xffffffffu, most > -126.f)) {
                    add_float32(sb, sc, ew);
                    return;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                float w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float e = fast_exp2(sc[u][j][x]);
                    l[j][x & 1] += e;
                    w[x] = FP8 ? fast_exp2(ew[u][j][x]) : e;
                }
                if constexpr (FP8) {
                    ph[u][j][0] = transpose8x8(pack_half2(w[0], w[1]));
                    ph[u][j][1] = transpose8x8(pack_half2(w[2], w[3]));
                } else {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        // the upper halves, and what is left plus 2^-24 of them: never 0 or of the other
                        // sign beside a weight, so that an infinite value stays one
                        constexpr float kRest = 1.f - 0x1p-24f;
                        const uint32_t h = __byte_perm(__float_as_uint(w[2 * y]), __float_as_uint(w[2 * y + 1]), 0x7632);
                        ph[u][j][y] = transpose8x8(h);
                        pl[u][j][y] = transpose8x8(pack_bf16x2(fmaf(-bf16_lo(h), kRest, w[2 * y]),
                                                               fmaf(-bf16_hi(h), kRest, w[2 * y + 1])));
                    }
                }
            }
        // ---- O^T += V^T P^T ----
        if constexpr (FP8) {
            constexpr int N = D / 8;   // dims of this lane: g * N ..
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                const uint8_t* vs = sb + u * 2 * Stage::KV + Stage::KV;
                uint32_t v[4][N / 4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int r = 2 * t + (y & 1) + 8 * (y >> 1);
                    if constexpr (N == 16) {
                        const uint4 w = *reinterpret_cast<const uint4*>(vs + Stage::at(r, g));
                        v[y][0] = w.x; v[y][1] = w.y; v[y][2] = w.z; v[y][3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(vs + Stage::at(r, g >> 1) + (g & 1) * 8);
                        v[y][0] = w.x; v[y][1] = w.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    // dims 2 i, 2 i + 1 of the four keys: (key 2t, key 2t + 1) pairs, then 2t + 8, 2t + 9
                    const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                    uint32_t f[4];
                    e4m3x4_to_half2(__byte_perm(v[0][i / 2], v[1][i / 2], sel), f[0], f[1]);
                    e4m3x4_to_half2(__byte_perm(v[2][i / 2], v[3][i / 2], sel), f[2], f[3]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma_f16(o[j][i], f, ph[u][j][0], ph[u][j][1]);
                }
            }
        } else {
            const int r = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t f[4];
                ldmatrix4_trans(f, sa + Stage::KV + Stage::at(r, 2 * i + ((lane >> 3) & 1)));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma_bf16(o[j][i], f, ph[0][j][0], ph[0][j][1]);
                    mma_bf16(o[j][i], f, pl[0][j][0], pl[0][j][1]);
                }
            }
        }
    };

    // The descriptions of items that are in the ring but not started yet wait in shared memory
    // beside it: at most STAGES of them, one per stage.
    int4* queue = reinterpret_cast<int4*>(smem + (size_t)kRowWarps * STAGES * Stage::BYTES) + warp * STAGES * 3;
    int q_in = 0, q_out = 0;
    auto push = [&]() {   // the item that fetch() just took
        if (it_valid && lane == 0) {
            queue[3 * q_in] = it_a;
            queue[3 * q_in + 1] = it_b;
            queue[3 * q_in + 2] = make_int4(it_hk, 0, 0, 0);
        }
        q_in = q_in + 1 == STAGES ? 0 : q_in + 1;
    };

    fetch();
    int cs = 0, is = 0;
    auto step_issue = [&]() {
        if (it_valid && it_v == it_b.y) push();
        issue(is);
        is = is + 1 == STAGES ? 0 : is + 1;
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) step_issue();
    while (true) {
        cp_async_wait<STAGES - 2>();
        __syncwarp();
        step_issue();
        const int4 meta = *reinterpret_cast<const int4*>(wsm + cs * Stage::BYTES + Stage::META);
        if (meta.x == -1) break;
        if (meta.y & 1) {
            start(queue[3 * q_out], queue[3 * q_out + 1], queue[3 * q_out + 2].x);
            q_out = q_out + 1 == STAGES ? 0 : q_out + 1;
        }
        if (meta.x >= 0) consume(cs, meta);
        if (meta.y & 2) epilogue();
        cs = cs + 1 == STAGES ? 0 : cs + 1;
    }
    cp_async_wait<0>();
    pdl_launch_dependents();
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
template <int D, bool FP8, int NT>
constexpr int row_smem() {
    return kRowWarps * (kRowStages * (RowStage<D, FP8, NT>::BYTES + 48) + RowStage<D, FP8, NT>::Q_BYTES);
}

template <int D, bool FP8, int NT>
cudaError_t launch_rows(const RowParams& p, long long max_items, cudaStream_t stream) {
    static std::once_flag once[64];
    static int per_sm[64];
    int dev = 0;
    cudaGetDevice(&dev);
    dev &= 63;
    auto kern = row_attention_kernel<D, FP8, NT>;
    constexpr int smem = row_smem<D, FP8, NT>();
    std::call_once(once[dev], [&] {
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kRowWarps * 32, smem) != cudaSuccess) n = 1;
        per_sm[dev] = std::max(1, n);
    });
    const long long want = (max_items + kRowWarps - 1) / kRowWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max(1LL, std::min<long long>((long long)device_sm_count() * per_sm[dev], want)));
    cfg.blockDim = dim3(kRowWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.planned ? 1 : 0;   // behind its plan kernel
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

struct RowGeometry {
    int nt, chunk, s_max;
    size_t counter, nsplit, items, lse_part, o_part, total;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// 16-key tiles per partition, from host-side bounds only (a captured call keeps its launches and
// its workspace, and a sequence's partitions do not depend on the others' lengths).  `pairs`
// sequences times KV heads see `seen` tiles each at most.
//  - Up to a quarter as many pairs as warps: as many partitions as keep every item in one round,
//    less a twelfth for lengths that the host does not know (8 contexts of 32 k keys in 8 bits: 24
//    partitions each 107 us, 27 109, 30, where a second round begins, 146, 64 124; 40 of 4 k: 5
//    69 us, 4 75, 8 83, 12 82; 40 of 0.5 to 4 k: 5 53 us, 12 60).
//  - More: 22 tiles, many rounds of items whose varying lengths even the rounds out (64 contexts
//    of 0.5 to 4 k keys: 73 us; 28 tiles 77, 18 tiles 80, 37 tiles 84; 56: 67 us, 3 partitions
//    75).
// Four tiles at least: shorter items cost more than the warps they fill; and up to 8 tiles stay
// whole, since that saves the combine and a chunk's plan (one context of 128 keys 13.7 us, two
// partitions 14.7; 4 chunks of 5 tokens at 128 keys 17.5 and 20.1, at 256 keys 23.4 and 20.1).
//
// Warps that a B200 holds at head_dim 128: 3 CTAs per SM for 8 rows and 2 for more.  (At head_dim 64
// the register file has room for 4, and 3 with 16 e4m3 rows, so that "one round" leaves some of the
// warps idle there; partitions for them have not been measured.)
constexpr long long row_resident_warps(int nt) { return 148LL * kRowWarps * (nt == 1 ? 3 : 2); }
int row_chunk_tiles(long long pairs, long long seen, int nt, int num_splits) {
    if (num_splits > 0) return (int)std::max(1LL, (seen + num_splits - 1) / num_splits);
    const long long warps = row_resident_warps(nt);
    if (seen <= 8) return (int)seen;
    long long chunk = 22;
    const long long parts = warps * 11 / 12 / std::max(1LL, pairs);
    if (parts >= 4) {
        chunk = std::max(4LL, (seen + parts - 1) / parts);
    }
    return (int)std::min(chunk, seen);
}

RowGeometry row_geometry(int batch, int total_q, int max_q, int hq, int hkv, int head_dim, int max_ctx,
                         int window, int sinks, int num_splits) {
    RowGeometry r{};
    const int rows = max_q * std::max(1, hq / hkv);   // of a KV head: at most 24, longer chunks go to the tiles
    r.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 3;
    // 16-key tiles that a sequence's tokens can see
    long long seen = ((long long)std::max(0, max_ctx) + kTileKeys - 1) / kTileKeys;
    if (window > 0)
        seen = std::min(seen, ((long long)window + std::max(1, max_q) + kTileKeys - 2) / kTileKeys + 1 +
                                  ((long long)sinks + kTileKeys - 1) / kTileKeys);
    seen = std::max(1LL, seen);
    r.chunk = row_chunk_tiles((long long)batch * hkv, seen, r.nt, num_splits);
    // the partition index travels in 15 bits
    r.chunk = (int)std::max<long long>(r.chunk, (seen + 32766) / 32767);
    r.s_max = (int)((seen + r.chunk - 1) / r.chunk);
    size_t off = 256;
    r.counter = 0;
    r.nsplit = off; off = align256(off + sizeof(int32_t) * (size_t)total_q);
    r.items = off; off = align256(off + 2 * sizeof(int4) * (size_t)batch * r.s_max);
    r.lse_part = off; off = align256(off + (r.s_max > 1 ? sizeof(float) * (size_t)total_q * hq * r.s_max : 0));
    r.o_part = off; off = align256(off + (r.s_max > 1 ? sizeof(float) * (size_t)total_q * hq * r.s_max * head_dim : 0));
    r.total = off;
    return r;
}

}  // namespace

size_t row_attention_workspace_bytes(int batch, int total_q, int max_q, int hq, int hkv, int head_dim,
                                     int max_ctx, int window, int sinks, int num_splits) {
    return row_geometry(batch, total_q, max_q, hq, hkv, head_dim, max_ctx, window, sinks, num_splits).total;
}

nvpa_status_t run_row_attention(const WindowCall& c, cudaStream_t stream) {
    const RowGeometry r = row_geometry(c.batch, c.total_q, c.max_seqlen_q, c.hq, c.hkv, c.head_dim,
                                       c.max_context_len, c.window, c.num_sinks, c.num_splits);
    if (c.workspace_bytes < r.total) {
        set_error("workspace too small: %zu bytes given, %zu needed", c.workspace_bytes, r.total);
        return NVPA_ERR_WORKSPACE_TOO_SMALL;
    }
    const long long max_items = (long long)c.batch * r.s_max * c.hkv;
    if (max_items > 0x7fffffffLL / 2) {
        set_error("more than 2^30 work items");
        return NVPA_ERR_UNSUPPORTED;
    }
    uint8_t* ws = static_cast<uint8_t*>(c.workspace);
    RowParams p{};
    p.q = static_cast<const uint16_t*>(c.q);
    p.k_cache = c.k_cache;
    p.v_cache = c.v_cache;
    p.k_scales = c.k_scales;
    p.v_scales = c.v_scales;
    p.block_tables = c.block_tables;
    p.context_lens = c.context_lens;
    p.cu_q = c.cu_seqlens_q;
    p.out = static_cast<uint16_t*>(c.out);
    p.lse_out = c.lse_out;
    p.counter = reinterpret_cast<int32_t*>(ws + r.counter);
    p.nsplit = reinterpret_cast<int32_t*>(ws + r.nsplit);
    p.items = reinterpret_cast<int4*>(ws + r.items);
    p.lse_part = reinterpret_cast<float*>(ws + r.lse_part);
    p.o_part = reinterpret_cast<float*>(ws + r.o_part);
    p.err = c.err_flag;
    p.batch = c.batch;
    p.total_q = c.total_q;
    p.max_q = c.max_seqlen_q;
    p.hq = c.hq;
    p.hkv = c.hkv;
    p.group = c.hq / c.hkv;
    p.max_blocks = c.max_blocks_per_seq;
    p.num_blocks = c.num_blocks;
    p.block_size = c.block_size;
    p.block_shift = __builtin_ctz((unsigned)c.block_size);
    p.max_ctx = c.max_context_len;
    // (a window as long as the longest context hides nothing)
    p.window = c.window >= c.max_context_len ? 0 : c.window;
    p.sinks = std::min(c.num_sinks, c.max_context_len);
    p.max_entries = c.batch * r.s_max;
    p.planned = c.batch > kRowWarps * 32 || max_items > row_resident_warps(r.nt);
    p.chunk = r.chunk;
    p.s_max = r.s_max;
    p.scale_log2 = c.scale * kLog2e;
    cudaError_t e = cudaSuccess;
    if (p.planned) {
        // (its time is barriers and load latency: fewer warps where they suffice, 0.4 us)
        row_plan_kernel<<<1, c.batch <= 256 ? 256 : 1024, 0, stream>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_failure(e, "row attention plan launch");
        count_launches(1);
    } else if (c.cu_seqlens_q != nullptr && r.s_max > 1) {
        // rows that no sequence owns have no partitions (the workers write the others' counts)
        e = cudaMemsetAsync(p.nsplit, 0, sizeof(int32_t) * (size_t)c.total_q, stream);
        if (e != cudaSuccess) return cuda_failure(e, "row attention memset");
    }
    const bool fp8 = c.k_scales != nullptr;
    e = cudaErrorInvalidValue;
#define NVPA_CASE(DD, FF, NN) \
    if (c.head_dim == DD && fp8 == FF && r.nt == NN) e = launch_rows<DD, FF, NN>(p, max_items, stream);
    NVPA_CASE(128, false, 1) NVPA_CASE(128, false, 2) NVPA_CASE(128, true, 1) NVPA_CASE(128, true, 2)
    NVPA_CASE(64, false, 1) NVPA_CASE(64, false, 2) NVPA_CASE(64, true, 1) NVPA_CASE(64, true, 2)
    NVPA_CASE(128, true, 3) NVPA_CASE(64, true, 3)   // (bf16: up to 16 rows)
#undef NVPA_CASE
    if (e != cudaSuccess) return cuda_failure(e, "row attention launch");
    if (r.s_max > 1) {
        AttnParams cp{};
        cp.out = p.out;
        cp.lse_out = p.lse_out;
        cp.o_part = p.o_part;
        cp.lse_part = p.lse_part;
        cp.nsplit = p.nsplit;
        cp.batch = c.total_q;
        cp.hq = c.hq;
        cp.s_max = r.s_max;
        e = launch_decode_combine(cp, c.head_dim, stream);
        if (e != cudaSuccess) return cuda_failure(e, "row attention combine launch");
        count_launches(1);
    }
    return NVPA_OK;
}

}  // namespace nvpa
