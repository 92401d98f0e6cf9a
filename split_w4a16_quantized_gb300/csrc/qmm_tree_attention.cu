// Attention of drafted token trees over the paged KV cache
// (qmm_tree_attention).
//
//   O[i, h] = sum_l p_l V[l, h / QG],  p = softmax over the visible l of
//             scale * q[i, h] . K[l, h / QG]
//
// Token i sees every slot below lens[b], and slot lens[b] + j where j is i or
// one of its ancestors.  The QG query heads of a KV head and the n tokens of a
// sequence are the R = n QG rows of one product with that head's keys, so each
// K and V row is read once for all of them: R flop per byte of a BF16 cache,
// HBM-bound up to a few hundred rows.
//
// Work split.  A work item is (sequence b, KV head g, tile of kRows rows), of
// ceil(L_b / 64) tiles of 64 positions, L_b = lens[b] + n_b.  Lengths live on
// the device and differ widely in a batch, so the grid does not know them: it
// is a fixed number of CTAs, and the tiles of all items, laid end to end, are
// cut into that many equal runs.  Each CTA sums the batch's tile counts, finds
// its run and walks it; the copies run ahead across item borders.  An item
// inside one run is written to O.  An item that a border cuts leaves a partial
// softmax state (maximum, sum, unnormalized output, FP32) per run, at most two
// a CTA, and the merge kernel adds them in run order: the bits do not depend
// on timing.  Equal runs keep every SM busy to the end whatever the lengths,
// and the workspace is two states per CTA whatever the batch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"
#include "qmm_paged.cuh"
#include "qmm_sm100.cuh"

namespace qmm {

// Tiled tensor map helper (qmm_w4a16_tc.cu)
bool encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* ptr,
                  const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                  CUtensorMapSwizzle swizzle);

namespace {

constexpr int kTile = 64;      // positions per tile
constexpr int kRows = 16;      // query rows per work item
constexpr int kWarps = 4;      // compute warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kKeys = kTile / kWarps;   // positions per compute warp
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
constexpr int kMinRun = 2;     // tiles of the shortest run
constexpr int kWords = kMaxTree / 32;

struct TreeParams {
    PagedDims d;
    const __nv_bfloat16* q;
    __nv_bfloat16* O;
    const int *cu, *parents;
    float* ws;    // partial states: m [2 ctas][kRows], l the same, o [2 ctas][kRows][D]
    int* status;
    int64_t q_stride;
    int N, T, Hq, QG, ctas;
    int box_shift;   // log2 of the positions of one copy: min(page, tile)
    float qscale;    // scale * log2(e) * k_scale
    float vscale;
};

// ---- work split ----------------------------------------------------------------

struct Seq {
    int first, n;      // its rows of q
    int len, total;    // cached tokens; with the new ones
    int tiles;         // of 64 positions
    int row_tiles;
};

__device__ __forceinline__ Seq sequence(const TreeParams& p, int b) {
    Seq s;
    token_range(p.cu, p.N, p.T, b, &s.first, &s.n);
    s.len = cached_tokens(p.d, b);
    s.total = s.len + s.n < p.d.cap ? s.len + s.n : p.d.cap;
    s.tiles = (s.total + kTile - 1) / kTile;
    s.row_tiles = (s.n * p.QG + kRows - 1) / kRows;
    return s;
}
__device__ __forceinline__ long long tiles_of(const TreeParams& p, const Seq& s) {
    return static_cast<long long>(s.tiles) * s.row_tiles * p.d.Hkv;
}

// Sum of v over the block and over the threads before this one.  Every thread
// of the block calls it; red is kThreads / 32 values of shared memory.
template <int kN>
__device__ __forceinline__ long long block_scan(long long v, long long* red, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kN / 32; ++w) {
        if (w < warp) before += red[w];
        all += red[w];
    }
    *total = all;
    return before + x - v;
}

__device__ __forceinline__ long long run_length(const TreeParams& p, long long all) {
    const long long r = (all + p.ctas - 1) / p.ctas;
    return r < kMinRun ? kMinRun : r;
}

// A CTA's place in the list of tiles.
struct Run {
    int b;            // sequence
    long long at;     // tile within the sequence's list
    long long left;   // tiles of the run still to do
};

// The CTA's run: whole block; sh: shared scratch.
struct RunShared {
    long long red[kThreads / 32];
    long long at;
    int b;
};
__device__ __forceinline__ Run find_run(const TreeParams& p, RunShared& sh) {
    const int per = (p.d.B + kThreads - 1) / kThreads;
    const int b0 = min(p.d.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.d.B, b0 + per);
    long long mine = 0, all;
    for (int b = b0; b < b1; ++b) mine += tiles_of(p, sequence(p, b));
    if (threadIdx.x == 0) sh.b = -1;
    const long long before = block_scan<kThreads>(mine, sh.red, &all);
    const long long len = run_length(p, all);
    const long long start = len * blockIdx.x;
    if (start >= before && start < before + mine) {
        // this thread's sequences hold the start
        long long at = start - before;
        for (int b = b0; b < b1; ++b) {
            const long long t = tiles_of(p, sequence(p, b));
            if (at < t) {
                sh.b = b;
                sh.at = at;
                break;
            }
            at -= t;
        }
    }
    __syncthreads();
    Run r;
    r.b = sh.b;
    r.at = sh.at;
    r.left = r.b < 0 ? 0 : (all - start < len ? all - start : len);
    return r;
}

// The next stretch of one work item in the run.
struct Stretch {
    Seq s;
    int b, g, row0;    // sequence, KV head, first row
    int t0, t1;        // tiles
};
__device__ __forceinline__ bool next_stretch(const TreeParams& p, Run& r, Stretch* x) {
    if (r.left <= 0) return false;
    x->s = sequence(p, r.b);
    while (r.at >= tiles_of(p, x->s)) {
        r.at -= tiles_of(p, x->s);
        if (++r.b >= p.d.B) return false;   // (not reached: the run ends with the list)
        x->s = sequence(p, r.b);
    }
    const int item = static_cast<int>(r.at / x->s.tiles);
    x->b = r.b;
    x->g = item / x->s.row_tiles;
    x->row0 = (item % x->s.row_tiles) * kRows;
    x->t0 = static_cast<int>(r.at % x->s.tiles);
    const long long end = x->t0 + r.left;
    x->t1 = end < x->s.tiles ? static_cast<int>(end) : x->s.tiles;
    r.at += x->t1 - x->t0;
    r.left -= x->t1 - x->t0;
    return true;
}

// ---- shared memory tiles ----------------------------------------------------

template <int D, bool kFp8>
struct Cfg {
    static constexpr int ROW = D * (kFp8 ? 1 : 2);          // bytes of a cache row
    static constexpr int BOX = ROW < 128 ? ROW : 128;       // row bytes of one copy
    static constexpr int BOXES = ROW / BOX;
    static constexpr int TILE = kTile * ROW;                // one K (or V) tile
    static constexpr int STAGE = 2 * TILE;
    static constexpr int KS = D / 16;                       // k-steps of Q K^T
    static constexpr int NB = D / 8;                        // n-blocks of P V
    // Byte offset of 16-byte chunk c of row r: boxes of kTile rows, the chunk
    // index permuted by the copy's swizzle (128-byte rows: with r mod 8;
    // 64-byte rows: with (r / 2) mod 4).
    static __device__ __forceinline__ uint32_t off(int r, int c) {
        if (BOX == 128)
            return static_cast<uint32_t>((c >> 3) * (kTile * 128) + r * 128 +
                                         (((c & 7) ^ (r & 7)) << 4));
        return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    }
};

template <int D>
struct Smem {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    int have[kStages];                 // pages of the stage's tile that exist, one bit a copy
    float wm[kWarps][kRows];
    float wl[kWarps][kRows];
    uint32_t anc[kRows][kWords];       // ancestors (and self) of each row's token
    int16_t par[kMaxTree];
    RunShared run;
    alignas(16) float ex[kWarps][kRows][D / kWarps];   // outputs on their way to another warp
};

// 4-D tile load (c0 innermost), completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_t(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// d += a * b, m16n8k16, FP32 accumulate, F16 or BF16 operands.
template <bool kF16>
__device__ __forceinline__ void mma16816(float d[4], const uint32_t a[4], uint32_t b0,
                                         uint32_t b1) {
    if (kF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        mma_bf16_16816(d, a, b0, b1);
}

// Two E4M3 numbers (the low 16 bits) as an F16 pair; every E4M3 number is an F16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
    return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Maximum that every later exp2 can subtract: 0 while nothing is visible.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// ---- the kernel -------------------------------------------------------------
//
// CTA: 4 compute warps and one copy warp, as the contiguous decode kernel.
//   - The copy warp loads tiles of 64 positions into a 3-stage ring, one 4-D
//     copy per page piece and 128-byte column block, each by its own lane.  A
//     lane looks up one table entry of the next 32 pieces at a time.  A
//     missing page (or a piece past the last position) is copied from outside
//     the map, which fills zeros; the stage's bits tell the compute warps.
//   - Compute warp w takes positions 16w .. 16w+15 of a tile and keeps its own
//     softmax state; scores in log2 units, exp2.
//   - BF16 cache: BF16 products, P as two BF16 terms (hi + lo), about 16 bits.
//     E4M3 cache: the values are exact in F16, so the products run in F16; a
//     row of q is scaled by a power of two to a maximum in [1, 2) first, so
//     rounding it to F16 (11 bits, 2^-25 absolute) loses nothing of its 8 bits
//     but what lies 2^-17 below the row's maximum, and P is one F16 term.
//   - When a stretch ends the 4 states are merged: each warp collects a quarter
//     of the columns from the other three.
// Every wait is bounded (1 s): a wait that runs out sets the status word and
// the CTA winds down after its copies in flight have landed.
template <int D, bool kFp8, bool kHalf>   // kHalf: at most 8 rows are in use
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    tree_attn_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ TreeParams p) {
    using C = Cfg<D, kFp8>;
    constexpr int KS = C::KS, NB = C::NB, NQ = NB / kWarps;
    constexpr int H = kHalf ? 1 : 2;   // row halves: rows gr and gr + 8
    extern __shared__ uint8_t tree_smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(tree_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(ring + kStages * C::STAGE);
    __shared__ int abort_flag;
    volatile int* abort = &abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_trigger();
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], kWarps);
        }
        mbar_fence_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    pdl_wait();
    __syncthreads();
    Run run = find_run(p, sm.run);
    const int box = 1 << p.box_shift;            // positions of one copy
    const int pieces = kTile >> p.box_shift;     // copies of a tile, per column block and pool
    Stretch x;

    if (warp == kWarps) {
        // ---- copy warp ----
        const uint32_t ring_a = smem_addr(ring);
        // this lane's copy of a tile: piece, K or V, column block
        const int my_piece = lane / (2 * C::BOXES), my_rest = lane % (2 * C::BOXES);
        const int my_pool = my_rest / C::BOXES, my_box = my_rest % C::BOXES;
        // (8 pieces x 4 copies fill the 32 lanes exactly)
        const bool copies = my_piece < pieces;
        const uint32_t my_off = my_pool * C::TILE + my_box * (kTile * C::BOX) +
                                (my_piece << p.box_shift) * C::BOX;
        int it = 0;   // tiles copied so far
        while (next_stretch(p, run, &x)) {
            // table entries of 32 pieces, and of the 32 after them
            const int c_end = (x.s.total + box - 1) >> p.box_shift;   // pieces that hold positions
            const int* row = p.d.table + static_cast<int64_t>(x.b) * p.d.max_pages;
            auto entry = [&](int c) {
                return c < c_end ? row[(c << p.box_shift) >> p.d.page_shift] : -1;
            };
            int c0 = x.t0 * pieces;
            int cur = entry(c0 + lane), nxt = entry(c0 + 32 + lane);
            for (int t = x.t0; t < x.t1; ++t, ++it) {
                if (t * pieces >= c0 + 32) {
                    c0 += 32;
                    cur = nxt;
                    nxt = entry(c0 + 32 + lane);
                }
                const int st = it % kStages;
                if (it >= kStages &&
                    !mbar_wait_warp(&sm.empty[st], ((it / kStages) & 1) ^ 1, abort, p.status))
                    break;
                const int at = t * pieces - c0;
                const uint32_t ok = __ballot_sync(0xffffffffu, cur >= 0 && cur < p.d.num_pages);
                const int page = __shfl_sync(0xffffffffu, cur, (at + my_piece) & 31);
                if (lane == 0) {
                    sm.have[st] = static_cast<int>((ok >> at) & ((1u << pieces) - 1u));
                    mbar_arrive_expect_tx(&sm.full[st], C::STAGE);
                }
                __syncwarp();
                if (copies) {
                    // the compute warps read (and may have zeroed) the stage
                    // with ordinary accesses
                    fence_proxy_async_smem();
                    const int pos = (t * kTile) + (my_piece << p.box_shift);
                    const bool real = (ok >> (at + my_piece)) & 1u;
                    tma_load_4d(ring_a + st * C::STAGE + my_off, my_pool ? &vmap : &kmap,
                                &sm.full[st], my_box * (C::BOX / (kFp8 ? 1 : 2)),
                                pos & ((1 << p.d.page_shift) - 1), x.g,
                                real ? page : p.d.num_pages);
                }
            }
            if (*abort) break;
        }
        if (*abort && lane == 0) {  // let the copies in flight land before the CTA exits
            for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
                mbar_wait(&sm.full[j % kStages], (j / kStages) & 1, nullptr, p.status);
        }
    } else {
        // ---- compute warps ----
        const int gr = lane >> 2, tq = lane & 3;   // fragment row, column pair
        const uint32_t ring_a = smem_addr(ring);
        const int mj = lane >> 3, mr = lane & 7;   // ldmatrix: matrix, row
        const int kb = warp * kKeys;               // the warp's first position in a tile
        int it = 0;
        while (next_stretch(p, run, &x)) {
            const int rows = min(kRows, x.s.n * p.QG - x.row0);
            // ---- ancestors of the rows' tokens, where the stretch reaches the
            // drafted slots; a chain needs none ----
            int node[H];
#pragma unroll
            for (int h = 0; h < H; ++h) node[h] = (x.row0 + min(gr + 8 * h, rows - 1)) / p.QG;
            if (p.parents && x.t1 * kTile > x.s.len) {
                for (int i = tid; i < x.s.n; i += 32 * kWarps) {
                    const int v = p.parents[x.s.first + i];
                    sm.par[i] = static_cast<int16_t>(v >= 0 && v < i ? v : -1);
                }
                named_bar_sync(1, 32 * kWarps);
                if (tid < rows) {
                    uint32_t w[kWords];
#pragma unroll
                    for (int j = 0; j < kWords; ++j) w[j] = 0;
                    for (int i = (x.row0 + tid) / p.QG; i >= 0; i = sm.par[i]) {
#pragma unroll
                        for (int j = 0; j < kWords; ++j)
                            if (j == i >> 5) w[j] |= 1u << (i & 31);
                    }
#pragma unroll
                    for (int j = 0; j < kWords; ++j) sm.anc[tid][j] = w[j];
                }
                named_bar_sync(1, 32 * kWarps);
            }
            // ---- A operand of S: rows of q, k = head dims ----
            // E4M3: dims 4 tq .. 4 tq + 3 of each 16 take the fragment's two
            // column pairs, as the 8-bit keys' loads lay them out.
            uint32_t qa[KS][2 * H];
            float qs[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int r = x.row0 + gr + 8 * h;
                const bool on = gr + 8 * h < rows;
                const __nv_bfloat16* qv =
                    p.q + (on ? (x.s.first + r / p.QG) * p.q_stride + (x.g * p.QG + r % p.QG) * D : 0);
                float big = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t lo, hi;
                    if (kFp8) {
                        const uint2 v = *reinterpret_cast<const uint2*>(qv + ks * 16 + 4 * tq);
                        lo = v.x;
                        hi = v.y;
                    } else {
                        lo = *reinterpret_cast<const uint32_t*>(qv + ks * 16 + 2 * tq);
                        hi = *reinterpret_cast<const uint32_t*>(qv + ks * 16 + 8 + 2 * tq);
                    }
                    qa[ks][h] = on ? lo : 0u;
                    qa[ks][H + h] = on ? hi : 0u;
                    if (kFp8) {
                        const uint32_t a = lo & 0x7fff7fffu, c = hi & 0x7fff7fffu;
                        big = fmaxf(big, fmaxf(fmaxf(__uint_as_float(a << 16),
                                                     __uint_as_float(a & 0xffff0000u)),
                                               fmaxf(__uint_as_float(c << 16),
                                                     __uint_as_float(c & 0xffff0000u))));
                    }
                }
                qs[h] = p.qscale;
                if (kFp8) {
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    // 2^e <= big < 2^(e+1); a row of zeros, or one that holds
                    // infinities or NaN, is left as it is
                    int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
                    e = big > 0.f && e < 128 ? max(-126, min(126, e)) : 0;
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    qs[h] *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t v = qa[ks][i * H + h];
                            qa[ks][i * H + h] = pack_f16x2(__uint_as_float(v << 16) * down,
                                                           __uint_as_float(v & 0xffff0000u) * down);
                        }
                }
            }
            float o[NB][2 * H];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2 * H; ++i) o[nb][i] = 0.f;
            float m_run[H], l_run[H];   // l_run: this lane's share of the row's sum
#pragma unroll
            for (int h = 0; h < H; ++h) m_run[h] = -INFINITY, l_run[h] = 0.f;

            for (int t = x.t0; t < x.t1; ++t, ++it) {
                const int st = it % kStages;
                if (__any_sync(0xffffffffu, *abort) ||
                    !mbar_wait_warp(&sm.full[st], (it / kStages) & 1, abort, p.status))
                    break;
                const int pos0 = t * kTile + kb;             // the warp's first position
                const int valid = x.s.total - pos0;          // how many of its 16 exist
                if (valid > 0) {
                    const uint32_t kt = ring_a + st * C::STAGE, vt = kt + C::TILE;
                    const uint32_t have = static_cast<uint32_t>(sm.have[st]);
                    const bool plain = have == (1u << pieces) - 1u && pos0 + kKeys <= x.s.len;
                    if (valid < kKeys) {
                        // slots past the last position may hold anything, and
                        // 0 * NaN is not 0: their V rows become zeros
                        uint8_t* v = ring + st * C::STAGE + C::TILE;
                        for (int c = lane; c < (kKeys - valid) * (C::ROW / 16); c += 32)
                            *reinterpret_cast<uint4*>(v + C::off(kb + valid + c / (C::ROW / 16),
                                                                 c % (C::ROW / 16))) =
                                make_uint4(0, 0, 0, 0);
                        __syncwarp();
                    }
                    // S = Q K^T for the warp's 16 positions
                    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                    if (kFp8) {
                        // matrices: (positions j % 2, 16-dim step j / 2)
#pragma unroll
                        for (int k2 = 0; k2 < KS / 2; ++k2) {
                            uint32_t kf[4];
                            ldmatrix_x4(kf, kt + C::off(kb + (mj & 1) * 8 + mr, 2 * k2 + (mj >> 1)));
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int ks = 2 * k2 + i;
                                const uint32_t a[4] = {qa[ks][0], H == 2 ? qa[ks][H - 1] : 0u,
                                                       qa[ks][H], H == 2 ? qa[ks][2 * H - 1] : 0u};
#pragma unroll
                                for (int nb = 0; nb < 2; ++nb)
                                    mma16816<true>(sc[nb], a, e4m3x2_to_f16x2(kf[2 * i + nb] & 0xffffu),
                                                   e4m3x2_to_f16x2(kf[2 * i + nb] >> 16));
                            }
                        }
                    } else {
                        // matrices: (positions j / 2, dims j % 2)
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            uint32_t kf[4];
                            ldmatrix_x4(kf, kt + C::off(kb + (mj >> 1) * 8 + mr, 2 * ks + (mj & 1)));
                            const uint32_t a[4] = {qa[ks][0], H == 2 ? qa[ks][H - 1] : 0u, qa[ks][H],
                                                   H == 2 ? qa[ks][2 * H - 1] : 0u};
                            mma16816<false>(sc[0], a, kf[0], kf[1]);
                            mma16816<false>(sc[1], a, kf[2], kf[3]);
                        }
                    }
                    // online softmax of each row over the 16 positions
                    float pw[H][4], corr[H];
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = sc[e >> 1][2 * h + (e & 1)] * qs[h];
                        if (!plain) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int k = (e >> 1) * 8 + 2 * tq + (e & 1);
                                const int j = pos0 + k - x.s.len;   // drafted token, >= 0
                                bool see = k < valid && ((have >> ((kb + k) >> p.box_shift)) & 1u);
                                if (see && j >= 0)
                                    see = p.parents
                                              ? (sm.anc[min(gr + 8 * h, rows - 1)][j >> 5] >> (j & 31)) & 1u
                                              : j <= node[h];
                                if (!see) v[e] = -INFINITY;
                            }
                        }
                        float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const float mn = fmaxf(m_run[h], mx);
                        const float mf = finite_max(mn);
                        corr[h] = exp2f(m_run[h] - mf);
                        m_run[h] = mn;
                        float rs = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pw[h][e] = exp2f(v[e] - mf);
                            rs += pw[h][e];
                        }
                        l_run[h] = l_run[h] * corr[h] + rs;
                    }
                    // P as the A operand of P V (rows, k = positions)
                    uint32_t ph[4] = {0, 0, 0, 0}, pl[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float a = pw[h][2 * i], c = pw[h][2 * i + 1];
                            if (kFp8) {
                                ph[2 * i + h] = pack_f16x2(a, c);
                            } else {
                                const uint32_t w = pack_bf16x2(a, c);
                                ph[2 * i + h] = w;
                                pl[2 * i + h] = pack_bf16x2(a - __uint_as_float(w << 16),
                                                            c - __uint_as_float(w & 0xffff0000u));
                            }
                        }
                    // o = o * corr + P V
#pragma unroll
                    for (int db = 0; db < NB / 2; ++db) {
                        uint32_t vf[4];
                        if (kFp8) {
                            // matrices: (positions j % 2, 16-dim block j / 2); a
                            // register holds two positions x an (even, odd) pair
                            // of dims, which become two n-blocks
                            if (db % 2 == 0) {
                                uint32_t raw[4];
                                ldmatrix_x4_t(raw, vt + C::off(kb + (mj & 1) * 8 + mr, db + (mj >> 1)));
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint32_t a = __byte_perm(raw[2 * i], 0, 0x3120);
                                    const uint32_t c = __byte_perm(raw[2 * i + 1], 0, 0x3120);
                                    vf[0] = e4m3x2_to_f16x2(a & 0xffffu);
                                    vf[1] = e4m3x2_to_f16x2(c & 0xffffu);
                                    vf[2] = e4m3x2_to_f16x2(a >> 16);
                                    vf[3] = e4m3x2_to_f16x2(c >> 16);
#pragma unroll
                                    for (int n = 0; n < 2; ++n) {
                                        float* acc = o[2 * (db + i) + n];
                                        float d4[4] = {acc[0] * corr[0], acc[1] * corr[0],
                                                       H == 2 ? acc[2 * H - 2] * corr[H - 1] : 0.f,
                                                       H == 2 ? acc[2 * H - 1] * corr[H - 1] : 0.f};
                                        mma16816<true>(d4, ph, vf[2 * n], vf[2 * n + 1]);
#pragma unroll
                                        for (int q = 0; q < 2 * H; ++q) acc[q] = d4[q];
                                    }
                                }
                            }
                        } else {
                            // matrices: (positions j % 2, dims j / 2), transposed
                            ldmatrix_x4_t(vf, vt + C::off(kb + (mj & 1) * 8 + mr, 2 * db + (mj >> 1)));
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                float* acc = o[2 * db + n];
                                float d4[4] = {acc[0] * corr[0], acc[1] * corr[0],
                                               H == 2 ? acc[2 * H - 2] * corr[H - 1] : 0.f,
                                               H == 2 ? acc[2 * H - 1] * corr[H - 1] : 0.f};
                                mma16816<false>(d4, ph, vf[2 * n], vf[2 * n + 1]);
                                mma16816<false>(d4, pl, vf[2 * n], vf[2 * n + 1]);
#pragma unroll
                                for (int q = 0; q < 2 * H; ++q) acc[q] = d4[q];
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[st]);
            }

            // ---- merge the warps' states; warp w ends with columns
            // [w D/4, (w + 1) D/4) of every row ----
#pragma unroll
            for (int h = 0; h < H; ++h) {
                l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 1);
                l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 2);
                if (tq == 0) {
                    sm.wm[warp][gr + 8 * h] = m_run[h];
                    sm.wl[warp][gr + 8 * h] = l_run[h];
                }
            }
            named_bar_sync(1, 32 * kWarps);
            float M[H], den[H], fac[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                M[h] = -INFINITY;
                den[h] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M[h] = fmaxf(M[h], sm.wm[w][gr + 8 * h]);
                const float mf = finite_max(M[h]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    den[h] = fmaf(exp2f(sm.wm[w][gr + 8 * h] - mf), sm.wl[w][gr + 8 * h], den[h]);
                fac[h] = exp2f(m_run[h] - mf);
            }
            float acc[NQ][2 * H];
#pragma unroll
            for (int qq = 0; qq < kWarps; ++qq)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * H; ++i) {
                        o[qq * NQ + n][i] *= fac[i >> 1];
                        if (qq == warp) acc[n][i] = o[qq * NQ + n][i];
                    }
            // round i: warp w hands columns of warp (w + i) % 4 over
#pragma unroll
            for (int i = 1; i < kWarps; ++i) {
                const int to = (warp + i) % kWarps;
#pragma unroll
                for (int qq = 0; qq < kWarps; ++qq)
                    if (qq == to)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int h = 0; h < H; ++h)
                                *reinterpret_cast<float2*>(&sm.ex[to][gr + 8 * h][n * 8 + 2 * tq]) =
                                    make_float2(o[qq * NQ + n][2 * h], o[qq * NQ + n][2 * h + 1]);
                named_bar_sync(1, 32 * kWarps);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const float2 v =
                            *reinterpret_cast<const float2*>(&sm.ex[warp][gr + 8 * h][n * 8 + 2 * tq]);
                        acc[n][2 * h] += v.x;
                        acc[n][2 * h + 1] += v.y;
                    }
                named_bar_sync(1, 32 * kWarps);
            }
            // (the other warps may not have seen the flag yet: this one goes on to
            // the next stretch's barriers with them, and writes nothing)
            if (*abort) continue;
            // ---- O, or the partial state ----
            const bool whole = x.t0 == 0 && x.t1 == x.s.tiles;
            const int slot = 2 * blockIdx.x + (x.t0 == 0 ? 1 : 0);
            float* pm = p.ws + static_cast<size_t>(slot) * kRows;
            float* pl = pm + static_cast<size_t>(2) * p.ctas * kRows;
            float* po = p.ws + static_cast<size_t>(4) * p.ctas * kRows +
                        static_cast<size_t>(slot) * kRows * D;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int r = gr + 8 * h;
                if (r >= rows) continue;
                const float inv = whole ? (den[h] > 0.f ? p.vscale / den[h]
                                                        : (den[h] == 0.f ? 0.f : den[h]))
                                        : 1.f;
                if (!whole && warp == 0 && tq == 0) {
                    pm[r] = M[h];
                    pl[r] = den[h];
                }
                const int rr = x.row0 + r;
                __nv_bfloat16* out = p.O + (static_cast<int64_t>(x.s.first + rr / p.QG) * p.Hq +
                                            x.g * p.QG + rr % p.QG) * D;
#pragma unroll
                for (int n = 0; n < NQ; n += kFp8 ? 2 : 1) {
                    // columns: BF16 8 n + 2 tq + {0, 1}; E4M3 n-blocks 2i (even
                    // dims) and 2i + 1 (odd dims): 16 i + 4 tq + {0, 2}, {1, 3}
                    const int c = (warp * NQ + n) * 8 + (kFp8 ? 4 : 2) * tq;
                    if (kFp8) {
                        const int n1 = n + 1 < NQ ? n + 1 : n;
                        const float4 v = make_float4(acc[n][2 * h] * inv, acc[n1][2 * h] * inv,
                                                     acc[n][2 * h + 1] * inv, acc[n1][2 * h + 1] * inv);
                        if (whole)
                            *reinterpret_cast<uint2*>(out + c) =
                                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4*>(po + r * D + c) = v;
                    } else {
                        const float2 v = make_float2(acc[n][2 * h] * inv, acc[n][2 * h + 1] * inv);
                        if (whole)
                            *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(v.x, v.y);
                        else
                            *reinterpret_cast<float2*>(po + r * D + c) = v;
                    }
                }
            }
        }
    }
    __syncthreads();
}

// The items that a run border cuts: O = sum_c 2^(m_c - M) o_c / sum_c
// 2^(m_c - M) l_c over the runs c that hold a stretch, in ascending c.  One
// block per item; a block whose item lies in one run leaves at once.
constexpr int kMergeThreads = 128;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeParams p,
                                                                   int max_row_tiles) {
    __shared__ long long red[kMergeThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int rt = blockIdx.x % max_row_tiles, g = blockIdx.x / max_row_tiles, b = blockIdx.y;
    const Seq s = sequence(p, b);
    if (rt >= s.row_tiles) return;
    long long mine = 0, upto = 0, all, total;
    for (int i = threadIdx.x; i < p.d.B; i += kMergeThreads) {
        const long long t = tiles_of(p, sequence(p, i));
        mine += t;
        if (i < b) upto += t;
    }
    block_scan<kMergeThreads>(mine, red, &all);
    __syncthreads();
    block_scan<kMergeThreads>(upto, red, &total);
    const long long len = run_length(p, all);
    const long long start = total + (static_cast<long long>(g) * s.row_tiles + rt) * s.tiles;
    const int c0 = static_cast<int>(start / len), c1 = static_cast<int>((start + s.tiles - 1) / len);
    if (c0 == c1) return;
    const int rows = min(kRows, s.n * p.QG - rt * kRows);
    const float* pm = p.ws;
    const float* pl = pm + static_cast<size_t>(2) * p.ctas * kRows;
    const float* po = pl + static_cast<size_t>(2) * p.ctas * kRows;
    constexpr int V = D / 32;   // values per lane
    const int lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < rows; r += kMergeThreads / 32) {
        // run c's slot: its last stretch (1) where the item starts in it, else its first
        auto slot = [&](int c) {
            return static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * kRows + r;
        };
        float M = -INFINITY;
        for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, pm[slot(c)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        M = finite_max(M);
        float num[V], den = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) num[j] = 0.f;
        for (int c = c0; c <= c1; ++c) {
            const float f = exp2f(pm[slot(c)] - M);
            den = fmaf(f, pl[slot(c)], den);
            const float* o = po + slot(c) * D + lane * V;
#pragma unroll
            for (int j = 0; j < V; ++j) num[j] = fmaf(f, o[j], num[j]);
        }
        const float inv = den > 0.f ? p.vscale / den : (den == 0.f ? 0.f : den);
        const int rr = rt * kRows + r;
        __nv_bfloat16* out = p.O + (static_cast<int64_t>(s.first + rr / p.QG) * p.Hq + g * p.QG +
                                    rr % p.QG) * D + lane * V;
#pragma unroll
        for (int j = 0; j < V; j += 2)
            *reinterpret_cast<uint32_t*>(out + j) = pack_bf16x2(num[j] * inv, num[j + 1] * inv);
    }
}

template <int D, bool kFp8, bool kHalf>
int launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, cudaStream_t st) {
    using C = Cfg<D, kFp8>;
    auto kern = tree_attn_kernel<D, kFp8, kHalf>;
    const size_t smem = 1024 + static_cast<size_t>(kStages) * C::STAGE + sizeof(Smem<D>);
    static int ok = -1;
    static std::once_flag once;
    std::call_once(once, [&] {
        ok = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(smem)) == cudaSuccess;
    });
    if (ok != 1) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(p.ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    const int rc = cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p);
    if (rc != cudaSuccess) return rc;
    const int row_tiles = (p.T * p.QG + kRows - 1) / kRows;
    cudaLaunchConfig_t mc = {};
    LaunchAttrs mla;
    apply_pdl(mc, mla);
    mc.gridDim = dim3(static_cast<unsigned>(row_tiles) * p.d.Hkv, p.d.B, 1);
    mc.blockDim = dim3(kMergeThreads, 1, 1);
    mc.stream = st;
    return cudaLaunchKernelEx(&mc, tree_merge_kernel<D>, p, row_tiles);
}

template <int D, bool kFp8>
int launch_rows(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p,
                cudaStream_t st) {
    return p.T * p.QG <= 8 ? launch<D, kFp8, true>(kmap, vmap, p, st)
                           : launch<D, kFp8, false>(kmap, vmap, p, st);
}

}  // namespace

size_t tree_attention_workspace(int D, int rows, int num_sms) {
    (void)rows;
    return static_cast<size_t>(2) * kCtasPerSm * num_sms * kRows * (D + 2) * sizeof(float);
}

int launch_tree_attention(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N,
                          int T, int Hq, const int* cu, const int* parents, float scale,
                          float* ws, int num_sms, void* stream) {
    TreeParams p = {};
    p.status = tc_status_ptr();
    if (!p.status) return cudaErrorInvalidSymbol;
    p.d = paged_dims(c);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.O = static_cast<__nv_bfloat16*>(O);
    p.cu = cu;
    p.parents = parents;
    p.ws = ws;
    p.q_stride = q_stride;
    p.N = N;
    p.T = T;
    p.Hq = Hq;
    p.QG = Hq / c.Hkv;
    p.ctas = kCtasPerSm * num_sms;
    p.box_shift = p.d.page_shift < 6 ? p.d.page_shift : 6;
    p.qscale = scale * 1.4426950408889634f * c.k_scale;  // log2(e): exp2 of the scaled score
    p.vscale = c.v_scale;
    // K and V as [pages, heads, slots, D], copied a page piece and 128 bytes of
    // columns at a time
    const bool fp8 = c.dtype == QMM_CACHE_E4M3;
    const int e = fp8 ? 1 : 2, row = c.D * e;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.d.slot_stride * e),
                                   static_cast<cuuint64_t>(p.d.head_stride * e),
                                   static_cast<cuuint64_t>(p.d.page_stride * e)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>((row < 128 ? row : 128) / e),
                               static_cast<cuuint32_t>(1 << p.box_shift), 1, 1};
    const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                         : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = row < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap kmap, vmap;
    if (!encode_tiled(&kmap, type, 4, c.K, dims, strides, box, sw) ||
        !encode_tiled(&vmap, type, 4, c.V, dims, strides, box, sw))
        return cudaErrorInvalidValue;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (c.D == 128)
        return fp8 ? launch_rows<128, true>(kmap, vmap, p, st)
                   : launch_rows<128, false>(kmap, vmap, p, st);
    return fp8 ? launch_rows<64, true>(kmap, vmap, p, st) : launch_rows<64, false>(kmap, vmap, p, st);
}

}  // namespace qmm
