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
// Work split.  A work item is (sequence b, KV head g, tile of query rows), of
// ceil(L_b / tile) tiles of positions, L_b = lens[b] + n_b, and counts for its
// tiles and a few more units of work (its q, its output).  Lengths live on the
// device and differ widely in a batch, so the grid does not know them: it is a
// fixed number of CTAs, and the units of all items, laid end to end, are cut
// into that many equal runs.  Each CTA sums the batch's units, finds its run
// and walks it; the copies run ahead across item borders.  An item
// inside one run is written to O.  An item that a border cuts leaves a partial
// softmax state (maximum, sum, unnormalized output, FP32) per run, at most two
// a CTA, and the merge kernel adds them in run order: the bits do not depend
// on timing.  Equal runs keep every SM busy to the end whatever the lengths,
// and the workspace is two states per CTA whatever the batch.
#include <algorithm>
#include <limits>

#include "qmm.h"
#include "qmm_per_device.h"
#include "qmm_tree.cuh"

namespace qmm {

// Tiled tensor map helper (qmm_w4a16_tc.cu)
bool encode_tiled_promoted(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* ptr,
                           const cuuint64_t* dims, const cuuint64_t* strides,
                           const cuuint32_t* box, CUtensorMapSwizzle swizzle,
                           CUtensorMapL2promotion promotion);

namespace {

constexpr int kTile = 64;      // positions per tile
constexpr int kRows = 8;       // query rows per work item
constexpr int kWarps = 4;      // compute warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kKeys = kTile / kWarps;   // positions per compute warp
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;

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
    int pages[kTile / 8];              // of the tile being copied
    float wm[kWarps][kRows];
    float wl[kWarps][kRows];
    uint32_t anc[kRows][kWords];       // ancestors (and self) of each row's token
    int16_t par[kMaxTree];
    RunShared run;
    alignas(16) float ex[kWarps][kRows][D / kWarps];   // outputs on their way to another warp
};

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

// ---- the kernel -------------------------------------------------------------
//
// Up to 8 query rows per KV head (plain decode): half of an m16n8k16 fragment.
// CTA: 4 compute warps and one copy warp, as the contiguous decode kernel.  Bound
// by HBM where there is enough to read (32 sequences of 1024 to 8192 positions,
// BF16: 78 us, 5.8 TB/s), by start-up and the merge's launch where there is not
// (one of 1000: 9 us for both).  E4M3: 64 sequences of 1000 to 4000 take 71 us, floor
// 42; a tile's chain of waits, conversions, products and exp2 (940 clocks, HBM would
// need 610) with 8 compute warps an SM: 1.8 instructions a clock, most stalls on
// fixed latencies.
//   - The copy warp loads tiles of 64 positions into a 3-stage ring, one 4-D
//     copy per page piece and 128-byte column block.  A lane looks up one table
//     entry of the next 32 pieces at a time, one lane issues the copies.  A
//     missing page (or a piece past the last position) is copied from outside
//     the map, which fills zeros; the stage's bits tell the compute warps.
//   - Compute warp w takes positions 16w .. 16w+15 of a tile and keeps its own
//     softmax state; scores in log2 units, exp2.
//   - BF16 cache: BF16 products, P as two BF16 terms (hi + lo), about 16 bits.
//     E4M3 cache: the values are exact in F16, so the products run in F16; a
//     row of q is scaled by a power of two to a maximum in [1, 2) first, so
//     rounding it to F16 (11 bits, 2^-25 absolute) loses nothing of its 8 bits
//     but what lies 2^-17 below the row's maximum, and P is one F16 term,
//     times 2^15: weights down to 2^-29 of the largest keep 11 bits.
//   - When a stretch ends the 4 states are merged: each warp collects a quarter
//     of the columns from the other three.
// Every wait is bounded (1 s): a wait that runs out sets the status word and
// the CTA winds down after its copies in flight have landed.
template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    tree_attn_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ TreeParams p) {
    using C = Cfg<D, kFp8>;
    constexpr int KS = C::KS, NB = C::NB, NQ = NB / kWarps;
    extern __shared__ uint8_t tree_smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(tree_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(ring + kStages * C::STAGE);
    __shared__ int abort_flag;
    volatile int* abort = &abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    // (after the wait: the merge kernel plans with lens and cu before its own)
    pdl_trigger();
    __syncthreads();
    Run run = find_run<kThreads>(p, sm.run);
    const int pieces = kTile >> p.box_shift;     // copies of a tile, per column block and pool
    Stretch x;

    if (warp == kWarps) {
        // ---- copy warp ----
        const uint32_t ring_a = smem_addr(ring);
        int it = 0;   // tiles copied so far
        bool ok = true;
        while (ok && next_stretch(p, run, &x)) {
            PageWalk<kTile> walk;
            walk.start(p, x, lane);
            for (int t = x.t0; t < x.t1; ++t, ++it) {
                const uint32_t have = walk.tile(p, t, lane, sm.pages);
                const int st = it % kStages;
                ok = it < kStages ||
                     mbar_wait_warp(&sm.empty[st], ((it / kStages) & 1) ^ 1, abort, p.status);
                if (!ok) break;
                if (elect_one()) {
                    sm.have[st] = static_cast<int>(have);
                    // the compute warps read (and may have zeroed) the stage with
                    // ordinary accesses
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(&sm.full[st], C::STAGE);
                    constexpr int E = C::BOX / (kFp8 ? 1 : 2);
                    copy_tile<kTile, C::BOXES, C::BOX, E>(p, &kmap, &sm.full[st], ring_a + st * C::STAGE,
                                                   sm.pages, t, x.g);
                    copy_tile<kTile, C::BOXES, C::BOX, E>(p, &vmap, &sm.full[st],
                                                   ring_a + st * C::STAGE + C::TILE, sm.pages, t,
                                                   x.g);
                }
                __syncwarp();
            }
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
            const bool on = gr < rows;
            const int row = x.row0 + min(gr, rows - 1);
            const int node = row_node(p, row), head = x.g * p.QG + row - node * p.QG;
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
            // (rows 8 .. 15 of the fragment are zeros)
            uint32_t qa[KS][2];
            float qs = p.qscale, big = 0.f;
            {
                const __nv_bfloat16* qv = p.q + (x.s.first + node) * p.q_stride + head * D;
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
                    qa[ks][0] = on ? lo : 0u;
                    qa[ks][1] = on ? hi : 0u;
                    if (kFp8) {
                        const uint32_t a = lo & 0x7fff7fffu, c = hi & 0x7fff7fffu;
                        big = fmaxf(big, fmaxf(fmaxf(__uint_as_float(a << 16),
                                                     __uint_as_float(a & 0xffff0000u)),
                                               fmaxf(__uint_as_float(c << 16),
                                                     __uint_as_float(c & 0xffff0000u))));
                    }
                }
                if (kFp8) {
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    // 2^e <= big < 2^(e+1); a row of zeros, or one that holds
                    // infinities or NaN, is left as it is
                    int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
                    e = big > 0.f && e < 128 ? max(-126, min(126, e)) : 0;
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    qs = finite_factor(qs * __uint_as_float(static_cast<uint32_t>(127 + e) << 23));
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t v = qa[ks][i];
                            qa[ks][i] = pack_f16x2(__uint_as_float(v << 16) * down,
                                                           __uint_as_float(v & 0xffff0000u) * down);
                        }
                }
            }
            float o[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) o[nb][0] = o[nb][1] = 0.f;
            float m_run = -INFINITY, l_run = 0.f;   // l_run: this lane's share of the row's sum

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
                                const uint32_t a[4] = {qa[ks][0], 0u, qa[ks][1], 0u};
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
                            const uint32_t a[4] = {qa[ks][0], 0u, qa[ks][1], 0u};
                            mma16816<false>(sc[0], a, kf[0], kf[1]);
                            mma16816<false>(sc[1], a, kf[2], kf[3]);
                        }
                    }
                    // online softmax of each row over the 16 positions
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = sc[e >> 1][e & 1] * qs;
                    if (!plain) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = (e >> 1) * 8 + 2 * tq + (e & 1);
                            const int j = pos0 + k - x.s.len;   // drafted token, >= 0
                            bool see = k < valid && ((have >> ((kb + k) >> p.box_shift)) & 1u);
                            if (see && j >= 0)
                                see = p.parents ? (sm.anc[min(gr, rows - 1)][j >> 5] >> (j & 31)) & 1u
                                                : j <= node;
                            if (!see) v[e] = -INFINITY;
                        }
                    }
                    float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = fmaxf(m_run, mx), mf = finite_max(mn);
                    const float corr = fast_exp2(m_run - mf), by = mf - (kFp8 ? 15.f : 0.f);
                    m_run = mn;
                    float pw[4], rs = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pw[e] = fast_exp2(v[e] - by);
                        rs += pw[e];
                    }
                    l_run = l_run * corr + rs;
                    // P as the A operand of P V (rows, k = positions)
                    uint32_t ph[4] = {0, 0, 0, 0}, pl[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a = pw[2 * i], c = pw[2 * i + 1];
                        if (kFp8) {
                            ph[2 * i] = pack_f16x2(a, c);
                        } else {
                            const uint32_t w = pack_bf16x2(a, c);
                            ph[2 * i] = w;
                            pl[2 * i] = pack_bf16x2(a - __uint_as_float(w << 16),
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
                                        float d4[4] = {acc[0] * corr, acc[1] * corr, 0.f, 0.f};
                                        mma16816<true>(d4, ph, vf[2 * n], vf[2 * n + 1]);
                                        acc[0] = d4[0], acc[1] = d4[1];
                                    }
                                }
                            }
                        } else {
                            // matrices: (positions j % 2, dims j / 2), transposed
                            ldmatrix_x4_t(vf, vt + C::off(kb + (mj & 1) * 8 + mr, 2 * db + (mj >> 1)));
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                float* acc = o[2 * db + n];
                                float d4[4] = {acc[0] * corr, acc[1] * corr, 0.f, 0.f};
                                mma16816<false>(d4, ph, vf[2 * n], vf[2 * n + 1]);
                                mma16816<false>(d4, pl, vf[2 * n], vf[2 * n + 1]);
                                acc[0] = d4[0], acc[1] = d4[1];
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[st]);
            }

            // ---- merge the warps' states; warp w ends with columns
            // [w D/4, (w + 1) D/4) of every row ----
            l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
            l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
            if (tq == 0) {
                sm.wm[warp][gr] = m_run;
                sm.wl[warp][gr] = l_run;
            }
            named_bar_sync(1, 32 * kWarps);
            float M = -INFINITY, den = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.wm[w][gr]);
            const float mf = finite_max(M);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                den = fmaf(fast_exp2(sm.wm[w][gr] - mf), sm.wl[w][gr], den);
            const float fac = fast_exp2(m_run - mf);
            float acc[NQ][2];
#pragma unroll
            for (int qq = 0; qq < kWarps; ++qq)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        o[qq * NQ + n][i] *= fac;
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
                            *reinterpret_cast<float2*>(&sm.ex[to][gr][n * 8 + 2 * tq]) =
                                make_float2(o[qq * NQ + n][0], o[qq * NQ + n][1]);
                named_bar_sync(1, 32 * kWarps);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float2 v =
                        *reinterpret_cast<const float2*>(&sm.ex[warp][gr][n * 8 + 2 * tq]);
                    acc[n][0] += v.x;
                    acc[n][1] += v.y;
                }
                named_bar_sync(1, 32 * kWarps);
            }
            // (the other warps may not have seen the flag yet: this one goes on to
            // the next stretch's barriers with them, and writes nothing)
            if (*abort) continue;
            // ---- O, or the partial state ----
            const bool whole = x.t0 == 0 && x.t1 == x.s.tiles;
            const PartialAt part = partial_at<D>(p, 2 * blockIdx.x + (x.t0 == 0 ? 1 : 0));
            if (on) {
                const float inv =
                    whole ? (den > 0.f ? p.vscale / den : (den == 0.f ? 0.f : den)) : 1.f;
                if (!whole && warp == 0 && tq == 0) {
                    part.m[gr] = M;
                    part.l[gr] = den;
                }
                __nv_bfloat16* out =
                    p.O + (static_cast<int64_t>(x.s.first + node) * p.Hq + head) * D;
#pragma unroll
                for (int n = 0; n < NQ; n += kFp8 ? 2 : 1) {
                    // columns: BF16 8 n + 2 tq + {0, 1}; E4M3 n-blocks 2i (even
                    // dims) and 2i + 1 (odd dims): 16 i + 4 tq + {0, 2}, {1, 3}
                    const int c = (warp * NQ + n) * 8 + (kFp8 ? 4 : 2) * tq;
                    if (kFp8) {
                        const int n1 = n + 1 < NQ ? n + 1 : n;
                        const float4 v = make_float4(acc[n][0] * inv, acc[n1][0] * inv,
                                                     acc[n][1] * inv, acc[n1][1] * inv);
                        if (whole)
                            *reinterpret_cast<uint2*>(out + c) =
                                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4*>(part.at(gr, c)) = v;
                    } else {
                        const float2 v = make_float2(acc[n][0] * inv, acc[n][1] * inv);
                        if (whole)
                            *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(v.x, v.y);
                        else
                            *reinterpret_cast<float2*>(part.at(gr, c)) = v;
                    }
                }
            }
            __syncwarp();
        }
    }
    __syncthreads();
}

// The items that a run border cuts: O = sum_c 2^(m_c - M) o_c / sum_c
// 2^(m_c - M) l_c over the runs c that hold a stretch, in ascending c.  One
// block per item and 16 of its rows: a thread takes a row and every 16th (D =
// 128; 64: 8th) group of 4 columns.  Up to 256 sequences, a thread's one each, the
// plan is worked out while the attention kernel still runs (one token behind 1000:
// 9.4 us, behind the wait 10.0; 8 sequences of 8: 23.8 and 25.2).  That kernel's
// threads let this one start only after their own wait for everything before it, so
// lens and cu are final in L2, and are read there, not through an L1 that may hold
// older lines.  More sequences: behind the wait and through L1, where a block's many
// values come from (1024 of one token: 206 us, ahead from L2 214).  Bound by latency:
// one trip to the states, 2 to 3 us behind the attention kernel of a small call; 16
// sequences of 64 tokens (two states of most of 32768 rows, 33 MB): 20 us alone with
// a cold L2.
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 16;
constexpr int kMergeAhead = 4;   // states whose loads a thread has in flight
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    tree_merge_kernel(const __grid_constant__ TreeParams p, int max_row_tiles, int chunks) {
    __shared__ long long red[2][kMergeThreads / 32];
    __shared__ Seq own;
    __shared__ __align__(16) uint2 stage[kMergeRows][D / 4 + 2];   // BF16 rows, padded by 16 bytes
    const int chunk = blockIdx.x % chunks, item = blockIdx.x / chunks;
    const int rt = item % max_row_tiles, g = item / max_row_tiles, b = blockIdx.y;
    const bool ahead = p.d.B <= kMergeThreads;
    if (!ahead) {
        pdl_trigger();
        pdl_wait();
    }
    const int row0 = rt << p.row_shift;
    auto has_rows = [&](const Seq& x) {
        return rt < x.row_tiles && chunk * kMergeRows < min(1 << p.row_shift, x.n * p.QG - row0);
    };
    Seq s;
    long long all = 0, before = 0;
    if (p.d.B <= 32) {
        const int lane = threadIdx.x & 31;
        s = sequence<true>(p, min(lane, p.d.B - 1));
        const long long mine = lane < p.d.B ? units_of(p, s) : 0;
        before = __shfl_sync(0xffffffffu, warp_scan(mine, &all), b);
        s.first = __shfl_sync(0xffffffffu, s.first, b);
        s.n = __shfl_sync(0xffffffffu, s.n, b);
        s.tiles = __shfl_sync(0xffffffffu, s.tiles, b);
        s.row_tiles = __shfl_sync(0xffffffffu, s.row_tiles, b);
    } else if (ahead) {
        long long mine = 0;
        if (threadIdx.x < p.d.B) {
            s = sequence<true>(p, threadIdx.x);
            mine = units_of(p, s);
            if (threadIdx.x == b) own = s;
        }
        block_scan<kMergeThreads>(mine, red[0], &all);
        block_scan<kMergeThreads>(threadIdx.x < b ? mine : 0, red[1], &before);
        s = own;
    } else {
        s = sequence(p, b);
        if (has_rows(s)) {   // (the same for the whole block)
            long long mine = 0, upto = 0;
            for (int i = threadIdx.x; i < p.d.B; i += kMergeThreads) {
                const int u = units_of(p, sequence(p, i));
                mine += u;
                if (i < b) upto += u;
            }
            block_scan<kMergeThreads>(mine, red[0], &all);
            block_scan<kMergeThreads>(upto, red[1], &before);
        }
    }
    const int rows = min(1 << p.row_shift, s.n * p.QG - row0);
    int c0 = 0, c1 = 0;
    if (has_rows(s)) {
        const long long len = run_length(p, all);
        const int units = item_units(p, s);
        const long long start = before + static_cast<long long>(g * s.row_tiles + rt) * units;
        c0 = static_cast<int>((start + p.setup) / len);
        c1 = static_cast<int>((start + units - 1) / len);
    }
    if (ahead) {
        pdl_trigger();
        pdl_wait();
    }
    if (c0 == c1) return;
    constexpr int GROUPS = D / 4;
    constexpr int TURNS = GROUPS / (kMergeThreads / kMergeRows);   // column groups of a thread
    const int i = threadIdx.x % kMergeRows, r = chunk * kMergeRows + i;
    const int j0 = threadIdx.x / kMergeRows;
    if (r < rows) {
        auto part = [&](int c) { return partial_at<D>(p, 2 * c + (c == c0 ? 1 : 0)); };
        float M = -INFINITY;   // running: a pass of its own would cost a latency
        float4 num[TURNS];
        float den = 0.f;
#pragma unroll
        for (int u = 0; u < TURNS; ++u) num[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0; c <= c1; c += kMergeAhead) {
            float m[kMergeAhead], l[kMergeAhead];
            float4 o[kMergeAhead][TURNS];
#pragma unroll
            for (int k = 0; k < kMergeAhead; ++k) {
                m[k] = -INFINITY;
                if (c + k > c1) continue;
                const PartialAt x = part(c + k);
                m[k] = x.m[r];
                l[k] = x.l[r];
#pragma unroll
                for (int u = 0; u < TURNS; ++u)
                    o[k][u] = *reinterpret_cast<const float4*>(
                        x.at(r, 4 * (j0 + u * (kMergeThreads / kMergeRows))));
            }
            float top = M;
#pragma unroll
            for (int k = 0; k < kMergeAhead; ++k) top = fmaxf(top, m[k]);
            const float sub = finite_max(top), old = fast_exp2(M - sub);
            M = top;
            den *= old;
#pragma unroll
            for (int u = 0; u < TURNS; ++u) {
                num[u].x *= old;
                num[u].y *= old;
                num[u].z *= old;
                num[u].w *= old;
            }
#pragma unroll
            for (int k = 0; k < kMergeAhead; ++k) {
                if (c + k > c1) break;
                const float f = fast_exp2(m[k] - sub);
                den = fmaf(f, l[k], den);
#pragma unroll
                for (int u = 0; u < TURNS; ++u) {
                    num[u].x = fmaf(f, o[k][u].x, num[u].x);
                    num[u].y = fmaf(f, o[k][u].y, num[u].y);
                    num[u].z = fmaf(f, o[k][u].z, num[u].z);
                    num[u].w = fmaf(f, o[k][u].w, num[u].w);
                }
            }
        }
        const float inv = den > 0.f ? p.vscale / den : (den == 0.f ? 0.f : den);
#pragma unroll
        for (int u = 0; u < TURNS; ++u)
            stage[i][j0 + u * (kMergeThreads / kMergeRows)] =
                make_uint2(pack_bf16x2(num[u].x * inv, num[u].y * inv),
                           pack_bf16x2(num[u].z * inv, num[u].w * inv));
    }
    __syncthreads();
    constexpr int CH = D / 8;   // 16-byte chunks of a row
    const int ri = threadIdx.x / CH, c = threadIdx.x % CH;
    if (ri < kMergeRows && chunk * kMergeRows + ri < rows) {
        const int rr = row0 + chunk * kMergeRows + ri;
        const int64_t to = static_cast<int64_t>(s.first + rr / p.QG) * p.Hq + g * p.QG + rr % p.QG;
        *reinterpret_cast<uint4*>(p.O + to * D + 8 * c) =
            *reinterpret_cast<const uint4*>(&stage[ri][2 * c]);
    }
}

template <int D, bool kFp8>
int launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int device,
           cudaStream_t st) {
    using C = Cfg<D, kFp8>;
    auto kern = tree_attn_kernel<D, kFp8>;
    const size_t smem = 1024 + static_cast<size_t>(kStages) * C::STAGE + sizeof(Smem<D>);
    static PerDevice<bool> opted_in;
    if (!opted_in.get(device, [&] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(smem)) == cudaSuccess;
        }))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(p.ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p);
}

int launch_merge(const TreeParams& p, int D, cudaStream_t st) {
    const int rows = p.T * p.QG, item_rows = 1 << p.row_shift;
    const int row_tiles = (rows + item_rows - 1) >> p.row_shift;
    const int chunks = ((rows < item_rows ? rows : item_rows) + kMergeRows - 1) / kMergeRows;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(static_cast<unsigned>(row_tiles) * chunks * p.d.Hkv, p.d.B, 1);
    cfg.blockDim = dim3(kMergeThreads, 1, 1);
    cfg.stream = st;
    return D == 128 ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<128>, p, row_tiles, chunks)
                    : cudaLaunchKernelEx(&cfg, tree_merge_kernel<64>, p, row_tiles, chunks);
}

// The kernel for `rows` query rows per KV head, its rows per work item, CTAs
// per SM, shortest run and an item's fixed units.  Measured on both sides of each
// border with 32 sequences of 500 to 16000 positions, D = 128 (us), unless said:
//   8 rows: this file's kernel.  4 rows of one sequence of 1000: 9.6, the
//     tcgen05 kernel 12.2 (its start and drain are longer); 64 sequences of 1000
//     to 4000, E4M3: 73 and 81, BF16: 99 and 98.
//   9 to 128 rows: tcgen05, one group.  16 rows: 105, E4M3 77, with both row halves
//     of this file's fragments in use 132 and 113.  128 rows: 123, E4M3 109, with
//     two groups of a single CTA per SM 127 and 140.
//   more: two groups of 128 rows that share the K and V tiles.  256 rows: 143,
//     E4M3 154; one group that reads them twice 212 and 204.
// Shortest run: 6 units of the tcgen05 kernel (one sequence of 8 tokens behind 1000
// positions: 3 10.9, 6 11.7, 12 14.9; two of 16 behind 1000 to 4000: 17.3, 15.9,
// 17.1), 2 of this one (one token behind 1000: 1 11.0, 2 9.7, 4 10.5).
// Fixed units (what an item costs beside its tiles, in tiles: its q, drain and
// output): 4, with an E4M3 cache, whose tiles are cheaper and whose q has to be
// turned, 8 (256 rows: 2 191, 4 174, 8 154, 12 158; BF16, 64 ragged sequences of up to
// 5 tokens, D = 64: 2 125, 4 121, 8 124).
struct Variant {
    bool tc;
    int row_shift, tile_shift, ctas_per_sm, min_run, setup;
};
Variant variant(int rows, bool fp8) {
    if (rows <= kRows) return {false, 3, 6, kCtasPerSm, 2, 1};
    if (rows <= 128) return {true, 7, kTcTileShift, 2, 6, fp8 ? 8 : 4};
    return {true, 8, kTcTileShift, 1, 6, fp8 ? 8 : 4};
}

}  // namespace

size_t tree_attention_workspace(int D, int rows, int num_sms) {
    const Variant v = variant(rows, false);   // (the same for either type)
    return (static_cast<size_t>(2 * v.ctas_per_sm * num_sms) << v.row_shift) * (D + 2) *
           sizeof(float);
}

int launch_tree_attention(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N,
                          int T, int Hq, const int* cu, const int* parents, float scale,
                          float* ws, int num_sms, void* stream) {
    TreeParams p = {};
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return cudaErrorInvalidDevice;
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
    p.qg_inv = ((1u << 22) + p.QG - 1) / p.QG;
    const Variant var = variant(T * p.QG, c.dtype == QMM_CACHE_E4M3);
    p.ctas = var.ctas_per_sm * num_sms;
    p.row_shift = var.row_shift;
    p.tile_shift = var.tile_shift;
    p.min_run = var.min_run;
    p.setup = var.setup;
    p.box_shift = p.d.page_shift < p.tile_shift ? p.d.page_shift : p.tile_shift;
    // log2(e): exp2 of the scaled score.  Neither 0 nor infinity, whatever scale and
    // k_scale: times a masked score (-inf) or a score of 0 those would be NaN.
    const double factor = static_cast<double>(scale) * 1.4426950408889634 * c.k_scale;
    p.qscale = static_cast<float>(
        std::min(std::max(factor, static_cast<double>(std::numeric_limits<float>::denorm_min())),
                 static_cast<double>(std::numeric_limits<float>::max())));
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
    // L2 fetches what a copy reads and no neighbouring head with it: a row, where
    // the next slot's row is not the next in memory (E4M3, pages of [slot, head], 32
    // sequences of 16 tokens: 83.6 us, with 256 bytes 86.2; D = 64 65.4 and 68.8)
    const CUtensorMapL2promotion l2 = p.d.slot_stride == c.D || row >= 256
                                          ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                      : row == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                   : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    if (!encode_tiled_promoted(&kmap, type, 4, c.K, dims, strides, box, sw, l2) ||
        !encode_tiled_promoted(&vmap, type, 4, c.V, dims, strides, box, sw, l2))
        return cudaErrorInvalidValue;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc;
    if (var.tc)
        rc = launch_tree_tc(kmap, vmap, p, c.D, fp8, device, st);
    else if (c.D == 128)
        rc = fp8 ? launch<128, true>(kmap, vmap, p, device, st)
                 : launch<128, false>(kmap, vmap, p, device, st);
    else
        rc = fp8 ? launch<64, true>(kmap, vmap, p, device, st)
                 : launch<64, false>(kmap, vmap, p, device, st);
    return rc == cudaSuccess ? launch_merge(p, c.D, st) : rc;
}

}  // namespace qmm
