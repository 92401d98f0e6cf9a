// Tree attention for more than 16 query rows per KV head (qmm_tree_attention):
// the products on the 5th-generation tensor cores.
//
// The formulas and the work split are those of qmm_tree_attention.cu.  Here a
// work item is up to 128 or 256 rows, the MMA's M, and a tile is two MMAs with
// the accumulators in tensor memory:
//   S [128 x 64]  = Q [128 x D] K^T    A = Q in tensor memory, B = the K tile
//   O [128 x D]  += P [128 x 64] V     A = P in tensor memory, B = the V tile
// Rows past the item's are computed and dropped: at 128 rows a tile's products
// take about a fifth of the time its 32 KB of K and V take from HBM, so the
// padding is free where there are few rows, and full tiles are what it is for.
//
// One CTA per SM, 12 warps:
//   warp 0     copies: K and V tiles, each to its own slot of a ring
//   warp 1     issues the MMAs and owns the tensor memory
//   warps 2-3  E4M3 cache: convert the copied tiles to F16 in a second ring
//   warps 4-7, 8-11  two softmax groups of 128 threads, one thread a row
// Two streams of (Q, S/P, O) keep the tensor cores and the exponentials busy at
// the same time: while a group turns its S into P, the other stream's products
// run.  An item of more than 128 rows gives each stream half of the rows and
// the same tiles; an item of at most 128 gives both streams all rows and every
// other tile, and the groups add their two states at the end.
//   MMA order:  ... P0 V(i), Q0 K(i+1) | P1 V(i), Q1 K(i+1) ...
// P overwrites S in place (BF16 or F16 in half the columns); the MMAs run in
// issue order, so a group that sees S of its next tile also knows that its last
// P V is done, and may rescale O.
//
// A row's maximum is followed lazily: P = 2^(s - ref) with a reference that is
// raised only when a score passes it by more than 8, so P stays below 2^8 and O
// is rescaled a few times per item instead of every tile.  The result is the
// same but for rounding: sums are FP32, P is rounded to BF16 (F16 for an E4M3
// cache) whatever its scale.  One BF16 term of P, where the kernel for few rows
// keeps two: the second would double the P V products, and its error is that of
// rounding the output.
//
// Tensor memory (512 columns): Q 2 x 64, S/P 2 x 64, O 2 x 128 for D = 128.
#include <mutex>

#include "qmm.h"
#include "qmm_tree.cuh"

namespace qmm {
namespace {

constexpr int kTcThreads = 384;
constexpr int kConvWarps = 2;       // warps 2 and 3
constexpr int kSoftmaxWarp0 = 4;
constexpr int kHave = 16;           // tiles whose page bits are kept
constexpr float kLazy = 8.f;        // log2 units a score may pass the reference by

constexpr uint32_t kColQ = 0, kColS = 128, kColO = 256;   // stream s: + 64 s, + 64 s, + 128 s

template <int D, bool kFp8>
struct Tc {
    static constexpr int ROW = D * (kFp8 ? 1 : 2);
    static constexpr int BOX = ROW < 128 ? ROW : 128;
    static constexpr int BOXES = ROW / BOX;
    static constexpr int COPY = kTile * ROW;                 // bytes of a copied tile
    static constexpr int MMA = kTile * D * 2;                // of an MMA operand tile
    static constexpr int SLOTS = kFp8 ? 8 : (D == 128 ? 12 : 16);   // copy ring
    static constexpr int CONV = kFp8 ? 8 : 0;                // converted ring
    static constexpr int RING = SLOTS * COPY + CONV * MMA;
    static constexpr int KS = D / 16;
    static constexpr int COLS_Q = D / 2;                     // tensor memory columns of Q
};

template <int D, bool kFp8>
struct TcSmem {
    uint64_t full[Tc<D, kFp8>::SLOTS], empty[Tc<D, kFp8>::SLOTS];
    uint64_t cfull[8], cempty[8];       // converted ring
    uint64_t sfull[2];                  // S of a stream's next tile is there
    uint64_t pready[2];                 // P is, and O may take its product
    uint64_t ofull[2];                  // O is complete
    uint64_t qready;
    uint64_t drained;                   // abort: every MMA issued has ended
    uint32_t tmem;
    int have[kHave];                    // pages of a tile that exist, one bit a copy
    float m[2][128], l[2][128];
    int16_t par[kMaxTree];
    uint32_t anc[256][kWords + 1];      // a thread's own row: ancestors and itself
    RunShared run;
};

// Instruction descriptor: kind::f16, FP32 accumulate, K-major A in tensor
// memory, B K-major or (transposed) N-major.
__host__ __device__ constexpr uint32_t idesc(int N, bool f16, bool b_n_major) {
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) |
           ((b_n_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

// Shared-memory descriptor of a V tile as B, N-major with the 128-byte
// swizzle: rows are positions (the MMA's K), 64 values of the head wide; the
// next 64 values are kTile rows on (leading offset), the next 8 positions 1024
// bytes (stride offset).
__device__ __forceinline__ uint64_t sdesc_n_major(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
           (static_cast<uint64_t>((kTile * 128) >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// Offset of 16-byte chunk c of row r: copied tile (boxes of 64 rows), and
// operand tile (64 values, 128 bytes a row).
template <int BOX>
__device__ __forceinline__ uint32_t copy_off(int r, int c) {
    if (BOX == 128)
        return static_cast<uint32_t>((c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Positions of a tile (64 bits, from its first) that a row sees.
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeParams p) {
    using C = Tc<D, kFp8>;
    using Sm = TcSmem<D, kFp8>;
    constexpr int SLOTS = C::SLOTS, KS = C::KS;
    extern __shared__ uint8_t tree_tc_smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(tree_tc_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Sm& sm = *reinterpret_cast<Sm*>(ring + C::RING);
    __shared__ int abort_flag;
    volatile int* abort = &abort_flag;
    const uint32_t ring_a = smem_addr(ring);
    const uint32_t conv_a = ring_a + SLOTS * C::COPY;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], kFp8 ? kConvWarps : 1);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&sm.cfull[i], kConvWarps);
            mbar_init(&sm.cempty[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.sfull[s], 2);    // the commit, and the issuing thread
            mbar_init(&sm.pready[s], 4);
            mbar_init(&sm.ofull[s], 1);
        }
        mbar_init(&sm.qready, 8);
        mbar_init(&sm.drained, 1);
        mbar_fence_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    // Tensor memory is taken after the kernels before this one have ended, and
    // the next may start only once it is taken: a CTA that holds tensor memory
    // never waits for one that still needs it.
    pdl_wait();
    if (warp == 1) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = sm.tmem;
    Run run = find_run<kTcThreads>(p, sm.run);
    const int box = 1 << p.box_shift;
    const int pieces = kTile >> p.box_shift;
    Stretch x;

    if (warp == 0) {
        // ---- copies ----
        const int my_piece = lane / C::BOXES, my_box = lane % C::BOXES;
        const bool copies = my_piece < pieces;
        const uint32_t my_off = my_box * (kTile * C::BOX) + (my_piece << p.box_shift) * C::BOX;
        int it = 0, ks = 0;    // tiles; tiles whose K and V both went out
        int slot = 0, round = 0;
        bool ok_run = true;
        while (ok_run && next_stretch(p, run, &x)) {
            const int c_end = (x.s.total + box - 1) >> p.box_shift;
            const int* row = p.d.table + static_cast<int64_t>(x.b) * p.d.max_pages;
            auto entry = [&](int c) {
                return c < c_end ? row[(c << p.box_shift) >> p.d.page_shift] : -1;
            };
            int c0 = x.t0 * pieces;
            int cur = entry(c0 + lane), nxt = entry(c0 + 32 + lane);
            for (int t = x.t0; ok_run && t < x.t1; ++t, ++it) {
                if (t * pieces >= c0 + 32) {
                    c0 += 32;
                    cur = nxt;
                    nxt = entry(c0 + 32 + lane);
                }
                const int at = t * pieces - c0;
                const uint32_t ok = __ballot_sync(0xffffffffu, cur >= 0 && cur < p.d.num_pages);
                const int page = __shfl_sync(0xffffffffu, cur, (at + my_piece) & 31);
                const int pos = (t * kTile + (my_piece << p.box_shift)) &
                                ((1 << p.d.page_shift) - 1);
                const bool real = (ok >> ((at + my_piece) & 31)) & 1u;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (round > 0 && !mbar_wait_warp(&sm.empty[slot], (round - 1) & 1, abort, p.status)) {
                        ok_run = false;
                        break;
                    }
                    if (lane == 0) {
                        if (v == 0)
                            sm.have[it % kHave] = static_cast<int>((ok >> at) & ((1u << pieces) - 1u));
                        mbar_arrive_expect_tx(&sm.full[slot], C::COPY);
                    }
                    __syncwarp();
                    if (copies) {
                        // the slot may have been read or zeroed with ordinary accesses
                        fence_proxy_async_smem();
                        tma_load_4d(ring_a + slot * C::COPY + my_off, v ? &vmap : &kmap,
                                    &sm.full[slot], my_box * (C::BOX / (kFp8 ? 1 : 2)), pos, x.g,
                                    real ? page : p.d.num_pages);
                    }
                    ++ks;
                    if (++slot == SLOTS) slot = 0, ++round;
                }
            }
        }
        if (*abort && lane == 0) {  // let the copies in flight land before the CTA exits
            for (int j = ks > SLOTS ? ks - SLOTS : 0; j < ks; ++j)
                mbar_wait(&sm.full[j % SLOTS], (j / SLOTS) & 1, nullptr, p.status);
        }
    } else if (warp == 1) {
        // ---- MMAs ----
        // operand tiles in the order K(0), V(0), K(1), V(1), ... of the run
        constexpr int OPS = kFp8 ? C::CONV : SLOTS;
        uint64_t* full = kFp8 ? sm.cfull : sm.full;
        uint64_t* empty = kFp8 ? sm.cempty : sm.empty;
        const uint32_t op_a = kFp8 ? conv_a : ring_a;
        constexpr uint32_t iqk = idesc(kTile, kFp8, false);
        constexpr uint32_t ipv = idesc(D, kFp8, true);
        int base = 0;                   // tiles of the run before this stretch
        int np[2] = {0, 0}, nq = 0;     // P's and Q's taken
        bool go = true;
        auto wait_op = [&](int j) {
            return mbar_wait_warp(&full[j % OPS], (j / OPS) & 1, abort, p.status);
        };
        auto qk = [&](int s, int j) {   // S of stream s from operand tile j
            if (lane == 0) {
                const uint32_t b = op_a + (j % OPS) * C::MMA;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    umma_bf16_tmem_a(tmem + kColS + 64 * s, tmem + kColQ + 64 * s + 8 * k,
                                     sdesc_kmajor_sw128(b + (k >> 2) * (kTile * 128) + (k & 3) * 32),
                                     iqk, k > 0);
            }
        };
        auto pv = [&](int s, int j, bool first) {
            if (lane == 0) {
                const uint32_t b = op_a + (j % OPS) * C::MMA;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    umma_bf16_tmem_a(tmem + kColO + 128 * s, tmem + kColS + 64 * s + 8 * k,
                                     sdesc_n_major(b + k * 2048), ipv, !first || k > 0);
            }
        };
        auto release = [&](int j) {
            if (lane == 0) umma_commit(&empty[j % OPS]);
        };
        auto s_done = [&](int s) {
            if (lane == 0) {
                umma_commit(&sm.sfull[s]);
                // this thread has seen the tile's copy complete, and with it the
                // copy warp's page bits: hand that on
                mbar_arrive(&sm.sfull[s]);
            }
        };
        while (go && next_stretch(p, run, &x)) {
            const int nt = x.t1 - x.t0;
            const bool both = x.s.n * p.QG - x.row0 > 128;   // two halves of the rows
            if (!mbar_wait_warp(&sm.qready, nq & 1, abort, p.status)) break;
            ++nq;
            tc_fence_after();
            // first S of each stream
            for (int i = 0; go && i < (both ? 1 : min(nt, 2)); ++i) {
                const int j = 2 * (base + i);
                if (!(go = wait_op(j))) break;
                qk(both ? 0 : i, j);
                s_done(both ? 0 : i);
                if (both) {
                    qk(1, j);
                    s_done(1);
                }
                release(j);
            }
            for (int i = 0; go && i < nt; ++i) {
                for (int u = 0; go && u < (both ? 2 : 1); ++u) {
                    const int s = both ? u : i & 1;
                    const int next = i + (both ? 1 : 2);     // the stream's next tile
                    const bool last = both ? u == 1 : true;  // last reader of the tile
                    if (!(go = mbar_wait_warp(&sm.pready[s], np[s] & 1, abort, p.status))) break;
                    ++np[s];
                    if (!(go = wait_op(2 * (base + i) + 1))) break;
                    tc_fence_after();
                    pv(s, 2 * (base + i) + 1, i < (both ? 1 : 2));
                    if (last) release(2 * (base + i) + 1);
                    if (next < nt) {
                        if (!(go = wait_op(2 * (base + next)))) break;
                        qk(s, 2 * (base + next));
                        s_done(s);
                        if (last) release(2 * (base + next));
                    } else if (lane == 0) {
                        umma_commit(&sm.ofull[s]);
                    }
                }
            }
            base += nt;
        }
        if (*abort) {  // MMAs in flight end before the tensor memory goes back
            if (lane == 0) {
                umma_commit(&sm.drained);
                mbar_wait(&sm.drained, 0, nullptr, p.status);
            }
            __syncwarp();
        }
    } else if (warp < kSoftmaxWarp0) {
        // ---- E4M3 -> F16 ----
        if (kFp8) {
            const int t64 = tid - 64;
            int j = 0;
            bool go = true;
            while (go && next_stretch(p, run, &x)) {
                for (int t = x.t0; go && t < x.t1; ++t) {
                    const int valid = x.s.total - t * kTile;
                    for (int v = 0; v < 2; ++v, ++j) {
                        if (!(go = mbar_wait_warp(&sm.full[j % SLOTS], (j / SLOTS) & 1, abort,
                                                  p.status)))
                            break;
                        const int cs = j % 8;
                        if (j >= 8 && !(go = mbar_wait_warp(&sm.cempty[cs], ((j / 8) & 1) ^ 1, abort,
                                                            p.status)))
                            break;
                        const uint8_t* src = ring + (j % SLOTS) * C::COPY;
                        uint8_t* dst = ring + SLOTS * C::COPY + cs * C::MMA;
                        // thread: row t64, every 16-value chunk
                        uint4 in[D / 16];
#pragma unroll
                        for (int c = 0; c < D / 16; ++c)
                            in[c] = *reinterpret_cast<const uint4*>(src + copy_off<C::BOX>(t64, c));
                        if (t64 >= valid) {
                            // slots past the last position may hold anything, and
                            // 0 * NaN is not 0
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) in[c] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            const uint32_t w[4] = {in[c].x, in[c].y, in[c].z, in[c].w};
                            uint32_t f[8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                f[2 * i] = e4m3x2_to_f16x2(w[i] & 0xffffu);
                                f[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
                            }
                            *reinterpret_cast<uint4*>(dst + copy_off<128>(t64, 2 * c)) =
                                make_uint4(f[0], f[1], f[2], f[3]);
                            *reinterpret_cast<uint4*>(dst + copy_off<128>(t64, 2 * c + 1)) =
                                make_uint4(f[4], f[5], f[6], f[7]);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sm.empty[j % SLOTS]);
                            mbar_arrive(&sm.cfull[cs]);
                        }
                    }
                }
            }
        }
    } else {
        // ---- softmax groups ----
        const int s = (warp - kSoftmaxWarp0) >> 2;
        const int gt = tid - 32 * kSoftmaxWarp0;          // 0 .. 255
        const int r128 = (warp & 3) * 32 + lane;          // row of the stream = tensor memory lane
        const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + quarter + kColS + 64 * s;
        const uint32_t tQ = tmem + quarter + kColQ + 64 * s;
        const uint32_t tO = tmem + quarter + kColO;       // stream 0's; stream 1's + 128
        int base = 0;             // tiles of the run before this stretch
        int ns = 0, no = 0;       // S's and O's taken
        auto waits = [&](uint64_t* bar, int phase) {
            return !__any_sync(0xffffffffu, *abort) && mbar_wait_warp(bar, phase, abort, p.status);
        };
        while (next_stretch(p, run, &x)) {
            const int nt = x.t1 - x.t0;
            const int rows = min(1 << p.row_shift, x.s.n * p.QG - x.row0);
            const bool both = x.s.n * p.QG - x.row0 > 128;
            const int r = both ? r128 + 128 * s : r128;              // row of the item
            const bool on = r < rows;
            const bool warp_on = __any_sync(0xffffffffu, on);
            const int node = (x.row0 + (on ? r : 0)) / p.QG;
            const int head = x.g * p.QG + (x.row0 + (on ? r : 0)) % p.QG;
            // ---- ancestors, where the stretch reaches the drafted slots ----
            if (x.t1 * kTile > x.s.len) {
                if (p.parents) {
                    named_bar_sync(1, 256);   // the last stretch's walks are done
                    for (int i = gt; i < x.s.n; i += 256) {
                        const int v = p.parents[x.s.first + i];
                        sm.par[i] = static_cast<int16_t>(v >= 0 && v < i ? v : -1);
                    }
                    named_bar_sync(1, 256);
                }
                uint32_t w[kWords];
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    w[j] = p.parents ? 0u : static_cast<uint32_t>(low_bits(node + 1 - 32 * j));
                if (p.parents)
                    for (int i = node; i >= 0; i = sm.par[i]) {
#pragma unroll
                        for (int j = 0; j < kWords; ++j)
                            if (j == i >> 5) w[j] |= 1u << (i & 31);
                    }
#pragma unroll
                for (int j = 0; j < kWords; ++j) sm.anc[gt][j] = w[j];
            }
            // ---- Q to tensor memory ----
            float qs = p.qscale;
            if (warp_on) {
                const __nv_bfloat16* qv = p.q + (x.s.first + node) * p.q_stride + head * D;
                float down = 1.f;
                if (kFp8) {
                    // F16 keeps 11 bits between 2^-14 and 2^16: with the row's
                    // maximum brought to [1, 2), rounding to it is 2^-25 at most
                    float big = 0.f;
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4*>(qv + 8 * c);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            big = fmaxf(big, fmaxf(__uint_as_float((w[i] & 0x7fffu) << 16),
                                                   __uint_as_float(w[i] & 0x7fff0000u)));
                    }
                    int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
                    e = big > 0.f && e < 128 ? max(-126, min(126, e)) : 0;
                    down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    qs *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                }
#pragma unroll
                for (int c = 0; c < C::COLS_Q; c += 16) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const uint4 v = *reinterpret_cast<const uint4*>(qv + 2 * (c + i));
                        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
                    }
                    if (kFp8)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * down,
                                              __uint_as_float(w[i] & 0xffff0000u) * down);
                    tmem_st16(tQ + c, w);
                }
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.qready);

            float ref = -INFINITY, sum = 0.f;
            int mine = 0;   // tiles of this stream
            for (int i = both ? 0 : s; i < nt; i += both ? 1 : 2, ++mine) {
                if (!waits(&sm.sfull[s], ns & 1)) break;
                ++ns;
                tc_fence_after();
                const int t = x.t0 + i;
                const int valid = x.s.total - t * kTile;
                if (!kFp8 && valid < kTile) {
                    // slots past the last position may hold anything, and 0 * NaN
                    // is not 0: their V rows become zeros before P V reads them
                    const int j = 2 * (base + i) + 1;
                    if (!waits(&sm.full[j % SLOTS], (j / SLOTS) & 1)) break;
                    uint8_t* v = ring + (j % SLOTS) * C::COPY;
                    for (int c = gt & 127; c < (kTile - valid) * (C::ROW / 16); c += 128)
                        *reinterpret_cast<uint4*>(v + copy_off<C::BOX>(valid + c / (C::ROW / 16),
                                                                       c % (C::ROW / 16))) =
                            make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                if (warp_on) {
                    uint32_t v[64];
#pragma unroll
                    for (int c = 0; c < 64; c += 16) tmem_ld16(tS + c, v + c);
                    // what the row sees of the tile
                    const uint32_t have = static_cast<uint32_t>(sm.have[(base + i) % kHave]);
                    const int past = t * kTile + kTile - x.s.len;   // drafted positions and beyond
                    uint64_t see = ~0ull;
                    if (past > 0) {
                        // history, then the ancestors' bits from token j0 on
                        const int j0 = t * kTile - x.s.len;
                        const int hist = j0 < 0 ? -j0 : 0;
                        const int from = j0 > 0 ? j0 : 0;
                        uint64_t bits = 0;
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            const int w = (from >> 5) + k;
                            const uint64_t b = w < kWords ? sm.anc[gt][w] : 0u;
                            const int sh = 32 * k - (from & 31);
                            bits |= sh >= 0 ? (sh < 64 ? b << sh : 0ull) : b >> -sh;
                        }
                        see = (hist < 64 ? bits << hist : 0ull) | low_bits(hist);
                        see &= low_bits(valid);
                    }
                    if (have != (1u << pieces) - 1u)
                        for (int k = 0; k < pieces; ++k)
                            if (!((have >> k) & 1u)) see &= ~(low_bits(box) << (k << p.box_shift));
                    tmem_ld_wait();
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    if (__any_sync(0xffffffffu, see != ~0ull)) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!((see >> c) & 1ull)) v[c] = 0xff800000u;   // -inf
                    }
#pragma unroll
                    for (int c = 0; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(v[c]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * qs;
                    // raise the reference
                    const bool raise = top > ref + kLazy || (ref == -INFINITY && top != -INFINITY);
                    if (__any_sync(0xffffffffu, raise)) {
                        const float now = fmaxf(ref, top);
                        const float f = now == -INFINITY ? 1.f : fast_exp2(ref - now);
                        sum *= f;
                        ref = now;
                        if (mine > 0) {
                            const uint32_t o = tO + 128 * s;
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t w[16];
                                tmem_ld16(o + c, w);
                                tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
                                tmem_st16(o + c, w);
                            }
                            tmem_st_wait();
                        }
                    }
                    const float sub = finite_max(ref);
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t pw[32];
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const float a = fast_exp2(fmaf(__uint_as_float(v[c]), qs, -sub));
                        const float b = fast_exp2(fmaf(__uint_as_float(v[c + 1]), qs, -sub));
                        part[c / 2 & 3] += a + b;
                        pw[c / 2] = kFp8 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
                    }
                    sum += (part[0] + part[1]) + (part[2] + part[3]);
                    tmem_st16(tS, pw);
                    tmem_st16(tS + 16, pw + 16);
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.pready[s]);
            }
            base += nt;
            if (mine > 0) {
                waits(&sm.ofull[s], no & 1);
                ++no;
                tc_fence_after();
            }
            // ---- O, or the partial state.  With tiles shared out, both groups
            // exchange their statistics and each adds half of the columns ----
            float f0 = 1.f, f1 = 0.f, M = ref, den = sum;
            int c_lo = 0, c_hi = D;
            bool two = false;
            if (!both) {
                // (a group without tiles leaves its place alone: the other one may
                // still be reading it for the stretch before)
                if (mine > 0) {
                    sm.m[s][r128] = ref;
                    sm.l[s][r128] = sum;
                }
                tc_fence_before();
                named_bar_sync(1, 256);
                tc_fence_after();
                two = nt > 1;
                const float m0 = sm.m[0][r128], m1 = two ? sm.m[1][r128] : -INFINITY;
                M = fmaxf(m0, m1);
                const float mf = finite_max(M);
                f0 = fast_exp2(m0 - mf);
                f1 = fast_exp2(m1 - mf);
                den = f0 * sm.l[0][r128] + (two ? f1 * sm.l[1][r128] : 0.f);
                c_lo = s * (D / 2);
                c_hi = c_lo + D / 2;
            }
            if (warp_on && !__any_sync(0xffffffffu, *abort)) {
                const bool whole = x.t0 == 0 && x.t1 == x.s.tiles;
                const PartialAt part = partial_at<D>(p, 2 * blockIdx.x + (x.t0 == 0 ? 1 : 0));
                const float inv =
                    whole ? (den > 0.f ? p.vscale / den : (den == 0.f ? 0.f : den)) : 1.f;
                if (on && !whole && c_lo == 0) {
                    part.m[r] = M;
                    part.l[r] = den;
                }
                __nv_bfloat16* out = p.O + (static_cast<int64_t>(x.s.first + node) * p.Hq + head) * D;
                float* po = part.o + static_cast<size_t>(r) * D;
                const uint32_t o0 = both ? tO + 128 * s : tO;
#pragma unroll 1
                for (int c = c_lo; c < c_hi; c += 16) {
                    uint32_t a[16], b[16];
                    tmem_ld16(o0 + c, a);
                    if (two) tmem_ld16(tO + 128 + c, b);
                    tmem_ld_wait();
                    float y[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        y[k] = __uint_as_float(a[k]) * f0;
                        if (two) y[k] = fmaf(__uint_as_float(b[k]), f1, y[k]);
                        y[k] *= inv;
                    }
                    if (on && whole) {
#pragma unroll
                        for (int k = 0; k < 16; k += 8)
                            *reinterpret_cast<uint4*>(out + c + k) = make_uint4(
                                pack_bf16x2(y[k], y[k + 1]), pack_bf16x2(y[k + 2], y[k + 3]),
                                pack_bf16x2(y[k + 4], y[k + 5]), pack_bf16x2(y[k + 6], y[k + 7]));
                    } else if (on) {
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            *reinterpret_cast<float4*>(po + c + k) =
                                make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                    }
                }
            }
            // The next stretch's products start when every warp of both groups has
            // brought its Q: until then O, m and l stay as they are.
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, bool kFp8>
int launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, cudaStream_t st) {
    using C = Tc<D, kFp8>;
    auto kern = tree_tc_kernel<D, kFp8>;
    const size_t smem = 1024 + static_cast<size_t>(C::RING) + sizeof(TcSmem<D, kFp8>);
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
    cfg.blockDim = dim3(kTcThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p);
}

}  // namespace

int launch_tree_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int D,
                   bool fp8, cudaStream_t st) {
    if (D == 128) return fp8 ? launch<128, true>(kmap, vmap, p, st) : launch<128, false>(kmap, vmap, p, st);
    return fp8 ? launch<64, true>(kmap, vmap, p, st) : launch<64, false>(kmap, vmap, p, st);
}

}  // namespace qmm
