// Weights of the slots for more than 8 query rows per KV head (qmm_scored_attention),
// behind tree attention, which leaves each row's lse:
//
//   mass[b, g, s] = decay mass[b, g, s] + sum_r 2^(q_r . K_s f - lse_r)
//
// over the rows r of the sequence's KV head, f the factor that makes a score of a
// product.  Every product is one of tree attention's, but here the positions are the
// MMA's M and the rows its N: S^T [128 x N] = K tile [128 x D] Q^T.  A thread then holds
// a position's scores for all rows, so the sum over rows stays in its registers and the
// sums leave as 128 neighbouring floats, without a reduction between threads.
//
// A CTA an SM walks an equal run of the batch's (sequence, KV head, tile of 128
// positions) list.  Positions do not depend on one another, so nothing is merged; more
// than 256 rows are blocks of 256 that add to the same thread's slots one after the
// other.  Roles:
//   warp 0       copies K tiles into a ring
//   warp 1       issues the MMAs, owns the tensor memory: two buffers of 256 columns, or
//                four of 128, so that products run ahead of the sums
//   warps 2-3    bring a block's q (for an E4M3 cache as two E4M3 terms) and lse
//   warps 4-11   two groups of 128 threads that take turns with the tiles
//
// The last up to 32 tokens of 8 prompts of 2000 to 16000 (128 rows, 108 MB of K): the call
// takes 75 us, 41 of them the attention kernel, 28 this one where it cannot overlap (floor
// 16).  A tile of 128 positions and rows takes 990 clocks: 510 are its products, 300 waits
// for K; the rest is the start, 9,000 clocks of a kernel alone: plan, q and the first copies.
// All but lse is there before the merge has ended, so the start runs beside it (75 us, behind
// it 82).
#include <algorithm>

#include "qmm.h"
#include "qmm_per_device.h"
#include "qmm_tree_tc.cuh"

namespace qmm {
namespace {

constexpr int kTileShift = 7;
constexpr int kTile = 1 << kTileShift;   // positions
constexpr int kBlockShift = 8;
constexpr int kBlock = 1 << kBlockShift;   // query rows of a block
constexpr int kThreads = 384;
constexpr int kMaxSlots = 12;
constexpr int kHave = 32;                // tiles whose page bits are kept
constexpr int kSetup = 2;                // units an item counts for beside its tiles

template <int D, bool kFp8>
struct Mt {
    static constexpr int ROW = D * (kFp8 ? 1 : 2);      // bytes of a cache row
    static constexpr int BOX = ROW < 128 ? ROW : 128;   // row bytes of one copy
    static constexpr int BOXES = ROW / BOX;
    static constexpr int SLOT = kTile * ROW;
};

struct MassParams {
    TreeParams t;
    float* mass;
    int64_t mass_stride;
    float decay;
    int q_rows;    // rows of q kept: the call's largest block, a multiple of 32
    int slots;     // of the ring
    int buffers;   // of scores
    int q_buffers; // 1 or 2 blocks' q
};

struct MassSmem {
    uint64_t kfull[kMaxSlots], kempty[kMaxSlots];
    uint64_t dfull[4], dfree[4];       // scores of a tile are there; have been read
    uint64_t qready[2];                // even and odd blocks' q and lse are there
    uint64_t lfree[2];                 // have been read by all
    uint64_t qfree[2];                 // by buffer of q: the block's products are done
    uint64_t drained;                  // abort: every MMA issued has ended
    uint32_t tmem;
    int abort;
    int have[kHave];                   // pages of a tile that exist, one bit a copy
    int pages[2][16];                  // of the tiles being copied
    alignas(16) float nl[2][kBlock];   // -lse of a block's rows
    alignas(16) float qs[2][kBlock];   // E4M3: factor on their scores
    long long red[kThreads / 32];
    long long at;
    int b;
};
constexpr int kSmemHead = (sizeof(MassSmem) + 1023) / 1024 * 1024;

// ---- work split: tiles of an item, each as many units as it has blocks of rows --------

__device__ __forceinline__ int blocks_of(const Seq& s) { return s.row_tiles > 1 ? s.row_tiles : 1; }
__device__ __forceinline__ int mass_item(const Seq& s) {
    return s.total > 0 ? s.tiles * blocks_of(s) + kSetup : 0;
}
struct MassRun {
    Seq s;
    int b;
    long long at, left;   // unit within the sequence's list; units still to do
};
__device__ __forceinline__ MassRun find_mass_run(const TreeParams& p, MassSmem& sm) {
    const int tid = threadIdx.x;
    const int per = (p.d.B + kThreads - 1) / kThreads;
    const int b0 = min(p.d.B, tid * per), b1 = min(p.d.B, b0 + per);
    long long mine = 0, all;
    for (int b = b0; b < b1; ++b)
        mine += static_cast<long long>(mass_item(sequence<true>(p, b))) * p.d.Hkv;
    if (tid == 0) sm.b = -1;
    long long before = block_scan<kThreads>(mine, sm.red, &all);
    const long long len = (all + p.ctas - 1) / p.ctas, start = len * blockIdx.x;
    if (start >= before && start < before + mine)
        for (int b = b0; b < b1; ++b) {
            const long long u = static_cast<long long>(mass_item(sequence<true>(p, b))) * p.d.Hkv;
            if (start < before + u) {
                sm.b = b;
                sm.at = start - before;
                break;
            }
            before += u;
        }
    __syncthreads();
    MassRun r;
    r.b = sm.b;
    r.at = sm.at;
    r.left = r.b < 0 ? 0 : (all - start < len ? all - start : len);
    if (r.b >= 0) r.s = sequence<true>(p, r.b);
    return r;
}
// The next tiles of one item in the run: those whose first unit lies in it.
__device__ __forceinline__ bool next_tiles(const TreeParams& p, MassRun& r, Stretch* x) {
    while (r.left > 0) {
        const int item = mass_item(r.s);
        if (r.at >= static_cast<long long>(item) * p.d.Hkv) {
            r.at -= static_cast<long long>(item) * p.d.Hkv;
            if (++r.b >= p.d.B) return false;   // (not reached: the run ends with the list)
            r.s = sequence<true>(p, r.b);
            continue;
        }
        const int w = blocks_of(r.s);
        const int g = static_cast<int>(r.at / item), u0 = static_cast<int>(r.at - static_cast<long long>(g) * item);
        const int u1 = r.left < item - u0 ? static_cast<int>(u0 + r.left) : item;
        r.at += u1 - u0;
        r.left -= u1 - u0;
        x->s = r.s;
        x->b = r.b;
        x->g = g;
        x->t0 = u0 > kSetup ? (u0 - kSetup + w - 1) / w : 0;
        x->t1 = u1 > kSetup ? (u1 - kSetup + w - 1) / w : 0;
        if (x->t1 > x->t0) return true;
    }
    return false;
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ MassParams mp) {
    using C = Mt<D, kFp8>;
    extern __shared__ uint8_t mass_smem_raw[];
    uint8_t* base_s = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(mass_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    MassSmem& sm = *reinterpret_cast<MassSmem*>(base_s);
    const TreeParams& p = mp.t;
    uint8_t* q_s = base_s + kSmemHead;
    const int q_box = mp.q_rows * C::BOX;                 // (E4M3: the second term follows the first)
    const int q_bytes = mp.q_rows * D * 2;
    uint8_t* k_s = q_s + mp.q_buffers * q_bytes;
    volatile int* abort = &sm.abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        sm.abort = 0;
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&sm.kfull[i], 1);
            mbar_init(&sm.kempty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm.dfull[i], 2);    // the commit, and the issuing thread
            mbar_init(&sm.dfree[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.lfree[i], 8);
            mbar_init(&sm.qready[i], 2);
            mbar_init(&sm.qfree[i], 1);
        }
        mbar_init(&sm.drained, 1);
        mbar_fence_init();
        tma_prefetch_map(&kmap);
    }
    // Everything but lse was final before the attention kernel let the merge start (its
    // threads wait first, and only then let others start), so all of this kernel's work up to
    // the scores may run beside the merge, from L2: only the warps that read lse and that
    // touch the weights wait.  Tensor memory: the attention kernel's CTAs all have theirs by
    // then, and the merge needs none.  The dependency wait has no limit, and no wait that has one
    // starts ahead of it where it needs what comes behind: the limit times this launch alone.
    if (warp == 1) {
        tmem_alloc(&sm.tmem, 2 * kBlock);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = sm.tmem;
    MassRun run = find_mass_run(p, sm);
    const int pieces = kTile >> p.box_shift;
    Stretch x = {};
    auto wait_one = [&](uint64_t* bar, int phase) {
        return mbar_probe(bar, phase) || mbar_wait(bar, phase, abort, p.status);
    };
    auto waits = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, mbar_probe(bar, phase)) ||
               mbar_wait_warp(bar, phase, abort, p.status);
    };

    if (warp == 0) {
        // ---- copies ----
        Cursor kc;
        int it = 0;   // tiles copied, or asked for
        int nk = 0;   // of the issuing thread: copied
        bool ok = true;
        while (ok && next_tiles(p, run, &x)) {
            for (int rb = 0; ok && rb < blocks_of(x.s); ++rb) {
                PageWalk<kTile, true> walk;
                walk.start(p, x, lane);
                for (int t = x.t0; ok && t < x.t1; ++t, ++it) {
                    if (it == mp.slots) pdl_wait();   // (the first slot to wait for)
                    const uint32_t have = walk.tile(p, t, lane, sm.pages[it & 1]);
                    if (elect_one() && wait_one(&sm.kempty[kc.slot], kc.phase ^ 1)) {
                        sm.have[it % kHave] = static_cast<int>(have);
                        mbar_arrive_expect_tx(&sm.kfull[kc.slot], C::SLOT);
                        copy_tile<kTile, C::BOXES, C::BOX, C::BOX / (kFp8 ? 1 : 2)>(
                            p, &kmap, &sm.kfull[kc.slot], smem_addr(k_s + kc.slot * C::SLOT),
                            sm.pages[it & 1], t, x.g);
                        ++nk;
                    }
                    kc.next(mp.slots);
                    ok = !__any_sync(0xffffffffu, *abort);
                }
            }
        }
        if (!ok && elect_one()) {  // let the copies in flight land before the CTA exits
            for (int j = max(0, nk - mp.slots); j < nk; ++j)
                mbar_wait(&sm.kfull[j % mp.slots], (j / mp.slots) & 1, nullptr, p.status);
        }
    } else if (warp == 1) {
        // ---- MMAs: one thread waits and issues ----
        if (elect_one()) {
            const uint64_t q_desc = sdesc_k_major<C::BOX>(smem_addr(q_s));
            const uint64_t k_desc = sdesc_k_major<C::BOX>(smem_addr(k_s));
            Cursor kc;
            int nb = 0;            // blocks
            uint32_t used = 0, phase = 0;   // of each buffer: written before; its next wait
            bool go = true;
            pdl_wait();
            while (go && next_tiles(p, run, &x)) {
                const int rows = x.s.n * p.QG;
                for (int rb = 0; go && rb < blocks_of(x.s); ++rb, ++nb) {
                    const int n = max(16, (min(kBlock, rows - (rb << kBlockShift)) + 15) & ~15);
                    const uint32_t id = idesc(n, kFp8 ? 0u : 1u, false);
                    const int qb = nb & (mp.q_buffers - 1);
                    if (!(go = wait_one(&sm.qready[nb & 1], (nb >> 1) & 1))) break;
                    const uint64_t q0 = q_desc + static_cast<uint32_t>((qb * q_bytes) >> 4);
                    for (int t = x.t0; t < x.t1; ++t) {
                        const int i = (t - x.t0) & (mp.buffers - 1);
                        if ((used >> i) & 1u) {
                            if (!(go = wait_one(&sm.dfree[i], (phase >> i) & 1u))) break;
                            phase ^= 1u << i;
                        }
                        if (!(go = wait_one(&sm.kfull[kc.slot], kc.phase))) break;
                        used |= 1u << i;
                        tc_fence_after();
                        const uint64_t a = k_desc + static_cast<uint32_t>(kc.slot * C::SLOT >> 4);
                        const uint32_t d = tmem + (2 * kBlock / mp.buffers) * i;
                        if (kFp8) {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int k = 0; k < D / 32; ++k)
                                    umma_ss<true>(d, a + ((k * 32) >> 4),
                                                  q0 + static_cast<uint32_t>((h * q_box + k * 32) >> 4),
                                                  id, h > 0 || k > 0);
                        } else {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                umma_ss<false>(d, a + (((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4),
                                               q0 + static_cast<uint32_t>(((k >> 2) * q_box + (k & 3) * 32) >> 4),
                                               id, k > 0);
                        }
                        umma_commit(&sm.kempty[kc.slot]);
                        umma_commit(&sm.dfull[i]);
                        if (t + 1 == x.t1) umma_commit(&sm.qfree[qb]);
                        // this thread has seen the tile's copy complete, and with it the
                        // page bits, and the block's lse: hand that on
                        mbar_arrive(&sm.dfull[i]);
                        kc.next(mp.slots);
                    }
                }
            }
            if (!go) {  // MMAs in flight end before the tensor memory goes back
                umma_commit(&sm.drained);
                mbar_wait(&sm.drained, 0, nullptr, p.status);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // ---- q and lse of each block ----
        const int t64 = tid - 64;
        bool go = true;
        int nb = 0;
        while (go && next_tiles(p, run, &x)) {
            const int all = x.s.n * p.QG;
            for (int rb = 0; go && rb < blocks_of(x.s); ++rb, ++nb) {
                const int r0 = rb << kBlockShift, rows = min(kBlock, all - r0);
                const int qb = nb & (mp.q_buffers - 1), use = nb >> (mp.q_buffers - 1);
                if (use > 0 && !(go = waits(&sm.qfree[qb], (use - 1) & 1))) break;
                if (nb > 1 && !(go = waits(&sm.lfree[nb & 1], ((nb >> 1) - 1) & 1))) break;
                fence_proxy_async_smem();
                uint8_t* const q_at = q_s + qb * q_bytes;
                // this thread's rows of the block, `step` apart, without a division each: a
                // row further is D values on, a token further q_stride - QG D more
                auto each_row = [&](int start, int step, int count, auto&& f) {
                    int node = (r0 + start) / p.QG, head = r0 + start - node * p.QG;
                    const __nv_bfloat16* src = p.q + (x.s.first + node) * p.q_stride +
                                               static_cast<int64_t>(x.g * p.QG + head) * D;
                    const int dn = step / p.QG, dh = step - dn * p.QG;
                    const int64_t by = dn * p.q_stride + static_cast<int64_t>(dh) * D;
                    const int64_t wrap = p.q_stride - static_cast<int64_t>(p.QG) * D;
#pragma unroll 4
                    for (int r = start; r < count; r += step) {
                        f(r, src);
                        src += by;
                        head += dh;
                        if (head >= p.QG) {
                            head -= p.QG;
                            src += wrap;
                        }
                    }
                };
                if (kFp8) {
                    // a group of lanes a row, 16 values a lane
                    constexpr int LPR = D / 16, STEP = 64 / LPR;
                    const int c = t64 % LPR;
                    // (whole passes: a row's lanes exchange its largest value)
                    each_row(t64 / LPR, STEP, (rows + STEP - 1) / STEP * STEP,
                             [&](int r, const __nv_bfloat16* src) {
                        uint4 a = make_uint4(0, 0, 0, 0), b = a;
                        if (r < rows) {
                            a = __ldcg(reinterpret_cast<const uint4*>(src) + 2 * c);
                            b = __ldcg(reinterpret_cast<const uint4*>(src) + 2 * c + 1);
                        }
                        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                        uint32_t big = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) big = bf16_magnitude(big, w[i]);
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1)
                            big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
                        float qs = p.qscale;
                        const float up = e4m3_scaling(big, &qs);
                        uint32_t t[2][4];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t hi, lo;
                            e4m3_terms(w[i], up, &hi, &lo);
                            if (i % 2 == 0) t[0][i / 2] = hi, t[1][i / 2] = lo;
                            else t[0][i / 2] |= hi << 16, t[1][i / 2] |= lo << 16;
                        }
                        if (r < rows) {
                            uint8_t* at = q_at + tile_off<C::BOX, kBlock>(r, c);
                            *reinterpret_cast<uint4*>(at) = make_uint4(t[0][0], t[0][1], t[0][2], t[0][3]);
                            *reinterpret_cast<uint4*>(at + q_box) =
                                make_uint4(t[1][0], t[1][1], t[1][2], t[1][3]);
                            if (c == 0) sm.qs[nb & 1][r] = qs;
                        }
                    });
                } else {
                    constexpr int CH = D / 8, STEP = 64 / CH;   // 16-byte chunks of a row; rows a pass
                    const int c = t64 % CH;
                    const uint32_t dst = smem_addr(q_at) + (c >> 3) * q_box;
                    each_row(t64 / CH, STEP, rows, [&](int r, const __nv_bfloat16* src) {
                        cp_async16(dst + tile_off<128, kBlock>(r, c & 7), src + 8 * c, true);
                    });
                    cp_async_commit();
                }
                if (nb == 0) pdl_wait();
                for (int r = t64; r < rows; r += 64) {
                    const int node = (r0 + r) / p.QG;
                    sm.nl[nb & 1][r] = -*stat_at(p, x.b, node, x.g * p.QG + r0 + r - node * p.QG);
                }
                if (!kFp8) cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.qready[nb & 1]);
            }
        }
    } else {
        // ---- sums: thread = position of a tile ----
        const int grp = (warp - 4) >> 2;
        const int gt = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        int nb = 0, it0 = 0;   // blocks; tiles before this block
        uint32_t phase = 0;    // of each buffer's next wait
        bool go = true;
        pdl_wait();
        while (go && next_tiles(p, run, &x)) {
            const int all = x.s.n * p.QG, nt = x.t1 - x.t0;
            float* mass = mp.mass + (static_cast<int64_t>(x.b) * p.d.Hkv + x.g) * mp.mass_stride;
            for (int rb = 0; go && rb < blocks_of(x.s); ++rb, ++nb, it0 += nt) {
                const int r0 = rb << kBlockShift, rows = min(kBlock, all - r0);
                // A warp whose group has no tile in the block goes through it all the same, and
                // no further ahead than this: block n + 2's q comes only once every warp is
                // through block n, so none arrives twice for one phase of lfree.
                if (!(go = waits(&sm.qready[nb & 1], (nb >> 1) & 1))) break;
                const float* nl = sm.nl[nb & 1];
                const float* qsr = sm.qs[nb & 1];
                for (int t = x.t0 + grp; t < x.t1; t += 2) {
                    const int pos = t * kTile + gt;
                    // what stands there: old weights, or those of the blocks before
                    float sum = 0.f;
                    if (pos < x.s.total && (rb > 0 || (pos < x.s.len && mp.decay != 0.f)))
                        sum = (rb > 0 ? 1.f : mp.decay) * mass[pos];
                    const int buf = (t - x.t0) & (mp.buffers - 1);   // (as odd as the group)
                    const uint32_t tS = lanes + (2 * kBlock / mp.buffers) * buf;
                    if (!(go = waits(&sm.dfull[buf], (phase >> buf) & 1u))) break;
                    phase ^= 1u << buf;
                    tc_fence_after();
                    const uint32_t have = static_cast<uint32_t>(sm.have[(it0 + t - x.t0) % kHave]);
                    const bool there = (have >> (gt >> p.box_shift)) & 1u;
                    // first row that sees the position: all see the cached ones, a chain's
                    // token those up to its own
                    const int from = max(0, pos - x.s.len) * p.QG - r0;
                    const bool cut = (t + 1) * kTile > x.s.len + 1;
                    F2 acc[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
                    auto chunk = [&](const uint32_t* v, int c0, bool check) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 n4 = *reinterpret_cast<const float4*>(nl + c0 + c);
                            float4 q4 = make_float4(p.qscale, p.qscale, p.qscale, p.qscale);
                            if (kFp8) q4 = *reinterpret_cast<const float4*>(qsr + c0 + c);
                            float2 y[2];
                            y[0] = split(fma2(f2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                              f2(q4.x, q4.y), f2(n4.x, n4.y)));
                            y[1] = split(fma2(f2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])),
                                              f2(q4.z, q4.w), f2(n4.z, n4.w)));
                            if (check) {
                                const int r = c0 + c;
                                if (r < from || r >= rows) y[0].x = -INFINITY;
                                if (r + 1 < from || r + 1 >= rows) y[0].y = -INFINITY;
                                if (r + 2 < from || r + 2 >= rows) y[1].x = -INFINITY;
                                if (r + 3 < from || r + 3 >= rows) y[1].y = -INFINITY;
                            }
                            acc[0] = add2(acc[0], f2(fast_exp2(y[0].x), fast_exp2(y[0].y)));
                            acc[1] = add2(acc[1], f2(fast_exp2(y[1].x), fast_exp2(y[1].y)));
                        }
                    };
                    for (int c0 = 0; c0 < rows; c0 += 64) {
                        uint32_t v[64];
                        tmem_ld32(tS + c0, v);
                        if (c0 + 32 < rows) tmem_ld32(tS + c0 + 32, v + 32);
                        tmem_ld_wait();
                        if (c0 + 64 >= rows) {   // all has been read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sm.dfree[buf]);
                        }
                        const bool check = cut || c0 + 64 > rows;
                        if (check) chunk(v, c0, true);
                        else chunk(v, c0, false);
                        if (c0 + 32 < rows) {
                            if (check) chunk(v + 32, c0 + 32, true);
                            else chunk(v + 32, c0 + 32, false);
                        }
                    }
                    if (rows <= 0 && lane == 0) mbar_arrive(&sm.dfree[buf]);
                    const float2 s2 = split(add2(acc[0], acc[1]));
                    if (pos < x.s.total) mass[pos] = there ? sum + (s2.x + s2.y) : sum;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.lfree[nb & 1]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 2 * kBlock);
}

template <int D, bool kFp8>
int launch(const CUtensorMap& kmap, MassParams p, int device, cudaStream_t st) {
    using C = Mt<D, kFp8>;
    auto kern = mass_tc_kernel<D, kFp8>;
    static PerDevice<int> limits;
    const int limit =
        limits.get(device, [&] { return set_max_dynamic_smem(reinterpret_cast<const void*>(kern)); });
    p.q_rows = std::min(kBlock, (p.t.T * p.t.QG + 31) / 32 * 32);
    // two blocks' q where they are small: the next item's comes while this one's tiles run
    p.q_buffers = p.q_rows <= kBlock / 2 ? 2 : 1;
    const int fixed = 1024 + kSmemHead + p.q_buffers * p.q_rows * D * 2;
    p.slots = std::min((limit - fixed) / C::SLOT, kMaxSlots);
    p.buffers = p.q_rows <= kBlock / 2 ? 4 : 2;
    if (limit < 0 || p.slots < 2) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(p.t.ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = fixed + static_cast<size_t>(p.slots) * C::SLOT;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, kmap, p);
}

}  // namespace

int launch_mass_tc(const qmm_kv_cache& c, const void* q, int64_t q_stride, int N, int T, int Hq,
                   const int* cu, float scale, const float* lse, float* mass, int64_t mass_stride,
                   float decay, int num_sms, void* stream) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return cudaErrorInvalidDevice;
    MassParams p = {};
    CUtensorMap kmap, vmap;
    const int rc = tree_setup(c, q, q_stride, nullptr, N, T, Hq, cu, nullptr, scale, nullptr, num_sms,
                              kBlockShift, kTileShift, 1, kSetup, &p.t, &kmap, &vmap);
    if (rc != cudaSuccess) return rc;
    p.t.lse = const_cast<float*>(lse);
    p.mass = mass;
    p.mass_stride = mass_stride;
    p.decay = decay;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (c.D == 128)
        return c.dtype == QMM_CACHE_E4M3 ? launch<128, true>(kmap, p, device, st)
                                         : launch<128, false>(kmap, p, device, st);
    return c.dtype == QMM_CACHE_E4M3 ? launch<64, true>(kmap, p, device, st)
                                     : launch<64, false>(kmap, p, device, st);
}

}  // namespace qmm
