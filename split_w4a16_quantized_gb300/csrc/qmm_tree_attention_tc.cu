// Tree attention for more than 8 query rows per KV head (qmm_tree_attention):
// the products on the 5th-generation tensor cores.
//
// The formulas and the work split are those of qmm_tree_attention.cu.  Here a
// work item is up to 128 or 256 rows, the MMA's M once or twice, and a tile is
// 64 positions:
//   S [128 x 64] = Q [128 x D] K^T    Q and the K tile in shared memory
//   O [128 x D] += P [128 x 64] V     P in tensor memory, V in shared memory
// with S and O accumulated in tensor memory.  Rows past the item's are computed
// and dropped: at 128 rows a tile's products (630 clocks, D = 128) take half the
// time its K and V take from HBM, so padding costs little where there are few
// rows.
//
// Roles of a CTA:
//   warp 0      copies: K and V tiles into a ring each
//   warp 1      issues the MMAs and owns the tensor memory
//   warps 2-3   bring the next item's q; E4M3 cache: turn V tiles into F16
//   one or two softmax groups of 128 threads, a thread a row; E4M3 cache: turn
//     their rows of q into two terms first
// A group has two buffers of S: while it turns one into P, the products of the
// other run, and with them the 130 to 480 clocks a commit takes to be seen.  P
// overwrites S in place (BF16 or F16 in half the columns).
//   MMA order of a group:  ... P(i) V(i), Q K(i+2) | P(i+1) V(i+1), Q K(i+3) ...
//   up to 128 rows: one group, two CTAs per SM, because each item ends with a few
//     thousand clocks in which its last products drain and its output is
//     written; the other CTA's products and copies run on meanwhile.
//   up to 256 rows: two groups with half of the rows each, which use the same K
//     and V tiles; one CTA per SM.
//
// An item's first scores need only its q and K: they are issued right behind
// the last products of the item before, while the group still writes that
// item's output.
//
// A row's maximum is followed lazily: P = 2^(s - ref) with a reference that is
// raised only when a score passes it by more than 8, so P stays below 2^8 and O
// is rescaled a few times per item instead of every tile.  The result is the
// same but for rounding: sums are FP32, P is rounded to BF16 (F16 for an E4M3
// cache) whatever its scale.  One BF16 term of P, where the kernel for few rows
// keeps two: its error is that of rounding the output (RMS 0.0022 of the outputs'
// RMS, with the second term 0.0017), and the second term would double the P V
// products: 16 sequences of 64 tokens 166 us instead of 128, 64 ragged ones of up to
// 5 tokens, D = 64, 142 instead of 118, 8 of 8 tokens 25.5 instead of 24.1.
// With shared prefixes (kShared) a BF16 cache's P keeps both terms: most of those calls
// are decode, a sequence's few rows are here for its neighbours' sake alone, and the
// tensor cores have room (64 sequences behind 8192 tokens: 46 us, with one term 42; 48 of
// 4 tokens behind five prefixes, D = 64: 105 and 88; error against 64 bits 0.00165 and
// 0.00226 of the outputs' RMS).  The second term takes the half of S that the first
// leaves.  An E4M3 cache's P is one F16 term there too: a second would take 73 us instead
// of 65 (24 sequences of up to 8 tokens behind 16000) for an error of 0.001665 instead of
// 0.001676, both of them the rounding of the output.
//
// What bounds it (152 SMs; a tile is 64 positions, D = 128; clocks a tile are those
// that 8000 more positions add to a history of 4000, 19 sequences of 8 KV heads).
//   BF16, up to 128 rows: HBM; 32 sequences of 16 tokens (64 rows), 500 to 16000
//     positions: 106 us, 5.8 TB/s.  Short ones: the start (5 us to the first
//     scores: plan, table, copy) and the merge; 8 of 8 tokens, 1500 to 4000:
//     24 us, floor 12.6.
//   BF16, 256 rows: the tensor cores with the hand-overs between their issue and
//     the softmax; 16 sequences of 64 tokens, 8000 positions: 122 to 129 us with the
//     merge, 1.05 to 1.11 PFLOP/s.  1,580 clocks a tile, of which an SM's products
//     need 1,240, 620 a group (measured alone and beside the softmax's tensor-memory
//     traffic); starting and ending takes as long as 20 tiles.
//   E4M3, up to 128 rows: shared memory.  The products read q again for every
//     tile (two terms, 32 KB) and V is converted through it (8 KB read, 16
//     written, 16 read): with K and the copies 104 KB, 830 clocks of an SM's
//     bandwidth a tile, of 900; 32 sequences of 16 tokens: 83 us, 3.7 TB/s.
//   E4M3, 256 rows: 1,660 clocks a tile, more than BF16's; 32 sequences of 64 tokens,
//     500 to 16000 positions: 153 us, floor 81.  The tensor pipe is active in 47 % of
//     the clocks and 1.8 instructions are issued a clock: neither is full, the two
//     groups and the conversion of V wait for one another.
//
// E4M3 cache.  Q K^T runs on the 8-bit keys as they are: a BF16 number has 8
// significant bits, so a row of q, scaled by a power of two to a maximum in
// [128, 256), is the sum of two E4M3 numbers, exactly for what lies within 2^-9
// of the row's maximum and to 2^-17 of that maximum below.  P V needs more bits
// of P than two E4M3 terms give far below the maximum (a long flat tail under
// one large weight would vanish), so V is converted to F16, exactly, and P is
// F16, times 2^7: at most 2^15, and 11 bits down to 2^-21 of the reference.
#include <algorithm>

#include "qmm.h"
#include "qmm_per_device.h"
#include "qmm_tree_tc.cuh"

namespace qmm {
namespace {

constexpr int kConvWarps = 2;
constexpr int kTile = 1 << kTcTileShift;   // positions
constexpr int kMaxSlots = 8;        // of one ring
constexpr int kHave = 32;           // tiles whose page bits are kept
constexpr float kLazy = 8.f;        // log2 units a score may pass the reference by

// kGroups: softmax groups (1: two CTAs per SM, up to 128 rows; 2: one CTA, 256).
template <int D, bool kFp8, int kGroups>
struct Tc {
    static constexpr int CTAS_PER_SM = kGroups == 1 ? 2 : 1;
    static constexpr int SOFTMAX0 = 4;                       // first softmax warp
    static constexpr int THREADS = 128 + 128 * kGroups;
    static constexpr int ROW = D * (kFp8 ? 1 : 2);           // bytes of a cache row
    static constexpr int BOX = ROW < 128 ? ROW : 128;        // row bytes of one copy
    static constexpr int BOXES = ROW / BOX;
    static constexpr int SLOT = kTile * ROW;                 // a copied tile
    static constexpr int CONV = kTile * D * 2;               // a converted V tile
    // tensor memory: two S/P buffers of each group, then an O of each
    static constexpr uint32_t COLS = 256 * kGroups, COL_O = 2 * kTile * kGroups;
    static_assert(kGroups * (2 * kTile + D) <= static_cast<int>(COLS), "tensor memory");
};

template <int kGroups>
struct TcSmem {
    uint64_t kfull[kMaxSlots], kempty[kMaxSlots], vfull[kMaxSlots], vempty[kMaxSlots];
    uint64_t cfull[2], cempty[2];
    uint64_t sfull[2 * kGroups];        // a buffer's next S is there
    uint64_t pready[2 * kGroups];       // its P is, and O may take the product
    uint64_t pvdone[kGroups];           // a group's product with V has ended
    uint64_t ofull[kGroups];            // a group's O is complete
    uint64_t qraw;                      // E4M3: an item's q is there, as BF16
    uint64_t qready, qfree;             // q is there; the item's products have read it
    uint64_t odone;                     // an item's O has been read by all
    uint64_t drained;                   // abort: every MMA issued has ended
    uint32_t tmem;
    int abort;
    int have[kHave];                    // pages of a tile that exist, one bit a copy
    int pages[2][16];                   // of the tiles being copied
    int16_t par[kMaxTree];
    alignas(16) uint4 stage[4 * kGroups][128];   // by warp: 32 rows x 32 BF16 columns of O
    uint32_t anc[128 * kGroups][kWords + 1];     // a thread's own row: ancestors and itself
    RunShared run;
};
template <int kGroups>
constexpr int kSmemHead = (sizeof(TcSmem<kGroups>) + 1023) / 1024 * 1024;

// A V tile of kRows positions as B, N-major with the 128-byte swizzle: rows are
// positions (the MMA's K), 64 values of the head wide; the next 64 values are
// kRows rows on (leading offset), the next 8 positions 1024 bytes (stride
// offset).
template <int kRows>
__device__ __forceinline__ uint64_t sdesc_n_major(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
           (static_cast<uint64_t>((kRows * 128) >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// What a pair of weights leaves of its first BF16 terms (`w`), as a pair of second ones.
__device__ __forceinline__ uint32_t rest_of(float a, float b, uint32_t w) {
    return pack_bf16x2(a - __uint_as_float(w << 16), b - __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint64_t low_bits(int n) {
    return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
}

// 64 of a row's bits, from bit `from` on (negative: zeros first).
__device__ __forceinline__ uint64_t bits_from(const uint32_t* anc, int from) {
    const int lead = from < 0 ? -from : 0;
    if (lead >= 64) return 0;
    if (from < 0) from = 0;
    uint64_t bits = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int w = (from >> 5) + k;
        const uint64_t b = w < kWords ? anc[w] : 0u;
        const int sh = 32 * k - (from & 31);
        bits |= sh >= 0 ? (sh < 64 ? b << sh : 0ull) : b >> -sh;
    }
    return bits << lead;
}

// Shared memory of a launch.  q_rows: rows kept of a group's Q (32, 64 or 128:
// the products read 128, and what follows stands for the rest, which nobody
// looks at).
struct Layout {
    int q_rows, conv_slots, k_slots, v_slots;
};

// kShared: with shared prefixes in the list of work; every item leaves a state, and a BF16
// cache's P is two terms.
template <int D, bool kFp8, int kGroups, bool kShared>
__global__ void __launch_bounds__(Tc<D, kFp8, kGroups>::THREADS, Tc<D, kFp8, kGroups>::CTAS_PER_SM)
    tree_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeParams p,
                   const Layout lay) {
    using C = Tc<D, kFp8, kGroups>;
    constexpr bool kTwo = kShared && !kFp8;   // P as two terms
    extern __shared__ uint8_t tree_tc_smem_raw[];
    uint8_t* base_s = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(tree_tc_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    TcSmem<kGroups>& sm = *reinterpret_cast<TcSmem<kGroups>*>(base_s);
    uint8_t* q_s = base_s + kSmemHead<kGroups>;
    const int q_box = lay.q_rows * C::BOX, q_bytes = lay.q_rows * D * 2;   // BF16, or two E4M3 terms
    uint8_t* conv_s = q_s + kGroups * q_bytes;
    uint8_t* k_s = conv_s + lay.conv_slots * C::CONV;
    uint8_t* v_s = k_s + lay.k_slots * C::SLOT;
    volatile int* abort = &sm.abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        sm.abort = 0;
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&sm.kfull[i], 1);
            mbar_init(&sm.kempty[i], 1);
            mbar_init(&sm.vfull[i], 1);
            mbar_init(&sm.vempty[i], kFp8 ? kConvWarps : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.cfull[i], kConvWarps);
            mbar_init(&sm.cempty[i], 1);
        }
        for (int s = 0; s < 2 * kGroups; ++s) {
            mbar_init(&sm.sfull[s], 2);    // the commit, and the issuing thread
            mbar_init(&sm.pready[s], 4);
        }
        for (int g = 0; g < kGroups; ++g) {
            mbar_init(&sm.pvdone[g], 1);
            mbar_init(&sm.ofull[g], 1);
        }
        mbar_init(&sm.qraw, 2);
        mbar_init(&sm.qready, kFp8 ? 4 * kGroups : 2);
        mbar_init(&sm.qfree, 1);
        mbar_init(&sm.odone, 4 * kGroups);
        mbar_init(&sm.drained, 1);
        mbar_fence_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    prefetch_plan(p, tid, C::THREADS);
    // Tensor memory is taken after the kernels before this one have ended, and
    // the next may start only once it is taken: a CTA that holds tensor memory
    // never waits for one that still needs it.
    pdl_wait();
    if (warp == 1) {
        tmem_alloc(&sm.tmem, C::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = sm.tmem;
    Run run = find_run<C::THREADS, kShared>(p, sm.run);
    const int pieces = kTile >> p.box_shift;
    Stretch x = {};
    // (test_wait answers in 60 clocks where the phase is complete, as it mostly
    // is; try_wait takes 170)
    auto wait_one = [&](uint64_t* bar, int phase) {
        return mbar_probe(bar, phase) || mbar_wait(bar, phase, abort, p.status);
    };
    auto waits = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, mbar_probe(bar, phase)) ||
               mbar_wait_warp(bar, phase, abort, p.status);
    };

    if (warp < C::SOFTMAX0) {
        if (warp == 0) {
            // ---- copies: one thread waits and issues (a vote or a block of its own
            // for each would cost 200 clocks, a sixth of a tile's time) ----
            // K runs a tile ahead of V, as the products want them (8 sequences of 8
            // tokens: 24.3 us, in step 26.4); not where V has yet to be converted
            // (E4M3, 32 of 16 tokens: in step 86, ahead 91) or tiles are half as
            // large (D = 64, 64 ragged of up to 5: in step 118, ahead 122).
            constexpr int kLead = kFp8 || D == 64 ? 0 : 1;
            Cursor kc, vc;
            int nk = 0, nv = 0;   // of the issuing thread: tiles of K and of V
            int it = 0;           // tiles of K
            int zeroed = 0;       // (BF16) V slots until one that was zeroed in part comes round
            bool ok = true;
            auto copy = [&](const CUtensorMap* map, uint64_t* bar, uint8_t* slot, int t) {
                mbar_arrive_expect_tx(bar, C::SLOT);
                copy_tile<kTile, C::BOXES, C::BOX, C::BOX / (kFp8 ? 1 : 2)>(
                    p, map, bar, smem_addr(slot), sm.pages[t & 1], t, x.g);
            };
            while (ok && next_stretch<kShared>(p, run, &x)) {
                PageWalk<kTile> walk;
                walk.template start<kShared>(p, x, lane);
                for (int t = x.t0 - kLead; ok && t < x.t1; ++t) {
                    const bool more = t + kLead < x.t1;
                    uint32_t have = 0;
                    if (more) have = walk.tile(p, t + kLead, lane, sm.pages[(t + kLead) & 1]);
                    if (elect_one()) {
                        bool go = true;
                        if (more && (go = wait_one(&sm.kempty[kc.slot], kc.phase ^ 1))) {
                            sm.have[it % kHave] = static_cast<int>(have);
                            copy(&kmap, &sm.kfull[kc.slot], k_s + kc.slot * C::SLOT, t + kLead);
                            ++nk;
                        }
                        if (go && t >= x.t0 && wait_one(&sm.vempty[vc.slot], vc.phase ^ 1)) {
                            // the slot was converted from with ordinary loads, or
                            // zeroed in part with ordinary stores
                            if (kFp8 || zeroed > 0) fence_proxy_async_smem();
                            copy(&vmap, &sm.vfull[vc.slot], v_s + vc.slot * C::SLOT, t);
                            ++nv;
                        }
                    }
                    if (more) {
                        kc.next(lay.k_slots);
                        ++it;
                    }
                    if (t >= x.t0) {
                        zeroed = (t + 1) * kTile > x.s.total ? lay.v_slots : max(0, zeroed - 1);
                        vc.next(lay.v_slots);
                    }
                    ok = !__any_sync(0xffffffffu, *abort);
                }
            }
            if (!ok && elect_one()) {  // let the copies in flight land before the CTA exits
                for (int j = max(0, nk - lay.k_slots); j < nk; ++j)
                    mbar_wait(&sm.kfull[j % lay.k_slots], (j / lay.k_slots) & 1, nullptr, p.status);
                for (int j = max(0, nv - lay.v_slots); j < nv; ++j)
                    mbar_wait(&sm.vfull[j % lay.v_slots], (j / lay.v_slots) & 1, nullptr, p.status);
            }
        } else if (warp == 1) {
            // ---- MMAs ----
            constexpr uint32_t iqk = idesc(kTile, kFp8 ? 0u : 1u, false);
            constexpr uint32_t ipv = idesc(D, kFp8 ? 0u : 1u, true);
            const uint64_t q_desc = sdesc_k_major<C::BOX>(smem_addr(q_s));
            const uint64_t k_desc = sdesc_k_major<C::BOX>(smem_addr(k_s));
            const uint64_t v_desc = sdesc_n_major<kTile>(smem_addr(kFp8 ? conv_s : v_s));
            uint64_t* vfull = kFp8 ? sm.cfull : sm.vfull;
            uint64_t* vempty = kFp8 ? sm.cempty : sm.vempty;
            constexpr int VSLOT = kFp8 ? C::CONV : C::SLOT;
            const int v_slots = kFp8 ? lay.conv_slots : lay.v_slots;
            Cursor kc, vc;
            int nq = 0;                     // Q's taken
            uint32_t pphase = 0;            // phase of the P of buffers 0 and 1, a bit each
            bool go = true;
            // S of group g's buffer `odd` from its rows and the K tile at kc
            auto qk = [&](int odd, int g) {
                const int s = 2 * g + odd;
                const uint64_t a = q_desc + static_cast<uint32_t>((q_bytes >> 4) * g);
                const uint64_t b = k_desc + static_cast<uint32_t>(kc.slot * C::SLOT >> 4);
                if (kFp8) {
                    // 32 values a step; q's two terms
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            umma_ss<true>(tmem + kTile * s,
                                          a + static_cast<uint32_t>((h * q_box + k * 32) >> 4),
                                          b + ((k * 32) >> 4), iqk, h > 0 || k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        umma_ss<false>(tmem + kTile * s,
                                       a + static_cast<uint32_t>(((k >> 2) * q_box + (k & 3) * 32) >> 4),
                                       b + (((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4), iqk, k > 0);
                }
                umma_commit(&sm.sfull[s]);
                // this thread has seen the tile's copy complete, and with it the
                // copy warp's page bits: hand that on
                mbar_arrive(&sm.sfull[s]);
            };
            // O of group g (+)= P of its buffer times the V tile at vc (kTwo: the first
            // terms' columns, then the second ones')
            auto pv = [&](int odd, int g, bool first) {
                const int s = 2 * g + odd;
                const uint64_t b = v_desc + static_cast<uint32_t>(vc.slot * VSLOT >> 4);
#pragma unroll
                for (int k = 0; k < (kTwo ? 2 : 1) * kTile / 16; ++k)
                    umma_bf16_tmem_a(tmem + C::COL_O + D * g, tmem + kTile * s + 8 * k,
                                     b + ((k % (kTile / 16) * 2048) >> 4), ipv, !first || k > 0);
            };
            // Two groups: one thread waits and issues, because a vote or an issuing
            // block of its own after each wait costs 200 clocks, in which the tensor
            // cores run dry (16 sequences of 64 tokens: 130 us, with votes 141).  One
            // group: the other CTA's products fill those gaps, and both CTAs' are
            // through sooner when a tile's are issued in one go by the whole warp (32
            // sequences of 16 tokens, E4M3: 86 us, one thread 91).
            constexpr bool kAlone = kGroups == 2;
            auto wait = [&](uint64_t* bar, int phase) {
                return kAlone ? wait_one(bar, phase) : waits(bar, phase);
            };
            auto issue = [&](auto&& f) {
                if (kAlone || elect_one()) f();
                if (!kAlone) __syncwarp();
            };
            if (!kAlone || elect_one()) {
                while (go && next_stretch<kShared>(p, run, &x)) {
                    const int nt = x.t1 - x.t0;
                    if (!(go = wait(&sm.qready, nq & 1))) break;
                    // the first S of each buffer
                    for (int i = 0; i < min(nt, 2); ++i) {
                        if (!(go = wait(&sm.kfull[kc.slot], kc.phase))) break;
                        tc_fence_after();
                        issue([&] {
#pragma unroll
                            for (int g = 0; g < kGroups; ++g) qk(i, g);
                            umma_commit(&sm.kempty[kc.slot]);
                            if (i + 1 == nt) umma_commit(&sm.qfree);
                        });
                        kc.next(lay.k_slots);
                    }
                    // O is free once the last stretch's has been read
                    if (go && nq > 0) go = wait(&sm.odone, (nq - 1) & 1);
                    ++nq;
                    for (int i = 0; go && i < nt; ++i) {
                        const int odd = i & 1;
                        const bool more = i + 2 < nt;   // the buffer gets another S
                        auto next_s = [&](int g) {
                            qk(odd, g);
                            if (g == kGroups - 1) umma_commit(&sm.kempty[kc.slot]);
                            if (g == kGroups - 1 && i + 3 == nt) umma_commit(&sm.qfree);
                        };
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) {
                            if (!(go = wait(&sm.pready[2 * g + odd], (pphase >> odd) & 1))) break;
                            if (g == 0 && !(go = wait(&vfull[vc.slot], vc.phase))) break;
                            // K has come by now, as a rule
                            const bool k_here =
                                !kAlone && more &&
                                __all_sync(0xffffffffu, mbar_probe(&sm.kfull[kc.slot], kc.phase));
                            tc_fence_after();
                            issue([&] {
                                pv(odd, g, i == 0);
                                if (g == kGroups - 1) umma_commit(&vempty[vc.slot]);
                                umma_commit(&sm.pvdone[g]);
                                if (i + 1 == nt) umma_commit(&sm.ofull[g]);
                                if (k_here) next_s(g);
                            });
                            if (more && !k_here) {
                                if (g == 0 && !(go = wait(&sm.kfull[kc.slot], kc.phase))) break;
                                issue([&] { next_s(g); });
                            }
                        }
                        pphase ^= 1u << odd;
                        vc.next(v_slots);
                        if (more) kc.next(lay.k_slots);
                    }
                }
                if (!go) {  // MMAs in flight end before the tensor memory goes back
                    issue([&] { umma_commit(&sm.drained); });
                    mbar_wait(&sm.drained, 0, nullptr, p.status);
                }
            }
            __syncwarp();
        } else {
            // ---- q of each item to shared memory, then its V tiles to F16 ----
            const int t64 = tid - 64;
            Cursor vc, cc;
            bool go = true;
            for (int k = 0; go && next_stretch<kShared>(p, run, &x); ++k) {
                const int rows = min(1 << p.row_shift, x.s.n * p.QG - x.row0);
                if (k > 0 && !waits(&sm.qfree, (k - 1) & 1)) break;
                if (k > 0) fence_proxy_async_smem();
                const __nv_bfloat16* q0 = p.q + x.s.first * p.q_stride + x.g * p.QG * D;
                // this thread's rows, STEP apart, without a division each: a row
                // further is D values on, a token further q_stride - QG D more
                auto each_row = [&](int start, int step, auto&& f) {
                    int node = row_node<kShared>(p, x.row0 + start);
                    int head = x.row0 + start - node * p.QG;
                    const __nv_bfloat16* src = q0 + node * p.q_stride + head * D;
                    const int dn = row_node<kShared>(p, step), dh = step - dn * p.QG;
                    const int64_t by = dn * p.q_stride + dh * D, wrap = p.q_stride - p.QG * D;
#pragma unroll 4
                    for (int r = start; r < rows; r += step) {
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
                    // A row's BF16 values are copied to where its two E4M3 terms
                    // will stand (as many bytes): the softmax threads turn them in
                    // place.
                    constexpr int LPR = D / 16, STEP = 64 / LPR;
                    const int c = t64 % LPR;
                    auto place = [&](int r) {
                        return q_s + (r >> 7) * q_bytes + tile_off<C::BOX, 128>(r & 127, c);
                    };
                    each_row(t64 / LPR, STEP, [&](int r, const __nv_bfloat16* src) {
                        const uint32_t dst = smem_addr(place(r));
                        cp_async16(dst, src + 16 * c, true);
                        cp_async16(dst + q_box, src + 16 * c + 8, true);
                    });
                    cp_async_commit();
                    cp_async_wait<0>();
                } else {
                    constexpr int CH = D / 8;        // 16-byte chunks of a row
                    constexpr int STEP = 64 / CH;    // rows a pass
                    const int c = t64 % CH;
                    const uint32_t dst = smem_addr(q_s);
                    each_row(t64 / CH, STEP, [&](int r, const __nv_bfloat16* src) {
                        cp_async16(dst + (r >> 7) * q_bytes + (c >> 3) * q_box +
                                       tile_off<128, 128>(r & 127, c & 7),
                                   src + 8 * c, true);
                    });
                    cp_async_commit();
                    cp_async_wait<0>();
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(kFp8 ? &sm.qraw : &sm.qready);
                // a thread takes a position
                for (int t = x.t0; kFp8 && t < x.t1; ++t) {
                    const int valid = x.s.total - t * kTile;
                    if (!(go = waits(&sm.vfull[vc.slot], vc.phase))) break;
                    if (!(go = waits(&sm.cempty[cc.slot], cc.phase ^ 1))) break;
                    const uint8_t* src = v_s + vc.slot * C::SLOT;
                    uint8_t* dst = conv_s + cc.slot * C::CONV;
#pragma unroll
                    for (int c0 = 0; c0 < D / 16; c0 += 4) {
                        uint4 in[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            in[c] = *reinterpret_cast<const uint4*>(
                                src + tile_off<C::BOX, kTile>(t64, c0 + c));
                            // slots past the last position may hold anything, and
                            // 0 * NaN is not 0
                            if (t64 >= valid) in[c] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t w[4] = {in[c].x, in[c].y, in[c].z, in[c].w};
                            uint32_t f[8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                f[2 * i] = e4m3x2_to_f16x2(w[i] & 0xffffu);
                                f[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
                            }
                            const int o = 2 * (c0 + c);
                            *reinterpret_cast<uint4*>(dst + tile_off<128, kTile>(t64, o)) =
                                make_uint4(f[0], f[1], f[2], f[3]);
                            *reinterpret_cast<uint4*>(dst + tile_off<128, kTile>(t64, o + 1)) =
                                make_uint4(f[4], f[5], f[6], f[7]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.vempty[vc.slot]);
                        mbar_arrive(&sm.cfull[cc.slot]);
                    }
                    vc.next(lay.v_slots);
                    cc.next(lay.conv_slots);
                }
            }
        }
    } else {
        // ---- softmax groups ----
        const int g = (warp - C::SOFTMAX0) >> 2;          // group
        const int gt = (warp & 3) * 32 + lane;            // thread of the group = tensor memory lane
        const uint32_t quarter = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t tO = quarter + C::COL_O + D * g;
        int base = 0;             // tiles of the run before this stretch
        int no = 0;               // O's taken
        uint32_t sphase = 0;      // phase of each buffer's S, a bit each
        int anc_b = -1, anc_row = 0;   // whose rows' ancestors stand in sm.anc
        uint32_t* const anc = sm.anc[tid - 32 * C::SOFTMAX0];
        for (int k = 0; next_stretch<kShared>(p, run, &x); ++k) {
            const int nt = x.t1 - x.t0;
            const int rows = min(1 << p.row_shift, x.s.n * p.QG - x.row0);
            const int r = gt + 128 * g;   // row of the item
            const bool on = r < rows;
            const bool warp_on = __any_sync(0xffffffffu, on);
            const int row = x.row0 + (on ? r : 0);
            const int node = row_node<kShared>(p, row), head = x.g * p.QG + row - node * p.QG;
            // ---- E4M3: the row of q as two terms ----
            float qs = p.qscale;
            if (kFp8) {
                if (waits(&sm.qraw, k & 1) && on) {
                    uint8_t* const row_s = q_s + g * q_bytes;
                    uint32_t big = 0;   // largest magnitude, as bits: NaN above all
#pragma unroll 4
                    for (int c = 0; c < D / 16; ++c)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 w = *reinterpret_cast<const uint4*>(
                                row_s + h * q_box + tile_off<C::BOX, 128>(gt, c));
                            big = bf16_magnitude(bf16_magnitude(big, w.x), w.y);
                            big = bf16_magnitude(bf16_magnitude(big, w.z), w.w);
                        }
                    const float up = e4m3_scaling(big, &qs);
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint4* const at = reinterpret_cast<uint4*>(row_s + tile_off<C::BOX, 128>(gt, c));
                        uint4* const at2 = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(at) + q_box);
                        const uint4 a = *at, b = *at2;
                        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                        uint32_t t[2][4];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t hi, lo;
                            e4m3_terms(w[i], up, &hi, &lo);
                            if (i % 2 == 0) t[0][i / 2] = hi, t[1][i / 2] = lo;
                            else t[0][i / 2] |= hi << 16, t[1][i / 2] |= lo << 16;
                        }
                        *at = make_uint4(t[0][0], t[0][1], t[0][2], t[0][3]);
                        *at2 = make_uint4(t[1][0], t[1][1], t[1][2], t[1][3]);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.qready);
            }
            // ---- ancestors, where the stretch reaches the drafted slots: the same
            // for all heads of a sequence ----
            if (x.t1 * kTile > x.s.len && (x.b != anc_b || x.row0 != anc_row) &&
                !(kShared && x.b < p.pre.G)) {
                anc_b = x.b;
                anc_row = x.row0;
                if (p.parents) {
                    named_bar_sync(1, 128 * kGroups);   // the last walks are done
                    for (int i = tid - 32 * C::SOFTMAX0; i < x.s.n; i += 128 * kGroups) {
                        const int v = p.parents[x.s.first + i];
                        sm.par[i] = static_cast<int16_t>(v >= 0 && v < i ? v : -1);
                    }
                    named_bar_sync(1, 128 * kGroups);
                }
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    anc[j] = p.parents ? 0u : static_cast<uint32_t>(low_bits(node + 1 - 32 * j));
                if (p.parents)
                    for (int i = node; i >= 0; i = sm.par[i]) anc[i >> 5] |= 1u << (i & 31);
            }

            float ref = -INFINITY, sum = 0.f;

            // One tile in the group's buffer s; `at` counts the tiles of the run.
            auto tile = [&](int s, int t, int at) {
                const uint32_t tS = quarter + kTile * (2 * g + s);
                uint32_t v[kTile];
#pragma unroll
                for (int c = 0; c < kTile; c += 32) tmem_ld32(tS + c, v + c);
                // what the row sees of the tile
                const uint32_t have = static_cast<uint32_t>(sm.have[at % kHave]);
                const int j0 = t * kTile - x.s.len;   // drafted token of the first position
                const int valid = x.s.total - t * kTile;
                const bool cut = j0 + kTile > 0 || have != (1u << pieces) - 1u;
                tmem_ld_wait();
                if (cut) {
#pragma unroll
                    for (int h = 0; h < kTile; h += 64) {
                        // history, then the ancestors
                        uint64_t see = ~0ull;
                        const int j = j0 + h;
                        if (j + 64 > 0)
                            see = (low_bits(-j) | bits_from(anc, j)) & low_bits(valid - h);
                        for (int q = 0; q < pieces; ++q)
                            if (!((have >> q) & 1u)) {
                                const int lo = (q << p.box_shift) - h;
                                see &= ~(low_bits(lo + (1 << p.box_shift)) & ~low_bits(lo));
                            }
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!((see >> c) & 1ull)) v[h + c] = 0xff800000u;   // -inf
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kTile; c += 2)
                    mx[c / 2 & 3] = max3(mx[c / 2 & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * qs;
                // raise the reference, row by row: a row's result must not depend
                // on its neighbours (those past the item's rows hold anything)
                const bool raise = on && top > ref + kLazy;
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise ? fast_exp2(ref - top) : 1.f;
                    sum *= f;
                    if (raise) ref = top;
                    if (t > x.t0) {
                        // (this S's products ran ahead of the last P V)
                        waits(&sm.pvdone[g], (at - 1) & 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t w[16];
                            tmem_ld16(tO + c, w);
                            tmem_ld_wait();
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                w[q] = __float_as_uint(__uint_as_float(w[q]) * f);
                            tmem_st16(tO + c, w);
                        }
                        tmem_st_wait();
                    }
                }
                const float sub = finite_max(ref) - (kFp8 ? kTcLift : 0.f);
                const F2 q2 = f2(qs, qs), s2 = f2(-sub, -sub);
                F2 part[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
                constexpr int kPart = kTwo ? 16 : 32;   // (with two terms 32 spill)
#pragma unroll
                for (int h = 0; h < kTile; h += kPart) {
                    uint32_t pw[kPart / 2], pl[kPart / 2];
#pragma unroll
                    for (int c = 0; c < kPart; c += 2) {
                        const float2 y = split(fma2(
                            f2(__uint_as_float(v[h + c]), __uint_as_float(v[h + c + 1])), q2, s2));
                        const float a = fast_exp2(y.x), b = fast_exp2(y.y);
                        part[c / 2 & 1] = add2(part[c / 2 & 1], f2(a, b));
                        pw[c / 2] = kFp8 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
                        if (kTwo) pl[c / 2] = rest_of(a, b, pw[c / 2]);
                    }
                    if constexpr (kTwo) {
                        tmem_st8(tS + h / 2, pw);
                        tmem_st8(tS + kTile / 2 + h / 2, pl);
                    } else {
                        tmem_st16(tS + h / 2, pw);
                    }
                }
                const float2 more = split(add2(part[0], part[1]));
                sum += more.x + more.y;
                tmem_st_wait();
            };

            for (int i = 0; i < nt; ++i) {
                const int s = i & 1;
                if (!waits(&sm.sfull[2 * g + s], (sphase >> s) & 1)) break;
                sphase ^= 1u << s;
                tc_fence_after();
                const int t = x.t0 + i;
                const int valid = x.s.total - t * kTile;
                if (!kFp8 && valid < kTile) {
                    // slots past the last position may hold anything, and 0 * NaN
                    // is not 0: their V rows become zeros before P V reads them
                    const int j = base + i;
                    if (!waits(&sm.vfull[j % lay.v_slots], (j / lay.v_slots) & 1)) break;
                    uint8_t* v = v_s + (j % lay.v_slots) * C::SLOT;
                    for (int c = gt; c < (kTile - valid) * (C::ROW / 16); c += 128)
                        *reinterpret_cast<uint4*>(
                            v + tile_off<C::BOX, kTile>(valid + c / (C::ROW / 16), c % (C::ROW / 16))) =
                            make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                if (warp_on) tile(s, t, base + i);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.pready[2 * g + s]);
            }
            base += nt;
            waits(&sm.ofull[g], no & 1);
            ++no;
            tc_fence_after();
            // ---- O, or the partial state ----
            const bool whole = x.t0 == 0 && x.t1 == x.s.tiles;
            const bool writes = on && !*abort;
            if (warp_on && !whole) {
                const PartialAt part = partial_at<D>(p, 2 * blockIdx.x + (x.t0 == 0 ? 1 : 0));
                if (writes) {
                    part.m[r] = ref;
                    part.l[r] = sum;
                }
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t y[32];
                    tmem_ld32(tO + c, y);
                    tmem_ld_wait();
                    if (writes)
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            *reinterpret_cast<uint4*>(part.at(r, c + q)) =
                                make_uint4(y[q], y[q + 1], y[q + 2], y[q + 3]);
                }
            } else if (kShared) {
                const DirectAt at = direct_at<D>(
                    p, x.b < p.pre.G, static_cast<int64_t>(x.s.first + node) * p.Hq + head);
                if (writes) {
                    *at.m = ref;
                    *at.l = sum;
                }
#pragma unroll 1
                for (int c = 0; warp_on && c < D; c += 32) {
                    uint32_t y[32];
                    tmem_ld32(tO + c, y);
                    tmem_ld_wait();
                    if (writes)
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            *reinterpret_cast<uint4*>(at.o + c + q) =
                                make_uint4(y[q], y[q + 1], y[q + 2], y[q + 3]);
                }
            } else if (warp_on) {
                // a warp's 32 rows x 32 columns turn in shared memory: 8 rows of 64
                // bytes a store instead of 32 of 16
                const float inv = sum > 0.f ? p.vscale / sum : (sum == 0.f ? 0.f : sum);
                if (p.lse && writes) *stat_at(p, x.b, node, head) = stat_of(p, ref, sum);
                const int64_t row_at = static_cast<int64_t>(x.s.first + node) * p.Hq + head;
                const uint32_t mask = __ballot_sync(0xffffffffu, writes);
                uint4* const stage = sm.stage[warp - C::SOFTMAX0];
                auto swz = [](int row, int j) { return row * 4 + ((j + (row >> 1)) & 3); };
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t y[32];
                    tmem_ld32(tO + c, y);
                    tmem_ld_wait();
                    auto pair = [&](int q) {
                        return pack_bf16x2(__uint_as_float(y[q]) * inv, __uint_as_float(y[q + 1]) * inv);
                    };
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        stage[swz(lane, q)] = make_uint4(pair(8 * q), pair(8 * q + 2), pair(8 * q + 4),
                                                         pair(8 * q + 6));
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int from = q * 8 + (lane >> 2);
                        const int64_t to = __shfl_sync(0xffffffffu, row_at, from);
                        if ((mask >> from) & 1u)
                            *reinterpret_cast<uint4*>(p.O + to * D + c + 8 * (lane & 3)) =
                                stage[swz(from, lane & 3)];
                    }
                    __syncwarp();
                }
            }
            // the next stretch's P V waits for all warps
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.odone);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::COLS);
}

template <int D, bool kFp8, int kGroups, bool kShared>
int launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int device,
           cudaStream_t st) {
    using C = Tc<D, kFp8, kGroups>;
    auto kern = tree_tc_kernel<D, kFp8, kGroups, kShared>;
    static PerDevice<int> limits;
    const int limit =
        limits.get(device, [&] { return set_max_dynamic_smem(reinterpret_cast<const void*>(kern)); });
    // the rings share what Q and the converted tiles leave; two CTAs of an SM
    // have 114 KB each, 1 KB of it the system's
    const int room = C::CTAS_PER_SM == 1 ? limit : std::min(limit, 113 * 1024);
    Layout lay;
    const int rows = (kShared ? p.N : p.T) * p.QG;
    lay.q_rows = kGroups == 2 || rows > 64 ? 128 : (rows > 32 ? 64 : 32);
    const int fixed = 1024 + kSmemHead<kGroups> + kGroups * lay.q_rows * D * 2;
    // two converted tiles where that leaves two slots to either ring (32 sequences
    // of 32 tokens, 128 rows: 112 us, with one tile and three slots 119)
    lay.conv_slots = kFp8 ? ((room - fixed - 2 * C::CONV) / C::SLOT >= 4 ? 2 : 1) : 0;
    const int slots = (room - fixed - lay.conv_slots * C::CONV) / C::SLOT;
    if (limit < 0 || slots < 4) return cudaErrorInvalidValue;
    lay.v_slots = std::min(slots / 2, kMaxSlots);
    lay.k_slots = std::min(slots - lay.v_slots, kMaxSlots);
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(p.ctas, 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = fixed + static_cast<size_t>(lay.conv_slots) * C::CONV +
                           static_cast<size_t>(lay.k_slots + lay.v_slots) * C::SLOT;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p, lay);
}

template <int D, bool kFp8>
int launch_groups(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int device,
                  cudaStream_t st) {
    return p.row_shift == 7 ? launch<D, kFp8, 1, false>(kmap, vmap, p, device, st)
                            : launch<D, kFp8, 2, false>(kmap, vmap, p, device, st);
}

}  // namespace

int launch_tree_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int D,
                   bool fp8, int device, cudaStream_t st) {
    if (D == 128)
        return fp8 ? launch_groups<128, true>(kmap, vmap, p, device, st)
                   : launch_groups<128, false>(kmap, vmap, p, device, st);
    return fp8 ? launch_groups<64, true>(kmap, vmap, p, device, st)
               : launch_groups<64, false>(kmap, vmap, p, device, st);
}

int launch_prefix_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int D,
                     bool fp8, int device, cudaStream_t st) {
    if (D == 128)
        return fp8 ? launch<128, true, 1, true>(kmap, vmap, p, device, st)
                   : launch<128, false, 1, true>(kmap, vmap, p, device, st);
    return fp8 ? launch<64, true, 1, true>(kmap, vmap, p, device, st)
               : launch<64, false, 1, true>(kmap, vmap, p, device, st);
}

}  // namespace qmm
