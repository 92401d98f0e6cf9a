// Writes into the paged KV cache: append with the per-head norm and the
// rotary position (qmm_kv_append), and the commit of an accepted path
// (qmm_tree_accept).
//
// Append.  Per head x of D values: y = x w / sqrt(mean(x^2) + eps), then each
// pair (a, c) turns by its angle, (a cos - c sin, c cos + a sin).  A few
// operations per value read and written once: the call is bound by the bytes
// of q, k, v and the cache rows, if the instructions per value are few.  A head
// row is held by D / 8 lanes, and a lane holds four pairs: values [4 j, 4 j + 4)
// of both halves of the rotated part, or eight neighbours where pairs are
// neighbours or nothing turns.  So a pair never crosses lanes, the lane's four
// cosines and sines serve all its rows, and the arithmetic runs on two values
// an instruction (f32x2).  The first rows are asked for before the chain of
// loads (range, length, page) that says where they go.  16384 tokens of 32 q and 8
// k and v heads, D = 128: 77 us, 5.3 TB/s (a plain copy of as many bytes: 68); into an
// E4M3 cache 83 us, floor 56 (each stored value is divided by its scale); one token:
// 3.1 us in a graph, latency.
//
// Positions of several axes (qmm_kv_append_axes): pair j turns by the position of
// axis[j], so neighbouring pairs may take their cosines and sines from different rows of
// the table.  A token's threads gather them once, a value each, and share them (9001 tokens
// of 40 heads into an E4M3 cache: 49.0 us, each lane its own 50.4, timed in turn; floor 30.5.  Bound by
// instructions, 70 % of the issue slots: norm, rotation and the division by the scale).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"
#include "qmm_paged.cuh"
#include "qmm_paged_host.h"

namespace qmm {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendQ = 4;   // q rows whose loads a lane has in flight, beside a k and a v row

struct AppendParams {
    PagedDims d;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* q_out;
    void *K, *V;
    const int *cu, *positions;
    const float* cos_sin;
    const __nv_bfloat16 *q_norm, *k_norm;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int N, T, Hq;
    int per_token;  // lane groups that share a token
    int rows, dim, interleaved;
    float eps, k_scale, v_scale;
    int axes;            // positions of a token, [axes][N]
    uint32_t axis4[16];  // axis of each pair, a byte each: those of lane l's four pairs
};

// Eight BF16 values of a lane as its four pairs: a = the pairs' first values
// (two and two), c = their partners.  Interleaved: the pairs are neighbours in
// memory; otherwise lo and hi are the two halves' pieces.
struct Pairs {
    F2 a[2], c[2];
};
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
template <bool kInter>
__device__ __forceinline__ Pairs pairs_of(uint2 lo, uint2 hi) {
    Pairs p;
    if (kInter) {
        p.a[0] = f2(bf_lo(lo.x), bf_lo(lo.y)), p.c[0] = f2(bf_hi(lo.x), bf_hi(lo.y));
        p.a[1] = f2(bf_lo(hi.x), bf_lo(hi.y)), p.c[1] = f2(bf_hi(hi.x), bf_hi(hi.y));
    } else {
        p.a[0] = f2(bf_lo(lo.x), bf_hi(lo.x)), p.a[1] = f2(bf_lo(lo.y), bf_hi(lo.y));
        p.c[0] = f2(bf_lo(hi.x), bf_hi(hi.x)), p.c[1] = f2(bf_lo(hi.y), bf_hi(hi.y));
    }
    return p;
}
// The same values in memory order: lo then hi, four each.
template <bool kInter>
__device__ __forceinline__ void values_of(const Pairs& p, float x[8]) {
    const float2 a0 = split(p.a[0]), a1 = split(p.a[1]), c0 = split(p.c[0]), c1 = split(p.c[1]);
    if (kInter) {
        x[0] = a0.x, x[1] = c0.x, x[2] = a0.y, x[3] = c0.y;
        x[4] = a1.x, x[5] = c1.x, x[6] = a1.y, x[7] = c1.y;
    } else {
        x[0] = a0.x, x[1] = a0.y, x[2] = a1.x, x[3] = a1.y;
        x[4] = c0.x, x[5] = c0.y, x[6] = c1.x, x[7] = c1.y;
    }
}

// x / scale to the nearest E4M3 number, at most +-448 (ties to even)
__device__ __forceinline__ uint32_t e4m3x4(const float* x, float scale) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] / scale, x[1] / scale),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] / scale, x[3] / scale),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

template <int D, bool kFp8, bool kInter, bool kAxes>
__global__ void __launch_bounds__(kAppendThreads, 8) kv_append_kernel(const AppendParams p) {
    constexpr int L = D / 8;                        // lanes of a head row
    constexpr int kGroups = kAppendThreads / L;     // lane groups of the block
    pdl_trigger();
    const int lane = threadIdx.x % L;
    const int group = threadIdx.x / L;
    const int step = p.per_token;                   // lane groups of a token
    const int sub = group & (step - 1);
    int tok = blockIdx.x * (kGroups / step) + group / step;
    pdl_wait();
    // A group's lanes leave together or not at all; the shuffles below name
    // only the group's own lanes.  (kAxes: behind the barrier; until then a group
    // without a token looks at the last one)
    bool alive = tok < p.N;
    if (!kAxes && !alive) return;
    if (kAxes) tok = min(tok, p.N - 1);
    const uint32_t mask = ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);

    // where the lane's two pieces of four values start
    const bool turns = 8 * lane < p.dim;
    const int at_lo = !kInter && turns ? 4 * lane : 8 * lane;
    const int at_hi = !kInter && turns ? p.dim / 2 + 4 * lane : 8 * lane + 4;
    const int Hq = p.Hq, Hkv = p.d.Hkv;
    const __nv_bfloat16* qrow = p.q + tok * p.q_stride;
    const __nv_bfloat16* krow = p.k + tok * p.k_stride;
    const __nv_bfloat16* vrow = p.v + tok * p.v_stride;
    struct In {
        uint2 lo, hi;
    };
    // (ordinary loads: q_out may be q, and the read-only path is not for memory
    // that the kernel writes)
    auto load = [&](const __nv_bfloat16* row, int h) {
        In x;
        x.lo = *reinterpret_cast<const uint2*>(row + h * D + at_lo);
        x.hi = *reinterpret_cast<const uint2*>(row + h * D + at_hi);
        return x;
    };
    In qi[kAppendQ], ki, vi;
#pragma unroll
    for (int u = 0; u < kAppendQ; ++u)
        if (sub + u * step < Hq) qi[u] = load(qrow, sub + u * step);
    if (sub < Hkv) ki = load(krow, sub), vi = load(vrow, sub);

    int b, i;
    if (!p.cu) {
        b = tok / p.T;
        i = tok - b * p.T;
    } else {
        // the ranges ascend: as many of cu[1..B] as are <= tok lie before it
        int before = 0;
        for (int j = 1 + lane; j <= p.d.B; j += L) before += p.cu[j] <= tok;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) before += __shfl_xor_sync(mask, before, o);
        if (!kAxes && before >= p.d.B) return;
        alive = alive && before < p.d.B;
        b = kAxes ? min(before, p.d.B - 1) : before;
        i = tok - max(p.cu[b], 0);   // clamped as token_range does
        if (!kAxes && i < 0) return;
        alive = alive && i >= 0;
    }
    int pos_given = 0;   // kAxes: of axis `lane`
    if (kAxes) {
        if (lane < p.axes) pos_given = p.positions[static_cast<int64_t>(lane) * p.N + tok];
    } else if (p.positions) {
        pos_given = p.positions[tok];
    }
    const int len = cached_tokens(p.d, b);
    const int pos = kAxes || p.positions ? pos_given : len + i;
    const bool off_table = p.dim > 0 && (pos < 0 || pos >= p.rows);
    if (kAxes) alive = !__any_sync(mask, off_table) && alive;
    else if (off_table) return;
    // (len <= cap < 2^31 - 65535 and i < N: the sum is tested before it is used)
    const int64_t slot = static_cast<int64_t>(len) + i;
    const int64_t at = slot < p.d.cap ? slot_offset(p.d, b, static_cast<int>(slot)) : -1;

    // cosines and sines of the lane's four pairs
    F2 cs[2], sn[2], ns[2];
    if (kAxes) {
        __shared__ __align__(16) float cs_s[kGroups][D];   // by token of the block
        float* const mine = cs_s[group / step];
        if (alive)
            for (int v = sub * L + lane; v < p.dim; v += step * L) {
                const int pair = v < p.dim / 2 ? v : v - p.dim / 2;
                const int axis = (p.axis4[pair >> 2] >> (8 * (pair & 3))) & 0xffu;
                const int at_axis = p.positions[static_cast<int64_t>(axis) * p.N + tok];
                mine[v] = p.cos_sin[static_cast<int64_t>(at_axis) * p.dim + v];
            }
        __syncthreads();
        if (!alive) return;
        if (turns) {
            const float4 c4 = *reinterpret_cast<const float4*>(mine + 4 * lane);
            const float4 s4 = *reinterpret_cast<const float4*>(mine + p.dim / 2 + 4 * lane);
            cs[0] = f2(c4.x, c4.y), cs[1] = f2(c4.z, c4.w);
            sn[0] = f2(s4.x, s4.y), sn[1] = f2(s4.z, s4.w);
            ns[0] = f2(-s4.x, -s4.y), ns[1] = f2(-s4.z, -s4.w);
        }
    } else if (turns) {
        const float* row = p.cos_sin + static_cast<int64_t>(pos) * p.dim + 4 * lane;
        const float4 c4 = *reinterpret_cast<const float4*>(row);
        const float4 s4 = *reinterpret_cast<const float4*>(row + p.dim / 2);
        cs[0] = f2(c4.x, c4.y), cs[1] = f2(c4.z, c4.w);
        sn[0] = f2(s4.x, s4.y), sn[1] = f2(s4.z, s4.w);
        ns[0] = f2(-s4.x, -s4.y), ns[1] = f2(-s4.z, -s4.w);
    }
    // norm (weights w, or none) and rotation
    auto turned = [&](const In& in, const __nv_bfloat16* w, float x[8]) {
        Pairs y = pairs_of<kInter>(in.lo, in.hi);
        if (w) {
            const uint2 wl = __ldg(reinterpret_cast<const uint2*>(w + at_lo));
            const uint2 wh = __ldg(reinterpret_cast<const uint2*>(w + at_hi));
            F2 s2 = mul2(y.a[0], y.a[0]);
            s2 = fma2(y.a[1], y.a[1], s2);
            s2 = fma2(y.c[0], y.c[0], s2);
            s2 = fma2(y.c[1], y.c[1], s2);
            const float2 s1 = split(s2);
            float ss = s1.x + s1.y;
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
            const float rms = rsqrtf(ss * (1.f / D) + p.eps);
            const F2 r2 = f2(rms, rms);
            const Pairs wp = pairs_of<kInter>(wl, wh);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                y.a[j] = mul2(mul2(y.a[j], r2), wp.a[j]);
                y.c[j] = mul2(mul2(y.c[j], r2), wp.c[j]);
            }
        }
        if (turns) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const F2 a = y.a[j], c = y.c[j];
                y.a[j] = fma2(c, ns[j], mul2(a, cs[j]));
                y.c[j] = fma2(a, sn[j], mul2(c, cs[j]));
            }
        }
        values_of<kInter>(y, x);
    };

    for (int h0 = sub; h0 < Hq; h0 += kAppendQ * step) {
        if (h0 != sub) {
#pragma unroll
            for (int u = 0; u < kAppendQ; ++u)
                if (h0 + u * step < Hq) qi[u] = load(qrow, h0 + u * step);
        }
#pragma unroll
        for (int u = 0; u < kAppendQ; ++u) {
            const int h = h0 + u * step;
            if (h >= Hq) break;
            float x[8];
            turned(qi[u], p.q_norm, x);
            __nv_bfloat16* out = p.q_out + tok * p.q_out_stride + h * D;
            *reinterpret_cast<uint2*>(out + at_lo) =
                make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
            *reinterpret_cast<uint2*>(out + at_hi) =
                make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        }
    }
    if (at < 0) return;   // no slot: nothing is stored
    auto store = [&](void* pool, int h, const float x[8], float scale) {
        const int64_t e = at + h * p.d.head_stride;
        if (kFp8) {
            uint8_t* out = static_cast<uint8_t*>(pool) + e;
            *reinterpret_cast<uint32_t*>(out + at_lo) = e4m3x4(x, scale);
            *reinterpret_cast<uint32_t*>(out + at_hi) = e4m3x4(x + 4, scale);
        } else {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(pool) + e;
            *reinterpret_cast<uint2*>(out + at_lo) =
                make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
            *reinterpret_cast<uint2*>(out + at_hi) =
                make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        }
    };
    for (int h = sub; h < Hkv; h += step) {
        if (h != sub) ki = load(krow, h), vi = load(vrow, h);
        float x[8];
        turned(ki, p.k_norm, x);
        store(p.K, h, x, p.k_scale);
        const Pairs v = pairs_of<false>(vi.lo, vi.hi);
        values_of<false>(v, x);
        store(p.V, h, x, p.v_scale);
    }
}

// ---- accepted path -----------------------------------------------------------

constexpr int kAcceptThreads = 256;
constexpr int kAcceptRows = 8;  // rows a lane group has in flight

struct AcceptParams {
    PagedDims d;
    const int *tokens, *targets, *parents, *cu;
    int *path, *count, *next, *new_lens;
    int N, T, n, per_block, row_bytes, elem;
    int outputs;
    uint8_t* pools[2 * kMaxAcceptCaches];  // K and V of each cache
};

// One block: the walk of sequence blockIdx.y (every block of a sequence walks
// it: a few hundred bytes and a handful of steps, less than a second launch
// or a hand-over between blocks), then the moves of its share of the (cache,
// K or V, head) columns.  Row j takes row path[j] >= j of the same column, and
// a column belongs to one lane group that goes through j in order: a row is
// read before any later step could overwrite it, so the moves are in place.
__global__ void __launch_bounds__(kAcceptThreads)
    tree_accept_kernel(const __grid_constant__ AcceptParams p) {
    __shared__ int tok[kMaxTree], tgt[kMaxTree], par[kMaxTree], path[kMaxTree];
    __shared__ int64_t src[kMaxTree], dst[kMaxTree];  // element offsets, -1: no page
    __shared__ int count_s, moves_s;
    const int tid = threadIdx.x, b = blockIdx.y;
    pdl_trigger();
    pdl_wait();
    int first, n;
    token_range(p.cu, p.N, p.T, b, &first, &n);
    for (int i = tid; i < n; i += kAcceptThreads) {
        tok[i] = p.tokens[first + i];
        tgt[i] = p.targets[first + i];
        par[i] = p.parents ? p.parents[first + i] : i - 1;
    }
    __syncthreads();
    if (tid < 32) {
        int count = 0, cur = 0;
        if (n > 0) {
            if (tid == 0) path[0] = 0;
            count = 1;
            // children lie behind their parent: each chunk of 32 tokens is
            // looked at from cur + 1 on, and the walk ends at the last token
            for (int c0 = 1; c0 < n;) {
                const int i = c0 + tid;
                const uint32_t hit = __ballot_sync(
                    0xffffffffu, i < n && par[i] == cur && tok[i] == tgt[cur]);
                if (hit) {
                    cur = c0 + __ffs(hit) - 1;
                    if (tid == 0) path[count] = cur;
                    ++count;
                    c0 = cur + 1;
                } else {
                    c0 += 32;
                }
            }
        }
        if (tid == 0) count_s = count;
        if (p.outputs && blockIdx.x == 0 && tid == 0) {
            p.count[b] = count;
            if (p.next) p.next[b] = count > 0 ? tgt[cur] : -1;
        }
    }
    __syncthreads();
    const int count = count_s;
    const int len = cached_tokens(p.d, b);
    if (p.outputs && blockIdx.x == 0) {
        for (int j = tid; j < p.T; j += kAcceptThreads)
            p.path[static_cast<int64_t>(b) * p.T + j] = j < count ? path[j] : -1;
        // (an int holds it: len <= cap, and cap + 256 < 2^31)
        if (p.new_lens && tid == 0) p.new_lens[b] = len + count;
    }
    // the rows that move, in order
    if (tid < 32) {
        int moves = 0;
        for (int j0 = 0; j0 < count; j0 += 32) {
            const int j = j0 + tid;
            int64_t from = -1, to = -1;
            if (j < count && path[j] != j) {
                from = slot_offset(p.d, b, len + path[j]);
                to = slot_offset(p.d, b, len + j);
            }
            const bool moved = from >= 0 && to >= 0;
            const uint32_t bits = __ballot_sync(0xffffffffu, moved);
            if (moved) {
                const int at = moves + __popc(bits & ((1u << tid) - 1u));
                src[at] = from;
                dst[at] = to;
            }
            moves += __popc(bits);
        }
        if (tid == 0) moves_s = moves;
    }
    __syncthreads();
    const int moves = moves_s;
    const int lanes = p.row_bytes / 16;
    const int lane = tid % lanes;
    const int cols = 2 * p.n * p.d.Hkv;
    const int last = min(cols, (static_cast<int>(blockIdx.x) + 1) * p.per_block);
    for (int c = blockIdx.x * p.per_block + tid / lanes; c < last; c += kAcceptThreads / lanes) {
        uint8_t* pool = p.pools[c / p.d.Hkv] + (c % p.d.Hkv) * p.d.head_stride * p.elem + 16 * lane;
        for (int j0 = 0; j0 < moves; j0 += kAcceptRows) {
            uint4 x[kAcceptRows];
#pragma unroll
            for (int u = 0; u < kAcceptRows; ++u)
                if (j0 + u < moves) x[u] = *reinterpret_cast<const uint4*>(pool + src[j0 + u] * p.elem);
#pragma unroll
            for (int u = 0; u < kAcceptRows; ++u)
                if (j0 + u < moves) *reinterpret_cast<uint4*>(pool + dst[j0 + u] * p.elem) = x[u];
        }
    }
}

}  // namespace

int launch_kv_append(const qmm_kv_cache& c, const void* q, const void* k, const void* v,
                     void* q_out, int N, int Hq, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, int64_t q_out_stride, const int* cu, const int* positions,
                     const qmm_rope* rope, const qmm_rope_axes* axes, void* stream) {
    AppendParams p = {};
    p.d = paged_dims(c);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.K = c.K;
    p.V = c.V;
    p.cu = cu;
    p.positions = positions;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.N = N;
    p.T = N / c.B;
    p.Hq = Hq;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    if (rope) {
        p.cos_sin = rope->cos_sin;
        p.q_norm = static_cast<const __nv_bfloat16*>(rope->q_norm);
        p.k_norm = static_cast<const __nv_bfloat16*>(rope->k_norm);
        p.rows = rope->rows;
        p.dim = rope->dim;
        p.interleaved = rope->interleaved;
        p.eps = rope->eps;
    }
    if (axes) {
        p.axes = axes->axes;
        for (int j = 0; j < rope->dim / 2; ++j)
            p.axis4[j / 4] |= static_cast<uint32_t>(axes->axis[j]) << (8 * (j % 4));
    }
    // lane groups per token: one per head row where the call is small (latency:
    // one token of 8 heads 2.4 us, with fewer groups 3.0), else as few as leave
    // kAppendQ q rows, or one k and v row, a group (bytes in flight: 2452 tokens of
    // 24 heads, D = 64: 5.4 us, with a group a row 6.8)
    const int groups = kAppendThreads / (c.D / 8), rows = Hq > c.Hkv ? Hq : c.Hkv;
    const bool small = static_cast<int64_t>(N) * rows <= 4 * 152 * groups;
    p.per_token = 1;
    while (p.per_token < groups &&
           (p.per_token * (small ? 1 : kAppendQ) < Hq || p.per_token < c.Hkv))
        p.per_token *= 2;
    const int tokens = groups / p.per_token;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3((N - 1) / tokens + 1, 1, 1);
    cfg.blockDim = dim3(kAppendThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    const bool fp8 = c.dtype == QMM_CACHE_E4M3, inter = rope && rope->interleaved;
    auto run = [&](auto kernel) { return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p)); };
    auto pick = [&](auto d, auto with_axes) {
        constexpr int D = decltype(d)::value;
        constexpr bool A = decltype(with_axes)::value;
        return fp8 ? (inter ? run(kv_append_kernel<D, true, true, A>) : run(kv_append_kernel<D, true, false, A>))
                   : (inter ? run(kv_append_kernel<D, false, true, A>) : run(kv_append_kernel<D, false, false, A>));
    };
    using D128 = std::integral_constant<int, 128>;
    using D64 = std::integral_constant<int, 64>;
    if (axes)
        return c.D == 128 ? pick(D128{}, std::true_type{}) : pick(D64{}, std::true_type{});
    return c.D == 128 ? pick(D128{}, std::false_type{}) : pick(D64{}, std::false_type{});
}

int launch_tree_accept(const qmm_kv_cache* caches, int n, const int* tokens, const int* targets,
                       const int* parents, const int* cu, int N, int T, int* path, int* count,
                       int* next, int* new_lens, bool outputs, void* stream) {
    const qmm_kv_cache& c = caches[0];
    AcceptParams p = {};
    p.d = paged_dims(c);
    p.tokens = tokens;
    p.targets = targets;
    p.parents = parents;
    p.cu = cu;
    p.path = path;
    p.count = count;
    p.next = next;
    p.new_lens = new_lens;
    p.N = N;
    p.T = T;
    p.n = n;
    p.elem = c.dtype == QMM_CACHE_E4M3 ? 1 : 2;
    p.row_bytes = c.D * p.elem;
    p.outputs = outputs;
    for (int i = 0; i < n; ++i) {
        p.pools[2 * i] = static_cast<uint8_t*>(caches[i].K);
        p.pools[2 * i + 1] = static_cast<uint8_t*>(caches[i].V);
    }
    // columns per block: a block's walk and table look-ups take longer than its
    // moves, so the blocks fill the SMs once (4 of them each) and no more (64
    // sequences, 36 layers: 13.9 us; 2 blocks an SM 17.9, 8 15.6)
    const int64_t cols = static_cast<int64_t>(2) * n * c.Hkv;
    const int groups = kAcceptThreads / (p.row_bytes / 16);
    const int64_t share = (cols * c.B - 1) / (4 * 152) + 1;
    p.per_block = static_cast<int>((share - 1) / groups + 1) * groups;
    while ((cols - 1) / p.per_block + 1 > 65535) p.per_block *= 2;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(static_cast<unsigned>((cols - 1) / p.per_block + 1), c.B, 1);
    cfg.blockDim = dim3(kAcceptThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    return cudaLaunchKernelEx(&cfg, tree_accept_kernel, p);
}

}  // namespace qmm
