// Attention that adds up the weight each slot receives (qmm_scored_attention).
//
//   mass[b, g, s] = decay mass[b, g, s] + sum over tokens i and heads h of g of
//                   2^(score(i, h, s) - lse(i, h))
//
// with scores in log2 units and lse = log2 sum_s 2^score.  The weights are known only
// once a row's whole history has been seen, so there are two passes over the scores:
//   up to 8 query rows per KV head (plain decode): the attention kernel leaves the scores,
//     4 bytes a row and position beside the 4 D of K and V, and the merge kernel's other
//     blocks add the weights up;
//     (32 sequences of 1024 to 8192: 89 us, floor 68, tree attention alone 78; scores formed
//     again from K 223.  64 of 300 to 12000, E4M3, D = 64, 8 rows: 88 us, floor 33: 70 the
//     attention kernel, bound as for tree attention by a tile's chain of conversions,
//     products and exp2; the scores are as many bytes as a quarter of K and V.)
//   more rows: the scores are formed again from K (qmm_mass_tc.cu), behind attention and
//     merge, which leave each row's lse.
#include "qmm.h"
#include "qmm_tree_merge.cuh"

namespace qmm {
namespace {

// ---- up to 8 rows ----
//
// One launch behind the attention kernel, whose first block wrote down what lies before
// each sequence.  The first blocks take equal runs of the batch's chunks of positions: a
// warp a row for its lse, from the states or, where one run held the item, from the
// attention kernel; then a thread 4 positions of a chunk.  The others finish the outputs
// of items that a run border cuts: a block an item or, where those are more, a border.
constexpr int kFinishThreads = 256;
static_assert(kChunk == 4 * kFinishThreads, "a thread takes 4 positions");

struct FinishParams {
    TreeParams t;
    float* mass;
    int64_t mass_stride;
    float decay;
    int adders;   // blocks that add up weights
    int by_item;  // the others take an item each, or a border between runs
};

// What lies before each sequence, of units of work and of chunks.  Up to 32 sequences:
// every warp works it out for itself, a lane a sequence, ahead of the dependency wait and
// so from L2 (one sequence of 1000: 9.7 us, as written down by the attention kernel 11.4);
// more: as written down.
struct Lists {
    const TreeParams& t;
    const bool few;
    long long units = 0, chunks = 0, all_units = 0, all_chunks = 0;   // before this lane's
    int my_units = 0;
    long long my_chunks = 0;
    __device__ __forceinline__ explicit Lists(const TreeParams& tp) : t(tp), few(tp.d.B <= 32) {
        if (!few) return;
        const int lane = threadIdx.x & 31;
        if (lane < t.d.B) {
            const Seq s = sequence<true>(t, lane);
            my_units = units_of(t, s);
            my_chunks = chunks_of(t, s);
        }
        units = warp_scan(my_units, &all_units);
        chunks = warp_scan(my_chunks, &all_chunks);
    }
    // (behind the wait)
    __device__ __forceinline__ void load() {
        if (few) return;
        all_units = t.plan[t.d.B];
        all_chunks = t.chunks[t.d.B];
    }
    __device__ __forceinline__ long long units_before(int b) const {
        return few ? __shfl_sync(0xffffffffu, units, b) : t.plan[b];
    }
    __device__ __forceinline__ long long chunks_before(int b) const {
        return few ? __shfl_sync(0xffffffffu, chunks, b) : t.chunks[b];
    }
    // The sequence that holds unit (or chunk) `at`, -1 behind the last.  Whole block.
    __device__ __forceinline__ int find(bool unit, long long at, int* found) const {
        if (few) {
            const long long from = unit ? units : chunks, n = unit ? my_units : my_chunks;
            const uint32_t hit = __ballot_sync(0xffffffffu, at >= from && at < from + n);
            return hit ? __ffs(hit) - 1 : -1;
        }
        const long long* before = unit ? t.plan : t.chunks;
        if (threadIdx.x == 0) *found = -1;
        __syncthreads();
        for (int b = threadIdx.x; b < t.d.B; b += kFinishThreads)
            if (at >= before[b] && at < before[b + 1]) *found = b;
        __syncthreads();
        return *found;
    }
};

template <int D>
__device__ __forceinline__ void finish_output(const FinishParams& p, const Lists& lists, int at) {
    constexpr int ROWS = 1 << kFewRowShift;
    __shared__ __align__(16) uint2 stage[ROWS][D / 4 + 2];
    __shared__ int found;
    const TreeParams& t = p.t;
    const int tid = threadIdx.x;
    const long long run = run_length(t, lists.all_units), unit = run * (at + 1);
    const int b = p.by_item ? at / t.d.Hkv : lists.find(true, unit, &found);
    if (b < 0) return;
    const Seq s = sequence(t, b);
    if (s.n == 0) return;
    const long long before = lists.units_before(b);
    const int g = p.by_item ? at % t.d.Hkv : static_cast<int>((unit - before) / item_units(t, s));
    const Runs c = runs_of(t, s, before, g, run);
    if (c.c0 == c.c1 || (!p.by_item && c.c0 != at)) return;   // whole, or of an earlier border
    const int rows = s.n * t.QG;
    constexpr int JUMP = kFinishThreads / ROWS;
    constexpr int TURNS = D / 4 / JUMP > 0 ? D / 4 / JUMP : 1;
    const int i = tid % ROWS, j0 = tid / ROWS;
    if (i < rows && j0 < D / 4) {
        Acc<TURNS> acc;
        acc.add_all(c.c1 - c.c0 + 1, j0, JUMP,
                    [&](int k) { return run_state<D>(t, c.c0 + k, c.c0, i); });
        const float inv = acc.inverse(t.vscale);
#pragma unroll
        for (int u = 0; u < TURNS; ++u)
            stage[i][j0 + u * JUMP] =
                make_uint2(pack_bf16x2(acc.num[u].x * inv, acc.num[u].y * inv),
                           pack_bf16x2(acc.num[u].z * inv, acc.num[u].w * inv));
    }
    __syncthreads();
    constexpr int CH = D / 8;   // 16-byte chunks of a row
    const int ri = tid / CH, ch = tid % CH;
    if (ri < rows) {
        const int node = ri / t.QG;
        const int64_t to = static_cast<int64_t>(s.first + node) * t.Hq + g * t.QG + ri - node * t.QG;
        *reinterpret_cast<uint4*>(t.O + to * D + 8 * ch) =
            *reinterpret_cast<const uint4*>(&stage[ri][2 * ch]);
    }
}

template <int D>
__global__ void __launch_bounds__(kFinishThreads, 3)
    scored_finish_kernel(const __grid_constant__ FinishParams p) {
    constexpr int ROWS = 1 << kFewRowShift;
    __shared__ float lse_s[ROWS];
    __shared__ int found;
    const TreeParams& t = p.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Lists lists(t);
    pdl_trigger();
    pdl_wait();
    lists.load();
    if (static_cast<int>(blockIdx.x) >= p.adders) {
        finish_output<D>(p, lists, static_cast<int>(blockIdx.x) - p.adders);
        return;
    }
    const long long all_chunks = lists.all_chunks, run = run_length(t, lists.all_units);
    const long long share = (all_chunks + p.adders - 1) / p.adders, start = share * blockIdx.x;
    int b = lists.find(false, start, &found);
    if (b < 0) return;
    Seq s = sequence(t, b);
    long long before = lists.units_before(b), at = start - lists.chunks_before(b);
    long long left = all_chunks - start < share ? all_chunks - start : share;
    const int all_rows = t.T * t.QG;
    while (left > 0) {
        while (at >= chunks_of(t, s)) {
            at -= chunks_of(t, s);
            if (++b >= t.d.B) return;   // (not reached: the run ends with the list)
            s = sequence(t, b);
            before = lists.units_before(b);
        }
        const int per_head = (s.total + kChunk - 1) / kChunk;
        const int g = static_cast<int>(at / per_head);
        const int k0 = static_cast<int>(at - static_cast<long long>(g) * per_head);
        const int k1 = static_cast<int>(left < per_head - k0 ? k0 + left : per_head);
        at += k1 - k0;
        left -= k1 - k0;
        const int rows = s.n * t.QG, total = s.total;
        // each row's lse
        __syncthreads();
        if (warp < rows) {
            const Runs c = runs_of(t, s, before, g, run);
            const int node = warp / t.QG;
            if (c.c0 == c.c1) {
                if (lane == 0) lse_s[warp] = *stat_at(t, b, node, g * t.QG + warp - node * t.QG);
            } else {
                float M = -INFINITY, den = 0.f;
                for (int k = c.c0 + lane; k <= c.c1; k += 32) {
                    const PartialAt x = partial_at<D>(t, 2 * k + (k == c.c0 ? 1 : 0));
                    const float m = x.m[warp], l = x.l[warp];
                    const float top = fmaxf(M, m), sub = finite_max(top);
                    den = fmaf(den, fast_exp2(M - sub), fast_exp2(m - sub) * l);
                    M = top;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const float m = __shfl_xor_sync(0xffffffffu, M, o);
                    const float l = __shfl_xor_sync(0xffffffffu, den, o);
                    const float top = fmaxf(M, m), sub = finite_max(top);
                    den = fmaf(den, fast_exp2(M - sub), fast_exp2(m - sub) * l);
                    M = top;
                }
                if (lane == 0) lse_s[warp] = stat_of(t, M, den);
            }
        }
        __syncthreads();
        const int64_t col = static_cast<int64_t>(b) * t.d.Hkv + g;
        const float* scores = t.scores + col * all_rows * t.score_stride;
        float* mass = p.mass + col * p.mass_stride;
        for (int k = k0; k < k1; ++k) {
            const int64_t pos = static_cast<int64_t>(k) * kChunk + 4 * tid;
            if (pos >= total) continue;
            float w[4] = {0.f, 0.f, 0.f, 0.f};
            // (a multiple of 4 slots is the caller's: the slots and the strides are)
            float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.decay != 0.f) old = *reinterpret_cast<const float4*>(mass + pos);
            float4 v[ROWS];   // all in flight at once
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (r < rows)
                    v[r] = *reinterpret_cast<const float4*>(scores + r * t.score_stride + pos);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if (r >= rows) break;
                const float lse = lse_s[r];
                if (lse == lse) {
                    w[0] += fast_exp2(v[r].x - lse), w[1] += fast_exp2(v[r].y - lse);
                    w[2] += fast_exp2(v[r].z - lse), w[3] += fast_exp2(v[r].w - lse);
                } else {   // NaN for what the row sees (out of its sight: -inf)
                    w[0] += v[r].x == -INFINITY ? 0.f : lse, w[1] += v[r].y == -INFINITY ? 0.f : lse;
                    w[2] += v[r].z == -INFINITY ? 0.f : lse, w[3] += v[r].w == -INFINITY ? 0.f : lse;
                }
            }
            if (p.decay != 0.f) {
                if (pos < s.len) w[0] = fmaf(p.decay, old.x, w[0]);
                if (pos + 1 < s.len) w[1] = fmaf(p.decay, old.y, w[1]);
                if (pos + 2 < s.len) w[2] = fmaf(p.decay, old.z, w[2]);
                if (pos + 3 < s.len) w[3] = fmaf(p.decay, old.w, w[3]);
            }
            if (pos + 3 < total)
                *reinterpret_cast<float4*>(mass + pos) = make_float4(w[0], w[1], w[2], w[3]);
            else
                for (int i = 0; i < 4 && pos + i < total; ++i) mass[pos + i] = w[i];
        }
    }
}

size_t scores_floats(const qmm_kv_cache& c, int rows) {
    const int64_t cap = static_cast<int64_t>(c.max_pages) * c.page_size;
    const int64_t stride = (cap + (1 << kFewTileShift) - 1) >> kFewTileShift << kFewTileShift;
    return static_cast<size_t>(c.B) * c.Hkv * rows * stride;
}

}  // namespace

// Behind the attention's states: lse [B][T][Hq], and the scores for few rows.
static size_t lse_floats(const qmm_kv_cache& c, int T, int Hq) {
    return (static_cast<size_t>(c.B) * T * Hq + 3) / 4 * 4;
}

// One list of B + 1 values of 64 bits.
static size_t plan_floats(int B) { return (2 * (static_cast<size_t>(B) + 1) + 3) / 4 * 4; }

size_t scored_attention_workspace(const qmm_kv_cache& c, int T, int Hq, int num_sms) {
    const int rows = T * (Hq / c.Hkv);
    return tree_attention_workspace(c.D, rows, num_sms) +
           (lse_floats(c, T, Hq) +
            (rows <= 1 << kFewRowShift ? scores_floats(c, rows) + 2 * plan_floats(c.B) : 0)) *
               sizeof(float);
}

static int launch_few_rows(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N,
                           int T, int Hq, const int* cu, float scale, float* mass,
                           int64_t mass_stride, float decay, float* ws, float* lse, int num_sms,
                           void* stream) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return cudaErrorInvalidDevice;
    const bool fp8 = c.dtype == QMM_CACHE_E4M3;
    FinishParams p = {};
    CUtensorMap kmap, vmap;
    int rc = tree_setup(c, q, q_stride, O, N, T, Hq, cu, nullptr, scale, ws,
                        kFewCtasPerSm * num_sms, kFewRowShift, kFewTileShift, kFewMinRun, kFewSetup,
                        &p.t, &kmap, &vmap);
    if (rc != cudaSuccess) return rc;
    p.t.lse = lse;
    p.t.lift = fp8 ? kFewLift : 0.f;
    float* const plan = lse + lse_floats(c, T, Hq);
    p.t.plan = reinterpret_cast<long long*>(plan);
    p.t.chunks = reinterpret_cast<long long*>(plan + plan_floats(c.B));
    p.t.scores = plan + 2 * plan_floats(c.B);
    p.t.score_stride = (static_cast<int64_t>(p.t.d.cap) + (1 << kFewTileShift) - 1) >>
                       kFewTileShift << kFewTileShift;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = launch_tree_scores(kmap, vmap, p.t, c.D, fp8, device, st);
    if (rc != cudaSuccess) return rc;
    p.mass = mass;
    p.mass_stride = mass_stride;
    p.decay = decay;
    // equal runs for one wave of blocks, three an SM, beside those of the outputs
    const int64_t chunks = (static_cast<int64_t>(p.t.d.cap) + kChunk - 1) / kChunk * c.B * c.Hkv;
    p.adders = static_cast<int>(chunks < 3 * num_sms ? chunks : 3 * num_sms);
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    const int64_t items = static_cast<int64_t>(c.B) * c.Hkv;
    p.by_item = items < p.t.ctas;
    cfg.gridDim = dim3(static_cast<unsigned>(p.adders + (p.by_item ? items : p.t.ctas - 1)), 1, 1);
    cfg.blockDim = dim3(kFinishThreads, 1, 1);
    cfg.stream = st;
    return c.D == 128 ? cudaLaunchKernelEx(&cfg, scored_finish_kernel<128>, p)
                      : cudaLaunchKernelEx(&cfg, scored_finish_kernel<64>, p);
}

int launch_scored_attention(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N,
                            int T, int Hq, const int* cu, float scale, float* mass,
                            int64_t mass_stride, float decay, float* ws, int num_sms,
                            void* stream) {
    float* lse = ws + tree_attention_workspace(c.D, T * (Hq / c.Hkv), num_sms) / sizeof(float);
    if (T * (Hq / c.Hkv) <= 1 << kFewRowShift)
        return launch_few_rows(c, q, q_stride, O, N, T, Hq, cu, scale, mass, mass_stride, decay, ws,
                               lse, num_sms, stream);
    const int rc = launch_tree_attention(c, q, q_stride, O, N, T, Hq, cu, nullptr, scale, ws,
                                         num_sms, stream, lse);
    if (rc != cudaSuccess) return rc;
    return launch_mass_tc(c, q, q_stride, N, T, Hq, cu, scale, lse, mass, mass_stride, decay,
                          num_sms, stream);
}

}  // namespace qmm
