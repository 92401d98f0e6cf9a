// Eviction from the paged KV cache by the weight each slot has received
// (qmm_kv_evict).
//
// A cache column (layer, sequence, KV head) of len slots goes back to `keep`: the
// first `sinks` and the last `recent` slots stay, and of those between the keep -
// sinks - recent with the largest weights, the lowest slot first among equals.
//
// Where rows go.  Attention does not look at the order of the slots, so only what
// lies behind the budget has to move: a chosen row below `line` = keep - recent stays,
// the evicted slots below it take the chosen rows from the line on, both in ascending
// order, and the recent rows follow in order at [line, keep).  So the last `recent`
// slots are the newest tokens at the next eviction too.  Moved are `recent` rows and
// the chosen ones between line and len - recent, instead of all rows behind the first
// evicted slot.
//
// Two kernels.  evict_select: a block a column finds the threshold by its bits, 8 a
// pass (a weight's bits, ordered as the weights are), then pairs evicted and chosen
// slots from two queues filled in ascending order, and moves the weights.  evict_move:
// blocks of (column, K or V, piece of the row's bytes) move the rows in ascending
// order of their targets, a batch at a time: all of a batch is in registers before any
// of it is stored.  A row moves to a lower slot, so a target is never the source of a
// later batch, and the batches before have read theirs.
#include <cuda_runtime.h>

#include <cstdint>

#include "qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"
#include "qmm_paged.cuh"
#include "qmm_paged_host.h"

namespace qmm {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kMoveThreads = 256;
constexpr int kMoveLanes = 4;  // lanes of a lane group: 64 bytes, a row's piece
constexpr int kMoveRows = 8;   // rows a lane group has in flight
constexpr int kBatch = kMoveThreads / kMoveLanes * kMoveRows;

struct EvictParams {
    PagedDims d;
    const float* mass;
    float* mass_out;
    int64_t layer_stride, row_stride;   // of the weights
    int *kept, *new_lens;
    int n, keep, sinks, recent;
    int first;                  // this launch's first layer
    int elem, slices;           // bytes a value; pieces of a row
    uint8_t* pools[2 * kMaxEvictCaches];   // K and V of each layer
};

// Weights in order: larger weight, larger number; both zeros alike, and NaN below all.
__device__ __forceinline__ uint32_t rank_of(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);   // (-0 + 0 = +0)
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// Sum of v over the threads before this one, and over the block.
__device__ __forceinline__ int scan_block(int v, int* red, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelectThreads / 32; ++w) {
        if (w < warp) before += red[w];
        all += red[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(kSelectThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int hist[256];
    __shared__ int red[kSelectThreads / 32];
    __shared__ int digit_s, above_s;
    __shared__ int queue[2][2 * kSelectThreads];   // evicted slots below the line, chosen ones behind
    const int tid = threadIdx.x;
    const int h = blockIdx.x % p.d.Hkv, layer = p.first + blockIdx.x / p.d.Hkv, b = blockIdx.y;
    pdl_trigger();
    pdl_wait();
    const int len = cached_tokens(p.d, b), keep = p.keep;
    const int64_t col = static_cast<int64_t>(b) * p.d.Hkv + h;
    const float* mass = p.mass + layer * p.layer_stride + col * p.row_stride;
    float* mass_out = p.mass_out + layer * p.layer_stride + col * p.row_stride;
    int* kept = p.kept + (static_cast<int64_t>(layer) * p.d.B * p.d.Hkv + col) * keep;
    if (layer == 0 && h == 0 && tid == 0) p.new_lens[b] = min(len, keep);
    if (len <= keep) {
        for (int64_t j = tid; j < keep; j += kSelectThreads) {
            kept[j] = j < len ? static_cast<int>(j) : -1;
            if (j < len && mass_out != mass) mass_out[j] = mass[j];
        }
        return;
    }
    const int m0 = p.sinks, m1 = len - p.recent;        // the slots in question
    const int want = keep - p.sinks - p.recent;         // how many of them stay
    const int line = keep - p.recent;

    // The want-th largest number: its digits from the top, 8 bits a pass.  `above`:
    // slots known to be larger.
    uint32_t top = 0;
    int above = 0;
    if (want > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (int64_t i = m0 + tid; i < m1; i += kSelectThreads) {
                const uint32_t r = rank_of(mass[i]);
                if (shift == 24 || (r >> (shift + 8)) == (top >> (shift + 8)))
                    atomicAdd(&hist[(r >> shift) & 255u], 1);
            }
            __syncthreads();
            // thread t < 256: how many lie in digits above 255 - t
            const int mine = tid < 256 ? hist[255 - tid] : 0;
            int all;
            const int before = scan_block(mine, red, &all);
            if (tid < 256 && above + before < want && above + before + mine >= want) {
                digit_s = 255 - tid;
                above_s = above + before;
            }
            __syncthreads();
            top |= static_cast<uint32_t>(digit_s) << shift;
            above = above_s;
            __syncthreads();
        }
    }
    // of the slots equal to it, the first `equal` stay
    const int equal = want - above;

    // Queues of evicted slots below the line and of chosen ones from it on; what both
    // hold is paired.  (below the line: sinks are chosen; there are as many evicted
    // there as chosen behind it)
    auto chosen = [&](int64_t i, bool in, int* ties) {   // whole block, ascending i
        const uint32_t r = in ? rank_of(mass[i]) : 0u;
        const bool tie = in && want > 0 && r == top;
        int all;
        const int before = scan_block(tie ? 1 : 0, red, &all);
        const bool yes = in && want > 0 && (r > top || (tie && *ties + before < equal));
        *ties += all;
        return yes;
    };
    // ties below the line come first
    int low_ties = 0, high_ties = 0;
    {
        int mine = 0;
        for (int64_t i = m0 + tid; i < line; i += kSelectThreads)
            mine += want > 0 && rank_of(mass[i]) == top;
        scan_block(mine, red, &high_ties);
    }
    for (int64_t j = tid; j < m0; j += kSelectThreads) kept[j] = static_cast<int>(j);
    for (int64_t j = line + tid; j < keep; j += kSelectThreads)
        kept[j] = static_cast<int>(j + (len - keep));
    int64_t low = m0, high = line;   // next slots to look at
    int held[2] = {0, 0};            // slots in each queue
    while (true) {
        // refill each queue to at least a slot, or to its end
        while (held[0] == 0 && low < line) {
            const int64_t i = low + tid;
            const bool in = i < line, yes = chosen(i, in, &low_ties);
            if (yes) kept[i] = static_cast<int>(i);
            int all;
            const int at = scan_block(in && !yes ? 1 : 0, red, &all);
            if (in && !yes) queue[0][at] = static_cast<int>(i);
            held[0] = all;
            low += kSelectThreads;
        }
        while (held[0] > 0 && held[1] < kSelectThreads && high < m1) {
            const int64_t i = high + tid;
            const bool yes = chosen(i, i < m1, &high_ties);
            int all;
            const int at = scan_block(yes ? 1 : 0, red, &all);
            if (yes) queue[1][held[1] + at] = static_cast<int>(i);
            held[1] += all;
            high += kSelectThreads;
        }
        __syncthreads();
        const int both = min(held[0], held[1]);
        if (both == 0) break;   // (no evicted slot is left)
        if (tid < both) kept[queue[0][tid]] = queue[1][tid];
        // what is left of either moves to its front
        int keep0 = 0, keep1 = 0, keep2 = 0;
        if (both + tid < held[0]) keep0 = queue[0][both + tid];
        if (both + tid < held[1]) keep1 = queue[1][both + tid];
        if (both + tid + kSelectThreads < held[1]) keep2 = queue[1][both + tid + kSelectThreads];
        __syncthreads();
        if (both + tid < held[0]) queue[0][tid] = keep0;
        if (both + tid < held[1]) queue[1][tid] = keep1;
        if (both + tid + kSelectThreads < held[1]) queue[1][tid + kSelectThreads] = keep2;
        held[0] -= both;
        held[1] -= both;
        __syncthreads();
    }
    __syncthreads();
    // the weights go with their slots, ascending: mass_out may be mass
    for (int64_t j0 = 0; j0 < keep; j0 += kSelectThreads) {
        const int64_t j = j0 + tid;
        const float w = j < keep ? mass[kept[j]] : 0.f;
        __syncthreads();
        if (j < keep) mass_out[j] = w;
    }
}

__global__ void __launch_bounds__(kMoveThreads, 4)
    evict_move_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int64_t src[kBatch], dst[kBatch];   // bytes from the column's start
    __shared__ int count_s;
    const int tid = threadIdx.x, b = blockIdx.y;
    int at = blockIdx.x;
    const int slice = at % p.slices;
    at /= p.slices;
    const int kv = at & 1;
    at >>= 1;
    const int h = at % p.d.Hkv, layer = at / p.d.Hkv;   // of this launch
    pdl_trigger();
    pdl_wait();
    const int len = cached_tokens(p.d, b), keep = p.keep;
    if (len <= keep) return;
    const int* kept = p.kept +
        ((static_cast<int64_t>(p.first + layer) * p.d.B + b) * p.d.Hkv + h) * keep;
    uint8_t* pool = p.pools[2 * layer + kv] + h * p.d.head_stride * p.elem +
                    (slice * kMoveLanes + tid % kMoveLanes) * 16;
    constexpr int kGroups = kMoveThreads / kMoveLanes;
    const int group = tid / kMoveLanes;
    if (tid == 0) count_s = 0;
    __syncthreads();
    for (int64_t j0 = p.sinks; j0 < keep;) {
        // the next batch of rows that move
        int count = 0;
        while (j0 < keep && count + kMoveThreads <= kBatch) {
            const int64_t j = j0 + tid;
            int64_t from = -1, to = -1;
            if (j < keep) {
                const int k = kept[j];
                if (k != j) {
                    from = slot_offset(p.d, b, k);
                    to = slot_offset(p.d, b, static_cast<int>(j));
                }
            }
            if (from >= 0 && to >= 0) {   // (a missing page on either side: not moved)
                const int i = atomicAdd(&count_s, 1);
                src[i] = from * p.elem;
                dst[i] = to * p.elem;
            }
            __syncthreads();
            count = count_s;
            __syncthreads();
            j0 += kMoveThreads;
        }
        if (tid == 0) count_s = 0;
        uint4 x[kMoveRows];
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            const int r = group + u * kGroups;
            if (r < count) x[u] = *reinterpret_cast<const uint4*>(pool + src[r]);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            const int r = group + u * kGroups;
            if (r < count) *reinterpret_cast<uint4*>(pool + dst[r]) = x[u];
        }
        __syncthreads();
    }
}

}  // namespace

int launch_kv_evict(const qmm_kv_cache* caches, int n, int first, const float* mass,
                    float* mass_out, int64_t layer_stride, int64_t row_stride, int keep, int sinks,
                    int recent, int* kept, int* new_lens, void* stream) {
    const qmm_kv_cache& c = caches[0];
    EvictParams p = {};
    p.d = paged_dims(c);
    p.mass = mass;
    p.mass_out = mass_out;
    p.layer_stride = layer_stride;
    p.row_stride = row_stride;
    p.kept = kept;
    p.new_lens = new_lens;
    p.n = n;
    p.keep = keep;
    p.sinks = sinks;
    p.recent = recent;
    p.first = first;
    p.elem = c.dtype == QMM_CACHE_E4M3 ? 1 : 2;
    p.slices = c.D * p.elem / (16 * kMoveLanes);
    for (int i = 0; i < n; ++i) {
        p.pools[2 * i] = static_cast<uint8_t*>(caches[i].K);
        p.pools[2 * i + 1] = static_cast<uint8_t*>(caches[i].V);
    }
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(static_cast<unsigned>(n * c.Hkv), c.B, 1);
    cfg.blockDim = dim3(kSelectThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    int rc = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
    if (rc != cudaSuccess) return rc;
    cfg.gridDim.x = static_cast<unsigned>(n * c.Hkv) * 2 * p.slices;
    cfg.blockDim = dim3(kMoveThreads, 1, 1);
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

}  // namespace qmm
