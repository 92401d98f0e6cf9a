// Writes into the paged KV cache: append with the per-head norm and the
// rotary position (qmm_kv_append), and the commit of an accepted path
// (qmm_tree_accept).
//
// Append.  Per head x of D values: y = x w / sqrt(mean(x^2) + eps), then each
// pair (a, c) turns by its angle, (a cos - c sin, c cos + a sin).  A few
// operations per value read and written once: the call is bound by the bytes
// of q, k, v and the cache rows.  A head row is held by D / 8 lanes, 16 bytes
// each, so that every access is one full 128-bit one; the partner of a value
// in a pair sits in the same lane (interleaved pairs) or in the lane dim / 16
// further (halves), reached by shuffles.  A lane keeps its cosines and sines
// for all the rows it handles, and its next rows' loads are issued together.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"
#include "qmm_paged.cuh"

namespace qmm {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 4;  // head rows whose loads a lane has in flight

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
};

__device__ __forceinline__ void unpack8(const uint4& u, float x[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float x[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// x / scale to the nearest E4M3 number, at most +-448 (ties to even)
__device__ __forceinline__ uint32_t e4m3x4(const float* x, float scale) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] / scale, x[1] / scale),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] / scale, x[3] / scale),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    constexpr int L = D / 8;                        // lanes of a head row
    constexpr int kGroups = kAppendThreads / L;     // lane groups of the block
    pdl_trigger();
    const int lane = threadIdx.x % L;
    const int group = threadIdx.x / L;
    const int sub = group % p.per_token;
    const int tok = blockIdx.x * (kGroups / p.per_token) + group / p.per_token;
    pdl_wait();
    // A group's lanes leave together or not at all; the shuffles below name
    // only the group's own lanes.
    if (tok >= p.N) return;
    const uint32_t mask = (L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u))
                          << ((threadIdx.x & 31) / L * L);
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
        if (before >= p.d.B) return;
        b = before;
        i = tok - p.cu[b];
        if (i < 0) return;
    }
    const int len = cached_tokens(p.d, b);
    const int pos = p.positions ? p.positions[tok] : len + i;
    if (p.dim > 0 && (pos < 0 || pos >= p.rows)) return;
    // (len <= cap < 2^31 - 65535 and i < N: the sum is tested before it is used)
    const int64_t slot = static_cast<int64_t>(len) + i;
    const int64_t at = slot < p.d.cap ? slot_offset(p.d, b, static_cast<int>(slot)) : -1;

    // the lane's cosines and sines: of pair j for its value 2j or 2j + 1
    // (interleaved), of pair (8 lane + j) mod (dim / 2) otherwise
    const bool turns = 8 * lane < p.dim;
    const int half = p.dim / 16;  // lanes of half a rotated head
    float cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = 1.f, sn[j] = 0.f;
    if (turns) {
        const float* row = p.cos_sin + static_cast<int64_t>(pos) * p.dim;
        if (p.interleaved) {
            const float4 c4 = *reinterpret_cast<const float4*>(row + 4 * lane);
            const float4 s4 = *reinterpret_cast<const float4*>(row + p.dim / 2 + 4 * lane);
            cs[0] = cs[1] = c4.x, cs[2] = cs[3] = c4.y, cs[4] = cs[5] = c4.z, cs[6] = cs[7] = c4.w;
            sn[0] = sn[1] = s4.x, sn[2] = sn[3] = s4.y, sn[4] = sn[5] = s4.z, sn[6] = sn[7] = s4.w;
        } else {
            const float* c = row + 8 * (lane < half ? lane : lane - half);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 c4 = *reinterpret_cast<const float4*>(c + j);
                const float4 s4 = *reinterpret_cast<const float4*>(c + p.dim / 2 + j);
                cs[j] = c4.x, cs[j + 1] = c4.y, cs[j + 2] = c4.z, cs[j + 3] = c4.w;
                sn[j] = s4.x, sn[j + 1] = s4.y, sn[j + 2] = s4.z, sn[j + 3] = s4.w;
            }
        }
    }
    // the first half (even values) subtracts its partner's product
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (p.interleaved ? j % 2 == 0 : lane < half) sn[j] = -sn[j];
    const int partner = turns && !p.interleaved ? (lane < half ? lane + half : lane - half) : lane;

    // head rows of the token: Hq of q, Hkv of k, Hkv of v
    const int Hkv = p.d.Hkv, all = p.Hq + 2 * Hkv;
    const __nv_bfloat16* qrow = p.q + tok * p.q_stride + 8 * lane;
    const __nv_bfloat16* krow = p.k + tok * p.k_stride + 8 * lane;
    const __nv_bfloat16* vrow = p.v + tok * p.v_stride + 8 * lane;
    for (int r0 = sub; r0 < all; r0 += kAppendRows * p.per_token) {
        uint4 in[kAppendRows];
#pragma unroll
        for (int u = 0; u < kAppendRows; ++u) {
            const int r = r0 + u * p.per_token;
            if (r < all)
                in[u] = *reinterpret_cast<const uint4*>(
                    r < p.Hq ? qrow + r * D
                             : (r < p.Hq + Hkv ? krow + (r - p.Hq) * D : vrow + (r - p.Hq - Hkv) * D));
        }
#pragma unroll
        for (int u = 0; u < kAppendRows; ++u) {
            const int r = r0 + u * p.per_token;
            if (r >= all) break;
            const int kind = r < p.Hq ? 0 : (r < p.Hq + Hkv ? 1 : 2);
            if (kind > 0 && at < 0) break;  // no slot: this row and the later ones store nothing
            float x[8];
            unpack8(in[u], x);
            const __nv_bfloat16* w = kind == 0 ? p.q_norm : (kind == 1 ? p.k_norm : nullptr);
            if (w) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
                const float rms = rsqrtf(ss * (1.f / D) + p.eps);
                float wf[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(w + 8 * lane)), wf);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * rms * wf[j];
            }
            if (kind < 2 && p.dim > 0) {
                float y[8];
                if (p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
                } else {
                    // (a lane past dim is its own partner)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y[j] = __shfl_sync(mask, x[j], partner, L);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = turns ? fmaf(y[j], sn[j], x[j] * cs[j]) : x[j];
            }
            if (kind == 0) {
                *reinterpret_cast<uint4*>(p.q_out + tok * p.q_out_stride + r * D + 8 * lane) = pack8(x);
            } else {
                const int h = kind == 1 ? r - p.Hq : r - p.Hq - Hkv;
                const int64_t e = at + h * p.d.head_stride + 8 * lane;
                void* pool = kind == 1 ? p.K : p.V;
                if (kFp8) {
                    const float sc = kind == 1 ? p.k_scale : p.v_scale;
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + e) =
                        make_uint2(e4m3x4(x, sc), e4m3x4(x + 4, sc));
                } else {
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pool) + e) = pack8(x);
                }
            }
        }
    }
}

// ---- accepted path -----------------------------------------------------------

constexpr int kAcceptThreads = 256;
constexpr int kAcceptRows = 4;  // rows a lane group has in flight

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
    __shared__ int count_s;
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
    for (int j = tid; j < count; j += kAcceptThreads) {
        src[j] = slot_offset(p.d, b, len + path[j]);
        dst[j] = slot_offset(p.d, b, len + j);
    }
    __syncthreads();
    const int lanes = p.row_bytes / 16;
    const int lane = tid % lanes;
    const int cols = 2 * p.n * p.d.Hkv;
    const int last = min(cols, (static_cast<int>(blockIdx.x) + 1) * p.per_block);
    for (int c = blockIdx.x * p.per_block + tid / lanes; c < last; c += kAcceptThreads / lanes) {
        uint8_t* pool = p.pools[c / p.d.Hkv];
        const int64_t head = (c % p.d.Hkv) * p.d.head_stride;
        for (int j0 = 0; j0 < count; j0 += kAcceptRows) {
            uint4 x[kAcceptRows];
#pragma unroll
            for (int u = 0; u < kAcceptRows; ++u) {
                const int j = j0 + u;
                if (j < count && path[j] != j && src[j] >= 0 && dst[j] >= 0)
                    x[u] = *reinterpret_cast<const uint4*>(pool + (src[j] + head) * p.elem + 16 * lane);
            }
#pragma unroll
            for (int u = 0; u < kAcceptRows; ++u) {
                const int j = j0 + u;
                if (j < count && path[j] != j && src[j] >= 0 && dst[j] >= 0)
                    *reinterpret_cast<uint4*>(pool + (dst[j] + head) * p.elem + 16 * lane) = x[u];
            }
        }
    }
}

}  // namespace

int launch_kv_append(const qmm_kv_cache& c, const void* q, const void* k, const void* v,
                     void* q_out, int N, int Hq, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, int64_t q_out_stride, const int* cu, const int* positions,
                     const qmm_rope* rope, void* stream) {
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
    const int groups = kAppendThreads / (c.D / 8);
    p.per_token = 1;
    while (p.per_token < groups && p.per_token < Hq + 2 * c.Hkv) p.per_token *= 2;
    const int tokens = groups / p.per_token;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3((N - 1) / tokens + 1, 1, 1);
    cfg.blockDim = dim3(kAppendThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    const bool fp8 = c.dtype == QMM_CACHE_E4M3;
    if (c.D == 128)
        return fp8 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<128, true>, p)
                   : cudaLaunchKernelEx(&cfg, kv_append_kernel<128, false>, p);
    return fp8 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<64, true>, p)
               : cudaLaunchKernelEx(&cfg, kv_append_kernel<64, false>, p);
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
    // one column per lane group where that leaves the grid within 64K blocks
    const int64_t cols = static_cast<int64_t>(2) * n * c.Hkv;
    p.per_block = kAcceptThreads / (p.row_bytes / 16);
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
