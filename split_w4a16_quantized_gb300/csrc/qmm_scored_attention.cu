// Attention that adds up the weight each slot receives (qmm_scored_attention).
//
//   mass[b, g, s] = decay mass[b, g, s] + sum over tokens i and heads h of g of
//                   2^(score(i, h, s) - lse(i, h))
//
// with scores in log2 units and lse = log2 sum_s 2^score, which tree attention leaves
// for every row beside its output.  The weights are known only once a row's whole
// history has been seen, so the scores are formed again from K behind the attention
// kernels: a thread a position, which holds its key and goes through the query rows.
#include "qmm.h"
#include "qmm_tree.cuh"

namespace qmm {
namespace {

constexpr int kMassThreads = 128;
constexpr int kMassRows = 8;   // query rows in shared memory at a time

struct MassParams {
    PagedDims d;
    const __nv_bfloat16* q;
    const uint8_t* K;
    const int* cu;
    const float* lse;   // [B][T][Hq]
    float* mass;
    int64_t q_stride, mass_stride;
    int N, T, Hq, QG;
    float qscale, decay;
};

template <int D, bool kFp8>
__global__ void __launch_bounds__(kMassThreads)
    mass_kernel(const __grid_constant__ MassParams p) {
    __shared__ float q_s[kMassRows][D];
    __shared__ float lse_s[kMassRows];
    const int tid = threadIdx.x, g = blockIdx.y, b = blockIdx.z;
    pdl_trigger();
    pdl_wait();
    int first, n;
    token_range(p.cu, p.N, p.T, b, &first, &n);
    const int len = cached_tokens(p.d, b);
    const int total = len + n < p.d.cap ? len + n : p.d.cap;
    const int rows = n * p.QG;
    float* mass = p.mass + (static_cast<int64_t>(b) * p.d.Hkv + g) * p.mass_stride;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kMassThreads; t0 < total;
         t0 += static_cast<int64_t>(gridDim.x) * kMassThreads) {
        const int pos = static_cast<int>(t0) + tid;   // (total <= cap < 2^31 - 65535)
        const int64_t at = pos < total ? slot_offset(p.d, b, pos) : -1;
        // the key: D values as BF16 pairs, or as E4M3 bytes
        constexpr int W = D * (kFp8 ? 1 : 2) / 16;
        uint4 key[W];
#pragma unroll
        for (int i = 0; i < W; ++i)
            key[i] = at < 0 ? make_uint4(0, 0, 0, 0)
                            : reinterpret_cast<const uint4*>(
                                  p.K + (at + g * p.d.head_stride) * (kFp8 ? 1 : 2))[i];
        float sum = 0.f;
        for (int r0 = 0; r0 < rows; r0 += kMassRows) {
            __syncthreads();
            for (int i = tid; i < kMassRows * D; i += kMassThreads) {
                const int r = r0 + i / D;
                float v = 0.f;
                if (r < rows)
                    v = __bfloat162float(p.q[(first + r / p.QG) * p.q_stride +
                                             (g * p.QG + r % p.QG) * D + i % D]);
                q_s[i / D][i % D] = v;
            }
            if (tid < kMassRows && r0 + tid < rows) {
                const int r = r0 + tid;
                lse_s[tid] = p.lse[(static_cast<int64_t>(b) * p.T + r / p.QG) * p.Hq + g * p.QG +
                                   r % p.QG];
            }
            __syncthreads();
            for (int k = 0; k < kMassRows && r0 + k < rows; ++k) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const uint32_t w[4] = {key[i].x, key[i].y, key[i].z, key[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (kFp8) {
                            const uint32_t lo = e4m3x2_to_f16x2(w[j] & 0xffffu);
                            const uint32_t hi = e4m3x2_to_f16x2(w[j] >> 16);
                            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                            const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                            const float* qv = &q_s[k][16 * i + 4 * j];
                            s = fmaf(a.x, qv[0], s), s = fmaf(a.y, qv[1], s);
                            s = fmaf(c.x, qv[2], s), s = fmaf(c.y, qv[3], s);
                        } else {
                            const float* qv = &q_s[k][8 * i + 2 * j];
                            s = fmaf(__uint_as_float(w[j] << 16), qv[0], s);
                            s = fmaf(__uint_as_float(w[j] & 0xffff0000u), qv[1], s);
                        }
                    }
                }
                const int node = (r0 + k) / p.QG;
                if (at >= 0 && (pos < len || pos - len <= node))
                    sum += fast_exp2(fmaf(s, p.qscale, -lse_s[k]));
            }
        }
        if (pos < total) {
            if (pos < len && p.decay != 0.f) sum = fmaf(p.decay, mass[pos], sum);
            mass[pos] = sum;
        }
    }
}

}  // namespace

size_t scored_attention_workspace(const qmm_kv_cache& c, int T, int Hq, int num_sms) {
    return tree_attention_workspace(c.D, T * (Hq / c.Hkv), num_sms) +
           static_cast<size_t>(c.B) * T * Hq * sizeof(float);
}

int launch_scored_attention(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N,
                            int T, int Hq, const int* cu, float scale, float* mass,
                            int64_t mass_stride, float decay, float* ws, int num_sms,
                            void* stream) {
    float* lse = ws + tree_attention_workspace(c.D, T * (Hq / c.Hkv), num_sms) / sizeof(float);
    const int rc = launch_tree_attention(c, q, q_stride, O, N, T, Hq, cu, nullptr, scale, ws,
                                         num_sms, stream, lse);
    if (rc != cudaSuccess) return rc;
    MassParams p = {};
    p.d = paged_dims(c);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.K = static_cast<const uint8_t*>(c.K);
    p.cu = cu;
    p.lse = lse;
    p.mass = mass;
    p.q_stride = q_stride;
    p.mass_stride = mass_stride;
    p.N = N;
    p.T = T;
    p.Hq = Hq;
    p.QG = Hq / c.Hkv;
    p.qscale = score_factor(c, scale);
    p.decay = decay;
    const int64_t tiles = (static_cast<int64_t>(p.d.cap) + kMassThreads - 1) / kMassThreads;
    const int64_t most = 16LL * num_sms * 8 / (static_cast<int64_t>(c.B) * c.Hkv) + 1;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles < most ? tiles : most), c.Hkv, c.B);
    cfg.blockDim = dim3(kMassThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    auto run = [&](auto kernel) { return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p)); };
    if (c.D == 128)
        return c.dtype == QMM_CACHE_E4M3 ? run(mass_kernel<128, true>) : run(mass_kernel<128, false>);
    return c.dtype == QMM_CACHE_E4M3 ? run(mass_kernel<64, true>) : run(mass_kernel<64, false>);
}

}  // namespace qmm
