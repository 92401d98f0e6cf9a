// Attention of a batch whose sequences share long prefixes (qmm_prefix_attention).
//
//   O[i, h] = sum_l p_l V[l],  p = softmax over the prefix of the token's sequence and
//             what tree attention lets the token see of the sequence's own slots
//
// The softmax over both parts is the merge of a state (maximum, sum, unnormalized
// output) of each.  All tokens of a prefix's sequences see all of it, so a prefix is one
// more entry of tree attention's list of work, whose rows are the query rows of all its
// sequences, 128 to an item: its K and V are read once for 128 rows and not once for
// each sequence.  Equal runs of the whole list keep the SMs busy whatever the lengths of
// the prefixes and of what lies behind them: one launch of the tcgen05 kernel
// (qmm_tree_attention_tc.cu), for few rows too, whose padding it hides behind the bytes
// of their K and V.  Items that one run holds leave their state by (token, head), the
// others by run as in tree attention, and the merge here adds a row's own states and its
// prefix's, in that order and each in run order.
#include <algorithm>

#include "qmm.h"
#include "qmm_tree_merge.cuh"

namespace qmm {
namespace {

constexpr int kRowShift = 7;
constexpr int kCtasPerSm = 2;
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 16;

// A block takes 16 query rows of a sequence's KV head, a thread a row and every 16th
// (D = 128; 64: 8th) group of 4 columns.
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    prefix_merge_kernel(const __grid_constant__ TreeParams p, int chunks) {
    __shared__ long long red[3][kMergeThreads / 32];
    __shared__ int group_s;
    __shared__ __align__(16) uint2 stage[kMergeRows][D / 4 + 2];   // BF16 rows, padded by 16 bytes
    const int tid = threadIdx.x;
    const int chunk = blockIdx.x % chunks, g = blockIdx.x / chunks, b = blockIdx.y;
    pdl_trigger();
    pdl_wait();
    const Seq s = sequence<false, true>(p, p.pre.G + b);
    const int rows = s.n * p.QG, row0 = chunk * kMergeRows;
    if (row0 >= rows) return;   // (the same for the whole block)
    // the sequence's prefix: the first that holds it
    if (tid == 0) group_s = p.pre.G;
    __syncthreads();
    for (int j = tid; j < p.pre.G; j += kMergeThreads) {
        int b0, b1;
        group_range<false>(p, j, &b0, &b1);
        if (b >= b0 && b < b1) atomicMin(&group_s, j);
    }
    __syncthreads();
    const int grp = group_s;
    long long all = 0, before_own = 0, before_grp = 0;
    {
        long long a = 0, o = 0, q = 0;
        for (int j = tid; j < p.pre.G + p.d.B; j += kMergeThreads) {
            const long long u = units_of(p, sequence<false, true>(p, j));
            a += u;
            if (j < p.pre.G + b) o += u;
            if (j < grp) q += u;
        }
        block_scan<kMergeThreads>(a, red[0], &all);
        block_scan<kMergeThreads>(o, red[1], &before_own);
        block_scan<kMergeThreads>(q, red[2], &before_grp);
    }
    const long long len = run_length(p, all);
    Seq pre = {};
    if (grp < p.pre.G) pre = sequence<false, true>(p, grp);

    constexpr int GROUPS = D / 4;
    constexpr int TURNS = GROUPS / (kMergeThreads / kMergeRows);   // column groups of a thread
    constexpr int JUMP = kMergeThreads / kMergeRows;
    const int i = tid % kMergeRows, r = row0 + i, j0 = tid / kMergeRows;
    if (r < rows) {
        const int node = r / p.QG, head = g * p.QG + r - node * p.QG;
        Acc<TURNS> acc;
        // the states of one entry's item that holds the row (row `at` of the entry)
        auto take = [&](const Seq& e, long long before, int at, int part) {
            const int rt = at >> p.row_shift, in = at & ((1 << p.row_shift) - 1);
            const Runs c = runs_of(p, e, before, g * e.row_tiles + rt, len);
            if (c.c0 == c.c1) {
                const DirectAt x =
                    direct_at<D>(p, part, static_cast<int64_t>(s.first + node) * p.Hq + head);
                float4 o[1][TURNS];
#pragma unroll
                for (int u = 0; u < TURNS; ++u)
                    o[0][u] = *reinterpret_cast<const float4*>(x.o + 4 * (j0 + u * JUMP));
                acc.template add<1>(x.m, x.l, o, 1);
                return;
            }
            acc.template add_runs<D>(p, c, in, j0, JUMP);
        };
        take(s, before_own, r, 0);
        const int64_t at = static_cast<int64_t>(s.first - pre.first + node) * p.QG + r - node * p.QG;
        if (pre.row_tiles > 0 && at >= 0 && at < static_cast<int64_t>(pre.n) * p.QG)
            take(pre, before_grp, static_cast<int>(at), 1);
        const float inv = acc.inverse(p.vscale);
#pragma unroll
        for (int u = 0; u < TURNS; ++u)
            stage[i][j0 + u * JUMP] =
                make_uint2(pack_bf16x2(acc.num[u].x * inv, acc.num[u].y * inv),
                           pack_bf16x2(acc.num[u].z * inv, acc.num[u].w * inv));
    }
    __syncthreads();
    constexpr int CH = D / 8;   // 16-byte chunks of a row
    const int ri = tid / CH, c = tid % CH, rr = row0 + ri;
    if (ri < kMergeRows && rr < rows) {
        const int64_t to = static_cast<int64_t>(s.first + rr / p.QG) * p.Hq + g * p.QG + rr % p.QG;
        *reinterpret_cast<uint4*>(p.O + to * D + 8 * c) =
            *reinterpret_cast<const uint4*>(&stage[ri][2 * c]);
    }
}

}  // namespace

static size_t slot_floats(int D, int num_sms) {
    return (static_cast<size_t>(2 * kCtasPerSm * num_sms) << kRowShift) * (D + 2);
}

size_t prefix_attention_workspace(int D, int64_t rows, int num_sms) {
    return (slot_floats(D, num_sms) + 2 * static_cast<size_t>(rows) * (D + 2)) * sizeof(float);
}

int launch_prefix_attention(const qmm_kv_cache& c, const qmm_prefix& pre, const void* q,
                            int64_t q_stride, void* O, int N, int T, int Hq, const int* cu,
                            const int* parents, float scale, float* ws, int num_sms,
                            void* stream) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return cudaErrorInvalidDevice;
    const bool fp8 = c.dtype == QMM_CACHE_E4M3;
    TreeParams p;
    CUtensorMap kmap, vmap;
    int rc = tree_setup(c, q, q_stride, O, N, T, Hq, cu, parents, scale, ws, kCtasPerSm * num_sms,
                        kRowShift, kTcTileShift, 6, fp8 ? 8 : 4, &p, &kmap, &vmap);
    if (rc != cudaSuccess) return rc;
    p.pre.table = pre.table;
    p.pre.lens = pre.lens;
    p.pre.first = pre.first;
    p.pre.G = pre.G;
    p.pre.max_pages = pre.max_pages;
    p.pre.cap = pre.max_pages * c.page_size;
    p.pre.direct = ws + slot_floats(c.D, num_sms);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = launch_prefix_tc(kmap, vmap, p, c.D, fp8, device, st);
    if (rc != cudaSuccess) return rc;
    const int chunks = (T * p.QG + kMergeRows - 1) / kMergeRows;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(static_cast<unsigned>(chunks) * c.Hkv, c.B, 1);
    cfg.blockDim = dim3(kMergeThreads, 1, 1);
    cfg.stream = st;
    return c.D == 128 ? cudaLaunchKernelEx(&cfg, prefix_merge_kernel<128>, p, chunks)
                      : cudaLaunchKernelEx(&cfg, prefix_merge_kernel<64>, p, chunks);
}

}  // namespace qmm
