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
// (qmm_tree_attention_tc.cu), for a sequence's few rows too, whose padding it hides behind
// the bytes of their K and V.  Items that one run holds leave their state by (token, head),
// the others by run as in tree attention; the merge adds a row's own states and its
// prefix's, in that order and each in run order.  Which runs hold an item follows from the
// units before its entry, which the attention launch's first block writes down: its CTAs
// take all registers, so the merge could not work them out while that launch runs (64
// sequences, one BF16 term of a weight: 42 us, each merge block summing the list 46).
//
// What bounds it: the chain of a tile in a CTA.  64 sequences behind 8192 tokens: 46 us,
// floor 20 (HBM), in tiles of 2690 clocks each of which the softmax takes 1850 with both
// terms of its weights and waits 570 for scores (tensor pipe active 44 %), then 7 us of merge,
// a chain of four trips to L2.  24 sequences of up to 8 tokens behind 16000, E4M3: 65 us, floor
// 13.5; a tile takes 1940 clocks of a CTA, 1020 of them softmax, an SM's two CTAs 1000 (tensor
// pipe active 35 %).  48 of 4 tokens behind five prefixes, D = 64: 105 us, floor 27; 1940 clocks,
// with the softmax at work for 1290 of them.  Measured and slower, with one BF16 term of a weight
// (42, 65 and 88 us): two groups of 128 rows and one CTA an SM (61, 64, 115 us: items of few rows
// follow one another without overlap); the sequences' own part and the prefixes as two launches
// side by side (64, 98, 136: two waves of CTAs, each with its start and end); tiles that count by
// their rows (50, 80, 107: a few rows' tile takes a CTA as long as a full one).
#include <algorithm>

#include "qmm.h"
#include "qmm_tree_merge.cuh"

namespace qmm {
namespace {

constexpr int kRowShift = 7;
constexpr int kCtasPerSm = 2;   // of either kernel
// The kernel for 8 rows takes calls of up to 8 query rows per KV head in all, and more where
// the prefixes' tables are so short that reading them once for 8 rows costs less than the
// tcgen05 kernel's longer start: slots of a table, and slots of all KV heads times the 8 rows'
// pieces.  One prefix, BF16, the kernel for 8 rows and the tcgen05 kernel, us (measured for 2, 8
// and 32 KV heads, 12 to 128 rows, 250 to 8000 slots; the rule's choice at most 7 % behind):
//   8 KV heads, 16 rows   500 slots 10.1 15.7   4000 15.7 18.7   8000 21.5 20.5
//               64 rows   500 slots 12.8 16.1   1000 16.4 17.0   2000 19.7 17.3
//   32 KV heads, 16 rows  500 slots 12.7 16.6   1000 16.3 17.4   2000 19.5 18.8
//   2 KV heads, 16 rows   500 slots  8.9 14.9   4000 15.7 16.6   8000 21.9 18.8
// (8 rows: 8 KV heads 8000 slots 18.4 20.2, 20000 28.7 28.8; 2 KV heads 8000 21.3 18.5.)
constexpr int64_t kFewSlots = 4096, kFewReads = 96 * 1024;
// A block takes ROWS query rows of a sequence's KV head, a thread a row and every 16th
// (D = 128; 64: each) group of 4 columns.
template <int D, int ROWS>
__global__ void __launch_bounds__(16 * ROWS)
    prefix_merge_kernel(const __grid_constant__ TreeParams p, int chunks) {
    __shared__ __align__(16) uint2 stage[ROWS][D / 4 + 2];   // BF16 rows, padded by 16 bytes
    const int tid = threadIdx.x, lane = tid & 31;
    const int chunk = blockIdx.x % chunks, g = blockIdx.x / chunks, b = blockIdx.y;
    pdl_trigger();
    pdl_wait();
    const Seq s = sequence<false, true>(p, p.pre.G + b);
    const long long before_own = p.plan[p.pre.G + b];
    const long long len = run_length(p, p.plan[p.pre.G + p.d.B]);
    // the first prefix that holds the sequence
    int group = -1;
    for (int j0 = 0; group < 0 && j0 < p.pre.G; j0 += 32) {
        int b0 = 0, b1 = 0;
        if (j0 + lane < p.pre.G) group_range<false>(p, j0 + lane, &b0, &b1);
        const uint32_t hit = __ballot_sync(0xffffffffu, b >= b0 && b < b1);
        if (hit) group = j0 + __ffs(hit) - 1;
    }
    Seq shared = {};
    long long before_pre = 0;
    if (group >= 0) {
        shared = sequence<false, true>(p, group);
        before_pre = p.plan[group];
    }
    const int rows = s.n * p.QG, row0 = chunk * ROWS;
    if (row0 >= rows) return;   // (the same for the whole block)

    constexpr int JUMP = 16;               // threads of a row
    constexpr int TURNS = D / 4 / JUMP;    // column groups of a thread
    const int i = tid % ROWS, r = row0 + i, j0 = tid / ROWS;
    if (r < rows) {
        const int node = r / p.QG, head = g * p.QG + r - node * p.QG;
        const int64_t row = static_cast<int64_t>(s.first + node) * p.Hq + head;
        // the runs that hold the row's item of the sequence, and of its prefix
        const Runs co = runs_of(p, s, before_own, g * s.row_tiles + (r >> p.row_shift), len);
        const int at = (s.first - shared.first + node) * p.QG + r - node * p.QG;
        Runs cp = {0, -1};
        if (shared.row_tiles > 0 && at >= 0 && at < shared.n * p.QG)
            cp = runs_of(p, shared, before_pre, g * shared.row_tiles + (at >> p.row_shift), len);
        const int mine = co.c1 - co.c0 + 1, all = mine + cp.c1 - cp.c0 + 1;
        Acc<TURNS> acc;
        acc.add_all(all, j0, JUMP, [&](int k) -> StateAt {
            const bool of_own = k < mine;
            if (of_own ? co.c0 == co.c1 : cp.c0 == cp.c1) {
                const DirectAt d = direct_at<D>(p, of_own ? 0 : 1, row);
                return {d.m, d.l, d.o, 4};
            }
            return of_own ? run_state<D>(p, co.c0 + k, co.c0, r & ((1 << p.row_shift) - 1))
                          : run_state<D>(p, cp.c0 + k - mine, cp.c0, at & ((1 << p.row_shift) - 1));
        });
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
    if (ri < ROWS && rr < rows) {
        const int64_t to = static_cast<int64_t>(s.first + rr / p.QG) * p.Hq + g * p.QG + rr % p.QG;
        *reinterpret_cast<uint4*>(p.O + to * D + 8 * c) =
            *reinterpret_cast<const uint4*>(&stage[ri][2 * c]);
    }
}

}  // namespace

static size_t slot_floats(int D, int num_sms) {
    return (static_cast<size_t>(2 * kCtasPerSm * num_sms) << kRowShift) * (D + 2);
}

// States by run, states by (token, head) of the sequences' own part and the prefixes', and
// the units before each entry (no more prefixes than sequences).
static size_t direct_floats(int D, int64_t rows) { return 2 * static_cast<size_t>(rows) * (D + 2); }

size_t prefix_attention_workspace(int D, int64_t rows, int B, int num_sms) {
    return (slot_floats(D, num_sms) + direct_floats(D, rows)) * sizeof(float) +
           (2 * static_cast<size_t>(B) + 2) * sizeof(long long);
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
    const int QG = Hq / c.Hkv;
    const int64_t pieces = (static_cast<int64_t>(N) * QG + (1 << kFewRowShift) - 1) >> kFewRowShift;
    const int64_t slots = static_cast<int64_t>(pre.max_pages) * c.page_size;
    const bool few = T * QG <= 1 << kFewRowShift &&
                     (pieces == 1 || (slots <= kFewSlots && pieces * slots * c.Hkv <= kFewReads));
    int rc = few ? tree_setup(c, q, q_stride, O, N, T, Hq, cu, parents, scale, ws,
                              kFewCtasPerSm * num_sms, kFewRowShift, kFewTileShift, kFewMinRun,
                              kFewSetup, &p, &kmap, &vmap)
                 : tree_setup(c, q, q_stride, O, N, T, Hq, cu, parents, scale, ws,
                              kCtasPerSm * num_sms, kRowShift, kTcTileShift, 6, fp8 ? 8 : 4, &p,
                              &kmap, &vmap);
    if (rc != cudaSuccess) return rc;
    p.pre.table = pre.table;
    p.pre.lens = pre.lens;
    p.pre.first = pre.first;
    p.pre.G = pre.G;
    p.pre.max_pages = pre.max_pages;
    p.pre.cap = pre.max_pages * c.page_size;
    p.pre.direct = ws + slot_floats(c.D, num_sms);
    p.plan = reinterpret_cast<long long*>(
        p.pre.direct + direct_floats(c.D, static_cast<int64_t>(N) * Hq));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = few ? launch_tree_few_shared(kmap, vmap, p, c.D, fp8, device, st)
             : launch_prefix_tc(kmap, vmap, p, c.D, fp8, device, st);
    if (rc != cudaSuccess) return rc;
    const int rows = T * p.QG, block_rows = rows <= 8 ? 8 : 16;
    const int chunks = (rows + block_rows - 1) / block_rows;
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs la;
    apply_pdl(cfg, la);
    cfg.gridDim = dim3(static_cast<unsigned>(chunks) * c.Hkv, c.B, 1);
    cfg.blockDim = dim3(16 * block_rows, 1, 1);
    cfg.stream = st;
    auto run = [&](auto kernel) {
        return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p, chunks));
    };
    if (c.D == 128)
        return rows <= 8 ? run(prefix_merge_kernel<128, 8>) : run(prefix_merge_kernel<128, 16>);
    return rows <= 8 ? run(prefix_merge_kernel<64, 8>) : run(prefix_merge_kernel<64, 16>);
}

}  // namespace qmm
