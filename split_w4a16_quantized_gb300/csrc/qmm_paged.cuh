// The paged KV cache on the device: token ranges of a batch and addresses of
// slots, shared by the append, tree attention and accept kernels.
#pragma once

#include <cstdint>

#include "qmm.h"

namespace qmm {

struct PagedDims {
    const int* table;
    const int* lens;
    int64_t page_stride, head_stride, slot_stride;  // elements
    int B, num_pages, max_pages, page_shift, Hkv;
    int cap;  // slots of a sequence's table
};

inline PagedDims paged_dims(const qmm_kv_cache& c) {
    PagedDims d;
    d.table = c.table;
    d.lens = c.lens;
    // a dimension of one row has no stride: whatever the caller holds there
    // (views of one head or one page) must not reach an address or a map
    d.page_stride = c.num_pages > 1 ? c.page_stride : c.D;
    d.head_stride = c.Hkv > 1 ? c.head_stride : c.D;
    d.slot_stride = c.page_size > 1 ? c.slot_stride : c.D;
    d.B = c.B;
    d.num_pages = c.num_pages;
    d.max_pages = c.max_pages;
    d.page_shift = 0;
    while ((1 << d.page_shift) < c.page_size) ++d.page_shift;
    d.Hkv = c.Hkv;
    d.cap = c.max_pages * c.page_size;
    return d;
}

// Two FP32 values in one register pair, and arithmetic on both at once.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// A value of lens or cu.  kFromL2: at GPU scope, past this SM's L1, for a kernel
// that reads it before its own dependency wait.
template <bool kFromL2>
__device__ __forceinline__ int plan_value(const int* at) {
    if (!kFromL2) return *at;
    int v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(at));
    return v;
}

// Tokens in the cache of sequence b before the call.
template <bool kFromL2 = false>
__device__ __forceinline__ int cached_tokens(const PagedDims& d, int b) {
    const int len = plan_value<kFromL2>(d.lens + b);
    return len < 0 ? 0 : (len > d.cap ? d.cap : len);
}

// New tokens of sequence b: rows [first, first + n).  cu's values are the
// caller's device data, so they are clamped to the N rows there are.
template <bool kFromL2 = false>
__device__ __forceinline__ void token_range(const int* cu, int N, int T, int b, int* first,
                                            int* n) {
    if (!cu) {
        *first = b * T;
        *n = T;
        return;
    }
    int a = plan_value<kFromL2>(cu + b), e = plan_value<kFromL2>(cu + b + 1);
    a = a < 0 ? 0 : (a > N ? N : a);
    e = e < a ? a : (e > N ? N : e);
    *first = a;
    *n = e - a < T ? e - a : T;
}

// Element offset of slot s of sequence b for head 0, or -1 where it has no page.
__device__ __forceinline__ int64_t slot_offset(const PagedDims& d, int b, int s) {
    const int pi = s >> d.page_shift;
    if (s < 0 || pi >= d.max_pages) return -1;
    const int page = d.table[static_cast<int64_t>(b) * d.max_pages + pi];
    if (page < 0 || page >= d.num_pages) return -1;
    return page * d.page_stride + (s & ((1 << d.page_shift) - 1)) * d.slot_stride;
}

}  // namespace qmm
