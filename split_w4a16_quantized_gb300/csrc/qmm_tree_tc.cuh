// The tcgen05 pieces that tree attention and the pass over the weights share:
// descriptors of operands in shared memory, products, loads of tensor memory, and a row
// of q as two E4M3 terms.
#pragma once

#include "qmm_tree.cuh"

namespace qmm {

// A ring position.
struct Cursor {
    int slot = 0, phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) slot = 0, phase ^= 1;
    }
};

// Instruction descriptor, FP32 accumulate, M = 128, K-major A, B K-major or
// N-major; format 0: F16 (kind::f16) or E4M3 (kind::f8f6f4), 1: BF16.
__host__ __device__ constexpr uint32_t idesc(int N, uint32_t format, bool b_n_major) {
    return (1u << 4) | (format << 7) | (format << 10) | ((b_n_major ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

// Shared-memory descriptor, K-major rows of kRow (128 or 64) bytes with the
// swizzle of that width; 8 rows apart: 8 kRow bytes.
template <int kRow>
__device__ __forceinline__ uint64_t sdesc_k_major(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>((8 * kRow) >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(kRow == 128 ? 2 : 4) << 61);
}
// D[tmem] (+)= A[smem] B[smem].
template <bool kF8>
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    if (kF8)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// 32 lanes x 32 columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
// 8 columns of each of 32 lanes.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(
                     taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                 "r"(v[7])
                 : "memory");
}
// Offset of 16-byte chunk c of row r in a tile of kRows rows: boxes of kBox
// bytes a row, the chunk permuted by the swizzle of that width.
template <int kBox, int kRows>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    if (kBox == 128)
        return static_cast<uint32_t>((c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// The scaling of a row of q for two E4M3 terms, from the bits of its largest magnitude
// (`big`; NaN above all): `up` takes the largest to [128, 256), qs becomes the factor on
// the row's scores.  A row that holds infinities or NaN becomes NaN (what its softmax
// would be).
__device__ __forceinline__ float e4m3_scaling(uint32_t big, float* qs) {
    // 2^e <= big < 2^(e+1)
    int e = static_cast<int>(big >> 23) - 127;
    const bool bad = e >= 128;
    e = big > 0 && !bad ? max(-110, e) : 0;
    *qs = finite_factor(*qs * __uint_as_float(static_cast<uint32_t>(120 + e) << 23));
    return bad ? __int_as_float(0x7fffffff)
               : __uint_as_float(static_cast<uint32_t>(134 - e) << 23);
}
__device__ __forceinline__ uint32_t bf16_magnitude(uint32_t big, uint32_t w) {
    return max(big, max((w & 0x7fffu) << 16, w & 0x7fff0000u));
}
// Two BF16 values (a pair's bits) times `up` as two E4M3 terms each: the first is the
// value rounded to 4 significant bits, the second what is left of it (at most 4 bits),
// both to a multiple of E4M3's smallest, 2^-9.
__device__ __forceinline__ void e4m3_terms(uint32_t w, float up, uint32_t* hi, uint32_t* lo) {
    const float f0 = __uint_as_float(w << 16) * up;
    const float f1 = __uint_as_float(w & 0xffff0000u) * up;
    *hi = __nv_cvt_float2_to_fp8x2(make_float2(f0, f1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t back = e4m3x2_to_f16x2(*hi);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&back));
    *lo = __nv_cvt_float2_to_fp8x2(make_float2(f0 - h.x, f1 - h.y), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace qmm
