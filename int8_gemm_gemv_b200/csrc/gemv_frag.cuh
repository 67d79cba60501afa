// Device code shared by the kernels that stream E4M3 weights past a few rows of
// FP16 activations with warp-level MMAs (gemv_fp8.cu, moe_fp8.cu).  A warp
// works on a chunk of 16 weight rows x 64 bytes of K: lane (g, t) holds bytes
// [16t, 16t + 16) of rows g and g + 8, and the same K positions of its
// activation row, so the order of K inside an MMA is the same for both.
#pragma once

#include "bsq_common.cuh"

namespace bsq {
namespace gv {

constexpr int CH = 64;  // weight bytes (= K elements) of one warp chunk

// Byte offset of 16-byte unit t of row r in a chunk [rows][64 B], 64-byte
// swizzle (unit t of row r sits at unit t ^ ((r >> 1) & 3)).
__device__ __forceinline__ uint32_t w_off(int r, int t) { return (uint32_t)(r * CH + ((t ^ ((r >> 1) & 3)) << 4)); }
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
    return r;
}

__device__ __forceinline__ uint4 ldg_nc_v4(const void *p) {
    uint4 r;
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// Four E4M3 bytes (byte 0 = lowest K index) -> two FP16x2 (bytes 0, 1 in
// lo; bytes 2, 3 in hi), exact: every E4M3 value is an FP16 normal or zero.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t four, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

// Two BF16 values times the power of two f, rounded to FP16x2: exact when
// the scaled value is representable, which the caller's choice of f makes
// true for every element within 2^31 of its row's largest magnitude.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2_scaled(uint32_t two, float f) {
    const uint64_t v = ((uint64_t)(two & 0xFFFF0000u) << 32) | (uint64_t)(two << 16);  // {lo, hi} as FP32
    uint64_t p;
    const uint64_t ff = ((uint64_t)__float_as_uint(f) << 32) | __float_as_uint(f);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(v), "l"(ff));
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float((uint32_t)(p >> 32))),
        "f"(__uint_as_float((uint32_t)p)));
    return r;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^e for -127 <= e <= 127 (2^-127 is the one subnormal needed).
__device__ __forceinline__ float pow2i(int e) {
    return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(0x00400000u);
}

// The power of two 2^s that puts a row's largest magnitude (given as BF16
// bits) in [2^14, 2^15): the row times 2^s converts to FP16 without overflow,
// and exactly for every element within 2^31 of that magnitude.  Zero rows
// get s = 0.
__device__ __forceinline__ int row_shift(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 7) - 127;  // floor(log2); BF16 subnormals count as 2^-127
    return amax_bits == 0 ? 0 : min(14 - e, 127);
}

// A lane's share of one chunk: weight rows g and g + 8 (16 E4M3 bytes each)
// and the FP16 activation fragments of rows g (xa) and g + 8 (xb, MT == 2),
// 16 elements each, at the same 16 K positions.
template <int MT>
struct Frag {
    uint4 wa, wb;
    uint32_t xa[8], xb[8];
};

// d[i] (+)= W[16 rows of the chunk] x X[8 rows of n-tile i]^T over the
// chunk's 64 K positions.
template <int MT>
__device__ __forceinline__ void chunk_mma(float (&d)[MT][4], const Frag<MT> &f) {
    const uint32_t a_w[4] = {f.wa.x, f.wa.y, f.wa.z, f.wa.w};
    const uint32_t b_w[4] = {f.wb.x, f.wb.y, f.wb.z, f.wb.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint32_t a[4];
        e4m3x4_to_f16x2(a_w[j], a[0], a[2]);  // row g:   k 4j, 4j+1 | 4j+2, 4j+3
        e4m3x4_to_f16x2(b_w[j], a[1], a[3]);  // row g+8: the same K
        mma_f16_16816(d[0], a, f.xa[2 * j], f.xa[2 * j + 1]);
        if (MT == 2) mma_f16_16816(d[MT - 1], a, f.xb[2 * j], f.xb[2 * j + 1]);
    }
}

template <int MT>
__device__ __forceinline__ void x_to_f16(const uint4 (&v)[2], float f, uint32_t (&o)[8]) {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int j = 0; j < 8; j++) o[j] = bf16x2_to_f16x2_scaled(w[j], f);
}

}  // namespace gv
}  // namespace bsq
