// Producers of FP8 activations for the block-scaled and row-scaled FP8 GEMMs,
// all one pass over their input:
//   rmsnorm_residual_quant_fp8  h = BF16(x + residual); RMS norm; E4M3 codes
//                               with one FP32 scale per 128 or per row
//   quant_act_fp8_per128        BF16 -> E4M3, one FP32 scale per 128
//   silu_mul_quant_fp8_per128   silu(gate) * up -> E4M3, one scale per 128
//
// Codes are those of the correctly rounded quotient y / s, s = amax / 448,
// found without a division per element (quant_codes.cuh; its argument needs no
// more of the numerator than being FP32).
//
// Eight lanes hold one group of 128, sixteen consecutive elements (a "unit")
// each: 32 bytes loaded and 16 stored per lane, three shuffles for the amax.
//
// Launched with programmatic stream serialization: a GEMM behind may set up
// while these run, and these wait for the kernel before them before they touch
// memory.
#include "quant_codes.cuh"

namespace bsq {

namespace {

using namespace qc;

struct Unit {
    uint32_t w[8];  // sixteen BF16 values, element 2j in the low half of w[j]
};

// 32 bytes through two 16-byte loads (only 16-byte alignment is asked of the
// caller's pointers).
__device__ __forceinline__ Unit ld_unit(const uint16_t *p) {
    const uint4 a = ld_nc_v4(p), b = ld_nc_v4(p + 8);
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
// The same for memory that this kernel may write later (in-place residuals).
__device__ __forceinline__ Unit ld_unit_rw(const uint16_t *p) {
    const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ Unit zero_unit() { return {{0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}}; }

__device__ __forceinline__ void unpack_unit(const Unit &v, float (&y)[16]) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
        y[2 * j] = lo_bf16(v.w[j]);
        y[2 * j + 1] = hi_bf16(v.w[j]);
    }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
// E4M3 codes of four values, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(uint64_t a, uint64_t b) {
    return (uint32_t)f32x2_to_e4m3x2(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32))) |
           (uint32_t)f32x2_to_e4m3x2(__uint_as_float((uint32_t)b), __uint_as_float((uint32_t)(b >> 32))) << 16;
}

// Sixteen E4M3 codes of y / s; s == 0 (an all-zero group) gives zeros.
// With r = rcp.approx(s), within 2^-23, the products y r (1 -+ 2^-20) lie on
// either side of RN(y / s) (their own roundings are 2^-24 each): where the
// codes of both agree they are the answer, for all sixteen in one comparison.
// Otherwise the pairs that differ are settled one by one.  (A branch per pair,
// at 2^-16, instead: SiLU 2048 x 17408 9% and norm 8192 x 5120 3% slower.)
__device__ __forceinline__ uint4 codes_16(const float (&y)[16], float s) {
    if (s == 0.0f) return make_uint4(0u, 0u, 0u, 0u);
    const Bracket br = bracket_of(s);
    uint32_t w[4];
    if (br.ok) {
        const float l = __fmul_rn(br.r, 1.0f - 0x1p-20f), h = __fmul_rn(br.r, 1.0f + 0x1p-20f);
        const uint64_t ll = f32x2_pack(l, l), hh = f32x2_pack(h, h);
        uint32_t d[4];  // bits in which the two codes differ
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint64_t a = f32x2_pack(y[4 * j], y[4 * j + 1]), b = f32x2_pack(y[4 * j + 2], y[4 * j + 3]);
            w[j] = e4m3x4(mul2(a, ll), mul2(b, ll));
            d[j] = w[j] ^ e4m3x4(mul2(a, hh), mul2(b, hh));
        }
        if ((d[0] | d[1] | d[2] | d[3]) != 0u) {
#pragma unroll
            for (int p = 0; p < 8; p++) {
                const uint32_t dp = (d[p >> 1] >> (16 * (p & 1))) & 0xFFFFu;
                if (dp != 0u) {
                    float p0 = __fmul_rn(y[2 * p], l), p1 = __fmul_rn(y[2 * p + 1], l);
                    pair_boundaries<5, 8>(y[2 * p], y[2 * p + 1], s, p0, p1, 0u, dp);
                    const uint32_t c = f32x2_to_e4m3x2(p0, p1);
                    w[p >> 1] = p & 1 ? (w[p >> 1] & 0xFFFFu) | c << 16 : (w[p >> 1] & 0xFFFF0000u) | c;
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            w[j] = (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(y[4 * j], s), __fdiv_rn(y[4 * j + 1], s)) |
                   (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(y[4 * j + 2], s), __fdiv_rn(y[4 * j + 3], s)) << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The larger value, NaN where either is: a group with a NaN gets a NaN scale
// and NaN codes, as in the quantiser, whose maximum of the BF16 bits ranks NaN
// highest.  (fmaxf drops NaN, and a group of nothing else would become zeros.)
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

__device__ __forceinline__ float amax_16(const float (&y)[16]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) m = max_nan(m, fabsf(y[i]));
    return m;
}

// Max over the eight lanes of a group.
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

constexpr int kThreads = 256;

// One lane per unit and UNROLL units per lane, all loads first; group g of the
// flattened [m, k] matrix is entry g of the scale matrix.  The eight lanes of
// a group are in or out of range together; the shuffles name all lanes, so
// every lane of a warp reaches them.
template <int UNROLL>
__global__ void __launch_bounds__(kThreads) k_quant_act_fp8_per128(const uint16_t *__restrict__ in,
                                                                   uint8_t *__restrict__ q,
                                                                   float *__restrict__ scale, int64_t units) {
    launch_dependents();
    dependency_wait();
    const int64_t u0 = (int64_t)blockIdx.x * kThreads * UNROLL + threadIdx.x;
    Unit v[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; i++) {
        const int64_t u = u0 + i * kThreads;
        v[i] = u < units ? ld_unit(in + 16 * u) : zero_unit();
    }
#pragma unroll
    for (int i = 0; i < UNROLL; i++) {
        const int64_t u = u0 + i * kThreads;
        // the amax from the BF16 bits: magnitudes order as they do
        uint32_t mx = max(amax_bits_8(make_uint4(v[i].w[0], v[i].w[1], v[i].w[2], v[i].w[3])),
                          amax_bits_8(make_uint4(v[i].w[4], v[i].w[5], v[i].w[6], v[i].w[7])));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const float s = __fdiv_rn(__uint_as_float(mx << 16), 448.0f);
        if (u >= units) continue;
        float y[16];
        unpack_unit(v[i], y);
        *reinterpret_cast<uint4 *>(q + 16 * u) = codes_16(y, s);
        if ((threadIdx.x & 7) == 0) scale[u >> 3] = s;
    }
}

// silu(g) * u.  With z = exp(-|g|) in (0, 1], sigmoid(g) is 1 / (1 + z) or z /
// (1 + z): the reciprocal's argument lies in [1, 2], where the approximate one
// is good to an ulp and nothing overflows.
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float z = expf(-fabsf(g));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + z));
    return g * (g < 0.0f ? z * r : r) * u;
}

// gate_up rows are [gate (k) | up (k)].
template <int UNROLL>
__global__ void __launch_bounds__(kThreads) k_silu_mul_quant_fp8_per128(const uint16_t *__restrict__ gate_up,
                                                                        uint8_t *__restrict__ q,
                                                                        float *__restrict__ scale, int k,
                                                                        int64_t units) {
    launch_dependents();
    dependency_wait();
    const int64_t u0 = (int64_t)blockIdx.x * kThreads * UNROLL + threadIdx.x;
    const uint32_t per_row = (uint32_t)k >> 4;
    Unit g[UNROLL], up[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; i++) {
        const int64_t u = u0 + i * kThreads;
        // the division is 32-bit while the matrix has fewer than 2^32 units
        const int64_t row = units <= 0xFFFFFFFFll ? (int64_t)((uint32_t)u / per_row) : u / per_row;
        const uint16_t *p = gate_up + row * k + 16 * u;  // row * 2k + 16 * (u - row * per_row)
        g[i] = u < units ? ld_unit(p) : zero_unit();
        up[i] = u < units ? ld_unit(p + k) : zero_unit();
    }
#pragma unroll
    for (int i = 0; i < UNROLL; i++) {
        const int64_t u = u0 + i * kThreads;
        float y[16];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            y[2 * j] = silu_mul(lo_bf16(g[i].w[j]), lo_bf16(up[i].w[j]));
            y[2 * j + 1] = silu_mul(hi_bf16(g[i].w[j]), hi_bf16(up[i].w[j]));
        }
        const float s = __fdiv_rn(group_max(amax_16(y)), 448.0f);
        if (u >= units) continue;
        *reinterpret_cast<uint4 *>(q + 16 * u) = codes_16(y, s);
        if ((threadIdx.x & 7) == 0) scale[u >> 3] = s;
    }
}

// ---------------------------------------------------------------------------
// RMS norm.  A row is held in registers as BF16 between the sum of squares and
// the codes, KEEP units per thread: one warp per row (eight rows per CTA, no
// barrier) up to K = 1024, else one CTA per row.
//
// The squares are added in an order that follows from K alone (a unit's
// sixteen in turn, 32 units by halves, then those sums by halves), however
// many units a thread holds, so a row alone and in a batch gives the same
// bits.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Two sums over the warp, added as warp_sum does: a's in lanes 0 to 15, b's in
// lanes 16 to 31.
__device__ __forceinline__ float warp_sum2(float a, float b, int lane) {
    float v = lane & 16 ? b : a;
    v += __shfl_xor_sync(0xFFFFFFFFu, lane & 16 ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

constexpr int kRowsPerCta = 8;  // of the one-warp form

template <int KEEP, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 32 * kRowsPerCta : 1024)
    k_rmsnorm_residual_quant_fp8(const uint16_t *x, const uint16_t *residual,
                                             const uint16_t *__restrict__ gain, float eps, uint16_t *residual_out,
                                             uint8_t *__restrict__ q, float *__restrict__ scale, int per_row, int m,
                                             int k) {
    __shared__ float sums[WARP_ROW ? 1 : 32 * KEEP], maxima[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * kRowsPerCta + warp : blockIdx.x;
    const int tid = WARP_ROW ? lane : threadIdx.x, nt = WARP_ROW ? 32 : blockDim.x;
    const int units = k >> 4;
    launch_dependents();
    dependency_wait();
    if (row >= m) return;

    Unit h[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; i++) {
        const int u = tid + i * nt;
        h[i] = u < units ? ld_unit_rw(x + row * k + 16 * u) : zero_unit();
    }
    if (residual != nullptr) {
        Unit r[KEEP];
#pragma unroll
        for (int i = 0; i < KEEP; i++) {
            const int u = tid + i * nt;
            r[i] = u < units ? ld_unit_rw(residual + row * k + 16 * u) : zero_unit();
        }
#pragma unroll
        for (int i = 0; i < KEEP; i++)
#pragma unroll
            for (int j = 0; j < 8; j++)
                h[i].w[j] = pack_bf16x2(__fadd_rn(lo_bf16(h[i].w[j]), lo_bf16(r[i].w[j])),
                                        __fadd_rn(hi_bf16(h[i].w[j]), hi_bf16(r[i].w[j])));
    }
    float sq[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; i++) {
        const int u = tid + i * nt;
        if (residual_out != nullptr && u < units) {
            uint4 *o = reinterpret_cast<uint4 *>(residual_out + row * k + 16 * u);
            o[0] = make_uint4(h[i].w[0], h[i].w[1], h[i].w[2], h[i].w[3]);
            o[1] = make_uint4(h[i].w[4], h[i].w[5], h[i].w[6], h[i].w[7]);
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            sq[i] = fmaf(lo_bf16(h[i].w[j]), lo_bf16(h[i].w[j]), j == 0 ? 0.0f : sq[i]);
            sq[i] = fmaf(hi_bf16(h[i].w[j]), hi_bf16(h[i].w[j]), sq[i]);
        }
    }
    float ss = 0.0f;
    if (WARP_ROW) {
#pragma unroll
        for (int i = 0; i < KEEP; i++) ss += sq[i];
    } else {
        // units 32 c .. 32 c + 31 to sums[c]: warp + i * warps is the c of a warp's i-th units
        const int warps = nt >> 5, all = KEEP * warps;
        if (KEEP == 1) {
            const float v = warp_sum(sq[0]);
            if (lane == 0) sums[warp] = v;
        } else {
#pragma unroll
            for (int i = 0; i < KEEP; i += 2) {
                const float v = warp_sum2(sq[i], sq[i + (KEEP > 1)], lane);
                if ((lane & 15) == 0) sums[warp + (i + (lane >> 4)) * warps] = v;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KEEP; i++) ss += lane + 32 * i < all ? sums[lane + 32 * i] : 0.0f;
    }
    ss = warp_sum(ss);
    const float mean = __fdiv_rn(ss, (float)k) + eps;
    // (a row of zeros without eps: zeros, not 0 * inf; a sum that overflowed, or
    // a NaN in the row: NaN, not zeros)
    const float f = mean == 0.0f ? 0.0f : mean < INFINITY ? rsqrtf(mean) : __uint_as_float(0x7FFFFFFFu);
    auto normed = [&](int i, float(&y)[16]) {
        const int u = tid + i * nt;
        const Unit g = u < units ? ld_unit(gain + 16 * u) : zero_unit();
#pragma unroll
        for (int j = 0; j < 8; j++) {
            y[2 * j] = __fmul_rn(__fmul_rn(lo_bf16(h[i].w[j]), f), lo_bf16(g.w[j]));
            y[2 * j + 1] = __fmul_rn(__fmul_rn(hi_bf16(h[i].w[j]), f), hi_bf16(g.w[j]));
        }
    };
    float s = 0.0f;
    if (per_row) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < KEEP; i++) {
            float y[16];
            normed(i, y);
            mx = max_nan(mx, amax_16(y));
        }
        mx = warp_max(mx);
        if (!WARP_ROW) {
            if (lane == 0) maxima[warp] = mx;
            __syncthreads();
            mx = warp_max(lane < (nt >> 5) ? maxima[lane] : 0.0f);
        }
        s = __fdiv_rn(mx, 448.0f);
        if (tid == 0) scale[row] = s;
    }
#pragma unroll
    for (int i = 0; i < KEEP; i++) {
        const int u = tid + i * nt;
        float y[16];
        normed(i, y);
        if (!per_row) {
            s = __fdiv_rn(group_max(amax_16(y)), 448.0f);
            if (u < units && (u & 7) == 0) scale[row * (k >> 7) + (u >> 3)] = s;
        }
        if (u < units) *reinterpret_cast<uint4 *>(q + row * k + 16 * u) = codes_16(y, s);
    }
}

template <class... P, class... A>
cudaError_t launch_pss(void (*kernel)(P...), int64_t grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (e == cudaSuccess) note_launch();
    return e;
}

// Units per lane: two where the units are three times the threads the SMs hold
// or more (836 rows of 17408: quantiser 10.9 us, 11.3 with one, SiLU 15.7 and
// 15.8; 4096 rows: 39.6 and 43.9, 63.4 and 67.3, the quantiser with four
// 55.0), one below (512 rows: quantiser 7.9 us, 8.2 with two, SiLU 10.5 and
// 10.7; 128 rows: 3.6 and 4.6, 4.5 and 5.9).
bool two_units(int64_t units) { return units >= (int64_t)sm_count() * 2048 * 3; }
int64_t grid_for_units(int64_t units, int unroll) { return (units + (int64_t)kThreads * unroll - 1) / (kThreads * unroll); }

}  // namespace

cudaError_t launch_quant_act_fp8_per128(const uint16_t *a, uint8_t *q, float *scale, int m, int k, cudaStream_t s) {
    const int64_t units = (int64_t)m * k / 16;
    return two_units(units)
               ? launch_pss(k_quant_act_fp8_per128<2>, grid_for_units(units, 2), kThreads, s, a, q, scale, units)
               : launch_pss(k_quant_act_fp8_per128<1>, grid_for_units(units, 1), kThreads, s, a, q, scale, units);
}

cudaError_t launch_silu_mul_quant_fp8_per128(const uint16_t *gate_up, uint8_t *q, float *scale, int m, int k,
                                             cudaStream_t s) {
    const int64_t units = (int64_t)m * k / 16;
    return two_units(units) ? launch_pss(k_silu_mul_quant_fp8_per128<2>, grid_for_units(units, 2), kThreads, s, gate_up,
                                         q, scale, k, units)
                            : launch_pss(k_silu_mul_quant_fp8_per128<1>, grid_for_units(units, 1), kThreads, s, gate_up,
                                         q, scale, k, units);
}

cudaError_t launch_rmsnorm_residual_quant_fp8(const uint16_t *x, const uint16_t *residual, const uint16_t *gain,
                                              float eps, uint16_t *residual_out, uint8_t *q, float *scale, int group,
                                              int m, int k, cudaStream_t s) {
    const int units = k >> 4, per_row = group == 0;
    auto warp_rows = [&](auto kernel) {
        return launch_pss(kernel, ((int64_t)m + kRowsPerCta - 1) / kRowsPerCta, 32 * kRowsPerCta, s, x, residual, gain,
                          eps, residual_out, q, scale, per_row, m, k);
    };
    auto cta_rows = [&](auto kernel, int keep) {
        return launch_pss(kernel, m, (units + 32 * keep - 1) / (32 * keep) * 32, s, x, residual, gain, eps, residual_out,
                          q, scale, per_row, m, k);
    };
    if (units <= 32) return warp_rows(k_rmsnorm_residual_quant_fp8<1, true>);
    if (units <= 64) return warp_rows(k_rmsnorm_residual_quant_fp8<2, true>);
    // One unit per thread for short rows (4000 rows: 160 units 15.3 us, 15.8
    // with two; 168 units 16.8 and 16.4), for no more rows than SMs (1024 units:
    // 148 rows 5.0 and 5.1, 160 rows 8.1 and 7.0), and, for a medium length,
    // while the rows have no more than 1024 units per SM (320 units: 470 rows
    // 5.3 and 6.7, 600 rows 6.2 and 6.8, 1000 rows 9.5 and 9.4, 4000 rows 28.7
    // and 26.2); else two, which keep more loads in flight per warp (4000 x
    // 1024 units: 78.0 us, 109.1 with one).  The lengths that count as medium
    // end where such batches stop gaining (470 rows: 384 units 6.0 and 6.9, 392
    // units 6.6 and 6.4, 512 units 7.7 and 7.1).  Scale per row.
    const int64_t sms = sm_count();
    if (units <= 160 || (units <= 384 && (int64_t)m * units <= 1024 * sms) || (units <= 1024 && m <= sms))
        return cta_rows(k_rmsnorm_residual_quant_fp8<1, false>, 1);
    if (units <= 1024 * 2) return cta_rows(k_rmsnorm_residual_quant_fp8<2, false>, 2);
    return cta_rows(k_rmsnorm_residual_quant_fp8<4, false>, 4);
}

}  // namespace bsq
