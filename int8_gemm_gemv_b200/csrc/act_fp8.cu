// Producers of FP8 activations for the block-scaled and row-scaled FP8 GEMMs,
// all one pass over their input:
//   rmsnorm_residual_quant_fp8  h = BF16(x + residual); RMS norm; E4M3 codes
//                               with one FP32 scale per 128 or per row
//   quant_act_fp8_per128        BF16 -> E4M3, one FP32 scale per 128
//   silu_mul_quant_fp8_per128   silu(gate) * up -> E4M3, one scale per 128
//
// Codes are those of the correctly rounded quotient y / s, s = amax / 448,
// found without a division per element (quant_codes.cuh).
//
// Eight lanes hold one group of 128, sixteen consecutive elements each: a
// 32-byte load and a 16-byte store per lane, three shuffles for the amax.
#include "quant_codes.cuh"

namespace bsq {

namespace {

using namespace qc;

struct Bf16x16 {
    uint32_t w[8];  // sixteen BF16 values, element 2j in the low half of w[j]
};

// 32 bytes through two 16-byte loads (only 16-byte alignment is asked of the
// caller's pointers).
__device__ __forceinline__ Bf16x16 ld16(const uint16_t *p) {
    const uint4 a = ld_nc_v4(p), b = ld_nc_v4(p + 8);
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// Sixteen E4M3 codes of y / s; s == 0 (an all-zero group) gives zeros.
__device__ __forceinline__ uint4 codes_16(const float (&y)[16], float s) {
    if (s == 0.0f) return make_uint4(0u, 0u, 0u, 0u);
    const Bracket br = bracket_of(s);
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        lo[i] = y[i];
        hi[i] = y[8 + i];
    }
    const uint2 a = e4m3_codes_8(lo, s, br), b = e4m3_codes_8(hi, s, br);
    return make_uint4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ float amax_16(const float (&y)[16]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) m = fmaxf(m, fabsf(y[i]));
    return m;
}

// Max over the eight lanes of a group.
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

__device__ __forceinline__ void unpack_16(const Bf16x16 &v, float (&y)[16]) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
        y[2 * j] = lo_bf16(v.w[j]);
        y[2 * j + 1] = hi_bf16(v.w[j]);
    }
}

constexpr int kThreads = 256;

// One lane per sixteen elements; m * k / 16 lanes in all.  Group g of the
// flattened [m, k] matrix is row-major group g of the scale matrix.
__global__ void __launch_bounds__(kThreads) k_quant_act_fp8_per128(const uint16_t *__restrict__ in,
                                                                   uint8_t *__restrict__ q,
                                                                   float *__restrict__ scale, int64_t units) {
    // whole groups of eight lanes are in or out together; the shuffles name
    // all lanes, so every lane of a warp stays in the loop
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t u0 = (int64_t)blockIdx.x * kThreads; u0 < units; u0 += stride) {
        const int64_t u = u0 + threadIdx.x;
        const bool in_range = u < units;
        float y[16];
        unpack_16(in_range ? ld16(in + 16 * u) : Bf16x16{}, y);
        const float s = __fdiv_rn(group_max(amax_16(y)), 448.0f);
        if (!in_range) continue;
        *reinterpret_cast<uint4 *>(q + 16 * u) = codes_16(y, s);
        if ((threadIdx.x & 7) == 0) scale[u >> 3] = s;
    }
}

// gate_up rows are [gate (k) | up (k)].
__global__ void __launch_bounds__(kThreads) k_silu_mul_quant_fp8_per128(const uint16_t *__restrict__ gate_up,
                                                                        uint8_t *__restrict__ q,
                                                                        float *__restrict__ scale, int k,
                                                                        int64_t units) {
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    const int per_row = k >> 4;
    for (int64_t u0 = (int64_t)blockIdx.x * kThreads; u0 < units; u0 += stride) {
        const int64_t u = u0 + threadIdx.x;
        const bool in_range = u < units;
        const int64_t row = u / per_row, c = u - row * per_row;
        const uint16_t *g = gate_up + row * 2 * k + 16 * c;
        float gv[16], y[16];
        unpack_16(in_range ? ld16(g) : Bf16x16{}, gv);
        unpack_16(in_range ? ld16(g + k) : Bf16x16{}, y);
#pragma unroll
        for (int i = 0; i < 16; i++) y[i] *= __fdiv_rn(gv[i], 1.0f + expf(-gv[i]));
        const float s = __fdiv_rn(group_max(amax_16(y)), 448.0f);
        if (!in_range) continue;
        *reinterpret_cast<uint4 *>(q + 16 * u) = codes_16(y, s);
        if ((threadIdx.x & 7) == 0) scale[u >> 3] = s;
    }
}

// ---------------------------------------------------------------------------
// One CTA per row; the row is read twice here.
__device__ __forceinline__ float cta_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < kThreads / 32; i++) v += red[i];
    return v;
}

__global__ void __launch_bounds__(kThreads)
    k_rmsnorm_residual_quant_fp8(const uint16_t *x, const uint16_t *residual, const uint16_t *__restrict__ gain,
                                 float eps, uint16_t *residual_out, uint8_t *__restrict__ q,
                                 float *__restrict__ scale, int per_row, int k) {
    __shared__ float red[kThreads / 32], red_max[kThreads / 32];
    const int64_t row = blockIdx.x;
    const int units = k >> 4;
    extern __shared__ uint4 row_h[];  // the row of h, BF16
    float ss = 0.0f;
    for (int u = threadIdx.x; u < 2 * units; u += kThreads) {
        const int64_t o = row * k + 8 * (int64_t)u;
        uint4 h = *reinterpret_cast<const uint4 *>(x + o);
        if (residual != nullptr) {
            const uint4 r = *reinterpret_cast<const uint4 *>(residual + o);
            h = make_uint4(pack_bf16x2(lo_bf16(h.x) + lo_bf16(r.x), hi_bf16(h.x) + hi_bf16(r.x)),
                           pack_bf16x2(lo_bf16(h.y) + lo_bf16(r.y), hi_bf16(h.y) + hi_bf16(r.y)),
                           pack_bf16x2(lo_bf16(h.z) + lo_bf16(r.z), hi_bf16(h.z) + hi_bf16(r.z)),
                           pack_bf16x2(lo_bf16(h.w) + lo_bf16(r.w), hi_bf16(h.w) + hi_bf16(r.w)));
        }
        row_h[u] = h;
        if (residual_out != nullptr) *reinterpret_cast<uint4 *>(residual_out + o) = h;
        float f[8];
        unpack_bf16_8(h, f);
        for (int i = 0; i < 8; i++) ss = fmaf(f[i], f[i], ss);
    }
    ss = cta_sum(ss, red);
    const float r = rsqrtf(ss / (float)k + eps);
    auto normed = [&](int u, float(&y)[16]) {
        const uint4 a = row_h[2 * u], b = row_h[2 * u + 1];
        unpack_16({{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}, y);
        float g[16];
        unpack_16(ld16(gain + 16 * u), g);
        for (int i = 0; i < 16; i++) y[i] = y[i] * r * g[i];
    };
    float s = 0.0f;
    float y[16];
    if (per_row) {
        float mx = 0.0f;
        for (int u = threadIdx.x; u < units; u += kThreads) {
            normed(u, y);
            mx = fmaxf(mx, amax_16(y));
        }
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        if ((threadIdx.x & 31) == 0) red_max[threadIdx.x >> 5] = mx;
        __syncthreads();
        for (int i = 0; i < kThreads / 32; i++) mx = fmaxf(mx, red_max[i]);
        s = __fdiv_rn(mx, 448.0f);
        if (threadIdx.x == 0) scale[row] = s;
    }
    for (int u0 = 0; u0 < units; u0 += kThreads) {
        const int u = u0 + threadIdx.x;
        for (int i = 0; i < 16; i++) y[i] = 0.0f;
        if (u < units) normed(u, y);
        if (!per_row) {
            s = __fdiv_rn(group_max(amax_16(y)), 448.0f);
            if (u < units && (u & 7) == 0) scale[row * (k >> 7) + (u >> 3)] = s;
        }
        if (u < units) *reinterpret_cast<uint4 *>(q + row * k + 16 * u) = codes_16(y, s);
    }
}

int grid_for_units(int64_t units) {
    const int64_t g = (units + kThreads - 1) / kThreads, most = (int64_t)sm_count() * 8;
    return (int)(g < most ? g : most);
}

}  // namespace

cudaError_t launch_quant_act_fp8_per128(const uint16_t *a, uint8_t *q, float *scale, int m, int k, cudaStream_t s) {
    const int64_t units = (int64_t)m * k / 16;
    k_quant_act_fp8_per128<<<grid_for_units(units), kThreads, 0, s>>>(a, q, scale, units);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_silu_mul_quant_fp8_per128(const uint16_t *gate_up, uint8_t *q, float *scale, int m, int k,
                                             cudaStream_t s) {
    const int64_t units = (int64_t)m * k / 16;
    k_silu_mul_quant_fp8_per128<<<grid_for_units(units), kThreads, 0, s>>>(gate_up, q, scale, k, units);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_rmsnorm_residual_quant_fp8(const uint16_t *x, const uint16_t *residual, const uint16_t *gain,
                                              float eps, uint16_t *residual_out, uint8_t *q, float *scale, int group,
                                              int m, int k, cudaStream_t s) {
    static DeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(k_rmsnorm_residual_quant_fp8, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    2 * kRmsMaxK);
    });
    if (e != cudaSuccess) return e;
    k_rmsnorm_residual_quant_fp8<<<m, kThreads, (size_t)k * 2, s>>>(x, residual, gain, eps, residual_out, q, scale,
                                                                    group == 0, k);
    note_launch();
    return cudaGetLastError();
}

}  // namespace bsq
