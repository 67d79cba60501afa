// Block-scaled FP8 GEMM: activations with one FP32 scale per 1 x 128, weight
// with one per 128 x 128,
//   C[m, n] = sum_b a_scale[m, b] w_scale[n / 128, b] sum_{k in block b} e4m3(A[m, k]) e4m3(W[n, k])
//
// Plain form: 64 x 64 tiles on the FP32 lanes, each block of 128 summed apart
// and folded with its two scales.
#include "bsq_common.cuh"

namespace bsq {

namespace {

constexpr int BM = 64, BN = 64, BK = 32, kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    k_fp8_gemm_blockscaled(const uint8_t *__restrict__ A, const float *__restrict__ a_scale,
                           const uint8_t *__restrict__ W, const float *__restrict__ w_scale,
                           uint16_t *__restrict__ out, int M, int N, int K) {
    __shared__ float sa[BK][BM + 1], sw[BK][BN + 1];
    const int m0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int kbn = K >> 7;
    float acc[4][4] = {}, part[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += BK) {
        for (int i = threadIdx.x; i < BM * BK / 4; i += kThreads) {
            const int r = i / (BK / 4), c = 4 * (i % (BK / 4));
            const uint32_t va = m0 + r < M ? *reinterpret_cast<const uint32_t *>(A + (int64_t)(m0 + r) * K + k0 + c) : 0;
            const uint32_t vw = n0 + r < N ? *reinterpret_cast<const uint32_t *>(W + (int64_t)(n0 + r) * K + k0 + c) : 0;
            for (int j = 0; j < 4; j++) {
                sa[c + j][r] = e4m3_to_f32((uint8_t)(va >> (8 * j)));
                sw[c + j][r] = e4m3_to_f32((uint8_t)(vw >> (8 * j)));
            }
        }
        __syncthreads();
        for (int kk = 0; kk < BK; kk++)
            for (int i = 0; i < 4; i++)
                for (int j = 0; j < 4; j++) part[i][j] = fmaf(sa[kk][4 * ty + i], sw[kk][4 * tx + j], part[i][j]);
        __syncthreads();
        if (((k0 + BK) & 127) == 0) {
            const int b = k0 >> 7;
            const float ws = w_scale[(int64_t)(n0 >> 7) * kbn + b];
            for (int i = 0; i < 4; i++) {
                const int m = min(m0 + 4 * ty + i, M - 1);
                const float s = a_scale[(int64_t)m * kbn + b] * ws;
                for (int j = 0; j < 4; j++) {
                    acc[i][j] = fmaf(part[i][j], s, acc[i][j]);
                    part[i][j] = 0.0f;
                }
            }
        }
    }
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++) {
            const int m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
            if (m < M && n < N) out[(int64_t)m * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i][j]));
        }
}

}  // namespace

cudaError_t launch_fp8_gemm_blockscaled(const uint8_t *a, const float *a_scale, const uint8_t *w,
                                        const float *w_scale, uint16_t *out, int m, int n, int k, cudaStream_t s) {
    k_fp8_gemm_blockscaled<<<dim3((n + BN - 1) / BN, (m + BM - 1) / BM), kThreads, 0, s>>>(a, a_scale, w, w_scale, out,
                                                                                          m, n, k);
    note_launch();
    return cudaGetLastError();
}

}  // namespace bsq
