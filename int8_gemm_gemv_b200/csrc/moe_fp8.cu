// Mixture-of-experts feed-forward for at most 16 tokens, block-FP8 weights:
//   ids[t] = the topk largest router logits of token t (ties: lowest index)
//   p[t, j] = exp(l_j - max) / sum, over all experts or over the chosen ones
//   act[t, j] = silu(Wg[e_j] x_t) * (Wu[e_j] x_t)
//   out[t] = sum_j p[t, j] Wd[e_j] act[t, j]
//
// Plain form: one warp per token routes, one warp per intermediate element,
// one warp per output element.
#include <cfloat>
#include <cmath>

#include "bsq_common.cuh"

namespace bsq {

namespace {

struct Routing {
    int32_t id[kMoeMaxTokens * kMoeMaxTopk];
    float weight[kMoeMaxTokens * kMoeMaxTopk];
};

// Order-preserving key of a logit: NaN counts as -inf, -0 as +0.
__device__ __forceinline__ uint32_t logit_key(float l) {
    l = (l != l) ? -INFINITY : l + 0.0f;
    const uint32_t b = __float_as_uint(l);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// exp(l - max): 1 at the maximum itself (also where both are +inf), 0 where
// every logit is -inf.
__device__ __forceinline__ float route_exp(float l, float mx) {
    if (mx == -INFINITY) return 0.0f;
    return l == mx ? 1.0f : expf(l - mx);
}

__global__ void k_moe_route(MoeArgs a, Routing *R) {
    const int t = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (t >= a.tokens) return;
    constexpr int PER = kMoeMaxExperts / 32;
    uint32_t key[PER];
    for (int i = 0; i < PER; i++) {
        const int e = lane + 32 * i;
        key[i] = e < a.experts ? logit_key(a.logits[t * a.experts + e]) : 0u;
    }
    uint32_t taken = 0;
    float mx = 0.0f, sum = 0.0f, sum_all = 0.0f;
    for (int j = 0; j < a.topk; j++) {
        uint32_t best = 0;
        for (int i = 0; i < PER; i++)
            if (!((taken >> i) & 1)) best = max(best, key[i]);
        best = __reduce_max_sync(0xFFFFFFFFu, best);
        int e = 1 << 30;
        for (int i = PER - 1; i >= 0; i--)
            if (!((taken >> i) & 1) && key[i] == best && lane + 32 * i < a.experts) e = lane + 32 * i;
        e = __reduce_min_sync(0xFFFFFFFFu, e);
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        const float l = key_logit(best);
        if (j == 0) mx = l;
        const float p = route_exp(l, mx);
        sum += p;
        if (lane == 0) {
            R->id[t * a.topk + j] = e;
            R->weight[t * a.topk + j] = p;
        }
    }
    for (int i = 0; i < PER; i++)
        if (lane + 32 * i < a.experts) sum_all += route_exp(key_logit(key[i]), mx);
    for (int o = 16; o > 0; o >>= 1) sum_all += __shfl_xor_sync(0xFFFFFFFFu, sum_all, o);
    if (!a.renormalise) sum = sum_all;
    __syncwarp();
    for (int j = lane; j < a.topk; j += 32) {
        const float p = sum > 0.0f ? R->weight[t * a.topk + j] / sum : 0.0f;
        R->weight[t * a.topk + j] = p;
        if (a.topk_ids) a.topk_ids[t * a.topk + j] = R->id[t * a.topk + j];
        if (a.topk_weights) a.topk_weights[t * a.topk + j] = p;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__global__ void k_moe_gate_up(MoeArgs a, const Routing *R, float *act) {
    const int lane = threadIdx.x & 31, pair = blockIdx.y;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = pair / a.topk;
    const int64_t e = R->id[pair];
    const int hb = a.hidden >> 7;
    float v[2];
    for (int part = 0; part < 2; part++) {
        const int64_t row = (2 * e + part) * a.inter + i;
        float acc = 0.0f;
        for (int k = lane; k < a.hidden; k += 32)
            acc += bf16_bits_to_f32(a.x[(int64_t)t * a.hidden + k]) * e4m3_to_f32(a.w_gu[row * a.hidden + k]) *
                   a.s_gu[(row >> 7) * hb + (k >> 7)];
        v[part] = warp_sum(acc);
    }
    if (lane == 0) act[(int64_t)pair * a.inter + i] = v[0] / (1.0f + expf(-v[0])) * v[1];
}

__global__ void k_moe_down(MoeArgs a, const Routing *R, const float *act) {
    const int lane = threadIdx.x & 31, t = blockIdx.y;
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int ib = a.inter >> 7;
    float sum = 0.0f;
    for (int j = 0; j < a.topk; j++) {
        const int pair = t * a.topk + j;
        const float p = R->weight[pair];
        if (p == 0.0f) continue;
        const int64_t row = (int64_t)R->id[pair] * a.hidden + n;
        float acc = 0.0f;
        for (int k = lane; k < a.inter; k += 32)
            acc += act[(int64_t)pair * a.inter + k] * e4m3_to_f32(a.w_d[row * a.inter + k]) *
                   a.s_d[(row >> 7) * ib + (k >> 7)];
        sum += p * warp_sum(acc);
    }
    if (lane == 0) a.out[(int64_t)t * a.hidden + n] = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
}

}  // namespace

size_t fp8_moe_workspace_bytes(int tokens, int hidden, int inter, int topk) {
    (void)hidden;
    return ((sizeof(Routing) + 255) & ~size_t(255)) + (size_t)tokens * topk * inter * sizeof(float);
}

cudaError_t launch_fp8_moe_blockscaled(const MoeArgs &a, cudaStream_t s) {
    Routing *R = static_cast<Routing *>(a.workspace);
    float *act = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + ((sizeof(Routing) + 255) & ~size_t(255)));
    k_moe_route<<<1, 32 * a.tokens, 0, s>>>(a, R);
    k_moe_gate_up<<<dim3(a.inter / 8, a.tokens * a.topk), 256, 0, s>>>(a, R, act);
    k_moe_down<<<dim3(a.hidden / 8, a.tokens), 256, 0, s>>>(a, R, act);
    note_launch();
    note_launch();
    note_launch();
    return cudaGetLastError();
}

}  // namespace bsq
