// Mixture-of-experts feed-forward for at most 16 tokens, block-FP8 weights:
//   ids[t] = the topk largest router logits of token t (ties: lowest index)
//   p[t, j] = exp(l_j - max) / sum, over all experts or over the chosen ones
//   act[t, j] = silu(Wg[e_j] x_t) * (Wu[e_j] x_t)
//   out[t] = sum_j p[t, j] Wd[e_j] act[t, j]
//
// The reached experts' weights, read once, are the whole cost, so both kernels
// are streaming reads built like the FP8 GEMV: one CTA per SM, a TMA producer
// warp that fills a ring with boxes of 16 weight rows x up to 1 KB of K, up to
// 32 KB to a slot, and eight consumer warps that split a box's K into its
// 128-wide scale blocks (E4M3 -> FP16 exactly, FP16 MMAs with FP32 sums, each
// block's sum times its scale).  The MMA's eight columns are tokens that chose
// the expert (more than eight: it is listed, and read, twice).
// Measured (back to back in a graph): 16 tokens, 57 of 64 experts of 5120 x
// 1408 reached: 230 us, 5.3 TB/s, of which the routing takes 6 and the
// activations' maxima 7; 1 token, 2048 x 768, 64 experts, 8 choices: 20.7 us,
// two kernels' latency around some 6 us of streaming.
//
//   k_moe_gate_up  every CTA routes all tokens by itself (some hundred
//                  instructions per token), then takes an equal share of the
//                  (expert, 16 intermediate rows) pairs: a box of gate rows
//                  and one of up rows give silu(g) * u on the spot.  act is
//                  kept as FP16 times a power of two per 16 values, 11
//                  significant bits: the down product's MMAs are FP16, and a
//                  second FP16 for the rest would double them for about a tenth
//                  of the output's own BF16 rounding.
//   k_moe_down     an output tile of 64 or 128 rows runs over all reached experts'
//                  K, so a token's experts add up in registers.  act enters
//                  the MMAs at one power of two per token and scale block,
//                  undone in the FP32 fold of that block, so a block's bits do
//                  not depend on how large the others are.  The (tile,
//                  expert, K) steps are cut into equal shares, one per CTA,
//                  also inside a tile: the 80 tiles of 5120 outputs alone
//                  would occupy 80 of 148 SMs.  CTAs that share a tile leave
//                  their FP32 sums in the workspace, and the last one to come
//                  adds them in share order, so the result does not depend on
//                  which was last.  No CTA waits for another.
//
// Both are launched with programmatic stream serialization.  The first lets
// the second start as its own CTAs run out; that one reads the logits and the
// weights, which the first does not write, and waits for it before act.
#include <cmath>

#include "gemv_frag.cuh"

#include <cuda_fp16.h>

namespace bsq {

namespace {

using namespace gv;

// Eight consumer warps, so that each has the registers to run a slot's boxes
// as independent chains of MMAs (sixteen warps, one scale block of one box
// each, were slower).
constexpr int kConsumers = 8;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int SB = 128;        // K of one scale block: two 64-byte chunks
constexpr int kMaxSlots = 16;
constexpr int kMaxActive = kMoeMaxTokens * kMoeMaxTopk;
constexpr int kRed = 8704;     // floats of the warps' partial sums; the routing keys before that
constexpr int kSums = 512;     // floats of a group's sums: tiles x 16 rows x 8 columns
// Down kernel: a warp sums kOwn rows of an output tile; the tile's rows follow
// from how many scale blocks of K the warps take side by side.
constexpr int kOwn = 64;
constexpr int tile_rows(int wide) { return kOwn * kConsumers / wide; }
constexpr int kMinTile = tile_rows(8), kMaxTile = tile_rows(4);
static_assert(kRed >= kMoeMaxTokens * kMoeMaxExperts && kRed >= kConsumers * kSums, "shared buffers");

static __device__ unsigned int g_timeouts;

constexpr uint32_t kNoColumn = 0xFFFFFFFFu;

struct alignas(16) Route {
    float weight[kMoeMaxTokens][kMoeMaxTopk];
    uint16_t id[kMoeMaxTokens][kMoeMaxTopk];
    uint32_t slot[kMoeMaxExperts];     // by expert: its tokens, then its place in the list
    // the reached experts, in order; one with more than eight tokens is listed
    // twice, with its first eight and with the others
    uint16_t expert[kMaxActive];
    uint16_t tokens[kMaxActive];       // a bit each
    uint32_t column[kMaxActive][8];    // its c-th token: (token << 16) | pair (token * topk + choice), or kNoColumn
    int warp_count[kMoeMaxExperts / 32];
    int active;
};

struct alignas(16) Bars {
    uint64_t full[kMaxSlots];
    uint64_t empty[kMaxSlots];
    uint32_t rowmax[kMoeMaxTokens];
    uint32_t abort;
    uint32_t last;  // this CTA finishes the tile
};

// Ring geometry: a slot holds boxes of 16 weight rows x `blocks` scale blocks
// of K (box_bytes each), as many as the kernel has per step or pair; `steps`
// along K, `slots` in the ring.
struct Ring {
    int blocks, steps, slots;
    __host__ __device__ int box_bytes() const { return blocks * 16 * SB; }
};

__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
}
// 32 bytes (32-byte aligned) through L2 where p holds, else zeros; no branch.
__device__ __forceinline__ void ld_32b_if(bool p, const void *src, uint32_t (&v)[8]) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %9, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "mov.b32 %4, 0;\n\tmov.b32 %5, 0;\n\tmov.b32 %6, 0;\n\tmov.b32 %7, 0;\n\t"
        "@p ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t}"
        : "=&r"(v[0]), "=&r"(v[1]), "=&r"(v[2]), "=&r"(v[3]), "=&r"(v[4]), "=&r"(v[5]), "=&r"(v[6]), "=&r"(v[7])
        : "l"(src), "r"((int)p)
        : "memory");
}

// ---------------------------------------------------------------- routing --

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

// Routes every token and lists the reached experts.  Up to kRankLimit tokens x
// experts^2 the choice is by counting, all threads at once; beyond that by
// rounds of a warp-wide maximum (whole routing, 64 experts, 8 choices: 1 token
// 2.9 us by counting, 4.4 by rounds; 16 tokens 8.0 and 6.6).
constexpr int kRankLimit = 1 << 15;
// `keys`: kMoeMaxTokens x kMoeMaxExperts words.  Called by all threads of the
// CTA.
__device__ __forceinline__ void route(const MoeArgs &a, Route *R, uint32_t *keys) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < kMoeMaxExperts; e += kThreads) R->slot[e] = 0;
    for (int i = threadIdx.x; i < kMaxActive * 8; i += kThreads) R->column[0][i] = kNoColumn;
    const int E = a.experts, quads = (E + 3) >> 2;
    for (int i = threadIdx.x; i < a.tokens * 4 * quads; i += kThreads) {
        const int t = i / (4 * quads), e = i - t * 4 * quads;
        keys[t * kMoeMaxExperts + e] = e < E ? logit_key(__ldg(a.logits + (int64_t)t * E + e)) : 0u;
    }
    __syncthreads();
    if (a.tokens * E * E <= kRankLimit) {
        // every (token, expert) counts the experts before its own
        for (int i = threadIdx.x; i < a.tokens * E; i += kThreads) {
            const int t = i / E, e = i - t * E;
            const uint4 *k4 = reinterpret_cast<const uint4 *>(keys + t * kMoeMaxExperts);
            const uint32_t own = keys[t * kMoeMaxExperts + e];
            int rank = 0;
            for (int q = 0; q < quads; q++) {
                const uint4 k = k4[q];
                // among equals a lower index comes first (no key is the largest word)
                rank += (k.x >= own + (4 * q >= e)) + (k.y >= own + (4 * q + 1 >= e)) +
                        (k.z >= own + (4 * q + 2 >= e)) + (k.w >= own + (4 * q + 3 >= e));
            }
            if (rank < a.topk) R->id[t][rank] = (uint16_t)e;
        }
    } else {
        // a warp per token takes the largest again and again
        for (int t = warp; t < a.tokens; t += kThreads / 32) {
            uint32_t *key = keys + t * kMoeMaxExperts;
            uint32_t taken = 0;  // bit i: expert lane + 32 i
            for (int j = 0; j < a.topk; j++) {
                uint32_t best = 0;
                int at = lane;
                for (int i = 0, e = lane; e < E; i++, e += 32)
                    if (key[e] > best && !((taken >> i) & 1)) {
                        best = key[e];
                        at = e;
                    }
                const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
                const int e = __reduce_min_sync(0xFFFFFFFFu, best == top ? at : kMoeMaxExperts);
                if ((e & 31) == lane) {
                    taken |= 1u << (e >> 5);
                    R->id[t][j] = (uint16_t)e;
                }
            }
        }
    }
    __syncthreads();
    // the weights, a warp per token: lane j has the j-th choice
    for (int t = warp; t < a.tokens; t += kThreads / 32) {
        const uint32_t *key = keys + t * kMoeMaxExperts;
        const float mx = key_logit(key[R->id[t][0]]);
        const int id = lane < a.topk ? R->id[t][lane] : 0;
        const float mine = lane < a.topk ? route_exp(key_logit(key[id]), mx) : 0.0f;
        float sum = a.renormalise ? mine : 0.0f;
        if (!a.renormalise)
            for (int e = lane; e < E; e += 32) sum += route_exp(key_logit(key[e]), mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane < a.topk) {
            const float w = sum > 0.0f ? __fdiv_rn(mine, sum) : 0.0f;
            R->weight[t][lane] = w;
            // an expert that adds nothing is not read
            if (w > 0.0f) atomicOr(&R->slot[id], 1u << t);
        }
    }
    __syncthreads();
    constexpr int HALVES = kMoeMaxExperts / (32 * kConsumers);
    uint32_t mask[HALVES], one[HALVES], two[HALVES];
    if (warp < kConsumers) {
#pragma unroll
        for (int i = 0; i < HALVES; i++) {
            mask[i] = R->slot[i * 32 * kConsumers + threadIdx.x];
            one[i] = __ballot_sync(0xFFFFFFFFu, mask[i] != 0);
            two[i] = __ballot_sync(0xFFFFFFFFu, __popc(mask[i]) > 8);
            if (lane == 0) R->warp_count[i * kConsumers + warp] = __popc(one[i]) + __popc(two[i]);
        }
    }
    __syncthreads();
    if (warp < kConsumers) {
#pragma unroll
        for (int i = 0; i < HALVES; i++) {
            const int w = i * kConsumers + warp, e = i * 32 * kConsumers + (int)threadIdx.x;
            const uint32_t below = (1u << lane) - 1u;
            const int before = lane < w ? R->warp_count[lane] : 0;  // (at most 16 warps' counts)
            const int at = (int)__reduce_add_sync(0xFFFFFFFFu, before) + __popc(one[i] & below) + __popc(two[i] & below);
            uint32_t first = mask[i];
            while (__popc(first) > 8) first &= ~(0x80000000u >> __clz(first));
            if (mask[i]) {
                R->expert[at] = (uint16_t)e;
                R->tokens[at] = (uint16_t)first;
                if (first != mask[i]) {
                    R->expert[at + 1] = (uint16_t)e;
                    R->tokens[at + 1] = (uint16_t)(mask[i] & ~first);
                }
                R->slot[e] = at;
            }
            if (e == kMoeMaxExperts - 1) R->active = at + (mask[i] != 0) + (first != mask[i]);
        }
    }
    __syncthreads();
    const int t = threadIdx.x >> 4, j = threadIdx.x & 15;
    if (t < a.tokens && j < a.topk && R->weight[t][j] > 0.0f) {
        int at = R->slot[R->id[t][j]];
        at += !((R->tokens[at] >> t) & 1);
        R->column[at][__popc(R->tokens[at] & ((1u << t) - 1u))] = (uint32_t)(t << 16 | (t * a.topk + j));
    }
    __syncthreads();
}
static_assert(kMoeMaxExperts % (32 * kConsumers) == 0 && kMoeMaxExperts / 32 <= 32 && kMoeMaxTopk == 16 &&
                  32 * kConsumers >= kMoeMaxTokens * kMoeMaxTopk,
              "routing by one CTA");

// ------------------------------------------------------------------- ring --

// Consumer side of the ring: every consumer warp takes its part of every slot.
struct Taker {
    int s = 0;
    uint32_t ph = 0;
    uint32_t empty0;  // the give-back barriers, by cluster address (the plain form of the arrival
                      // waits some 160 cycles for the warp's other memory operations)
    __device__ __forceinline__ Taker(Bars *S) : empty0(mapa_shared(smem_u32(&S->empty[0]), 0)) {}
    // Waits for the next slot; returns its address in shared memory.
    __device__ __forceinline__ uint32_t take(Bars *S, uint32_t ring, int slot_bytes) {
        mbar_wait_or_abort(&S->full[s], ph, &S->abort, &g_timeouts);
        __syncwarp();
        return ring + (uint32_t)s * slot_bytes;
    }
    // Gives it back.
    __device__ __forceinline__ void give_back(int slots, int lane) {
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(empty0 + 8 * s);
        if (++s == slots) {
            s = 0;
            ph ^= 1;
        }
    }
};

// d (+)= 16 rows x 64 of K times eight tokens; a_w, b_w the E4M3 bytes of rows
// g and g + 8, x the FP16 activations.
__device__ __forceinline__ void chunk_mma_8(float (&d)[4], const uint4 &wa, const uint4 &wb, const uint32_t (&x)[8]) {
    const uint32_t a_w[4] = {wa.x, wa.y, wa.z, wa.w};
    const uint32_t b_w[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint32_t a[4];
        e4m3x4_to_f16x2(a_w[j], a[0], a[2]);
        e4m3x4_to_f16x2(b_w[j], a[1], a[3]);
        mma_f16_16816(d, a, x[2 * j], x[2 * j + 1]);
    }
}

// Two boxes of the next slot: acc[box] += scale[box] * (this warp's scale
// block, two chunks, of the box) x the activation fragments x[chunk], as four
// independent chains of MMAs.  `offset` is that block's place in the slot.
// With COLS the sums of the lane's two columns (tokens) are also multiplied by
// col, powers of two.
template <bool COLS>
__device__ __forceinline__ void slot_mma(Taker &take, Bars *S, uint32_t ring, int slot_bytes, int slots, int box_bytes,
                                         int offset, bool active, int lane, const uint32_t (&x)[2][8],
                                         const float (&scale)[2], const float (&col)[2], float (&acc0)[4],
                                         float (&acc1)[4]) {
    const uint32_t at = take.take(S, ring, slot_bytes) + offset;
    const int g = lane >> 2, t = lane & 3;
    uint4 w[2][2][2];  // [box][chunk][row g, g + 8]
    if (active) {
#pragma unroll
        for (int v = 0; v < 2; v++)
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const uint32_t chunk = at + v * box_bytes + c * 16 * CH;
                w[v][c][0] = lds_v4(chunk + w_off(g, t));
                w[v][c][1] = lds_v4(chunk + w_off(g + 8, t));
            }
    }
    take.give_back(slots, lane);
    if (!active) return;
    float d[2][2][4] = {};  // [box][chunk]
#pragma unroll
    for (int c = 0; c < 2; c++)
#pragma unroll
        for (int v = 0; v < 2; v++) chunk_mma_8(d[v][c], w[v][c][0], w[v][c][1], x[c]);
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float d0 = d[0][0][k] + d[0][1][k], d1 = d[1][0][k] + d[1][1][k];
        acc0[k] = COLS ? __fmaf_rn(d0 * scale[0], col[k & 1], acc0[k]) : __fmaf_rn(d0, scale[0], acc0[k]);
        acc1[k] = COLS ? __fmaf_rn(d1 * scale[1], col[k & 1], acc1[k]) : __fmaf_rn(d1, scale[1], acc1[k]);
    }
}

// Producer side, one thread.
struct Giver {
    int s = 0;
    uint32_t ph = 1;
    uint32_t it = 0;
    // BOXES boxes, box b at weight row row0 + b * apart
    template <int BOXES>
    __device__ __forceinline__ bool give(Bars *S, uint8_t *ring, int box_bytes, int slots, const CUtensorMap *tm,
                                         int row0, int apart, int chunk) {
        const int slot_bytes = BOXES * box_bytes;
        if (!mbar_wait(&S->empty[s], ph, &g_timeouts) || *(volatile uint32_t *)&S->abort) return false;
        mbar_arrive_expect_tx(&S->full[s], slot_bytes);
#pragma unroll
        for (int b = 0; b < BOXES; b++)
            tma_load_3d(ring + (size_t)s * slot_bytes + b * box_bytes, tm, &S->full[s], 0, row0 + b * apart, chunk);
        if (++s == slots) {
            s = 0;
            ph ^= 1;
        }
        it++;
        return true;
    }
    // wait out the copies still in flight so that none lands after exit
    __device__ __forceinline__ void give_up(Bars *S, int slots) {
        S->abort = 1;
        for (uint32_t i = it > (uint32_t)slots ? it - slots : 0; i < it; i++)
            mbar_wait(&S->full[i % slots], (i / slots) & 1, &g_timeouts);
    }
};

__device__ __forceinline__ void init_bars(Bars *S, int slots) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < slots; s++) {
            mbar_init(&S->full[s], 1);
            mbar_init(&S->empty[s], kConsumers);
        }
        for (int m = 0; m < kMoeMaxTokens; m++) S->rowmax[m] = 0;
        S->abort = 0;
        fence_mbar_init();
    }
}

// The warps' partial sums of `n` outputs (an output's index is (tile * 4 + r)
// * 32 + lane, as the MMA leaves it), added in warp order.
template <int TG>
__device__ __forceinline__ void reduce_warps(const float (&acc)[TG][4], float *red, float *sums, int warp, int lane,
                                             int n) {
    consumers_sync();  // the previous group's sums have been read
#pragma unroll
    for (int u = 0; u < TG; u++)
#pragma unroll
        for (int r = 0; r < 4; r++) red[((warp * TG + u) * 4 + r) * 32 + lane] = acc[u][r];
    consumers_sync();
    for (int v = threadIdx.x; v < n; v += 32 * kConsumers) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kConsumers; w++) sum += red[w * TG * 128 + v];
        sums[v] = sum;
    }
    consumers_sync();
}

// Share b of g of `all` steps: equal to within one, none empty while b < all.
struct Share {
    int begin, end;
};
__device__ __forceinline__ Share share_of(int all, int b, int g) {
    const int per = all / g, more = all - per * g;
    const int begin = b * per + min(b, more);
    return {begin, begin + per + (b < more)};
}
// The share that step u lies in.
__device__ __forceinline__ int share_at(int all, int u, int g) {
    const int per = all / g, more = all - per * g;
    return u < more * (per + 1) ? u / (per + 1) : more + (u - more * (per + 1)) / per;
}

// The token of a column, -1 without one.
__device__ __forceinline__ int token_of(uint32_t column) { return column == kNoColumn ? -1 : (int)(column >> 16); }

// Workspace layout.
struct Ws {
    __half *act;       // [tokens * topk, inter], times a power of two per 16
    uint8_t *act_exp;  // [tokens * topk, inter / 16]: exponent field of the 16 values' largest
    int *count;        // [output tiles] shares of a tile that have come
    float *part;       // [CTAs][2][tile rows x tokens] FP32 sums of shared tiles
};

// The power of two for 16 (or a scale block of) act values whose largest has
// this FP32 exponent field: brings it to [2^14, 2^15).
__device__ __forceinline__ int exp_shift(int e) { return min(14 - (e - 127), 127); }

// ---------------------------------------------------------------- gate, up --
//   tmW  [experts * 2 inter] rows x hidden, as (64 B, rows, hidden / 64), box
//        (64, 16, 2 ring.blocks)
__global__ void __launch_bounds__(kThreads, 1)
    k_moe_gate_up(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ MoeArgs a, Ring ring, Ws ws) {
    constexpr int PG = 2, TG = 2 * PG;  // (gate, up) tile pairs sharing one pass over x; a slot holds one pair
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int box_bytes = ring.box_bytes(), slot_bytes = 2 * box_bytes;
    float *red = reinterpret_cast<float *>(base + (size_t)ring.slots * slot_bytes);
    float *sums = red + kRed;
    Route *R = reinterpret_cast<Route *>(sums + kSums);
    Bars *S = reinterpret_cast<Bars *>(R + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = a.hidden, I = a.inter, T = a.tokens;
    init_bars(S, ring.slots);
    __syncthreads();
    dependency_wait();
    // the down kernel may start where CTAs run out; it reads nothing that this
    // one writes before it has completed, and everything before this one has
    launch_dependents();

    route(a, R, reinterpret_cast<uint32_t *>(red));

    // this CTA's share of the (expert, 16 rows) units
    const int per_expert = I >> 4;
    const Share mine = share_of(R->active * per_expert, blockIdx.x, gridDim.x);
    const int u_begin = mine.begin, u_end = mine.end;

    if (warp == kConsumers) {
        if (elect_one()) {
            prefetch_tensormap(&tmW);
            Giver give;
            bool ok = true;
            for (int u = u_begin; u < u_end && ok;) {
                const int ai = u / per_expert, r = u - ai * per_expert;
                const int n = min(min(PG, per_expert - r), u_end - u);
                const int row = (int)R->expert[ai] * 2 * I + 16 * r;
                for (int q = 0; q < ring.steps && ok; q++)
                    for (int p = 0; p < n && ok; p++)
                        ok = give.give<2>(S, base, box_bytes, ring.slots, &tmW, row + 16 * p, I, q * ring.blocks * 2);
                u += n;
            }
            if (!ok) give.give_up(S, ring.slots);
        }
        return;
    }

    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring_at = smem_u32(base);
    const int hb = H >> 7;
    // this lane's activations of step q for token m, [chunk][16-byte half]
    // (without a token, and past the end of K, some other valid ones: they are
    // multiplied by zero, or not used; no branch)
    auto load_x = [&](int m, int q, uint4(&x)[2][2]) {
        const int kb = min(q * ring.blocks + warp, hb - 1);
        const uint16_t *p = a.x + (int64_t)max(m, 0) * H + kb * SB + 16 * t;
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
            for (int h = 0; h < 2; h++) x[c][h] = ldg_nc_v4(p + CH * c + 8 * h);
    };
    // the scales of this warp's block of step q for the group that starts at row
    // unit r of the listed expert ai (a unit's 16 rows lie in one scale block;
    // a group's may not)
    auto load_scales = [&](int ai, int r, int q, float(&sc)[TG]) {
        const int kb = min(q * ring.blocks + warp, hb - 1);
#pragma unroll
        for (int p = 0; p < PG; p++) {
            const int64_t row = (int64_t)R->expert[ai] * 2 * I + 16 * min(r + p, per_expert - 1);
            const float *s = a.s_gu + (row >> 7) * hb + kb;
            sc[2 * p] = __ldg(s);
            sc[2 * p + 1] = __ldg(s + (int64_t)(I >> 7) * hb);
        }
    };
    Taker take(S);
    uint4 nx[2][2];
    float nsc[TG];
    int m_next = -1, ai = u_begin / per_expert, r = u_begin - ai * per_expert;
    if (u_begin < u_end) {
        m_next = token_of(R->column[ai][g]);
        load_x(m_next, 0, nx);
        load_scales(ai, r, 0, nsc);
    }
    // each token's largest magnitude, found by all consumer warps together (the
    // first weight copies are on their way)
    {
        constexpr int B = 10;  // 16-byte loads of a lane in flight
        const int parts = T < kConsumers ? kConsumers / T : 1;
        const int units = H >> 3, per = (units + parts - 1) / parts;
        for (int task = warp; task < T * parts; task += kConsumers) {
            const int m = task % T, p = task / T;
            const int u0 = p * per, u1 = min(units, u0 + per);
            const uint4 *xr = reinterpret_cast<const uint4 *>(a.x + (int64_t)m * H);
            uint32_t mx = 0;
            for (int u = u0 + lane; u < u1; u += 32 * B) {
                uint4 v[B];
#pragma unroll
                for (int j = 0; j < B; j++) v[j] = u + 32 * j < u1 ? ldg_nc_v4(xr + u + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < B; j++)
                    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[j].x & 0x7FFF7FFFu, v[j].y & 0x7FFF7FFFu),
                                               __vmaxu2(v[j].z & 0x7FFF7FFFu, v[j].w & 0x7FFF7FFFu)));
            }
            mx = max(mx & 0xFFFFu, mx >> 16);
            mx = __reduce_max_sync(0xFFFFFFFFu, mx);
            if (lane == 0) atomicMax(&S->rowmax[m], mx);
        }
    }
    if (blockIdx.x == 0) {
        const int t = threadIdx.x >> 4, j = threadIdx.x & 15;
        if (t < T && j < a.topk) {
            if (a.topk_ids) a.topk_ids[t * a.topk + j] = R->id[t][j];
            if (a.topk_weights) a.topk_weights[t * a.topk + j] = R->weight[t][j];
        }
        for (int i = threadIdx.x; i < H / kMinTile; i += 32 * kConsumers) ws.count[i] = 0;
    }

    consumers_sync();
    for (int u = u_begin; u < u_end;) {
        const int n = min(min(PG, per_expert - r), u_end - u);
        const int ai1 = r + n == per_expert ? ai + 1 : ai, r1 = r + n == per_expert ? 0 : r + n;  // the next group
        const int my = m_next;  // this lane's token
        const float xs = my < 0 ? 0.0f : pow2i(row_shift(S->rowmax[my]));
        float acc[TG][4] = {};
        for (int q = 0; q < ring.steps; q++) {
            uint32_t f[2][8];
#pragma unroll
            for (int c = 0; c < 2; c++) x_to_f16<1>(nx[c], xs, f[c]);
            float sc[PG][2];
#pragma unroll
            for (int v = 0; v < TG; v++) sc[v >> 1][v & 1] = nsc[v];
            // the next step's, one step ahead
            if (q + 1 < ring.steps) {
                load_x(my, q + 1, nx);
                load_scales(ai, r, q + 1, nsc);
            } else if (u + n < u_end) {
                m_next = token_of(R->column[ai1][g]);
                load_x(m_next, 0, nx);
                load_scales(ai1, r1, 0, nsc);
            }
            const bool active = warp < ring.blocks && q * ring.blocks + warp < hb;
#pragma unroll
            for (int p = 0; p < PG; p++) {
                if (p >= n) break;
                slot_mma<false>(take, S, ring_at, slot_bytes, ring.slots, box_bytes, warp * 2 * 16 * CH, active, lane, f,
                                sc[p], {1.0f, 1.0f}, acc[2 * p], acc[2 * p + 1]);
            }
        }
        reduce_warps<TG>(acc, red, sums, warp, lane, 2 * n * 128);
        // silu(gate) * up: a warp takes one (pair, column parity), a lane rows
        // g and g + 8 of column 2 t + parity
        if (warp < 2 * n) {
            const int p = warp >> 1, c = warp & 1;
            const uint32_t col = R->column[ai][2 * t + c];
            const int m = token_of(col);
            const float unscale = pow2i(-row_shift(S->rowmax[max(m, 0)]));
            const float *gs = sums + (2 * p * 4 + c) * 32 + lane, *us = gs + 128;
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const float gate = gs[64 * k] * unscale, up = us[64 * k] * unscale;
                v[k] = __fdiv_rn(gate, 1.0f + expf(-gate)) * up;
            }
            float mx = fmaxf(fabsf(v[0]), fabsf(v[1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
            if (m >= 0) {
                const int64_t pair = col & 0xFFFFu;
                const int ex = (int)(__float_as_uint(mx) >> 23);
                const float s = pow2i(exp_shift(ex));
                __half *dst = ws.act + pair * I + 16 * (r + p) + g;
                dst[0] = __float2half_rn(v[0] * s);
                dst[8] = __float2half_rn(v[1] * s);
                if (g == 0) ws.act_exp[pair * per_expert + r + p] = (uint8_t)ex;
            }
        }
        u += n;
        ai = ai1;
        r = r1;
    }
}

// -------------------------------------------------------------------- down --
//   tmW  [experts * hidden] rows x inter, as (64 B, rows, inter / 64), box
//        (64, 16, 2 ring.blocks)
// The eight warps take WIDE scale blocks of K side by side, 8 / WIDE row halves
// each: WIDE 8 and tiles of 64 rows, or WIDE 4 and tiles of 128 (one scale
// block), where that leaves fewer warps without a block.
template <int WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    k_moe_down(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ MoeArgs a, Ring ring, Ws ws) {
    constexpr int ROW = kMoeMaxTokens + 1;  // floats of an output row's sums (odd: rows fall into different banks)
    constexpr int TILE = tile_rows(WIDE), PART = TILE * kMoeMaxTokens;
    constexpr int WARP_SUMS = kOwn * ROW, PER = PART / (32 * kConsumers);
    constexpr int BOXES = 16 / WIDE;  // of a slot; two slots per step
    static_assert(WIDE == 4 || WIDE == 8, "a tile lies in one scale block and a slot holds 32 KB");
    static_assert(kConsumers * WARP_SUMS <= kRed && PER * 32 * kConsumers == PART, "sums of a tile");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int box_bytes = ring.box_bytes(), slot_bytes = BOXES * box_bytes;
    float *red = reinterpret_cast<float *>(base + (size_t)ring.slots * slot_bytes);
    Route *R = reinterpret_cast<Route *>(red + kRed);
    Bars *S = reinterpret_cast<Bars *>(R + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = a.hidden, I = a.inter, T = a.tokens;
    init_bars(S, ring.slots);
    __syncthreads();
    route(a, R, reinterpret_cast<uint32_t *>(red));  // the logits were there before the previous kernel started

    // this CTA's share of the (tile, expert, K step) sequence; no share
    // is empty, which the count of a shared tile's shares relies on
    const int steps = R->active * ring.steps, all = steps * (H / TILE);  // of one tile, of all
    const int shares = max(min((int)gridDim.x, all), 1);
    const Share mine = (int)blockIdx.x < shares ? share_of(all, blockIdx.x, shares) : Share{all, all};
    const int u_begin = mine.begin, u_end = mine.end;

    if (warp == kConsumers) {
        if (elect_one()) {
            prefetch_tensormap(&tmW);
            Giver give;
            bool ok = true;
            int tile = steps ? u_begin / steps : 0;
            const int st = u_begin - tile * steps;
            int ai = st / ring.steps, q = st - ai * ring.steps;
            for (int u = u_begin; u < u_end && ok; u++) {
                const int row = (int)R->expert[ai] * H + TILE * tile;
                for (int h = 0; h < 2 && ok; h++)
                    ok = give.give<BOXES>(S, base, box_bytes, ring.slots, &tmW, row + 16 * BOXES * h, 16, q * ring.blocks * 2);
                if (++q == ring.steps) {
                    q = 0;
                    if (++ai == R->active) {
                        ai = 0;
                        tile++;
                    }
                }
            }
            if (!ok) give.give_up(S, ring.slots);
            dependency_wait();  // no CTA ends before the previous kernel has
            launch_dependents();
        }
        return;
    }

    dependency_wait();
    launch_dependents();
    if (all == 0) {  // no token has an expert
        for (int64_t i = (int64_t)blockIdx.x * 32 * kConsumers + threadIdx.x; i < (int64_t)T * H;
             i += (int64_t)gridDim.x * 32 * kConsumers)
            a.out[i] = 0;
        return;
    }
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring_at = smem_u32(base);
    const int hb = H >> 7, ib = I >> 7;
    // A warp takes scale block wb of a step, and rows 32 wr .. + 31 of each slot.
    const int wb = warp % WIDE, wr = warp / WIDE;
    const int offset = 2 * wr * box_bytes + wb * 2 * 16 * CH;
    // A step's input of this lane: its token's act, 2 x 16 FP16 values, the
    // exponents of the block's eight groups, and the block's weight scale.
    struct Input {
        uint32_t v[2][8];
        uint2 ex;
        float sc;
    };
    // a place in the sequence
    struct Pos {
        int tile, ai, q;
    };
    auto advance = [&](Pos &p) {
        if (++p.q == ring.steps) {
            p.q = 0;
            if (++p.ai == R->active) {
                p.ai = 0;
                p.tile++;
            }
        }
    };
    auto load = [&](const Pos &p, Input &o) {
        // (past the end of K some other valid values, not used; no branch)
        const int kb = min(p.q * ring.blocks + wb, ib - 1);
        const uint32_t col = R->column[p.ai][g];
        const int pair = col == kNoColumn ? 0 : (int)(col & 0xFFFFu);
        const __half *src = ws.act + (int64_t)pair * I + kb * SB + 16 * t;
#pragma unroll
        for (int c = 0; c < 2; c++) ld_32b_if(col != kNoColumn, src + CH * c, o.v[c]);
        o.ex = __ldcg(reinterpret_cast<const uint2 *>(ws.act_exp + (int64_t)pair * (I >> 4)) + kb);
        // (the tile's rows lie in one scale block)
        o.sc = __ldg(a.s_d + ((int64_t)R->expert[p.ai] * hb + p.tile * TILE / 128) * ib + kb);
    };
    // Sixteen act values brought to their scale block's power of two, which the
    // fold undoes: the factor 2^-d, exact down to FP16's subnormals (2^-24,
    // where the block's largest is 2^14 or more; a whole block may be as far
    // from another as FP32 goes).  From 2^-25 on FP16 has no such factor, so it
    // is taken as two.
    auto to_block = [&](const uint32_t(&v)[8], uint32_t exps, int block_shift, uint32_t(&o)[8]) {
        const int d = min(max(exp_shift((int)((exps >> (8 * t)) & 0xFFu)) - block_shift, 0), 40), d0 = min(d, 24);
        const __half2 f0 = __float2half2_rn(pow2i(-d0)), f1 = __float2half2_rn(pow2i(d0 - d));
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const __half2 h = __hmul2(__hmul2(*reinterpret_cast<const __half2 *>(&v[j]), f1), f0);
            o[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
    };

    // This warp's sums of its rows of the tile, [row][token]; an expert's products gather
    // in registers over its K steps and are added here, weighted, per token.
    float *own = red + warp * WARP_SUMS;
    auto clear = [&] {
        for (int i = lane; i < WARP_SUMS; i += 32) own[i] = 0.0f;
        __syncwarp();
    };
    Taker take(S);
    Pos cur, ahead;
    cur.tile = u_begin / steps;
    const int st = u_begin - cur.tile * steps;
    cur.ai = st / ring.steps;
    cur.q = st - cur.ai * ring.steps;
    int first = st;  // the tile's first step here
    float acc[kOwn / 16][4] = {};
    clear();
    Input in;  // one step ahead
    ahead = cur;
    if (u_begin < u_end) load(ahead, in);
    advance(ahead);
    // The tile's sums over the warps, in warp order.  A tile shared with other
    // CTAs: leave them in the workspace, count, and add everybody's if last.
    auto finish_tile = [&](int tile, bool shared) {
        consumers_sync();
        float sum[PER];
#pragma unroll
        for (int h = 0; h < PER; h++) {
            const int v = threadIdx.x + h * 32 * kConsumers, r = v >> 4;
            // slot r / SLOT's row 32 wr + i is row 32 (r / SLOT) + i of the warps with that wr
            constexpr int SLOT = 16 * BOXES;
            const float *from =
                red + r % SLOT / 32 * WIDE * WARP_SUMS + (r / SLOT * 32 + (r & 31)) * ROW + (v & 15);
            sum[h] = 0.0f;
#pragma unroll
            for (int w = 0; w < WIDE; w++) sum[h] += from[w * WARP_SUMS];
        }
        if (shared) {
            const int b0 = share_at(all, tile * steps, shares), b1 = share_at(all, (tile + 1) * steps - 1, shares);
            float *part = ws.part + ((int64_t)blockIdx.x * 2 + (first == 0)) * PART;
#pragma unroll
            for (int h = 0; h < PER; h++) __stcg(part + threadIdx.x + h * 32 * kConsumers, sum[h]);
            __threadfence();
            consumers_sync();
            if (threadIdx.x == 0) S->last = atomicAdd(ws.count + tile, 1) == b1 - b0;
            consumers_sync();
            if (S->last) {
                __threadfence();
#pragma unroll
                for (int h = 0; h < PER; h++) sum[h] = 0.0f;
                // (of its two slots the share with the tile's first step took
                // 1, the others 0; four shares' loads are in flight together)
                constexpr int JB = 4;
                for (int b = b0; b <= b1; b += JB) {
                    float v[JB][PER];
#pragma unroll
                    for (int j = 0; j < JB; j++) {
                        const float *p = ws.part + ((int64_t)min(b + j, b1) * 2 + (b + j == b0)) * PART + threadIdx.x;
#pragma unroll
                        for (int h = 0; h < PER; h++) v[j][h] = __ldcg(p + h * 32 * kConsumers);
                    }
#pragma unroll
                    for (int j = 0; j < JB; j++)
#pragma unroll
                        for (int h = 0; h < PER; h++)
                            if (b + j <= b1) sum[h] += v[j][h];
                }
            }
        }
        if (!shared || S->last) {
#pragma unroll
            for (int h = 0; h < PER; h++) {
                const int v = threadIdx.x + h * 32 * kConsumers, m = v & 15;
                if (m < T) a.out[(int64_t)m * H + TILE * tile + (v >> 4)] = __bfloat16_as_ushort(__float2bfloat16_rn(sum[h]));
            }
        }
        consumers_sync();  // everybody's sums, and the flag, have been read
        clear();
    };
    auto step = [&](int u) {
        // the block's largest exponent, its power of two, and how that is undone
        // for this lane's columns 2t and 2t + 1 (without a token: zeros times
        // some power of two)
        uint32_t mx = __vmaxu4(in.ex.x, in.ex.y);
        mx = __vmaxu4(mx, mx >> 16);
        const int shift = exp_shift((int)max(mx & 0xFFu, (mx >> 8) & 0xFFu));
        const float undo = pow2i(-shift);
        const float cols[2] = {__shfl_sync(0xFFFFFFFFu, undo, 8 * t), __shfl_sync(0xFFFFFFFFu, undo, 8 * t + 4)};
        uint32_t f[2][8];
#pragma unroll
        for (int c = 0; c < 2; c++) to_block(in.v[c], c ? in.ex.y : in.ex.x, shift, f[c]);
        const float sc[2] = {in.sc, in.sc};
        if (u + 1 < u_end) load(ahead, in);
        advance(ahead);
        const bool active = wb < ring.blocks && cur.q * ring.blocks + wb < ib;
#pragma unroll
        for (int h = 0; h < 2; h++)
            slot_mma<true>(take, S, ring_at, slot_bytes, ring.slots, box_bytes, offset, active, lane, f, sc, cols,
                           acc[2 * h], acc[2 * h + 1]);
        const int tile = cur.tile, ai = cur.ai;
        advance(cur);
        if (cur.ai == ai && cur.tile == tile && u + 1 < u_end) return;
        // the expert's last step here: columns 2t and 2t + 1, rows g and g + 8
#pragma unroll
        for (int c = 0; c < 2; c++) {
            const uint32_t to = R->column[ai][2 * t + c];
            if (to != kNoColumn) {
                const int m = (int)(to >> 16);
                const float cf = R->weight[m][(int)(to & 0xFFFFu) - m * a.topk];
                float *o = own + g * ROW + m;
#pragma unroll
                for (int r = 0; r < kOwn / 8; r++) o[8 * r * ROW] = __fmaf_rn(acc[r >> 1][2 * (r & 1) + c], cf, o[8 * r * ROW]);
            }
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < kOwn / 16; r++) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.0f;
        if (cur.tile == tile && u + 1 < u_end) return;
        finish_tile(tile, first != 0 || cur.tile == tile);
        first = 0;
    };
    for (int u = u_begin; u < u_end; u++) step(u);
}

// -------------------------------------------------------------------- host --

constexpr size_t kSmemMax = 232448;
constexpr size_t kFixed = 1024 + (kRed + kSums) * 4 + sizeof(Route) + sizeof(Bars);  // all but the ring

// Boxes of equal size, at most `wide` scale blocks of K, and as many slots (of
// `boxes` boxes) as fit.
Ring ring_for(int k, int wide, int boxes) {
    Ring r;
    const int blocks = k / SB;
    r.steps = (blocks + wide - 1) / wide;
    r.blocks = (blocks + r.steps - 1) / r.steps;
    const int room = (int)((kSmemMax - kFixed) / ((size_t)boxes * r.box_bytes()));
    r.slots = room < kMaxSlots ? room : kMaxSlots;
    return r;
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

size_t ws_layout(void *p, int tokens, int hidden, int inter, int topk, Ws *ws) {
    const size_t pairs = (size_t)tokens * topk;
    const size_t act = align256(pairs * inter * sizeof(__half)), ex = align256(pairs * (inter / 16)),
                 count = align256((size_t)hidden / kMinTile * sizeof(int)),
                 part = (size_t)sm_count() * 2 * kMaxTile * kMoeMaxTokens * sizeof(float);
    if (ws) {
        uint8_t *b = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 255) & ~uintptr_t(255));
        ws->act = reinterpret_cast<__half *>(b);
        ws->act_exp = b + act;
        ws->count = reinterpret_cast<int *>(b + act + ex);
        ws->part = reinterpret_cast<float *>(b + act + ex + count);
    }
    return 255 + act + ex + count + part;
}

template <class F>
cudaError_t launch_one(F kernel, const uint8_t *w, int64_t rows, int k, int wide, int boxes, const MoeArgs &a,
                       const Ws &ws, cudaStream_t s) {
    const Ring ring = ring_for(k, wide, boxes);
    alignas(64) CUtensorMap tm;
    const uint64_t d[3] = {CH, (uint64_t)rows, (uint64_t)k / CH}, st[2] = {(uint64_t)k, CH};
    const uint32_t box[3] = {CH, 16, (uint32_t)(2 * ring.blocks)};
    if (!make_tmap(&tm, w, 1, 3, d, st, box, 64)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sm_count());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kFixed + (size_t)ring.slots * boxes * ring.box_bytes();
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm, a, ring, ws);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace

uint32_t take_timeouts_moe() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    cudaMemcpyToSymbol(g_timeouts, &zero, sizeof(zero));
    return v;
}

size_t fp8_moe_workspace_bytes(int tokens, int hidden, int inter, int topk) {
    return ws_layout(nullptr, tokens, hidden, inter, topk, nullptr);
}

cudaError_t launch_fp8_moe_blockscaled(const MoeArgs &a, cudaStream_t s) {
    static DeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        const cudaError_t err =
            cudaFuncSetAttribute(k_moe_gate_up, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
        if (err != cudaSuccess) return err;
        const cudaError_t err8 =
            cudaFuncSetAttribute(k_moe_down<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
        if (err8 != cudaSuccess) return err8;
        return cudaFuncSetAttribute(k_moe_down<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    });
    if (e != cudaSuccess) return e;
    Ws ws;
    ws_layout(a.workspace, a.tokens, a.hidden, a.inter, a.topk, &ws);
    e = launch_one(k_moe_gate_up, a.w_gu, (int64_t)a.experts * 2 * a.inter, a.hidden, kConsumers, 2, a, ws, s);
    if (e != cudaSuccess) return e;
    // Four blocks of K side by side where eight leave more warps idle (inter
    // 1408, eleven blocks: 11 of 12 against 11 of 16; 16 tokens of 5120 x 1408
    // x 64 experts 5.2 TB/s against 5.0), else eight, with smaller tiles to
    // share and join (1 token, 2048 x 768 x 64: 22.3 us against 23.4).
    const int blocks = a.inter / SB;
    const bool four = (blocks + 3) / 4 * 4 < (blocks + 7) / 8 * 8;
    const int64_t rows = (int64_t)a.experts * a.hidden;
    return four ? launch_one(k_moe_down<4>, a.w_d, rows, a.inter, 4, 4, a, ws, s)
                : launch_one(k_moe_down<8>, a.w_d, rows, a.inter, 8, 2, a, ws, s);
}

}  // namespace bsq
