// Block-scaled FP8 GEMM on the sm_100a tensor cores: activations with one
// FP32 scale per 1 x 128, weight with one per 128 x 128,
//   C[m, n] = sum_b a_scale[m, b] w_scale[n / 128, b] sum_{k in block b} e4m3(A[m, k]) e4m3(W[n, k])
//
// The tensor cores sum one block of 128 at a time into tensor memory; the
// FP32 lanes fold each block with its scales into accumulators that stay in
// registers.  An output tile is one weight scale block wide, so a block's two
// scales multiply to one factor per row and the fold is one FMA per output.
//
// CTA pairs (clusters of two SMs), persistent over 256 x 128 output tiles.
// One pair MMA (tcgen05.mma.cta_group::2, 256 x 128 x 32) runs on both SMs'
// tensor cores; each CTA holds 128 rows of A and 64 of the tile's 128 weight
// rows and receives 128 x 128 of the products in its tensor memory.
// Per CTA (384 threads):
//   warp 0      TMA producer, a ring of STAGES stages of GB = 2 K blocks (32
//               KB of A, 16 KB of W), counted on the even CTA's barrier
//   warp 1      tensor memory for the pair; in the even CTA, one elected
//               thread issues the MMAs: per stage two blocks of four 256 x 128
//               x 32 into one of NBUF = 2 buffers (of two 128-column blocks:
//               all 512 columns)
//   warp 2      brings the activation and weight scales into shared memory,
//               four blocks at a time (one load per activation row and fold
//               thread, straight from global memory, cost more than the MMAs)
//   warps 4..11 fold and epilogue: warp w owns lane group w % 4 (32 rows) and
//               64 columns, (w - 4) / 4; output through swizzled shared memory
//               and TMA stores (plain stores where a row is not a multiple of
//               16 bytes)
// Per SM and K block the MMAs take 256 cycles and the fold's 16,384 FMAs 64 to
// 128 of the FP32 lanes' cycles; a block takes about 455.  What is between is
// the round of a buffer: MMAs, commit, the waiting warps' wake-up, two
// tensor-memory loads of 64 columns, the arrival at the even CTA.  Two blocks
// per stage halve the rounds, and the issue takes about 50 cycles per MMA
// (elected thread, precomputed descriptor words), under the 64 that it runs.
// 4096 x 17408 x 5120: 344 to 358 us by operands' values in a burst (2.04 to
// 2.12 PFLOP/s), 408 when repeated for seconds, where the power limit holds the
// clock at 1.43 GHz; 225 at twice the BF16 rate of a plain product.  Tiles of 256 x 256 (fold of 128 registers per thread, 16 or 8
// warps), one block per stage, and two tiles in turn were not faster.
//
// Launched with programmatic stream serialization: every role waits for the
// previous kernel (griddepcontrol.wait) before its first global access.
// Every mbarrier wait is bounded; on a timeout the kernel records it, stops
// issuing work, drains what it issued, frees tensor memory and exits.
#include <cstring>

#include "bsq_common.cuh"

namespace bsq {

namespace {

static __device__ unsigned int g_timeouts;

// Pair MMA: D (128 lanes of each CTA) (+)= A (128 rows in each CTA) x
// B (N rows, half in each CTA), E4M3, issued by the even CTA.  The low words
// of the descriptors (start address) vary; the high word is the same for all.
__device__ __forceinline__ void mma_f8f6f4_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t desc_hi,
                                                uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(desc_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

namespace pair {

constexpr int BM = 128;       // rows of A per CTA (256 per pair)
constexpr int BN = 128;       // output columns per tile: one scale block
constexpr int BK = 128;       // one scale block, in bytes = elements
constexpr int GB = 2;         // K blocks of one stage, one round of the barriers
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK, B_BYTES = BN / 2 * BK;  // of one K block
constexpr int STAGE_BYTES = GB * (A_BYTES + B_BYTES);
constexpr int NBUF = 2, TMEM_COLS = NBUF * GB * BN;
constexpr int kFoldWarps = 8, kThreads = 32 * (4 + kFoldWarps);
// output staging: per fold warp one TMA store box of 32 rows x 32 columns
// (64-byte rows, 64-byte swizzle), used twice per tile
constexpr int OUT_BOX_COLS = 32, OUT_BOX_ROWS = 32, OUT_BOX_BYTES = OUT_BOX_COLS * 2 * OUT_BOX_ROWS;

constexpr int SG = 4, SSLOTS = 3;  // scale blocks per slot, slots

struct Smem {
    float4 sa[SSLOTS][BM];  // this CTA's rows, SG consecutive blocks each
    float4 sw[SSLOTS];
    uint64_t sfull[SSLOTS], sempty[SSLOTS];
    uint64_t full[STAGES];   // even CTA: both CTAs' A and W tiles landed
    uint64_t empty[STAGES];  // both: the pair MMAs of this stage are done
    uint64_t tfull[NBUF];    // both: a block's products are in tensor memory
    uint64_t tempty[NBUF];   // even CTA: both CTAs have read them
    uint64_t drain;
    uint32_t tmem_base;
    uint32_t abort;
};
constexpr size_t kSmemBytes = 1024 + (size_t)STAGES * STAGE_BYTES + kFoldWarps * OUT_BOX_BYTES + sizeof(Smem);
static_assert(kSmemBytes <= 232448, "shared memory per block");

__device__ __forceinline__ bool aborted(volatile Smem *s) { return s->abort != 0; }

__device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, Smem *S) {
    mbar_wait_or_abort(bar, parity, &S->abort, &g_timeouts);
}

__global__ void __launch_bounds__(kThreads, 1)
    k_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
           const __grid_constant__ CUtensorMap tmOut, int use_tma_store, const float *__restrict__ a_scale,
           const float *__restrict__ w_scale, uint16_t *__restrict__ out, int M, int N, int K) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *out_stage = base + (size_t)STAGES * STAGE_BYTES;
    Smem *S = reinterpret_cast<Smem *>(out_stage + kFoldWarps * OUT_BOX_BYTES);
    auto a_tile = [&](int s) { return base + (size_t)s * STAGE_BYTES; };
    auto b_tile = [&](int s) { return base + (size_t)s * STAGE_BYTES + GB * A_BYTES; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int tiles_m = (M + 2 * BM - 1) / (2 * BM), tiles_n = (N + BN - 1) / BN;
    const int num_tiles = tiles_m * tiles_n;
    const int nkb = K / BK, ngr = (nkb + GB - 1) / GB;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(&S->full[s], 1);
            mbar_init(&S->empty[s], 1);
        }
        for (int i = 0; i < NBUF; i++) {
            mbar_init(&S->tfull[i], 1);
            mbar_init(&S->tempty[i], 2 * kFoldWarps);
        }
        for (int i = 0; i < SSLOTS; i++) {
            mbar_init(&S->sfull[i], 1);
            mbar_init(&S->sempty[i], kFoldWarps);
        }
        mbar_init(&S->drain, 1);
        S->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&S->tmem_base, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    launch_dependents();  // only now: a dependent must not take the tensor memory first
    dependency_wait();    // every role: the bounded waits start with this kernel's own work
    const uint32_t tmem = S->tmem_base;
    auto leader = [&](uint64_t *bar) { return mapa_shared(smem_u32(bar), 0); };

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (elect_one()) {
            prefetch_tensormap(&tmA);
            prefetch_tensormap(&tmB);
            const uint32_t full0 = leader(&S->full[0]);
            uint32_t it = 0, ph = 1;
            int s = 0;
            bool ok = true, ready = mbar_test(&S->empty[0], 1);
            for (int t = pair; t < num_tiles && ok; t += npairs) {
                const int mt = t % tiles_m, nt = t / tiles_m;
                const int arow = mt * 2 * BM + (int)rank * BM, brow = nt * BN + (int)rank * (BN / 2);
                for (int g = 0; g < ngr; g++, it++) {
                    if (!ready && (!mbar_wait(&S->empty[s], ph, &g_timeouts) || aborted(S))) {
                        ok = false;
                        break;
                    }
                    // the next slot's barrier, read while this slot's copies are issued
                    const int s1 = s + 1 == STAGES ? 0 : s + 1;
                    const uint32_t ph1 = s1 == 0 ? ph ^ 1 : ph;
                    ready = mbar_test(&S->empty[s1], ph1);
                    if (rank == 0) mbar_arrive_expect_tx(&S->full[s], 2 * STAGE_BYTES);
                    const uint32_t bar = full0 + 8 * s;
                    // [block][row][128 B]; a block past K is filled with zeros
                    tma_load_3d_pair(a_tile(s), &tmA, bar, 0, arow, g * GB);
                    tma_load_3d_pair(b_tile(s), &tmB, bar, 0, brow, g * GB);
                    s = s1;
                    ph = ph1;
                }
            }
            if (!ok) {
                S->abort = 1;
                // let the copies in flight land before either CTA can exit
                // (the even CTA's barriers count both CTAs' copies)
                const uint32_t first = it > STAGES ? it - STAGES : 0;
                if (rank == 0)
                    for (uint32_t i = first; i < it; i++)
                        mbar_wait(&S->full[i % STAGES], (i / STAGES) & 1, &g_timeouts);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------ pair MMA issuer (even CTA)
        if (rank == 0 && elect_one()) {
            const uint32_t idesc = idesc_e4m3(2 * BM, BN);
            const uint64_t desc0 = sdesc_k_sw128(smem_u32(a_tile(0)));
            const uint32_t desc_hi = (uint32_t)(desc0 >> 32);
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            bool ok = true, ready = false;
            for (int t = pair; t < num_tiles && ok; t += npairs) {
                for (int g = 0; g < ngr; g++) {
                    if (!ready && (!mbar_wait(&S->full[s], ph, &g_timeouts) ||
                                   !mbar_wait(&S->tempty[b], bph, &g_timeouts) || aborted(S))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // the next stage's barriers, read while this one's MMAs
                    // are issued
                    const int s1 = s + 1 == STAGES ? 0 : s + 1, b1 = (b + 1) % NBUF;
                    const uint32_t ph1 = s1 == 0 ? ph ^ 1 : ph, bph1 = b1 == 0 ? bph ^ 1 : bph;
                    const bool r0 = mbar_test(&S->full[s1], ph1), r1 = mbar_test(&S->tempty[b1], bph1);
                    const uint32_t ad = (uint32_t)desc0 + s * (STAGE_BYTES >> 4), bd = ad + (GB * A_BYTES >> 4);
#pragma unroll
                    for (int u = 0; u < GB; u++)
#pragma unroll
                        for (int j = 0; j < 4; j++)  // 32 bytes of K each: 2 in the descriptor's address field
                            mma_f8f6f4_pair(tmem + (b * GB + u) * BN, ad + u * (A_BYTES >> 4) + 2 * j,
                                            bd + u * (B_BYTES >> 4) + 2 * j, desc_hi, idesc, j != 0);
                    tc_commit_pair_multicast(&S->tfull[b], 0x3);
                    tc_commit_pair_multicast(&S->empty[s], 0x3);
                    ready = r0 && r1;
                    s = s1, b = b1;
                    ph = ph1, bph = bph1;
                }
            }
            if (!ok) S->abort = 1;
            // wait for every tensor-core operation this thread issued
            tc_commit_pair_multicast(&S->drain, 0x1);
            mbar_wait(&S->drain, 0, &g_timeouts);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------- scales
        const bool vec = (nkb & 3) == 0 &&
                         ((reinterpret_cast<uintptr_t>(a_scale) | reinterpret_cast<uintptr_t>(w_scale)) & 15) == 0;
        uint32_t g = 0;
        bool ok = true;
        for (int t = pair; t < num_tiles && ok; t += npairs) {
            const int mt = t % tiles_m, nt = t / tiles_m;
            // rows and columns past the end take a valid scale; their products are zero or never stored
            const float *sa[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                sa[i] = a_scale + (int64_t)min(mt * 2 * BM + (int)rank * BM + 32 * i + lane, M - 1) * nkb;
            const float *sw = w_scale + (int64_t)nt * nkb;
            for (int kb = 0; kb < nkb; kb += SG, g++) {
                // loads first: they are in flight while the slot is waited for
                auto four = [&](const float *p) {  // zeros past the last block
                    if (vec) return __ldg(reinterpret_cast<const float4 *>(p + kb));
                    return make_float4(__ldg(p + kb), kb + 1 < nkb ? __ldg(p + kb + 1) : 0.0f,
                                       kb + 2 < nkb ? __ldg(p + kb + 2) : 0.0f, kb + 3 < nkb ? __ldg(p + kb + 3) : 0.0f);
                };
                float4 v[4], vw;
#pragma unroll
                for (int i = 0; i < 4; i++) v[i] = four(sa[i]);
                if (lane == 0) vw = four(sw);
                const int s = g % SSLOTS;
                ok = mbar_wait(&S->sempty[s], ((g / SSLOTS) & 1) ^ 1, &g_timeouts) && !aborted(S);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; i++) S->sa[s][32 * i + lane] = v[i];
                if (lane == 0) S->sw[s] = vw;
                __syncwarp();
                if (lane == 0) mbar_arrive(&S->sfull[s]);
            }
        }
        if (!ok && lane == 0) S->abort = 1;
    } else if (warp >= 4) {
        // ------------------------------------------------- fold + epilogue
        // lane group q, column half h
        const int q = warp & 3, h = (warp - 4) >> 2;
        uint8_t *stage = out_stage + (warp - 4) * OUT_BOX_BYTES;
        const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + h * 64;
        const uint32_t tempty0 = leader(&S->tempty[0]);
        // arrivals through the cluster address even where the barrier is this
        // CTA's: the plain form takes 160 cycles here, this one none
        const uint32_t sempty0 = mapa_shared(smem_u32(&S->sempty[0]), rank);
        if (use_tma_store && lane == 0) prefetch_tensormap(&tmOut);
        uint32_t bph = 0, sph = 0;
        int b = 0, ss = 0;
        bool ready = false;
        for (int t = pair; t < num_tiles; t += npairs) {
            const int mt = t % tiles_m, nt = t / tiles_m;
            const int row0 = mt * 2 * BM + (int)rank * BM + 32 * q;  // first row of this warp
            const int col0 = nt * BN + h * 64;
            float2 acc[32];
#pragma unroll
            for (int i = 0; i < 32; i++) acc[i] = make_float2(0.0f, 0.0f);
            for (int kb0 = 0; kb0 < nkb; kb0 += SG) {
                wait_or_abort(&S->sfull[ss], sph, S);
                const float4 xa = S->sa[ss][32 * q + lane], xw = S->sw[ss];
                float f0 = xa.x * xw.x, f1 = xa.y * xw.y;
                const float f2 = xa.z * xw.z, f3 = xa.w * xw.w;
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(sempty0 + 8 * ss);
                if (++ss == SSLOTS) {
                    ss = 0;
                    sph ^= 1;
                }
#pragma unroll 1
                for (int j = 0; j < min(SG, nkb - kb0); j += GB) {
                    if (!ready) wait_or_abort(&S->tfull[b], bph, S);
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t src = tbase + b * GB * BN;
                    uint32_t r[64];
                    auto fold = [&](float f1) {
                        const float2 ff = make_float2(f1, f1);
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            fma2(acc[i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), ff);
                    };
                    tmem_ld_32x32b_x64(src, r);
                    tmem_ld_wait();
                    fold(f0);
                    tmem_ld_32x32b_x64(src + BN, r);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * b);
                    // the next stage's barrier, read while this one is folded
                    b = (b + 1) % NBUF;
                    bph ^= b == 0;
                    ready = mbar_test(&S->tfull[b], bph);
                    fold(f1);  // (past an odd last block: zeros times a scale of zero)
                    f0 = f2, f1 = f3;
                }
            }
            // every lane leaves together
            if (__any_sync(0xFFFFFFFFu, aborted(S))) break;
            // box bx holds columns [32 bx, 32 bx + 32) of the warp's 32 x 64
            // block; lane = row; 16-byte unit u of a row sits at u ^ ((row >> 1) & 3)
#pragma unroll
            for (int bx = 0; bx < 2; bx++) {
                if (lane == 0) bulk_wait_group_read0();  // the previous store has read the box
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const float2 *v = acc + 16 * bx + 4 * u;
                    *reinterpret_cast<uint4 *>(stage + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
                        make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                   pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
                }
                const int col = col0 + bx * OUT_BOX_COLS;
                if (use_tma_store) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < M && col < N) {
                        tma_store_2d(&tmOut, stage, col, row0);
                        bulk_commit_group();
                    }
                } else {
                    // plain stores, a row's 32 columns together: lane = column
                    __syncwarp();
                    // (by the thread that holds the row: 678 us instead of 79
                    // at 4096 x 17407 x 256, 290 instead of 108 at 4096 x 5121
                    // x 5120)
                    const int rows = min(32, M - row0);
                    uint16_t *o = out + (int64_t)row0 * N + col + lane;
                    if (col + lane < N)
#pragma unroll 8
                        for (int r = 0; r < rows; r++, o += N)
                            *o = *reinterpret_cast<const uint16_t *>(
                                stage + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + 2 * (lane & 7));
                    __syncwarp();
                }
            }
        }
        if (lane == 0) bulk_wait_group0();  // stores complete before the CTA exits
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no pair MMA or cross-CTA signal is in flight after this
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

// CTA pairs that can be resident at once (cached per device).
int max_pairs(cudaLaunchConfig_t cfg) {
    // a racing first call computes the same value twice; the store is atomic
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    const bool cacheable = dev >= 0 && dev < kMaxDevices;
    if (cacheable) {
        const int c = cached[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    cfg.gridDim = dim3(sm_count());
    if (cudaOccupancyMaxActiveClusters(&n, k_gemm, &cfg) != cudaSuccess || n <= 0) n = sm_count() / 2;
    if (cacheable) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch(const uint8_t *a, const float *a_scale, const uint8_t *w, const float *w_scale, uint16_t *out,
                   int m, int n, int k, cudaStream_t s) {
    alignas(64) CUtensorMap tA, tB, tO;
    // TMA stores need 16-byte output rows
    const int use_tma_store = (n % 8) == 0;
    memset(&tO, 0, sizeof(tO));
    if (use_tma_store) {
        const uint64_t d[2] = {(uint64_t)n, (uint64_t)m}, st[1] = {(uint64_t)n * 2};
        const uint32_t box[2] = {OUT_BOX_COLS, OUT_BOX_ROWS};
        if (!make_tmap(&tO, out, 2, 2, d, st, box, 64)) return cudaErrorInvalidValue;
    }
    if (!make_tmap_rows_chunks(&tA, a, k, m, BM, GB) || !make_tmap_rows_chunks(&tB, w, k, n, BN / 2, GB))
        return cudaErrorInvalidValue;
    static DeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(k_gemm, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int most = max_pairs(cfg);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    const int tiles = ((m + 2 * BM - 1) / (2 * BM)) * ((n + BN - 1) / BN);
    cfg.gridDim = dim3(2 * (tiles < most ? tiles : most));
    return cudaLaunchKernelEx(&cfg, k_gemm, tA, tB, tO, use_tma_store, a_scale, w_scale, out, m, n, k);
}

}  // namespace pair

}  // namespace

uint32_t take_timeouts_gemm_fp8_block() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    cudaMemcpyToSymbol(g_timeouts, &zero, sizeof(zero));
    return v;
}

// The swapped-operand kernel up to 64 rows (64 x 17408 x 5120: 19.6 us against
// 23.7 here, 65 rows 32.1 against 24.0; 64 x 5120 x 5120: 11.5 against 13.1),
// and beyond while its tiles of 128 x 32 outputs fit one to an SM (x 5120 x
// 5120: 96 rows, 120 tiles, 12.9 against 13.4; 128 rows, 160 tiles, 17.3
// against 13.5; x 2112 x 5120: 128 rows, 68 tiles, 10.5 against 12.7; 256 rows,
// 136 tiles, 12.7 both; 320 rows, 170 tiles, 17.6 against 12.8).  K moves this
// bound little (x 5120 x 17408: 96 rows 36.0 against 34.9, 128 rows 51.1
// against 35.0; x 5120 x 1408: 96 rows 5.7 against 7.0, 128 rows 7.0 against
// 7.2).  Back to back in a graph, weights rotated past L2.
cudaError_t launch_fp8_gemm_blockscaled(const uint8_t *a, const float *a_scale, const uint8_t *w,
                                        const float *w_scale, uint16_t *out, int m, int n, int k, cudaStream_t s) {
    const int64_t small_tiles = (int64_t)((n + 127) / 128) * ((m + 31) / 32);
    const cudaError_t e = m <= 64 || small_tiles <= sm_count()
                              ? launch_fp8_gemm_blockscaled_small(a, a_scale, w, w_scale, out, m, n, k, s)
                              : pair::launch(a, a_scale, w, w_scale, out, m, n, k, s);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace bsq
