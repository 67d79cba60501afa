// Block-scaled FP8 GEMM on the sm_100a tensor cores: activations with one
// FP32 scale per 1 x 128, weight with one per 128 x 128,
//   C[m, n] = sum_b a_scale[m, b] w_scale[n / 128, b] sum_{k in block b} e4m3(A[m, k]) e4m3(W[n, k])
//
// The tensor cores sum one block of 128 at a time into tensor memory; the
// FP32 lanes fold each block with its scales into accumulators that stay in
// registers.  In a 256-column tile a thread holds one output row and 128
// columns, all inside one 128-wide scale block, so a block's two scales
// multiply to one factor per thread and the fold is one FMA per output.
//
// CTA pairs (clusters of two SMs), persistent over 256 x 256 output tiles.
// One pair MMA (tcgen05.mma.cta_group::2, 256 x 256 x 32) runs on both SMs'
// tensor cores; each CTA holds 128 rows of A and 128 of the tile's 256 weight
// rows and receives 128 x 256 of the products in its tensor memory.
// Per CTA (384 threads):
//   warp 0      TMA producer, a six-stage ring of one K block each (16 KB of
//               A, 16 KB of W), counted on the even CTA's barrier
//   warp 1      tensor memory for the pair; in the even CTA, lane 0 issues
//               four MMAs per block into one of two 256-column buffers, so
//               the next block's products overlap this block's fold
//   warps 4..11 fold and epilogue: warp w owns lane group w % 4 and column
//               half (w - 4) / 4; output through swizzled shared memory and
//               TMA stores (plain stores where a row is not a multiple of 16
//               bytes)
// Per SM and K block the MMAs take 512 cycles and the fold's 32,768 FMAs 256
// of the FP32 lanes' cycles.
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

template <int R> __device__ __forceinline__ void setmaxnreg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R> __device__ __forceinline__ void setmaxnreg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// (d0, d1) += (a0, a1) * (b0, b1), packed
__device__ __forceinline__ void fma2(float2 &d, float2 a, float2 b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(*reinterpret_cast<uint64_t *>(&d))
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
}

// Pair MMA: D (128 lanes of each CTA) (+)= A (128 rows in each CTA) x
// B (N rows, half in each CTA), E4M3, issued by the even CTA.
__device__ __forceinline__ void mma_f8f6f4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

namespace pair {

constexpr int BM = 128;       // rows of A per CTA (256 per pair)
constexpr int BN = 256;       // output columns per tile
constexpr int BNH = BN / 2;   // weight rows per CTA
constexpr int BK = 128;       // one scale block, in bytes = elements
constexpr int STAGES = 6;
constexpr int A_BYTES = BM * BK, B_BYTES = BNH * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int NBUF = 2, TMEM_COLS = 512;
constexpr int kFoldWarps = 8, kThreads = 32 * (4 + kFoldWarps);
// Launched with 168 registers a thread; warps 0-3 drop to 56, the two fold
// warpgroups take 224: 128 * 56 + 256 * 224 = 384 * 168.  The launcher checks
// the compiled count.
constexpr int kLaunchRegs = 168, kCtlRegs = 56, kFoldRegs = 224;
static_assert(128 * kCtlRegs + 32 * kFoldWarps * kFoldRegs <= kThreads * kLaunchRegs, "register split");
// output staging: per fold warp one TMA store box of 32 rows x 64 columns
constexpr int OUT_BOX_COLS = 64, OUT_BOX_ROWS = 32, OUT_BOX_BYTES = OUT_BOX_COLS * 2 * OUT_BOX_ROWS;

struct Smem {
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

__global__ void __launch_bounds__(kThreads, 1)
    k_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
           const __grid_constant__ CUtensorMap tmOut, int use_tma_store, const float *__restrict__ a_scale,
           const float *__restrict__ w_scale, uint16_t *__restrict__ out, int M, int N, int K) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *out_stage = base + (size_t)STAGES * STAGE_BYTES;
    Smem *S = reinterpret_cast<Smem *>(out_stage + kFoldWarps * OUT_BOX_BYTES);
    auto a_tile = [&](int s) { return base + (size_t)s * STAGE_BYTES; };
    auto b_tile = [&](int s) { return base + (size_t)s * STAGE_BYTES + A_BYTES; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int tiles_m = (M + 2 * BM - 1) / (2 * BM), tiles_n = (N + BN - 1) / BN;
    const int num_tiles = tiles_m * tiles_n;
    const int nkb = K / BK;

    launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(&S->full[s], 1);
            mbar_init(&S->empty[s], 1);
        }
        for (int b = 0; b < NBUF; b++) {
            mbar_init(&S->tfull[b], 1);
            mbar_init(&S->tempty[b], 2 * kFoldWarps);
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
    const uint32_t tmem = S->tmem_base;
    auto leader = [&](uint64_t *bar) { return mapa_shared(smem_u32(bar), 0); };
    if (warp < 4) setmaxnreg_dec<kCtlRegs>();

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (lane == 0) {
            prefetch_tensormap(&tmA);
            prefetch_tensormap(&tmB);
            dependency_wait();
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; t < num_tiles && ok; t += npairs) {
                const int mt = t % tiles_m, nt = t / tiles_m;
                const int arow = mt * 2 * BM + (int)rank * BM, brow = nt * BN + (int)rank * BNH;
                for (int kb = 0; kb < nkb; kb++, it++) {
                    const int s = it % STAGES;
                    if (!mbar_wait(&S->empty[s], ((it / STAGES) & 1) ^ 1, &g_timeouts) || aborted(S)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&S->full[s], 2 * STAGE_BYTES);
                    const uint32_t bar = leader(&S->full[s]);
                    tma_load_2d_pair(a_tile(s), &tmA, bar, kb * BK, arow);
                    tma_load_2d_pair(b_tile(s), &tmB, bar, kb * BK, brow);
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
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = idesc_e4m3(2 * BM, BN);
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; t < num_tiles && ok; t += npairs) {
                for (int kb = 0; kb < nkb; kb++, it++) {
                    const int s = it % STAGES, b = it % NBUF;
                    if (!mbar_wait(&S->full[s], (it / STAGES) & 1, &g_timeouts) ||
                        !mbar_wait_cluster(&S->tempty[b], ((it / NBUF) & 1) ^ 1, &g_timeouts) || aborted(S)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(a_tile(s)), b0 = smem_u32(b_tile(s));
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        mma_f8f6f4_pair(tmem + b * BN, sdesc_k_sw128(a0 + 32 * j), sdesc_k_sw128(b0 + 32 * j), idesc,
                                        j != 0);
                    tc_commit_pair_multicast(&S->empty[s], 0x3);
                    tc_commit_pair_multicast(&S->tfull[b], 0x3);
                }
            }
            if (!ok) S->abort = 1;
            // wait for every tensor-core operation this thread issued
            tc_commit_pair_multicast(&S->drain, 0x1);
            mbar_wait(&S->drain, 0, &g_timeouts);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------- fold + epilogue
        setmaxnreg_inc<kFoldRegs>();
        const int q = warp & 3, h = (warp - 4) >> 2;
        uint8_t *stage = out_stage + (warp - 4) * OUT_BOX_BYTES;
        const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + h * 128;
        if (lane == 0) prefetch_tensormap(&tmOut);
        dependency_wait();
        uint32_t it = 0;
        bool ok = true;
        for (int t = pair; t < num_tiles && ok; t += npairs) {
            const int mt = t % tiles_m, nt = t / tiles_m;
            const int row0 = mt * 2 * BM + (int)rank * BM + 32 * q;  // first row of this warp
            const int col0 = nt * BN + h * 128;
            // rows and columns past the end read a valid scale; their products are zero or never stored
            const float *sa = a_scale + (int64_t)min(row0 + lane, M - 1) * nkb;
            const float *sw = w_scale + (int64_t)(min(col0, N - 1) >> 7) * nkb;
            float2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; i++) acc[i] = make_float2(0.0f, 0.0f);
            float sa_n = __ldg(sa), sw_n = __ldg(sw);
            for (int kb = 0; kb < nkb; kb++, it++) {
                const int b = it % NBUF;
                const float f = sa_n * sw_n;
                const float2 ff = make_float2(f, f);
                if (kb + 1 < nkb) {
                    sa_n = __ldg(sa + kb + 1);
                    sw_n = __ldg(sw + kb + 1);
                }
                // (no abort-flag read here: if another role gives up, nothing more is committed and this
                // bounded wait ends the fold)
                ok = mbar_wait(&S->tfull[b], (it / NBUF) & 1, &g_timeouts);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = tbase + b * BN;
                uint32_t r0[32], r1[32];
                auto fold = [&](const uint32_t(&r)[32], int c) {
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        fma2(acc[16 * c + i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), ff);
                };
                tmem_ld_32x32b_x32(src, r0);
                tmem_ld_wait();
                tmem_ld_32x32b_x32(src + 32, r1);
                fold(r0, 0);
                tmem_ld_wait();
                tmem_ld_32x32b_x32(src + 64, r0);
                fold(r1, 1);
                tmem_ld_wait();
                tmem_ld_32x32b_x32(src + 96, r1);
                fold(r0, 2);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(leader(&S->tempty[b]));
                fold(r1, 3);
            }
            if (!ok) {
                if (lane == 0) S->abort = 1;
                break;
            }
            if (use_tma_store) {
                // box bx holds columns [64 bx, 64 bx + 64) of the warp's 32 x 128
                // block; lane = row; 16-byte unit u of a row sits at u ^ (row & 7)
#pragma unroll
                for (int bx = 0; bx < 2; bx++) {
                    if (lane == 0) bulk_wait_group_read0();  // the previous store has read the box
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 8; u++) {
                        const float2 *v = acc + 32 * bx + 4 * u;
                        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) =
                            make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                       pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < M && col0 + bx * OUT_BOX_COLS < N) {
                        tma_store_2d(&tmOut, stage, col0 + bx * OUT_BOX_COLS, row0);
                        bulk_commit_group();
                    }
                }
            } else if (row0 + lane < M) {
                uint16_t *orow = out + (int64_t)(row0 + lane) * N;
#pragma unroll
                for (int i = 0; i < 64; i++) {
                    const int n = col0 + 2 * i;
                    if (n < N) orow[n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i].x));
                    if (n + 1 < N) orow[n + 1] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i].y));
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
    if (use_tma_store && !make_tmap_2d(&tO, out, 2, n, m, (uint64_t)n * 2, OUT_BOX_COLS, OUT_BOX_ROWS, true, false))
        return cudaErrorInvalidValue;
    if (!make_tmap_2d(&tA, a, 1, k, m, k, BK, BM, true, false) || !make_tmap_2d(&tB, w, 1, k, n, k, BK, BNH, true, false))
        return cudaErrorInvalidValue;
    static DeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        cudaFuncAttributes fa;
        cudaError_t err = cudaFuncGetAttributes(&fa, k_gemm);
        if (err != cudaSuccess) return err;
        // a register split above the launch's total would wait forever
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
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

cudaError_t launch_fp8_gemm_blockscaled(const uint8_t *a, const float *a_scale, const uint8_t *w,
                                        const float *w_scale, uint16_t *out, int m, int n, int k, cudaStream_t s) {
    const cudaError_t e = pair::launch(a, a_scale, w, w_scale, out, m, n, k, s);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace bsq
