// Block-scaled FP8 GEMM for few activation rows: the same product as
// gemm_fp8_block.cu with the operands swapped (128 weight rows as the MMA's M
// operand, NT activation rows as its N operand) and K split over the CTAs of
// a cluster.
//
// Up to some hundred activation rows the weight stream is the cost, and N / 128
// tiles alone would not occupy the SMs: a 5120-row weight has 40.  So S CTAs
// (a cluster of 1 to 8) share a tile, each streaming its share of the K
// blocks; their FP32 sums are added through distributed shared memory in rank
// order, so the result does not depend on timing and no workspace is needed.
// Small rings let two CTAs share an SM.  16 x 5120 x 5120: 8.9 us back to back in
// a graph with the weight rotated past L2 (6.8 with it in L2), where a kernel
// that only reads the weight takes 5.6 and the copy peak 4.0: what is above the
// stream is the start of the ring behind the previous kernel and the join of a
// tile's sums.
//
// Per CTA (384 threads):
//   warp 0      TMA producer: one K block per stage (16 KB of W, NT x 128
//               bytes of A), as many stages as the launcher found room for
//   warp 1      tensor memory; one elected thread issues four 128 x NT x 32
//               MMAs per block into one of NBUF buffers
//   warp 2      scales: a_scale * w_scale of each activation row, four K
//               blocks at a time, into shared memory
//   warps 4..11 fold and epilogue: warp w owns weight rows 32 (w % 4) ..
//               and columns (w - 4) / 4 * NT / 2 ..; lane = weight row, so an
//               output store covers 32 consecutive columns of one row
#include <cstring>

#include "bsq_common.cuh"

namespace bsq {

namespace {

constexpr int BW = 128;  // weight rows per tile: one scale block
constexpr int BK = 128;  // one scale block of K
constexpr int W_BYTES = BW * BK;
constexpr int kFoldWarps = 8, kThreads = 32 * (4 + kFoldWarps);
constexpr int kMaxStages = 12, SG = 4, SSLOTS = 3;
constexpr int kMaxSplit = 8;

static __device__ unsigned int g_timeouts;

template <int NT> struct Cfg {
    static constexpr int A_BYTES = NT * BK, STAGE_BYTES = W_BYTES + A_BYTES;
    static constexpr int NBUF = 4;
    // 64 or 128 of 512: at most three CTAs of 384 threads fit an SM's registers,
    // so none of a cluster ever waits for columns that another cluster's CTA
    // holds while that one waits for its own peers
    static constexpr int TMEM_COLS = NBUF * NT;
    static constexpr int CW = NT / 2;            // columns of one fold warp
};

template <int NT> struct Smem {
    float f[SSLOTS][SG][NT];  // a_scale * w_scale
    uint64_t sfull[SSLOTS], sempty[SSLOTS];
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t tfull[Cfg<NT>::NBUF], tempty[Cfg<NT>::NBUF];
    uint64_t drain;
    uint32_t tmem_base;
    uint32_t abort;
};

// ring (also the NT x 128 FP32 sums at the end), then the barriers
template <int NT> size_t smem_bytes(int stages) {
    return 1024 + (size_t)stages * Cfg<NT>::STAGE_BYTES + sizeof(Smem<NT>);
}

template <int NT> __device__ __forceinline__ bool aborted(volatile Smem<NT> *s) { return s->abort != 0; }

template <int NT> __device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, Smem<NT> *S) {
    mbar_wait_or_abort(bar, parity, &S->abort, &g_timeouts);
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[8]) { tmem_ld_32x32b_x8(taddr, r); }
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(taddr, r); }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

//   grid: x = S * (row tiles), y = activation tiles; clusters of S along x
template <int NT>
__global__ void __launch_bounds__(kThreads, 2)
    k_gemm_small(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, int stages,
                 const float *__restrict__ a_scale, const float *__restrict__ w_scale, uint16_t *__restrict__ out,
                 int M, int N, int K) {
    using C = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Smem<NT> *S = reinterpret_cast<Smem<NT> *>(base + (size_t)stages * C::STAGE_BYTES);
    auto w_tile = [&](int s) { return base + (size_t)s * C::STAGE_BYTES; };
    auto a_tile = [&](int s) { return base + (size_t)s * C::STAGE_BYTES + W_BYTES; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int nkb_all = K / BK;
    const int kb0 = (int)((int64_t)nkb_all * rank / split), nkb = (int)((int64_t)nkb_all * (rank + 1) / split) - kb0;
    const int n0 = (int)(blockIdx.x / split) * BW, m0 = (int)blockIdx.y * NT;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; s++) {
            mbar_init(&S->full[s], 1);
            mbar_init(&S->empty[s], 1);
        }
        for (int b = 0; b < C::NBUF; b++) {
            mbar_init(&S->tfull[b], 1);
            mbar_init(&S->tempty[b], kFoldWarps);
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
        tmem_alloc(&S->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    launch_dependents();  // only now: a dependent must not take the tensor memory first
    const uint32_t tmem = S->tmem_base;
    dependency_wait();

    if (warp == 0) {
        if (elect_one()) {
            prefetch_tensormap(&tmW);
            prefetch_tensormap(&tmA);
            int s = 0;
            uint32_t ph = 1;
            int it = 0;
            bool ok = true;
            for (; it < nkb; it++) {
                if (!mbar_wait(&S->empty[s], ph, &g_timeouts) || aborted<NT>(S)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&S->full[s], C::STAGE_BYTES);
                tma_load_2d(w_tile(s), &tmW, &S->full[s], (kb0 + it) * BK, n0);
                tma_load_2d(a_tile(s), &tmA, &S->full[s], (kb0 + it) * BK, m0);
                if (++s == stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (!ok) {
                S->abort = 1;
                // let the copies in flight land before the CTA can exit
                for (int i = it > stages ? it - stages : 0; i < it; i++)
                    mbar_wait(&S->full[i % stages], (i / stages) & 1, &g_timeouts);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t idesc = idesc_e4m3(BW, NT);
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            bool ok = true;
            for (int it = 0; it < nkb; it++) {
                if (!mbar_wait(&S->full[s], ph, &g_timeouts) || !mbar_wait(&S->tempty[b], bph, &g_timeouts) ||
                    aborted<NT>(S)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t wd = sdesc_k_sw128(smem_u32(w_tile(s))), ad = wd + (W_BYTES >> 4);
#pragma unroll
                for (int j = 0; j < 4; j++)  // 32 bytes of K each: 2 in the descriptor's address field
                    mma_f8f6f4(tmem + b * NT, wd + 2 * j, ad + 2 * j, idesc, j != 0);
                tc_commit(&S->tfull[b]);
                tc_commit(&S->empty[s]);
                if (++s == stages) {
                    s = 0;
                    ph ^= 1;
                }
                b = (b + 1) % C::NBUF;
                bph ^= b == 0;
            }
            if (!ok) S->abort = 1;
            // wait for every tensor-core operation this thread issued
            tc_commit(&S->drain);
            mbar_wait(&S->drain, 0, &g_timeouts);
        }
    } else if (warp == 2) {
        // scales of SG blocks at a time
        const float *sw = w_scale + (int64_t)(n0 >> 7) * nkb_all + kb0;
        int s = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int g0 = 0; g0 < nkb; g0 += SG) {
            // loads first: they are in flight while the slot is waited for
            float v[SG], w[SG];
#pragma unroll
            for (int j = 0; j < SG; j++) w[j] = g0 + j < nkb ? __ldg(sw + g0 + j) : 0.0f;
            // rows past the end take a valid scale; they are never stored
            const float *sa = a_scale + (int64_t)min(m0 + lane, M - 1) * nkb_all + kb0 + g0;
#pragma unroll
            for (int j = 0; j < SG; j++) v[j] = g0 + j < nkb ? __ldg(sa + j) : 0.0f;
            ok = mbar_wait(&S->sempty[s], ph, &g_timeouts) && !aborted<NT>(S);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane < NT)
#pragma unroll
                for (int j = 0; j < SG; j++) S->f[s][j][lane] = v[j] * w[j];
            __syncwarp();
            if (lane == 0) mbar_arrive(&S->sfull[s]);
            if (++s == SSLOTS) {
                s = 0;
                ph ^= 1;
            }
        }
        if (!ok && lane == 0) S->abort = 1;
    } else if (warp >= 4) {
        constexpr int CW = C::CW;
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + h * CW;
        // arrivals through the cluster address: the plain form waits some 160
        // cycles for the warp's other memory operations
        const uint32_t tempty0 = mapa_shared(smem_u32(&S->tempty[0]), rank);
        const uint32_t sempty0 = mapa_shared(smem_u32(&S->sempty[0]), rank);
        float2 acc[CW / 2];
#pragma unroll
        for (int i = 0; i < CW / 2; i++) acc[i] = make_float2(0.0f, 0.0f);
        int b = 0, ss = 0;
        uint32_t bph = 0, sph = 0;
        for (int it = 0; it < nkb; it++) {
            if (it % SG == 0) wait_or_abort<NT>(&S->sfull[ss], sph, S);
            wait_or_abort<NT>(&S->tfull[b], bph, S);
            __syncwarp();
            tc_fence_after();
            uint32_t r[CW];
            ld_cols(tbase + b * NT, r);
            const float4 *fp = reinterpret_cast<const float4 *>(&S->f[ss][it % SG][h * CW]);
            float4 f[CW / 4];
#pragma unroll
            for (int i = 0; i < CW / 4; i++) f[i] = fp[i];
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * b);
#pragma unroll
            for (int i = 0; i < CW / 4; i++) {
                fma2(acc[2 * i], make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])),
                     make_float2(f[i].x, f[i].y));
                fma2(acc[2 * i + 1], make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])),
                     make_float2(f[i].z, f[i].w));
            }
            b = (b + 1) % C::NBUF;
            bph ^= b == 0;
            if (it % SG == SG - 1 || it == nkb - 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(sempty0 + 8 * ss);
                if (++ss == SSLOTS) {
                    ss = 0;
                    sph ^= 1;
                }
            }
        }
        const int n = n0 + 32 * q + lane;
        if (split == 1) {
            if (n < N) {
#pragma unroll
                for (int c = 0; c < CW; c++) {
                    const int m = m0 + h * CW + c;
                    const float v = c & 1 ? acc[c / 2].y : acc[c / 2].x;
                    if (m < M) out[(int64_t)m * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                }
            }
        } else {
            // this CTA's sums, [column][weight row], over the ring: every
            // copy has landed and every MMA has read it (its products have
            // been folded)
            float *part = reinterpret_cast<float *>(base);
#pragma unroll
            for (int c = 0; c < CW; c++)
                part[(h * CW + c) * BW + 32 * q + lane] = c & 1 ? acc[c / 2].y : acc[c / 2].x;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (split > 1) {
        cluster_sync();  // every CTA's sums are written
        // CTA `rank` finishes columns rank, rank + split, ...: the sums are
        // added in rank order
        const int cols = min(NT, M - m0);
        const uint32_t part = smem_u32(base);
        if (threadIdx.x < 2 * BW) {
            const int row = threadIdx.x & (BW - 1);
            for (int c = rank + split * (int)(threadIdx.x / BW); c < cols; c += 2 * split) {
                const uint32_t at = part + 4 * (c * BW + row);
                float v[kMaxSplit];
#pragma unroll
                for (int r = 0; r < kMaxSplit; r++)
                    if (r < split) v[r] = ld_cluster_f32(mapa_shared(at, r));
                float sum = v[0];
#pragma unroll
                for (int r = 1; r < kMaxSplit; r++)
                    if (r < split) sum += v[r];
                if (n0 + row < N)
                    out[(int64_t)(m0 + c) * N + n0 + row] = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
            }
        }
        cluster_sync();  // no CTA leaves while another reads its sums
    }
}

constexpr size_t kWholeSm = 226 * 1024, kHalfSm = 112 * 1024;

template <int NT> int ring_stages(size_t room) {
    const int n = (int)((room - 1024 - sizeof(Smem<NT>)) / Cfg<NT>::STAGE_BYTES);
    return n < kMaxStages ? n : kMaxStages;
}

struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Launch(int split, int tiles_n, int tiles_m, size_t smem, cudaStream_t s) {
        cfg.gridDim = dim3(split * tiles_n, tiles_m);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = split;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
};

// Clusters of `split` CTAs that can be resident at once (cached per device).
// Two CTAs share an SM here (half of its shared memory, a third of its
// registers and at most 128 of its 512 tensor-memory columns each), but the
// occupancy query counts one per SM for a kernel that allocates tensor memory,
// whatever its size, so its answer is doubled: the step in the measured times
// comes there (40 tiles: 6 x 40 CTAs 9.0 us, 7 x 40 14.0; 80 tiles of 64 x
// 5120 x 17408: 3 x 80 23 us, 4 x 80 35).
template <int NT> int max_clusters(int split) {
    // a racing first call computes the same value twice; the store is atomic
    static std::atomic<int> cached[kMaxDevices][kMaxSplit + 1];
    int dev = 0;
    cudaGetDevice(&dev);
    const bool cacheable = dev >= 0 && dev < kMaxDevices;
    if (cacheable) {
        const int c = cached[dev][split].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    Launch l(split, sm_count(), 1, smem_bytes<NT>(ring_stages<NT>(kHalfSm)), nullptr);
    l.cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_gemm_small<NT>, &l.cfg) != cudaSuccess || n <= 0) n = 1;
    n *= 2;
    if (cacheable) cached[dev][split].store(n, std::memory_order_relaxed);
    return n;
}

// CTAs per tile: as many as can all be resident at once (a cluster too many
// makes a second round, see above), but 1 where one CTA per tile nearly fills
// the SMs already (17408 x 5120, 136 tiles: 17.4 us at 16 rows, 18.2 with two;
// 17.5 and 19.5 at 32 rows) or where the ring holds
// all of a tile's K anyway (64 x 5120 x 1408: 5.3 us, 7.1 with three), and
// never below five K blocks each.
template <int NT> int split_for(int64_t tiles, int nkb) {
    if (4 * tiles >= 3 * (int64_t)sm_count() || nkb <= kMaxStages) return 1;
    for (int split = nkb / 5 < kMaxSplit ? nkb / 5 : kMaxSplit; split > 1; split--)
        if (tiles <= max_clusters<NT>(split)) return split;
    return 1;
}

template <int NT>
cudaError_t launch_nt(const uint8_t *a, const float *a_scale, const uint8_t *w, const float *w_scale, uint16_t *out,
                      int m, int n, int k, cudaStream_t s) {
    alignas(64) CUtensorMap tW, tA;
    if (!make_tmap_2d(&tW, w, 1, k, n, k, BK, BW, true, false) || !make_tmap_2d(&tA, a, 1, k, m, k, BK, NT, true, false))
        return cudaErrorInvalidValue;
    static DeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(k_gemm_small<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWholeSm);
    });
    if (e != cudaSuccess) return e;
    const int tiles_n = (n + BW - 1) / BW, tiles_m = (m + NT - 1) / NT, nkb = k / BK;
    const int64_t tiles = (int64_t)tiles_n * tiles_m;
    const int split = split_for<NT>(tiles, nkb);
    // a whole SM's shared memory when every CTA has an SM to itself (clusters
    // do not fill every SM: 17 tiles of 16 x 2112 x 17408, 8 x 17 CTAs, took
    // 17.1 us with whole SMs, 10.5 with halves), half of it otherwise, and no
    // more than the K blocks a CTA has
    int stages = ring_stages<NT>(2 * tiles <= max_clusters<NT>(split) ? kWholeSm : kHalfSm);
    // (the sums of a split tile need NT * 512 bytes of ring: at most two stages)
    const int per_cta = (nkb + split - 1) / split;
    stages = stages < per_cta ? stages : (per_cta > 2 ? per_cta : 2);
    Launch l(split, tiles_n, tiles_m, smem_bytes<NT>(stages), s);
    return cudaLaunchKernelEx(&l.cfg, k_gemm_small<NT>, tW, tA, stages, a_scale, w_scale, out, m, n, k);
}

static_assert(2 * Cfg<32>::STAGE_BYTES >= 32 * BW * 4 && 2 * Cfg<16>::STAGE_BYTES >= 16 * BW * 4, "sums in the ring");

}  // namespace

uint32_t take_timeouts_gemm_fp8_block_small() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    cudaMemcpyToSymbol(g_timeouts, &zero, sizeof(zero));
    return v;
}

// Activation rows of a tile: 16 up to 16 rows, else 32 (tiles of 64 and 128
// were slower at every size: the fold then needs more registers than two CTAs
// per SM leave).
cudaError_t launch_fp8_gemm_blockscaled_small(const uint8_t *a, const float *a_scale, const uint8_t *w,
                                              const float *w_scale, uint16_t *out, int m, int n, int k,
                                              cudaStream_t s) {
    return m <= 16 ? launch_nt<16>(a, a_scale, w, w_scale, out, m, n, k, s)
                   : launch_nt<32>(a, a_scale, w, w_scale, out, m, n, k, s);
}

}  // namespace bsq
