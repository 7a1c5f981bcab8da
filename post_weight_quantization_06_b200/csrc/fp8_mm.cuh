// Product of two e4m3 matrices with block scales on the 5th-generation tensor cores
// (gptq_fp8_matmul):
//   Y[i][j] = sum_b sA[i][b] sB[j / 128][b] sum_{l in b} A[i][l] B[j][l],   blocks b of 128
//
// The scales change with every block of K, so a block's product (four tcgen05.mma of K = 32 into a
// fresh TMEM accumulator) is read back, scaled and added to fp32 sums in registers by the
// "promotion" warps while the next block's MMAs run into another accumulator.
#pragma once

#include "hessian_tc.cuh"
#include "serve_common.cuh"

namespace gptq {
namespace serve {

using tc::cluster_sync_all;
using tc::mbar_arrive;
using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;
using tc::mma_commit;
using tc::smem_u32;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tma_load_2d;
using tc::tmem_alloc;
using tc::tmem_dealloc;
using tc::tmem_relinquish;

constexpr int MM_BK = 128;                 // codes (= bytes) of K per stage: one scale block
constexpr int MM_SCALE_SLOTS = 8;          // ring of scale vectors

// kind::f8f6f4, D fp32, A and B e4m3, both K-major.
__host__ __device__ constexpr uint32_t mm_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// K-major operand in the 128-byte swizzle: rows of 128 bytes, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t mm_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)((1024 >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
__device__ __forceinline__ void mma_e4m3(uint32_t dtmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// 16 columns of this thread's TMEM lane, without the wait; mm_wait_ld16 ties the wait to them.
__device__ __forceinline__ void mm_ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void mm_wait_ld16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(on ? 4 : 0)
                 : "memory");
}
// The lane's earlier cp.async copies count as one arrival on `bar` once they have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

struct MmArgs {
    const float *sA, *sB;
    void *Y;
    long long ldy;
    int m, n, kb;            // kb: blocks of K
    int tiles_n;             // 128-row tiles of B
    int split;               // CTAs of a cluster, each with a part of the K blocks
    long long wait_limit;
};

// ---------------------------------------------------------------------------------------
// Few rows of A (decode): the weights' rows are the MMA's 128 rows and NT tokens its columns, so
// a 128 x NT tile costs only the weight's bytes. The blocks of K are split over the `split` CTAs of a
// cluster, which add their sums through distributed shared memory in a fixed order.
//
// Warps: 0 TMA, 1 TMEM and MMA, 2-5 promotion (32 weight rows each), 6 scales.
// ---------------------------------------------------------------------------------------
constexpr int NARROW_THREADS = 224;

template <int NT>
struct NarrowShape {
    static constexpr int W_BYTES = 128 * MM_BK;
    static constexpr int X_BYTES = NT * MM_BK;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int STAGES = NT <= 32 ? 9 : NT <= 64 ? 8 : 6;
    static constexpr int SLOT = NT + 4;   // scales of NT tokens, then the weight tile's
    static constexpr int BUFS = NT <= 64 ? 4 : 2;
    static constexpr int TMEM = NT * BUFS < 32 ? 32 : NT * BUFS;
    static constexpr int BARS = 2 * STAGES + 2 * BUFS + 2 * MM_SCALE_SLOTS + 2;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES +
                                   sizeof(float) * MM_SCALE_SLOTS * SLOT + 8 * BARS + 64;
    static_assert(SMEM <= 232448, "fits the shared memory of one CTA");
    static_assert((TMEM & (TMEM - 1)) == 0 && TMEM <= 512, "a TMEM allocation");
    static_assert(NT * 128 * 4 <= STAGES * STAGE_BYTES, "partial sums fit the stages");
};

template <int NT, typename TY>
__global__ void __launch_bounds__(NARROW_THREADS, 1)
fp8_mm_narrow_kernel(const __grid_constant__ CUtensorMap wmap,
                     const __grid_constant__ CUtensorMap xmap, const __grid_constant__ MmArgs a) {
    using S = NarrowShape<NT>;
    extern __shared__ __align__(1024) unsigned char mm_smem[];
    unsigned char *stages = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(mm_smem) + 1023) & ~uintptr_t(1023));
    float *scale_ring = reinterpret_cast<float *>(stages + S::STAGES * S::STAGE_BYTES);
    uint64_t *full = reinterpret_cast<uint64_t *>(scale_ring + MM_SCALE_SLOTS * S::SLOT);
    uint64_t *empty = full + S::STAGES;
    uint64_t *acc_full = empty + S::STAGES;
    uint64_t *acc_empty = acc_full + S::BUFS;
    uint64_t *s_full = acc_empty + S::BUFS;
    uint64_t *s_empty = s_full + MM_SCALE_SLOTS;
    uint64_t *mma_done = s_empty + MM_SCALE_SLOTS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = a.split > 1 ? (int)tc::cluster_rank() : 0;
    const int tile = (int)(blockIdx.x / (unsigned)a.split);
    const int tn = tile % a.tiles_n, tm = tile / a.tiles_n;
    const int n0 = tn * 128, m0 = tm * NT;
    const int b0 = (int)((long long)a.kb * part / a.split);
    const int nb = (int)((long long)a.kb * (part + 1) / a.split) - b0;  // this CTA's blocks

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < S::BUFS; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 4); }
        for (int i = 0; i < MM_SCALE_SLOTS; ++i) { mbar_init(&s_full[i], 32); mbar_init(&s_empty[i], 4); }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, S::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // the next kernel may start its own set-up now: this CTA holds its TMEM already
    pdl_launch_next();
    pdl_wait_prev();

    float acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = 0.f;

    if (warp == 0) {
        if (lane == 0) {
            for (int it = 0; it < nb; ++it) {
                const int st = it % S::STAGES;
                if (*abort_flag) break;
                if (!mbar_wait(&empty[st], (uint32_t)((it / S::STAGES) & 1) ^ 1u, a.wait_limit)) {
                    report(GPTQ_ERR_TIMEOUT, 11);
                    *abort_flag = 1;
                    break;
                }
                unsigned char *w = stages + st * S::STAGE_BYTES;
                mbar_expect_tx(&full[st], S::STAGE_BYTES);
                tma_load_2d(&wmap, &full[st], w, (b0 + it) * MM_BK, n0);
                tma_load_2d(&xmap, &full[st], w + S::W_BYTES, (b0 + it) * MM_BK, m0);
            }
            if (*abort_flag) {
                // copies in flight land within microseconds: before the shared memory goes away
                const long long t0 = clock64();
                while (clock64() - t0 < 2000000) { }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int it = 0; it < nb && !*abort_flag; ++it) {
                const int b = it % S::BUFS, st = it % S::STAGES;
                if (!mbar_wait(&acc_empty[b], (uint32_t)((it / S::BUFS) & 1) ^ 1u, a.wait_limit) ||
                    !mbar_wait(&full[st], (uint32_t)((it / S::STAGES) & 1), a.wait_limit)) {
                    report(GPTQ_ERR_TIMEOUT, 12);
                    *abort_flag = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t w = smem_u32(stages + st * S::STAGE_BYTES);
#pragma unroll
                for (int k = 0; k < MM_BK / 32; ++k)
                    mma_e4m3(tmem + (uint32_t)(b * NT), mm_desc(w + 32 * k),
                             mm_desc(w + S::W_BYTES + 32 * k), mm_idesc(128, NT), k > 0);
                mma_commit(&empty[st]);
                mma_commit(&acc_full[b]);
            }
            mma_commit(mma_done);
            mbar_wait(mma_done, 0, a.wait_limit);
        }
    } else if (warp == 6) {
        for (int it = 0; it < nb && !*abort_flag; ++it) {
            const int sl = it % MM_SCALE_SLOTS;
            if (!mbar_wait(&s_empty[sl], (uint32_t)((it / MM_SCALE_SLOTS) & 1) ^ 1u, a.wait_limit)) {
                if (lane == 0) report(GPTQ_ERR_TIMEOUT, 13);
                *abort_flag = 1;
                break;
            }
            float *d = scale_ring + sl * S::SLOT;
#pragma unroll
            for (int j = lane; j < NT; j += 32) {
                const bool on = m0 + j < a.m;
                cp_async4(d + j, a.sA + (on ? (long long)(m0 + j) * a.kb + b0 + it : 0), on);
            }
            if (lane == 0) cp_async4(d + NT, a.sB + (long long)tn * a.kb + b0 + it, true);
            cp_async_arrive(&s_full[sl]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        const int q = warp & 3;
        for (int it = 0; it < nb && !*abort_flag; ++it) {
            const int b = it % S::BUFS, sl = it % MM_SCALE_SLOTS;
            if (!mbar_wait(&s_full[sl], (uint32_t)((it / MM_SCALE_SLOTS) & 1), a.wait_limit) ||
                !mbar_wait(&acc_full[b], (uint32_t)((it / S::BUFS) & 1), a.wait_limit)) {
                if (lane == 0) report(GPTQ_ERR_TIMEOUT, 14);
                *abort_flag = 1;
                break;
            }
            __syncwarp();
            tc_fence_after();
            const float *d = scale_ring + sl * S::SLOT;
            const float sw = d[NT];
            const uint32_t t = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * NT);
#pragma unroll
            for (int c = 0; c < NT; c += 16) {
                uint32_t r[16];
                mm_ld16(t + c, r);
                mm_wait_ld16(r);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 s = *reinterpret_cast<const float4 *>(d + c + j);
                    acc[c + j] = fmaf(__uint_as_float(r[j]), s.x * sw, acc[c + j]);
                    acc[c + j + 1] = fmaf(__uint_as_float(r[j + 1]), s.y * sw, acc[c + j + 1]);
                    acc[c + j + 2] = fmaf(__uint_as_float(r[j + 2]), s.z * sw, acc[c + j + 2]);
                    acc[c + j + 3] = fmaf(__uint_as_float(r[j + 3]), s.w * sw, acc[c + j + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) { mbar_arrive(&acc_empty[b]); mbar_arrive(&s_empty[sl]); }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, S::TMEM);

    const bool adds = warp >= 2 && warp < 6;
    const int row = 32 * (warp & 3) + lane;  // of the weight tile
    TY *Y = static_cast<TY *>(a.Y);
    if (a.split == 1) {
        if (adds && n0 + row < a.n) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (m0 + j < a.m) Y[(long long)(m0 + j) * a.ldy + n0 + row] = narrow<TY>(acc[j]);
        }
        return;
    }
    // the stages are free: every copy was waited for and every MMA is done
    float *sum = reinterpret_cast<float *>(stages);
    if (adds) {
#pragma unroll
        for (int j = 0; j < NT; ++j) sum[j * 128 + row] = acc[j];
    }
    cluster_sync_all();
    for (int i = part * NARROW_THREADS + (int)threadIdx.x; i < NT * 128; i += a.split * NARROW_THREADS) {
        const int j = i >> 7, r = i & 127;
        float v[8];
#pragma unroll
        for (int p = 0; p < 8; ++p)
            v[p] = p < a.split ? ld_cluster_f32(tc::map_to_rank(sum + i, (uint32_t)p)) : 0.f;
        float t = v[0];
#pragma unroll
        for (int p = 1; p < 8; ++p)
            if (p < a.split) t += v[p];
        if (m0 + j < a.m && n0 + r < a.n) Y[(long long)(m0 + j) * a.ldy + n0 + r] = narrow<TY>(t);
    }
    cluster_sync_all();  // no CTA leaves while another still reads its sums
}

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------
inline bool mm_map(CUtensorMap *map, const void *p, long long rows, long long k, long long ld,
                   int box_rows) {
    tc::EncodeTiledFn enc = tc::encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {(cuuint32_t)MM_BK, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, typename TY>
inline int mm_narrow(const void *A, long long lda, const void *B, long long ldb, long long k,
                     MmArgs a, cudaStream_t s) {
    using S = NarrowShape<NT>;
    CUtensorMap wmap, xmap;
    if (!mm_map(&wmap, B, a.n, k, ldb, 128) || !mm_map(&xmap, A, a.m, k, lda, NT)) return GPTQ_ERR_CUDA;
    auto kernel = fp8_mm_narrow_kernel<NT, TY>;
    GPTQ_SMEM_LIMIT(kernel, S::SMEM);
    a.tiles_n = ceil_div(a.n, 128);
    const long long tiles = (long long)a.tiles_n * ceil_div(a.m, NT);
    // as many parts of K as fill the SMs, at most a portable cluster's eight
    long long split = device_sm_count() / tiles;
    if (split > 8) split = 8;
    if (split > a.kb) split = a.kb;
    if (split < 1) split = 1;
    a.split = (int)split;
    if (tiles * split > 0x7fffffffLL) return GPTQ_ERR_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(NARROW_THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, wmap, xmap, a);
    const int st = launch_status();
    return e == cudaSuccess ? st : GPTQ_ERR_CUDA;
}

template <typename TY>
inline int mm_type(const void *A, long long lda, const void *B, long long ldb, long long k, MmArgs a,
                   cudaStream_t s) {
    if (a.m <= 16) return mm_narrow<16, TY>(A, lda, B, ldb, k, a, s);
    if (a.m <= 32) return mm_narrow<32, TY>(A, lda, B, ldb, k, a, s);
    if (a.m <= 64) return mm_narrow<64, TY>(A, lda, B, ldb, k, a, s);
    return mm_narrow<128, TY>(A, lda, B, ldb, k, a, s);
}

inline int fp8_matmul(const void *A, long long lda, const float *sA, const void *B, long long ldb,
                      const float *sB, long long m, long long n, long long k, void *Y, int y_dtype,
                      long long ldy, cudaStream_t s) {
    if (k == 0) {
        const size_t b = (size_t)serve_dtype_bytes(y_dtype);
        return cudaMemset2DAsync(Y, (size_t)ldy * b, 0, (size_t)n * b, (size_t)m, s) == cudaSuccess
                   ? GPTQ_OK : GPTQ_ERR_CUDA;
    }
    MmArgs a;
    a.sA = sA;
    a.sB = sB;
    a.Y = Y;
    a.ldy = ldy;
    a.m = (int)m;
    a.n = (int)n;
    a.kb = (int)((k + MM_BK - 1) / MM_BK);
    a.tiles_n = a.split = 0;
    // a wait longer than ~2 s at the 1.9 GHz clock means a lost signal, not a slow kernel
    a.wait_limit = tc::env_ll("GPTQ_WAIT_LIMIT_CYCLES", 4000000000LL);
    switch (y_dtype) {
        case GPTQ_BF16: return mm_type<__nv_bfloat16>(A, lda, B, ldb, k, a, s);
        case GPTQ_F16: return mm_type<__half>(A, lda, B, ldb, k, a, s);
        default: return mm_type<float>(A, lda, B, ldb, k, a, s);
    }
}

}  // namespace serve
}  // namespace gptq
