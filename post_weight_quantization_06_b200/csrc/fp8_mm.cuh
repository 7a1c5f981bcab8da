// Product of two e4m3 matrices with block scales on the 5th-generation tensor cores
// (gptq_fp8_matmul):
//   Y[i][j] = sum_b sA[i][b] sB[j / 128][b] sum_{l in b} A[i][l] B[j][l],   blocks b of 128
//
// The scales change with every block of K, so a block's product (four tcgen05.mma of K = 32 into a
// fresh TMEM accumulator) is read back, scaled and added to fp32 sums in registers by the
// "promotion" warps while the next block's MMAs run into another accumulator.
#pragma once

#include <algorithm>
#include <type_traits>

#include "hessian_tc.cuh"
#include "serve_common.cuh"

namespace gptq {
namespace serve {

using tc::cluster_sync_all;
using tc::mbar_arrive;
using tc::mbar_expect_tx;
using tc::mbar_init;
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
// One lane of a converged warp. The producer's and the issuer's loops are run by whole warps, with
// this lane alone issuing: under `lane == 0` the compiler cannot keep descriptors and addresses
// in uniform registers, and an iteration of four MMAs took 900 cycles.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ bool mm_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for the phase with this parity, called by a whole warp. False, with the abort flag set, if
// `limit` cycles pass first (recorded with `site`) or another role gave up. The answer is the same in
// every lane: what follows are loops that a warp leaves together and instructions that want all its
// lanes.
__device__ __forceinline__ bool mm_wait(uint64_t *bar, uint32_t parity, long long limit,
                                        volatile int *abort_flag, int site) {
    const uint32_t addr = smem_u32(bar);
    if (__all_sync(0xffffffffu, mm_try(addr, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, mm_try(addr, parity))) {
        const bool late = clock64() - t0 > limit;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
            if (late) report(GPTQ_ERR_TIMEOUT, site);
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}
// The same for one lane, whose warp does not go by the answer and meets before anything that wants
// all its lanes (a vote in the pair kernel's promotion cost 3 %).
__device__ __forceinline__ bool mm_wait_lane(uint64_t *bar, uint32_t parity, long long limit,
                                             volatile int *abort_flag, int site) {
    const uint32_t addr = smem_u32(bar);
    if (mm_try(addr, parity)) return true;
    const long long t0 = clock64();
    while (!mm_try(addr, parity)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            report(GPTQ_ERR_TIMEOUT, site);
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}
// The issuer's last wait: all its MMAs are complete, after an abort too, before the TMEM is released.
__device__ __forceinline__ void mm_wait_mmas(uint64_t *mma_done, long long limit, volatile int *abort_flag,
                                             int site) {
    const uint32_t addr = smem_u32(mma_done);
    if (mm_try(addr, 0)) return;
    if (tc::mbar_wait(mma_done, 0, limit)) return;
    report(GPTQ_ERR_TIMEOUT, site);
    *abort_flag = 1;
}
// After an abort, once all roles have met: copies in flight land within microseconds, before the
// shared memory is used for something else or goes away. (The producer cannot say whether there are
// any: it may have left long before another role gave up.)
__device__ __forceinline__ void mm_drain(volatile int *abort_flag) {
    if (!*abort_flag) return;
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) { }
}
// Position in a ring of N with the parity of its current round.
template <int N>
struct Ring {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) { i = 0; phase ^= 1u; }
    }
};
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
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b),
                 "f"(c), "f"(d)
                 : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// acc (two fp32) += t * s, both halves
__device__ __forceinline__ void fma2(uint64_t &acc, uint32_t t0, uint32_t t1, uint64_t s2) {
    asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
        : "+l"(acc)
        : "r"(t0), "r"(t1), "l"(s2));
}
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ void mm_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
                 "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
                 "}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                       "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
                       "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                       "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                       "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
__device__ __forceinline__ void mm_wait_ld32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]),
          "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
          "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
          "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
          "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
          "+r"(r[31])::"memory");
}
// Four values of a row of Y from column col on, those before n.
template <typename TY>
__device__ __forceinline__ void store_y4(TY *y, int col, int n, float4 v) {
    const TY t[4] = {narrow<TY>(v.x), narrow<TY>(v.y), narrow<TY>(v.z), narrow<TY>(v.w)};
    if (col + 4 <= n) {
        if (sizeof(TY) == 4) *reinterpret_cast<uint4 *>(y) = *reinterpret_cast<const uint4 *>(t);
        else *reinterpret_cast<uint2 *>(y) = *reinterpret_cast<const uint2 *>(t);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < n) y[i] = t[i];
    }
}
// 32 rows x 128 bytes of shared memory in the 128-byte swizzle to Y at (x, y); one bulk group.
__device__ __forceinline__ void mm_store_2d(const CUtensorMap *map, const void *src, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(smem_u32(src)), "r"(x), "r"(y)
        : "memory");
}
// The same slice by ordinary stores, for rows of Y that TMA does not take (a pitch that is no
// multiple of 16 bytes): `rows` rows, `cols` columns from y on, one value a lane. (32-bit words,
// with the single 16-bit values that rows starting between two words need at their ends, took twice
// as long: 5000 x 3001 x 777 58 us to 32 us.)
template <typename TY>
__device__ __forceinline__ void store_slice(TY *y, long long ldy, const unsigned char *slice, int rows,
                                            int cols, int lane) {
    constexpr int AT_ONCE = 8;   // rows whose values are on their way from shared memory together
    constexpr int S = 4 / sizeof(TY);
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += AT_ONCE) {
        TY w[AT_ONCE][S];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)   // r0 is a multiple of 8: row r0 + i has swizzle i
#pragma unroll
            for (int h = 0; h < S; ++h) {
                const int at = (lane + 32 * h) * (int)sizeof(TY);
                w[i][h] = *reinterpret_cast<const TY *>(slice + (r0 + i) * 128 + (at ^ (i << 4)));
            }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i, y += ldy)
#pragma unroll
            for (int h = 0; h < S; ++h)
                if (r0 + i < rows && lane + 32 * h < cols) y[lane + 32 * h] = w[i][h];
    }
}

struct MmArgs {
    const float *sA, *sB;
    void *Y;
    long long ldy;
    int m, n, kb;            // kb: blocks of K
    int nb128;               // blocks of 128 columns of Y
    int tiles_m, tiles_n;
    int split;               // CTAs of a cluster, each with a part of the K blocks
    int vec, vec16;          // four values can be stored at once; TMA takes the rows of Y
    int stall_at, stall_n;   // test hook: barriers whose phases want one arrival too many
    long long wait_limit;
};

// ---------------------------------------------------------------------------------------
// Few rows of A (decode): the weights' rows are the MMA's 128 rows and NT tokens its columns, so
// a tile costs only the weight's bytes. The blocks of K are split over the `split` CTAs of a
// cluster; each sends its sums to the CTA that owns the token, which adds them in the order of
// the parts. (64 rows a CTA, to split less, took as long or longer at every size tried.) Bytes of
// the weight should bound it; at one token what a launch costs from its set-up to the exchange in
// the cluster does: 1 x 2048 x 6144 in 5.2 us with the weight in the L2, 6.2 us from DRAM (2.0 TB/s; an empty launch of
// this shape 3 us), 1 x 8192 x 8192 in 12 and 15 us (4.4 TB/s).
//
// Warps: 0 TMA, 1 TMEM and MMA, 2-5 promotion (32 weight rows each), 6 scales.
// ---------------------------------------------------------------------------------------
constexpr int NARROW_THREADS = 224;

template <int NT>
struct NarrowShape {
    static constexpr int W_BYTES = 128 * MM_BK;
    static constexpr int STAGE_BYTES = W_BYTES + NT * MM_BK;
    static constexpr int STAGES = NT <= 16 ? 10 : 8;
    static constexpr int SLOT = NT + 4;   // scales of NT tokens, then the weight tile's
    static constexpr int BUFS = 4;
    static constexpr int TMEM = NT * BUFS;
    static constexpr int BARS = 2 * STAGES + 2 * BUFS + 2 * MM_SCALE_SLOTS + 1;
    static constexpr int RED = (NT + 7) * 128;   // floats received from the cluster
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + sizeof(float) * RED +
                                   sizeof(float) * MM_SCALE_SLOTS * SLOT + 8 * BARS + 64;
    static_assert(SMEM <= 232448, "fits the shared memory of one CTA");
    static_assert((TMEM & (TMEM - 1)) == 0 && TMEM >= 32 && TMEM <= 512, "a TMEM allocation");
};

template <int NT, typename TY>
__global__ void __launch_bounds__(NARROW_THREADS, 1)
fp8_mm_narrow_kernel(const __grid_constant__ CUtensorMap wmap,
                     const __grid_constant__ CUtensorMap xmap, const __grid_constant__ MmArgs a) {
    using S = NarrowShape<NT>;
    extern __shared__ __align__(1024) unsigned char mm_smem[];
    unsigned char *stages = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(mm_smem) + 1023) & ~uintptr_t(1023));
    float *red = reinterpret_cast<float *>(stages + S::STAGES * S::STAGE_BYTES);
    float *scale_ring = red + S::RED;
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

    if (warp == 0) {
        for (int i = lane; i < S::BARS; i += 32) {
            uint64_t *b = full + i;
            const uint32_t count = (b >= acc_empty && b < s_full) || (b >= s_empty && b < mma_done)
                                       ? 4u
                                       : (b >= s_full && b < s_empty) ? 32u : 1u;
            mbar_init(b, count + ((unsigned)(i - a.stall_at) < (unsigned)a.stall_n));
        }
        if (lane == 0) *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
    } else if (warp == 1) {
        tmem_alloc(tmem_slot, S::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the CTAs of a cluster have to be there before one writes to another (waited for below)
    if (a.split > 1) cluster_arrive();
    const uint32_t tmem = *tmem_slot;
    // the next kernel may start its own set-up now: this CTA holds its TMEM already
    pdl_launch_next();
    pdl_wait_prev();

    float acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = 0.f;

    if (warp == 0) {
        const bool one = elect_one();
        Ring<S::STAGES> st;
        for (int it = 0; it < nb; ++it, st.next()) {
            if (!mm_wait(&empty[st.i], st.phase ^ 1u, a.wait_limit, abort_flag, 11)) break;
            if (one) {
                unsigned char *w = stages + st.i * S::STAGE_BYTES;
                mbar_expect_tx(&full[st.i], S::STAGE_BYTES);
                tma_load_2d(&wmap, &full[st.i], w, (b0 + it) * MM_BK, n0);
                tma_load_2d(&xmap, &full[st.i], w + S::W_BYTES, (b0 + it) * MM_BK, m0);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        const bool one = elect_one();
        Ring<S::STAGES> st;
        Ring<S::BUFS> b;
        for (int it = 0; it < nb; ++it, st.next(), b.next()) {
            if (!mm_wait(&acc_empty[b.i], b.phase ^ 1u, a.wait_limit, abort_flag, 12) ||
                !mm_wait(&full[st.i], st.phase, a.wait_limit, abort_flag, 13))
                break;
            tc_fence_after();
            if (one) {
                const uint32_t w = smem_u32(stages + st.i * S::STAGE_BYTES);
                const uint64_t wd = mm_desc(w), xd = mm_desc(w + S::W_BYTES);
#pragma unroll
                for (int k = 0; k < MM_BK / 32; ++k)   // 32 codes: 32 bytes further, in units of 16
                    mma_e4m3(tmem + (uint32_t)(b.i * NT), wd + 2 * k, xd + 2 * k, mm_idesc(128, NT),
                             k > 0);
                mma_commit(&empty[st.i]);
                mma_commit(&acc_full[b.i]);
            }
            __syncwarp();
        }
        if (one) mma_commit(mma_done);
        mm_wait_mmas(mma_done, a.wait_limit, abort_flag, 14);
    } else if (warp == 6) {
        Ring<MM_SCALE_SLOTS> sl;
        const float *sw = a.sB + (long long)tn * a.kb + b0;
        for (int it = 0; it < nb; ++it, sl.next()) {
            if (!mm_wait(&s_empty[sl.i], sl.phase ^ 1u, a.wait_limit, abort_flag, 15)) break;
            float *d = scale_ring + sl.i * S::SLOT;
#pragma unroll
            for (int j = lane; j < NT; j += 32) {
                const bool on = m0 + j < a.m;
                cp_async4(d + j, a.sA + (on ? (long long)(m0 + j) * a.kb + b0 + it : 0), on);
            }
            if (lane == 0) cp_async4(d + NT, sw + it, true);
            cp_async_arrive(&s_full[sl.i]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        const int q = warp & 3;
        Ring<MM_SCALE_SLOTS> sl;
        Ring<S::BUFS> b;
        for (int it = 0; it < nb; ++it, sl.next(), b.next()) {
            if (!mm_wait(&s_full[sl.i], sl.phase, a.wait_limit, abort_flag, 16) ||
                !mm_wait(&acc_full[b.i], b.phase, a.wait_limit, abort_flag, 17))
                break;
            __syncwarp();
            tc_fence_after();
            const float *d = scale_ring + sl.i * S::SLOT;
            const float sw = d[NT];
            const uint32_t t = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b.i * NT);
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
            if (lane == 0) { mbar_arrive(&acc_empty[b.i]); mbar_arrive(&s_empty[sl.i]); }
        }
    }
    __syncwarp();

    const bool adds = warp >= 2 && warp < 6;
    const int row = 32 * (warp & 3) + lane;  // of the weight tile
    const int mt = a.m - m0 < NT ? a.m - m0 : NT;
    TY *Y = static_cast<TY *>(a.Y) + (long long)m0 * a.ldy + n0;
    if (a.split == 1) {
        if (adds && n0 + row < a.n) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (j < mt) Y[(long long)j * a.ldy + row] = narrow<TY>(acc[j]);
        }
    } else {
        const int own = (NT + a.split - 1) / a.split;   // tokens of a CTA, at most
        cluster_wait();
        if (adds) {
            int dst = 0, at = part * own;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j < mt) st_cluster(tc::map_to_rank(red + at * 128 + row, (uint32_t)dst), acc[j]);
                if (++dst == a.split) { dst = 0; ++at; }
            }
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        // token part + split * l, the parts in order
        for (int i = threadIdx.x; i < own * 128; i += NARROW_THREADS) {
            const int j = part + a.split * (i >> 7), r = i & 127;
            if (j >= mt || n0 + r >= a.n) continue;
            float t = red[i];
            for (int p = 1; p < a.split; ++p) t += red[p * own * 128 + i];
            Y[(long long)j * a.ldy + r] = narrow<TY>(t);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    mm_drain(abort_flag);
    if (warp == 1) tmem_dealloc(tmem, S::TMEM);
}

// ---------------------------------------------------------------------------------------
// More rows of A than a decode batch, too few tiles for the pair kernel: 128 x 128 tiles of Y,
// one CTA each, the rows of A on the TMEM lanes, so that a promotion thread has one row and its
// scale is one number per block. The blocks of K can be split over a cluster as above. A block takes
// about 400 cycles of promotion (256 of MMAs), a launch 3 us and the rows of Y 1.5 us: 777 x 1500 x 2900
// in 12 us, 64 x 6144 x 2048 in 9 us.
//
// Warps: 0 TMA, 1 TMEM and MMA, 2 scales, 4-11 promotion (32 rows x 64 columns each).
// ---------------------------------------------------------------------------------------
constexpr int TILE_THREADS = 384;
constexpr int TILE_STAGES = 6;
constexpr int TILE_STAGE_BYTES = 2 * 128 * MM_BK;
constexpr int TILE_BUFS = 4;
constexpr int TILE_SLOT = 128 + 4;
constexpr int TILE_BARS = 2 * TILE_STAGES + 2 * TILE_BUFS + 2 * MM_SCALE_SLOTS + 1;
constexpr int TILE_PITCH = 132;   // floats of a row of sums in shared memory: no bank conflicts
constexpr size_t TILE_SMEM = 1024 + (size_t)TILE_STAGES * TILE_STAGE_BYTES +
                             sizeof(float) * MM_SCALE_SLOTS * TILE_SLOT + 8 * TILE_BARS + 64;
static_assert(TILE_SMEM <= 232448, "fits the shared memory of one CTA");
static_assert((128 + 7) * TILE_PITCH * 4 <= TILE_STAGES * TILE_STAGE_BYTES, "sums fit the stages");

template <typename TY>
__global__ void __launch_bounds__(TILE_THREADS, 1)
fp8_mm_tile_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ MmArgs a) {
    extern __shared__ __align__(1024) unsigned char mm_smem[];
    unsigned char *stages = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(mm_smem) + 1023) & ~uintptr_t(1023));
    float *scale_ring = reinterpret_cast<float *>(stages + TILE_STAGES * TILE_STAGE_BYTES);
    uint64_t *full = reinterpret_cast<uint64_t *>(scale_ring + MM_SCALE_SLOTS * TILE_SLOT);
    uint64_t *empty = full + TILE_STAGES;
    uint64_t *acc_full = empty + TILE_STAGES;
    uint64_t *acc_empty = acc_full + TILE_BUFS;
    uint64_t *s_full = acc_empty + TILE_BUFS;
    uint64_t *s_empty = s_full + MM_SCALE_SLOTS;
    uint64_t *mma_done = s_empty + MM_SCALE_SLOTS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = a.split > 1 ? (int)tc::cluster_rank() : 0;
    const int tile = (int)(blockIdx.x / (unsigned)a.split);
    const int tn = tile % a.tiles_n, tm = tile / a.tiles_n;
    const int n0 = tn * 128, m0 = tm * 128;
    const int b0 = (int)((long long)a.kb * part / a.split);
    const int nb = (int)((long long)a.kb * (part + 1) / a.split) - b0;

    if (warp == 0) {
        for (int i = lane; i < TILE_BARS; i += 32) {
            uint64_t *b = full + i;
            const uint32_t count = (b >= acc_empty && b < s_full) || (b >= s_empty && b < mma_done)
                                       ? 8u : (b >= s_full && b < s_empty) ? 32u : 1u;
            mbar_init(b, count + ((unsigned)(i - a.stall_at) < (unsigned)a.stall_n));
        }
        if (lane == 0) *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
    } else if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_next();
    pdl_wait_prev();

    uint64_t acc[32];   // 64 columns of one row, in pairs
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = 0;

    if (warp == 0) {
        const bool one = elect_one();
        Ring<TILE_STAGES> st;
        for (int it = 0; it < nb; ++it, st.next()) {
            if (!mm_wait(&empty[st.i], st.phase ^ 1u, a.wait_limit, abort_flag, 21)) break;
            if (one) {
                unsigned char *sa = stages + st.i * TILE_STAGE_BYTES;
                mbar_expect_tx(&full[st.i], TILE_STAGE_BYTES);
                tma_load_2d(&amap, &full[st.i], sa, (b0 + it) * MM_BK, m0);
                tma_load_2d(&bmap, &full[st.i], sa + 128 * MM_BK, (b0 + it) * MM_BK, n0);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        const bool one = elect_one();
        Ring<TILE_STAGES> st;
        Ring<TILE_BUFS> b;
        for (int it = 0; it < nb; ++it, st.next(), b.next()) {
            if (!mm_wait(&acc_empty[b.i], b.phase ^ 1u, a.wait_limit, abort_flag, 22) ||
                !mm_wait(&full[st.i], st.phase, a.wait_limit, abort_flag, 23))
                break;
            tc_fence_after();
            if (one) {
                const uint32_t w = smem_u32(stages + st.i * TILE_STAGE_BYTES);
                const uint64_t ad = mm_desc(w), bd = mm_desc(w + 128 * MM_BK);
#pragma unroll
                for (int k = 0; k < MM_BK / 32; ++k)
                    mma_e4m3(tmem + (uint32_t)(b.i * 128), ad + 2 * k, bd + 2 * k,
                             mm_idesc(128, 128), k > 0);
                mma_commit(&empty[st.i]);
                mma_commit(&acc_full[b.i]);
            }
            __syncwarp();
        }
        if (one) mma_commit(mma_done);
        mm_wait_mmas(mma_done, a.wait_limit, abort_flag, 24);
    } else if (warp == 2) {
        Ring<MM_SCALE_SLOTS> sl;
        for (int it = 0; it < nb; ++it, sl.next()) {
            if (!mm_wait(&s_empty[sl.i], sl.phase ^ 1u, a.wait_limit, abort_flag, 25)) break;
            float *d = scale_ring + sl.i * TILE_SLOT;
#pragma unroll
            for (int j = lane; j < 128; j += 32) {
                const bool on = m0 + j < a.m;
                cp_async4(d + j, a.sA + (on ? (long long)(m0 + j) * a.kb + b0 + it : 0), on);
            }
            if (lane == 0) cp_async4(d + 128, a.sB + (long long)tn * a.kb + b0 + it, true);
            cp_async_arrive(&s_full[sl.i]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4) {
        const int q = warp & 3, h = (warp - 4) >> 2;
        Ring<MM_SCALE_SLOTS> sl;
        Ring<TILE_BUFS> b;
        for (int it = 0; it < nb; ++it, sl.next(), b.next()) {
            if (!mm_wait(&s_full[sl.i], sl.phase, a.wait_limit, abort_flag, 26) ||
                !mm_wait(&acc_full[b.i], b.phase, a.wait_limit, abort_flag, 27))
                break;
            __syncwarp();
            tc_fence_after();
            const float *d = scale_ring + sl.i * TILE_SLOT;
            const float s = d[32 * q + lane] * d[128];
            const uint64_t s2 = pair_of(s, s);
            const uint32_t t = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b.i * 128 + 64 * h);
            uint32_t r0[32], r1[32];
            mm_ld32(t, r0);
            mm_ld32(t + 32, r1);
            mm_wait_ld32(r0);
            mm_wait_ld32(r1);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) { mbar_arrive(&acc_empty[b.i]); mbar_arrive(&s_empty[sl.i]); }
#pragma unroll
            for (int j = 0; j < 16; ++j) fma2(acc[j], r0[2 * j], r0[2 * j + 1], s2);
#pragma unroll
            for (int j = 0; j < 16; ++j) fma2(acc[16 + j], r1[2 * j], r1[2 * j + 1], s2);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    mm_drain(abort_flag);
    if (warp == 1) tmem_dealloc(tmem, 512);

    // Sums by row through shared memory (the stages are free: every copy was waited for or drained and
    // every MMA is done), then whole rows to Y. Row i belongs to CTA i % split of the cluster.
    float *sum = reinterpret_cast<float *>(stages);
    const int own = (128 + a.split - 1) / a.split;
    if (a.split > 1) cluster_sync_all();
    if (warp >= 4) {
        const int i = 32 * (warp & 3) + lane, h = (warp - 4) >> 2;
        float *d = sum + ((long long)part * own + i / a.split) * TILE_PITCH + 64 * h;
        if (a.split > 1) {
            const uint32_t to = tc::map_to_rank(d, (uint32_t)(i % a.split));
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float2 u = unpair(acc[j]), v = unpair(acc[j + 1]);
                st_cluster4(to + 8 * j, u.x, u.y, v.x, v.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float2 u = unpair(acc[j]), v = unpair(acc[j + 1]);
                *reinterpret_cast<float4 *>(d + 2 * j) = make_float4(u.x, u.y, v.x, v.y);
            }
        }
    }
    if (a.split > 1) cluster_sync_all();
    else __syncthreads();
    for (int l = warp; l < own; l += TILE_THREADS / 32) {
        const int i = part + a.split * l;
        if (i >= 128 || m0 + i >= a.m) continue;
        const float *d = sum + (long long)l * TILE_PITCH;
        TY *y = static_cast<TY *>(a.Y) + (long long)(m0 + i) * a.ldy + n0;
        if (a.vec) {   // four columns a lane
            const int c = 4 * lane;
            float4 v = *reinterpret_cast<const float4 *>(d + c);
            for (int p = 1; p < a.split; ++p) {
                const float4 w = *reinterpret_cast<const float4 *>(d + (long long)p * own * TILE_PITCH + c);
                v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
            }
            store_y4(y + c, n0 + c, a.n, v);
        } else {       // rows that are not aligned: neighbouring lanes store neighbouring columns
#pragma unroll
            for (int c = lane; c < 128; c += 32) {
                float v = d[c];
                for (int p = 1; p < a.split; ++p) v += d[(long long)p * own * TILE_PITCH + c];
                if (n0 + c < a.n) y[c] = narrow<TY>(v);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------
// Many rows: 256 x 256 tiles of Y by a CTA pair (tcgen05 cta_group::2), persistent. CTA r holds
// rows 128 r .. of the pair's A and B; the leader's 256 x 256 x 32 MMAs read both CTAs' shared
// memory and leave rows 128 r .. of the tile in CTA r's TMEM. A block of K takes the tensor cores
// 512 cycles; in that time a promotion thread reads 128 columns of its row from one of two
// accumulators and adds them to 128 sums in registers (setmaxnreg: 232 for the promotion warps,
// 40 for the others, together the 168 x 384 of the launch). A warp of its own brings the scales to
// shared memory, four blocks at a time and up to sixteen ahead; loaded by the promotion threads
// themselves, four blocks ahead, they cost 5 % with 48 blocks a tile and 15 % with three, where a
// tile's first scales were waited for. Their ring takes the place of a fifth stage of A and B.
//
// With two accumulators (all of TMEM) what bounds a block is the way from its last MMA to the
// release of its accumulator, about 840 cycles, then the 1000 W power limit. One CTA per
// 128 x 256 tile has the shorter way (its commits and arrivals stay on the SM) but moves half as
// much again; on random data it was 6 % slower. Accumulators of 128 columns, four of them, were
// slower still: every wait and arrival doubles; so were sixteen promotion warps of 64 columns.
// 16384 x 2048 x 6144 in 174 us (2370 TFLOP/s, tensor pipe busy 62 % of the time), 204 us in a loop
// that heats the card to its limit.
//
// Warps: 0 TMA, 1 TMEM and (leader) MMA, 2 scales, 4-11 promotion (32 rows x 128 columns each). A
// tile's sums are rounded into shared memory and leave by TMA while the next tile runs.
// ---------------------------------------------------------------------------------------
constexpr int PAIR_THREADS = 384;
constexpr int PAIR_STAGES = 4;
constexpr int PAIR_A_BYTES = 128 * MM_BK;
constexpr int PAIR_STAGE_BYTES = 2 * 128 * MM_BK;   // this CTA's halves of A and B
constexpr int PAIR_GROUPS = 4;                      // ring of scales, four blocks each
constexpr int PAIR_SCALES = 130;                    // float4: 128 rows, two blocks of columns
constexpr int PAIR_BARS = 2 * PAIR_STAGES + 4 + 2 * PAIR_GROUPS + 1;
constexpr int PAIR_SLICE = 32 * 128;                // 128 bytes of 32 rows, 128-byte swizzle
constexpr int PAIR_OUT = 8 * 2 * PAIR_SLICE;        // two slices per promotion warp
constexpr size_t PAIR_SMEM = 1024 + (size_t)PAIR_STAGES * PAIR_STAGE_BYTES + PAIR_OUT +
                             sizeof(float4) * PAIR_GROUPS * PAIR_SCALES + 8 * PAIR_BARS + 64;
static_assert(PAIR_SMEM <= 232448, "fits the shared memory of one CTA");
constexpr int PAIR_GROUP = 8;   // tile rows that are walked together, column by column

// Tile t in groups of PAIR_GROUP tile rows, so that the tiles in flight share rows and columns
// that the L2 holds.
__device__ __forceinline__ void pair_tile(const MmArgs &a, int t, int &tm, int &tn) {
    const int per = PAIR_GROUP * a.tiles_n, g = t / per, r = t - g * per;
    const int h = min(PAIR_GROUP, a.tiles_m - g * PAIR_GROUP);
    tn = r / h;
    tm = g * PAIR_GROUP + (r - tn * h);
}

__device__ __forceinline__ void mma_e4m3_pair(uint32_t dtmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtmem),
        "l"(adesc), "l"(bdesc), "r"(mm_idesc(256, 256)), "r"(accumulate));
}
// Arrival on a barrier of the pair's leader. What it orders are TMEM loads that have completed
// (tcgen05.wait::ld), so the default scope will do: a release at cluster scope fences the thread's
// memory first and cost the promotion a thousand cycles a block.
__device__ __forceinline__ void mm_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The scales of up to four blocks of a row, `left` of them there, to shared memory.
__device__ __forceinline__ void load_scales(float4 *d, const float *src, int left, bool vec) {
    if (vec) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(d)), "l"(src) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async4(reinterpret_cast<float *>(d) + i, src + (i < left ? i : 0), i < left);
    }
}

// acc += s * the 128 columns at taddr, 32 at a time, the next 32 on their way meanwhile; the
// accumulator is released when the last have arrived.
__device__ __forceinline__ void pair_promote(uint32_t taddr, float s, float (&acc)[128],
                                             uint32_t release, int lane) {
    uint32_t r0[32], r1[32];
    __syncwarp();
    tc_fence_after();
    mm_ld32(taddr, r0);
    mm_wait_ld32(r0);
    mm_ld32(taddr + 32, r1);
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(r0[j]), s, acc[j]);
    mm_wait_ld32(r1);
    mm_ld32(taddr + 64, r0);
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[32 + j] = fmaf(__uint_as_float(r1[j]), s, acc[32 + j]);
    mm_wait_ld32(r0);
    mm_ld32(taddr + 96, r1);
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[64 + j] = fmaf(__uint_as_float(r0[j]), s, acc[64 + j]);
    mm_wait_ld32(r1);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mm_arrive_remote(release);
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[96 + j] = fmaf(__uint_as_float(r1[j]), s, acc[96 + j]);
}

template <typename TY>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
fp8_mm_pair_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ CUtensorMap ymap, const __grid_constant__ MmArgs a) {
    extern __shared__ __align__(1024) unsigned char mm_smem[];
    unsigned char *stages = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(mm_smem) + 1023) & ~uintptr_t(1023));
    unsigned char *out = stages + PAIR_STAGES * PAIR_STAGE_BYTES;
    float4 *scales = reinterpret_cast<float4 *>(out + PAIR_OUT);
    uint64_t *full = reinterpret_cast<uint64_t *>(scales + PAIR_GROUPS * PAIR_SCALES);
    uint64_t *empty = full + PAIR_STAGES;
    uint64_t *acc_full = empty + PAIR_STAGES;   // 2
    uint64_t *acc_empty = acc_full + 2;         // 2
    uint64_t *s_full = acc_empty + 2;
    uint64_t *s_empty = s_full + PAIR_GROUPS;
    uint64_t *mma_done = s_empty + PAIR_GROUPS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = a.tiles_m * a.tiles_n;
    const uint32_t rank = tc::cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (warp == 0) {
        for (int i = lane; i < PAIR_BARS; i += 32) {
            uint64_t *b = full + i;
            const uint32_t count = b >= acc_empty && b < s_full ? 16u
                                   : b >= s_empty && b < mma_done ? 8u
                                   : b >= s_full && b < s_empty ? 32u : 1u;
            mbar_init(b, count + ((unsigned)(i - a.stall_at) < (unsigned)a.stall_n));
        }
        if (lane == 0) *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
    } else if (warp == 1) {
        tc::tmem_alloc_pair(tmem_slot, 512);
        tc::tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any remote arrive or TMA
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_next();
    pdl_wait_prev();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            const bool one = elect_one();
            Ring<PAIR_STAGES> st;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int tm, tn;
                pair_tile(a, t, tm, tn);
                for (int kb = 0; kb < a.kb; ++kb, st.next()) {
                    ok = mm_wait(&empty[st.i], st.phase ^ 1u, a.wait_limit, abort_flag, 31);
                    if (!ok) break;
                    if (one) {
                        unsigned char *sa = stages + st.i * PAIR_STAGE_BYTES;
                        // the leader's barrier counts both CTAs' bytes
                        if (rank == 0) mbar_expect_tx(&full[st.i], 2 * PAIR_STAGE_BYTES);
                        const uint32_t fb = tc::map_to_rank(&full[st.i], 0);
                        const int r0 = 128 * (int)rank;
                        tc::tma_load_2d_pair(&amap, fb, sa, kb * MM_BK, tm * 256 + r0);
                        tc::tma_load_2d_pair(&bmap, fb, sa + PAIR_A_BYTES, kb * MM_BK, tn * 256 + r0);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 1 && rank == 0) {
            const bool one = elect_one();
            Ring<PAIR_STAGES> st;
            Ring<2> b;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                for (int kb = 0; kb < a.kb; ++kb, st.next(), b.next()) {
                    ok = mm_wait(&full[st.i], st.phase, a.wait_limit, abort_flag, 32) &&
                         mm_wait(&acc_empty[b.i], b.phase ^ 1u, a.wait_limit, abort_flag, 33);
                    if (!ok) break;
                    tc_fence_after();
                    if (one) {
                        const uint32_t w = smem_u32(stages + st.i * PAIR_STAGE_BYTES);
                        const uint64_t ad = mm_desc(w), bd = mm_desc(w + PAIR_A_BYTES);
#pragma unroll
                        for (int k = 0; k < MM_BK / 32; ++k)
                            mma_e4m3_pair(tmem + (uint32_t)(b.i * 256), ad + 2 * k, bd + 2 * k, k > 0);
                        tc::mma_commit_pair(&acc_full[b.i], 0x3);
                        tc::mma_commit_pair(&empty[st.i], 0x3);
                    }
                    __syncwarp();
                }
            }
            // all MMAs complete before the TMEM is released
            if (one) tc::mma_commit_pair(mma_done, 0x1);
            mm_wait_mmas(mma_done, a.wait_limit, abort_flag, 34);
        } else if (warp == 2) {
            Ring<PAIR_GROUPS> sl;
            bool ok = true;
            const bool vec = (a.kb & 3) == 0 &&
                             ((reinterpret_cast<uintptr_t>(a.sA) | reinterpret_cast<uintptr_t>(a.sB)) & 15u) == 0;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int tm, tn;
                pair_tile(a, t, tm, tn);
                const int m0 = tm * 256 + 128 * (int)rank;
                for (int kb = 0; kb < a.kb; kb += 4, sl.next()) {
                    ok = mm_wait(&s_empty[sl.i], sl.phase ^ 1u, a.wait_limit, abort_flag, 36);
                    if (!ok) break;
                    float4 *d = scales + sl.i * PAIR_SCALES;
                    // rows and columns behind the last take its scales: what they scale is not stored
#pragma unroll
                    for (int j = 0; j < 128; j += 32)
                        load_scales(d + j + lane, a.sA + (long long)min(m0 + j + lane, a.m - 1) * a.kb + kb,
                                    a.kb - kb, vec);
                    if (lane < 2)
                        load_scales(d + 128 + lane, a.sB + (long long)min(2 * tn + lane, a.nb128 - 1) * a.kb + kb,
                                    a.kb - kb, vec);
                    cp_async_arrive(&s_full[sl.i]);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int q = warp & 3, h = (warp - 4) >> 2;
        unsigned char *slices = out + (warp - 4) * 2 * PAIR_SLICE;
        int turn = 0;
        const uint32_t release = tc::map_to_rank(acc_empty, 0);
        uint32_t n = 0;   // blocks so far: accumulator n & 1
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(128 * h);
        Ring<PAIR_GROUPS> sl;
        for (int t = pair; t < tiles; t += pairs) {
            int tm, tn;
            pair_tile(a, t, tm, tn);
            const int m0 = tm * 256 + 128 * (int)rank + 32 * q, n0 = tn * 256 + 128 * h;
            float acc[128];   // 128 columns of one row
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
#pragma unroll 1
            for (int kb = 0; kb < a.kb; kb += 4) {
                mm_wait_lane(&s_full[sl.i], sl.phase, a.wait_limit, abort_flag, 37);
                float4 sc = scales[sl.i * PAIR_SCALES + 32 * q + lane];
                const float4 sb = scales[sl.i * PAIR_SCALES + 128 + h];
                sc.x *= sb.x; sc.y *= sb.y; sc.z *= sb.z; sc.w *= sb.w;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[sl.i]);
                sl.next();
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (u > 0 && kb + u >= a.kb) break;
                    // no way out after an abort (its later waits return at once): a branch that
                    // leaves the loop made the compiler move the 128 sums about
                    mm_wait_lane(&acc_full[n & 1], (n >> 1) & 1, a.wait_limit, abort_flag, 35);
                    pair_promote(tq + (n & 1) * 256, u == 0 ? sc.x : u == 1 ? sc.y : u == 2 ? sc.z : sc.w,
                                 acc, release + 8 * (n & 1), lane);
                    ++n;
                }
            }
            // 128 bytes of a row at a time: rounded, written to a slice, and on their way
            constexpr int E = 16 / sizeof(TY), C = 8 * E;   // values of 16 and of 128 bytes
#pragma unroll
            for (int c = 0; c < 128 / C; ++c) {
                if (n0 + C * c >= a.n || m0 >= a.m) continue;   // the same in the whole warp
                // the slices take turns: the last TMA store but one, from this one, has read it
                unsigned char *slice = slices + (turn & 1) * PAIR_SLICE;
                // TMA stores whole 16-byte pieces, the last of a row too: past the columns
                const bool tma = a.vec16 && (n0 + C * c + C <= a.n || a.n % E == 0);
                if (a.vec16 && lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    TY v[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] = narrow<TY>(acc[C * c + E * j + e]);
                    *reinterpret_cast<uint4 *>(slice + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                        *reinterpret_cast<const uint4 *>(v);
                }
                if (tma) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mm_store_2d(&ymap, slice, n0 + C * c, m0);
                    ++turn;
                } else {
                    __syncwarp();
                    store_slice(static_cast<TY *>(a.Y) + (long long)m0 * a.ldy + n0 + C * c, a.ldy, slice,
                                min(32, a.m - m0), a.n - n0 - C * c, lane);
                    __syncwarp();
                }
            }
        }
        if (a.vec16 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    mm_drain(abort_flag);
    cluster_sync_all();  // the peer's TMEM, barriers and shared memory outlive every access
    tc_fence_after();
    if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
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

// Y in boxes of 32 rows x 128 bytes.
template <typename TY>
inline bool mm_out_map(CUtensorMap *map, const MmArgs &a) {
    tc::EncodeTiledFn enc = tc::encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)a.n, (cuuint64_t)a.m};
    const cuuint64_t strides[1] = {(cuuint64_t)a.ldy * sizeof(TY)};
    const cuuint32_t box[2] = {128 / sizeof(TY), 32};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType t = std::is_same<TY, float>::value    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : std::is_same<TY, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return enc(map, t, 2, a.Y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... P, typename... V>
inline int mm_launch(void (*kernel)(P...), long long ctas, int cluster, int threads, size_t smem,
                     cudaStream_t s, const V &...args) {
    if (ctas > 0x7fffffffLL) return GPTQ_ERR_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    const int st = launch_status();
    return e == cudaSuccess ? st : GPTQ_ERR_CUDA;
}

// CTAs with an SM's shared memory that run at once in clusters of `size`: from the occupancy call
// on a B200 of 148 SMs, whose clusters do not cross the borders of its SM groups (larger clusters
// leave SMs idle: seven, 105), and in proportion for other counts. It only chooses the parts of K.
inline int mm_resident(int size) {
    static const int on148[9] = {0, 148, 148, 135, 132, 130, 132, 105, 120};
    return on148[size] * device_sm_count() / 148;
}
// Parts of K for `tiles` tiles: the least cost, rounds of CTAs x (blocks of a CTA and what a round
// costs besides) and what adding the parts up costs; all in blocks of a CTA.
inline int mm_split(long long tiles, int kb, int round, int add, long long &cost) {
    int best = 1;
    cost = -1;
    for (int s = 1; s <= 8 && s <= kb; ++s) {
        const int at_once = mm_resident(s) / s * s;
        if (at_once < s) continue;
        const long long c = (tiles * s + at_once - 1) / at_once * ((kb + s - 1) / s + round) + (s > 1 ? add : 0);
        if (cost < 0 || c < cost) { cost = c; best = s; }
    }
    return best;
}

// Test hook: kind `a.stall_n` of barrier (1 accumulator full, 2 stage full, 3 stage empty, 4 scales full,
// 5 accumulator empty; 0 none) as the range of a kernel's barriers, which lie in this order: stages full and
// empty, accumulators full and empty, scales full and empty.
inline void mm_stall(MmArgs &a, int stages, int bufs, int slots) {
    const int at[6] = {0, 2 * stages, 0, stages, 2 * stages + 2 * bufs, 2 * stages + bufs};
    const int n[6] = {0, bufs, stages, stages, slots, bufs};
    const int kind = a.stall_n > 0 && a.stall_n < 6 ? a.stall_n : 0;
    a.stall_at = at[kind];
    a.stall_n = n[kind];
}

template <int NT, typename TY>
inline int mm_narrow(const void *A, long long lda, const void *B, long long ldb, long long k,
                     MmArgs a, cudaStream_t s) {
    using S = NarrowShape<NT>;
    a.tiles_m = ceil_div(a.m, NT);
    a.tiles_n = ceil_div(a.n, 128);
    long long cost;   // a block 0.24 us, a round 3 us, the sum over the cluster 0.5 us
    a.split = mm_split((long long)a.tiles_n * a.tiles_m, a.kb, 12, 2, cost);
    mm_stall(a, S::STAGES, S::BUFS, MM_SCALE_SLOTS);
    CUtensorMap wmap, xmap;
    if (!mm_map(&wmap, B, a.n, k, ldb, 128) || !mm_map(&xmap, A, a.m, k, lda, NT)) return GPTQ_ERR_CUDA;
    auto kernel = fp8_mm_narrow_kernel<NT, TY>;
    GPTQ_SMEM_LIMIT(kernel, S::SMEM);
    return mm_launch(kernel, (long long)a.tiles_n * a.tiles_m * a.split, a.split, NARROW_THREADS, S::SMEM, s,
                     wmap, xmap, a);
}

template <typename TY>
inline int mm_tile(const void *A, long long lda, const void *B, long long ldb, long long k, MmArgs a,
                   int split, cudaStream_t s) {
    a.tiles_m = ceil_div(a.m, 128);
    a.tiles_n = ceil_div(a.n, 128);
    a.split = split;
    mm_stall(a, TILE_STAGES, TILE_BUFS, MM_SCALE_SLOTS);
    CUtensorMap amap, bmap;
    if (!mm_map(&amap, A, a.m, k, lda, 128) || !mm_map(&bmap, B, a.n, k, ldb, 128)) return GPTQ_ERR_CUDA;
    auto kernel = fp8_mm_tile_kernel<TY>;
    GPTQ_SMEM_LIMIT(kernel, TILE_SMEM);
    return mm_launch(kernel, (long long)a.tiles_m * a.tiles_n * a.split, a.split, TILE_THREADS, TILE_SMEM, s,
                     amap, bmap, a);
}

template <typename TY>
inline int mm_pair(const void *A, long long lda, const void *B, long long ldb, long long k, MmArgs a,
                   cudaStream_t s) {
    a.tiles_m = ceil_div(a.m, 256);
    a.tiles_n = ceil_div(a.n, 256);
    const long long tiles = (long long)a.tiles_m * a.tiles_n;
    if (tiles > 0x7fffffffLL - 1024) return GPTQ_ERR_ARG;
    a.split = 1;
    mm_stall(a, PAIR_STAGES, 2, PAIR_GROUPS);
    CUtensorMap amap, bmap, ymap = {};
    if (!mm_map(&amap, A, a.m, k, lda, 128) || !mm_map(&bmap, B, a.n, k, ldb, 128)) return GPTQ_ERR_CUDA;
    if (a.vec16 && !mm_out_map<TY>(&ymap, a)) return GPTQ_ERR_CUDA;
    auto kernel = fp8_mm_pair_kernel<TY>;
    GPTQ_SMEM_LIMIT(kernel, PAIR_SMEM);
    const long long pairs = std::min<long long>(tiles, device_sm_count() / 2);
    return mm_launch(kernel, 2 * pairs, 2, PAIR_THREADS, PAIR_SMEM, s, amap, bmap, ymap, a);
}

template <typename TY>
inline int mm_type(const void *A, long long lda, const void *B, long long ldb, long long k, MmArgs a,
                   cudaStream_t s) {
    // up to 32 rows the narrow kernel: 1 x 2048 x 6144 5.2 us, 32 rows 7.0 us (tile kernel 10.3 us);
    // at 64 rows of 6144 x 2048 the tile kernel is ahead, 9.1 us to 11.4 us
    if (a.m <= 16) return mm_narrow<16, TY>(A, lda, B, ldb, k, a, s);
    if (a.m <= 32) return mm_narrow<32, TY>(A, lda, B, ldb, k, a, s);
    // The tile kernel takes 0.22 us a block, 4.5 us a round of CTAs, 2.5 us for the sum over a
    // cluster; the pair kernel 0.44 us a block, 1 us a tile and 5 us once.
    // Pair to tile: 2048 x 2048 x 6144 26 us to 41, 512 x 6144 x 2048 12.2 to 19.4, 3001 x 2048 x 256
    // 7.3 to 14.6; 777 x 1500 x 2900 15.0 to 12.4, 1024 x 2048 x 6144 24.3 to 20.8, 128 x 6144 x 2048
    // 13.0 to 9.7.
    long long tile;
    const int split = mm_split((long long)ceil_div(a.m, 128) * ceil_div(a.n, 128), a.kb, 20, 11, tile);
    const long long tiles = (long long)ceil_div(a.m, 256) * ceil_div(a.n, 256), pairs = device_sm_count() / 2;
    const long long pair = (tiles + pairs - 1) / pairs * (2 * a.kb + 5) + 22;
    if (pair < tile) return mm_pair<TY>(A, lda, B, ldb, k, a, s);
    return mm_tile<TY>(A, lda, B, ldb, k, a, split, s);
}

inline int fp8_matmul(const void *A, long long lda, const float *sA, const void *B, long long ldb,
                      const float *sB, long long m, long long n, long long k, void *Y, int y_dtype,
                      long long ldy, cudaStream_t s) {
    const int size = serve_dtype_bytes(y_dtype);
    if (k == 0)
        return cudaMemset2DAsync(Y, (size_t)ldy * size, 0, (size_t)n * size, (size_t)m, s) == cudaSuccess
                   ? GPTQ_OK : GPTQ_ERR_CUDA;
    MmArgs a = {};
    a.sA = sA;
    a.sB = sB;
    a.Y = Y;
    a.ldy = ldy;
    a.m = (int)m;
    a.n = (int)n;
    a.kb = (int)((k + MM_BK - 1) / MM_BK);
    a.nb128 = ceil_div(n, 128);
    a.vec = ldy % 4 == 0 && reinterpret_cast<uintptr_t>(Y) % (4 * size) == 0;
    a.vec16 = ldy * size % 16 == 0 && reinterpret_cast<uintptr_t>(Y) % 16 == 0;
    // a wait longer than ~2 s at the 1.9 GHz clock means a lost signal, not a slow kernel
    static const long long wait_limit = tc::env_ll("GPTQ_WAIT_LIMIT_CYCLES", 4000000000LL);
    a.wait_limit = wait_limit;
    a.stall_n = (int)tc::env_ll("GPTQ_TEST_STALL", 0);   // made a range of barriers by mm_stall
    switch (y_dtype) {
        case GPTQ_BF16: return mm_type<__nv_bfloat16>(A, lda, B, ldb, k, a, s);
        case GPTQ_F16: return mm_type<__half>(A, lda, B, ldb, k, a, s);
        default: return mm_type<float>(A, lda, B, ldb, k, a, s);
    }
}

}  // namespace serve
}  // namespace gptq
