// A matrix to e4m3 codes with one scale for each block of block_rows x 128 (gptq_fp8_quantize).
//
//   s = max(max |x| / 448, 2^-126), r = 1 / s, code = e4m3(x r)
//
// One pass: a block stays in registers between its maximum and its codes. Bytes bound it: b + 1
// for each value of b bytes.
#pragma once

#include "serve_common.cuh"

namespace gptq {
namespace serve {

struct Fp8QuantArgs {
    const void *X;
    long long rows, cols, ldx, ldc;
    unsigned char *codes;
    float *scales;
    uint32_t kb;        // blocks of 128 per row
    long long units;    // rows * kb (block_rows 1) or block rows * kb
    int vec_in, vec_out;
};

__device__ __forceinline__ void store_codes8(unsigned char *p, bool vec, int have, uint2 c) {
    if (vec) {
        *reinterpret_cast<uint2 *>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < have) p[i] = (unsigned char)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

constexpr int FQ_THREADS = 256;
constexpr int FQ_UNITS = 4;  // units in flight per half warp

// block_rows 1: a half warp per block, eight values per lane; each half warp takes FQ_UNITS
// blocks, all loaded before the first is worked on.
template <typename T>
__global__ void __launch_bounds__(FQ_THREADS) fp8_quantize_rows_kernel(Fp8QuantArgs a) {
    pdl_launch_next();
    pdl_wait_prev();
    const int lane = threadIdx.x & 31, l = lane & 15;
    const long long half = ((long long)blockIdx.x * FQ_THREADS + threadIdx.x) >> 4;
    const long long halves = (long long)gridDim.x * (FQ_THREADS / 16);
    Raw8<T> raw[FQ_UNITS];
    uint32_t row[FQ_UNITS], b[FQ_UNITS];
    int have[FQ_UNITS];
#pragma unroll
    for (int i = 0; i < FQ_UNITS; ++i) {
        const long long u = half + i * halves;
        have[i] = -1;
        row[i] = b[i] = 0;
        if (u < a.units) {
            row[i] = (uint32_t)u / a.kb;
            b[i] = (uint32_t)u - row[i] * a.kb;
            const long long c = (long long)b[i] * 128 + 8 * l;
            have[i] = (int)max(0LL, min(8LL, a.cols - c));
        }
        const T *p = static_cast<const T *>(a.X) + (long long)row[i] * a.ldx + (long long)b[i] * 128 + 8 * l;
        load8(p, a.vec_in && have[i] == 8, have[i], raw[i]);
    }
#pragma unroll
    for (int i = 0; i < FQ_UNITS; ++i) {
        float v[8];
        widen8(raw[i], v);
        uint32_t m = amax_bits8(v);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (__any_sync(0xffffffffu, m >= INF_BITS)) {
            const bool bad = m >= INF_BITS;
            m = amax_finite8(v);
#pragma unroll
            for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (bad && l == 0 && have[i] >= 0) report(GPTQ_ERR_NONFINITE, row[i]);
        }
        const float s = e4m3_scale(m);
        const uint2 c = e4m3_codes8(v, __frcp_rn(s));
        if (have[i] < 0) continue;
        if (l == 0) a.scales[(long long)row[i] * a.kb + b[i]] = s;
        store_codes8(a.codes + (long long)row[i] * a.ldc + (long long)b[i] * 128 + 8 * l,
                     a.vec_out && have[i] == 8, have[i], c);
    }
}

// block_rows 128: a CTA per block, 64 values per thread (rows t / 16 + 16 i, columns 8 (t % 16)).
template <typename T>
__global__ void __launch_bounds__(FQ_THREADS) fp8_quantize_tiles_kernel(Fp8QuantArgs a) {
    pdl_launch_next();
    pdl_wait_prev();
    __shared__ uint32_t wmax[2][FQ_THREADS / 32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint32_t br = blockIdx.x / a.kb, b = blockIdx.x - br * a.kb;
    const long long c = (long long)b * 128 + 8 * (t & 15);
    const int have = (int)max(0LL, min(8LL, a.cols - c));
    Raw8<T> raw[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long r = (long long)br * 128 + (t >> 4) + 16 * i;
        const int n = r < a.rows ? have : 0;
        load8(static_cast<const T *>(a.X) + (n ? r * a.ldx + c : 0), a.vec_in && n == 8, n, raw[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        widen8(raw[i], v);
        m = max(m, amax_bits8(v));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) wmax[0][warp] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < FQ_THREADS / 32; ++w) m = max(m, wmax[0][w]);
    if (m >= INF_BITS) {  // the same in every thread
        m = 0;
        for (int i = 0; i < 8; ++i) {
            float v[8];
            widen8(raw[i], v);
            if (amax_bits8(v) >= INF_BITS)
                report(GPTQ_ERR_NONFINITE, (long long)br * 128 + (t >> 4) + 16 * i);
            m = max(m, amax_finite8(v));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) wmax[1][warp] = m;
        __syncthreads();
        m = 0;
        for (int w = 0; w < FQ_THREADS / 32; ++w) m = max(m, wmax[1][w]);
    }
    const float s = e4m3_scale(m), r = __frcp_rn(s);
    if (t == 0) a.scales[blockIdx.x] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long row = (long long)br * 128 + (t >> 4) + 16 * i;
        if (row >= a.rows || have == 0) continue;
        float v[8];
        widen8(raw[i], v);
        // an infinity becomes the format's NaN: its product with r would saturate
        if (amax_bits8(v) >= INF_BITS) amax_finite8(v);
        store_codes8(a.codes + row * a.ldc + c, a.vec_out && have == 8, have, e4m3_codes8(v, r));
    }
}

template <typename T>
inline int fp8_quantize_launch(const Fp8QuantArgs &a, int block_rows, cudaStream_t s) {
    if (block_rows == 1) {
        const long long per = FQ_THREADS / 16 * FQ_UNITS;
        return launch_kernel(fp8_quantize_rows_kernel<T>, dim3((unsigned)((a.units + per - 1) / per)),
                             dim3(FQ_THREADS), 0, s, true, a);
    }
    return launch_kernel(fp8_quantize_tiles_kernel<T>, dim3((unsigned)a.units), dim3(FQ_THREADS), 0,
                         s, true, a);
}

inline int fp8_quantize(const void *X, int x_dtype, long long rows, long long cols, long long ldx,
                        int block_rows, void *codes, long long ldc, float *scales, cudaStream_t s) {
    Fp8QuantArgs a;
    a.X = X;
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    a.ldc = ldc;
    a.codes = static_cast<unsigned char *>(codes);
    a.scales = scales;
    a.kb = (uint32_t)((cols + 127) / 128);
    a.units = (block_rows == 1 ? rows : (rows + 127) / 128) * (long long)a.kb;
    const int b = serve_dtype_bytes(x_dtype);
    a.vec_in = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (ldx * b) % 16 == 0;
    a.vec_out = (reinterpret_cast<uintptr_t>(codes) & 7u) == 0 && ldc % 8 == 0;
    switch (x_dtype) {
        case GPTQ_BF16: return fp8_quantize_launch<__nv_bfloat16>(a, block_rows, s);
        case GPTQ_F16: return fp8_quantize_launch<__half>(a, block_rows, s);
        default: return fp8_quantize_launch<float>(a, block_rows, s);
    }
}

}  // namespace serve
}  // namespace gptq
