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
    const void *X, *X_end;   // X_end: behind the last value
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
constexpr int FQ_LANES = 4;

// block_rows 1: L lanes per block, 128 / L values each (pieces of eight l, l + L, ... of the block's
// sixteen). The scale, its reciprocal and the block's place cost some 70 instructions, which at
// 8 values a lane was more than all the rest: 16384 x 6144 bf16 took 88 us, with 32 it takes 51 us
// (5.9 TB/s; with 64, fewer lanes have a load on its way, 64 us).
template <typename T, int L>
__global__ void __launch_bounds__(FQ_THREADS) fp8_quantize_rows_kernel(Fp8QuantArgs a) {
    pdl_launch_next();
    pdl_wait_prev();
    constexpr int V = 16 / L;
    const int l = threadIdx.x & (L - 1);
    const long long u = ((long long)blockIdx.x * FQ_THREADS + threadIdx.x) / L;
    const bool live = u < a.units;
    const uint32_t row = live ? (uint32_t)u / a.kb : 0, b = live ? (uint32_t)u - row * a.kb : 0;
    const int left = live ? (int)min(128LL, a.cols - (long long)b * 128) : 0;   // columns of the block
    const bool whole = left == 128;
    const T *x = static_cast<const T *>(a.X) + (long long)row * a.ldx + (long long)b * 128;
    Raw8<T> raw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (l + L * i);
        const int have = whole ? 8 : max(0, min(8, left - c));
        if (whole && a.vec_in) load8(x + c, true, 8, raw[i]);
        else if (a.vec_in || have < 8 || !load8_shifted(x + c, a.X, a.X_end, raw[i]))
            load8(have ? x + c : x, a.vec_in && have == 8, have, raw[i]);
    }
    Amax<T> am;
#pragma unroll
    for (int i = 0; i < V; ++i) am.add(raw[i]);
    float m = am.value();
#pragma unroll
    for (int o = L >> 1; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool bad = !finitef(m);
    if (__any_sync(0xffffffffu, bad)) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v[8];
            widen8(raw[i], v);
            m = fmaxf(m, amax_finite8(v));
        }
#pragma unroll
        for (int o = L >> 1; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (bad && l == 0) report(GPTQ_ERR_NONFINITE, row);
    }
    if (!live) return;
    const float s = e4m3_scale(m), r = __frcp_rn(s);
    if (l == 0) a.scales[(long long)row * a.kb + b] = s;
    unsigned char *y = a.codes + (long long)row * a.ldc + (long long)b * 128;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (l + L * i);
        float v[8];
        widen8(raw[i], v);
        // an infinity becomes the format's NaN: its product with r would saturate
        if (bad) amax_finite8(v);
        const uint2 q = e4m3_codes8(v, r);
        if (whole && a.vec_out) *reinterpret_cast<uint2 *>(y + c) = q;
        else store_codes8(y + c, a.vec_out && left - c >= 8, left - c, q);
    }
}

// block_rows 128: a CTA per block, 32 values per thread (rows t / 16 + 32 i, columns 8 (t % 16)). A CTA
// loads, then computes: several per SM overlap. Three of 512 threads for 16-bit types (8192 x 8192
// bf16 in 45 us, 5000 x 3001 in 18 us; four of 256, whose unaligned loads spill, 43 and 20 us), two for fp32
// (2047 x 6100 in 14 us, 8192 x 8192 in 57 us = 5.9 TB/s; one of 1024, 90 us).
constexpr int FQ_TILE_THREADS = 512;
template <typename T>
__global__ void __launch_bounds__(FQ_TILE_THREADS, sizeof(T) == 2 ? 3 : 2) fp8_quantize_tiles_kernel(Fp8QuantArgs a) {
    pdl_launch_next();
    pdl_wait_prev();
    __shared__ float wmax[2][FQ_TILE_THREADS / 32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint32_t br = blockIdx.x / a.kb, b = blockIdx.x - br * a.kb;
    const long long c = (long long)b * 128 + 8 * (t & 15);
    const int have = (int)max(0LL, min(8LL, a.cols - c));
    constexpr int V = 2048 / FQ_TILE_THREADS, R = FQ_TILE_THREADS / 16;   // vectors of a thread, rows between them
    Raw8<T> raw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const long long r = (long long)br * 128 + (t >> 4) + R * i;
        const int n = r < a.rows ? have : 0;
        const T *x = static_cast<const T *>(a.X) + (n ? r * a.ldx + c : 0);
        if (a.vec_in || n < 8 || !load8_shifted(x, a.X, a.X_end, raw[i]))
            load8(x, a.vec_in && n == 8, n, raw[i]);
    }
    Amax<T> am;
#pragma unroll
    for (int i = 0; i < V; ++i) am.add(raw[i]);
    float m = am.value();
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) wmax[0][warp] = m;
    __syncthreads();
    m = 0.f;
#pragma unroll
    for (int w = 0; w < FQ_TILE_THREADS / 32; ++w) m = max_nan(m, wmax[0][w]);
    const bool bad = !finitef(m);   // the same in every thread
    if (bad) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v[8];
            widen8(raw[i], v);
            Amax<T> one;
            one.add(raw[i]);
            if (!finitef(one.value()))
                report(GPTQ_ERR_NONFINITE, (long long)br * 128 + (t >> 4) + R * i);
            m = fmaxf(m, amax_finite8(v));
        }
        m = warp_max(m);
        if (lane == 0) wmax[1][warp] = m;
        __syncthreads();
        m = 0.f;
        for (int w = 0; w < FQ_TILE_THREADS / 32; ++w) m = fmaxf(m, wmax[1][w]);
    }
    const float s = e4m3_scale(m), r = __frcp_rn(s);
    if (t == 0) a.scales[blockIdx.x] = s;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const long long row = (long long)br * 128 + (t >> 4) + R * i;
        if (row >= a.rows || have == 0) continue;
        float v[8];
        widen8(raw[i], v);
        if (bad) amax_finite8(v);
        store_codes8(a.codes + row * a.ldc + c, a.vec_out && have == 8, have, e4m3_codes8(v, r));
    }
}

template <typename T>
inline int fp8_quantize_launch(const Fp8QuantArgs &a, int block_rows, cudaStream_t s) {
    if (block_rows == 1) {
        const long long per = FQ_THREADS / FQ_LANES;
        return launch_kernel(fp8_quantize_rows_kernel<T, FQ_LANES>, dim3((unsigned)((a.units + per - 1) / per)),
                             dim3(FQ_THREADS), 0, s, true, a);
    }
    return launch_kernel(fp8_quantize_tiles_kernel<T>, dim3((unsigned)a.units), dim3(FQ_TILE_THREADS), 0,
                         s, true, a);
}

inline int fp8_quantize(const void *X, int x_dtype, long long rows, long long cols, long long ldx,
                        int block_rows, void *codes, long long ldc, float *scales, cudaStream_t s) {
    Fp8QuantArgs a;
    a.X = X;
    a.X_end = static_cast<const char *>(X) + ((rows - 1) * ldx + cols) * serve_dtype_bytes(x_dtype);
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
