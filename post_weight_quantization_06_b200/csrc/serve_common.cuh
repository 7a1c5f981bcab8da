// Shared pieces of the serving operators (8-bit block product, quantized cache): vectors of eight
// values of the three input types, the conversion to e4m3, division by a number fixed per call.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "gptq_serve.h"

namespace gptq {
namespace serve {

constexpr float E4M3_MAX = 448.f;
constexpr float SCALE_MIN = 1.17549435e-38f;  // 2^-126: a scale and its reciprocal stay normal

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }

// Eight values as they lie in memory: one 16-byte word of a 16-bit type, two of fp32.
template <typename T>
struct Raw8 {
    static constexpr int WORDS = 8 * sizeof(T) / 16;
    uint4 w[WORDS];
};

// `vec`: all eight are there and p is 16-byte aligned. Otherwise the first `have` (0..8) are
// loaded one by one and the others are zero. (Plain loads throughout: these kernels may start while
// the one before them still writes, which the read-only path does not allow.)
template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, int have, Raw8<T> &r) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < Raw8<T>::WORDS; ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else {
        T *e = reinterpret_cast<T *>(r.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < have ? p[i] : narrow<T>(0.f);
    }
}
// All eight from an address of any alignment of T: the aligned 16-byte words around them, shifted
// into place. False, with nothing read, where a word would reach outside [lo, hi).
template <typename T>
__device__ __forceinline__ bool load8_shifted(const T *p, const void *lo, const void *hi, Raw8<T> &r) {
    constexpr int N = 4 * Raw8<T>::WORDS;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const char *at = reinterpret_cast<const char *>(p) - off;
    if (at < static_cast<const char *>(lo) || at + 4 * N + 16 > static_cast<const char *>(hi)) return false;
    uint32_t w[N + 4];
#pragma unroll
    for (int i = 0; i < N + 4; i += 4) {
        const uint4 q = *reinterpret_cast<const uint4 *>(at + 4 * i);
        w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
    }
#pragma unroll
    for (int i = 0; i < N + 2; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < N + 1; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
    uint32_t *o = reinterpret_cast<uint32_t *>(r.w);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = sizeof(T) == 4 ? w[i] : __funnelshift_r(w[i], w[i + 1], 8 * (off & 2));
    return true;
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T> &r, float *v) {
    const T *e = reinterpret_cast<const T *>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = widen(e[i]);
}
// Eight fp32 values rounded to T and stored.
template <typename T>
__device__ __forceinline__ void store8(T *p, bool vec, const float *v) {
    Raw8<T> r;
    T *e = reinterpret_cast<T *>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = narrow<T>(v[i]);
    if (vec) {
#pragma unroll
        for (int i = 0; i < Raw8<T>::WORDS; ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = e[i];
    }
}

// Maximum and minimum that let a NaN through: whether a group is finite is then seen from its
// range, without a test per value.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// Largest |x|, and smallest and largest x, of vectors of eight; 16-bit types two at a time.
template <typename T>
struct Amax {
    float m = 0.f;
    __device__ __forceinline__ void add(const Raw8<T> &r) {
        const T *e = reinterpret_cast<const T *>(r.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(e[i]));
    }
    __device__ __forceinline__ float value() const { return m; }
};
template <typename T>
struct MinMax {
    float mn = 0.f, mx = 0.f;
    __device__ __forceinline__ void add(const Raw8<T> &r) {
        const T *e = reinterpret_cast<const T *>(r.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mn = min_nan(mn, e[i]);
            mx = max_nan(mx, e[i]);
        }
    }
    __device__ __forceinline__ float low() const { return mn; }
    __device__ __forceinline__ float high() const { return mx; }
};
#define SERVE_PACKED_RANGE(T, T2)                                                            \
    template <>                                                                              \
    struct Amax<T> {                                                                         \
        uint32_t m = 0;                                                                      \
        __device__ __forceinline__ void add(const Raw8<T> &r) {                              \
            const T2 *e = reinterpret_cast<const T2 *>(r.w);                                 \
            T2 t = *reinterpret_cast<T2 *>(&m);                                              \
            _Pragma("unroll") for (int i = 0; i < 4; ++i) t = __hmax2_nan(t, __habs2(e[i])); \
            m = *reinterpret_cast<uint32_t *>(&t);                                           \
        }                                                                                    \
        __device__ __forceinline__ float value() const {                                     \
            const T2 t = *reinterpret_cast<const T2 *>(&m);                                  \
            return max_nan(widen(t.x), widen(t.y));                                          \
        }                                                                                    \
    };                                                                                       \
    template <>                                                                              \
    struct MinMax<T> {                                                                       \
        uint32_t mn = 0, mx = 0;                                                             \
        __device__ __forceinline__ void add(const Raw8<T> &r) {                              \
            const T2 *e = reinterpret_cast<const T2 *>(r.w);                                 \
            T2 a = *reinterpret_cast<T2 *>(&mn), b = *reinterpret_cast<T2 *>(&mx);           \
            _Pragma("unroll") for (int i = 0; i < 4; ++i) {                                  \
                a = __hmin2_nan(a, e[i]);                                                    \
                b = __hmax2_nan(b, e[i]);                                                    \
            }                                                                                \
            mn = *reinterpret_cast<uint32_t *>(&a);                                          \
            mx = *reinterpret_cast<uint32_t *>(&b);                                          \
        }                                                                                    \
        __device__ __forceinline__ float low() const {                                       \
            const T2 t = *reinterpret_cast<const T2 *>(&mn);                                 \
            return min_nan(widen(t.x), widen(t.y));                                          \
        }                                                                                    \
        __device__ __forceinline__ float high() const {                                      \
            const T2 t = *reinterpret_cast<const T2 *>(&mx);                                 \
            return max_nan(widen(t.x), widen(t.y));                                          \
        }                                                                                    \
    };
SERVE_PACKED_RANGE(__nv_bfloat16, __nv_bfloat162)
SERVE_PACKED_RANGE(__half, __half2)
#undef SERVE_PACKED_RANGE

// The largest of the finite |v|; the others become NaN. For groups that are not finite.
__device__ __forceinline__ float amax_finite8(float *v) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!finitef(v[i])) v[i] = __uint_as_float(0x7fffffffu);
        else a = fmaxf(a, fabsf(v[i]));
    }
    return a;
}

__device__ __forceinline__ float e4m3_scale(float amax) {
    return fmaxf(__fdiv_rn(amax, E4M3_MAX), SCALE_MIN);
}

// x r truncated to fp32 with the last bit set where the truncation dropped something: rounding
// that to e4m3 rounds the exact product (a nearest product could itself land on a border
// between two codes, which would then be decided by the even one).
__device__ __forceinline__ float mul_sticky(float x, float r) {
    uint32_t p = __float_as_uint(__fmul_rz(x, r));
    const float d = __fmaf_rn(x, r, -__uint_as_float(p));
    asm("{\n\t.reg .pred q;\n\tsetp.neu.f32 q, %1, 0f00000000;\n\t@q or.b32 %0, %0, 1;\n\t}" : "+r"(p) : "f"(d));
    return __uint_as_float(p);
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}
// Eight e4m3 codes of v under the reciprocal scale r, the first in the lowest byte.
__device__ __forceinline__ uint2 e4m3_codes8(const float *v, float r) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = e4m3_pair(mul_sticky(v[2 * i], r), mul_sticky(v[2 * i + 1], r));
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// n / d by a multiplication, exact for n * d < 2^32 (the error of the rounded-up reciprocal,
// below d / 2^32 per unit of n, then never reaches the next whole number).
struct FastDiv {
    uint32_t d, m;
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return m ? __umulhi(n, m) : n; }
};
inline FastDiv fast_div(uint32_t d) {
    return FastDiv{d, d > 1 ? (uint32_t)((0x100000000ull + d - 1) / d) : 0u};
}

inline bool serve_dtype_ok(int t) { return t == GPTQ_BF16 || t == GPTQ_F32 || t == GPTQ_F16; }
inline int serve_dtype_bytes(int t) { return t == GPTQ_F32 ? 4 : 2; }

}  // namespace serve
}  // namespace gptq
