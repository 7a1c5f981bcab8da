// The quantized cache of keys and values (gptq_cache_write, gptq_cache_read).
//
// Write: a unit is one group of one head of one token of K or V. A power of two of lanes holds
// it, up to 48 values each, between its range and its codes: one pass over the values. Read: a unit
// is 8 or 16 values.
//   int:  s = max((mx - mn) / maxq, 2^-126), z = rint(-mn maxq / (mx - mn)),
//         c = clamp(rint(x / s + z)), value s (c - z)
//   e4m3: s = max(max |x| / 448, 2^-126), c = e4m3(x / s), value s c
// Both are bound by bytes for long calls and by the latency of slot -> data -> store for a
// decode step; a CTA takes a few whole tokens, so that the slots are looked at once per token.
#pragma once

#include <algorithm>
#include <type_traits>

#include "serve_common.cuh"

namespace gptq {
namespace serve {

constexpr int CACHE_THREADS = 256;
constexpr int CACHE_MAX_TB = 8;      // tokens of a CTA
constexpr int CACHE_MAX_HD = 65536;  // heads * head_dim: unit numbers stay exact in FastDiv

struct CachePlane {
    const void *x;         // values (read: null)
    void *y;               // values (write: null)
    long long ts, hs;      // strides of x or y in elements
    unsigned char *codes;
    float *scales;
    uint8_t *zeros;
    int vec;               // x or y takes 16-byte (1) or 32-byte (2) accesses
};

struct CacheArgs {
    CachePlane p[2];
    const int64_t *slots;
    int32_t *claims;
    long long n_slots;
    int tokens, heads, dim, group;  // group: values that share a scale
    int tb;                         // tokens of a CTA
    FastDiv per_token, per_plane, per_head, per_group;  // units (see each kernel)
    int w;                          // lanes of a unit (write)
    int vec;                        // codes take 16-byte accesses (read)
    int full;                       // every lane has all its vectors, aligned (write)
    int clear;                      // rows of no slot are set to zero (read)
};

// ---------------------------------------------------------------------------------------
// Which token of a call stays in a slot that several of them name: the last. Up to
// GPTQ_CACHE_UNCLAIMED tokens each CTA compares its own tokens' slots with the later ones (two
// loads a thread; 512 tokens of 8 x 128 in 3.9 us); beyond that the comparisons would outgrow the
// copy, and the tokens first claim their slots: claims[slot] = the largest token + 1 (513 tokens in
// 4.2 us, a launch more).
// ---------------------------------------------------------------------------------------
__global__ void cache_claim_kernel(const int64_t *slots, int tokens, long long n_slots,
                                   int32_t *claims) {
    pdl_launch_next();
    pdl_wait_prev();
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t >= tokens) return;
    const long long s = slots[t];
    if (s >= 0 && s < n_slots) atomicMax(&claims[s], t + 1);
}

// slot[j] of the CTA's tokens t0 + j, or -1 where the token is not written (also where beaten[j]).
__device__ __forceinline__ void cache_resolve(const CacheArgs &a, int t0, int nt, long long *slot,
                                              int *beaten) {
    const int tid = threadIdx.x;
    if (tid < nt) {
        long long s = a.slots[t0 + tid];
        if (s >= a.n_slots) {
            report(GPTQ_ERR_ARG, t0 + tid);
            s = -1;
        }
        if (a.claims && s >= 0) {
            // only the winner clears the claim, so a loser can read its own number never
            if (*(volatile int32_t *)&a.claims[s] == t0 + tid + 1) a.claims[s] = 0;
            else s = -1;
        }
        slot[tid] = s;
        beaten[tid] = 0;
    }
    __syncthreads();
    if (!a.claims) {
        for (int i = t0 + 1 + tid; i < a.tokens; i += CACHE_THREADS) {
            const long long s = a.slots[i];
            for (int j = 0; j < nt; ++j)
                if (i > t0 + j && s == slot[j]) beaten[j] = 1;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------------------
constexpr float CACHE_MAGIC = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number

// The whole number nearest to -mn maxq / (mx - mn), ties to even: a symmetric range lies on the
// border between two, and rounded operands would pick either. In fp64 both products and the
// difference are exact; the quotient's whole number is corrected by the remainder.
__device__ __forceinline__ float cache_zero(float mn, float mx, float maxq, double) {
    const double num = -(double)mn * (double)maxq, den = (double)mx - (double)mn;
    int q = (int)rintf(__fdiv_rn(-mn, mx - mn) * maxq);
    const double d = 2.0 * (num - (double)q * den);
    if (d > den || (d == den && (q & 1))) ++q;
    else if (d < -den || (d == -den && (q & 1))) --q;
    return (float)min(max(q, 0), (int)maxq);
}
// The same in fp32 for values of 16-bit types (at most 11 bits): the product has 19, and the
// difference is exact unless the exponents are 13 or more apart, where the quotient is far from
// a border. A power of two keeps the product from overflowing. A quotient that rounds to a border
// is decided by the sign of the remainder.
__device__ __forceinline__ float cache_zero(float mn, float mx, float maxq, float) {
    const float k = mx - mn > 1.f ? 0.00390625f : 1.f;
    const float num = -mn * k * maxq, den = (mx - mn) * k;
    const float q = __fdiv_rn(num, den);
    float z = rintf(q);
    if (fabsf(q - z) == 0.5f) {
        const float r = fmaf(-q, den, num);
        if (r != 0.f) z = q + (r > 0.f ? 0.5f : -0.5f);
    }
    return fminf(fmaxf(z, 0.f), maxq);
}

// Min-max grid of a group: scale, its reciprocal, zero-point. `edge`: an end of the range lies so
// near the middle between a code and one that does not exist that codes have to be clamped.
// False where the range is not finite.
template <typename T>
__device__ __forceinline__ bool cache_grid(float mn, float mx, float maxq, float &s, float &r,
                                           float &z, bool &edge) {
    if (mx == mn) { mn = -1.f; mx = 1.f; }   // both zero: the range starts from there
    const float range = mx - mn;
    if (!finitef(range)) return false;
    s = fmaxf(__fdiv_rn(range, maxq), SCALE_MIN);
    r = __frcp_rn(s);
    typedef typename std::conditional<sizeof(T) == 2, float, double>::type Z;
    z = cache_zero(mn, mx, maxq, Z());
    edge = fabsf(fmaf(mn, r, z)) > 0.499f || fabsf(fmaf(mx, r, z - maxq)) > 0.499f;
    return true;
}

// Where a unit's values are, and what it is.
struct WriteUnit {
    uint32_t j, pl, h, g;
    bool live;
    __device__ __forceinline__ void place(const CacheArgs &a, uint32_t u, uint32_t units) {
        live = u < units;
        if (!live) u = 0;
        j = a.per_token.div(u);
        const uint32_t rem = u - j * a.per_token.d;
        pl = a.per_plane.div(rem);
        const uint32_t hg = rem - pl * a.per_plane.d;
        h = a.per_head.div(hg);
        g = hg - h * a.per_head.d;
    }
    template <int V, typename T>
    __device__ __forceinline__ void load(const CacheArgs &a, int t0, int l, int nvec, Raw8<T> *raw) const {
        const CachePlane &p = a.p[pl];
        const T *x = static_cast<const T *>(p.x) + (long long)(t0 + (int)j) * p.ts +
                     (long long)h * p.hs + (long long)g * a.group;
        if (a.full) {   // units that do not exist read the first token's
            x += 8 * l;
#pragma unroll
            for (int i = 0; i < V; ++i) load8(x + i * 8 * a.w, true, 8, raw[i]);
            return;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = l + i * a.w;
            const bool on = live && v < nvec;
            load8(x + (on ? 8 * v : 0), on && p.vec, on ? 8 : 0, raw[i]);
        }
    }
};

// CTAs an SM with V vectors of eight a lane. At 16 bits the min-max forms spill 4 to 24 bytes a thread under
// these bounds. Five instead of six with V = 4: 2048 tokens of 8 x 128 at 8 bits 6.5 us instead of 7.3, at
// e4m3 6.3 and 6.6; 32768 tokens 42.8 and 43.2, at e4m3 44.5 and 42.8.
template <typename T>
__host__ __device__ constexpr int cache_write_ctas(int V) {
    return sizeof(T) == 2 ? (V == 4 ? 6 : 5) : (V == 4 ? 4 : 3);
}
template <typename T, int FMT, int V>
__global__ void __launch_bounds__(CACHE_THREADS, cache_write_ctas<T>(V))
cache_write_kernel(const __grid_constant__ CacheArgs a) {
    __shared__ long long slot[CACHE_MAX_TB];
    __shared__ int beaten[CACHE_MAX_TB];
    pdl_launch_next();
    pdl_wait_prev();
    const int t0 = blockIdx.x * a.tb;
    const int nt = min(a.tb, a.tokens - t0);
    const int w = a.w, l = threadIdx.x & (w - 1);
    const uint32_t units = (uint32_t)nt * a.per_token.d;
    const uint32_t step = CACHE_THREADS / w;
    const int nvec = a.group >> 3;
    // the first values are on their way while the slots are looked at
    WriteUnit at0;
    Raw8<T> raw[V];
    at0.place(a, threadIdx.x / w, units);
    at0.load<V>(a, t0, l, nvec, raw);
    cache_resolve(a, t0, nt, slot, beaten);
    for (uint32_t u0 = 0; u0 < units; u0 += step) {
        if (u0) {
            at0.place(a, u0 + threadIdx.x / w, units);
            at0.load<V>(a, t0, l, nvec, raw);
        }
        const uint32_t j = at0.j, h = at0.h, g = at0.g;
        const CachePlane &p = a.p[at0.pl];
        const long long sl = at0.live && !beaten[j] ? slot[j] : -1;
        float s, r, z = 0.f;
        bool bad, edge = false;
        if (FMT == GPTQ_CACHE_E4M3) {
            Amax<T> am;
#pragma unroll
            for (int i = 0; i < V; ++i) am.add(raw[i]);
            float m = am.value();
            for (int o = w >> 1; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            bad = !finitef(m);
            if (__any_sync(0xffffffffu, bad)) {
                m = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float v[8];
                    widen8(raw[i], v);
                    m = fmaxf(m, amax_finite8(v));
                }
                for (int o = w >> 1; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            s = e4m3_scale(m);
            r = __frcp_rn(s);
        } else {
            constexpr float maxq = FMT == GPTQ_CACHE_INT4 ? 15.f : 255.f;
            MinMax<T> mm;
#pragma unroll
            for (int i = 0; i < V; ++i) mm.add(raw[i]);
            float mn = mm.low(), mx = mm.high();
            for (int o = w >> 1; o; o >>= 1) {
                mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            bad = !cache_grid<T>(mn, mx, maxq, s, r, z, edge);
            edge = __any_sync(0xffffffffu, edge || bad);
            if (bad) {
                s = __uint_as_float(0x7fffffffu);
                r = 0.f;
                z = 0.f;
            }
        }
        if (sl < 0) continue;
        if (bad && l == 0) report(GPTQ_ERR_NONFINITE, t0 + (int)j);
        const long long row = sl * a.heads + h;
        if (l == 0) {
            const long long m = row * a.per_head.d + g;
            p.scales[m] = s;
            if (FMT != GPTQ_CACHE_E4M3) p.zeros[m] = (uint8_t)z;
        }
        unsigned char *code = p.codes + ((row * a.dim + (long long)g * a.group) >> (FMT == GPTQ_CACHE_INT4));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = l + i * w;
            if (!a.full && v >= nvec) continue;
            float f[8];
            widen8(raw[i], f);
            if (FMT == GPTQ_CACHE_E4M3) {
                if (bad) amax_finite8(f);
                *reinterpret_cast<uint2 *>(code + 8 * v) = e4m3_codes8(f, r);
            } else {
                // x r + z rounded once, to a whole number in the low bits
                constexpr float maxq = FMT == GPTQ_CACHE_INT4 ? 15.f : 255.f;
                uint32_t c[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e] = __float_as_uint(fmaf(f[e], r, CACHE_MAGIC + z));
                if (edge) {
                    // a group that is not finite (r = 0, and NaN here at most) gets code 0
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        c[e] = bad ? 0u : __float_as_uint(fminf(fmaxf(__uint_as_float(c[e]), CACHE_MAGIC),
                                                                CACHE_MAGIC + maxq));
                }
                if (FMT == GPTQ_CACHE_INT8) {
                    const uint32_t lo = __byte_perm(__byte_perm(c[0], c[1], 0x0040),
                                                    __byte_perm(c[2], c[3], 0x0040), 0x5410);
                    const uint32_t hi = __byte_perm(__byte_perm(c[4], c[5], 0x0040),
                                                    __byte_perm(c[6], c[7], 0x0040), 0x5410);
                    *reinterpret_cast<uint2 *>(code + 8 * v) = make_uint2(lo, hi);
                } else {
                    // the low byte of c0 + 16 c1 is both codes: the bits above them in c0 and c1
                    // (2^23's) lie beyond it
                    const uint32_t lo = __byte_perm(c[0] + 16 * c[1], c[2] + 16 * c[3], 0x0040);
                    const uint32_t hi = __byte_perm(c[4] + 16 * c[5], c[6] + 16 * c[7], 0x0040);
                    *reinterpret_cast<uint32_t *>(code + 4 * v) = __byte_perm(lo, hi, 0x5410);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------------
// read
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void store32(void *p, const uint4 &a, const uint4 &b) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
// Eight values of one word (4 bits) or two (8 bits), in fp32. An output of 16 bits rounds them a second
// time: 0 to 9 of 100000 values then come out one step from the nearest one. A sticky last bit, as the
// quantizer has it, would avoid that at four instructions a value instead of one: 131072 tokens of
// 8 x 128 at 8 bits 137 us, 127 us without; 8192 tokens at 4 bits 10.8 and 8.9 us.
template <int FMT>
__device__ __forceinline__ void decode8(uint2 c, float s, float z, float *f) {
    if (FMT == GPTQ_CACHE_E4M3) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = e < 2 ? c.x : c.y;
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w >> (16 * (e & 1)))));
            const __half2 hv = *reinterpret_cast<const __half2 *>(&h2);
            f[2 * e] = __low2float(hv) * s;
            f[2 * e + 1] = __high2float(hv) * s;
        }
    } else {
        // a code in the low bits of 2^23 is 2^23 + code: the difference is exact
        const float bias = 8388608.f + z;
        if (FMT == GPTQ_CACHE_INT4) {
            // the even codes and the odd ones, a byte each
            const uint32_t odd = (c.x >> 4) & 0x0f0f0f0fu;
            c.x &= 0x0f0f0f0fu;
            c.y = odd;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool second = FMT == GPTQ_CACHE_INT4 ? e & 1 : e > 3;
            const uint32_t at = FMT == GPTQ_CACHE_INT4 ? e >> 1 : e & 3;
            const uint32_t q = __byte_perm(second ? c.y : c.x, 0x4b000000u, 0x7440u | at);
            f[e] = (__uint_as_float(q) - bias) * s;
        }
    }
}

// Zeros in place of unit `rem` of token t (units as in the next kernel). Apart from its loop, where
// an address taken before the loads, for both uses, cost 1 to 3 %.
template <typename T, int U>
__device__ __noinline__ void cache_clear(const CacheArgs &a, int t, uint32_t rem) {
    const uint32_t pl = a.per_plane.div(rem), v = rem - pl * a.per_plane.d, h = a.per_head.div(v);
    const CachePlane &p = a.p[pl];
    T *y = static_cast<T *>(p.y) + (long long)t * p.ts + (long long)h * p.hs + 8 * U * (v - h * a.per_head.d);
    const float zero[8] = {};
#pragma unroll
    for (int k = 0; k < U; ++k) store8(y + 8 * k, p.vec != 0, zero);
}

// One unit is 8 U values; per_token.d units per token over the planes, per_plane.d per plane,
// per_head.d per head, and per_group.d of them share a scale. U = 2 where heads and groups are
// multiples of 16: what a unit's place costs is then shared by 16 values, and its 16-bit output
// is one 32-byte store. A thread does one unit after another: several at once took more registers
// than they saved waiting (131072 tokens of 8 x 128 at 8 bits: four at once 172 us, one 127 us).
template <typename T, int FMT, int U>
__global__ void __launch_bounds__(CACHE_THREADS, 8) cache_read_kernel(const __grid_constant__ CacheArgs a) {
    pdl_launch_next();
    pdl_wait_prev();
    const int t0 = blockIdx.x * a.tb;
    const int nt = min(a.tb, a.tokens - t0);
    const uint32_t units = (uint32_t)nt * a.per_token.d;
    const int row = a.heads * a.dim, meta = a.heads * (a.dim / a.group);
    for (uint32_t u = threadIdx.x; u < units; u += CACHE_THREADS) {
        const uint32_t j = a.per_token.div(u), rem = u - j * a.per_token.d;
        const long long sl = a.slots[t0 + (int)j];
        if (sl < 0 || sl >= a.n_slots) {
            if (sl >= 0 && rem == 0) report(GPTQ_ERR_ARG, t0 + (int)j);
            if (a.clear) cache_clear<T, U>(a, t0 + (int)j, rem);
            continue;
        }
        const uint32_t pl = a.per_plane.div(rem), v = rem - pl * a.per_plane.d;
        const CachePlane &p = a.p[pl];
        const long long at = sl * row + 8LL * U * v;
        uint2 c[U];
        if (FMT == GPTQ_CACHE_INT4) {
            if (U == 2) {
                const uint2 q = *reinterpret_cast<const uint2 *>(p.codes + (at >> 1));
                c[0].x = q.x;
                c[U - 1].x = q.y;
            } else {
                c[0].x = *reinterpret_cast<const uint32_t *>(p.codes + (at >> 1));
            }
        } else if (U == 2 && a.vec) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p.codes + at);
            c[0] = make_uint2(q.x, q.y);
            c[U - 1] = make_uint2(q.z, q.w);
        } else {
#pragma unroll
            for (int k = 0; k < U; ++k) c[k] = *reinterpret_cast<const uint2 *>(p.codes + at + 8 * k);
        }
        const long long m = sl * meta + a.per_group.div(v);
        const float s = p.scales[m];
        const float z = FMT != GPTQ_CACHE_E4M3 ? (float)p.zeros[m] : 0.f;
        const uint32_t h = a.per_head.div(v);
        T *y = static_cast<T *>(p.y) + (long long)(t0 + (int)j) * p.ts + (long long)h * p.hs +
               8 * U * (v - h * a.per_head.d);
        float f[8 * U];
#pragma unroll
        for (int k = 0; k < U; ++k) decode8<FMT>(c[k], s, z, f + 8 * k);
        if (U == 2 && sizeof(T) == 2 && p.vec == 2) {
            uint4 o[2];
            T *e = reinterpret_cast<T *>(o);
#pragma unroll
            for (int k = 0; k < 8 * U; ++k) e[k & 15] = narrow<T>(f[k]);
            store32(y, o[0], o[1]);
        } else {
#pragma unroll
            for (int k = 0; k < U; ++k) store8(y + 8 * k, p.vec != 0, f + 8 * k);
        }
    }
}

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------
// Tokens of a CTA: as many as its threads take at once (`per_token` threads each), more where that
// leaves several CTAs per SM all the same.
inline int cache_tokens_per_cta(int tokens, long long per_token) {
    const int once = (int)std::max(1LL, std::min<long long>(CACHE_MAX_TB, CACHE_THREADS / per_token));
    const int most = tokens / (device_sm_count() * 8) / once * once;
    return std::min(CACHE_MAX_TB, std::max(once, most));
}

template <typename T, int FMT>
inline int cache_write_launch(CacheArgs &a, cudaStream_t s) {
    // Four or six vectors of eight a lane: what a group costs once (its grid) is shared by up to 48
    // values. Six where that leaves fewer of them empty (heads of 80, 96, 192) and four would take more
    // lanes than the device holds at once; up to there more lanes are the shorter way. With four and six,
    // bf16 at 4 bits: 16 x 80, 1024 tokens 7.1 and 7.2 us, 2048 8.8 and 8.2, 32768 76 and 55; 8 x 96, 2048 tokens
    // 6.9 and 8.0, 8192 13.0 and 11.4; 8 x 192, 1024 tokens 6.6 and 6.6, 2048 8.5 and 7.6. (At 513 tokens
    // six would be ahead for 8 x 192, 5.5 and 4.8 us, and behind for 8 x 96, 4.3 and 4.5.)
    const int nvec = a.group / 8;
    int w4 = 1, w6 = 1;
    while (4 * w4 < nvec) w4 *= 2;
    while (6 * w6 < nvec) w6 *= 2;
    const long long at_once = (long long)device_sm_count() * cache_write_ctas<T>(4) * CACHE_THREADS;
    const bool six = 6 * w6 < 4 * w4 && (long long)a.tokens * a.per_token.d * w4 > at_once;
    a.w = six ? w6 : w4;
    a.full = nvec == (six ? 6 : 4) * a.w && a.p[0].vec && (!a.p[1].x || a.p[1].vec);
    a.tb = cache_tokens_per_cta(a.tokens, (long long)a.per_token.d * a.w);
    const dim3 grid((a.tokens + a.tb - 1) / a.tb);
    if (six) return launch_kernel(cache_write_kernel<T, FMT, 6>, grid, dim3(CACHE_THREADS), 0, s, true, a);
    return launch_kernel(cache_write_kernel<T, FMT, 4>, grid, dim3(CACHE_THREADS), 0, s, true, a);
}
template <typename T>
inline int cache_write_fmt(CacheArgs &a, int format, cudaStream_t s) {
    switch (format) {
        case GPTQ_CACHE_INT4: return cache_write_launch<T, GPTQ_CACHE_INT4>(a, s);
        case GPTQ_CACHE_INT8: return cache_write_launch<T, GPTQ_CACHE_INT8>(a, s);
        default: return cache_write_launch<T, GPTQ_CACHE_E4M3>(a, s);
    }
}
inline int cache_write(CacheArgs &a, int x_dtype, int format, cudaStream_t s) {
    const int groups = a.dim / a.group, planes = a.p[1].x ? 2 : 1;
    a.per_head = fast_div(groups);
    a.per_plane = fast_div((uint32_t)a.heads * groups);
    a.per_token = fast_div((uint32_t)planes * a.heads * groups);
    a.per_group = fast_div(1);
    if (a.tokens > GPTQ_CACHE_UNCLAIMED) {
        if (int st = launch_kernel(cache_claim_kernel, dim3((a.tokens + 255) / 256), dim3(256), 0, s,
                                   true, a.slots, a.tokens, a.n_slots, a.claims))
            return st;
    } else {
        a.claims = nullptr;
    }
    switch (x_dtype) {
        case GPTQ_BF16: return cache_write_fmt<__nv_bfloat16>(a, format, s);
        case GPTQ_F16: return cache_write_fmt<__half>(a, format, s);
        default: return cache_write_fmt<float>(a, format, s);
    }
}

template <typename T, int U>
inline int cache_read_fmt(CacheArgs &a, int format, cudaStream_t s) {
    const dim3 grid((a.tokens + a.tb - 1) / a.tb), block(CACHE_THREADS);
    switch (format) {
        case GPTQ_CACHE_INT4:
            return launch_kernel(cache_read_kernel<T, GPTQ_CACHE_INT4, U>, grid, block, 0, s, true, a);
        case GPTQ_CACHE_INT8:
            return launch_kernel(cache_read_kernel<T, GPTQ_CACHE_INT8, U>, grid, block, 0, s, true, a);
        default:
            return launch_kernel(cache_read_kernel<T, GPTQ_CACHE_E4M3, U>, grid, block, 0, s, true, a);
    }
}
template <typename T>
inline int cache_read_type(CacheArgs &a, int format, int unit, cudaStream_t s) {
    return unit == 2 ? cache_read_fmt<T, 2>(a, format, s) : cache_read_fmt<T, 1>(a, format, s);
}
inline int cache_read(CacheArgs &a, int y_dtype, int format, cudaStream_t s) {
    const int planes = a.p[1].y ? 2 : 1;
    const int unit = a.dim % 16 == 0 && a.group % 16 == 0 ? 2 : 1;
    a.per_head = fast_div(a.dim / (8 * unit));
    a.per_plane = fast_div((uint32_t)a.heads * (a.dim / (8 * unit)));
    a.per_token = fast_div((uint32_t)planes * a.heads * (a.dim / (8 * unit)));
    a.per_group = fast_div(a.group / (8 * unit));
    a.tb = cache_tokens_per_cta(a.tokens, a.per_token.d);
    a.claims = nullptr;
    a.w = 1;
    // 16 codes at once
    a.vec = ((reinterpret_cast<uintptr_t>(a.p[0].codes) | reinterpret_cast<uintptr_t>(a.p[1].codes)) & 15u) == 0;
    switch (y_dtype) {
        case GPTQ_BF16: return cache_read_type<__nv_bfloat16>(a, format, unit, s);
        case GPTQ_F16: return cache_read_type<__half>(a, format, unit, s);
        default: return cache_read_type<float>(a, format, unit, s);
    }
}

}  // namespace serve
}  // namespace gptq
