// Device helpers shared by the scan's kernels.
//
// Thread layout of every scan kernel: K adjacent lanes hold one channel, each
// S = 4 of its states (n <= 4 K, the states behind n are zeros: a = 1, B = C
// = 0), so a CTA of NT threads holds NT / K channels and walks the tokens of
// one chunk. What depends on (token, channel) alone (the softplus, the gate)
// is computed once per element by another mapping of the threads, token-major
// and coalesced, and passed through shared memory.
#pragma once

#include <cfloat>

#include "ssm.h"

namespace la {

constexpr int SCAN_S = 4;            // states per thread
constexpr float SCAN_LOG2E = 1.4426950408889634f;
constexpr float SCAN_LN2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A log2 e, the decay's rate per dt. An infinite A (a state that forgets at once)
// is the lowest number, so that the dt of 0 that stands for a row behind a
// sequence's end is a decay of 1 there too. A dt of 126 2^-128 = 3.7e-37 or more
// still makes it 0; the decay of a smaller one is not.
__device__ __forceinline__ float decay_rate(float A)
{
    const float r = A * SCAN_LOG2E;
    return r < -FLT_MAX ? -FLT_MAX : r;
}

// Pairs of fp32 in one 64-bit register, for the packed instructions: one issue
// slot for two operations.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack(float a, float b)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(f2 v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 x)
{
    float a, b;
    unpack(x, a, b);
    return pack(ex2(a), ex2(b));
}

// sigmoid(x) = 1 / (1 + 2^(-x log2 e)); a large negative x gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid_f(float x)
{
    return rcp(1.f + ex2(-SCAN_LOG2E * x));
}

// exp(-|x|): the product |x| log2 e is rounded to fp32, an error of up to
// 2^-24 |x| log2 e in the exponent; its rest, from two multiply-adds more, is put
// back by a first-order factor. |x| counts as at most 100, which spares the case
// of an infinite product; from 87.34 on the result, below 2^-126, is 0.
__device__ __forceinline__ f2 exp_neg_abs2(float x, float y)
{
    constexpr float LO = 1.9259629e-8f;  // log2 e - fp32(log2 e)
    const f2 t = pack(fminf(fabsf(x), 100.f), fminf(fabsf(y), 100.f));
    const f2 c = pack(-SCAN_LOG2E, -SCAN_LOG2E);
    const f2 hi = mul2(t, c);
    const f2 lo = fma2(t, pack(-LO, -LO), fma2(t, c, mul2(hi, pack(-1.f, -1.f))));
    const f2 e = ex2_2(hi);
    return fma2(mul2(e, lo), pack(SCAN_LN2, SCAN_LN2), e);
}
// max(x, 0), NaN for NaN.
__device__ __forceinline__ float relu_nan(float x)
{
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
    return r;
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) <= 1. The logarithm by
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, which keeps the relative
// precision of small results. atanh(s) / s is a polynomial of degree 4 in q = s^2
// <= 1/9, a minimax fit (Remez exchange) whose constant term was then set to 1;
// its relative error is between -8.0e-9 and 5e-10. Where e is 0 (x below -87.34)
// so is the result. The derivative, sigmoid(x), is 1 / (1 + e) or e / (1 + e).
__device__ __forceinline__ f2 atanh_ratio(f2 q)
{
    f2 p = fma2(q, pack(0.14095774f, 0.14095774f), pack(0.13978833f, 0.13978833f));
    p = fma2(p, q, pack(0.20012558f, 0.20012558f));
    p = fma2(p, q, pack(0.33333156f, 0.33333156f));
    return fma2(p, q, pack(1.f, 1.f));
}
__device__ __forceinline__ f2 log1p_part(f2 e)
{
    float a, b;
    unpack(add2(e, pack(2.f, 2.f)), a, b);
    const f2 s = mul2(e, pack(rcp(a), rcp(b)));
    return mul2(mul2(s, pack(2.f, 2.f)), atanh_ratio(mul2(s, s)));
}
__device__ __forceinline__ f2 softplus2(f2 v)
{
    float x, y;
    unpack(v, x, y);
    return add2(log1p_part(exp_neg_abs2(x, y)), pack(relu_nan(x), relu_nan(y)));
}
// With its derivative.
__device__ __forceinline__ f2 softplus2(f2 v, f2& slope)
{
    float x, y, e0, e1, a, b;
    unpack(v, x, y);
    const f2 e = exp_neg_abs2(x, y);
    unpack(e, e0, e1);
    unpack(add2(e, pack(1.f, 1.f)), a, b);
    // x < 0: e / (1 + e); NaN: itself
    slope = mul2(pack(rcp(a), rcp(b)), pack(x >= 0.f ? 1.f : x < 0.f ? e0 : x,
                                            y >= 0.f ? 1.f : y < 0.f ? e1 : y));
    return add2(log1p_part(e), pack(relu_nan(x), relu_nan(y)));
}
__device__ __forceinline__ float softplus_f(float x)
{
    float y, unused;
    unpack(softplus2(pack(x, 0.f)), y, unused);
    return y;
}
__device__ __forceinline__ f2 sigmoid2(f2 x)
{
    float a, b;
    unpack(add2(ex2_2(mul2(x, pack(-SCAN_LOG2E, -SCAN_LOG2E))), pack(1.f, 1.f)), a, b);
    return pack(rcp(a), rcp(b));
}
// Sum V values over the M lanes that differ in the bits [STEP, STEP M) of the
// lane number. Each step halves the values that a lane keeps, so V values
// cost about V shuffles instead of V log2 M. On return lane l holds, in v[0
// .. V/min(V,M) ), the totals with the indices that `reduced_index` names.
template <int V, int M, int STEP>
__device__ __forceinline__ void lane_reduce(float* v, int lane)
{
    int count = V;
#pragma unroll
    for (int m = M / 2; m >= 1; m >>= 1) {
        const int bit = m * STEP;
        if (count > 1) {
            count >>= 1;
            const bool up = lane & bit;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                if (i < count) {
                    const float send = up ? v[i] : v[i + count];
                    const float keep = up ? v[i + count] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
        }
    }
}
// Index of the first value that a lane holds after lane_reduce<V, M, STEP>.
template <int V, int M, int STEP> __device__ __forceinline__ int reduced_index(int lane)
{
    int count = V, at = 0;
#pragma unroll
    for (int m = M / 2; m >= 1; m >>= 1) {
        if (count > 1) {
            count >>= 1;
            if (lane & (m * STEP)) at += count;
        }
    }
    return at;
}
// Whether a lane is the one that writes (more lanes than values hold copies).
template <int V, int M, int STEP> __device__ __forceinline__ bool reduced_writer(int lane)
{
    return M <= V || (lane & ((M / V - 1) * STEP)) == 0;
}

// Two adjacent channels of a token as loaded: one access where VEC (every row
// of every tensor then starts on such a pair), else two.
template <typename T, bool VEC> struct Pair;
template <bool VEC> struct Pair<__nv_bfloat16, VEC> {
    uint32_t w;
    __device__ __forceinline__ void load(const char* p, uint32_t next)
    {
        if (VEC) w = *reinterpret_cast<const uint32_t*>(p);
        else w = *reinterpret_cast<const uint16_t*>(p) |
                 (uint32_t) * reinterpret_cast<const uint16_t*>(p + next) << 16;
    }
    __device__ __forceinline__ f2 get() const
    {
        return pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};
template <bool VEC> struct Pair<float, VEC> {
    f2 v;
    __device__ __forceinline__ void load(const char* p, uint32_t next)
    {
        if (VEC) v = *reinterpret_cast<const f2*>(p);
        else v = pack(*reinterpret_cast<const float*>(p), *reinterpret_cast<const float*>(p + next));
    }
    __device__ __forceinline__ f2 get() const { return v; }
};

// Four states of one channel at p (n of them in all, this thread's start at
// m0); vectors when a row of n states keeps 16-byte alignment. FULL: n is known
// to be a multiple of four above m0.
template <bool FULL = false>
__device__ __forceinline__ void load_states(float* v, const float* p, int m0, int n)
{
    if (FULL || (n & 3) == 0) {
        const float4 x = FULL || m0 < n ? *reinterpret_cast<const float4*>(p + m0) : make_float4(0, 0, 0, 0);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = m0 + i < n ? p[m0 + i] : 0.f;
    }
}
template <bool FULL = false>
__device__ __forceinline__ void store_states(float* p, const float* v, int m0, int n)
{
    if (FULL || (n & 3) == 0) {
        if (FULL || m0 < n) *reinterpret_cast<float4*>(p + m0) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (m0 + i < n) p[m0 + i] = v[i];
    }
}

// Lanes per channel for n states.
inline int scan_lanes(int n) { return n <= 4 ? 1 : n <= 8 ? 2 : n <= 16 ? 4 : n <= 32 ? 8 : 16; }

#define LA_SCAN_DISPATCH_K(n, CALL)                                                              \
    switch (scan_lanes(n)) {                                                                     \
    case 1: CALL(1); break;                                                                      \
    case 2: CALL(2); break;                                                                      \
    case 4: CALL(4); break;                                                                      \
    case 8: CALL(8); break;                                                                      \
    default: CALL(16); break;                                                                    \
    }

}  // namespace la
