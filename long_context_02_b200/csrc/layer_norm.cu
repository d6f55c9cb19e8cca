// Layer norm forward and backward (formulas in lightning.h).
//
// Streams bound by HBM. A row is held in registers by TPR threads (a warp for
// short rows, so that no barrier is needed), at most PER elements each, loaded
// once: the mean, then the centred sum of squares, then the output come from
// the registers. Rows are read in 16-byte vectors when F allows, else element
// by element.
//
// Backward: the row's two means give dx; dweight and dbias are sums down the
// columns, which a CTA gathers in registers over the rows it walks and writes
// as one partial row each; a second launch adds the partial rows.
#include "ssm_scan.cuh"

namespace la {
namespace {

template <typename T, int V> struct Vec {
    T e[V];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (V * sizeof(T) == 16)
            *reinterpret_cast<uint4*>(e) = __ldcs(reinterpret_cast<const uint4*>(p));
        else e[0] = *p;
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(e[i]); }
};

template <typename T, int V> __device__ __forceinline__ void store_vec(T* p, const float* v)
{
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 2) {
        __align__(16) __nv_bfloat162 h[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<uint4*>(h));
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            __stcs(reinterpret_cast<float4*>(p + i), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
    }
}

// V weights from p on; in vectors when V allows.
template <int V> __device__ __forceinline__ void load_weights(float* v, const float* p)
{
    if constexpr (V == 1) {
        v[0] = __ldg(p);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(v + i) = __ldg(reinterpret_cast<const float4*>(p + i));
    }
}

// V elements at p as pairs.
template <typename T, int V> __device__ __forceinline__ void load_pairs(f2* v, const T* p)
{
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        if constexpr (sizeof(T) == 2)
            v[i] = pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else v[i] = pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
}

// 16 bytes to shared memory, asynchronously.
__device__ __forceinline__ void copy16(void* to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from)
                 : "memory");
}

// Sum over a warp.
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T, typename To, int TPR, int NT, int V, int CH>
__global__ void __launch_bounds__(NT) norm_kernel(const T* x, const float* __restrict__ weight,
                                                  const float* __restrict__ bias, float eps,
                                                  To* y, float* mean, float* rstd,
                                                  long long rows, int F)
{
    __shared__ float3 part[NT / 32];  // of each warp: elements, mean, centred squares
    const int tid = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
    if (row >= rows) return;  // whole warps: rows share a CTA only when TPR is a warp
    const T* xr = x + row * F;
    Vec<T, V> xs[CH];
    float sum = 0.f, count = 0.f;
#pragma unroll
    for (int m = 0; m < CH; ++m) {
        const int c = (tid + TPR * m) * V;
        if (c < F) xs[m].load(xr + c);
    }
#pragma unroll
    for (int m = 0; m < CH; ++m)
        if ((tid + TPR * m) * V < F) {
            count += V;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += xs[m].get(i);
        }
    // Each warp's mean and squares about it; with N_w, m_w, q_w of the warps the
    // row's mean is sum N_w m_w / F and its squares sum q_w + N_w (m_w - mean)^2,
    // so that one barrier serves both.
    sum = warp_sum(sum);
    if (TPR > 32) count = warp_sum(count);
    float mu = TPR > 32 ? (count > 0.f ? sum / count : 0.f) : sum / F, sq = 0.f;
#pragma unroll
    for (int m = 0; m < CH; ++m)
        if ((tid + TPR * m) * V < F) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = xs[m].get(i) - mu;
                sq = fmaf(d, d, sq);
            }
        }
    sq = warp_sum(sq);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float3(count, mu, sq);
        __syncthreads();
        mu = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) mu = fmaf(part[i].x, part[i].y, mu);
        mu /= F;
        sq = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) {
            const float d = part[i].y - mu;
            sq += fmaf(part[i].x * d, d, part[i].z);
        }
    }
    const float rs = rsqrtf(sq / F + eps);
#pragma unroll
    for (int m = 0; m < CH; ++m) {
        const int c = (tid + TPR * m) * V;
        if (c < F) {
            float out[V], w[V], b[V];
            load_weights<V>(w, weight + c);
            if (bias) load_weights<V>(b, bias + c);
#pragma unroll
            for (int i = 0; i < V; ++i)
                out[i] = fmaf((xs[m].get(i) - mu) * rs, w[i], bias ? b[i] : 0.f);
            store_vec<To, V>(y + row * F + c, out);
        }
    }
    if (mean && tid == 0) {
        mean[row] = mu;
        rstd[row] = rs;
    }
}

// One CTA walks every `gridDim.x`-th row. Its rows come through shared memory,
// STAGES - 1 of them on their way while one is worked on; each thread copies
// the elements that it will use itself, so that only the row's two sums need a
// barrier. With one stage (where F allows no vectors, or shared memory does not
// hold two rows of each) the rows are loaded directly.
template <typename T, typename To, int NT, int V, int CH, int STAGES>
__global__ void __launch_bounds__(NT) norm_backward_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ weight,
    const float* __restrict__ mean, const float* __restrict__ rstd, To* __restrict__ dx,
    float* __restrict__ dw_part, float* __restrict__ db_part, long long rows, int F)
{
    constexpr int H = (V * CH + 1) / 2;  // pairs of elements per thread
    constexpr bool VECTORS = V > 1, RING = STAGES > 1;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float2 red[2][NT / 32];
    const int tid = threadIdx.x;
    const f2 zero = pack(0.f, 0.f);
    f2 dw[H], db[H], w[H];
#pragma unroll
    for (int h = 0; h < H; ++h) dw[h] = db[h] = w[h] = zero;
#pragma unroll
    for (int m = 0; m < CH; ++m) {
        const int c = (tid + NT * m) * V;
        if constexpr (VECTORS) {
            float v[V];
            if (c < F) {
                load_weights<V>(v, weight + c);
#pragma unroll
                for (int i = 0; i < V; i += 2) w[(m * V + i) / 2] = pack(v[i], v[i + 1]);
            }
        }
    }
    if constexpr (!VECTORS) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int c0 = tid + NT * 2 * h, c1 = c0 + NT;
            w[h] = pack(c0 < F ? weight[c0] : 0.f, c1 < F ? weight[c1] : 0.f);
        }
    }
    // stage s: this CTA's row of x, then of dy
    T* const ring = reinterpret_cast<T*>(smem);
    auto fetch = [&](int stage, long long row) {
        if constexpr (RING) {
            if (row < rows) {
#pragma unroll
                for (int m = 0; m < CH; ++m) {
                    const int c = (tid + NT * m) * V;
                    if (c < F) {
                        copy16(ring + (long long)(2 * stage) * F + c, x + row * F + c);
                        copy16(ring + (long long)(2 * stage + 1) * F + c, dy + row * F + c);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    const long long step = gridDim.x;
    long long row = blockIdx.x;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) fetch(s, row + s * step);
    float mu = row < rows ? mean[row] : 0.f, rs = row < rows ? rstd[row] : 0.f;
    int stage = 0, turn = 0;
#pragma unroll 1
    for (; row < rows; row += step, turn ^= 1) {
        const long long next = row + step;
        const float mu_next = next < rows ? mean[next] : 0.f;
        const float rs_next = next < rows ? rstd[next] : 0.f;
        f2 xv[H], gv[H];
        if constexpr (VECTORS) {
            const T *xr = x + row * F, *gr = dy + row * F;
            if constexpr (RING) {
                asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
                xr = ring + (long long)(2 * stage) * F;
                gr = xr + F;
            }
#pragma unroll
            for (int m = 0; m < CH; ++m) {
                const int c = (tid + NT * m) * V;
#pragma unroll
                for (int i = 0; i < V / 2; ++i) xv[m * V / 2 + i] = gv[m * V / 2 + i] = zero;
                if (c < F) {
                    load_pairs<T, V>(xv + m * V / 2, xr + c);
                    load_pairs<T, V>(gv + m * V / 2, gr + c);
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int c0 = tid + NT * 2 * h, c1 = c0 + NT;
                const T *xr = x + row * F, *gr = dy + row * F;
                xv[h] = pack(c0 < F ? to_f32(xr[c0]) : 0.f, c1 < F ? to_f32(xr[c1]) : 0.f);
                gv[h] = pack(c0 < F ? to_f32(gr[c0]) : 0.f, c1 < F ? to_f32(gr[c1]) : 0.f);
            }
        }
        // The stage before this one was used up a row ago.
        fetch((stage + STAGES - 1) % STAGES, row + (STAGES - 1) * step);
        const f2 minus_mu = pack(-mu, -mu), scale = pack(rs, rs);
        f2 s1 = zero, s2 = zero;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            xv[h] = mul2(add2(xv[h], minus_mu), scale);
            dw[h] = fma2(gv[h], xv[h], dw[h]);
            db[h] = add2(db[h], gv[h]);
            gv[h] = mul2(gv[h], w[h]);
            s1 = add2(s1, gv[h]);
            s2 = fma2(gv[h], xv[h], s2);
        }
        float a0, a1, b0, b1;
        unpack(s1, a0, a1);
        unpack(s2, b0, b1);
        float m1 = warp_sum(a0 + a1), m2 = warp_sum(b0 + b1);
        if constexpr (NT > 32) {
            // Two sets of slots in turn: a warp may be a row ahead of another.
            if ((tid & 31) == 0) red[turn][tid >> 5] = make_float2(m1, m2);
            __syncthreads();
            m1 = m2 = 0.f;
#pragma unroll
            for (int i = 0; i < NT / 32; ++i) m1 += red[turn][i].x, m2 += red[turn][i].y;
        }
        m1 /= F;
        m2 /= F;
        const f2 minus_m1 = pack(-m1, -m1), minus_m2 = pack(-m2, -m2);
#pragma unroll
        for (int h = 0; h < H; ++h)
            xv[h] = mul2(fma2(xv[h], minus_m2, add2(gv[h], minus_m1)), scale);
        To* const out = dx + row * F;
        if constexpr (VECTORS) {
#pragma unroll
            for (int m = 0; m < CH; ++m) {
                const int c = (tid + NT * m) * V;
                if (c < F) {
                    float v[V];
#pragma unroll
                    for (int i = 0; i < V; i += 2) unpack(xv[(m * V + i) / 2], v[i], v[i + 1]);
                    store_vec<To, V>(out + c, v);
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int c0 = tid + NT * 2 * h, c1 = c0 + NT;
                float v0, v1;
                unpack(xv[h], v0, v1);
                if (c0 < F) out[c0] = from_f32<To>(v0);
                if (c1 < F) out[c1] = from_f32<To>(v1);
            }
        }
        mu = mu_next;
        rs = rs_next;
        stage = (stage + 1) % STAGES;
    }
    float* const dwp = dw_part + (long long)blockIdx.x * F;
    float* const dbp = db_part + (long long)blockIdx.x * F;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        float w0, w1, b0, b1;
        unpack(dw[h], w0, w1);
        unpack(db[h], b0, b1);
        if constexpr (VECTORS) {
            const int m = 2 * h / V, c = (tid + NT * m) * V + 2 * h % V;
            if (c < F) {
                *reinterpret_cast<float2*>(dwp + c) = make_float2(w0, w1);
                *reinterpret_cast<float2*>(dbp + c) = make_float2(b0, b1);
            }
        } else {
            const int c0 = tid + NT * 2 * h, c1 = c0 + NT;
            if (c0 < F) dwp[c0] = w0, dbp[c0] = b0;
            if (c1 < F) dwp[c1] = w1, dbp[c1] = b1;
        }
    }
}

// Threads of the backward, for at most 16 elements each (a row's, its gradient's
// and two sums per column are in registers).
int back_threads(int F)
{
    return F <= 512 ? 32 : F <= 2048 ? 128 : F <= 4096 ? 256 : F <= 8192 ? 512 : 1024;
}

// Stages of the backward's ring: what fits beside the SM's other CTAs.
template <typename T> constexpr int stages(int V, int nt)
{
    return V == 1 ? 1 : sizeof(T) == 2 ? (nt > 512 ? 3 : 4) : (nt > 512 ? 1 : 3);
}

// CTAs of the backward, each with a partial row of dweight and dbias: as many as
// are resident at once, 512 threads per SM (1024 where a row takes them).
int back_ctas(long long rows, int F)
{
    const int nt = back_threads(F), per_sm = nt >= 512 ? 1 : 512 / nt;
    return (int)(rows < 148LL * per_sm ? rows : 148LL * per_sm);
}

}  // namespace

size_t norm_backward_workspace(long long rows, int F)
{
    return 2 * align_up((size_t)back_ctas(rows, F) * F * 4, 256);
}

// Threads per row so that a thread holds at most 32 elements.
#define LA_NORM_FORWARD(T, To, V)                                                                \
    do {                                                                                         \
        if (F <= 1024) LA_CALL(T, To, 32, 128, V, 32 / V);                                       \
        else if (F <= 2048) LA_CALL(T, To, 32, 128, V, 64 / V);                                  \
        else if (F <= 4096) LA_CALL(T, To, 128, 128, V, 32 / V);                                 \
        else if (F <= 8192) LA_CALL(T, To, 256, 256, V, 32 / V);                                 \
        else LA_CALL(T, To, 512, 512, V, 32 / V);                                                \
    } while (0)
#define LA_NORM_TYPES(SIZES)                                                                     \
    if (in_t == LA_F32) { if (F % 4 == 0) SIZES(float, float, 4); else SIZES(float, float, 1); } \
    else if (out_t == LA_F32) {                                                                  \
        if (F % 8 == 0) SIZES(__nv_bfloat16, float, 8); else SIZES(__nv_bfloat16, float, 1);     \
    } else {                                                                                     \
        if (F % 8 == 0) SIZES(__nv_bfloat16, __nv_bfloat16, 8);                                  \
        else SIZES(__nv_bfloat16, __nv_bfloat16, 1);                                             \
    }

cudaError_t launch_layer_norm(const void* x, const float* weight, const float* bias, float eps,
                              void* y, float* mean, float* rstd, long long rows, int F, int in_t,
                              int out_t, cudaStream_t stream)
{
#define LA_CALL(T, To, TPR, NT, V, CH)                                                           \
    norm_kernel<T, To, TPR, NT, V, CH>                                                           \
        <<<(unsigned)((rows + NT / TPR - 1) / (NT / TPR)), NT, 0, stream>>>(                     \
            (const T*)x, weight, bias, eps, (To*)y, mean, rstd, rows, F)
    LA_NORM_TYPES(LA_NORM_FORWARD)
#undef LA_CALL
    count_launch();
    return cudaGetLastError();
}

#define LA_NORM_BACKWARD(T, To, V)                                                               \
    do {                                                                                         \
        switch (back_threads(F)) {                                                               \
        case 32: LA_CALL(T, To, 32, V, 16 / V, stages<T>(V, 32)); break;                         \
        case 128: LA_CALL(T, To, 128, V, 16 / V, stages<T>(V, 128)); break;                      \
        case 256: LA_CALL(T, To, 256, V, 16 / V, stages<T>(V, 256)); break;                      \
        case 512: LA_CALL(T, To, 512, V, 16 / V, stages<T>(V, 512)); break;                      \
        default: LA_CALL(T, To, 1024, V, 16 / V, stages<T>(V, 1024)); break;                     \
        }                                                                                        \
    } while (0)

// A launch with the ring's shared memory (two rows per stage).
template <typename T, typename To, int NT, int V, int CH, int STAGES>
cudaError_t launch_backward(const void* dy, const void* x, const float* weight, const float* mean,
                            const float* rstd, void* dx, float* dw, float* db, long long rows,
                            int F, int ctas, cudaStream_t stream)
{
    auto kernel = norm_backward_kernel<T, To, NT, V, CH, STAGES>;
    const int smem = STAGES > 1 ? STAGES * 2 * F * (int)sizeof(T) : 0;
    if (smem > 40 * 1024) {  // beside the static slots of the sums
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<ctas, NT, smem, stream>>>((const T*)dy, (const T*)x, weight, mean, rstd, (To*)dx, dw,
                                       db, rows, F);
    return cudaGetLastError();
}

cudaError_t launch_layer_norm_backward(const void* dy, const void* x, const float* weight,
                                       const float* mean, const float* rstd, void* dx,
                                       float* dweight, float* dbias, long long rows, int F,
                                       int in_t, int out_t, void* ws, cudaStream_t stream)
{
    const int ctas = back_ctas(rows, F);
    float* dw = (float*)ws;
    float* db = (float*)((char*)ws + align_up((size_t)ctas * F * 4, 256));
    if (rows > 0) {
        cudaError_t e;
#define LA_CALL(T, To, NT, V, CH, STAGES)                                                        \
    e = launch_backward<T, To, NT, V, CH, STAGES>(dy, x, weight, mean, rstd, dx, dw, db, rows, F, \
                                                  ctas, stream)
        LA_NORM_TYPES(LA_NORM_BACKWARD)
#undef LA_CALL
        count_launch();
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_column_sum(dw, dweight, ctas, F, stream);
    if (e == cudaSuccess && dbias) e = launch_column_sum(db, dbias, ctas, F, stream);
    return e;
}

}  // namespace la
