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
#include "ssm.h"

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

// Sum over a row's TPR threads, in a fixed order; `red` has a slot per warp.
template <int TPR> __device__ __forceinline__ float row_sum(float v, float* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v += red[i];
    }
    return v;
}

template <typename T, typename To, int TPR, int NT, int V, int CH>
__global__ void __launch_bounds__(NT) norm_kernel(const T* x, const float* __restrict__ weight,
                                                  const float* __restrict__ bias, float eps,
                                                  To* y, float* mean, float* rstd,
                                                  long long rows, int F)
{
    __shared__ float red[2][NT / 32];
    const int tid = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
    if (row >= rows) return;  // whole warps: rows share a CTA only when TPR is a warp
    const T* xr = x + row * F;
    Vec<T, V> xs[CH];
    float sum = 0.f;
#pragma unroll
    for (int m = 0; m < CH; ++m) {
        const int c = (tid + TPR * m) * V;
        if (c < F) xs[m].load(xr + c);
    }
#pragma unroll
    for (int m = 0; m < CH; ++m)
        if ((tid + TPR * m) * V < F) {
#pragma unroll
            for (int i = 0; i < V; ++i) sum += xs[m].get(i);
        }
    const float mu = row_sum<TPR>(sum, red[0]) / F;
    float sq = 0.f;
#pragma unroll
    for (int m = 0; m < CH; ++m)
        if ((tid + TPR * m) * V < F) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = xs[m].get(i) - mu;
                sq = fmaf(d, d, sq);
            }
        }
    const float rs = rsqrtf(row_sum<TPR>(sq, red[1]) / F + eps);
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

template <typename T, typename To, int TPR, int NT, int V, int CH>
__global__ void __launch_bounds__(NT) norm_backward_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ weight,
    const float* __restrict__ mean, const float* __restrict__ rstd, To* __restrict__ dx,
    float* __restrict__ dw_part, float* __restrict__ db_part, long long rows, int F)
{
    __shared__ float red[2][2][NT / 32];
    const int tid = threadIdx.x % TPR;
    const int strand = blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
    const int strands = gridDim.x * (NT / TPR);
    float dw[CH][V], db[CH][V];
#pragma unroll
    for (int m = 0; m < CH; ++m)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[m][i] = db[m][i] = 0.f;
    int turn = 0;
#pragma unroll 1
    for (long long row = strand; row < rows; row += strands, turn ^= 1) {
        Vec<T, V> xs[CH], gs[CH];
#pragma unroll
        for (int m = 0; m < CH; ++m) {
            const int c = (tid + TPR * m) * V;
            if (c < F) {
                xs[m].load(x + row * F + c);
                gs[m].load(dy + row * F + c);
            }
        }
        const float mu = mean[row], rs = rstd[row];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int m = 0; m < CH; ++m) {
            const int c = (tid + TPR * m) * V;
            if (c < F) {
                float w[V];
                load_weights<V>(w, weight + c);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float v = (xs[m].get(i) - mu) * rs, g = gs[m].get(i);
                    const float e = g * w[i];
                    s1 += e;
                    s2 = fmaf(e, v, s2);
                    dw[m][i] = fmaf(g, v, dw[m][i]);
                    db[m][i] += g;
                }
            }
        }
        // Two alternating sets of slots: a warp may be a row ahead of another.
        s1 = row_sum<TPR>(s1, red[turn][0]);
        s2 = row_sum<TPR>(s2, red[turn][1]);
        const float m1 = s1 / F, m2 = s2 / F;
#pragma unroll
        for (int m = 0; m < CH; ++m) {
            const int c = (tid + TPR * m) * V;
            if (c < F) {
                float out[V], w[V];
                load_weights<V>(w, weight + c);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float v = (xs[m].get(i) - mu) * rs;
                    out[i] = rs * (gs[m].get(i) * w[i] - m1 - v * m2);
                }
                store_vec<To, V>(dx + row * F + c, out);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < CH; ++m) {
        const int c = (tid + TPR * m) * V;
        if (c < F) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dw_part[(long long)strand * F + c + i] = dw[m][i];
                db_part[(long long)strand * F + c + i] = db[m][i];
            }
        }
    }
}

// Partial rows of the backward: one per strand of rows. Two CTAs per SM; a
// warp-per-row CTA holds four strands.
int back_strands(long long rows, int F)
{
    const long long most = F <= 512 ? 148 * 8 : 148 * 2;
    long long n = rows < most ? rows : most;
    if (F <= 512) n = (n + 3) / 4 * 4;
    return (int)n;
}

}  // namespace

size_t norm_backward_workspace(long long rows, int F)
{
    return 2 * align_up((size_t)back_strands(rows, F) * F * 4, 256);
}

// Threads per row so that a thread holds at most 32 elements.
#define LA_NORM_FORWARD(T, To, V)                                                                \
    do {                                                                                         \
        if (F <= 1024) LA_CALL(T, To, 32, 128, V, 32 / V);                                       \
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

// At most 16 elements per thread: a row, its gradient and two sums per column.
#define LA_NORM_BACKWARD(T, To, V)                                                               \
    do {                                                                                         \
        if (F <= 512) LA_CALL(T, To, 32, 128, V, 16 / V);                                        \
        else if (F <= 2048) LA_CALL(T, To, 128, 128, V, 16 / V);                                 \
        else if (F <= 4096) LA_CALL(T, To, 256, 256, V, 16 / V);                                 \
        else if (F <= 8192) LA_CALL(T, To, 512, 512, V, 16 / V);                                 \
        else LA_CALL(T, To, 1024, 1024, V, 16 / V);                                              \
    } while (0)

cudaError_t launch_layer_norm_backward(const void* dy, const void* x, const float* weight,
                                       const float* mean, const float* rstd, void* dx,
                                       float* dweight, float* dbias, long long rows, int F,
                                       int in_t, int out_t, void* ws, cudaStream_t stream)
{
    const int strands = back_strands(rows, F);
    float* dw = (float*)ws;
    float* db = (float*)((char*)ws + align_up((size_t)strands * F * 4, 256));
    if (rows > 0) {
#define LA_CALL(T, To, TPR, NT, V, CH)                                                           \
    norm_backward_kernel<T, To, TPR, NT, V, CH><<<strands / (NT / TPR), NT, 0, stream>>>(        \
        (const T*)dy, (const T*)x, weight, mean, rstd, (To*)dx, dw, db, rows, F)
        LA_NORM_TYPES(LA_NORM_BACKWARD)
#undef LA_CALL
        count_launch();
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_column_sum(dw, dweight, strands, F, stream);
    if (e == cudaSuccess && dbias) e = launch_column_sum(db, dbias, strands, F, stream);
    return e;
}

}  // namespace la
