// Layer norm forward and backward (formulas in lightning.h).
//
// Streams bound by HBM. Rows are read once, in 16-byte vectors when F allows,
// else element by element; the mean, the centred squares and the output come
// from registers or shared memory. Up to 1024 features (2048 for few rows) a
// warp holds a row, so that no barrier is needed; beyond, a CTA does. Many rows
// are walked by CTAs that stay, several rows at a time, with the weights in
// registers (they are fp32, twice as wide as bf16 rows) and the next rows on
// their way into shared memory: a grid of one CTA per row took 230-310 us where
// this takes 185-203 (32K rows of 8192, bf16, 5.3-5.8 TB/s).
//
// Backward: the row's two means give dx; dweight and dbias are sums down the
// columns, which a CTA gathers in registers over the rows it walks and writes
// as one partial row each; a second launch adds the partial rows. 16K rows of
// 8192, bf16: 154-168 us, 4.8-5.2 TB/s.
//
// Beyond 8192 features 1024 threads leave 64 registers each: the ring spills (bf16
// 220 to 228 bytes stored, fp32 32) and the backward too (272 in bf16, 384 in
// fp32, which has no ring there; 400 to 420 without vectors). Widths that are no
// whole vectors, 8 in bf16 or 4 in fp32, take single elements and no ring however
// many rows there are.
#include "ssm_scan.cuh"

namespace la {
namespace {

constexpr int MOST_SHARED = 200 * 1024;  // of dynamic shared memory that a ring asks for

// From so many rows on the forward pass walks them through shared memory.
constexpr long long LA_RING_ROWS = 148 * 8;

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

// A thread's share of a row, as stored: CH vectors of V elements, TPR vectors
// apart; read as pairs. Without vectors (V = 1) a pair is two elements TPR apart.
// Elements behind the row's end are zeros.
template <typename T, int TPR, int V, int CH> struct Share {
    static constexpr int H = (V * CH + 1) / 2;
    static constexpr int N = V == 1 ? CH : CH * V * (int)sizeof(T) / 4;
    uint32_t w[N];

    // Column of a half of pair h.
    __device__ __forceinline__ static int column(int tid, int h, int half)
    {
        return V == 1 ? tid + TPR * (2 * h + half) : (tid + TPR * (2 * h / V)) * V + 2 * h % V + half;
    }
    __device__ __forceinline__ void load(const T* p, int tid, int F)
    {
#pragma unroll
        for (int m = 0; m < CH; ++m) {
            const int c = (tid + TPR * m) * V;
            if constexpr (V == 1) {
                const float v = c < F ? to_f32(p[c]) : 0.f;
                w[m] = __float_as_uint(v);
            } else {
                uint4 q = make_uint4(0, 0, 0, 0);
                if (c < F) q = __ldcs(reinterpret_cast<const uint4*>(p + c));
                w[4 * m] = q.x, w[4 * m + 1] = q.y, w[4 * m + 2] = q.z, w[4 * m + 3] = q.w;
            }
        }
    }
    __device__ __forceinline__ f2 get(int h) const
    {
        if constexpr (V > 1 && sizeof(T) == 2)
            return pack(__uint_as_float(w[h] << 16), __uint_as_float(w[h] & 0xffff0000u));
        else
            return pack(__uint_as_float(w[2 * h]),
                        2 * h + 1 < N ? __uint_as_float(w[2 * h + 1]) : 0.f);
    }
    __device__ __forceinline__ f2 sum() const
    {
        f2 s = get(0);
#pragma unroll
        for (int h = 1; h < H; ++h) s = add2(s, get(h));
        return s;
    }
    // Squares about `mean`; pairs behind the row's end (or halves, without
    // vectors) do not count.
    __device__ __forceinline__ f2 squares(float mean, int tid, int F) const
    {
        f2 s = pack(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            f2 d = add2(get(h), pack(-mean, -mean));
            if (V == 1) {
                float a, b;
                unpack(d, a, b);
                d = pack(column(tid, h, 0) < F ? a : 0.f, column(tid, h, 1) < F ? b : 0.f);
                s = fma2(d, d, s);
            } else if (column(tid, h, 0) < F) {
                s = fma2(d, d, s);
            }
        }
        return s;
    }
};
// y = (x - mean) rstd weight + bias of R rows' shares; the weights are read once.
template <typename T, typename To, int TPR, int V, int CH, int R>
__device__ __forceinline__ void write_rows(const Share<T, TPR, V, CH>* xs, To* y,
                                           const float* weight, const float* bias, const float* mean,
                                           const float* rstd, int tid, int rows, int F)
{
#pragma unroll
    for (int m = 0; m < (V == 1 ? CH / 2 : CH); ++m) {
        constexpr int P = V == 1 ? 1 : V / 2;  // pairs
        const int c = V == 1 ? tid + TPR * 2 * m : (tid + TPR * m) * V;
        if (c >= F) continue;
        f2 w[P], b[P];
        const int next = c + TPR;  // the second of a pair without vectors
        if constexpr (V == 1) {
            w[0] = pack(weight[c], next < F ? weight[next] : 0.f);
            b[0] = pack(bias ? bias[c] : 0.f, bias && next < F ? bias[next] : 0.f);
        } else {
            float v[V];
            load_weights<V>(v, weight + c);
#pragma unroll
            for (int i = 0; i < P; ++i) w[i] = pack(v[2 * i], v[2 * i + 1]), b[i] = pack(0.f, 0.f);
            if (bias) {
                load_weights<V>(v, bias + c);
#pragma unroll
                for (int i = 0; i < P; ++i) b[i] = pack(v[2 * i], v[2 * i + 1]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= rows) continue;
            float out[2 * P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const f2 v = mul2(add2(xs[r].get(m * P + i), pack(-mean[r], -mean[r])),
                                  pack(rstd[r], rstd[r]));
                unpack(fma2(v, w[i], b[i]), out[2 * i], out[2 * i + 1]);
            }
            To* const p = y + (long long)r * F;
            if constexpr (V == 1) {
                p[c] = from_f32<To>(out[0]);
                if (next < F) p[next] = from_f32<To>(out[1]);
            } else {
                store_vec<To, V>(p + c, out);
            }
        }
    }
}

// 16 bytes of a row as stored, V elements; read as pairs.
template <typename T, int V> struct Raw {
    uint4 q;
    __device__ __forceinline__ void load(const T* p, bool ok)
    {
        q = make_uint4(0, 0, 0, 0);
        if (ok) q = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ f2 get(int i) const
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        if constexpr (sizeof(T) == 2)
            return pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else return pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

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

// One warp per row.
template <typename T, typename To, int V, int CH>
__global__ void __launch_bounds__(128) norm_warp_kernel(const T* x, const float* __restrict__ weight,
                                                        const float* __restrict__ bias, float eps,
                                                        To* y, float* mean, float* rstd,
                                                        long long rows, int F)
{
    const int tid = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    Share<T, 32, V, CH> xs;
    xs.load(x + row * F, tid, F);
    float a, b;
    unpack(xs.sum(), a, b);
    const float mu = warp_sum(a + b) / F;
    unpack(xs.squares(mu, tid, F), a, b);
    const float rs = rsqrtf(warp_sum(a + b) / F + eps);
    write_rows<T, To, 32, V, CH, 1>(&xs, y + row * F, weight, bias, &mu, &rs, tid, 1, F);
    if (mean && tid == 0) {
        mean[row] = mu;
        rstd[row] = rs;
    }
}

// Totals of R values over the CTA's warps: lane l reads warp l's.
template <int NW, int R> __device__ __forceinline__ void across_warps(float* v)
{
#pragma unroll
    for (int o = NW / 2; o >= 1; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
}

// One CTA per row, 16 elements per thread. One barrier serves both statistics:
// each warp leaves its mean m_w and its squares q_w about it; with N_w elements
// the row's mean is sum N_w m_w / F, and its squares are sum q_w + N_w (m_w -
// mean)^2.
template <typename T, typename To, int NT, int V, int CH>
__global__ void __launch_bounds__(NT) norm_kernel(const T* x, const float* __restrict__ weight,
                                                  const float* __restrict__ bias, float eps, To* y,
                                                  float* mean, float* rstd, long long rows, int F)
{
    constexpr int NW = NT / 32;
    __shared__ float3 part[NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    Share<T, NT, V, CH> xs;
    xs.load(x + row * F, tid, F);
    float count = 0.f, a, b;
#pragma unroll
    for (int m = 0; m < CH; ++m)
        if ((tid + NT * m) * V < F) count += V;
    count = warp_sum(count);
    unpack(xs.sum(), a, b);
    float mu = warp_sum(a + b);
    mu = count > 0.f ? mu / count : 0.f;
    unpack(xs.squares(mu, tid, F), a, b);
    float sq = warp_sum(a + b);
    if (lane == 0) part[warp] = make_float3(count, mu, sq);
    __syncthreads();
    const float3 p = part[lane & (NW - 1)];
    mu = p.x * p.y;
    across_warps<NW, 1>(&mu);
    mu /= F;
    sq = fmaf(p.x * (p.y - mu), p.y - mu, p.z);
    across_warps<NW, 1>(&sq);
    const float rs = rsqrtf(sq / F + eps);
    write_rows<T, To, NT, V, CH, 1>(&xs, y + row * F, weight, bias, &mu, &rs, tid, 1, F);
    if (mean && tid == 0) {
        mean[row] = mu;
        rstd[row] = rs;
    }
}

// Many rows: a CTA walks them, R at a time, with its columns' weights in
// registers. Rows come through shared memory, STAGES - 1 sets of them on their
// way while one is worked on; each thread copies the elements that it will use
// itself, so that only the statistics need a barrier, as in norm_kernel.
template <typename T, typename To, int NT, int V, int CH, int STAGES, int R>
__global__ void __launch_bounds__(NT, NT < 512 ? 512 / NT : 1)
    norm_ring_kernel(const T* x, const float* __restrict__ weight, const float* __restrict__ bias,
                     float eps, To* y, float* mean, float* rstd, long long rows, int F)
{
    constexpr int NW = NT / 32, H = V * CH / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float2 part[2][R][NW];
    __shared__ float counts[NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    f2 w[H], b[H];
    float count = 0.f;
#pragma unroll
    for (int m = 0; m < CH; ++m) {
        const int c = (tid + NT * m) * V;
        float v[V], u[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = u[i] = 0.f;
        if (c < F) {
            count += V;
            load_weights<V>(v, weight + c);
            if (bias) load_weights<V>(u, bias + c);
        }
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            w[(m * V + i) / 2] = pack(v[i], v[i + 1]);
            b[(m * V + i) / 2] = pack(u[i], u[i + 1]);
        }
    }
    count = warp_sum(count);
    const float inverse = count > 0.f ? 1.f / count : 0.f;
    if (lane == 0) counts[warp] = count;
    T* const ring = reinterpret_cast<T*>(smem);  // [stage][row][F]
    auto fetch = [&](int stage, long long row) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (row + r < rows) {
#pragma unroll
                for (int m = 0; m < CH; ++m) {
                    const int c = (tid + NT * m) * V;
                    if (c < F)
                        copy16(ring + (long long)(stage * R + r) * F + c, x + (row + r) * F + c);
                }
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const long long step = (long long)gridDim.x * R;
    long long row = (long long)blockIdx.x * R;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) fetch(s, row + s * step);
    int stage = 0, turn = 0;
#pragma unroll 1
    for (; row < rows; row += step, turn ^= 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        Raw<T, V> xs[R][CH];  // zeros behind a row's end
        float mu[R], sq[R], mw[R], lo, hi;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f2 s = pack(0.f, 0.f);
#pragma unroll
            for (int m = 0; m < CH; ++m) {
                const int c = (tid + NT * m) * V;
                xs[r][m].load(ring + (long long)(stage * R + r) * F + c, c < F);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) s = add2(s, xs[r][m].get(i));
            }
            unpack(s, lo, hi);
            mu[r] = lo + hi;
        }
        across_warps<32, R>(mu);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] *= inverse;
            f2 s = pack(0.f, 0.f);
#pragma unroll
            for (int m = 0; m < CH; ++m) {
                if ((tid + NT * m) * V < F) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const f2 d = add2(xs[r][m].get(i), pack(-mu[r], -mu[r]));
                        s = fma2(d, d, s);
                    }
                }
            }
            unpack(s, lo, hi);
            sq[r] = lo + hi;
        }
        across_warps<32, R>(sq);
        // Two sets of slots in turn: a warp may be a set of rows ahead of another.
        if (lane == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) part[turn][r][warp] = make_float2(mu[r], sq[r]);
        }
        __syncthreads();
        const float n_w = counts[lane & (NW - 1)];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 p = part[turn][r][lane & (NW - 1)];
            mw[r] = p.x;
            mu[r] = n_w * p.x;
            sq[r] = p.y;
        }
        across_warps<NW, R>(mu);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] /= F;
            const float d = mw[r] - mu[r];
            sq[r] = fmaf(n_w * d, d, sq[r]);
        }
        across_warps<NW, R>(sq);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sq[r] = rsqrtf(sq[r] / F + eps);
            if (row + r >= rows) continue;
#pragma unroll
            for (int m = 0; m < CH; ++m) {
                const int c = (tid + NT * m) * V;
                float out[V];
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const f2 d =
                        mul2(add2(xs[r][m].get(i), pack(-mu[r], -mu[r])), pack(sq[r], sq[r]));
                    const int h = m * V / 2 + i;
                    unpack(fma2(d, w[h], b[h]), out[2 * i], out[2 * i + 1]);
                }
                if (c < F) store_vec<To, V>(y + (row + r) * F + c, out);
            }
            if (mean && tid == 0) {
                mean[row + r] = mu[r];
                rstd[row + r] = sq[r];
            }
        }
        // The stage before this one was read for the last time a turn ago.
        fetch((stage + STAGES - 1) % STAGES, row + (STAGES - 1) * step);
        stage = (stage + 1) % STAGES;
    }
}

// One CTA walks the rows, R at a time. They come through shared memory, STAGES -
// 1 sets of them on their way while one is worked on; each thread copies the
// elements that it will use itself, so that only the rows' sums need a barrier.
// With one stage (where F allows no vectors, or shared memory does not hold two
// sets) the rows are loaded directly.
template <typename T, typename To, int NT, int V, int CH, int STAGES, int R>
__global__ void __launch_bounds__(NT, NT < 512 ? 512 / NT : 1) norm_backward_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ weight,
    const float* __restrict__ mean, const float* __restrict__ rstd, To* __restrict__ dx,
    float* __restrict__ dw_part, float* __restrict__ db_part, long long rows, int F)
{
    constexpr int H = (V * CH + 1) / 2;  // pairs of elements per thread and row
    constexpr int NW = NT / 32;
    constexpr bool VECTORS = V > 1, RING = STAGES > 1;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float2 red[2][R][NW];
    const int tid = threadIdx.x, lane = tid & 31;
    const f2 zero = pack(0.f, 0.f);
    // Without vectors a pair is the elements NT apart.
    const auto column = [&](int h, int half) {
        return VECTORS ? (tid + NT * (2 * h / V)) * V + 2 * h % V + half : tid + NT * (2 * h + half);
    };
    f2 dw[H], db[H], w[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        dw[h] = db[h] = zero;
        const int c0 = column(h, 0), c1 = column(h, 1);
        w[h] = pack(c0 < F ? weight[c0] : 0.f, c1 < F ? weight[c1] : 0.f);
    }
    T* const ring = reinterpret_cast<T*>(smem);  // [stage][row][x, dy][F]
    auto fetch = [&](int stage, long long row) {
        if constexpr (RING) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (row + r < rows) {
                    T* const to = ring + (long long)(stage * R + r) * 2 * F;
#pragma unroll
                    for (int m = 0; m < CH; ++m) {
                        const int c = (tid + NT * m) * V;
                        if (c < F) {
                            copy16(to + c, x + (row + r) * F + c);
                            copy16(to + F + c, dy + (row + r) * F + c);
                        }
                    }
                }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    const long long step = (long long)gridDim.x * R;
    long long row = (long long)blockIdx.x * R;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) fetch(s, row + s * step);
    float mu[R], rs[R], mu_next[R], rs_next[R];
    auto stats = [&](long long at, float* m, float* s) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = at + r < rows ? mean[at + r] : 0.f;
            s[r] = at + r < rows ? rstd[at + r] : 0.f;
        }
    };
    stats(row, mu, rs);
    int stage = 0, turn = 0;
#pragma unroll 1
    for (; row < rows; row += step, turn ^= 1) {
        stats(row + step, mu_next, rs_next);
        if constexpr (RING) asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        // x and dy of a row as stored (without vectors: as pairs), zeros where there
        // are none. Rows in shared memory are read twice, for the sums and for dx,
        // rather than kept in registers.
        Raw<T, V> xs[CH], gs[CH];
        f2 x1[H] = {}, g1[H] = {};
        auto load = [&](int r) {
            const bool ok = row + r < rows;
            const T *xr = x + (row + r) * F, *gr = dy + (row + r) * F;
            if constexpr (RING) {
                xr = ring + (long long)(stage * R + r) * 2 * F;
                gr = xr + F;
            }
            if constexpr (VECTORS) {
#pragma unroll
                for (int m = 0; m < CH; ++m) {
                    const int c = (tid + NT * m) * V;
                    xs[m].load(xr + c, ok && c < F);
                    gs[m].load(gr + c, ok && c < F);
                }
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int c0 = column(h, 0), c1 = column(h, 1);
                    const bool k0 = ok && c0 < F, k1 = ok && c1 < F;
                    x1[h] = pack(k0 ? to_f32(xr[c0]) : 0.f, k1 ? to_f32(xr[c1]) : 0.f);
                    g1[h] = pack(k0 ? to_f32(gr[c0]) : 0.f, k1 ? to_f32(gr[c1]) : 0.f);
                }
            }
        };
        auto value = [&](int r, int h) {
            f2 v;
            if constexpr (VECTORS) v = xs[2 * h / V].get(h % (V / 2));
            else v = x1[h];
            return mul2(add2(v, pack(-mu[r], -mu[r])), pack(rs[r], rs[r]));
        };
        auto grad = [&](int h) {
            if constexpr (VECTORS) return gs[2 * h / V].get(h % (V / 2));
            else return g1[h];
        };
        float m1[R], m2[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            load(r);
            f2 s1 = zero, s2 = zero;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const f2 v = value(r, h), g = grad(h);
                dw[h] = fma2(g, v, dw[h]);
                db[h] = add2(db[h], g);
                const f2 e = mul2(g, w[h]);
                s1 = add2(s1, e);
                s2 = fma2(e, v, s2);
            }
            float a, b;
            unpack(s1, a, b);
            m1[r] = a + b;
            unpack(s2, a, b);
            m2[r] = a + b;
        }
        across_warps<32, R>(m1);
        across_warps<32, R>(m2);
        if constexpr (NW > 1) {
            // Two sets of slots in turn: a warp may be a set of rows ahead of another.
            if (lane == 0) {
#pragma unroll
                for (int r = 0; r < R; ++r) red[turn][r][tid >> 5] = make_float2(m1[r], m2[r]);
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 v = red[turn][r][lane & (NW - 1)];
                m1[r] = v.x;
                m2[r] = v.y;
            }
            across_warps<NW, R>(m1);
            across_warps<NW, R>(m2);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (RING || R > 1) load(r);
            f2 dxv[H];
            const f2 minus_m1 = pack(-m1[r] / F, -m1[r] / F), minus_m2 = pack(-m2[r] / F, -m2[r] / F);
            const f2 scale = pack(rs[r], rs[r]);
            To* const out = dx + (row + r) * F;
#pragma unroll
            for (int h = 0; h < H; ++h)
                dxv[h] = mul2(fma2(value(r, h), minus_m2, fma2(grad(h), w[h], minus_m1)), scale);
            if (row + r >= rows) continue;
            if constexpr (VECTORS) {
#pragma unroll
                for (int m = 0; m < CH; ++m) {
                    const int c = (tid + NT * m) * V;
                    if (c < F) {
                        float v[V];
#pragma unroll
                        for (int i = 0; i < V; i += 2) unpack(dxv[(m * V + i) / 2], v[i], v[i + 1]);
                        store_vec<To, V>(out + c, v);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int c0 = column(h, 0), c1 = column(h, 1);
                    float v0, v1;
                    unpack(dxv[h], v0, v1);
                    if (c0 < F) out[c0] = from_f32<To>(v0);
                    if (c1 < F) out[c1] = from_f32<To>(v1);
                }
            }
        }
        // The stage before this one was read for the last time a turn ago.
        fetch((stage + STAGES - 1) % STAGES, row + (STAGES - 1) * step);
#pragma unroll
        for (int r = 0; r < R; ++r) mu[r] = mu_next[r], rs[r] = rs_next[r];
        stage = (stage + 1) % STAGES;
    }
    float* const dwp = dw_part + (long long)blockIdx.x * F;
    float* const dbp = db_part + (long long)blockIdx.x * F;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        float w0, w1, b0, b1;
        unpack(dw[h], w0, w1);
        unpack(db[h], b0, b1);
        const int c0 = column(h, 0), c1 = column(h, 1);
        if (c0 < F) dwp[c0] = w0, dbp[c0] = b0;
        if (c1 < F) dwp[c1] = w1, dbp[c1] = b1;
    }
}

// Threads of the backward, for at most 16 elements each (a row's, its gradient's
// and two sums per column are in registers); without vectors for 8, where 1024
// threads allow it, since no ring hides those loads.
int back_threads(int F)
{
    return F <= 512 ? 32 : F <= 2048 ? 128 : F <= 4096 ? 256 : F <= 8192 ? 512 : 1024;
}

// Rows that a CTA of the backward takes at once, and stages of its ring: what
// shared memory holds beside the SM's other CTAs.
template <typename T> constexpr int back_rows(int V, int nt)
{
    return V > 1 && sizeof(T) == 2 && nt <= 512 ? 2 : 1;
}
template <typename T> constexpr int back_stages(int V, int nt)
{
    return V == 1 ? 1 : nt <= 512 ? 3 : sizeof(T) == 2 ? 3 : 1;
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

template <typename T, typename To, int NT, int V>
cudaError_t launch_ring(const void* x, const float* weight, const float* bias, float eps, void* y,
                        float* mean, float* rstd, long long rows, int F, cudaStream_t stream)
{
    constexpr int R = sizeof(T) == 2 ? (NT > 512 ? 2 : 4) : (NT > 512 ? 1 : 2), STAGES = 3;
    auto kernel = norm_ring_kernel<T, To, NT, V, 16 / V, STAGES, R>;
    const int smem = STAGES * R * F * (int)sizeof(T);
    cudaError_t e = allow_shared((const void*)kernel, MOST_SHARED);
    if (e != cudaSuccess) return e;
    const long long sets = (rows + R - 1) / R, most = 148 * (NT < 512 ? 512 / NT : 1);
    kernel<<<(unsigned)(sets < most ? sets : most), NT, smem, stream>>>(
        (const T*)x, weight, bias, eps, (To*)y, mean, rstd, rows, F);
    return cudaGetLastError();
}

// Few rows: a warp each up to 2048 features, a CTA each beyond. Many: rings.
#define LA_NORM_FORWARD(T, To, V)                                                                \
    do {                                                                                         \
        const bool many = V > 1 && rows >= LA_RING_ROWS;                                         \
        if (F <= 1024) LA_WARP(T, To, V, 32 / V);                                                \
        else if (F <= 2048 && !many) LA_WARP(T, To, V, 64 / V);                                  \
        else if (F <= 2048) LA_RING(T, To, 128, V);                                              \
        else if (F <= 4096 && many) LA_RING(T, To, 256, V);                                      \
        else if (F <= 4096) LA_CALL(T, To, 256, V);                                              \
        else if (F <= 8192 && many) LA_RING(T, To, 512, V);                                      \
        else if (F <= 8192) LA_CALL(T, To, 512, V);                                              \
        else if (many) LA_RING(T, To, 1024, V);                                                  \
        else LA_CALL(T, To, 1024, V);                                                            \
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
#define LA_WARP(T, To, V, CH)                                                                    \
    norm_warp_kernel<T, To, V, CH><<<(unsigned)((rows + 3) / 4), 128, 0, stream>>>(              \
        (const T*)x, weight, bias, eps, (To*)y, mean, rstd, rows, F)
#define LA_CALL(T, To, NT, V)                                                                    \
    norm_kernel<T, To, NT, V, 16 / V><<<(unsigned)rows, NT, 0, stream>>>(                        \
        (const T*)x, weight, bias, eps, (To*)y, mean, rstd, rows, F)
#define LA_RING(T, To, NT, V)                                                                    \
    do {                                                                                         \
        if constexpr (V > 1)                                                                     \
            e = launch_ring<T, To, NT, V>(x, weight, bias, eps, y, mean, rstd, rows, F, stream); \
    } while (0)
    cudaError_t e = cudaSuccess;
    LA_NORM_TYPES(LA_NORM_FORWARD)
#undef LA_CALL
#undef LA_RING
#undef LA_WARP
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

#define LA_NORM_BACKWARD(T, To, V)                                                               \
    do {                                                                                         \
        constexpr int E = V == 1 ? 8 : 16;                                                       \
        switch (back_threads(V == 1 && F <= 8192 ? 2 * F : F)) {                                 \
        case 32: LA_CALL(T, To, 32, V, E); break;                                                \
        case 128: LA_CALL(T, To, 128, V, E); break;                                              \
        case 256: LA_CALL(T, To, 256, V, E); break;                                              \
        case 512: LA_CALL(T, To, 512, V, E); break;                                              \
        default:                                                                                 \
            if (V == 1 && F <= 8192) LA_CALL(T, To, 1024, V, E);                                 \
            else LA_CALL(T, To, 1024, V, 16);                                                    \
            break;                                                                               \
        }                                                                                        \
    } while (0)

// A launch with the ring's shared memory.
template <typename T, typename To, int NT, int V, int CH, int STAGES, int R>
cudaError_t launch_backward(const void* dy, const void* x, const float* weight, const float* mean,
                            const float* rstd, void* dx, float* dw, float* db, long long rows,
                            int F, int ctas, cudaStream_t stream)
{
    auto kernel = norm_backward_kernel<T, To, NT, V, CH, STAGES, R>;
    const int smem = STAGES > 1 ? STAGES * R * 2 * F * (int)sizeof(T) : 0;
    if (smem > 40 * 1024) {  // beside the static slots of the sums
        cudaError_t e = allow_shared((const void*)kernel, MOST_SHARED);
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
#define LA_CALL(T, To, NT, V, E)                                                                 \
    e = launch_backward<T, To, NT, V, E / V, back_stages<T>(V, NT), back_rows<T>(V, NT)>(        \
        dy, x, weight, mean, rstd, dx, dw, db, rows, F, ctas, stream)
        LA_NORM_TYPES(LA_NORM_BACKWARD)
#undef LA_CALL
        count_launch();
        if (e != cudaSuccess) return e;
    }
    SumJobs sums;
    sums.add(dw, dweight, ctas, F);
    sums.add(db, dbias, ctas, F);
    return launch_column_sums(sums, stream);
}

}  // namespace la
