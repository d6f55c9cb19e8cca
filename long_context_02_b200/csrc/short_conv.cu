// Short causal convolution of each channel, over prompts, for single tokens
// and backward (formulas in lightning.h).
//
// Streams of 2 (forward) or 3 (backward) values per (token, channel): bound by
// HBM. A thread owns V adjacent channels (one 16-byte vector where pointers and
// strides allow it, else one channel) and walks a tile of tokens with the last
// W inputs in registers, so that each input is loaded once; only the W - 1
// rows before a tile are loaded twice. Tiles cut the packed rows without
// regard to sequences: at a sequence's first token the window is reloaded from
// its incoming state.
#include "ssm.h"

namespace la {
namespace {

constexpr int NT = 128;
constexpr int TILE = 64;       // tokens per thread, forward
constexpr int BACK_TILE = 64;  // tokens per thread, backward
constexpr int AHEAD = 8;       // rows loaded before any of them is used

struct ConvArgs {
    const void* x;
    long long ld_x;
    const float* weight;
    const float* bias;
    const void* state_in;
    void* y;
    void* state_out;
    SeqView view;
    int D, silu, cblocks;
    long long tiles;
    // backward
    const void* dy;
    long long ld_dy;
    const void* dstate_out;
    void* dx;
    void* dstate_in;
    float* dw_part;  // [tiles][D][W]
    float* db_part;  // [tiles][D]
};

// V values of type T at p, as stored.
template <typename T, int V> struct Row {
    static constexpr int BYTES = V * sizeof(T);
    union {
        T e[V];
        uint4 q;
        uint2 d;
        uint32_t w;
    };
    __device__ __forceinline__ Row() {}
    __device__ __forceinline__ void load(const T* p)
    {
        if (BYTES == 16) q = __ldcs(reinterpret_cast<const uint4*>(p));
        else e[0] = *p;
    }
    __device__ __forceinline__ void zero()
    {
        if (BYTES == 16) q = make_uint4(0, 0, 0, 0);
        else e[0] = T(0.f);
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if (BYTES == 16) __stcs(reinterpret_cast<uint4*>(p), q);
        else *p = e[0];
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(e[i]); }
    __device__ __forceinline__ void set(int i, float v) { e[i] = from_f32<T>(v); }
};

template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const float* v)
{
    if constexpr (V * sizeof(T) > 16) {  // eight fp32 outputs of eight bf16 inputs
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
    } else {
        Row<T, V> r;
#pragma unroll
        for (int i = 0; i < V; ++i) r.set(i, v[i]);
        r.store(p);
    }
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// CTAs [0, tiles * cblocks) convolve; the CTAs behind them write state_out.
template <typename T, typename To, int W, int V>
__global__ void __launch_bounds__(NT) conv_kernel(ConvArgs a)
{
    const int cb = blockIdx.x % a.cblocks;
    const long long tile = blockIdx.x / a.cblocks;
    const int c = (cb * NT + threadIdx.x) * V;
    if (c >= a.D) return;
    const T* x = (const T*)a.x + c;
    const T* st = a.state_in ? (const T*)a.state_in + c : nullptr;
    long long start, end;
    if (tile >= a.tiles) {
        const int s = (int)(tile - a.tiles);
        a.view.range(s, start, end);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            const long long tok = end - (W - 1) + r;  // before the sequence: from its state
            Row<T, V> row;
            if (tok >= start) row.load(x + tok * a.ld_x);
            else if (st) row.load(st + ((long long)s * (W - 1) + (tok - start + W - 1)) * a.D);
            else row.zero();
            row.store((T*)a.state_out + ((long long)s * (W - 1) + r) * a.D + c);
        }
        return;
    }
    float w[W][V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = a.weight[(long long)(c + i) * W + j];
        b[i] = a.bias ? a.bias[c + i] : 0.f;
    }
    const long long t0 = tile * TILE;
    const long long t1 = t0 + TILE < a.view.total ? t0 + TILE : a.view.total;
    int s = a.view.find(t0);
    if (s >= a.view.num_seqs) return;
    a.view.range(s, start, end);

    float win[W][V];  // inputs t - (W - 1) .. t
    // The W - 1 inputs before row t of sequence s.
    auto fill = [&](long long t) {
#pragma unroll
        for (int j = 1; j < W; ++j) {
            const long long tok = t - W + j;
            Row<T, V> row;
            if (tok >= start) row.load(x + tok * a.ld_x);
            else if (st) row.load(st + ((long long)s * (W - 1) + (tok - start + W - 1)) * a.D);
            else row.zero();
#pragma unroll
            for (int i = 0; i < V; ++i) win[j][i] = row.get(i);
        }
    };
    fill(t0);
#pragma unroll 1
    for (long long t = t0; t < t1; t += AHEAD) {
        Row<T, V> rows[AHEAD];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            if (t + q < t1) rows[q].load(x + (t + q) * a.ld_x);
            else rows[q].zero();
        }
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const long long tok = t + q;
            if (tok >= t1) return;
            if (tok >= end) {  // the next sequence that holds this row
                do {
                    if (++s >= a.view.num_seqs) return;
                    a.view.range(s, start, end);
                } while (tok >= end);
                fill(tok);
            }
            float out[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][i] = win[j + 1][i];
                win[W - 1][i] = rows[q].get(i);
                float p = b[i];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                out[i] = a.silu ? p * sigmoid(p) : p;
            }
            store_row<To, V>((To*)a.y + tok * a.D + c, out);
        }
    }
}

template <typename T, typename To, int W, int V>
__global__ void __launch_bounds__(NT) conv_step_kernel(ConvArgs a)
{
    const int c = (blockIdx.x % a.cblocks * NT + threadIdx.x) * V;
    const long long s = blockIdx.x / a.cblocks;
    if (c >= a.D) return;
    Row<T, V> rows[W];
    T* st = (T*)a.state_out + s * (W - 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[j].load(st + (long long)j * a.D);
    rows[W - 1].load((const T*)a.x + s * a.ld_x + c);
    float out[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float p = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j)
            p = fmaf(a.weight[(long long)(c + i) * W + j], rows[j].get(i), p);
        out[i] = a.silu ? p * sigmoid(p) : p;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[j + 1].store(st + (long long)j * a.D);
    store_row<To, V>((To*)a.y + s * a.D + c, out);
}

// A tile is walked from its last row to its first, with q_t .. q_{t+W-1} in
// registers: dx_t needs the q of the W - 1 rows after it, which are computed
// again where the tile ends inside a sequence. The weight's gradient is summed
// over the tile's own rows and written as a partial sum. CTAs behind the tiles
// write dstate_in: the rows before a sequence's first token.
template <typename T, typename To, int W, int V>
__global__ void __launch_bounds__(NT) conv_backward_kernel(ConvArgs a)
{
    const int cb = blockIdx.x % a.cblocks;
    const long long tile = blockIdx.x / a.cblocks;
    const int c = (cb * NT + threadIdx.x) * V;
    if (c >= a.D) return;
    const T* x = (const T*)a.x + c;
    const T* dy = (const T*)a.dy + c;
    const T* st = a.state_in ? (const T*)a.state_in + c : nullptr;
    const T* dst = a.dstate_out ? (const T*)a.dstate_out + c : nullptr;
    float w[W][V], b[V], dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = a.weight[(long long)(c + i) * W + j], dw[j][i] = 0.f;
        b[i] = a.bias ? a.bias[c + i] : 0.f;
        db[i] = 0.f;
    }
    int s;
    long long start, end;
    float win[W][V], q[W][V];  // inputs t - (W-1) .. t; q_t .. q_{t+W-1}
    // Input row `tok` of sequence s, before its start from the state.
    auto input = [&](long long tok) {
        Row<T, V> row;
        if (tok >= start) row.load(x + tok * a.ld_x);
        else if (st && tok - start >= -(W - 1))
            row.load(st + ((long long)s * (W - 1) + (tok - start + W - 1)) * a.D);
        else row.zero();
        return row;
    };
    // Gradient that state_out sends to input row `tok`.
    auto from_state = [&](long long tok, float* v) {
        const long long r = tok - (end - (W - 1));
        if (!dst || r < 0) return;
        Row<T, V> row;
        row.load(dst + ((long long)s * (W - 1) + r) * a.D);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += row.get(i);
    };
    auto pull = [&](float* v) {  // sum_j w_j q_{t + W-1-j}
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) v[i] = fmaf(w[j][i], q[W - 1 - j][i], v[i]);
        }
    };
    // One row: window and q move down to row t, whose oldest input and dy are given.
    auto step = [&](const Row<T, V>& oldest, const Row<T, V>& grad) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = W - 1; j > 0; --j) win[j][i] = win[j - 1][i], q[j][i] = q[j - 1][i];
            win[0][i] = oldest.get(i);
            float g = grad.get(i);
            if (a.silu) {
                float p = b[i];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                const float sg = sigmoid(p);
                g *= sg * fmaf(p, 1.f - sg, 1.f);
            }
            q[0][i] = g;
        }
    };
    // Before row `last` of sequence s: no q after it, and its window but the oldest.
    auto open = [&](long long last) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const Row<T, V> row = input(last - (W - 2) + j);
#pragma unroll
            for (int i = 0; i < V; ++i) win[j][i] = row.get(i);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) q[j][i] = 0.f;
    };

    if (tile >= a.tiles) {
        s = (int)(tile - a.tiles);
        a.view.range(s, start, end);
        // Rows start + W - 2 down to start - (W - 1); the last W - 1 are the state's.
        long long t = start + W - 2 < end - 1 ? start + W - 2 : end - 1;
        open(t);
        for (; t >= start; --t) {
            Row<T, V> g;
            g.load(dy + t * a.ld_dy);
            step(input(t - (W - 1)), g);
        }
        for (; t >= start - (W - 1); --t) {
            Row<T, V> g;
            g.zero();
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = W - 1; j > 0; --j) q[j][i] = q[j - 1][i];
                q[0][i] = 0.f;
            }
            float v[V];
            pull(v);
            from_state(t, v);
            store_row<To, V>((To*)a.dstate_in +
                                 ((long long)s * (W - 1) + (t - start + W - 1)) * a.D + c, v);
        }
        return;
    }

    const long long t0 = tile * BACK_TILE;
    long long t1 = t0 + BACK_TILE < a.view.total ? t0 + BACK_TILE : a.view.total;
    // The sequence of the last row that has one.
    s = a.view.find(t1 - 1);
    if (s >= a.view.num_seqs) {
        s = a.view.num_seqs - 1;
        a.view.range(s, start, end);
        if (end < t1) t1 = end;
        if (t1 > t0) s = a.view.find(t1 - 1);
    }
    if (t1 > t0 && s < a.view.num_seqs) {
        a.view.range(s, start, end);
        // rows after the tile in the same sequence
        long long t = t1 - 1 + (W - 1) < end - 1 ? t1 - 1 + (W - 1) : end - 1;
        open(t);
        for (; t >= t1; --t) {
            Row<T, V> g;
            g.load(dy + t * a.ld_dy);
            step(input(t - (W - 1)), g);
        }
#pragma unroll 1
        for (; t >= t0;) {
            if (t < start) {  // an earlier sequence's last row
                do {
                    if (--s < 0) break;
                    a.view.range(s, start, end);
                } while (t < start || end == start);
                if (s < 0) break;
                open(t);
            }
            const long long low = start > t0 ? start : t0;
            long long n = t - low + 1;
            if (n > AHEAD / 2) n = AHEAD / 2;
            Row<T, V> xs[AHEAD / 2], gs[AHEAD / 2];
#pragma unroll
            for (int k = 0; k < AHEAD / 2; ++k)
                if (k < n) {
                    xs[k] = input(t - k - (W - 1));
                    gs[k].load(dy + (t - k) * a.ld_dy);
                }
#pragma unroll
            for (int k = 0; k < AHEAD / 2; ++k)
                if (k < n) {
                    step(xs[k], gs[k]);
                    float v[V];
                    pull(v);
                    from_state(t - k, v);
                    store_row<To, V>((To*)a.dx + (t - k) * a.D + c, v);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][i] = fmaf(q[0][i], win[j][i], dw[j][i]);
                        db[i] += q[0][i];
                    }
                }
            t -= n;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) a.dw_part[(tile * a.D + c + i) * W + j] = dw[j][i];
        a.db_part[tile * a.D + c + i] = db[i];
    }
}

bool vec16(const void* p, long long ld, size_t e)
{
    return ((uintptr_t)p & 15) == 0 && (ld * e & 15) == 0;
}

// Calls F<T, To, W, V>: V channels per thread, a 16-byte vector of the inputs
// when every row of every tensor starts on one, else 1.
#define LA_CONV_CASE(F, T, To, W, VEC)                                                           \
    if (vec) F(T, To, W, VEC);                                                                   \
    else F(T, To, W, 1)
#define LA_CONV_TYPES(F, W)                                                                      \
    if (p.in_t == LA_F32) { LA_CONV_CASE(F, float, float, W, 4); }                               \
    else if (p.out_t == LA_F32) { LA_CONV_CASE(F, __nv_bfloat16, float, W, 8); }                 \
    else { LA_CONV_CASE(F, __nv_bfloat16, __nv_bfloat16, W, 8); }
#define LA_CONV_DISPATCH(F)                                                                      \
    if (p.W == 2) { LA_CONV_TYPES(F, 2) }                                                        \
    else if (p.W == 3) { LA_CONV_TYPES(F, 3) }                                                   \
    else { LA_CONV_TYPES(F, 4) }

ConvArgs base_args(const ConvProblem& p, bool vec)
{
    ConvArgs a{};
    a.x = p.x;
    a.ld_x = p.ld_x;
    a.weight = p.weight;
    a.bias = p.bias;
    a.view = p.view;
    a.D = p.D;
    a.silu = p.silu;
    const int V = vec ? (p.in_t == LA_BF16 ? 8 : 4) : 1;
    a.cblocks = (p.D + NT * V - 1) / (NT * V);
    return a;
}

bool use_vectors(const ConvProblem& p)
{
    const size_t e = p.in_t == LA_BF16 ? 2 : 4;
    return (p.D * e & 15) == 0 && vec16(p.x, p.ld_x, e);
}

}  // namespace

cudaError_t launch_short_conv(const ConvProblem& p, const void* state_in, void* y,
                              void* state_out, cudaStream_t stream)
{
    const bool vec = use_vectors(p);
    ConvArgs a = base_args(p, vec);
    a.state_in = state_in;
    a.y = y;
    a.state_out = state_out;
    a.tiles = (p.view.total + TILE - 1) / TILE;
    const long long grid = (a.tiles + (state_out ? p.view.num_seqs : 0)) * a.cblocks;
    if (grid == 0) return cudaSuccess;
#define LA_CALL(T, To, W, V) conv_kernel<T, To, W, V><<<(unsigned)grid, NT, 0, stream>>>(a)
    LA_CONV_DISPATCH(LA_CALL)
#undef LA_CALL
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_short_conv_step(const ConvProblem& p, void* state, void* y,
                                   cudaStream_t stream)
{
    const bool vec = use_vectors(p);
    ConvArgs a = base_args(p, vec);
    a.state_out = state;
    a.y = y;
    const unsigned grid = (unsigned)((long long)p.view.num_seqs * a.cblocks);
#define LA_CALL(T, To, W, V) conv_step_kernel<T, To, W, V><<<grid, NT, 0, stream>>>(a)
    LA_CONV_DISPATCH(LA_CALL)
#undef LA_CALL
    count_launch();
    return cudaGetLastError();
}

size_t conv_backward_workspace(int D, long long total, int W)
{
    const size_t tiles = (size_t)((total + BACK_TILE - 1) / BACK_TILE);
    return align_up(tiles * D * W * 4, 256) + align_up(tiles * D * 4, 256);
}

cudaError_t launch_short_conv_backward(const ConvProblem& p, const void* dy, long long ld_dy,
                                       const void* state_in, const void* dstate_out, void* dx,
                                       float* dweight, float* dbias, void* dstate_in, void* ws,
                                       cudaStream_t stream)
{
    const bool vec = use_vectors(p) && vec16(dy, ld_dy, p.in_t == LA_BF16 ? 2 : 4);
    ConvArgs a = base_args(p, vec);
    a.state_in = state_in;
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.dstate_out = dstate_out;
    a.dx = dx;
    a.dstate_in = dstate_in;
    a.tiles = (p.view.total + BACK_TILE - 1) / BACK_TILE;
    a.dw_part = (float*)ws;
    a.db_part = (float*)((char*)ws + align_up((size_t)a.tiles * p.D * p.W * 4, 256));
    const long long grid = (a.tiles + (dstate_in ? p.view.num_seqs : 0)) * a.cblocks;
    if (grid > 0) {
#define LA_CALL(T, To, W, V) conv_backward_kernel<T, To, W, V><<<(unsigned)grid, NT, 0, stream>>>(a)
        LA_CONV_DISPATCH(LA_CALL)
#undef LA_CALL
        count_launch();
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_column_sum(a.dw_part, dweight, (int)a.tiles, (long long)p.D * p.W, stream);
    if (e == cudaSuccess && dbias)
        e = launch_column_sum(a.db_part, dbias, (int)a.tiles, p.D, stream);
    return e;
}

}  // namespace la
