// Short causal convolution of each channel, over prompts, for single tokens
// and backward (formulas in lightning.h).
//
// Streams of 2 (forward) or 3 (backward) values per (token, channel): bound by
// HBM. A thread owns V = 4 adjacent channels (one vector where pointers and
// strides allow it, else one channel) and walks a tile of tokens with the last
// W inputs in registers, so that each input is loaded once; only the W - 1
// rows before a tile are loaded twice. Tiles cut the packed rows without
// regard to sequences: at a sequence's first token the window is reloaded from
// its incoming state.
//
// Measured, bf16, W = 4: 4 x 8K tokens of 8192 channels 191-203 us, 5.3-5.6 TB/s.
// The backward of 2 x 8K takes 202-206 us, 3.9-4.0 TB/s. Neither memory (42% of
// DRAM's peak) nor issue (50% of the cycles) is full: its 128 registers leave 14
// warps per SM, whose latencies set the pace, over about 27 instructions per
// element where the formula has 12 in pairs. Two channels per thread, for more
// warps per SM, took 250 us. In fp32 four channels spill (W = 4 236 bytes stored,
// W = 3 76).
#include "ssm_scan.cuh"

namespace la {
namespace {

constexpr int NT = 128;
constexpr int AHEAD = 8;        // rows in flight per thread while the rows before them are used
constexpr int BACK_AHEAD = 4;   // the same, backward (two rows each)

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
    int tile;  // rows per CTA
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

// V values of type T at p, as stored, read as pairs (a single value is a pair
// with a zero).
template <typename T, int V> struct Row {
    union {
        uint4 q;
        uint2 d;
        uint32_t w[4];
        T one;
    };
    __device__ __forceinline__ Row() {}
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (V == 1) one = *p;
        else if constexpr (V * sizeof(T) == 16) q = __ldcs(reinterpret_cast<const uint4*>(p));
        else d = __ldcs(reinterpret_cast<const uint2*>(p));
    }
    __device__ __forceinline__ void zero()
    {
        if constexpr (V == 1) one = T(0.f);
        else if constexpr (V * sizeof(T) == 16) q = make_uint4(0, 0, 0, 0);
        else d = make_uint2(0, 0);
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if constexpr (V == 1) *p = one;
        else if constexpr (V * sizeof(T) == 16) __stcs(reinterpret_cast<uint4*>(p), q);
        else __stcs(reinterpret_cast<uint2*>(p), d);
    }
    __device__ __forceinline__ f2 get(int i) const
    {
        if constexpr (V == 1) return pack(to_f32(one), 0.f);
        else if constexpr (sizeof(T) == 2)
            return pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else return pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const f2* v)
{
    float x[V + 1];
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) unpack(v[i], x[2 * i], x[2 * i + 1]);
    if constexpr (V == 1) {
        *p = from_f32<T>(x[0]);
    } else if constexpr (sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(x[2], x[3]);
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                       *reinterpret_cast<const uint32_t*>(&hi)));
    }
}

// Weights [D][W] and biases of V channels from c on, as pairs of channels.
template <int W, int V>
__device__ __forceinline__ void load_weights(const float* weight, const float* bias, int c,
                                             f2 (*w)[(V + 1) / 2], f2* b)
{
    float x[V * W], y[V + 1];
    if constexpr (V == 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) x[j] = weight[(long long)c * W + j];
        y[0] = bias ? bias[c] : 0.f;
        y[1] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < V * W; i += 4)
            *reinterpret_cast<float4*>(x + i) =
                *reinterpret_cast<const float4*>(weight + (long long)c * W + i);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = bias ? bias[c + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            w[j][i] = pack(x[2 * i * W + j], V == 1 ? 0.f : x[((2 * i + 1) % V) * W + j]);
        b[i] = pack(y[2 * i], y[2 * i + 1]);
    }
}

// CTAs [0, tiles * cblocks) convolve; the CTAs behind them write state_out.
template <typename T, typename To, int W, int V>
__global__ void __launch_bounds__(NT) conv_kernel(ConvArgs a)
{
    constexpr int H = (V + 1) / 2;  // pairs
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
    f2 w[W][H], b[H];
    load_weights<W, V>(a.weight, a.bias, c, w, b);
    const long long t0 = tile * a.tile;
    const long long t1 = t0 + a.tile < a.view.total ? t0 + a.tile : a.view.total;
    int s = a.view.find(t0);
    if (s >= a.view.num_seqs) return;

    // The tile's rows, one run per sequence.
    for (long long t = t0; t < t1; ++s) {
        if (s >= a.view.num_seqs) return;
        a.view.range(s, start, end);
        if (end <= t) continue;
        f2 win[W][H];  // inputs t - (W - 1) .. t
#pragma unroll
        for (int j = 1; j < W; ++j) {
            const long long tok = t - W + j;
            Row<T, V> row;
            if (tok >= start) row.load(x + tok * a.ld_x);
            else if (st) row.load(st + ((long long)s * (W - 1) + (tok - start + W - 1)) * a.D);
            else row.zero();
#pragma unroll
            for (int i = 0; i < H; ++i) win[j][i] = row.get(i);
        }
        const int n = (int)((end < t1 ? end : t1) - t);  // rows of this run
        const T* xp = x + t * a.ld_x;
        To* yp = (To*)a.y + t * a.D + c;
        auto row_out = [&](const Row<T, V>& in, int at) {
            f2 out[H];
#pragma unroll
            for (int i = 0; i < H; ++i) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][i] = win[j + 1][i];
                win[W - 1][i] = in.get(i);
                f2 p = b[i];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fma2(w[j][i], win[j][i], p);
                const f2 g = mul2(p, sigmoid2(p));
                out[i] = a.silu ? g : p;
            }
            store_row<To, V>(yp + (long long)at * a.D, out);
        };
        // Whole groups of rows, so that the window's shifts are a renaming of
        // registers; then the rest one by one.
        const int whole = n / AHEAD * AHEAD;
        Row<T, V> rows[AHEAD];
        auto load = [&](int at) {
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) rows[q].load(xp + (long long)(at + q) * a.ld_x);
        };
        if (whole) load(0);
#pragma unroll 1
        for (int at = 0; at < whole; at += AHEAD) {
            Row<T, V> now[AHEAD];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) now[q] = rows[q];
            if (at + AHEAD < whole) load(at + AHEAD);
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) row_out(now[q], at + q);
        }
#pragma unroll 1
        for (int at = whole; at < n; ++at) {
            Row<T, V> in;
            in.load(xp + (long long)at * a.ld_x);
            row_out(in, at);
        }
        t += n;
    }
}

template <typename T, typename To, int W, int V>
__global__ void __launch_bounds__(NT) conv_step_kernel(ConvArgs a)
{
    constexpr int H = (V + 1) / 2;
    const int c = (blockIdx.x % a.cblocks * NT + threadIdx.x) * V;
    const long long s = blockIdx.x / a.cblocks;
    if (c >= a.D) return;
    Row<T, V> rows[W];
    T* st = (T*)a.state_out + s * (W - 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[j].load(st + (long long)j * a.D);
    rows[W - 1].load((const T*)a.x + s * a.ld_x + c);
    f2 w[W][H], b[H], out[H];
    load_weights<W, V>(a.weight, a.bias, c, w, b);
#pragma unroll
    for (int i = 0; i < H; ++i) {
        f2 p = b[i];
#pragma unroll
        for (int j = 0; j < W; ++j) p = fma2(w[j][i], rows[j].get(i), p);
        out[i] = a.silu ? mul2(p, sigmoid2(p)) : p;
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
__global__ void __launch_bounds__(NT, 4) conv_backward_kernel(ConvArgs a)
{
    constexpr int H = (V + 1) / 2;
    const int cb = blockIdx.x % a.cblocks;
    const long long tile = blockIdx.x / a.cblocks;
    const int c = (cb * NT + threadIdx.x) * V;
    if (c >= a.D) return;
    const T* x = (const T*)a.x + c;
    const T* dy = (const T*)a.dy + c;
    const T* st = a.state_in ? (const T*)a.state_in + c : nullptr;
    const T* dst = a.dstate_out ? (const T*)a.dstate_out + c : nullptr;
    const f2 zero = pack(0.f, 0.f), one = pack(1.f, 1.f), minus = pack(-1.f, -1.f);
    f2 w[W][H], b[H], dw[W][H], db[H];
    load_weights<W, V>(a.weight, a.bias, c, w, b);
#pragma unroll
    for (int i = 0; i < H; ++i) {
        db[i] = zero;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = zero;
    }
    int s;
    long long start, end;
    f2 win[W][H], q[W][H];  // inputs t - (W-1) .. t; q_t .. q_{t+W-1}
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
    auto from_state = [&](long long tok, f2* v) {
        const long long r = tok - (end - (W - 1));
        if (!dst || r < 0) return;
        Row<T, V> row;
        row.load(dst + ((long long)s * (W - 1) + r) * a.D);
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = add2(v[i], row.get(i));
    };
    auto pull = [&](f2* v) {  // sum_j w_j q_{t + W-1-j}
#pragma unroll
        for (int i = 0; i < H; ++i) {
            v[i] = mul2(w[0][i], q[W - 1][i]);
#pragma unroll
            for (int j = 1; j < W; ++j) v[i] = fma2(w[j][i], q[W - 1 - j][i], v[i]);
        }
    };
    // One row: window and q move down to row t, whose oldest input and dy are given.
    auto step = [&](const Row<T, V>& oldest, const Row<T, V>& grad) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
#pragma unroll
            for (int j = W - 1; j > 0; --j) win[j][i] = win[j - 1][i], q[j][i] = q[j - 1][i];
            win[0][i] = oldest.get(i);
            const f2 g = grad.get(i);
            f2 p = b[i];
#pragma unroll
            for (int j = 0; j < W; ++j) p = fma2(w[j][i], win[j][i], p);
            // y'(p) = sg (1 + p (1 - sg))
            const f2 sg = sigmoid2(p);
            const f2 slope = mul2(sg, fma2(p, fma2(sg, minus, one), one));
            q[0][i] = a.silu ? mul2(g, slope) : g;
        }
    };
    // Before row `last` of sequence s: no q after it, and its window but the oldest.
    auto open = [&](long long last) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const Row<T, V> row = input(last - (W - 2) + j);
#pragma unroll
            for (int i = 0; i < H; ++i) win[j][i] = row.get(i);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) q[j][i] = zero;
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
#pragma unroll
            for (int i = 0; i < H; ++i) {
#pragma unroll
                for (int j = W - 1; j > 0; --j) q[j][i] = q[j - 1][i];
                q[0][i] = zero;
            }
            f2 v[H];
            pull(v);
            from_state(t, v);
            store_row<To, V>((To*)a.dstate_in +
                                 ((long long)s * (W - 1) + (t - start + W - 1)) * a.D + c, v);
        }
        return;
    }

    const long long t0 = tile * a.tile;
    long long t1 = t0 + a.tile < a.view.total ? t0 + a.tile : a.view.total;
    // The sequence of the last row that has one.
    s = a.view.find(t1 - 1);
    if (s >= a.view.num_seqs) {
        s = a.view.num_seqs - 1;
        a.view.range(s, start, end);
        if (end < t1) t1 = end;
        if (t1 > t0) s = a.view.find(t1 - 1);
    }
    // The tile's rows, one run per sequence, each from its last row down.
    for (long long t = t1 - 1; t >= t0; --s) {
        if (s < 0 || s >= a.view.num_seqs) break;
        a.view.range(s, start, end);
        if (start > t || end == start) continue;
        // rows after the tile in the same sequence
        long long after = t + (W - 1) < end - 1 ? t + (W - 1) : end - 1;
        open(after);
        for (; after > t; --after) {
            Row<T, V> g;
            g.load(dy + after * a.ld_dy);
            step(input(after - (W - 1)), g);
        }
        const long long low = start > t0 ? start : t0;
        const int n = (int)(t - low + 1);
        To* out = (To*)a.dx + t * a.D + c;
        auto finish = [&](To* to, long long with_state) {
            f2 v[H];
            pull(v);
            if (with_state >= 0) from_state(with_state, v);
            store_row<To, V>(to, v);
#pragma unroll
            for (int i = 0; i < H; ++i) {
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][i] = fma2(q[0][i], win[j][i], dw[j][i]);
                db[i] = add2(db[i], q[0][i]);
            }
        };
        // The rows that state_out holds, one by one; whole groups of rows, so that
        // the windows' shifts are a renaming of registers; the rest one by one.
        const long long held = t - end + W;
        const int head = dst && held > 0 ? (int)(held < n ? held : n) : 0;
        const int whole = head + (n - head) / BACK_AHEAD * BACK_AHEAD;
        auto single = [&](int at, bool with_state) {
            Row<T, V> g;
            g.load(dy + (t - at) * a.ld_dy);
            step(input(t - at - (W - 1)), g);
            finish(out - (long long)at * a.D, with_state ? t - at : -1);
        };
#pragma unroll 1
        for (int at = 0; at < head; ++at) single(at, true);
        Row<T, V> xs[BACK_AHEAD], gs[BACK_AHEAD];
        auto load = [&](long long tok) {
            const T* xp = x + (tok - (W - 1)) * a.ld_x;
            const T* gp = dy + tok * a.ld_dy;
            if (tok - (BACK_AHEAD - 1) - (W - 1) >= start) {
#pragma unroll
                for (int k = 0; k < BACK_AHEAD; ++k) xs[k].load(xp - (long long)k * a.ld_x);
            } else {
#pragma unroll
                for (int k = 0; k < BACK_AHEAD; ++k) xs[k] = input(tok - k - (W - 1));
            }
#pragma unroll
            for (int k = 0; k < BACK_AHEAD; ++k) gs[k].load(gp - (long long)k * a.ld_dy);
        };
        if (whole > head) load(t - head);
#pragma unroll 1
        for (int at = head; at < whole; at += BACK_AHEAD) {
            Row<T, V> xn[BACK_AHEAD], gn[BACK_AHEAD];
#pragma unroll
            for (int k = 0; k < BACK_AHEAD; ++k) xn[k] = xs[k], gn[k] = gs[k];
            if (at + BACK_AHEAD < whole) load(t - at - BACK_AHEAD);
#pragma unroll
            for (int k = 0; k < BACK_AHEAD; ++k) {
                step(xn[k], gn[k]);
                finish(out - (long long)(at + k) * a.D, -1);
            }
        }
#pragma unroll 1
        for (int at = whole; at < n; ++at) single(at, false);
        t -= n;
    }
    float out[2 * H][W], ob[2 * H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) unpack(dw[j][i], out[2 * i][j], out[2 * i + 1][j]);
        unpack(db[i], ob[2 * i], ob[2 * i + 1]);
    }
    float* dwp = a.dw_part + (tile * a.D + c) * W;
    float* dbp = a.db_part + tile * a.D + c;
    if constexpr (V == 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) dwp[j] = out[0][j];
        dbp[0] = ob[0];
    } else {
        const float* flat = &out[0][0];
#pragma unroll
        for (int i = 0; i < V * W; i += 4)
            *reinterpret_cast<float4*>(dwp + i) =
                make_float4(flat[i], flat[i + 1], flat[i + 2], flat[i + 3]);
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(dbp + i) = make_float4(ob[i], ob[i + 1], ob[i + 2], ob[i + 3]);
    }
}

// Whether every row of p starts on a vector of four elements.
bool on_vectors(const void* p, long long ld, size_t e)
{
    return (uintptr_t)p % (4 * e) == 0 && ld % 4 == 0;
}

// Calls F<T, To, W, V>: V = 4 channels per thread when every row of every
// tensor starts on a vector of four, else 1.
#define LA_CONV_CASE(F, T, To, W)                                                                \
    if (vec) F(T, To, W, 4);                                                                     \
    else F(T, To, W, 1)
#define LA_CONV_TYPES(F, W)                                                                      \
    if (p.in_t == LA_F32) { LA_CONV_CASE(F, float, float, W); }                               \
    else if (p.out_t == LA_F32) { LA_CONV_CASE(F, __nv_bfloat16, float, W); }                 \
    else { LA_CONV_CASE(F, __nv_bfloat16, __nv_bfloat16, W); }
#define LA_CONV_DISPATCH(F)                                                                      \
    if (p.W == 2) { LA_CONV_TYPES(F, 2) }                                                        \
    else if (p.W == 3) { LA_CONV_TYPES(F, 3) }                                                   \
    else { LA_CONV_TYPES(F, 4) }

// Rows per CTA: as many as make the CTAs a whole number of full waves of about
// `about` rows (`resident` CTAs run at once), at least 16.
int tile_rows(long long total, int cblocks, int resident, int about)
{
    const long long rows = total * cblocks;
    long long waves = (rows + (long long)resident * about / 2) / ((long long)resident * about);
    if (waves < 1) waves = 1;
    const long long t = (rows + resident * waves - 1) / (resident * waves);
    return (int)(t < 16 ? 16 : t);
}
constexpr int BACK_RESIDENT = 148 * 4, BACK_ABOUT = 128;

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
    const int V = vec ? 4 : 1;
    a.cblocks = (p.D + NT * V - 1) / (NT * V);
    return a;
}

bool use_vectors(const ConvProblem& p)
{
    return p.D % 4 == 0 && on_vectors(p.x, p.ld_x, p.in_t == LA_BF16 ? 2 : 4);
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
    const long long rows = p.view.total * a.cblocks;
    a.tile = rows >= 148 * 8 * 64 ? 64 : rows >= 148 * 8 * 32 ? 32 : 16;  // fill the SMs
    a.tiles = (p.view.total + a.tile - 1) / a.tile;
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
    size_t tiles = 0;  // whichever number of channels a thread takes
    for (int V : {1, 4}) {
        const int tile = tile_rows(total, (D + NT * V - 1) / (NT * V), BACK_RESIDENT, BACK_ABOUT);
        const size_t n = (size_t)((total + tile - 1) / tile);
        tiles = n > tiles ? n : tiles;
    }
    return align_up(tiles * D * W * 4, 256) + align_up(tiles * D * 4, 256);
}

cudaError_t launch_short_conv_backward(const ConvProblem& p, const void* dy, long long ld_dy,
                                       const void* state_in, const void* dstate_out, void* dx,
                                       float* dweight, float* dbias, void* dstate_in, void* ws,
                                       cudaStream_t stream)
{
    const bool vec = use_vectors(p) && on_vectors(dy, ld_dy, p.in_t == LA_BF16 ? 2 : 4);
    ConvArgs a = base_args(p, vec);
    a.state_in = state_in;
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.dstate_out = dstate_out;
    a.dx = dx;
    a.dstate_in = dstate_in;
    a.tile = tile_rows(p.view.total, a.cblocks, BACK_RESIDENT, BACK_ABOUT);
    a.tiles = (p.view.total + a.tile - 1) / a.tile;
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
    SumJobs sums;
    sums.add(a.dw_part, dweight, (int)a.tiles, (long long)p.D * p.W);
    sums.add(a.db_part, dbias, (int)a.tiles, p.D);
    return launch_column_sums(sums, stream);
}

}  // namespace la
