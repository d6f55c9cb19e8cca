// The selective scan over prompts and for single tokens.
//
//     dt = softplus(delta + bias),  h_t = exp(dt A) h_{t-1} + dt u B_t,
//     y_t = (C_t . h_t + D u) z sigmoid(z)
//
// A channel's n states are scanned token by token in registers: the chain
// from token to token is one multiply-add, everything else is off it. What
// bounds it is the exponentials: n per (token, channel) plus four for the
// softplus and the gate, at 16 per clock and SM.
//
// When the channels of all sequences do not fill the GPU, the sequences are
// cut into chunks: a first launch computes every chunk's state from zero (the
// first chunk's from the incoming state) and the sum of its dt, whose
// exponential exp(A sum dt) is the chunk's whole decay; the second launch
// folds the chunks before its own, h <- exp(A sum dt_c) h + h_c, and scans
// with outputs. That takes the exponentials twice, so it pays from about
// three chunks on.
#include <climits>

#include "ssm_scan.cuh"

namespace la {
namespace {

constexpr int NT = 128;  // scanning threads per CTA; as many serve them

struct ScanArgs {
    la_scan_inputs in;
    SeqView view;
    Chunks ch;
    const float* state_in;
    void* y;
    float* state_out;
    float* local;   // [items][D][n], chunked only
    float* dtsum;   // [items][D]
    int D, G, n, cpg;  // cpg: channel blocks per group
    int out_f32, vec;
};

// Two adjacent channels of a token as loaded: one access where `vec` (every
// row of every tensor then starts on such a pair), else two.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    uint32_t w;
    __device__ __forceinline__ void load(const char* base, uint32_t at, uint32_t next, bool vec)
    {
        if (vec) w = *reinterpret_cast<const uint32_t*>(base + at);
        else w = *reinterpret_cast<const uint16_t*>(base + at) |
                 (uint32_t) * reinterpret_cast<const uint16_t*>(base + at + next) << 16;
    }
    __device__ __forceinline__ float lo() const { return __uint_as_float(w << 16); }
    __device__ __forceinline__ float hi() const { return __uint_as_float(w & 0xffff0000u); }
};
template <> struct Pair<float> {
    float x, y;
    __device__ __forceinline__ void load(const char* base, uint32_t at, uint32_t next, bool vec)
    {
        if (vec) {
            const float2 v = *reinterpret_cast<const float2*>(base + at);
            x = v.x, y = v.y;
        } else {
            x = *reinterpret_cast<const float*>(base + at);
            y = *reinterpret_cast<const float*>(base + at + next);
        }
    }
    __device__ __forceinline__ float lo() const { return x; }
    __device__ __forceinline__ float hi() const { return y; }
};

// Named barriers of a CTA: `arrive` counts this warp in without waiting.
__device__ __forceinline__ void bar_sync(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(2 * NT) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(2 * NT) : "memory");
}

// A CTA's chunk and channels, the same for all its threads.
struct Place {
    int s, chunk, nchunks, item, g, c0, c_end;
    long long t0, t1;
};

// MODE 0: with outputs. MODE 1: the chunks' states only.
//
// The CTA's first NT threads scan, the other NT serve them, tile by tile of TT
// tokens through two sets of shared buffers. The servers turn pairs of channels
// into (dt, dt u), each twice in a row as the packed multiplies want them; the
// scanning threads carry four states of one channel each over the tile and
// leave their shares of C . h; the servers add the K shares, the skip and the
// gate and store. So the exponentials of the scan run while the next tile is
// made and the last one stored, and the next inputs are on their way.
template <int K> struct ScanTile {
    static constexpr int NP = SCAN_S * K, CC = NT / K;
    static constexpr int TT = K == 1 ? 8 : K == 2 ? 16 : 32;  // tokens
    ulonglong2 dtu[TT][CC];
    float b[TT][NP];
    float c[TT][NP];
    float y[TT][NT];
};

template <int K, int MODE>
__device__ __forceinline__ void scan_threads(const ScanArgs& a, const Place& p, ScanTile<K>* tiles)
{
    constexpr int S = SCAN_S, TT = ScanTile<K>::TT;
    const int tid = threadIdx.x;
    const int sch = tid / K, m0 = (tid % K) * S, sc = p.c0 + sch;
    const bool ok = sc < p.c_end, last = p.chunk == p.nchunks - 1;

    float A[S] = {0.f, 0.f, 0.f, 0.f}, h[S] = {0.f, 0.f, 0.f, 0.f};
    if (ok) load_states(A, a.in.A + (long long)sc * a.n, m0, a.n);
    const f2 log2e = pack(SCAN_LOG2E, SCAN_LOG2E);
    const f2 A01 = mul2(pack(A[0], A[1]), log2e), A23 = mul2(pack(A[2], A[3]), log2e);
    const long long slot = ((long long)p.item * a.D + sc) * a.n;
    if (ok) {
        const float* in = a.state_in ? a.state_in + ((long long)p.s * a.D + sc) * a.n : nullptr;
        if (MODE == 1) {
            // The last chunk's slot is free: it keeps the incoming state, which
            // may be overwritten in place before the first chunk reads it.
            if (in && (p.chunk == 0 || last)) load_states(h, in, m0, a.n);
            if (last) store_states(a.local + slot, h, m0, a.n);
        } else if (p.nchunks == 1) {
            if (in) load_states(h, in, m0, a.n);
        } else if (p.chunk == 0) {
            load_states(h, a.local + slot + (long long)(p.nchunks - 1) * a.D * a.n, m0, a.n);
        } else {
            const long long first = (long long)(p.item - p.chunk) * a.D + sc;
            load_states(h, a.local + first * a.n, m0, a.n);
#pragma unroll 4
            for (int c = 1; c < p.chunk; ++c) {
                float l[S], e[S];
                load_states(l, a.local + (first + (long long)c * a.D) * a.n, m0, a.n);
                const float d = a.dtsum[first + (long long)c * a.D];
                unpack(ex2_2(mul2(pack(d, d), A01)), e[0], e[1]);
                unpack(ex2_2(mul2(pack(d, d), A23)), e[2], e[3]);
#pragma unroll
                for (int i = 0; i < S; ++i) h[i] = fmaf(e[i], h[i], l[i]);
            }
        }
    }
    if (MODE == 1 && last) return;
    f2 h01 = pack(h[0], h[1]), h23 = pack(h[2], h[3]), dts = pack(0.f, 0.f);
    int turn = 0;
#pragma unroll 1
    for (long long t = p.t0; t < p.t1; t += TT, turn ^= 1) {
        ScanTile<K>& w = tiles[turn];
        bar_sync(1 + turn);
#pragma unroll 2
        for (int tb = 0; tb < TT; tb += 8) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const ulonglong2 d = w.dtu[tb + q][sch];
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&w.b[tb + q][m0]);
                h01 = fma2(ex2_2(mul2(d.x, A01)), h01, mul2(d.y, b.x));
                h23 = fma2(ex2_2(mul2(d.x, A23)), h23, mul2(d.y, b.y));
                if (MODE == 0) {
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&w.c[tb + q][m0]);
                    float lo, hi;
                    unpack(fma2(c.y, h23, mul2(c.x, h01)), lo, hi);
                    w.y[tb + q][tid] = lo + hi;
                } else {
                    dts = add2(dts, d.x);
                }
            }
        }
        bar_arrive(3 + turn);
    }
    if (!ok) return;
    unpack(h01, h[0], h[1]);
    unpack(h23, h[2], h[3]);
    if (MODE == 1) {
        float d, d_;
        unpack(dts, d, d_);
        store_states(a.local + slot, h, m0, a.n);
        if (m0 == 0) a.dtsum[(long long)p.item * a.D + sc] = d;
    } else if (last && a.state_out) {
        store_states(a.state_out + ((long long)p.s * a.D + sc) * a.n, h, m0, a.n);
    }
}

template <typename T, int K, int MODE>
__device__ __forceinline__ void serve_threads(const ScanArgs& a, const Place& p, ScanTile<K>* tiles)
{
    constexpr int NP = ScanTile<K>::NP, CC = ScanTile<K>::CC, TT = ScanTile<K>::TT;
    constexpr int RP = 2 * K;                       // rows between a thread's pairs
    constexpr int E = TT / RP;                      // pairs per thread
    constexpr int RB = NT / NP, EB = (TT + RB - 1) / RB;
    constexpr uint32_t TS = sizeof(T);
    const int tid = threadIdx.x - NT;
    const int pr = tid % (CC / 2), prow = tid / (CC / 2);
    const int ec = p.c0 + 2 * pr;
    // Channels behind the group's last read the last ones.
    const bool lo_ok = ec < p.c_end, hi_ok = ec + 1 < p.c_end;
    const int ch = lo_ok ? 2 * pr : p.c_end - p.c0 - (a.vec ? 2 : 1);
    const uint32_t ch_at = (uint32_t)ch * TS, next = hi_ok ? TS : 0;
    const uint32_t lu = (uint32_t)a.in.ld_u * TS, ld = (uint32_t)a.in.ld_delta * TS;
    const uint32_t lz = (uint32_t)a.in.ld_z * TS;
    const uint32_t lb = (uint32_t)a.in.ld_b * TS, lc = (uint32_t)a.in.ld_c * TS;
    const char* up = (const char*)a.in.u + ((long long)p.c0 + p.t0 * a.in.ld_u) * TS;
    const char* dp = (const char*)a.in.delta + ((long long)p.c0 + p.t0 * a.in.ld_delta) * TS;
    const char* zp = (const char*)a.in.z + ((long long)p.c0 + p.t0 * a.in.ld_z) * TS;
    const char* Bp = (const char*)a.in.B + ((long long)p.g * a.n + p.t0 * a.in.ld_b) * TS;
    const char* Cp = (const char*)a.in.C + ((long long)p.g * a.n + p.t0 * a.in.ld_c) * TS;
    const bool gated = a.in.z != nullptr, vec = a.vec;
    const int bm = tid % NP, brow = tid / NP;
    const bool bm_ok = bm < a.n;
    const uint32_t bm_at = (uint32_t)(bm_ok ? bm : 0) * TS;
    float bias[2] = {0.f, 0.f}, Dw[2] = {0.f, 0.f};
    if (a.in.delta_bias) {
        if (lo_ok) bias[0] = a.in.delta_bias[ec];
        if (hi_ok) bias[1] = a.in.delta_bias[ec + 1];
    }
    if (MODE == 0 && a.in.D) {
        if (lo_ok) Dw[0] = a.in.D[ec];
        if (hi_ok) Dw[1] = a.in.D[ec + 1];
    }

    // Loaded for the next tile; of this tile and of the last one.
    Pair<T> ru[E], rd[E], rz[E], cu[E], cz[E], pu[E], pz[E];
    T rB[EB], rC[EB];
    // Rows of a tile are counted from its first; rmax is the last that exists.
    auto load = [&](int rmax) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t row = min(prow + e * RP, rmax);
            ru[e].load(up, row * lu + ch_at, next, vec);
            rd[e].load(dp, row * ld + ch_at, next, vec);
            if (MODE == 0 && gated) rz[e].load(zp, row * lz + ch_at, next, vec);
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const uint32_t row = min(brow + e * RB, rmax);
            rB[e] = *reinterpret_cast<const T*>(Bp + (row * lb + bm_at));
            if (MODE == 0) rC[e] = *reinterpret_cast<const T*>(Cp + (row * lc + bm_at));
        }
        up += (long long)TT * lu;
        dp += (long long)TT * ld;
        zp += (long long)TT * lz;
        Bp += (long long)TT * lb;
        Cp += (long long)TT * lc;
    };
    // The outputs of the tile at t, whose shares are in w.
    auto finish = [&](long long t, const ScanTile<K>& w) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int row = prow + e * RP;
            float y[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                y[0] += w.y[row][2 * pr * K + k];
                y[1] += w.y[row][(2 * pr + 1) * K + k];
            }
            y[0] = fmaf(Dw[0], pu[e].lo(), y[0]);
            y[1] = fmaf(Dw[1], pu[e].hi(), y[1]);
            if (gated) {
                y[0] *= pz[e].lo() * sigmoid_f(pz[e].lo());
                y[1] *= pz[e].hi() * sigmoid_f(pz[e].hi());
            }
            if (t + row >= p.t1) continue;
            const long long at = (t + row) * a.D + ec;
            if (a.out_f32) {
                float* o = (float*)a.y + at;
                if (vec) {
                    if (lo_ok) *reinterpret_cast<float2*>(o) = make_float2(y[0], y[1]);
                } else {
                    if (lo_ok) o[0] = y[0];
                    if (hi_ok) o[1] = y[1];
                }
            } else {
                __nv_bfloat16* o = (__nv_bfloat16*)a.y + at;
                if (vec) {
                    if (lo_ok)
                        *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(y[0], y[1]);
                } else {
                    if (lo_ok) o[0] = __float2bfloat16_rn(y[0]);
                    if (hi_ok) o[1] = __float2bfloat16_rn(y[1]);
                }
            }
        }
    };

    int rmax = (int)(p.t1 - p.t0 < TT ? p.t1 - p.t0 : TT) - 1, turn = 0;
    if (p.t0 < p.t1) load(rmax);
#pragma unroll 1
    for (long long t = p.t0; t < p.t1; t += TT, turn ^= 1) {
        ScanTile<K>& w = tiles[turn];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (MODE == 0) pu[e] = cu[e], pz[e] = cz[e], cz[e] = rz[e];
            cu[e] = ru[e];
            const int row = prow + e * RP;
            float x = rd[e].lo() + bias[0], y = rd[e].hi() + bias[1];
            if (a.in.softplus) softplus2(x, y);
            float xu = x * cu[e].lo(), yu = y * cu[e].hi();
            if (row > rmax) x = y = xu = yu = 0.f;  // decay 1, nothing added
            w.dtu[row][2 * pr] = make_ulonglong2(pack(x, x), pack(xu, xu));
            w.dtu[row][2 * pr + 1] = make_ulonglong2(pack(y, y), pack(yu, yu));
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int row = brow + e * RB;
            if (TT % RB == 0 || row < TT) {
                w.b[row][bm] = bm_ok && row <= rmax ? to_f32(rB[e]) : 0.f;
                if (MODE == 0) w.c[row][bm] = bm_ok && row <= rmax ? to_f32(rC[e]) : 0.f;
            }
        }
        bar_arrive(1 + turn);
        if (t + TT < p.t1) {
            rmax = (int)(p.t1 - t - TT < TT ? p.t1 - t - TT : TT) - 1;
            load(rmax);
        }
        // The scan is done with the other set: it may be stored and filled again.
        if (t > p.t0) {
            bar_sync(3 + (turn ^ 1));
            if (MODE == 0) finish(t - TT, tiles[turn ^ 1]);
        }
    }
    if (p.t0 < p.t1) {
        const int final_turn = turn ^ 1;
        bar_sync(3 + final_turn);
        if (MODE == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) pu[e] = cu[e], pz[e] = cz[e];
            finish(p.t0 + (p.t1 - p.t0 - 1) / TT * TT, tiles[final_turn]);
        }
    }
}

template <typename T, int K, int MODE>
__global__ void __launch_bounds__(2 * NT, 2) scan_kernel(ScanArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    ScanTile<K>* tiles = reinterpret_cast<ScanTile<K>*>(smem);
    const int blocks = a.G * a.cpg, cb = blockIdx.x % blocks, Dg = a.D / a.G;
    Place p;
    p.item = blockIdx.x / blocks;
    p.s = a.ch.seq(p.item);
    if (p.s < 0) return;
    const int first = a.ch.first_of(p.s);
    p.chunk = p.item - first;
    p.nchunks = a.ch.end_of(p.s) - first;
    a.view.range(p.s, p.t0, p.t1);
    p.t0 += p.chunk * a.ch.len;
    if (p.t1 - p.t0 > a.ch.len) p.t1 = p.t0 + a.ch.len;
    p.g = cb / a.cpg;
    p.c0 = p.g * Dg + (cb % a.cpg) * ScanTile<K>::CC;
    p.c_end = (p.g + 1) * Dg;
    if (threadIdx.x < NT) scan_threads<K, MODE>(a, p, tiles);
    else if (MODE == 0 || p.chunk < p.nchunks - 1) serve_threads<T, K, MODE>(a, p, tiles);
}

// One token per sequence: the states are the traffic, one vector of four per
// thread, read and written once.
template <typename T, int K>
__global__ void __launch_bounds__(256) scan_step_kernel(la_scan_inputs in, float* state, void* y,
                                                        int B, int D, int G, int n, int out_f32)
{
    constexpr int S = SCAN_S;
    const int tid = threadIdx.x, lane = tid & 31;
    const int m0 = (tid % K) * S;
    const long long p = (long long)blockIdx.x * (256 / K) + tid / K;  // sequence * D + channel
    const bool ok = p < (long long)B * D;
    const int b = ok ? (int)(p / D) : 0, c = ok ? (int)(p % D) : 0, g = c / (D / G);
    float h[S], A[S], acc = 0.f;
    load_states(h, state + (ok ? p : 0) * n, m0, n);
    load_states(A, in.A + (long long)c * n, m0, n);
    const float u = to_f32(((const T*)in.u)[b * in.ld_u + c]);
    float dt = to_f32(((const T*)in.delta)[b * in.ld_delta + c]);
    const float z = in.z ? to_f32(((const T*)in.z)[b * in.ld_z + c]) : 0.f;
    const T* Bp = (const T*)in.B + b * in.ld_b + (long long)g * n;
    const T* Cp = (const T*)in.C + b * in.ld_c + (long long)g * n;
    if (in.delta_bias) dt += in.delta_bias[c];
    if (in.softplus) dt = softplus_f(dt);
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const bool in_n = m0 + i < n;
        const float bv = in_n ? to_f32(Bp[m0 + i]) : 0.f, cv = in_n ? to_f32(Cp[m0 + i]) : 0.f;
        h[i] = fmaf(ex2(dt * (A[i] * SCAN_LOG2E)), h[i], dt * u * bv);
        acc = fmaf(cv, h[i], acc);
    }
#pragma unroll
    for (int m = K / 2; m >= 1; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    if (!ok) return;
    store_states(state + p * n, h, m0, n);
    if (lane % K == 0) {
        float v = in.D ? fmaf(in.D[c], u, acc) : acc;
        if (in.z) v *= z * sigmoid_f(z);
        if (out_f32) ((float*)y)[p] = v;
        else ((__nv_bfloat16*)y)[p] = __float2bfloat16_rn(v);
    }
}

// Tables of a packed batch's chunks: one CTA.
__global__ void __launch_bounds__(1024) plan_chunks_kernel(SeqView v, long long len, int items,
                                                           int* first, int* seq_of)
{
    __shared__ int warp_sum[32];
    __shared__ int carry;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (tid == 0) carry = 0;
    __syncthreads();
    for (int base = 0; base < v.num_seqs; base += 1024) {
        const int s = base + tid;
        int x = 0;
        if (s < v.num_seqs) {
            long long t0, t1;
            v.range(s, t0, t1);
            const long long c = (t1 - t0 + len - 1) / len;
            x = (int)(c > 1 ? c : 1);
        }
        int sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane == 31) warp_sum[w] = sum;
        __syncthreads();
        int before = carry;
        for (int i = 0; i < w; ++i) before += warp_sum[i];
        int at = before + sum - x;  // offsets that are not sorted could pass the table's end
        if (s < v.num_seqs) first[s] = at < items ? at : items;
        __syncthreads();
        if (tid == 1023) carry = before + sum < items ? before + sum : items;
        __syncthreads();
    }
    if (tid == 0) first[v.num_seqs] = carry;
    __syncthreads();
    for (int i = tid; i < items; i += 1024) {
        int lo = 0, hi = v.num_seqs + 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= i) lo = mid + 1;
            else hi = mid;
        }
        seq_of[i] = lo > 0 && lo <= v.num_seqs ? lo - 1 : -1;
    }
}

struct ForwardPlan {
    long long len;  // tokens per chunk, 0: one chunk per sequence
    int items;
};

// How the forward scan is cut. One warp on each of the GPU's 592 schedulers is
// what a scan should have at least; chunks are made for two. A packed batch's
// lengths are not known here, so that it counts as one long sequence: where its
// sequences are shorter than a chunk, the first launch finds nothing to do.
ForwardPlan plan_forward(bool packed, int G, int D, long long total, int n, int num_seqs)
{
    constexpr long long SCHEDULERS = 148 * 4;
    const int K = scan_lanes(n), CC = NT / K;
    const long long warps = (long long)G * ((D / G + CC - 1) / CC) * (NT / 32);
    if (num_seqs == 0 || total == 0 || (packed ? 1 : num_seqs) * warps >= SCHEDULERS)
        return {0, num_seqs};
    long long want = (2 * SCHEDULERS + warps - 1) / warps;  // chunks in all
    if (want > 64) want = 64;
    long long len = ((total + want - 1) / want + 31) / 32 * 32;
    if (len < 64) len = 64;
    // Below three chunks the second walk costs what the cut gains.
    if ((packed ? total : total / num_seqs) <= 2 * len) return {0, num_seqs};
    return {len, (int)(total / len + num_seqs)};
}

// The pass over the chunks' states (if any) and the pass with outputs.
template <int K>
cudaError_t launch_tiles(void (*states)(ScanArgs), void (*outputs)(ScanArgs), const ScanArgs& a,
                         unsigned grid, cudaStream_t stream)
{
    constexpr int smem = 2 * (int)sizeof(ScanTile<K>);
    for (auto kernel : {states, outputs}) {
        if (!kernel) continue;
        cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kernel<<<grid, 2 * NT, smem, stream>>>(a);
        count_launch();
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_plan_chunks(const SeqView& v, long long len, int items, int* first, int* seq_of,
                               cudaStream_t stream)
{
    plan_chunks_kernel<<<1, 1024, 0, stream>>>(v, len, items, first, seq_of);
    count_launch();
    return cudaGetLastError();
}

size_t scan_backward_workspace(int G, int D, long long total, int n, int num_seqs);

size_t scan_workspace(bool backward, int G, int D, long long total, int n, int num_seqs)
{
    if (backward) return scan_backward_workspace(G, D, total, n, num_seqs);
    // The larger of what a packed and a dense batch take.
    const ForwardPlan f = plan_forward(true, G, D, total, n, num_seqs);
    if (f.len == 0) return 0;
    return align_up((size_t)f.items * D * n * 4, 256) + align_up((size_t)f.items * D * 4, 256) +
           align_up((size_t)(num_seqs + 1 + f.items) * 4, 256);
}

cudaError_t launch_scan(const ScanProblem& p, const float* state_in, void* y, float* state_out,
                        void* ws, cudaStream_t stream)
{
    const int K = scan_lanes(p.n), CC = NT / K, Dg = p.D / p.G;
    ScanArgs a{};
    a.in = p.in;
    a.view = p.view;
    a.state_in = state_in;
    a.y = y;
    a.state_out = state_out;
    a.D = p.D;
    a.G = p.G;
    a.n = p.n;
    a.cpg = (Dg + CC - 1) / CC;
    a.out_f32 = p.out_t == LA_F32;
    const size_t two = p.in_t == LA_BF16 ? 4 : 8;  // bytes of a pair of channels
    const auto pairs = [&](const void* q, long long ld) {
        return (uintptr_t)q % two == 0 && ld % 2 == 0;
    };
    a.vec = Dg % 2 == 0 && pairs(p.in.u, p.in.ld_u) && pairs(p.in.delta, p.in.ld_delta) &&
            (!p.in.z || pairs(p.in.z, p.in.ld_z));
    const ForwardPlan f = plan_forward(p.view.cu != nullptr, p.G, p.D, p.view.total, p.n,
                                       p.view.num_seqs);
    a.ch.len = LLONG_MAX / 2;
    a.ch.items = p.view.num_seqs;
    if (f.len) {
        char* w = (char*)ws;
        a.local = (float*)w;
        w += align_up((size_t)f.items * p.D * p.n * 4, 256);
        a.dtsum = (float*)w;
        w += align_up((size_t)f.items * p.D * 4, 256);
        a.ch.len = f.len;
        if (p.view.cu) {
            int* first = (int*)w;
            a.ch.items = f.items;
            a.ch.first = first;
            a.ch.seq_of = first + p.view.num_seqs + 1;
            cudaError_t e = launch_plan_chunks(p.view, f.len, f.items, first,
                                               first + p.view.num_seqs + 1, stream);
            if (e != cudaSuccess) return e;
        } else {
            const long long per = (p.view.N + f.len - 1) / f.len;
            a.ch.per_seq = per > 1 ? (int)per : 1;
            a.ch.items = a.ch.per_seq * p.view.num_seqs;
        }
    }
    const unsigned grid = (unsigned)((long long)a.ch.items * a.G * a.cpg);
    cudaError_t e = cudaSuccess;
#define LA_CALL(KK)                                                                              \
    do {                                                                                         \
        const bool low = p.in_t == LA_BF16;                                                      \
        e = launch_tiles<KK>(f.len ? (low ? scan_kernel<__nv_bfloat16, KK, 1>                    \
                                          : scan_kernel<float, KK, 1>)                           \
                                   : nullptr,                                                    \
                             low ? scan_kernel<__nv_bfloat16, KK, 0> : scan_kernel<float, KK, 0>, \
                             a, grid, stream);                                                   \
    } while (0)
    LA_SCAN_DISPATCH_K(p.n, LA_CALL)
#undef LA_CALL
    return e;
}

cudaError_t launch_scan_step(const ScanProblem& p, float* state, void* y, cudaStream_t stream)
{
    const int K = scan_lanes(p.n), CC = 256 / K, B = p.view.num_seqs;
    const unsigned grid = (unsigned)(((long long)B * p.D + CC - 1) / CC);
#define LA_CALL(KK)                                                                              \
    if (p.in_t == LA_BF16)                                                                       \
        scan_step_kernel<__nv_bfloat16, KK><<<grid, 256, 0, stream>>>(p.in, state, y, B, p.D,    \
                                                                      p.G, p.n,                  \
                                                                      p.out_t == LA_F32);        \
    else                                                                                         \
        scan_step_kernel<float, KK><<<grid, 256, 0, stream>>>(p.in, state, y, B, p.D, p.G, p.n,  \
                                                              1);
    LA_SCAN_DISPATCH_K(p.n, LA_CALL)
#undef LA_CALL
    count_launch();
    return cudaGetLastError();
}

}  // namespace la
