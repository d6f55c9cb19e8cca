// The selective scan over prompts and for single tokens.
//
//     dt = softplus(delta + bias),  h_t = exp(dt A) h_{t-1} + dt u B_t,
//     y_t = (C_t . h_t + D u) z sigmoid(z)
//
// A channel's n states are scanned token by token in registers: the chain
// from token to token is one multiply-add, everything else is off it. What
// bounds it is the special function unit, 16 results per clock and SM: n
// exponentials per (token, channel), and two each for the softplus and the
// gate. For n = 16 that is 4.3 ps per (token, channel) on 148 SMs at 1.965 GHz,
// against 1.2 ps for the bf16 inputs and outputs at 6.5 TB/s. Measured: 8 x 2K
// tokens of 8192 channels 797 us, 5.9 ps; 8K tokens of one sequence 505 us, 7.5
// ps (64 channels per CTA leave 20 SMs idle and one scanning warp to each
// scheduler of the others).
//
// When the channels of all sequences do not fill the GPU, the sequences are
// cut into chunks: a first launch computes every chunk's state from zero (the
// first chunk's from the incoming state) and the sum of its dt, whose
// exponential exp(A sum dt) is the chunk's whole decay; the second launch
// folds the chunks before its own, h <- exp(A sum dt_c) h + h_c, and scans
// with outputs. That takes the exponentials twice, so it pays from about
// three chunks on: 46K packed fp32 tokens of 1024 channels take 664 us (under the
// profiler, launch by launch, 4 for the table of chunks, 288 and 388), against
// 385 for the exponentials of both walks. Scanning and serving threads share one
// register budget, 80 with 256 servers and 96 with 512: the first launch spills
// for n above 4 (60 to 84 bytes stored), the second with fp32 inputs, 256
// servers and n up to 16 (132 to 156). What that costs has not been measured.
#include <climits>

#include "ssm_scan.cuh"

namespace la {
namespace {

constexpr int NT = 128;  // scanning threads per CTA

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
    int out_f32;
};

// Named barriers of a CTA: `arrive` counts this warp in without waiting.
template <int THREADS> __device__ __forceinline__ void bar_sync(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}
template <int THREADS> __device__ __forceinline__ void bar_arrive(int id)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}

// A CTA's chunk and channels, the same for all its threads.
struct Place {
    int s, chunk, nchunks, item, g, c0, c_end;
    long long t0, t1;
};

// One of the CTA's two sets of buffers, for TT tokens of CC channels: K lanes
// share two adjacent channels.
template <int K> struct ScanTile {
    static constexpr int NP = SCAN_S * K, CC = 2 * NT / K;
    static constexpr int TT = K == 1 ? 8 : K == 2 ? 16 : 32;
    float4 dt[TT][CC / 2];  // dt, dt u of the pair's first channel, then of its second
    float b[TT][NP];
    float c[TT][NP];
    f2 y[TT][NT];           // each scanning thread's share of C . h, for both channels
};

template <int K, int MODE, int SV>
__device__ __forceinline__ void scan_threads(const ScanArgs& a, const Place& p, ScanTile<K>* tiles)
{
    constexpr int S = SCAN_S, TT = ScanTile<K>::TT;
    const int tid = threadIdx.x;
    const int pr = tid / K, m0 = (tid % K) * S, c0 = p.c0 + 2 * pr;
    const bool last = p.chunk == p.nchunks - 1;

    float A[2][S], h[2][S];
    float* const local = a.local;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int i = 0; i < S; ++i) A[x][i] = h[x][i] = 0.f;
        const int c = c0 + x;
        if (c >= p.c_end) continue;
        load_states(A[x], a.in.A + (long long)c * a.n, m0, a.n);
#pragma unroll
        for (int i = 0; i < S; ++i) A[x][i] = decay_rate(A[x][i]);
        const float* in = a.state_in ? a.state_in + ((long long)p.s * a.D + c) * a.n : nullptr;
        const long long slot = ((long long)p.item * a.D + c) * a.n;
        if (MODE == 1) {
            // The last chunk's slot is free: it keeps the incoming state, which
            // may be overwritten in place before the first chunk reads it.
            if (in && (p.chunk == 0 || last)) load_states(h[x], in, m0, a.n);
            if (last) store_states(local + slot, h[x], m0, a.n);
        } else if (p.nchunks == 1) {
            if (in) load_states(h[x], in, m0, a.n);
        } else if (p.chunk == 0) {
            load_states(h[x], local + slot + (long long)(p.nchunks - 1) * a.D * a.n, m0, a.n);
        } else {
            const long long first = (long long)(p.item - p.chunk) * a.D + c;
            load_states(h[x], local + first * a.n, m0, a.n);
#pragma unroll 4
            for (int k = 1; k < p.chunk; ++k) {
                float l[S];
                load_states(l, local + (first + (long long)k * a.D) * a.n, m0, a.n);
                const float d = a.dtsum[first + (long long)k * a.D];
#pragma unroll
                for (int i = 0; i < S; ++i) h[x][i] = fmaf(ex2(d * A[x][i]), h[x][i], l[i]);
            }
        }
    }
    if (MODE == 1 && last) return;
    f2 hp[2][2], Ap[2][2], dts = pack(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        hp[x][0] = pack(h[x][0], h[x][1]), hp[x][1] = pack(h[x][2], h[x][3]);
        Ap[x][0] = pack(A[x][0], A[x][1]), Ap[x][1] = pack(A[x][2], A[x][3]);
    }
    int turn = 0;
#pragma unroll 1
    for (long long t = p.t0; t < p.t1; t += TT, turn ^= 1) {
        ScanTile<K>& w = tiles[turn];
        bar_sync<NT + SV>(1 + turn);
        // The inputs of the next Q tokens are read before the outputs of these
        // are written: the compiler keeps shared reads behind earlier writes.
        constexpr int Q = 2;
        struct In {
            float4 d;
            ulonglong2 b, c;
        } now[Q], then[Q];
        auto read = [&](int row, In* in) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                in[q].d = w.dt[row + q][pr];
                in[q].b = *reinterpret_cast<const ulonglong2*>(&w.b[row + q][m0]);
                if (MODE == 0) in[q].c = *reinterpret_cast<const ulonglong2*>(&w.c[row + q][m0]);
            }
        };
        read(0, then);
#pragma unroll
        for (int tb = 0; tb < TT; tb += Q) {
#pragma unroll
            for (int q = 0; q < Q; ++q) now[q] = then[q];
            if (tb + Q < TT) read(tb + Q, then);
            f2 y[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const float4 d = now[q].d;
                const f2 dt[2] = {pack(d.x, d.x), pack(d.z, d.z)};
                const f2 du[2] = {pack(d.y, d.y), pack(d.w, d.w)};
                float yx[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    hp[x][0] = fma2(ex2_2(mul2(dt[x], Ap[x][0])), hp[x][0], mul2(du[x], now[q].b.x));
                    hp[x][1] = fma2(ex2_2(mul2(dt[x], Ap[x][1])), hp[x][1], mul2(du[x], now[q].b.y));
                    if (MODE == 0) {
                        float lo, hi;
                        unpack(fma2(now[q].c.y, hp[x][1], mul2(now[q].c.x, hp[x][0])), lo, hi);
                        yx[x] = lo + hi;
                    }
                }
                if (MODE == 0) y[q] = pack(yx[0], yx[1]);
                else dts = add2(dts, pack(d.x, d.z));
            }
            if (MODE == 0) {
#pragma unroll
                for (int q = 0; q < Q; ++q) w.y[tb + q][tid] = y[q];
            }
        }
        bar_arrive<NT + SV>(3 + turn);
    }
    float d[2];
    unpack(dts, d[0], d[1]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int c = c0 + x;
        if (c >= p.c_end) continue;
        unpack(hp[x][0], h[x][0], h[x][1]);
        unpack(hp[x][1], h[x][2], h[x][3]);
        if (MODE == 1) {
            store_states(local + ((long long)p.item * a.D + c) * a.n, h[x], m0, a.n);
            if (m0 == 0) a.dtsum[(long long)p.item * a.D + c] = d[x];
        } else if (last && a.state_out) {
            store_states(a.state_out + ((long long)p.s * a.D + c) * a.n, h[x], m0, a.n);
        }
    }
}

template <typename T, int K, int MODE, bool VEC, int SV>
__device__ __forceinline__ void serve_threads(const ScanArgs& a, const Place& p, ScanTile<K>* tiles)
{
    using Tile = ScanTile<K>;
    constexpr int NP = Tile::NP, CP = Tile::CC / 2, TT = Tile::TT;
    constexpr int RP = SV / CP, E = (TT + RP - 1) / RP;  // rows between a thread's pairs; pairs
    constexpr int RB = SV / NP, EB = (TT + RB - 1) / RB;
    constexpr uint32_t TS = sizeof(T);
    const int tid = threadIdx.x - NT;
    const int pr = tid % CP, prow = tid / CP;
    const int ec = p.c0 + 2 * pr;
    // Channels behind the group's last read the last ones.
    const bool lo_ok = ec < p.c_end, hi_ok = ec + 1 < p.c_end;
    const int ch = lo_ok ? 2 * pr : p.c_end - p.c0 - (VEC ? 2 : 1);
    const uint32_t next = hi_ok ? TS : 0;
    const int bm = tid % NP, brow = tid / NP;
    const bool bm_ok = bm < a.n;
    // Addresses are a base that all threads share, which moves from tile to tile
    // and from row to row, and a thread's own 32-bit offset from it.
    const uint32_t lu = (uint32_t)a.in.ld_u * TS, ld = (uint32_t)a.in.ld_delta * TS;
    const uint32_t lz = (uint32_t)a.in.ld_z * TS;
    const uint32_t lb = (uint32_t)a.in.ld_b * TS, lc = (uint32_t)a.in.ld_c * TS;
    const char* up = (const char*)a.in.u + ((long long)p.c0 + p.t0 * a.in.ld_u) * TS;
    const char* dp = (const char*)a.in.delta + ((long long)p.c0 + p.t0 * a.in.ld_delta) * TS;
    const char* zp = (const char*)a.in.z + ((long long)p.c0 + p.t0 * a.in.ld_z) * TS;
    const char* Bp = (const char*)a.in.B + ((long long)p.g * a.n + p.t0 * a.in.ld_b) * TS;
    const char* Cp = (const char*)a.in.C + ((long long)p.g * a.n + p.t0 * a.in.ld_c) * TS;
    const uint32_t ch_at = ch * TS, bm_at = (bm_ok ? bm : 0) * TS;
    const uint32_t ou = prow * lu + ch_at, od = prow * ld + ch_at, oz = prow * lz + ch_at;
    const uint32_t ob = brow * lb + bm_at, oc = brow * lc + bm_at;
    const bool gated = MODE == 0 && a.in.z != nullptr;
    f2 bias = pack(0.f, 0.f), Dw = pack(0.f, 0.f);
    if (a.in.delta_bias && lo_ok)
        bias = pack(a.in.delta_bias[ec], hi_ok ? a.in.delta_bias[ec + 1] : 0.f);
    if (MODE == 0 && a.in.D && lo_ok) Dw = pack(a.in.D[ec], hi_ok ? a.in.D[ec + 1] : 0.f);

    Pair<T, VEC> ru[E], rd[E], rz[E], pu[E], pz[E];  // of the next tile; of the last one
    T rB[EB], rC[EB];
    // Rows of a tile are counted from its first; rows behind rmax read that one.
    auto load = [&](int rmax) {
        if (rmax == TT - 1 && TT % RB == 0 && TT % RP == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ru[e].load(up + (long long)(e * RP) * lu + ou, next);
                rd[e].load(dp + (long long)(e * RP) * ld + od, next);
                if (gated) rz[e].load(zp + (long long)(e * RP) * lz + oz, next);
            }
#pragma unroll
            for (int e = 0; e < EB; ++e) {
                rB[e] = *reinterpret_cast<const T*>(Bp + (long long)(e * RB) * lb + ob);
                if (MODE == 0)
                    rC[e] = *reinterpret_cast<const T*>(Cp + (long long)(e * RB) * lc + oc);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint32_t row = min(prow + e * RP, rmax);
                ru[e].load(up + (row * lu + ch_at), next);
                rd[e].load(dp + (row * ld + ch_at), next);
                if (gated) rz[e].load(zp + (row * lz + ch_at), next);
            }
#pragma unroll
            for (int e = 0; e < EB; ++e) {
                const uint32_t row = min(brow + e * RB, rmax);
                rB[e] = *reinterpret_cast<const T*>(Bp + (row * lb + bm_at));
                if (MODE == 0) rC[e] = *reinterpret_cast<const T*>(Cp + (row * lc + bm_at));
            }
        }
        up += (long long)TT * lu;
        dp += (long long)TT * ld;
        zp += (long long)TT * lz;
        Bp += (long long)TT * lb;
        Cp += (long long)TT * lc;
    };
    // The outputs of the tile at t, whose shares are in w.
    auto finish = [&](long long t, const Tile& w) {
        const int rows = (int)(p.t1 - t < TT ? p.t1 - t : TT);
        const int os = a.out_f32 ? 4 : 2;
        char* const out = (char*)a.y + (t * a.D + p.c0) * os;
        const uint32_t at = (uint32_t)(prow * a.D + 2 * pr) * os;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int row = prow + e * RP;
            if (row >= rows || !lo_ok) continue;
            f2 y;
            if constexpr (K == 1) {
                y = w.y[row][pr];
            } else {
                const ulonglong2* v = reinterpret_cast<const ulonglong2*>(&w.y[row][pr * K]);
                y = add2(v[0].x, v[0].y);
#pragma unroll
                for (int k = 1; k < K / 2; ++k) y = add2(y, add2(v[k].x, v[k].y));
            }
            y = fma2(Dw, pu[e].get(), y);
            if (gated) {
                const f2 z = pz[e].get();
                y = mul2(y, mul2(z, sigmoid2(z)));
            }
            char* const o = out + (long long)(e * RP) * a.D * os + at;
            float lo, hi;
            unpack(y, lo, hi);
            if (a.out_f32) {
                if (VEC) *reinterpret_cast<f2*>(o) = y;
                else {
                    reinterpret_cast<float*>(o)[0] = lo;
                    if (hi_ok) reinterpret_cast<float*>(o)[1] = hi;
                }
            } else {
                if (VEC) *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(lo, hi);
                else {
                    reinterpret_cast<__nv_bfloat16*>(o)[0] = __float2bfloat16_rn(lo);
                    if (hi_ok) reinterpret_cast<__nv_bfloat16*>(o)[1] = __float2bfloat16_rn(hi);
                }
            }
        }
    };

    int rmax = (int)(p.t1 - p.t0 < TT ? p.t1 - p.t0 : TT) - 1, turn = 0;
    if (p.t0 < p.t1) load(rmax);
#pragma unroll 1
    for (long long t = p.t0; t < p.t1; t += TT, turn ^= 1) {
        Tile& w = tiles[turn];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int row = prow + e * RP;
            f2 dt = add2(rd[e].get(), bias);
            if (a.in.softplus) dt = softplus2(dt);
            f2 du = mul2(dt, ru[e].get());
            if (row > rmax) dt = du = pack(0.f, 0.f);  // decay 1, nothing added
            float4 v;
            unpack(dt, v.x, v.z);
            unpack(du, v.y, v.w);
            if (TT % RP == 0 || row < TT) w.dt[row][pr] = v;
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int row = brow + e * RB;
            if (TT % RB == 0 || row < TT) {
                w.b[row][bm] = bm_ok && row <= rmax ? to_f32(rB[e]) : 0.f;
                if (MODE == 0) w.c[row][bm] = bm_ok && row <= rmax ? to_f32(rC[e]) : 0.f;
            }
        }
        bar_arrive<NT + SV>(1 + turn);
        // The scan is done with the other set: it may be stored and filled again.
        if (t > p.t0) {
            bar_sync<NT + SV>(3 + (turn ^ 1));
            if (MODE == 0) finish(t - TT, tiles[turn ^ 1]);
        }
        if (MODE == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) pu[e] = ru[e], pz[e] = rz[e];
        }
        if (t + TT < p.t1) {
            rmax = (int)(p.t1 - t - TT < TT ? p.t1 - t - TT : TT) - 1;
            load(rmax);
        }
    }
    if (p.t0 < p.t1) {
        const int final_turn = turn ^ 1;
        bar_sync<NT + SV>(3 + final_turn);
        if (MODE == 0) finish(p.t0 + (p.t1 - p.t0 - 1) / TT * TT, tiles[final_turn]);
    }
}

// MODE 0: with outputs. MODE 1: the chunks' states only.
//
// The CTA's first NT threads scan, the other SV serve them, tile by tile of TT
// tokens through two sets of shared buffers. The servers turn pairs of channels
// into dt and dt u; the scanning threads carry four states of two channels each
// over the tile and leave their shares of C . h; the servers add the K shares,
// the skip and the gate and store. So the exponentials of the scan run while the
// next tile is made and the last one stored. Two channels per thread, because
// what a thread reads from shared memory per token (B, C and its dt, dt u, a
// wavefront per word whether other lanes read the same word or not) otherwise
// takes longer than its exponentials: with one channel, 8K x 8192 took 681 us.
// 512 servers where every CTA has an SM to itself (505 us against 572 with 256),
// 256 where two CTAs share one (8 x 2K x 8192: 797 us against 943 with one).
template <typename T, int K, int MODE, bool VEC, int SV>
__global__ void __launch_bounds__(NT + SV, SV == 256 ? 2 : 1) scan_kernel(ScanArgs a)
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
    if (threadIdx.x < NT) scan_threads<K, MODE, SV>(a, p, tiles);
    else if (MODE == 0 || p.chunk < p.nchunks - 1) serve_threads<T, K, MODE, VEC, SV>(a, p, tiles);
}

// One token per sequence: the states are the traffic, one vector of four per
// thread and sequence, read and written once. A thread takes one channel of BB
// sequences, for which it reads the weights once and whose loads it starts
// together. What depends on the channel alone is shared out: each of the
// channel's K lanes makes dt, dt u and the gate of BB / K sequences, passes the
// former on, and finishes the output of the same ones. 256 sequences of 8192
// channels, 16 states: 61-63 us, 4.5-4.7 TB/s (every lane making every element
// 120 us, with bounds checks on whole vectors 95 us). It is latency that keeps it
// from the 44 us of its bytes: a CTA takes one group of sequences, waits for all
// its loads and has nothing on its way while it computes and stores.
constexpr int BB = 4;

// Four of B or C at p (the thread's first is m0 of n).
template <typename T, bool FULL>
__device__ __forceinline__ void load_four(float* v, const T* p, int m0, int n, bool vec)
{
    if (FULL || vec) {
        if constexpr (sizeof(T) == 2) {
            const uint2 w = FULL || m0 < n ? *reinterpret_cast<const uint2*>(p + m0)
                                           : make_uint2(0, 0);
            v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
            v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
            load_states<FULL>(v, p, m0, n);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = m0 + i < n ? to_f32(p[m0 + i]) : 0.f;
    }
}

// FULL: n = 4 K, and B and C are on vectors of four.
template <typename T, int K, bool FULL>
__global__ void __launch_bounds__(128) scan_step_kernel(la_scan_inputs in, float* state, void* y,
                                                        int B, int D, int G, int n, int cblocks,
                                                        bool vec, int out_f32)
{
    constexpr int S = SCAN_S, CC = 128 / K;
    constexpr int EL = K < BB ? BB / K : 1;  // sequences whose elements a lane makes
    const int tid = threadIdx.x, lane = tid & 31, m0 = (tid % K) * S;
    const int c_ = blockIdx.x % cblocks * CC + tid / K, b0 = blockIdx.x / cblocks * BB;
    const bool c_ok = c_ < D;
    const int c = c_ok ? c_ : D - 1, g = G == 1 ? 0 : c / (D / G);
    float h[BB][S], A[S], Bv[BB][S], Cv[BB][S];
    const float* hp = state + ((long long)b0 * D + c) * n;
#pragma unroll
    for (int i = 0; i < BB; ++i) {
        const long long b = min(b0 + i, B - 1) - b0;
        load_states<FULL>(h[i], hp + b * D * n, m0, n);
    }
    const int mine = b0 + reduced_index<BB, K, 1>(lane);
    float u[EL], d[EL], z[EL];
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        const long long b = min(mine + e, B - 1);
        u[e] = to_f32(((const T*)in.u)[b * in.ld_u + c]);
        d[e] = to_f32(((const T*)in.delta)[b * in.ld_delta + c]);
        z[e] = in.z ? to_f32(((const T*)in.z)[b * in.ld_z + c]) : 0.f;
    }
    const T* Bp = (const T*)in.B + b0 * in.ld_b + (long long)g * n;
    const T* Cp = (const T*)in.C + b0 * in.ld_c + (long long)g * n;
#pragma unroll
    for (int i = 0; i < BB; ++i) {
        const long long b = min(b0 + i, B - 1) - b0;
        load_four<T, FULL>(Bv[i], Bp + b * in.ld_b, m0, n, vec);
        load_four<T, FULL>(Cv[i], Cp + b * in.ld_c, m0, n, vec);
    }
    load_states<FULL>(A, in.A + (long long)c * n, m0, n);
#pragma unroll
    for (int s = 0; s < S; ++s) A[s] = decay_rate(A[s]);
    const float bias = in.delta_bias ? in.delta_bias[c] : 0.f;
    float acc[BB];
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        d[e] += bias;
        if (in.softplus) d[e] = softplus_f(d[e]);
    }
#pragma unroll
    for (int i = 0; i < BB; ++i) {
        constexpr int PER = K > BB ? K / BB : 1;  // lanes with the same sequence
        const int from = (lane & ~(K - 1)) + (K > BB ? i * PER : i / EL);
        const float dt = __shfl_sync(0xffffffffu, d[i % EL], from);
        const float du = dt * __shfl_sync(0xffffffffu, u[i % EL], from);
        acc[i] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            h[i][s] = fmaf(ex2(dt * A[s]), h[i][s], du * Bv[i][s]);
            acc[i] = fmaf(Cv[i][s], h[i][s], acc[i]);
        }
    }
    lane_reduce<BB, K, 1>(acc, lane);
    if (!c_ok) return;
    float* hq = state + ((long long)b0 * D + c) * n;
#pragma unroll
    for (int i = 0; i < BB; ++i)
        if (b0 + i < B) store_states<FULL>(hq + (long long)i * D * n, h[i], m0, n);
    if (!reduced_writer<BB, K, 1>(lane)) return;
    const float Dw = in.D ? in.D[c] : 0.f;
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        if (mine + e >= B) continue;
        float v = fmaf(Dw, u[e], acc[e]);
        if (in.z) v *= z[e] * sigmoid_f(z[e]);
        const long long p = (long long)(mine + e) * D + c;
        if (out_f32) ((float*)y)[p] = v;
        else ((__nv_bfloat16*)y)[p] = __float2bfloat16_rn(v);
    }
}

// Tables of a packed batch's chunks: one CTA.
__global__ void __launch_bounds__(1024) plan_chunks_kernel(SeqView v, long long len, int items,
                                                           int* first, int* seq_of)
{
    __shared__ long long warp_sum[32];  // offsets that are not sorted can pass 32 bits
    __shared__ int carry;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (tid == 0) carry = 0;
    __syncthreads();
    for (int base = 0; base < v.num_seqs; base += 1024) {
        const int s = base + tid;
        long long x = 0;
        if (s < v.num_seqs) {
            long long t0, t1;
            v.range(s, t0, t1);
            const long long c = (t1 - t0 + len - 1) / len;
            x = c > 1 ? c : 1;
        }
        long long sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane == 31) warp_sum[w] = sum;
        __syncthreads();
        long long before = carry;
        for (int i = 0; i < w; ++i) before += warp_sum[i];
        const long long at = before + sum - x;  // nor may they pass the table's end
        if (s < v.num_seqs) first[s] = (int)(at < items ? at : items);
        __syncthreads();
        if (tid == 1023) carry = (int)(before + sum < items ? before + sum : items);
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

constexpr int SMS = 148;

struct ForwardPlan {
    long long len;  // tokens per chunk, 0: one chunk per sequence
    int items;
};

// How the forward scan is cut: into about two CTAs per SM (three or four per SM
// took 817 and 671 us against 668 on the packed batch above). A packed batch's lengths are not known here, so
// that it counts as one long sequence: where its sequences are shorter than a
// chunk, the first launch finds nothing to do.
ForwardPlan plan_forward(bool packed, int G, int D, long long total, int n, int num_seqs)
{
    const int CC = 2 * NT / scan_lanes(n);
    const long long ctas = (long long)G * ((D / G + CC - 1) / CC);
    if (num_seqs == 0 || total == 0 || (packed ? 1 : num_seqs) * ctas * 2 > SMS)
        return {0, num_seqs};
    long long want = 2 * SMS / ctas;  // chunks in all: two CTAs per SM
    if (want > 64) want = 64;
    long long len = ((total + want - 1) / want + 31) / 32 * 32;
    if (len < 64) len = 64;
    // Below three chunks the second walk costs what the cut gains.
    if ((packed ? total : total / num_seqs) <= 2 * len) return {0, num_seqs};
    return {len, (int)(total / len + num_seqs)};
}

// The pass over the chunks' states (when cut) and the pass with outputs.
template <int K, int SV>
cudaError_t launch_tiles(void (*states)(ScanArgs), void (*outputs)(ScanArgs), const ScanArgs& a,
                         bool cut, unsigned grid, cudaStream_t stream)
{
    constexpr int smem = 2 * (int)sizeof(ScanTile<K>);
    for (auto kernel : {cut ? states : nullptr, outputs}) {
        if (!kernel) continue;
        cudaError_t e = allow_shared((const void*)kernel, smem);
        if (e != cudaSuccess) return e;
        kernel<<<grid, NT + SV, smem, stream>>>(a);
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
    const int K = scan_lanes(p.n), CC = 2 * NT / K, Dg = p.D / p.G;
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
    const bool vec = Dg % 2 == 0 && pairs(p.in.u, p.in.ld_u) && pairs(p.in.delta, p.in.ld_delta) &&
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
#define LA_TYPE(T, KK)                                                                           \
    if (!vec)                                                                                    \
        e = launch_tiles<KK, 256>(scan_kernel<T, KK, 1, false, 256>,                             \
                                  scan_kernel<T, KK, 0, false, 256>, a, f.len != 0, grid, stream); \
    else if (grid <= SMS)                                                                        \
        e = launch_tiles<KK, 512>(scan_kernel<T, KK, 1, true, 512>,                              \
                                  scan_kernel<T, KK, 0, true, 512>, a, f.len != 0, grid, stream); \
    else                                                                                         \
        e = launch_tiles<KK, 256>(scan_kernel<T, KK, 1, true, 256>,                              \
                                  scan_kernel<T, KK, 0, true, 256>, a, f.len != 0, grid, stream)
#define LA_CALL(KK)                                                                              \
    if (p.in_t == LA_BF16) { LA_TYPE(__nv_bfloat16, KK); }                                       \
    else { LA_TYPE(float, KK); }
    LA_SCAN_DISPATCH_K(p.n, LA_CALL)
#undef LA_CALL
#undef LA_TYPE
    return e;
}

cudaError_t launch_scan_step(const ScanProblem& p, float* state, void* y, cudaStream_t stream)
{
    const int K = scan_lanes(p.n), CC = 128 / K, B = p.view.num_seqs;
    const int cblocks = (p.D + CC - 1) / CC;
    const unsigned grid = (unsigned)((long long)cblocks * ((B + BB - 1) / BB));
    const size_t four = p.in_t == LA_BF16 ? 8 : 16;  // bytes of four of B or C
    const auto fours = [&](const void* q, long long ld) {
        return (uintptr_t)q % four == 0 && ld % 4 == 0;
    };
    const bool vec = p.n % 4 == 0 && fours(p.in.B, p.in.ld_b) && fours(p.in.C, p.in.ld_c);
    const int f32 = p.out_t == LA_F32;
#define LA_STEP(T, KK, FULL)                                                                     \
    scan_step_kernel<T, KK, FULL><<<grid, 128, 0, stream>>>(p.in, state, y, B, p.D, p.G, p.n,    \
                                                            cblocks, vec, f32)
#define LA_CALL(KK)                                                                              \
    if (vec && p.n == SCAN_S * KK) {                                                             \
        if (p.in_t == LA_BF16) LA_STEP(__nv_bfloat16, KK, true);                                 \
        else LA_STEP(float, KK, true);                                                           \
    } else {                                                                                     \
        if (p.in_t == LA_BF16) LA_STEP(__nv_bfloat16, KK, false);                                \
        else LA_STEP(float, KK, false);                                                          \
    }
    LA_SCAN_DISPATCH_K(p.n, LA_CALL)
#undef LA_CALL
#undef LA_STEP
    count_launch();
    return cudaGetLastError();
}

}  // namespace la
