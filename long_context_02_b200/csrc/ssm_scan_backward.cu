// Gradients of the selective scan (formulas in lightning.h).
//
// The sequences are cut into chunks of 32 to 128 tokens, all of them independent:
//  1. local pass: each chunk's state from zero, h_c, and that state before every
//     block of 8 tokens; the sums of dt to the same places, whose exponentials
//     exp(A sum dt) are the decays from the chunk's start; and the gradient that
//     the chunk's own outputs send to the state before it,
//     G_c = sum_t (prod_{s<=t} a_s) C_t dyz_t.
//  2. combine: forward over the chunks, the state before each; backward over
//     them, the gradient of the state after each (from dstate_out).
//  3. main pass: the blocks of a chunk from the last to the first. The state
//     before a block is its local part plus the decayed state before the chunk.
//     Half a block at a time, the second half first, a forward walk keeps the
//     states of 4 tokens in registers and a reverse walk carries the gradient;
//     the second half's states need a walk over the first half before. So the
//     exponentials are taken 20 times per 8 tokens here, with the local pass 3.5
//     times in all.
//  4. reductions of dB and dC over the channel blocks and of dA, dD and
//     ddelta_bias over the chunks, from partial sums in the workspace, in a
//     fixed order.
// As in the forward scan a thread holds four states of two channels: what it
// reads from shared memory per token, and the sums over channels (shuffles take
// the same path), would otherwise take longer than the exponentials.
//
// 2 x 4K tokens of 4096 channels, 16 states, bf16: 1,038 us (bytes alone 72 us;
// the exponentials of 3.5 walks and the elementwise ones 483 us), of which
// the local pass 250, combine 25, the main pass 735, the sums 30. No single unit
// bounds the main pass: its warps issue in 55% of the cycles, the special
// function unit is busy in 39%, shared memory in half of them, and four CTAs per
// SM instead of three gain nothing; fewer instructions do. One channel per
// thread took 2,104 us in all. For n up to 8 the main pass spills (fp32 124 bytes
// stored, bf16 32), for n up to 16 with fp32 inputs too (16 to 20).
//
// The workspace is mostly the states before the blocks, total / 8 D n fp32, and
// the partial sums of dB and dC, 2 cpg total G n fp32, where the channel blocks
// per group, cpg, grow with n: 3.1 GB for 32K tokens of 8192 channels with 16
// states, 18.5 GB with 64.
#include <climits>

#include "ssm_scan.cuh"

namespace la {
namespace {

constexpr int BLK = 8;    // tokens per block
constexpr int NT = 128;   // threads per CTA of the local and the main pass

struct BackArgs {
    la_scan_inputs in;
    SeqView view;
    Chunks ch;
    const void* dy;
    long long ld_dy;
    la_scan_grads out;
    float* hs;      // [items][D][n]: chunk states, then states before the chunks, then dA partials
    float* gs;      // [items][D][n]: G of the chunks, then gradients of the states after them
    float* dtsum;   // [items][D]
    float* ck;      // [items][len / BLK][D][n]: local state before each block but the first
    float* ckdt;    // [items][len / BLK][D]: sum of the chunk's dt before each block
    float* dDp;     // [items][D]
    float* dbp;     // [items][D]
    float* dBp;     // [cpg][total][G][n]
    float* dCp;
    int D, G, n, cpg;
    int out_f32;
};

// A CTA's chunk and channels.
struct Place {
    int item, c0, c_end, g, cbg;
    long long t0, t1;
    // An item of a packed batch's table behind its last chunk gets no tokens.
    __device__ __forceinline__ Place(const BackArgs& a, int CC)
    {
        const int blocks = a.G * a.cpg, cb = blockIdx.x % blocks, Dg = a.D / a.G;
        item = blockIdx.x / blocks;
        const int s = a.ch.seq(item);
        t0 = t1 = 0;
        if (s >= 0) {
            a.view.range(s, t0, t1);
            t0 += (item - a.ch.first_of(s)) * a.ch.len;
            if (t1 - t0 > a.ch.len) t1 = t0 + a.ch.len;
        }
        g = cb / a.cpg;
        cbg = cb % a.cpg;
        c0 = g * Dg + cbg * CC;
        c_end = (g + 1) * Dg;
    }
};

// The token inputs of a CTA, block by block of BLK tokens: each thread holds E
// pairs of channels and EB values of B and of C. Addresses are a base that all
// threads share and a thread's own 32-bit offset from it.
template <typename T, int K, bool VEC> struct Inputs {
    static constexpr int NP = SCAN_S * K, CC = 2 * NT / K, CP = CC / 2;
    static constexpr int RP = NT / CP;                        // rows between a thread's pairs
    static constexpr int E = (BLK + RP - 1) / RP;
    static constexpr int RB = NT / NP, EB = (BLK + RB - 1) / RB;
    static constexpr uint32_t TS = sizeof(T);
    Pair<T, VEC> u[E], d[E], z[E], y[E];
    T B[EB], C[EB];
    const char *up, *dp, *zp, *yp, *Bp, *Cp;
    uint32_t lu, ld, lz, ly, lb, lc, ch_at, bm_at, next;
    int prow, brow;
    bool gated, lo_ok, hi_ok;  // whether the pair's channels are the CTA's

    __device__ __forceinline__ Inputs(const BackArgs& a, const Place& p)
    {
        const int tid = threadIdx.x, pr = tid % CP, ec = p.c0 + 2 * pr;
        lo_ok = ec < p.c_end;
        hi_ok = ec + 1 < p.c_end;
        // Channels behind the group's last read the last ones.
        const int ch = lo_ok ? 2 * pr : p.c_end - p.c0 - (VEC ? 2 : 1);
        const int bm = tid % NP;
        prow = tid / CP;
        brow = tid / NP;
        next = hi_ok ? TS : 0;
        ch_at = ch * TS;
        bm_at = (bm < a.n ? bm : 0) * TS;
        lu = (uint32_t)a.in.ld_u * TS;
        ld = (uint32_t)a.in.ld_delta * TS;
        lz = (uint32_t)a.in.ld_z * TS;
        ly = (uint32_t)a.ld_dy * TS;
        lb = (uint32_t)a.in.ld_b * TS;
        lc = (uint32_t)a.in.ld_c * TS;
        up = (const char*)a.in.u + ((long long)p.c0 + p.t0 * a.in.ld_u) * TS;
        dp = (const char*)a.in.delta + ((long long)p.c0 + p.t0 * a.in.ld_delta) * TS;
        zp = (const char*)a.in.z + ((long long)p.c0 + p.t0 * a.in.ld_z) * TS;
        yp = (const char*)a.dy + ((long long)p.c0 + p.t0 * a.ld_dy) * TS;
        Bp = (const char*)a.in.B + ((long long)p.g * a.n + p.t0 * a.in.ld_b) * TS;
        Cp = (const char*)a.in.C + ((long long)p.g * a.n + p.t0 * a.in.ld_c) * TS;
        gated = a.in.z != nullptr;
    }
    // Block blk of the chunk; rows behind rmax (counted from the block's first) read that one.
    __device__ __forceinline__ void load(int blk, int rmax)
    {
        const long long r = (long long)blk * BLK;
        const char *u_ = up + r * lu, *d_ = dp + r * ld, *z_ = zp + r * lz, *y_ = yp + r * ly;
        const char *B_ = Bp + r * lb, *C_ = Cp + r * lc;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t row = min(prow + e * RP, rmax);
            u[e].load(u_ + (row * lu + ch_at), next);
            d[e].load(d_ + (row * ld + ch_at), next);
            y[e].load(y_ + (row * ly + ch_at), next);
            if (gated) z[e].load(z_ + (row * lz + ch_at), next);
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const uint32_t row = min(brow + e * RB, rmax);
            B[e] = *reinterpret_cast<const T*>(B_ + (row * lb + bm_at));
            C[e] = *reinterpret_cast<const T*>(C_ + (row * lc + bm_at));
        }
    }
};

// A block's inputs as the scanning threads read them.
template <int K> struct Block {
    static constexpr int NP = SCAN_S * K, CP = NT / K;
    float4 dt[BLK][CP];  // dt, dt u of the pair's first channel, then of its second
    f2 w[BLK][CP];       // dy times the gate
    float b[BLK][NP];
    float c[BLK][NP];
};

// What the main pass's elementwise end needs of a block, made with the rest: the
// exponentials are at hand there, and 1,080 us became 1,038 (with the outputs'
// addresses taken per row).
template <int K> struct Slopes {
    f2 dt[BLK][NT / K];  // d dt / d delta
    f2 z[BLK][NT / K];   // dy times the gate's derivative
};

template <typename T, int K, bool VEC>
__device__ __forceinline__ void fill_block(Block<K>& blk, const Inputs<T, K, VEC>& in, int n,
                                           int rmax, f2 bias, bool softplus,
                                           Slopes<K>* slopes = nullptr)
{
    using I = Inputs<T, K, VEC>;
    const int pr = threadIdx.x % I::CP, bm = threadIdx.x % I::NP;
#pragma unroll
    for (int e = 0; e < I::E; ++e) {
        const int row = in.prow + e * I::RP;
        if (BLK % I::RP && row >= BLK) continue;
        f2 dt = add2(in.d[e].get(), bias), w = in.y[e].get();
        if (slopes) {
            f2 slope = pack(1.f, 1.f);
            if (softplus) dt = softplus2(dt, slope);
            slopes->dt[row][pr] = slope;
        } else if (softplus) {
            dt = softplus2(dt);
        }
        f2 du = mul2(dt, in.u[e].get());
        if (in.gated) {
            const f2 z = in.z[e].get(), sg = sigmoid2(z), gate = mul2(z, sg);
            // (z sg)' = sg + z sg (1 - sg)
            if (slopes)
                slopes->z[row][pr] =
                    mul2(w, fma2(gate, fma2(sg, pack(-1.f, -1.f), pack(1.f, 1.f)), sg));
            w = mul2(w, gate);
        }
        if (row > rmax || !in.lo_ok) dt = du = w = pack(0.f, 0.f);  // decay 1, nothing added
        if (!in.hi_ok) {  // a channel of the next group adds nothing to this one's sums
            float lo, hi;
            unpack(dt, lo, hi);
            dt = pack(lo, 0.f);
            unpack(du, lo, hi);
            du = pack(lo, 0.f);
            unpack(w, lo, hi);
            w = pack(lo, 0.f);
        }
        float4 v;
        unpack(dt, v.x, v.z);
        unpack(du, v.y, v.w);
        blk.dt[row][pr] = v;
        blk.w[row][pr] = w;
    }
#pragma unroll
    for (int e = 0; e < I::EB; ++e) {
        const int row = in.brow + e * I::RB;
        if (BLK % I::RB && row >= BLK) continue;
        const bool ok = bm < n && row <= rmax;
        blk.b[row][bm] = ok ? to_f32(in.B[e]) : 0.f;
        blk.c[row][bm] = ok ? to_f32(in.C[e]) : 0.f;
    }
}

// A pair of channels' values of a [D] vector; zeros where there are none.
__device__ __forceinline__ f2 channel_pair(const float* v, int c, int c_end)
{
    return pack(v && c < c_end ? v[c] : 0.f, v && c + 1 < c_end ? v[c + 1] : 0.f);
}

// A log2 e of a thread's four states of two channels.
__device__ __forceinline__ void load_decays(f2 (*A)[2], const BackArgs& a, int c, int c_end, int m0)
{
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (c + x < c_end) load_states(v, a.in.A + (long long)(c + x) * a.n, m0, a.n);
        // States behind n: the decay is 1 but for an infinite dt, where it is 0 as
        // elsewhere; with A = 0 it would be NaN, and with it the channel's sums.
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (m0 + i >= a.n) v[i] = -FLT_MIN;
        A[x][0] = pack(decay_rate(v[0]), decay_rate(v[1]));
        A[x][1] = pack(decay_rate(v[2]), decay_rate(v[3]));
    }
}
__device__ __forceinline__ void load_pair(f2 (*v)[2], const float* p, const BackArgs& a,
                                          long long row, int c, int c_end, int m0)
{
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        if (c + x < c_end) load_states(s, p + (row * a.D + c + x) * a.n, m0, a.n);
        v[x][0] = pack(s[0], s[1]);
        v[x][1] = pack(s[2], s[3]);
    }
}
__device__ __forceinline__ void store_pair(float* p, f2 (*v)[2], const BackArgs& a, long long row,
                                           int c, int c_end, int m0)
{
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        float s[4];
        unpack(v[x][0], s[0], s[1]);
        unpack(v[x][1], s[2], s[3]);
        if (c + x < c_end) store_states(p + (row * a.D + c + x) * a.n, s, m0, a.n);
    }
}

template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(NT, 4) local_kernel(BackArgs a)
{
    using I = Inputs<T, K, VEC>;
    __shared__ Block<K> blocks[2];
    const Place p(a, I::CC);
    const int tid = threadIdx.x, pr = tid / K, m0 = (tid % K) * SCAN_S, c = p.c0 + 2 * pr;
    f2 A[2][2], h[2][2], G[2][2], P[2][2], dts = pack(0.f, 0.f);
    load_decays(A, a, c, p.c_end, m0);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) h[x][i] = G[x][i] = pack(0.f, 0.f), P[x][i] = pack(1.f, 1.f);
    I in(a, p);
    const f2 bias = channel_pair(a.in.delta_bias, p.c0 + 2 * (tid % I::CP), p.c_end);
    const int len = (int)(p.t1 - p.t0), nblk = (len + BLK - 1) / BLK;
    if (nblk > 0) in.load(0, min(BLK, len) - 1);
#pragma unroll 1
    for (int b = 0; b < nblk; ++b) {
        Block<K>& blk = blocks[b & 1];
        fill_block<T, K, VEC>(blk, in, a.n, min(BLK, len - b * BLK) - 1, bias, a.in.softplus);
        __syncthreads();
        if (b + 1 < nblk) in.load(b + 1, min(BLK, len - (b + 1) * BLK) - 1);
        if (b > 0) {
            const long long at = (long long)p.item * (a.ch.len / BLK) + b;
            store_pair(a.ck, h, a, at, c, p.c_end, m0);
            if (m0 == 0) {
                float d0, d1;
                unpack(dts, d0, d1);
                if (c < p.c_end) a.ckdt[at * a.D + c] = d0;
                if (c + 1 < p.c_end) a.ckdt[at * a.D + c + 1] = d1;
            }
        }
#pragma unroll
        for (int q = 0; q < BLK; ++q) {
            const float4 d = blk.dt[q][pr];
            float w[2];
            unpack(blk.w[q][pr], w[0], w[1]);
            const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&blk.b[q][m0]);
            const ulonglong2 cv = *reinterpret_cast<const ulonglong2*>(&blk.c[q][m0]);
            const float dt[2] = {d.x, d.z}, du[2] = {d.y, d.w};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const f2 e = ex2_2(mul2(pack(dt[x], dt[x]), A[x][i]));
                    h[x][i] = fma2(e, h[x][i], mul2(pack(du[x], du[x]), i ? bv.y : bv.x));
                    P[x][i] = mul2(P[x][i], e);
                    G[x][i] = fma2(P[x][i], mul2(pack(w[x], w[x]), i ? cv.y : cv.x), G[x][i]);
                }
            }
            dts = add2(dts, pack(dt[0], dt[1]));
        }
    }
    store_pair(a.hs, h, a, p.item, c, p.c_end, m0);
    store_pair(a.gs, G, a, p.item, c, p.c_end, m0);
    if (m0 == 0) {
        float d0, d1;
        unpack(dts, d0, d1);
        if (c < p.c_end) a.dtsum[(long long)p.item * a.D + c] = d0;
        if (c + 1 < p.c_end) a.dtsum[(long long)p.item * a.D + c + 1] = d1;
    }
}

// One thread per (channel, state) of a sequence.
__global__ void __launch_bounds__(128) combine_kernel(BackArgs a, const float* state_in,
                                                      const float* dstate_out)
{
    const long long DN = (long long)a.D * a.n;
    const int per = (int)((DN + 127) / 128);  // CTAs of a sequence
    const int s = blockIdx.x / per;
    const long long e = (long long)(blockIdx.x % per) * 128 + threadIdx.x;
    if (e >= DN) return;
    const int c = (int)(e / a.n);
    const float A2 = decay_rate(a.in.A[e]);
    const int first = a.ch.first_of(s), end = a.ch.end_of(s);
    float h = state_in ? state_in[s * DN + e] : 0.f;
    float g = dstate_out ? dstate_out[s * DN + e] : 0.f;
    // Both sweeps together, AHEAD chunks of each at a time: reads first, then the
    // writes to the same places.
    constexpr int AHEAD = 8;
    float hl[AHEAD], hd[AHEAD], gl[AHEAD], gd[AHEAD];
    const int chunks = end - first;
    for (int i = 0; i < chunks; i += AHEAD) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int at = min(i + k, chunks - 1);
            const long long up = first + at, down = end - 1 - at;
            hl[k] = a.hs[up * DN + e];
            hd[k] = a.dtsum[up * a.D + c];
            gl[k] = a.gs[down * DN + e];
            gd[k] = a.dtsum[down * a.D + c];
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (i + k >= chunks) break;
            a.hs[(first + i + k) * DN + e] = h;
            h = fmaf(ex2(A2 * hd[k]), h, hl[k]);
            a.gs[(end - 1 - i - k) * DN + e] = g;
            g = fmaf(ex2(A2 * gd[k]), g, gl[k]);
        }
    }
    if (a.out.dstate_in) a.out.dstate_in[s * DN + e] = g;
}

template <int K> struct MainShared {
    static constexpr int NP = SCAN_S * K;
    Block<K> in;
    // Each scanning thread's share of sum_m g B, of sum_m A log2 e a h g and of
    // C . h, for both channels.
    f2 gB[BLK][NT], gA[BLK][NT], y[BLK][NT];
    float red[NT / 32][BLK][2][NP];  // dB and dC, summed over each warp's channels
    Slopes<K> slopes;
};

// A pair of outputs at p.
template <bool VEC>
__device__ __forceinline__ void store_two(char* p, bool f32, bool hi, f2 v)
{
    float x, y;
    unpack(v, x, y);
    if (f32) {
        if (VEC) *reinterpret_cast<f2*>(p) = v;
        else {
            reinterpret_cast<float*>(p)[0] = x;
            if (hi) reinterpret_cast<float*>(p)[1] = y;
        }
    } else {
        if (VEC) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
        else {
            reinterpret_cast<__nv_bfloat16*>(p)[0] = __float2bfloat16_rn(x);
            if (hi) reinterpret_cast<__nv_bfloat16*>(p)[1] = __float2bfloat16_rn(y);
        }
    }
}

// ex2 that the compiler does not replace by the result of an earlier one: 64
// decays kept from the forward walk would not fit in registers.
__device__ __forceinline__ float ex2_again(float x)
{
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Sum of the K shares of a pair of channels.
template <int K> __device__ __forceinline__ f2 sum_shares(const f2* v)
{
    f2 s;
#pragma unroll
    for (int k = 0; k < K; k += 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(v + k);
        s = k ? add2(s, add2(x.x, x.y)) : add2(x.x, x.y);
    }
    return s;
}

template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(NT, 3) main_kernel(BackArgs a)
{
    using I = Inputs<T, K, VEC>;
    constexpr int S = SCAN_S, NP = I::NP, M = 32 / K;  // M: pairs of channels per warp
    constexpr int RC = M < 8 ? 8 / M : 1;              // dB, dC values per lane when reduced
    extern __shared__ __align__(16) unsigned char smem[];
    MainShared<K>& sh = *reinterpret_cast<MainShared<K>*>(smem);
    const Place p(a, I::CC);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pr = tid / K, m0 = (tid % K) * S, c = p.c0 + 2 * pr;
    const int epr = tid % I::CP, ec = p.c0 + 2 * epr;  // of the elementwise work

    f2 A[2][2], h0[2][2], carry[2][2], dA[2][2];
    load_decays(A, a, c, p.c_end, m0);
    load_pair(h0, a.hs, a, p.item, c, p.c_end, m0);
    load_pair(carry, a.gs, a, p.item, c, p.c_end, m0);
#pragma unroll
    for (int x = 0; x < 2; ++x) dA[x][0] = dA[x][1] = pack(0.f, 0.f);

    I in(a, p);
    const f2 bias = channel_pair(a.in.delta_bias, ec, p.c_end);
    const f2 Dw = channel_pair(a.in.D, ec, p.c_end);
    const f2 zero = pack(0.f, 0.f);
    f2 dD = zero, db = zero;
    // Where the chunk's outputs start, and this thread's offset in bytes.
    const int os = a.out_f32 ? 4 : 2;
    const long long out0 = (p.t0 * a.D + p.c0) * os;
    const uint32_t out_at = (uint32_t)(in.prow * a.D + 2 * epr) * os;
    // dB and dC: this thread's state and tensor, and its first token of a block.
    static_assert(2 * NP <= NT, "a token's values fit the threads");
    constexpr int RT = NT / (2 * NP);  // tokens per round
    const int bm = tid % NP, bwhich = tid / NP % 2, bq = tid / (2 * NP);
    const long long per_token = (long long)a.G * a.n;
    float* const bc_out = (bwhich ? a.dCp : a.dBp) +
                          ((long long)p.cbg * a.view.total + p.t0) * per_token + (long long)p.g * a.n + bm;
    const int len = (int)(p.t1 - p.t0), nblk = (len + BLK - 1) / BLK;
    if (nblk > 0) in.load(nblk - 1, len - (nblk - 1) * BLK - 1);
#pragma unroll 1
    for (int b = nblk - 1; b >= 0; --b) {
        const int rmax = min(BLK, len - b * BLK) - 1;
        fill_block<T, K, VEC>(sh.in, in, a.n, rmax, bias, a.in.softplus, &sh.slopes);
        Pair<T, VEC> cu[I::E];
#pragma unroll
        for (int e = 0; e < I::E; ++e) cu[e] = in.u[e];
        __syncthreads();
        if (b > 0) in.load(b - 1, BLK - 1);

        // The state before the block: its local part, and what is left of the
        // state before the chunk.
        f2 start[2][2];
        if (b == 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) start[x][0] = h0[x][0], start[x][1] = h0[x][1];
        } else {
            const long long at = (long long)p.item * (a.ch.len / BLK) + b;
            load_pair(start, a.ck, a, at, c, p.c_end, m0);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float d = c + x < p.c_end ? a.ckdt[at * a.D + c + x] : 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    start[x][i] = fma2(ex2_2(mul2(pack(d, d), A[x][i])), h0[x][i], start[x][i]);
            }
        }
        auto advance = [&](int q, const f2 (*from)[2], f2 (*to)[2]) {
            const float4 d = sh.in.dt[q][pr];
            const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&sh.in.b[q][m0]);
            const float dt[2] = {d.x, d.z}, du[2] = {d.y, d.w};
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float A0, A1;
                    unpack(A[x][i], A0, A1);
                    to[x][i] = fma2(pack(ex2_again(dt[x] * A0), ex2_again(dt[x] * A1)), from[x][i],
                                    mul2(pack(du[x], du[x]), i ? bv.y : bv.x));
                }
        };
        // What a token leaves is written while the next one is worked on, and after
        // that one's inputs are read: shared reads stay behind earlier writes, and
        // these wait for the shuffles.
        struct {
            float v[8];
            f2 gB, gA, y;
        } last = {};
        auto flush = [&](int q) {
            sh.gB[q][tid] = last.gB;
            sh.gA[q][tid] = last.gA;
            sh.y[q][tid] = last.y;
            lane_reduce<8, M, K>(last.v, lane);
            if (reduced_writer<8, M, K>(lane)) {
                const int at = reduced_index<8, M, K>(lane);
#pragma unroll
                for (int i = 0; i < RC; ++i)
                    sh.red[warp][q][(at + i) / S][m0 + (at + i) % S] = last.v[i];
            }
        };
        // Half a block at a time: its states stay in registers.
        constexpr int HALF = BLK / 2;
#pragma unroll 1
        for (int from = HALF; from >= 0; from -= HALF) {
            f2 hb[HALF + 1][2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x) hb[0][x][0] = start[x][0], hb[0][x][1] = start[x][1];
            if (from) {
#pragma unroll
                for (int q = 0; q < HALF; ++q) advance(q, hb[0], hb[0]);
            }
#pragma unroll
            for (int r = 0; r < HALF; ++r) advance(from + r, hb[r], hb[r + 1]);
#pragma unroll
            for (int r = HALF - 1; r >= 0; --r) {
                const int q = from + r;
                const float4 d = sh.in.dt[q][pr];
                float w[2];
                unpack(sh.in.w[q][pr], w[0], w[1]);
                const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&sh.in.b[q][m0]);
                const ulonglong2 cv = *reinterpret_cast<const ulonglong2*>(&sh.in.c[q][m0]);
                if (r < HALF - 1) flush(q + 1);
                const float dt[2] = {d.x, d.z}, du[2] = {d.y, d.w};
                f2 dB[2], dC[2];
                float gB[2], gA[2], y[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const f2 ww = pack(w[x], w[x]), dd = pack(dt[x], dt[x]), uu = pack(du[x], du[x]);
                    f2 sB, sA, sy;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const f2 Bm = i ? bv.y : bv.x, Cm = i ? cv.y : cv.x, ht = hb[r + 1][x][i];
                        const f2 g = fma2(Cm, ww, carry[x][i]);
                        dB[i] = x ? fma2(g, uu, dB[i]) : mul2(g, uu);
                        dC[i] = x ? fma2(ht, ww, dC[i]) : mul2(ht, ww);
                        sB = i ? fma2(g, Bm, sB) : mul2(g, Bm);
                        sy = i ? fma2(ht, Cm, sy) : mul2(ht, Cm);
                        float A0, A1;
                        unpack(A[x][i], A0, A1);
                        carry[x][i] = mul2(pack(ex2_again(dt[x] * A0), ex2_again(dt[x] * A1)), g);
                        const f2 gh = mul2(carry[x][i], hb[r][x][i]);
                        sA = i ? fma2(gh, A[x][i], sA) : mul2(gh, A[x][i]);
                        dA[x][i] = fma2(gh, dd, dA[x][i]);
                    }
                    float lo, hi;
                    unpack(sB, lo, hi);
                    gB[x] = lo + hi;
                    unpack(sA, lo, hi);
                    gA[x] = lo + hi;
                    unpack(sy, lo, hi);
                    y[x] = lo + hi;
                }
                last.gB = pack(gB[0], gB[1]);
                last.gA = pack(gA[0], gA[1]);
                last.y = pack(y[0], y[1]);
                unpack(dB[0], last.v[0], last.v[1]);
                unpack(dB[1], last.v[2], last.v[3]);
                unpack(dC[0], last.v[4], last.v[5]);
                unpack(dC[1], last.v[6], last.v[7]);
                if (r == 0) flush(q);
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < I::E; ++e) {
            const int row = in.prow + e * I::RP;
            if (row > rmax || !in.lo_ok) continue;
            const f2 u = cu[e].get(), w = sh.in.w[row][epr];
            const f2 gb = sum_shares<K>(&sh.gB[row][epr * K]);
            const f2 ga = sum_shares<K>(&sh.gA[row][epr * K]);
            const float4 dtv = sh.in.dt[row][epr];
            const f2 dt = pack(dtv.x, dtv.z);
            const f2 dd = mul2(fma2(ga, pack(SCAN_LN2, SCAN_LN2), mul2(u, gb)),
                               sh.slopes.dt[row][epr]);
            // The rows' part of the address is the same for all threads.
            const long long at = out0 + (long long)(b * BLK + e * I::RP) * a.D * os;
            if (in.gated) {
                const f2 y = fma2(Dw, u, sum_shares<K>(&sh.y[row][epr * K]));
                store_two<VEC>((char*)a.out.dz + at + out_at, a.out_f32, in.hi_ok,
                               mul2(sh.slopes.z[row][epr], y));
            }
            store_two<VEC>((char*)a.out.du + at + out_at, a.out_f32, in.hi_ok,
                           fma2(Dw, w, mul2(dt, gb)));
            store_two<VEC>((char*)a.out.ddelta + at + out_at, a.out_f32, in.hi_ok, dd);
            dD = fma2(w, u, dD);
            db = add2(db, dd);
        }
#pragma unroll
        for (int r = 0; r < BLK; r += RT) {
            const int q = r + bq;
            if (q > rmax || bm >= a.n) continue;
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < NT / 32; ++k) v += sh.red[k][q][bwhich][bm];
            bc_out[(b * BLK + q) * per_token] = v;
        }
        __syncthreads();
    }
    store_pair(a.hs, dA, a, p.item, c, p.c_end, m0);  // this thread's own slots, read above
    // dD and ddelta_bias of this chunk: RP threads hold one pair of channels.
    ulonglong2* pair = reinterpret_cast<ulonglong2*>(&sh.gB[0][0]);
    pair[tid] = make_ulonglong2(dD, db);
    __syncthreads();
    if (tid < I::CP && in.lo_ok) {
        f2 x = zero, y = zero;
#pragma unroll
        for (int k = 0; k < I::RP; ++k) {
            x = add2(x, pair[tid + k * I::CP].x);
            y = add2(y, pair[tid + k * I::CP].y);
        }
        float x0, x1, y0, y1;
        unpack(x, x0, x1);
        unpack(y, y0, y1);
        const long long at = (long long)p.item * a.D + ec;
        a.dDp[at] = x0;
        a.dbp[at] = y0;
        if (in.hi_ok) a.dDp[at + 1] = x1, a.dbp[at + 1] = y1;
    }
}

// Lanes per pair of channels.
int back_lanes(int n)
{
    return n <= 8 ? 2 : scan_lanes(n);
}

struct BackLayout {
    int len, items, cpg;
    size_t hs, gs, dtsum, ck, ckdt, dDp, dbp, dBp, dCp, first, bytes;
};

BackLayout back_layout(int G, int D, long long total, int n, int num_seqs)
{
    BackLayout l;
    const int CC = 2 * NT / back_lanes(n);
    l.cpg = (D / G + CC - 1) / CC;
    // Tokens per chunk: 128, or fewer while that leaves SMs without work (three
    // CTAs fit on each): a chunk is walked by one CTA from end to end.
    l.len = 128;
    while (l.len > 32 && (total / l.len + 1) * G * l.cpg < 3 * 148) l.len /= 2;
    l.items = (int)(total / l.len + num_seqs);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes, 256);
        return here;
    };
    const size_t states = (size_t)l.items * D * n * 4, chans = (size_t)l.items * D * 4;
    l.hs = take(states);
    l.gs = take(states);
    l.dtsum = take(chans);
    l.ck = take(states * (l.len / BLK));
    l.ckdt = take(chans * (l.len / BLK));
    l.dDp = take(chans);
    l.dbp = take(chans);
    const size_t slabs = (size_t)l.cpg * total * G * n * 4;
    l.dBp = take(slabs);
    l.dCp = take(slabs);
    l.first = take((size_t)(num_seqs + 1 + l.items) * 4);
    l.bytes = at;
    return l;
}

}  // namespace

size_t scan_backward_workspace(int G, int D, long long total, int n, int num_seqs)
{
    return back_layout(G, D, total, n, num_seqs).bytes;
}

cudaError_t launch_scan_backward(const ScanProblem& p, const float* state_in, const void* dy,
                                 long long ld_dy, const float* dstate_out,
                                 const la_scan_grads& out, void* ws, cudaStream_t stream)
{
    const int num_seqs = p.view.num_seqs;
    const BackLayout l = back_layout(p.G, p.D, p.view.total, p.n, num_seqs);
    char* w = (char*)ws;
    BackArgs a{};
    a.in = p.in;
    a.view = p.view;
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.out = out;
    a.hs = (float*)(w + l.hs);
    a.gs = (float*)(w + l.gs);
    a.dtsum = (float*)(w + l.dtsum);
    a.ck = (float*)(w + l.ck);
    a.ckdt = (float*)(w + l.ckdt);
    a.dDp = (float*)(w + l.dDp);
    a.dbp = (float*)(w + l.dbp);
    a.dBp = (float*)(w + l.dBp);
    a.dCp = (float*)(w + l.dCp);
    a.D = p.D;
    a.G = p.G;
    a.n = p.n;
    a.cpg = l.cpg;
    a.out_f32 = p.out_t == LA_F32;
    a.ch.len = l.len;
    if (p.view.cu) {
        int* first = (int*)(w + l.first);
        a.ch.items = l.items;
        a.ch.first = first;
        a.ch.seq_of = first + num_seqs + 1;
        if (num_seqs > 0) {
            cudaError_t e = launch_plan_chunks(p.view, l.len, l.items, first, first + num_seqs + 1,
                                               stream);
            if (e != cudaSuccess) return e;
        }
    } else if (num_seqs > 0) {
        const long long per = (p.view.N + l.len - 1) / l.len;
        a.ch.per_seq = per > 1 ? (int)per : 1;
        a.ch.items = a.ch.per_seq * num_seqs;
    }
    cudaError_t e = cudaSuccess;
    const long long DN = (long long)p.D * p.n;
    if (num_seqs > 0) {
        const unsigned grid = (unsigned)((long long)a.ch.items * p.G * a.cpg);
        const unsigned combine_grid = (unsigned)((DN + 127) / 128 * num_seqs);
        const size_t two = p.in_t == LA_BF16 ? 4 : 8;  // bytes of a pair of channels
        const auto pairs = [&](const void* q, long long ld) {
            return (uintptr_t)q % two == 0 && ld % 2 == 0;
        };
        const bool vec = p.D / p.G % 2 == 0 && pairs(p.in.u, p.in.ld_u) &&
                         pairs(p.in.delta, p.in.ld_delta) && pairs(dy, ld_dy) &&
                         (!p.in.z || pairs(p.in.z, p.in.ld_z));
#define LA_TYPE(T, KK)                                                                           \
    do {                                                                                         \
        auto local = vec ? local_kernel<T, KK, true> : local_kernel<T, KK, false>;               \
        auto main = vec ? main_kernel<T, KK, true> : main_kernel<T, KK, false>;                  \
        const int smem = (int)sizeof(MainShared<KK>);                                            \
        e = allow_shared((const void*)main, smem);                                               \
        if (e != cudaSuccess) return e;                                                          \
        local<<<grid, NT, 0, stream>>>(a);                                                       \
        combine_kernel<<<combine_grid, 128, 0, stream>>>(a, state_in, dstate_out);               \
        main<<<grid, NT, smem, stream>>>(a);                                                     \
    } while (0)
#define LA_CALL(KK)                                                                              \
    if (p.in_t == LA_BF16) LA_TYPE(__nv_bfloat16, KK);                                           \
    else LA_TYPE(float, KK)
        switch (back_lanes(p.n)) {
        case 2: LA_CALL(2); break;
        case 4: LA_CALL(4); break;
        case 8: LA_CALL(8); break;
        default: LA_CALL(16); break;
        }
#undef LA_CALL
#undef LA_TYPE
        count_launch(3);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const int rows = num_seqs > 0 ? a.ch.items : 0, bf16 = !a.out_f32;
    const long long cells = p.view.total * p.G * p.n;
    const int* held = p.view.cu ? p.view.cu + num_seqs : nullptr;
    SumJobs sums;
    if (num_seqs > 0) {
        sums.add(a.dBp, out.dB, a.cpg, cells, bf16, held, (long long)p.G * p.n);
        sums.add(a.dCp, out.dC, a.cpg, cells, bf16, held, (long long)p.G * p.n);
    }
    sums.add(a.hs, out.dA, rows, DN);
    sums.add(a.dDp, out.dD, rows, p.D);
    sums.add(a.dbp, out.ddelta_bias, rows, p.D);
    return launch_column_sums(sums, stream);
}

}  // namespace la
