// Gradients of the selective scan (formulas in lightning.h).
//
// The sequences are cut into chunks of LEN tokens, all of them independent:
//  1. local pass: each chunk's state from zero, h_c; the sum of its dt, whose
//     exponential exp(A sum dt) is the chunk's whole decay; and the gradient
//     that the chunk's own outputs send to the state before it,
//     G_c = sum_t (prod_{s<=t} a_s) C_t dyz_t.
//  2. combine: forward over the chunks, the state before each; backward over
//     them, the gradient of the state after each (from dstate_out).
//  3. main pass: per chunk, a forward walk that leaves the state before every
//     block of 8 tokens in shared memory, then the blocks from the last to the
//     first: forward again with the 8 states and decays in registers, and the
//     reverse recurrence over them. The exponentials are thus taken three times
//     (once per walk), which costs less than moving states or decays through
//     shared memory.
//  4. reductions of dB and dC over the channel blocks and of dA, dD and
//     ddelta_bias over the chunks, from partial sums in the workspace, in a
//     fixed order.
#include <climits>

#include "ssm_scan.cuh"

namespace la {
namespace {

constexpr int LEN = 128;  // tokens per chunk
constexpr int BLK = 8;    // tokens per block of the main pass
constexpr int NT1 = 128;  // threads of the local pass
constexpr int NT3 = 256;  // threads of the main pass

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
    float* dDp;     // [items][D]
    float* dbp;     // [items][D]
    float* dBp;     // [cpg][total][G][n]
    float* dCp;
    int D, G, n, cpg;
    int out_f32;
};

template <typename T>
__device__ __forceinline__ void store_out(void* p, long long i, float v, int f32)
{
    if (f32) ((float*)p)[i] = v;
    else ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(v);
}

// A CTA's chunk and channels.
struct Place {
    int c0, c_end, g, cbg;
    long long t0, t1;
    // An item of a packed batch's table behind its last chunk gets no tokens.
    __device__ __forceinline__ Place(const BackArgs& a, int item, int cb, int cpg, int CC)
    {
        const int s = a.ch.seq(item), Dg = a.D / a.G;
        t0 = t1 = 0;
        if (s >= 0) {
            a.view.range(s, t0, t1);
            t0 += (item - a.ch.first_of(s)) * a.ch.len;
            if (t1 - t0 > a.ch.len) t1 = t0 + a.ch.len;
        }
        g = cb / cpg;
        cbg = cb % cpg;
        c0 = g * Dg + cbg * CC;
        c_end = (g + 1) * Dg;
    }
};

template <typename T, int K>
__global__ void __launch_bounds__(NT1) local_kernel(BackArgs a, int cpg1)
{
    constexpr int S = SCAN_S, NP = S * K, CC = NT1 / K;
    constexpr int TT = K == 1 ? 8 : K == 2 || K == 16 ? 16 : 32;
    constexpr int E = TT * CC / NT1;
    constexpr int EB = (TT * NP + NT1 - 1) / NT1;
    __shared__ float2 dtu[TT][CC];
    __shared__ float dyz[TT][CC];
    __shared__ __align__(16) float bc[2][TT][NP];

    const int tid = threadIdx.x;
    const int blocks = a.G * cpg1;
    const int item = blockIdx.x / blocks;
    const Place p(a, item, blockIdx.x % blocks, cpg1, CC);
    const int sch = tid / K, m0 = (tid % K) * S, sc = p.c0 + sch;
    const bool sc_ok = sc < p.c_end;
    const int ech = tid % CC, etok = tid / CC, ec = p.c0 + ech;
    const bool ec_ok = ec < p.c_end;

    float A2[S] = {0.f, 0.f, 0.f, 0.f};
    if (sc_ok) load_states(A2, a.in.A + (long long)sc * a.n, m0, a.n);
    float h[S], G[S], P[S], dts = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) A2[i] *= SCAN_LOG2E, h[i] = G[i] = 0.f, P[i] = 1.f;

    const T* up = (const T*)a.in.u + ec;
    const T* dp = (const T*)a.in.delta + ec;
    const T* zp = a.in.z ? (const T*)a.in.z + ec : nullptr;
    const T* yp = (const T*)a.dy + ec;
    const T* Bp = (const T*)a.in.B + (long long)p.g * a.n;
    const T* Cp = (const T*)a.in.C + (long long)p.g * a.n;
    const float dbias = a.in.delta_bias && ec_ok ? a.in.delta_bias[ec] : 0.f;
    const long long t1 = p.t1;

    T ru[E], rd[E], rz[E], ry[E], rB[EB], rC[EB];
    auto load = [&](long long t) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const long long tok = t + e * K + etok;
            const bool ok = ec_ok && tok < t1;
            ru[e] = ok ? up[tok * a.in.ld_u] : T(0.f);
            rd[e] = ok ? dp[tok * a.in.ld_delta] : T(0.f);
            ry[e] = ok ? yp[tok * a.ld_dy] : T(0.f);
            rz[e] = ok && zp ? zp[tok * a.in.ld_z] : T(0.f);
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int idx = e * NT1 + tid, m = idx % NP;
            const long long tok = t + idx / NP;
            const bool ok = m < a.n && tok < t1 && idx < TT * NP;
            rB[e] = ok ? Bp[tok * a.in.ld_b + m] : T(0.f);
            rC[e] = ok ? Cp[tok * a.in.ld_c + m] : T(0.f);
        }
    };
    if (p.t0 < t1) load(p.t0);
    for (long long t = p.t0; t < t1; t += TT) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float dt = to_f32(rd[e]) + dbias;
            if (a.in.softplus) dt = softplus_f(dt);
            if (!ec_ok || t + e * K + etok >= t1) dt = 0.f;
            dtu[e * K + etok][ech] = make_float2(dt, dt * to_f32(ru[e]));
            float y = to_f32(ry[e]);
            const float z = to_f32(rz[e]);
            if (zp) y *= z * sigmoid_f(z);
            dyz[e * K + etok][ech] = y;
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int idx = e * NT1 + tid;
            if (idx < TT * NP) {
                (&bc[0][0][0])[idx] = to_f32(rB[e]);
                (&bc[1][0][0])[idx] = to_f32(rC[e]);
            }
        }
        __syncthreads();
        if (t + TT < t1) load(t + TT);
#pragma unroll 8
        for (int q = 0; q < TT; ++q) {
            const float2 d = dtu[q][sch];
            const float w = dyz[q][sch];
            const float4 b4 = *reinterpret_cast<const float4*>(&bc[0][q][m0]);
            const float4 c4 = *reinterpret_cast<const float4*>(&bc[1][q][m0]);
            const float bv[S] = {b4.x, b4.y, b4.z, b4.w}, cv[S] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const float e = ex2(d.x * A2[i]);
                h[i] = fmaf(e, h[i], d.y * bv[i]);
                P[i] *= e;
                G[i] = fmaf(P[i], w * cv[i], G[i]);
            }
            dts += d.x;
        }
        __syncthreads();
    }
    if (!sc_ok) return;
    const long long slot = (long long)item * a.D + sc;
    store_states(a.hs + slot * a.n, h, m0, a.n);
    store_states(a.gs + slot * a.n, G, m0, a.n);
    if (m0 == 0) a.dtsum[slot] = dts;
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
    const float A2 = a.in.A[e] * SCAN_LOG2E;
    const int first = a.ch.first_of(s), end = a.ch.end_of(s);
    float h = state_in ? state_in[s * DN + e] : 0.f;
    float g = dstate_out ? dstate_out[s * DN + e] : 0.f;
#pragma unroll 4
    for (int i = first; i < end; ++i) {
        const float local = a.hs[i * DN + e];
        const float decay = ex2(A2 * a.dtsum[(long long)i * a.D + c]);
        a.hs[i * DN + e] = h;
        h = fmaf(decay, h, local);
    }
#pragma unroll 4
    for (int i = end - 1; i >= first; --i) {
        const float local = a.gs[i * DN + e];
        const float decay = ex2(A2 * a.dtsum[(long long)i * a.D + c]);
        a.gs[i * DN + e] = g;
        g = fmaf(decay, g, local);
    }
    if (a.out.dstate_in) a.out.dstate_in[s * DN + e] = g;
}

template <int K> struct MainShared {
    static constexpr int NP = SCAN_S * K, CC = NT3 / K;
    static constexpr int TA = K == 1 ? 8 : K == 2 || K == 16 ? 16 : 32;
    float4 ck[LEN / BLK][NT3];  // states before each block
    union {
        struct {
            float2 dtu[TA][CC];
            float b[TA][NP];
        } a;
        struct {
            float2 dtu[BLK][CC];
            float dyz[BLK][CC];
            float bc[2][BLK][NP];
            float gB[BLK][CC], gA[BLK][CC], y[BLK][CC];
            float red[2][NT3 / 32][BLK][NP];  // dB and dC of each warp's channels
        } b;
    } u;
};

template <typename T, int K>
__global__ void __launch_bounds__(NT3, 2) main_kernel(BackArgs a)
{
    using Sh = MainShared<K>;
    constexpr int S = SCAN_S, NP = Sh::NP, CC = Sh::CC, TA = Sh::TA;
    constexpr int EA = TA * CC / NT3, EBA = (TA * NP + NT3 - 1) / NT3;
    constexpr int E = (BLK * CC + NT3 - 1) / NT3, EB = (BLK * NP + NT3 - 1) / NT3;
    constexpr int M = 32 / K;                     // channels per warp
    constexpr int RC = M < 8 ? 8 / M : 1;         // dB, dC values per lane after the reduction
    constexpr int RK = K < 4 ? 4 / K : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    Sh& sh = *reinterpret_cast<Sh*>(smem);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = a.G * a.cpg;
    const int item = blockIdx.x / blocks;
    const Place p(a, item, blockIdx.x % blocks, a.cpg, CC);
    const long long t0 = p.t0, t1 = p.t1;
    const int sch = tid / K, m0 = (tid % K) * S, sc = p.c0 + sch;
    const bool sc_ok = sc < p.c_end;
    const int ech = tid % CC, etok = tid / CC, ec = p.c0 + ech;
    const bool ec_ok = ec < p.c_end;
    const long long slot = (long long)item * a.D + sc;

    float A2[S] = {0.f, 0.f, 0.f, 0.f}, h[S] = {0.f, 0.f, 0.f, 0.f};
    float carry[S] = {0.f, 0.f, 0.f, 0.f}, dA[S] = {0.f, 0.f, 0.f, 0.f};
    if (sc_ok) {
        load_states(A2, a.in.A + (long long)sc * a.n, m0, a.n);
        load_states(h, a.hs + slot * a.n, m0, a.n);
        load_states(carry, a.gs + slot * a.n, m0, a.n);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) A2[i] *= SCAN_LOG2E;

    const T* up = (const T*)a.in.u + ec;
    const T* dp = (const T*)a.in.delta + ec;
    const T* zp = a.in.z ? (const T*)a.in.z + ec : nullptr;
    const T* yp = (const T*)a.dy + ec;
    const T* Bp = (const T*)a.in.B + (long long)p.g * a.n;
    const T* Cp = (const T*)a.in.C + (long long)p.g * a.n;
    const float dbias = a.in.delta_bias && ec_ok ? a.in.delta_bias[ec] : 0.f;
    const float Dw = a.in.D && ec_ok ? a.in.D[ec] : 0.f;

    // Forward walk: the state before each block.
    {
        T ru[EA], rd[EA], rB[EBA];
        auto load = [&](long long t) {
#pragma unroll
            for (int e = 0; e < EA; ++e) {
                const long long tok = t + e * K + etok;
                const bool ok = ec_ok && tok < t1;
                ru[e] = ok ? up[tok * a.in.ld_u] : T(0.f);
                rd[e] = ok ? dp[tok * a.in.ld_delta] : T(0.f);
            }
#pragma unroll
            for (int e = 0; e < EBA; ++e) {
                const int idx = e * NT3 + tid, m = idx % NP;
                const long long tok = t + idx / NP;
                const bool ok = m < a.n && tok < t1 && idx < TA * NP;
                rB[e] = ok ? Bp[tok * a.in.ld_b + m] : T(0.f);
            }
        };
        if (t0 < t1) load(t0);
        for (long long t = t0; t < t1; t += TA) {
#pragma unroll
            for (int e = 0; e < EA; ++e) {
                float dt = to_f32(rd[e]) + dbias;
                if (a.in.softplus) dt = softplus_f(dt);
                if (!ec_ok || t + e * K + etok >= t1) dt = 0.f;
                sh.u.a.dtu[e * K + etok][ech] = make_float2(dt, dt * to_f32(ru[e]));
            }
#pragma unroll
            for (int e = 0; e < EBA; ++e) {
                const int idx = e * NT3 + tid;
                if (idx < TA * NP) (&sh.u.a.b[0][0])[idx] = to_f32(rB[e]);
            }
            __syncthreads();
            if (t + TA < t1) load(t + TA);
#pragma unroll 1
            for (int tb = 0; tb < TA; tb += BLK) {
                const int blk = (int)(t - t0 + tb) / BLK;
                if (blk < LEN / BLK) sh.ck[blk][tid] = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
                for (int q = 0; q < BLK; ++q) {
                    const float2 d = sh.u.a.dtu[tb + q][sch];
                    const float4 b4 = *reinterpret_cast<const float4*>(&sh.u.a.b[tb + q][m0]);
                    const float bv[S] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                    for (int i = 0; i < S; ++i)
                        h[i] = fmaf(ex2(d.x * A2[i]), h[i], d.y * bv[i]);
                }
            }
            __syncthreads();
        }
    }

    // Blocks of 8 tokens, last to first.
    T ru[E], rd[E], rz[E], ry[E], rB[EB], rC[EB];
    auto load = [&](long long t) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int row = e * K + etok;
            const long long tok = t + row;
            const bool ok = ec_ok && tok < t1 && row < BLK;
            ru[e] = ok ? up[tok * a.in.ld_u] : T(0.f);
            rd[e] = ok ? dp[tok * a.in.ld_delta] : T(0.f);
            ry[e] = ok ? yp[tok * a.ld_dy] : T(0.f);
            rz[e] = ok && zp ? zp[tok * a.in.ld_z] : T(0.f);
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int idx = e * NT3 + tid, m = idx % NP;
            const long long tok = t + idx / NP;
            const bool ok = m < a.n && tok < t1 && idx < BLK * NP;
            rB[e] = ok ? Bp[tok * a.in.ld_b + m] : T(0.f);
            rC[e] = ok ? Cp[tok * a.in.ld_c + m] : T(0.f);
        }
    };
    float dD = 0.f, db = 0.f;
    const int nblk = (int)((t1 - t0 + BLK - 1) / BLK);
    if (nblk > 0) load(t0 + (nblk - 1) * BLK);
    auto& B = sh.u.b;
#pragma unroll 1
    for (int blk = nblk - 1; blk >= 0; --blk) {
        const long long t = t0 + blk * BLK;
        float eu[E], ed[E], edt[E], ez[E], ey[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int row = e * K + etok;
            eu[e] = to_f32(ru[e]);
            ed[e] = to_f32(rd[e]) + dbias;
            ez[e] = to_f32(rz[e]);
            ey[e] = to_f32(ry[e]);
            float dt = a.in.softplus ? softplus_f(ed[e]) : ed[e];
            if (!ec_ok || t + row >= t1) dt = 0.f;
            edt[e] = dt;
            if (row < BLK) {
                B.dtu[row][ech] = make_float2(dt, dt * eu[e]);
                B.dyz[row][ech] = zp ? ey[e] * ez[e] * sigmoid_f(ez[e]) : ey[e];
            }
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int idx = e * NT3 + tid;
            if (idx < BLK * NP) {
                (&B.bc[0][0][0])[idx] = to_f32(rB[e]);
                (&B.bc[1][0][0])[idx] = to_f32(rC[e]);
            }
        }
        __syncthreads();
        if (blk > 0) load(t - BLK);

        float hb[BLK][S], av[BLK][S];  // the state before each token, and its decay
        {
            const float4 c = sh.ck[blk][tid];
            h[0] = c.x, h[1] = c.y, h[2] = c.z, h[3] = c.w;
        }
#pragma unroll
        for (int q = 0; q < BLK; ++q) {
            const float2 d = B.dtu[q][sch];
            const float4 b4 = *reinterpret_cast<const float4*>(&B.bc[0][q][m0]);
            const float bv[S] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int i = 0; i < S; ++i) {
                hb[q][i] = h[i];
                av[q][i] = ex2(d.x * A2[i]);
                h[i] = fmaf(av[q][i], h[i], d.y * bv[i]);
            }
        }
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            float gB[4], gA[4], yv[4];
#pragma unroll
            for (int r = 3; r >= 0; --r) {
                const int q = half * 4 + r;
                const float2 d = B.dtu[q][sch];
                const float w = B.dyz[q][sch];
                const float4 b4 = *reinterpret_cast<const float4*>(&B.bc[0][q][m0]);
                const float4 c4 = *reinterpret_cast<const float4*>(&B.bc[1][q][m0]);
                const float bv[S] = {b4.x, b4.y, b4.z, b4.w}, cv[S] = {c4.x, c4.y, c4.z, c4.w};
                float v[8];
                gB[r] = gA[r] = yv[r] = 0.f;
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    const float ht = q == BLK - 1 ? h[i] : hb[q < BLK - 1 ? q + 1 : q][i];
                    const float g = fmaf(cv[i], w, carry[i]);
                    v[i] = g * d.y;
                    v[S + i] = w * ht;
                    yv[r] = fmaf(cv[i], ht, yv[r]);
                    gB[r] = fmaf(g, bv[i], gB[r]);
                    carry[i] = av[q][i] * g;
                    const float gh = carry[i] * hb[q][i];
                    gA[r] = fmaf(A2[i], gh, gA[r]);
                    dA[i] = fmaf(gh, d.x, dA[i]);
                }
                lane_reduce<8, M, K>(v, lane);
                if (reduced_writer<8, M, K>(lane)) {
                    const int at = reduced_index<8, M, K>(lane);
#pragma unroll
                    for (int x = 0; x < RC; ++x) {
                        const int idx = at + x;
                        B.red[idx / S][warp][q][m0 + idx % S] = v[x];
                    }
                }
            }
            lane_reduce<4, K, 1>(gB, lane);
            lane_reduce<4, K, 1>(gA, lane);
            lane_reduce<4, K, 1>(yv, lane);
            if (reduced_writer<4, K, 1>(lane)) {
                const int at = half * 4 + reduced_index<4, K, 1>(lane);
#pragma unroll
                for (int r = 0; r < RK; ++r) {
                    B.gB[at + r][sch] = gB[r];
                    B.gA[at + r][sch] = gA[r];
                    B.y[at + r][sch] = yv[r];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int row = e * K + etok;
            const long long tok = t + row;
            if (ec_ok && tok < t1 && row < BLK) {
                const float u = eu[e], gb = B.gB[row][ech];
                float w = ey[e];
                if (zp) {
                    const float sg = sigmoid_f(ez[e]), gate = ez[e] * sg;
                    const float y = fmaf(Dw, u, B.y[row][ech]);
                    store_out<T>(a.out.dz, tok * a.D + ec, w * y * (sg + gate * (1.f - sg)),
                                 a.out_f32);
                    w *= gate;
                }
                store_out<T>(a.out.du, tok * a.D + ec, fmaf(Dw, w, edt[e] * gb), a.out_f32);
                float dd = fmaf(SCAN_LN2, B.gA[row][ech], u * gb);
                if (a.in.softplus) dd *= sigmoid_f(ed[e]);
                store_out<T>(a.out.ddelta, tok * a.D + ec, dd, a.out_f32);
                dD = fmaf(w, u, dD);
                db += dd;
            }
        }
        for (int idx = tid; idx < 2 * BLK * NP; idx += NT3) {
            const int m = idx % NP, q = idx / NP % BLK, which = idx / (NP * BLK);
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < NT3 / 32; ++w) v += B.red[which][w][q][m];
            if (m < a.n && t + q < t1) {
                float* to = which ? a.dCp : a.dBp;
                to[(((long long)p.cbg * a.view.total + t + q) * a.G + p.g) * a.n + m] = v;
            }
        }
    }
    if (sc_ok) store_states(a.hs + slot * a.n, dA, m0, a.n);  // this thread's own, read above
    // dD and ddelta_bias of this chunk: K threads hold one channel's.
    __syncthreads();
    float* red = &B.red[0][0][0][0];
    float2* pair = reinterpret_cast<float2*>(red);
    pair[tid] = make_float2(dD, db);
    __syncthreads();
    if (tid < CC && ec_ok) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) x += pair[tid + k * CC].x, y += pair[tid + k * CC].y;
        a.dDp[(long long)item * a.D + ec] = x;
        a.dbp[(long long)item * a.D + ec] = y;
    }
}

// dB and dC: the sum of the channel blocks' slabs, for the rows of a sequence.
__global__ void __launch_bounds__(256) sum_bc_kernel(BackArgs a)
{
    const long long cols = (long long)a.G * a.n;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long rows = a.view.cu ? a.view.cu[a.view.num_seqs] : a.view.total;
    if (i >= a.view.total * cols || i / cols >= rows) return;
    const long long slab = a.view.total * cols;
    const float* in = (blockIdx.y ? a.dCp : a.dBp) + i;
    float v = 0.f;
#pragma unroll 8
    for (int r = 0; r < a.cpg; ++r) v += in[r * slab];
    store_out<float>(blockIdx.y ? a.out.dC : a.out.dB, i, v, a.out_f32);
}

// out[c] = sum of in[r][c]: 32 columns per CTA, 32 strands of rows.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* in, float* out,
                                                          int rows, long long cols)
{
    __shared__ float part[32][33];
    const int x = threadIdx.x, y = threadIdx.y;
    const long long c = (long long)blockIdx.x * 32 + x;
    float v = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int r = y; r < rows; r += 32) v += in[r * cols + c];
    }
    part[y][x] = v;
    __syncthreads();
    v = part[x][y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const long long oc = (long long)blockIdx.x * 32 + y;
    if (x == 0 && oc < cols) out[oc] = v;
}

struct BackLayout {
    int items, cpg;
    size_t hs, gs, dtsum, dDp, dbp, dBp, dCp, first, bytes;
};

BackLayout back_layout(int G, int D, long long total, int n, int num_seqs)
{
    BackLayout l;
    const int CC = NT3 / scan_lanes(n);
    l.items = (int)(total / LEN + num_seqs);
    l.cpg = (D / G + CC - 1) / CC;
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

cudaError_t launch_column_sum(const float* in, float* out, int rows, long long cols,
                              cudaStream_t stream)
{
    column_sum_kernel<<<(unsigned)((cols + 31) / 32), dim3(32, 32), 0, stream>>>(in, out, rows,
                                                                                cols);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_scan_backward(const ScanProblem& p, const float* state_in, const void* dy,
                                 long long ld_dy, const float* dstate_out,
                                 const la_scan_grads& out, void* ws, cudaStream_t stream)
{
    const int K = scan_lanes(p.n), num_seqs = p.view.num_seqs, Dg = p.D / p.G;
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
    a.dDp = (float*)(w + l.dDp);
    a.dbp = (float*)(w + l.dbp);
    a.dBp = (float*)(w + l.dBp);
    a.dCp = (float*)(w + l.dCp);
    a.D = p.D;
    a.G = p.G;
    a.n = p.n;
    a.cpg = l.cpg;
    a.out_f32 = p.out_t == LA_F32;
    a.ch.len = LEN;
    if (p.view.cu) {
        int* first = (int*)(w + l.first);
        a.ch.items = l.items;
        a.ch.first = first;
        a.ch.seq_of = first + num_seqs + 1;
        if (num_seqs > 0) {
            cudaError_t e = launch_plan_chunks(p.view, LEN, l.items, first, first + num_seqs + 1,
                                               stream);
            if (e != cudaSuccess) return e;
        }
    } else if (num_seqs > 0) {
        const long long per = (p.view.N + LEN - 1) / LEN;
        a.ch.per_seq = per > 1 ? (int)per : 1;
        a.ch.items = a.ch.per_seq * num_seqs;
    }
    cudaError_t e = cudaSuccess;
    const long long DN = (long long)p.D * p.n;
    if (num_seqs > 0) {
        const int CC1 = NT1 / K, cpg1 = (Dg + CC1 - 1) / CC1;
        const unsigned grid1 = (unsigned)((long long)a.ch.items * p.G * cpg1);
        const unsigned grid3 = (unsigned)((long long)a.ch.items * p.G * a.cpg);
        const unsigned grid2 = (unsigned)((DN + 127) / 128 * num_seqs);
#define LA_CALL(KK)                                                                              \
    do {                                                                                         \
        const int smem = (int)sizeof(MainShared<KK>);                                            \
        auto main = p.in_t == LA_BF16 ? main_kernel<__nv_bfloat16, KK> : main_kernel<float, KK>; \
        auto local =                                                                             \
            p.in_t == LA_BF16 ? local_kernel<__nv_bfloat16, KK> : local_kernel<float, KK>;       \
        e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);       \
        if (e != cudaSuccess) return e;                                                          \
        local<<<grid1, NT1, 0, stream>>>(a, cpg1);                                               \
        combine_kernel<<<grid2, 128, 0, stream>>>(a, state_in, dstate_out);                      \
        main<<<grid3, NT3, smem, stream>>>(a);                                                   \
    } while (0)
        LA_SCAN_DISPATCH_K(p.n, LA_CALL)
#undef LA_CALL
        count_launch(3);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if (p.view.total > 0) {
            const long long cells = p.view.total * p.G * p.n;
            sum_bc_kernel<<<dim3((unsigned)((cells + 255) / 256), 2), 256, 0, stream>>>(a);
            count_launch();
        }
    }
    const int rows = num_seqs > 0 ? a.ch.items : 0;
    if ((e = launch_column_sum(a.hs, out.dA, rows, DN, stream)) != cudaSuccess) return e;
    if (out.dD && (e = launch_column_sum(a.dDp, out.dD, rows, p.D, stream)) != cudaSuccess)
        return e;
    if (out.ddelta_bias) return launch_column_sum(a.dbp, out.ddelta_bias, rows, p.D, stream);
    return cudaSuccess;
}

}  // namespace la
