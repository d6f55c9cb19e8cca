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

constexpr int NT = 128;  // threads per CTA

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

// MODE 0: with outputs. MODE 1: the chunks' states only.
template <typename T, int K, int MODE>
__global__ void __launch_bounds__(NT) scan_kernel(ScanArgs a)
{
    constexpr int S = SCAN_S, NP = S * K, CC = NT / K;
    constexpr int TT = K == 1 ? 8 : K == 2 || K == 16 ? 16 : 32;  // tokens per tile
    constexpr int E = TT * CC / NT;                               // elements per thread
    constexpr int EB = (TT * NP + NT - 1) / NT;
    constexpr int YS = CC + 32 / K;  // padded row of the output tile
    constexpr int R = K < 8 ? 8 / K : 1;
    __shared__ float2 dtu[TT][CC];
    __shared__ __align__(16) float bc[2][TT][NP];
    __shared__ float ys[MODE == 0 ? TT : 1][YS];

    const int tid = threadIdx.x, lane = tid & 31;
    const int blocks = a.G * a.cpg;
    const int item = blockIdx.x / blocks, cb = blockIdx.x % blocks;
    const int s = a.ch.seq(item);
    if (s < 0) return;
    const int chunk = item - a.ch.first_of(s), nchunks = a.ch.end_of(s) - a.ch.first_of(s);
    const bool last = chunk == nchunks - 1;
    long long t0, t1;
    a.view.range(s, t0, t1);
    t0 += chunk * a.ch.len;
    if (t1 - t0 > a.ch.len) t1 = t0 + a.ch.len;

    const int g = cb / a.cpg, Dg = a.D / a.G;
    const int c0 = g * Dg + (cb % a.cpg) * CC, c_end = (g + 1) * Dg;
    // scan mapping
    const int sch = tid / K, m0 = (tid % K) * S, sc = c0 + sch;
    const bool sc_ok = sc < c_end;
    // element mapping
    const int ech = tid % CC, etok = tid / CC, ec = c0 + ech;
    const bool ec_ok = ec < c_end;

    float A2[S], h[S] = {0.f, 0.f, 0.f, 0.f};
    if (sc_ok) {
        load_states(A2, a.in.A + (long long)sc * a.n, m0, a.n);
#pragma unroll
        for (int i = 0; i < S; ++i) A2[i] *= SCAN_LOG2E;
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i) A2[i] = 0.f;
    }
    const long long slot = ((long long)item * a.D + sc) * a.n;
    if (sc_ok) {
        if (MODE == 1) {
            // The last chunk's slot is free: it keeps the incoming state, which
            // may be overwritten in place before the first chunk reads it.
            if (a.state_in && (chunk == 0 || last))
                load_states(h, a.state_in + ((long long)s * a.D + sc) * a.n, m0, a.n);
            if (last) store_states(a.local + slot, h, m0, a.n);
        } else if (nchunks == 1) {
            if (a.state_in)
                load_states(h, a.state_in + ((long long)s * a.D + sc) * a.n, m0, a.n);
        } else if (chunk == 0) {
            load_states(h, a.local + slot + (long long)(nchunks - 1) * a.D * a.n, m0, a.n);
        } else {
            const long long first = (long long)a.ch.first_of(s) * a.D + sc;
            load_states(h, a.local + first * a.n, m0, a.n);
#pragma unroll 4
            for (int c = 1; c < chunk; ++c) {
                float l[S];
                load_states(l, a.local + (first + (long long)c * a.D) * a.n, m0, a.n);
                const float d = a.dtsum[first + (long long)c * a.D];
#pragma unroll
                for (int i = 0; i < S; ++i) h[i] = fmaf(ex2(d * A2[i]), h[i], l[i]);
            }
        }
    }
    if (MODE == 1 && last) return;

    const T* up = (const T*)a.in.u + ec;
    const T* dp = (const T*)a.in.delta + ec;
    const T* zp = a.in.z ? (const T*)a.in.z + ec : nullptr;
    const T* Bp = (const T*)a.in.B + (long long)g * a.n;
    const T* Cp = (const T*)a.in.C + (long long)g * a.n;
    const float dbias = a.in.delta_bias && ec_ok ? a.in.delta_bias[ec] : 0.f;
    const float Dw = a.in.D && ec_ok ? a.in.D[ec] : 0.f;

    T ru[E], rd[E], rz[E], rB[EB], rC[EB];
    auto load = [&](long long t) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const long long tok = t + e * K + etok;
            const bool ok = ec_ok && tok < t1;
            ru[e] = ok ? up[tok * a.in.ld_u] : T(0.f);
            rd[e] = ok ? dp[tok * a.in.ld_delta] : T(0.f);
            if (MODE == 0) rz[e] = ok && zp ? zp[tok * a.in.ld_z] : T(0.f);
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int idx = e * NT + tid, m = idx % NP;
            const long long tok = t + idx / NP;
            const bool ok = m < a.n && tok < t1 && idx < TT * NP;
            rB[e] = ok ? Bp[tok * a.in.ld_b + m] : T(0.f);
            if (MODE == 0) rC[e] = ok ? Cp[tok * a.in.ld_c + m] : T(0.f);
        }
    };

    float dts = 0.f;
    if (t0 < t1) load(t0);
    for (long long t = t0; t < t1; t += TT) {
        float cu[E], cz[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            cu[e] = to_f32(ru[e]);
            if (MODE == 0) cz[e] = to_f32(rz[e]);
            float dt = to_f32(rd[e]) + dbias;
            if (a.in.softplus) dt = softplus_f(dt);
            if (!ec_ok || t + e * K + etok >= t1) dt = 0.f;
            dtu[e * K + etok][ech] = make_float2(dt, dt * cu[e]);
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            const int idx = e * NT + tid;
            if (idx < TT * NP) {
                (&bc[0][0][0])[idx] = to_f32(rB[e]);
                if (MODE == 0) (&bc[1][0][0])[idx] = to_f32(rC[e]);
            }
        }
        __syncthreads();
        if (t + TT < t1) load(t + TT);
#pragma unroll 1
        for (int tb = 0; tb < TT; tb += 8) {
            float acc[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float2 d = dtu[tb + q][sch];
                const float4 b4 = *reinterpret_cast<const float4*>(&bc[0][tb + q][m0]);
                const float bv[S] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                for (int i = 0; i < S; ++i) h[i] = fmaf(ex2(d.x * A2[i]), h[i], d.y * bv[i]);
                if (MODE == 0) {
                    const float4 c4 = *reinterpret_cast<const float4*>(&bc[1][tb + q][m0]);
                    acc[q] = fmaf(c4.x, h[0], c4.y * h[1]) + fmaf(c4.z, h[2], c4.w * h[3]);
                } else {
                    dts += d.x;
                }
            }
            if (MODE == 0) {
                lane_reduce<8, K, 1>(acc, lane);
                if (reduced_writer<8, K, 1>(lane)) {
                    const int at = reduced_index<8, K, 1>(lane);
#pragma unroll
                    for (int r = 0; r < R; ++r) ys[tb + at + r][sch] = acc[r];
                }
            }
        }
        __syncthreads();
        if (MODE == 0 && ec_ok) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int row = e * K + etok;
                const long long tok = t + row;
                if (tok < t1) {
                    float y = fmaf(Dw, cu[e], ys[row][ech]);
                    if (zp) y *= cz[e] * sigmoid_f(cz[e]);
                    if (a.out_f32) ((float*)a.y)[tok * a.D + ec] = y;
                    else ((__nv_bfloat16*)a.y)[tok * a.D + ec] = __float2bfloat16_rn(y);
                }
            }
        }
    }
    if (!sc_ok) return;
    if (MODE == 1) {
        store_states(a.local + slot, h, m0, a.n);
        if (m0 == 0) a.dtsum[(long long)item * a.D + sc] = dts;
    } else if (last && a.state_out) {
        store_states(a.state_out + ((long long)s * a.D + sc) * a.n, h, m0, a.n);
    }
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

// How the forward scan is cut. GPU_WARPS: four schedulers on 148 SMs.
ForwardPlan plan_forward(int G, int D, long long total, int n, int num_seqs)
{
    constexpr long long GPU_WARPS = 148 * 4;
    const int K = scan_lanes(n), CC = NT / K;
    const long long blocks = (long long)G * ((D / G + CC - 1) / CC);
    const long long warps = blocks * (NT / 32);
    if (num_seqs == 0 || warps * num_seqs >= GPU_WARPS) return {0, num_seqs};
    long long want = (2 * GPU_WARPS + warps - 1) / warps;  // chunks
    if (want > 64) want = 64;
    long long len = ((total + want - 1) / want + 31) / 32 * 32;
    if (len < 64) len = 64;
    if (len * num_seqs >= total && total / num_seqs * 2 < len * 3) return {0, num_seqs};
    return {len, (int)(total / len + num_seqs)};
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
    const ForwardPlan f = plan_forward(G, D, total, n, num_seqs);
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
    const ForwardPlan f = plan_forward(p.G, p.D, p.view.total, p.n, p.view.num_seqs);
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
#define LA_CALL(KK)                                                                              \
    if (p.in_t == LA_BF16) {                                                                     \
        if (f.len) scan_kernel<__nv_bfloat16, KK, 1><<<grid, NT, 0, stream>>>(a);                \
        scan_kernel<__nv_bfloat16, KK, 0><<<grid, NT, 0, stream>>>(a);                           \
    } else {                                                                                     \
        if (f.len) scan_kernel<float, KK, 1><<<grid, NT, 0, stream>>>(a);                        \
        scan_kernel<float, KK, 0><<<grid, NT, 0, stream>>>(a);                                   \
    }
    LA_SCAN_DISPATCH_K(p.n, LA_CALL)
#undef LA_CALL
    count_launch(f.len ? 2 : 1);
    return cudaGetLastError();
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
