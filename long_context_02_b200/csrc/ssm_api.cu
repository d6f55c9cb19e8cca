// C ABI of the state space layer: argument checks and dispatch. The public
// contract of every entry point is documented in include/lightning.h.
#include <cstdint>

#include "ssm.h"

namespace la {

namespace {

// Features and states that keep every index of a row, every count of chunks and
// every grid within 31 bits.
bool sizes_fit(int D, int num_seqs)
{
    return D <= LA_MAX_LD && (long long)num_seqs * D <= (1 << 30);
}

}  // namespace

size_t ssm_workspace_bytes(int op, int G, int D, long long total, int n, int num_seqs)
{
    if (D <= 0 || total < 0 || total > LA_MAX_TOKENS || D > LA_MAX_LD) return 0;
    switch (op) {
    case LA_OP_SCAN:
    case LA_OP_SCAN_BACKWARD:
        if (G <= 0 || D % G || n <= 0 || n > LA_MAX_SCAN_STATES || num_seqs < 0 ||
            !sizes_fit(D, num_seqs))
            return 0;
        return scan_workspace(op == LA_OP_SCAN_BACKWARD, G, D, total, n, num_seqs);
    case LA_OP_CONV_BACKWARD:
        if (n < 2 || n > 4) return 0;
        return conv_backward_workspace(D, total, n);
    case LA_OP_NORM_BACKWARD:
        if (D > LA_MAX_NORM_FEATURES) return 0;
        return norm_backward_workspace(total, D);
    default: return 0;
    }
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// Of a dense tensor whose slices along the first dimension have `count` elements of
// `size` bytes (weights: the whole tensor): aligned to the largest power of two, at
// most 16, that divides them. The kernels choose vectors by widths alone, so a width
// that allows none asks for no more than its elements' alignment.
bool dense(const void* p, long long count, size_t size)
{
    const size_t bytes = (size_t)count * size, most = bytes & (~bytes + 1);
    return aligned(p, most < 16 ? most : 16);
}
size_t elem(int t) { return t == LA_BF16 ? 2 : 4; }

int check_types(int in_t, int out_t)
{
    if ((in_t != LA_BF16 && in_t != LA_F32) || (out_t != LA_BF16 && out_t != LA_F32))
        return LA_ERR_INVALID_ARG;
    return in_t == LA_F32 && out_t != LA_F32 ? LA_ERR_UNSUPPORTED : LA_OK;
}

// Sequences and rows; fills the view.
int check_sequences(const int* cu, int num_seqs, long long total, int D, SeqView& v)
{
    if (num_seqs < 0 || total < 0 || D <= 0) return LA_ERR_INVALID_ARG;
    if (num_seqs == 0 && total > 0) return LA_ERR_INVALID_ARG;  // rows of no sequence
    if (!cu && num_seqs > 0 && total % num_seqs) return LA_ERR_INVALID_ARG;
    if (total > LA_MAX_TOKENS || !sizes_fit(D, num_seqs)) return LA_ERR_UNSUPPORTED;
    if (!aligned(cu, 4)) return LA_ERR_INVALID_ARG;
    v.cu = cu;
    v.num_seqs = num_seqs;
    v.total = total;
    v.N = num_seqs > 0 ? total / num_seqs : 0;
    return LA_OK;
}

int check_scan(const la_scan_inputs* in, long long rows, int D, int G, int n, int in_t, int out_t)
{
    if (!in || G <= 0 || D % G || n <= 0) return LA_ERR_INVALID_ARG;
    if (n > LA_MAX_SCAN_STATES) return LA_ERR_UNSUPPORTED;
    if (int st = check_types(in_t, out_t)) return st;
    if (!in->A || (rows > 0 && (!in->u || !in->delta || !in->B || !in->C)))
        return LA_ERR_INVALID_ARG;
    const size_t e = elem(in_t);
    if (!aligned(in->u, e) || !aligned(in->delta, e) || !aligned(in->z, e) || !aligned(in->B, e) ||
        !aligned(in->C, e) || !dense(in->A, (long long)D * n, 4) || !dense(in->D, D, 4) ||
        !dense(in->delta_bias, D, 4))
        return LA_ERR_INVALID_ARG;
    const long long bc = (long long)G * n;
    if (rows > 1 && (in->ld_u > LA_MAX_LD || in->ld_delta > LA_MAX_LD ||
                     (in->z && in->ld_z > LA_MAX_LD) || in->ld_b > LA_MAX_LD ||
                     in->ld_c > LA_MAX_LD))
        return LA_ERR_UNSUPPORTED;
    if (rows > 1 && (in->ld_u < D || in->ld_delta < D || (in->z && in->ld_z < D) ||
                     in->ld_b < bc || in->ld_c < bc))
        return LA_ERR_INVALID_ARG;
    return LA_OK;
}

int check_ws(const void* ws, size_t have, size_t need)
{
    return need > 0 && (!ws || have < need || !aligned(ws, 16)) ? LA_ERR_WORKSPACE : LA_OK;
}

int check_conv(const void* x, long long ld_x, const float* weight, const float* bias,
               long long rows, int D, int W, int in_t, int out_t)
{
    if (W <= 0) return LA_ERR_INVALID_ARG;
    if (W < 2 || W > 4) return LA_ERR_UNSUPPORTED;
    if (int st = check_types(in_t, out_t)) return st;
    if (!weight || (rows > 0 && !x)) return LA_ERR_INVALID_ARG;
    if (!aligned(x, elem(in_t)) || !dense(weight, (long long)D * W, 4) || !dense(bias, D, 4))
        return LA_ERR_INVALID_ARG;
    if (rows > 1 && ld_x > LA_MAX_LD) return LA_ERR_UNSUPPORTED;
    return rows > 1 && ld_x < D ? LA_ERR_INVALID_ARG : LA_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }
cudaStream_t stream_of(la_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

LA_API int la_selective_scan(const int* cu_seqlens, int num_seqs, const la_scan_inputs* in,
                             const float* state_in, void* y, float* state_out, long long total,
                             int D, int G, int n, int in_t, int out_t, void* workspace,
                             size_t ws_bytes, la_stream_t stream)
{
    reset_launches();
    ScanProblem p;
    int st = check_sequences(cu_seqlens, num_seqs, total, D, p.view);
    if (st != LA_OK || (st = check_scan(in, total, D, G, n, in_t, out_t)) != LA_OK) return st;
    if (total > 0 && !y) return LA_ERR_INVALID_ARG;
    const long long DN = (long long)D * n;
    if (!dense(y, D, elem(out_t)) || !dense(state_in, DN, 4) || !dense(state_out, DN, 4))
        return LA_ERR_INVALID_ARG;
    st = check_ws(workspace, ws_bytes, scan_workspace(false, G, D, total, n, num_seqs));
    if (st != LA_OK) return st;
    if (num_seqs == 0) return LA_OK;
    p.in = *in;
    p.D = D;
    p.G = G;
    p.n = n;
    p.in_t = in_t;
    p.out_t = out_t;
    return status_of(launch_scan(p, state_in, y, state_out, workspace, stream_of(stream)));
}

LA_API int la_selective_scan_step(const la_scan_inputs* in, float* state, void* y, int B, int D,
                                  int G, int n, int in_t, int out_t, la_stream_t stream)
{
    reset_launches();
    ScanProblem p;
    int st = check_sequences(nullptr, B, B, D, p.view);
    if (st != LA_OK || (st = check_scan(in, B, D, G, n, in_t, out_t)) != LA_OK) return st;
    if (B == 0) return LA_OK;
    if (!state || !y || !dense(state, (long long)D * n, 4) || !dense(y, D, elem(out_t)))
        return LA_ERR_INVALID_ARG;
    p.in = *in;
    p.D = D;
    p.G = G;
    p.n = n;
    p.in_t = in_t;
    p.out_t = out_t;
    return status_of(launch_scan_step(p, state, y, stream_of(stream)));
}

LA_API int la_selective_scan_backward(const int* cu_seqlens, int num_seqs,
                                      const la_scan_inputs* in, const float* state_in,
                                      const void* dy, long long ld_dy, const float* dstate_out,
                                      const la_scan_grads* out, long long total, int D, int G,
                                      int n, int in_t, int out_t, void* workspace,
                                      size_t ws_bytes, la_stream_t stream)
{
    reset_launches();
    ScanProblem p;
    int st = check_sequences(cu_seqlens, num_seqs, total, D, p.view);
    if (st != LA_OK || (st = check_scan(in, total, D, G, n, in_t, out_t)) != LA_OK) return st;
    if (!out || !out->dA || (total > 0 && (!dy || !out->du || !out->ddelta || !out->dB || !out->dC)))
        return LA_ERR_INVALID_ARG;
    if (total > 0 && !in->z != !out->dz) return LA_ERR_INVALID_ARG;
    if (!aligned(dy, elem(in_t)) || (total > 1 && ld_dy < D)) return LA_ERR_INVALID_ARG;
    if (total > 1 && ld_dy > LA_MAX_LD) return LA_ERR_UNSUPPORTED;
    const long long DN = (long long)D * n, GN = (long long)G * n;
    const size_t e = elem(out_t);
    if (!dense(state_in, DN, 4) || !dense(dstate_out, DN, 4) || !dense(out->du, D, e) ||
        !dense(out->ddelta, D, e) || !dense(out->dz, D, e) || !dense(out->dB, GN, e) ||
        !dense(out->dC, GN, e) || !dense(out->dA, DN, 4) || !dense(out->dD, D, 4) ||
        !dense(out->ddelta_bias, D, 4) || !dense(out->dstate_in, DN, 4))
        return LA_ERR_INVALID_ARG;
    st = check_ws(workspace, ws_bytes, scan_workspace(true, G, D, total, n, num_seqs));
    if (st != LA_OK) return st;
    p.in = *in;
    p.D = D;
    p.G = G;
    p.n = n;
    p.in_t = in_t;
    p.out_t = out_t;
    return status_of(launch_scan_backward(p, state_in, dy, ld_dy, dstate_out, *out, workspace,
                                          stream_of(stream)));
}

LA_API int la_short_conv(const int* cu_seqlens, int num_seqs, const void* x, long long ld_x,
                         const float* weight, const float* bias, const void* state_in, void* y,
                         void* state_out, long long total, int D, int W, int silu, int in_t,
                         int out_t, la_stream_t stream)
{
    reset_launches();
    ConvProblem p;
    int st = check_sequences(cu_seqlens, num_seqs, total, D, p.view);
    if (st != LA_OK || (st = check_conv(x, ld_x, weight, bias, total, D, W, in_t, out_t)) != LA_OK)
        return st;
    if (total > 0 && !y) return LA_ERR_INVALID_ARG;
    const long long rest = (long long)(W - 1) * D;  // of a state
    if (!dense(y, D, elem(out_t)) || !dense(state_in, rest, elem(in_t)) ||
        !dense(state_out, rest, elem(in_t)) ||
        (state_out && state_out == state_in))
        return LA_ERR_INVALID_ARG;
    if (num_seqs == 0) return LA_OK;
    p.x = x;
    p.ld_x = ld_x;
    p.weight = weight;
    p.bias = bias;
    p.D = D;
    p.W = W;
    p.silu = silu;
    p.in_t = in_t;
    p.out_t = out_t;
    return status_of(launch_short_conv(p, state_in, y, state_out, stream_of(stream)));
}

LA_API int la_short_conv_step(const void* x, long long ld_x, const float* weight,
                              const float* bias, void* state, void* y, int B, int D, int W,
                              int silu, int in_t, int out_t, la_stream_t stream)
{
    reset_launches();
    ConvProblem p;
    int st = check_sequences(nullptr, B, B, D, p.view);
    if (st != LA_OK || (st = check_conv(x, ld_x, weight, bias, B, D, W, in_t, out_t)) != LA_OK)
        return st;
    if (B == 0) return LA_OK;
    if (!state || !y || !dense(state, (long long)(W - 1) * D, elem(in_t)) ||
        !dense(y, D, elem(out_t)))
        return LA_ERR_INVALID_ARG;
    p.x = x;
    p.ld_x = ld_x;
    p.weight = weight;
    p.bias = bias;
    p.D = D;
    p.W = W;
    p.silu = silu;
    p.in_t = in_t;
    p.out_t = out_t;
    return status_of(launch_short_conv_step(p, state, y, stream_of(stream)));
}

LA_API int la_short_conv_backward(const int* cu_seqlens, int num_seqs, const void* dy,
                                  long long ld_dy, const void* x, long long ld_x,
                                  const float* weight, const float* bias, const void* state_in,
                                  const void* dstate_out, void* dx, float* dweight, float* dbias,
                                  void* dstate_in, long long total, int D, int W, int silu,
                                  int in_t, int out_t, void* workspace, size_t ws_bytes,
                                  la_stream_t stream)
{
    reset_launches();
    ConvProblem p;
    int st = check_sequences(cu_seqlens, num_seqs, total, D, p.view);
    if (st != LA_OK || (st = check_conv(x, ld_x, weight, bias, total, D, W, in_t, out_t)) != LA_OK)
        return st;
    if (!dweight || (total > 0 && (!dy || !dx))) return LA_ERR_INVALID_ARG;
    if (!aligned(dy, elem(in_t)) || (total > 1 && ld_dy < D)) return LA_ERR_INVALID_ARG;
    if (total > 1 && ld_dy > LA_MAX_LD) return LA_ERR_UNSUPPORTED;
    const long long rest = (long long)(W - 1) * D;  // of a state
    if (!dense(state_in, rest, elem(in_t)) || !dense(dstate_out, rest, elem(in_t)) ||
        !dense(dx, D, elem(out_t)) || !dense(dweight, (long long)D * W, 4) || !dense(dbias, D, 4) ||
        !dense(dstate_in, rest, elem(out_t)))
        return LA_ERR_INVALID_ARG;
    if ((st = check_ws(workspace, ws_bytes, conv_backward_workspace(D, total, W))) != LA_OK)
        return st;
    p.x = x;
    p.ld_x = ld_x;
    p.weight = weight;
    p.bias = bias;
    p.D = D;
    p.W = W;
    p.silu = silu;
    p.in_t = in_t;
    p.out_t = out_t;
    return status_of(launch_short_conv_backward(p, dy, ld_dy, state_in, dstate_out, dx, dweight,
                                                dbias, dstate_in, workspace, stream_of(stream)));
}

namespace {

int check_norm(const void* x, const float* weight, const float* bias, long long rows, int F,
               int in_t, int out_t)
{
    if (rows < 0 || F <= 0) return LA_ERR_INVALID_ARG;
    if (F > LA_MAX_NORM_FEATURES || rows > LA_MAX_TOKENS) return LA_ERR_UNSUPPORTED;
    if (int st = check_types(in_t, out_t)) return st;
    if (rows > 0 && (!x || !weight)) return LA_ERR_INVALID_ARG;
    return dense(x, F, elem(in_t)) && dense(weight, F, 4) && dense(bias, F, 4) ? LA_OK
                                                                               : LA_ERR_INVALID_ARG;
}

}  // namespace

LA_API int la_layer_norm(const void* x, const float* weight, const float* bias, float eps,
                         void* y, float* mean, float* rstd, long long rows, int F, int in_t,
                         int out_t, la_stream_t stream)
{
    reset_launches();
    int st = check_norm(x, weight, bias, rows, F, in_t, out_t);
    if (st != LA_OK) return st;
    if (!(eps >= 0.f) || eps > 3.0e38f) return LA_ERR_INVALID_ARG;  // also rejects NaN
    if (rows == 0) return LA_OK;
    if (!y || !mean != !rstd || (y == x && in_t != out_t)) return LA_ERR_INVALID_ARG;
    if (!dense(y, F, elem(out_t)) || !aligned(mean, 4) || !aligned(rstd, 4)) return LA_ERR_INVALID_ARG;
    return status_of(launch_layer_norm(x, weight, bias, eps, y, mean, rstd, rows, F, in_t, out_t,
                                       stream_of(stream)));
}

LA_API int la_layer_norm_backward(const void* dy, const void* x, const float* weight,
                                  const float* mean, const float* rstd, void* dx, float* dweight,
                                  float* dbias, long long rows, int F, int in_t, int out_t,
                                  void* workspace, size_t ws_bytes, la_stream_t stream)
{
    reset_launches();
    int st = check_norm(x, weight, dbias, rows, F, in_t, out_t);
    if (st != LA_OK) return st;
    if (!dweight || (rows > 0 && (!dy || !mean || !rstd || !dx))) return LA_ERR_INVALID_ARG;
    if (!dense(dy, F, elem(in_t)) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !dense(dx, F, elem(out_t)) || !dense(dweight, F, 4))
        return LA_ERR_INVALID_ARG;
    if ((st = check_ws(workspace, ws_bytes, norm_backward_workspace(rows, F))) != LA_OK) return st;
    return status_of(launch_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias,
                                                rows, F, in_t, out_t, workspace,
                                                stream_of(stream)));
}

}  // extern "C"
