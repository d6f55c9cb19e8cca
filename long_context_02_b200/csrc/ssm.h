// Internal types and launchers of the state space layer (selective scan,
// short convolution, layer norm); the public contract is in lightning.h.
#pragma once

#include "common.cuh"

namespace la {

// The sequences of a token-major tensor: dense (cu == nullptr, N tokens each)
// or packed by device offsets.
struct SeqView {
    const int* cu = nullptr;
    int num_seqs = 0;
    long long N = 0;      // dense: tokens per sequence
    long long total = 0;  // rows of the tensors

    // Rows [start, end) of sequence s; packed offsets are clamped to the tensor.
    __device__ __forceinline__ void range(int s, long long& start, long long& end) const
    {
        if (!cu) {
            start = (long long)s * N;
            end = start + N;
            return;
        }
        start = cu[s];
        end = cu[s + 1];
        start = start < 0 ? 0 : (start > total ? total : start);
        end = end < start ? start : (end > total ? total : end);
    }
    // The sequence that holds row t (num_seqs when none does): the last s with cu[s] <= t.
    __device__ __forceinline__ int find(long long t) const
    {
        if (!cu) return N > 0 ? (int)(t / N) : num_seqs;
        int lo = 0, hi = num_seqs + 1;  // cu[lo - 1] <= t < cu[hi]
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if ((long long)cu[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        return lo > 0 ? lo - 1 : num_seqs;
    }
};

// Sequences cut into chunks of `len` tokens, every sequence into at least one
// (an empty one has an empty chunk). Dense: per_seq chunks each. Packed: a
// table made on the device; without one (first == nullptr) one chunk each.
struct Chunks {
    long long len = 0;
    int items = 0;                 // chunks, or an upper bound of them (packed)
    int per_seq = 1;               // dense
    const int* first = nullptr;    // packed: [num_seqs + 1] first chunk of each sequence
    const int* seq_of = nullptr;   // packed: [items] sequence of each chunk, -1 behind the last

    __device__ __forceinline__ int seq(int item) const
    {
        return seq_of ? seq_of[item] : item / per_seq;
    }
    __device__ __forceinline__ int first_of(int s) const { return first ? first[s] : s * per_seq; }
    __device__ __forceinline__ int end_of(int s) const
    {
        const int e = first ? first[s + 1] : (s + 1) * per_seq;
        return e < items ? e : items;
    }
};

// Fill `first` and `seq_of` of a packed batch.
cudaError_t launch_plan_chunks(const SeqView& v, long long len, int items, int* first, int* seq_of,
                               cudaStream_t stream);

// Column sums out[c] = sum over r < rows of in[r][c], in a fixed order, of up to
// five matrices in one launch. Jobs without an output are left out.
struct SumJobs {
    struct Job {
        const float* in;
        void* out;
        int rows;
        long long cols;
        int bf16;  // dtype of out
        // Packed batch: only the columns of rows that a sequence holds, cu_end[0]
        // times `per_row` of them; the others are left as they were.
        const int* cu_end;
        long long per_row;
        long long first_block;
        int strands;  // threads that share a column's rows
    } job[5];
    int count = 0;
    long long blocks = 0;
    void add(const float* in, void* out, int rows, long long cols, int bf16 = 0,
             const int* cu_end = nullptr, long long per_row = 1);
};
cudaError_t launch_column_sums(const SumJobs& jobs, cudaStream_t stream);

// Dynamic shared memory beyond the default limit, once per kernel and device.
cudaError_t allow_shared(const void* kernel, int bytes);

size_t ssm_workspace_bytes(int op, int G, int D, long long total, int n, int num_seqs);

struct ScanProblem {
    la_scan_inputs in;
    SeqView view;
    int D, G, n;
    int in_t, out_t;
};

size_t scan_workspace(bool backward, int G, int D, long long total, int n, int num_seqs);
cudaError_t launch_scan(const ScanProblem& p, const float* state_in, void* y, float* state_out,
                        void* ws, cudaStream_t stream);
cudaError_t launch_scan_step(const ScanProblem& p, float* state, void* y, cudaStream_t stream);
cudaError_t launch_scan_backward(const ScanProblem& p, const float* state_in, const void* dy,
                                 long long ld_dy, const float* dstate_out,
                                 const la_scan_grads& out, void* ws, cudaStream_t stream);

struct ConvProblem {
    const void* x;
    long long ld_x;
    const float* weight;
    const float* bias;
    SeqView view;
    int D, W, silu;
    int in_t, out_t;
};

size_t conv_backward_workspace(int D, long long total, int W);
cudaError_t launch_short_conv(const ConvProblem& p, const void* state_in, void* y,
                              void* state_out, cudaStream_t stream);
cudaError_t launch_short_conv_step(const ConvProblem& p, void* state, void* y,
                                   cudaStream_t stream);
cudaError_t launch_short_conv_backward(const ConvProblem& p, const void* dy, long long ld_dy,
                                       const void* state_in, const void* dstate_out, void* dx,
                                       float* dweight, float* dbias, void* dstate_in, void* ws,
                                       cudaStream_t stream);

size_t norm_backward_workspace(long long rows, int F);
cudaError_t launch_layer_norm(const void* x, const float* weight, const float* bias, float eps,
                              void* y, float* mean, float* rstd, long long rows, int F, int in_t,
                              int out_t, cudaStream_t stream);
cudaError_t launch_layer_norm_backward(const void* dy, const void* x, const float* weight,
                                       const float* mean, const float* rstd, void* dx,
                                       float* dweight, float* dbias, long long rows, int F,
                                       int in_t, int out_t, void* ws, cudaStream_t stream);

}  // namespace la
