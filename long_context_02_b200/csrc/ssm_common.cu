// What the state space layer's operators share: column sums of partial results
// and the launch attribute for large shared memory.
#include <atomic>

#include "ssm.h"

namespace la {
namespace {

constexpr int NT = 256;

// Threads that share the rows of a column (a power of two): enough of them that
// there are 1024 threads per SM.
int strands_for(int rows, long long cols)
{
    int s = 1;
    while (s < 32 && 2 * s <= rows && cols * s < 148LL * 1024) s *= 2;
    return s;
}

__global__ void __launch_bounds__(NT) column_sums_kernel(SumJobs jobs)
{
    __shared__ float part[NT];
    int j = 0;
    while (j + 1 < jobs.count && (long long)blockIdx.x >= jobs.job[j + 1].first_block) ++j;
    const SumJobs::Job job = jobs.job[j];
    const int width = NT / job.strands;  // columns of this CTA
    const int x = threadIdx.x % width, y = threadIdx.x / width;
    const long long c = ((long long)blockIdx.x - job.first_block) * width + x;
    long long cols = job.cols;
    if (job.cu_end) {
        const long long held = (long long)job.cu_end[0] * job.per_row;
        cols = held < cols ? held : cols;
    }
    float v = 0.f;
    if (c < cols) {
#pragma unroll 16
        for (int r = y; r < job.rows; r += job.strands) v += job.in[r * job.cols + c];
    }
    if (job.strands > 1) {
        part[threadIdx.x] = v;
        __syncthreads();
        if (y != 0) return;
        v = 0.f;
        for (int i = 0; i < job.strands; ++i) v += part[i * width + x];
    }
    if (c >= cols) return;
    if (job.bf16) ((__nv_bfloat16*)job.out)[c] = __float2bfloat16_rn(v);
    else ((float*)job.out)[c] = v;
}

}  // namespace

void SumJobs::add(const float* in, void* out, int rows, long long cols, int bf16,
                  const int* cu_end, long long per_row)
{
    if (!out || cols == 0) return;
    const int strands = strands_for(rows, cols), per_block = NT / strands;
    job[count++] = {in, out, rows, cols, bf16, cu_end, per_row, blocks, strands};
    blocks += (cols + per_block - 1) / per_block;
}

cudaError_t launch_column_sums(const SumJobs& jobs, cudaStream_t stream)
{
    if (jobs.blocks == 0) return cudaSuccess;
    column_sums_kernel<<<(unsigned)jobs.blocks, NT, 0, stream>>>(jobs);
    count_launch();
    return cudaGetLastError();
}

cudaError_t allow_shared(const void* kernel, int bytes)
{
    // A small open-addressed set of (kernel, device); when it is full, or two
    // threads meet in it, the attribute is merely set again.
    static std::atomic<uintptr_t> done[1024];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uintptr_t key = (uintptr_t)kernel * 64 + (uintptr_t)(device & 63) + 1;
    for (int i = 0; i < 8; ++i) {
        auto& slot = done[(key * 0x9e3779b97f4a7c15ull >> 54) + i & 1023];
        uintptr_t seen = slot.load(std::memory_order_relaxed);
        if (seen == key) return cudaSuccess;
        if (seen == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e == cudaSuccess) slot.store(key, std::memory_order_relaxed);
            return e;
        }
    }
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace la
