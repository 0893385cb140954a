// Column sums of float32 matrices for gfx950: the last step of every
// parameter gradient (rows are the partial sums of the workgroups of an
// earlier kernel, written without atomics, so results do not depend on
// timing).
//
// out[m] = sum_r in[r stride + m].  A workgroup takes 64 columns: 16 lanes
// read 4 columns each (256 contiguous bytes a row), and 16 row groups take
// every 16th row, so that the few columns of a short parameter still have
// many loads in flight; the groups' sums meet in LDS in a fixed order.  Bound
// by the bytes of the partial sums.
#include "kda_block.h"
#include "kda_block_device.h"

namespace kda {
namespace {

constexpr int COLS = 64, GROUPS = 16, MAX_JOBS = 4;

struct Jobs {
    ColumnSum j[MAX_JOBS];
    unsigned first[MAX_JOBS + 1];   // first workgroup of each job
    int n;
};

__global__ void __launch_bounds__(256) column_sum_kernel(Jobs jobs)
{
    int k = 0;
    while (k + 1 < jobs.n && blockIdx.x >= jobs.first[k + 1]) ++k;
    const ColumnSum &job = jobs.j[k];
    const int g = threadIdx.x / 16, l = threadIdx.x % 16;
    const int64_t m = (int64_t)(blockIdx.x - jobs.first[k]) * COLS + 4 * l;
    const bool vec = !((job.cols | job.stride) & 3);   // whole 4-column groups, rows 16-byte aligned

    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (m < job.cols) {
        if (vec) {
#pragma unroll 4
            for (int64_t r = g; r < job.rows; r += GROUPS) {
                const float4 v = *reinterpret_cast<const float4 *>(job.in + r * job.stride + m);
                s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
            }
        } else {
            const int n = (int)(job.cols - m < 4 ? job.cols - m : 4);
#pragma unroll 2
            for (int64_t r = g; r < job.rows; r += GROUPS)
                for (int c = 0; c < n; ++c) s[c] += job.in[r * job.stride + m + c];
        }
    }
    __shared__ float part[GROUPS][COLS + 4];
#pragma unroll
    for (int c = 0; c < 4; ++c) part[g][4 * l + c] = s[c];
    __syncthreads();
    if (threadIdx.x < COLS) {
        const int64_t col = (int64_t)(blockIdx.x - jobs.first[k]) * COLS + threadIdx.x;
        if (col < job.cols) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) t += part[i][threadIdx.x];
            if (job.out_bf16) static_cast<uint16_t *>(job.out)[col] = f32_to_bf16(t);
            else static_cast<float *>(job.out)[col] = t;
        }
    }
}

}  // namespace

hipError_t launch_column_sums(const ColumnSum *jobs, int n, hipStream_t stream)
{
    Jobs a;
    a.n = 0;
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i) {
        if (!jobs[i].out || jobs[i].cols <= 0) continue;
        if (a.n == MAX_JOBS) return hipErrorInvalidValue;
        a.j[a.n] = jobs[i];
        a.first[a.n++] = (unsigned)blocks;
        blocks += (jobs[i].cols + COLS - 1) / COLS;
    }
    if (blocks == 0) return hipSuccess;
    if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    a.first[a.n] = (unsigned)blocks;
    column_sum_kernel<<<(unsigned)blocks, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kda
