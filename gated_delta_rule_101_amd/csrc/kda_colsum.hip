// Column sums of float32 matrices for gfx950: the last step of every
// parameter gradient (rows are the partial sums of the workgroups of an
// earlier kernel, written without atomics, so results do not depend on
// timing).
//
// out[m] = sum_r in[r stride + m].  A workgroup takes 4 L columns: L lanes read 4
// columns each and 256 / L row groups take every (256 / L)th row, so that few
// columns still have many loads in flight; the groups' sums meet in LDS in a
// fixed order.  L is 16 (256 contiguous bytes a row), or 4 where that leaves
// under 64 workgroups.  Where columns are many (the rows of B and C), a thread
// takes 4 columns and all their rows instead.  Where rows are many and
// workgroups few (a parameter of few channels), a first launch sums chunks of
// CHUNK rows, each into its own first row, and the second those rows: at 4096
// rows of 68 columns one launch took 170 us, a chain of 256 loads a thread.
// Bound by the bytes of the partial sums.
#include "kda_block.h"
#include "kda_block_device.h"

namespace kda {
namespace {

constexpr int MAX_JOBS = 5, CHUNK = 64;
constexpr int SERIAL = 256;   // L of jobs whose threads walk all rows

struct Jobs {
    ColumnSum j[MAX_JOBS];
    unsigned first[MAX_JOBS + 1];   // first workgroup of each job
    int lanes[MAX_JOBS];            // L
    int n;
};

__device__ __forceinline__ void put(const ColumnSum &job, int64_t col, float v)
{
    if (job.out_bf16) static_cast<uint16_t *>(job.out)[col] = f32_to_bf16(v);
    else static_cast<float *>(job.out)[col] = v;
}

// CHUNKS: workgroups of one column block take CHUNK rows each and write their
// sum over the chunk's first row, which no other workgroup reads.
template <bool CHUNKS>
__global__ void __launch_bounds__(256) column_sum_kernel(Jobs jobs)
{
    int k = 0;
    while (k + 1 < jobs.n && blockIdx.x >= jobs.first[k + 1]) ++k;
    const ColumnSum &job = jobs.j[k];
    const bool vec = !((job.cols | job.stride) & 3);   // whole 4-column groups, rows 16-byte aligned
    const int L = jobs.lanes[k], cols = 4 * L, groups = 256 / L;
    if (L == SERIAL) {
        const int64_t m = (int64_t)(blockIdx.x - jobs.first[k]) * cols + 4 * threadIdx.x;
        if (m >= job.cols) return;
        const int n = (int)(job.cols - m < 4 ? job.cols - m : 4);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        if (vec) {
#pragma unroll 8
            for (int64_t r = 0; r < job.rows; ++r) {
                const float4 v = *reinterpret_cast<const float4 *>(job.in + r * job.stride + m);
                s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
            }
        } else {
            for (int64_t r = 0; r < job.rows; ++r)
                for (int c = 0; c < n; ++c) s[c] += job.in[r * job.stride + m + c];
        }
        for (int c = 0; c < n; ++c) put(job, m + c, s[c]);
        return;
    }
    const int g = threadIdx.x / L, l = threadIdx.x % L;
    const unsigned blocks = (unsigned)((job.cols + cols - 1) / cols), id = blockIdx.x - jobs.first[k];
    const int64_t m0 = (int64_t)(id % blocks) * cols, m = m0 + 4 * l;
    const int64_t r0 = CHUNKS ? (int64_t)(id / blocks) * CHUNK : 0;
    const int64_t r1 = CHUNKS && r0 + CHUNK < job.rows ? r0 + CHUNK : job.rows;

    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (m < job.cols) {
        if (vec) {
#pragma unroll 4
            for (int64_t r = r0 + g; r < r1; r += groups) {
                const float4 v = *reinterpret_cast<const float4 *>(job.in + r * job.stride + m);
                s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
            }
        } else {
            const int n = (int)(job.cols - m < 4 ? job.cols - m : 4);
#pragma unroll 2
            for (int64_t r = r0 + g; r < r1; r += groups)
                for (int c = 0; c < n; ++c) s[c] += job.in[r * job.stride + m + c];
        }
    }
    __shared__ float part[256 * 5];   // [groups][cols + 4]
#pragma unroll
    for (int c = 0; c < 4; ++c) part[g * (cols + 4) + 4 * l + c] = s[c];
    __syncthreads();
    const int64_t col = m0 + threadIdx.x;
    if (threadIdx.x < cols && col < job.cols) {
        float t = 0.f;
#pragma unroll 8
        for (int i = 0; i < groups; ++i) t += part[i * (cols + 4) + threadIdx.x];
        if (CHUNKS) job.in[r0 * job.stride + col] = t;
        else put(job, col, t);
    }
}

template <bool CHUNKS> hipError_t run(const Jobs &jobs, int64_t blocks, hipStream_t stream)
{
    if (blocks == 0) return hipSuccess;
    column_sum_kernel<CHUNKS><<<(unsigned)blocks, 256, 0, stream>>>(jobs);
    return hipGetLastError();
}

// The jobs of both launches and their workgroups; false: too many to launch.
struct Plan {
    Jobs jobs, chunks;
    int64_t blocks, chunk_blocks;
};
bool plan(const ColumnSum *list, int n, Plan &p)
{
    Jobs &jobs = p.jobs, &chunks = p.chunks;
    jobs.n = chunks.n = 0;
    p.blocks = p.chunk_blocks = 0;
    for (int i = 0; i < n; ++i) {
        ColumnSum job = list[i];
        if (!job.out || job.cols <= 0) continue;
        if (jobs.n == MAX_JOBS) return false;
        const auto blocks_of = [&](int lanes) { return (job.cols + 4 * lanes - 1) / (4 * lanes); };
        const int lanes = blocks_of(16) < 64 ? 4 : blocks_of(16) >= 2048 && job.rows <= 1024 ? SERIAL : 16;
        const int64_t wide = blocks_of(lanes);
        if (job.rows > 16 * CHUNK && wide < 256) {
            chunks.j[chunks.n] = job;
            chunks.lanes[chunks.n] = lanes;
            chunks.first[chunks.n++] = (unsigned)p.chunk_blocks;
            job.rows = (job.rows + CHUNK - 1) / CHUNK;
            p.chunk_blocks += wide * job.rows;
            job.stride *= CHUNK;
        }
        jobs.j[jobs.n] = job;
        jobs.lanes[jobs.n] = lanes;
        jobs.first[jobs.n++] = (unsigned)p.blocks;
        p.blocks += wide;
    }
    return grid_fits(p.blocks, 256) && grid_fits(p.chunk_blocks, 256);
}

}  // namespace

bool column_sums_fit(const ColumnSum *list, int n)
{
    Plan p;
    return plan(list, n, p);
}

hipError_t launch_column_sums(const ColumnSum *list, int n, hipStream_t stream)
{
    Plan p;
    if (!plan(list, n, p)) return hipErrorNotSupported;
    const hipError_t e = run<true>(p.chunks, p.chunk_blocks, stream);
    return e != hipSuccess ? e : run<false>(p.jobs, p.blocks, stream);
}

}  // namespace kda
