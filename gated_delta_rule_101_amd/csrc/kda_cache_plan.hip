// A serving step's plan for gfx950, from the requests' lengths: rows, pages
// taken from the free list, block table entries, positions and cache slots.
//
//   need[b] = ceil((cached + added) / page) - ceil(cached / page)
//   q_start = exclusive sums of added, the pages of request b are those behind
//   the exclusive sum of need, counted from the free list's end.
//
// One launch, bound by latency: every workgroup forms the sums over all
// requests for itself (8 B bytes from L2, SPAN requests a round), so that no
// workgroup waits for another, and fills in its own 256 token rows and its own
// share of the per-request outputs.  A page's table entry is written by the
// row of its first token.  256 requests of one token 4.6 us, 2000 requests with
// 251000 tokens 11.7.
#include "kda_attn.h"
#include "kda_block.h"
#include "kda_block_device.h"

namespace kda {
namespace {

constexpr int ITEMS = 4, SPAN = 256 * ITEMS;

struct Pair {
    int64_t rows, pages;
};

// Inclusive sums over the workgroup's threads; `total` gets those of all.
__device__ __forceinline__ Pair scan256(Pair x, Pair (*wave)[4], int slot, Pair &total)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t r = __shfl_up(x.rows, d, 64), p = __shfl_up(x.pages, d, 64);
        if (lane >= d) { x.rows += r; x.pages += p; }
    }
    if (lane == 63) wave[slot][threadIdx.x / 64] = x;
    __syncthreads();
    total = {0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const Pair t = wave[slot][w];
        if (w < (int)threadIdx.x / 64) { x.rows += t.rows; x.pages += t.pages; }
        total.rows += t.rows;
        total.pages += t.pages;
    }
    return x;
}

__global__ void __launch_bounds__(256) kda_cache_plan_kernel(PlanArgs a, int shift)
{
    __shared__ Pair wave[2][4];
    __shared__ int64_t ends[SPAN];           // of the rows of a round's requests
    __shared__ int64_t first_page[SPAN];     // their first new page's place in the order of taking
    __shared__ int live[SPAN];               // served
    const int free_count = min(max(*a.free_count, 0), a.capacity);
    const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
    Pair before = {0, 0};
    int64_t taken = 0;                       // pages of served requests (of this thread's)
    bool placed = false;                     // this thread's row has a request
    int slot = 0;
    for (int b0 = 0; b0 < a.B; b0 += SPAN, slot ^= 1) {
        Pair mine[ITEMS], sum = {0, 0};
        int cached[ITEMS], added[ITEMS];
        bool ok[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int b = b0 + threadIdx.x * ITEMS + i;
            cached[i] = b < a.B ? a.cached[b] : 0;
            added[i] = b < a.B ? a.added[b] : 0;
            const int64_t c = cached[i], n = added[i], up = a.page - 1;     // a page is a power of two
            const int64_t want = (c + n + up) >> shift;
            ok[i] = c >= 0 && n >= 0 && want <= a.per;
            sum.rows += n > 0 ? n : 0;
            sum.pages += ok[i] ? want - ((c + up) >> shift) : 0;
            mine[i] = sum;
        }
        Pair total;
        const Pair upto = scan256(sum, wave, slot, total);
        const Pair base = {before.rows + upto.rows - sum.rows, before.pages + upto.pages - sum.pages};
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int at = threadIdx.x * ITEMS + i, b = b0 + at;
            const int64_t r0 = base.rows + (i ? mine[i - 1].rows : 0), p0 = base.pages + (i ? mine[i - 1].pages : 0);
            const int64_t r1 = base.rows + mine[i].rows, p1 = base.pages + mine[i].pages;
            const bool served = ok[i] && p1 <= free_count && r1 <= a.tokens;
            ends[at] = r1;
            first_page[at] = p0;
            live[at] = served;
            taken += served ? p1 - p0 : 0;
            // per-request outputs are dealt to the workgroups by rounds
            if (b < a.B && (b0 / SPAN) % gridDim.x == blockIdx.x) {
                a.q_start[b] = (int)(r0 < a.tokens ? r0 : a.tokens);
                a.context[b] = served ? cached[i] + added[i] : 0;
            }
        }
        __syncthreads();
        const int64_t r_end = before.rows + total.rows;
        if (!placed && row < a.tokens && row >= before.rows && row < r_end) {
            placed = true;
            int lo = 0, hi = min(SPAN, a.B - b0) - 1;      // the first request that ends behind this row
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (ends[mid] > row) hi = mid;
                else lo = mid + 1;
            }
            const int b = b0 + lo;
            int pos = -1, slot_of = -1;
            if (live[lo]) {
                const int c = a.cached[b];
                pos = c + (int)(row - (ends[lo] - a.added[b]));
                const int index = pos >> shift, have = (int)(((int64_t)c + a.page - 1) >> shift), in = pos & (a.page - 1);
                int *entry = a.table + (int64_t)b * a.per + index;
                int id;
                if (index >= have) {
                    id = a.free_pages[free_count - 1 - (first_page[lo] + index - have)];
                    if (in == 0) *entry = id;
                } else {
                    id = *entry;
                }
                const int64_t place = (int64_t)id * a.page + in;
                slot_of = place < 0 || place > 0x7fffffff ? -1 : (int)place;
            }
            a.positions[row] = pos;
            a.slots[row] = slot_of;
        }
        before.rows += total.rows;
        before.pages += total.pages;
        __syncthreads();
    }
    if (!placed && row < a.tokens) a.positions[row] = a.slots[row] = -1;   // rows behind the last request
    if (blockIdx.x == 0) {
        Pair total;
        scan256(Pair{taken, 0}, wave, slot, total);
        if (threadIdx.x == 0) {
            a.q_start[a.B] = (int)(before.rows < a.tokens ? before.rows : a.tokens);
            *a.free_left = free_count - (int)total.rows;
        }
    }
}

}  // namespace

hipError_t launch_cache_plan(const PlanArgs &a, hipStream_t stream)
{
    const int64_t blocks = a.tokens > 0 ? ((int64_t)a.tokens + 255) / 256 : 1;
    if (!grid_fits(blocks, 256)) return hipErrorNotSupported;
    hipLaunchKernelGGL(kda_cache_plan_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a, __builtin_ctz(a.page));
    return hipGetLastError();
}

}  // namespace kda
