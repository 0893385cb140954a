// The line of units that the attention kernels cut into shares: its arithmetic,
// for the device and, where it can be checked without one, for the host.
//
// A unit is 64 tokens of one sequence, key head and block of query rows; the line
// has sequences, heads, blocks and tokens in that order.  Lines are shorter than
// LINE_LIMIT units: the launchers refuse longer ones (line_fits), and where row
// starts that descend count some rows many times the sums saturate, so that such a
// line is seen to be too long and nothing of it is done.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// A sequence of the call: its first query row, queries and tokens in the cache,
// held inside the buffers whatever the device's numbers say.
struct Sequence {
    int first, queries, context;
};
// from, to: its row starts; room: tokens of its row of the table.
__host__ __device__ inline Sequence sequence_of(int from, int to, int tokens, int context, int64_t room)
{
    const auto clamp = [&](int x, int low) { return x < low ? low : x > tokens ? tokens : x; };
    const int first = clamp(from, 0), c = context > 0 ? context : 0;
    return Sequence{first, clamp(to, first) - first, c < room ? c : (int)room};
}
__host__ __device__ inline int tiles_of(const Sequence &s)       // contexts are below 2^31 - 256
{
    const int n = (s.context + 63) / 64;
    return n > 1 ? n : 1;
}
__host__ __device__ inline int blocks_of(const Sequence &s, int G, int rows)
{
    return (int)(((unsigned)s.queries * G + rows - 1) / rows);   // below 2^31 rows, and rows a power of two
}

constexpr unsigned LINE_LIMIT = 0x7fffffff;
// A sum of units, no more than the largest number.
__host__ __device__ inline unsigned units_add(unsigned a, unsigned b) { return a + b < a ? ~0u : a + b; }
// Units a share of a line of `units` (not none) in `rows` rows: `at_least` as many
// where rows are that long, as short rows stay whole.
__host__ __device__ inline int share_of(unsigned units, unsigned rows, unsigned workgroups, unsigned at_least)
{
    const unsigned even = (units + workgroups - 1) / workgroups, row = (units + rows - 1) / rows;
    const unsigned least = row < at_least ? row : at_least;
    return (int)(even > least ? even : least);
}
// The workgroup whose share has the last unit of a row of `tiles` that begins at place `at`.
__host__ __device__ inline int last_share(unsigned at, unsigned tiles, unsigned share) { return (int)((at + tiles - 1) / share); }

// A product of sizes, no more than the largest number.
inline int64_t times(int64_t a, int64_t b)
{
    int64_t x;
    return __builtin_mul_overflow(a, b, &x) ? INT64_MAX : x;
}
// Whether a line of blocks of `block` query rows is short enough, where row starts do
// not descend: a sequence adds less than one block to those of all rows.
inline bool line_fits(int64_t tiles, int64_t rows, int block, int B, int Hk)
{
    return times(times(tiles > 0 ? tiles : 1, Hk), rows / block + B) < (int64_t)LINE_LIMIT - 65535;
}
// Workgroups for a line of at most `units` units, of which the device holds `most` at once.
inline int shares(int64_t units, int most) { return units < most && units > 0 ? (int)units : most; }

}  // namespace kda
