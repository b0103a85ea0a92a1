// kv_step.hpp -- what the kernels of a model step share (append, attend,
// weights, evict): the layer's pool, block tables with their lengths on the
// device, and the new tokens' rows.
//
// Lengths, row ranges and groups are read from device memory, so a captured
// graph follows them; every value read is cut to the bound that the host
// gave, which sizes the grids and the workspaces, and no access depends on
// the device values alone.  A page id outside the pool makes its tokens
// invisible (or unwritten) and sets a fault bit.
#pragma once

#include "kv_common.hpp"

namespace kvmove {

using f32x4 = __attribute__((ext_vector_type(4))) float;
using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using gf32x4 = __attribute__((address_space(1))) f32x4;

struct PoolArg {
    uint64_t k_pages;        // uint64[L]: layer K pool addresses
    uint64_t v_pages;
    uint32_t num_pages;
    uint32_t page_size;
    uint32_t page_magic;     // t / page_size = (t * page_magic) >> page_shift for t < 2^31
    uint32_t page_shift;
    uint32_t heads;          // KV heads
    uint32_t dim;            // elements of a head
    int32_t layer;
};

struct TablesArg {
    uint64_t table;          // int32[n][stride]: page ids
    uint64_t lens;           // int32[n]: tokens cached
    int64_t stride;
    int32_t n;
    int32_t max_len;         // lens beyond it are cut to it
};

struct StepArg {
    TablesArg own;
    TablesArg prefix;
    uint64_t q_start;        // int32[own.n + 1]: first new-token row of each sequence
    uint64_t group_start;    // int32[prefix.n + 1]: first sequence of each group
    int32_t n_rows;
    int32_t max_new;         // rows of one sequence beyond it are not taken
    int32_t max_group_rows;  // rows of one group beyond it are not taken
};

struct Rows {
    int32_t first, count;
};

__device__ __forceinline__ int32_t clamp_i32(int32_t x, int32_t lo, int32_t hi)
{
    return x < lo ? lo : x > hi ? hi : x;
}

__device__ __forceinline__ int32_t table_len(const TablesArg& t, int32_t i)
{
    return clamp_i32(gptr<const gi32>(t.lens)[i], 0, t.max_len);
}

__device__ __forceinline__ Rows seq_rows(const StepArg& a, int32_t s)
{
    const int32_t b = clamp_i32(gptr<const gi32>(a.q_start)[s], 0, a.n_rows);
    const int32_t e = clamp_i32(gptr<const gi32>(a.q_start)[s + 1], b, a.n_rows);
    return {b, e - b < a.max_new ? e - b : a.max_new};
}

__device__ __forceinline__ Rows group_rows(const StepArg& a, int32_t g)
{
    const int32_t s0 = clamp_i32(gptr<const gi32>(a.group_start)[g], 0, a.own.n);
    const int32_t s1 = clamp_i32(gptr<const gi32>(a.group_start)[g + 1], s0, a.own.n);
    const int32_t b = clamp_i32(gptr<const gi32>(a.q_start)[s0], 0, a.n_rows);
    const int32_t e = clamp_i32(gptr<const gi32>(a.q_start)[s1], b, a.n_rows);
    return {b, e - b < a.max_group_rows ? e - b : a.max_group_rows};
}

__device__ __forceinline__ uint32_t page_of(const PoolArg& p, uint32_t t)
{
    return uint32_t((uint64_t(t) * p.page_magic) >> p.page_shift);
}

// First of the 64 neighbouring ranges [starts[i], starts[i + 1]), i < n, one of
// which holds x if any does.  Every round of loads leaves a 64th of them: none
// for up to 64 ranges, one for up to 4096.
__device__ __forceinline__ int32_t ranges_around(uint64_t starts, int32_t n, int32_t x)
{
    const int32_t lane = threadIdx.x & 63;
    int32_t lo = 0, span = n;
    while (span > 64) {
        const int32_t step = (span + 63) / 64, i = lane * step;
        const int32_t b = gptr<const gi32>(starts)[lo + (i < span ? i : 0)];
        const uint64_t m = __ballot(i < span && b <= x);
        if (m == 0) break;
        const int32_t at = (63 - __builtin_clzll(m)) * step;
        lo += at;
        span = span - at < step ? span - at : step;
    }
    return lo;
}

// The sequence that new-token row r belongs to, from one round of loads after
// ranges_around (lane i holds the i-th; the row's own is taken from the lane
// that holds it).  s < 0: none.
struct RowOwner {
    int32_t s, first, count, len;
};

__device__ __forceinline__ RowOwner row_owner(const StepArg& a, int32_t r)
{
    const int32_t i0 = ranges_around(a.q_start, a.own.n, r), i = i0 + int32_t(threadIdx.x & 63);
    int32_t b = 0, e = 0, n = 0;
    if (i < a.own.n) {
        b = gptr<const gi32>(a.q_start)[i];
        e = gptr<const gi32>(a.q_start)[i + 1];
        n = table_len(a.own, i);
    }
    const uint64_t m = __ballot(b <= r && r < e);
    if (m == 0) return {-1, 0, 0, 0};
    const int j = __builtin_ctzll(m);
    RowOwner o;
    o.s = i0 + j;
    o.first = clamp_i32(__builtin_amdgcn_readlane(b, j), 0, a.n_rows);
    o.count = clamp_i32(__builtin_amdgcn_readlane(e, j), o.first, a.n_rows) - o.first;
    o.count = o.count < a.max_new ? o.count : a.max_new;
    o.len = __builtin_amdgcn_readlane(n, j);
    if (r - o.first >= o.count) o.s = -1;
    return o;
}

__device__ __forceinline__ void raise_fault_lane(unsigned bit) { atomicOr(&g_kv_faults, bit); }

}  // namespace kvmove
