// kv_evict.hpp -- eviction by accumulated attention weight: of a sequence's n
// cached tokens, `keep` stay -- the `recent` newest ones and, of the others,
// those with the largest weights.
//
// The kept tokens have to end up in the first `keep` slots.  Attention does
// not care about the order of the slots (a key carries its position), so a
// kept token that already is in one of them stays where it is, and only the
// kept ones behind them move, into the slots that fall free: the k-th of
// them to the k-th free slot, both ascending.  That is the least that has to
// be moved, and since no slot is both read and written, all moves run at
// once and in place.
//
// evict_select   one workgroup per (layer, sequence, head): the keep-th
//                largest key by radix select (11, 11 and 10 bits, counts in
//                LDS), then the list of moves by running counts over the
//                slots; weights and positions go to their new slots;
// evict_move     the K and V rows of the moves, 16 bytes a thread.
//
// Bound: select reads 8 bytes a token (the weights again, from L2, for each
// digit) and waits on LDS counts; move is a scattered copy of rows.
#pragma once

#include "kv_order.hpp"
#include "kv_step.hpp"

namespace kvmove {

constexpr int kSelectBlock = 1024;
constexpr int kSelectBins = 2048;
constexpr int kMoveRowsBlock = 256;
constexpr int kMoveRowsPer = 4;        // moves of a thread in flight

struct EvictArgs {
    PoolArg pool;                      // layer: first layer
    TablesArg tab;
    uint64_t weights, positions;       // float32 / int32 [n_layers][n][heads][cap]
    uint64_t out_weights, out_positions;   // [n_layers][n][heads][out_cap]
    int64_t cap, out_cap;
    uint64_t out_lens;                 // int32[n]
    uint64_t counts;                   // uint32 per (layer, sequence, head): moves
    uint64_t moves;                    // uint32 pairs (to, from), max_moves per (layer, sequence, head)
    int32_t heads;                     // KV heads, or 1: all heads of a token stay or go together
    int32_t n_layers;
    int32_t keep, recent;
    int32_t max_moves;
};

// Order of the weights as unsigned integers: larger key, larger weight; -0 as
// 0, a NaN below all, a protected token above all.
__device__ __forceinline__ uint32_t weight_key(float w, bool protect)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);
    uint32_t k = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) k = 0;
    return protect ? 0xFFFFFFFFu : k;
}

// Sum of x over the workgroup's threads below this one, and over all of them.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* wave_sums, uint32_t& total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t v = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t y = __shfl_up(v, d);
        if (lane >= d) v += y;
    }
    __syncthreads();
    if (lane == 63) wave_sums[wave] = v;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSelectBlock / 64; ++w) {
        const uint32_t s = wave_sums[w];
        if (w < wave) before += s;
        total += s;
    }
    return before + v - x;
}

__global__ __launch_bounds__(kSelectBlock) void evict_select(EvictArgs a)
{
    __shared__ uint32_t bins[kSelectBins];
    __shared__ uint32_t wave_sums[kSelectBlock / 64];
    __shared__ int32_t found[2];
    const int32_t tid = threadIdx.x, job = blockIdx.x;
    const int32_t s = job / a.heads % a.tab.n;
    const int32_t n = table_len(a.tab, s), keep = a.keep;
    const gf32* w = gptr<const gf32>(a.weights) + job * a.cap;
    const gi32* p = gptr<const gi32>(a.positions) + job * a.cap;
    gf32* ow = gptr<gf32>(a.out_weights) + job * a.out_cap;
    gi32* op = gptr<gi32>(a.out_positions) + job * a.out_cap;
    const bool in_place = a.weights == a.out_weights;
    if (tid == 0 && job / a.heads < a.tab.n && job % a.heads == 0)
        gptr<gi32>(a.out_lens)[s] = n < keep ? n : keep;
    if (n <= keep) {
        if (!in_place)
            for (int32_t i = tid; i < n; i += kSelectBlock) {
                ow[i] = w[i];
                op[i] = p[i];
            }
        if (tid == 0) gptr<gu32>(a.counts)[job] = 0;
        return;
    }
    // the newest position; 64-bit so that no `recent` wraps around
    int32_t newest = INT32_MIN;
    for (int32_t i = tid; i < n; i += kSelectBlock) newest = p[i] > newest ? p[i] : newest;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t y = __shfl_xor(newest, d);
        newest = y > newest ? y : newest;
    }
    if ((tid & 63) == 0) wave_sums[tid >> 6] = uint32_t(newest);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kSelectBlock / 64; ++x) {
        const int32_t y = int32_t(wave_sums[x]);
        newest = y > newest ? y : newest;
    }
    const int64_t border = int64_t(newest) - a.recent;
    auto key_of = [&](int32_t i) { return weight_key(w[i], int64_t(p[i]) > border); };

    // the keep-th largest key: top 11 bits, then 11, then 10
    uint32_t prefix = 0, mask = 0;
    int32_t want = keep;                   // rank, from the largest, within what matches the prefix
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        __syncthreads();
        for (int32_t x = tid; x < kSelectBins; x += kSelectBlock) bins[x] = 0;
        __syncthreads();
        for (int32_t i = tid; i < n; i += kSelectBlock) {
            const uint32_t key = key_of(i);
            if ((key & mask) == prefix) atomicAdd(&bins[(key >> shift) & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        // thread x holds bins from the top: 2047 - 2x and 2046 - 2x
        const uint32_t c0 = bins[kSelectBins - 1 - 2 * tid], c1 = bins[kSelectBins - 2 - 2 * tid];
        uint32_t total;
        const uint32_t before = block_scan(c0 + c1, wave_sums, total);
        if (before < uint32_t(want) && uint32_t(want) <= before + c0) {
            found[0] = kSelectBins - 1 - 2 * tid;
            found[1] = want - before;
        } else if (before + c0 < uint32_t(want) && uint32_t(want) <= before + c0 + c1) {
            found[0] = kSelectBins - 2 - 2 * tid;
            found[1] = want - before - c0;
        }
        __syncthreads();
        prefix |= uint32_t(found[0]) << shift;
        mask |= ((1u << bits) - 1) << shift;
        want = found[1];
    }
    const uint32_t border_key = prefix;    // `want` of the tokens with this very key stay, the first ones

    // slots in order: what stays, and the moves
    gu32* moves = gptr<gu32>(a.moves) + int64_t(job) * a.max_moves * 2;
    uint32_t ties = 0, holes = 0, sources = 0;
    for (int32_t i0 = 0; i0 < n; i0 += kSelectBlock) {
        const int32_t i = i0 + tid;
        const uint32_t key = i < n ? key_of(i) : 0;
        const bool tie = i < n && key == border_key;
        uint32_t n_tie, n_both;
        const uint32_t tie_rank = ties + block_scan(tie, wave_sums, n_tie);
        const bool stays = i < n && (key > border_key || (tie && tie_rank < uint32_t(want)));
        const bool hole = i < keep && !stays, source = i >= keep && stays;
        // both counts in one scan: at most 1024 each
        const uint32_t rank = block_scan(uint32_t(hole) | uint32_t(source) << 16, wave_sums, n_both);
        const uint32_t to = holes + (rank & 0xFFFFu), from = sources + (rank >> 16);
        if (hole && to < uint32_t(a.max_moves)) moves[2 * to] = i;
        if (source && from < uint32_t(a.max_moves)) moves[2 * from + 1] = i;
        if (!in_place && i < keep && stays) {
            ow[i] = w[i];
            op[i] = p[i];
        }
        ties += n_tie;
        holes += n_both & 0xFFFFu;
        sources += n_both >> 16;
    }
    __threadfence_block();
    __syncthreads();
    holes = holes < uint32_t(a.max_moves) ? holes : uint32_t(a.max_moves);
    for (uint32_t x = tid; x < holes; x += kSelectBlock) {
        const uint32_t to = moves[2 * x], from = moves[2 * x + 1];
        ow[to] = w[from];
        op[to] = p[from];
    }
    if (tid == 0) gptr<gu32>(a.counts)[job] = holes;
}

// blockIdx.x: (layer, sequence, head); blockIdx.y: a share of its moves.
__global__ __launch_bounds__(kMoveRowsBlock) void evict_move(EvictArgs a)
{
    const int32_t job = blockIdx.x;
    // counts and slots come from the caller's workspace: cut to their bounds, so that calls that wrongly share one
    // cannot send an access outside
    uint32_t n = gptr<const gu32>(a.counts)[job];
    n = n < uint32_t(a.max_moves) ? n : uint32_t(a.max_moves);
    const int32_t h = job % a.heads, s = job / a.heads % a.tab.n, layer = a.pool.layer + job / a.heads / a.tab.n;
    const uint32_t width = a.pool.heads * a.pool.dim / a.heads;        // elements of a move
    const uint32_t vecs = width / 8;
    const uint64_t kb = gptr<const gu64>(a.pool.k_pages)[layer], vb = gptr<const gu64>(a.pool.v_pages)[layer];
    const gu32* moves = gptr<const gu32>(a.moves) + int64_t(job) * a.max_moves * 2;
    if (n == 0) return;
    if (bad_addr(kb) || bad_addr(vb)) {
        raise_fault(kFaultPool);
        return;
    }
    const uint64_t per_row = uint64_t(a.pool.heads) * a.pool.dim * 2;
    const uint64_t total = uint64_t(n) * vecs;
    auto row_of = [&](uint32_t slot) -> int64_t {
        if (slot >= uint32_t(a.tab.max_len)) return -1;
        const uint32_t pi = page_of(a.pool, slot);
        const int32_t page = gptr<const gi32>(a.tab.table)[s * a.tab.stride + pi];
        if (page < 0 || uint32_t(page) >= a.pool.num_pages) {
            raise_fault_lane(kFaultPage);
            return -1;
        }
        return int64_t(page) * a.pool.page_size + (slot - pi * a.pool.page_size);
    };
    for (uint64_t x0 = uint64_t(blockIdx.y) * kMoveRowsBlock * kMoveRowsPer; x0 < total;
         x0 += uint64_t(gridDim.y) * kMoveRowsBlock * kMoveRowsPer) {
        u32x4 kx[kMoveRowsPer], vx[kMoveRowsPer];
        uint64_t to[kMoveRowsPer];
#pragma unroll
        for (int u = 0; u < kMoveRowsPer; ++u) {
            const uint64_t x = x0 + u * kMoveRowsBlock + threadIdx.x;
            to[u] = ~0ull;
            if (x >= total) continue;
            const uint32_t m = uint32_t(x / vecs), v = uint32_t(x - uint64_t(m) * vecs);
            const int64_t rt = row_of(moves[2 * m]), rf = row_of(moves[2 * m + 1]);
            if (rt < 0 || rf < 0) continue;
            const uint64_t in_row = (uint64_t(h) * width + v * 8) * 2;
            to[u] = rt * per_row + in_row;
            kx[u] = *gptr<const gvec4>(kb + rf * per_row + in_row);
            vx[u] = *gptr<const gvec4>(vb + rf * per_row + in_row);
        }
#pragma unroll
        for (int u = 0; u < kMoveRowsPer; ++u)
            if (to[u] != ~0ull) {
                *gptr<gvec4>(kb + to[u]) = kx[u];
                *gptr<gvec4>(vb + to[u]) = vx[u];
            }
    }
}

}  // namespace kvmove
