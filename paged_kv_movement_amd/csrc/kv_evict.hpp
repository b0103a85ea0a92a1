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
// evict_select   one workgroup per (layer, sequence, head): the tokens' keys
//                (weights as ordered integers) once into LDS, the keep-th
//                largest by radix select (11, 11 and 10 bits, counts in LDS),
//                then each thread takes a run of slots and two sums over the
//                workgroup number the ties and the moves; weights and
//                positions go to their new slots.  A few tokens too many
//                (kFew, the steady state of decoding) are found one by one
//                instead, as the smallest key each time.
// evict_move     the K and V rows of the moves, 16 bytes a thread.  Where the
//                host's bound says that a row has at most kFusedMoves of
//                them, evict_select makes them itself.
//
// Bound: select, of latency: some twenty waits of a workgroup for loads, LDS
// counts and each other; 8.0 us for rows of 2049 with their moves, 25 for 256
// rows of up to 10000.  Move, of memory: a scattered copy of rows of head_dim
// elements, past the caches (each is read or written once: both kernels 134 us
// with the streaming policy, 147 without): 105 us for 440 MB of 256-byte rows,
// 4.2 TB/s.
#pragma once

#include "kv_order.hpp"
#include "kv_step.hpp"

namespace kvmove {

constexpr int kSelectBlock = 1024;
constexpr int kSelectWaves = kSelectBlock / 64;
constexpr int kSelectBins = 2048;
constexpr int kMoveRowsBlock = 256;
constexpr int kMoveRowsPer = 2;        // moves of a thread in flight: 139 us for what 4 or 8 move in 147
// Most moves of a row that evict_select makes itself: at most 64 of 16 rows take 14.4 us in one launch and 17.0 in two,
// 256 take 21.7 either way.
constexpr int kFusedMoves = 64;
// Tokens too many that are found one by one: one 12.0 us, two 12.2, four 16.6, where the selection takes 13.6.
constexpr int kFew = 2;

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
    uint32_t vecs;                     // 16-byte vectors of a moved row
    uint32_t vec_magic, vec_shift;     // x / vecs
    int32_t fused;
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
    for (int w = 0; w < kSelectWaves; ++w) {
        const uint32_t s = wave_sums[w];
        if (w < wave) before += s;
        total += s;
    }
    return before + v - x;
}

// Rows of a (layer, sequence, head): vectors [x, x + kMoveRowsPer * kThreads)
// by kThreads threads of the workgroup's moves (to, from).
struct RowMover {
    const EvictArgs& a;
    uint64_t kb, vb;
    int32_t s, h;

    __device__ __forceinline__ int64_t row_of(uint32_t slot) const
    {
        if (slot >= uint32_t(a.tab.max_len)) return -1;     // not from this call: see evict_move
        const uint32_t pi = page_of(a.pool, slot);
        const int32_t page = gptr<const gi32>(a.tab.table)[s * a.tab.stride + pi];
        if (uint32_t(page) >= a.pool.num_pages) {
            raise_fault_lane(kFaultPage);
            return -1;
        }
        return int64_t(page) * a.pool.page_size + (slot - pi * a.pool.page_size);
    }

    template <int kThreads, class Moves>
    __device__ __forceinline__ void run(Moves&& moves, uint32_t x0, uint32_t total) const
    {
        const uint64_t per_row = uint64_t(a.pool.heads) * a.pool.dim * 2, head = uint64_t(h) * a.vecs * 16;
        u32x4 kx[kMoveRowsPer], vx[kMoveRowsPer];
        uint64_t to[kMoveRowsPer], from[kMoveRowsPer];
#pragma unroll
        for (int u = 0; u < kMoveRowsPer; ++u) {
            const uint32_t x = x0 + u * kThreads + threadIdx.x;
            to[u] = from[u] = ~0ull;
            if (x >= total) continue;
            const uint32_t m = uint32_t((uint64_t(x) * a.vec_magic) >> a.vec_shift), v = x - m * a.vecs;
            const int64_t rt = row_of(moves(2 * m)), rf = row_of(moves(2 * m + 1));
            if (rt < 0 || rf < 0) continue;
            to[u] = rt * per_row + head + v * 16;
            from[u] = rf * per_row + head + v * 16;
        }
#pragma unroll
        for (int u = 0; u < kMoveRowsPer; ++u)
            if (from[u] != ~0ull) {
                kx[u] = __builtin_nontemporal_load(gptr<const gvec4>(kb + from[u]));
                vx[u] = __builtin_nontemporal_load(gptr<const gvec4>(vb + from[u]));
            }
#pragma unroll
        for (int u = 0; u < kMoveRowsPer; ++u)
            if (to[u] != ~0ull) {
                __builtin_nontemporal_store(kx[u], gptr<gvec4>(kb + to[u]));
                __builtin_nontemporal_store(vx[u], gptr<gvec4>(vb + to[u]));
            }
    }
};

__device__ __forceinline__ RowMover row_mover(const EvictArgs& a, int32_t job, bool& ok)
{
    const int32_t layer = a.pool.layer + job / a.heads / a.tab.n;
    const uint64_t kb = gptr<const gu64>(a.pool.k_pages)[layer], vb = gptr<const gu64>(a.pool.v_pages)[layer];
    ok = !bad_addr(kb) && !bad_addr(vb);
    if (!ok) raise_fault(kFaultPool);
    return {a, kb, vb, job / a.heads % a.tab.n, job % a.heads};
}

// kKeys: keys that fit the kernel's LDS; longer rows read weights and
// positions again wherever a key is needed.
template <int kKeys>
__global__ __launch_bounds__(kSelectBlock) void evict_select(EvictArgs a)
{
    __shared__ uint32_t keys[kKeys];
    __shared__ uint32_t bins[kSelectBins];
    __shared__ uint32_t wave_sums[kSelectWaves];
    __shared__ uint64_t wave_least[kSelectWaves];
    __shared__ int32_t found[2];
    __shared__ uint32_t few[2 * kFusedMoves];
    const int32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, job = blockIdx.x;
    const int32_t s = job / a.heads % a.tab.n;
    const gf32* w = gptr<const gf32>(a.weights) + job * a.cap;
    const gi32* p = gptr<const gi32>(a.positions) + job * a.cap;
    gf32* ow = gptr<gf32>(a.out_weights) + job * a.out_cap;
    gi32* op = gptr<gi32>(a.out_positions) + job * a.out_cap;
    const bool in_place = a.weights == a.out_weights;
    const int32_t n = table_len(a.tab, s), keep = a.keep;
    if (tid == 0 && job / a.heads < a.tab.n && job % a.heads == 0)
        gptr<gi32>(a.out_lens)[s] = n < keep ? n : keep;
    if (n <= keep || keep == 0) {              // all stay, or none
        if (!in_place && keep > 0)
            for (int32_t i = tid; i < n; i += kSelectBlock) {
                ow[i] = w[i];
                op[i] = p[i];
            }
        if (tid == 0) gptr<gu32>(a.counts)[job] = 0;
        return;
    }
    const bool in_lds = n <= kKeys;
    // the newest position; compared in 64 bits, so that no `recent` wraps around
    int32_t newest = INT32_MIN;
    for (int32_t i = tid; i < n; i += kSelectBlock) newest = p[i] > newest ? p[i] : newest;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t y = __shfl_xor(newest, d);
        newest = y > newest ? y : newest;
    }
    if (lane == 0) wave_sums[wave] = uint32_t(newest);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kSelectWaves; ++x) {
        const int32_t y = int32_t(wave_sums[x]);
        newest = y > newest ? y : newest;
    }
    const int64_t border = int64_t(newest) - a.recent;
    auto key_anew = [&](int32_t i) { return weight_key(w[i], int64_t(p[i]) > border); };
    if (in_lds)
        for (int32_t i = tid; i < n; i += kSelectBlock) keys[i] = key_anew(i);
    auto key_of = [&](int32_t i) { return in_lds ? keys[i] : key_anew(i); };
    gu32* moves = gptr<gu32>(a.moves) + int64_t(job) * a.max_moves * 2;
    uint32_t n_moves;

    if (n - keep <= kFew) {
        // the tokens that go, one by one: least key, of equal ones the last slot
        const int32_t gone_max = n - keep;
        int32_t gone[kFew];
        uint64_t above = 0;                    // what went before is below it
#pragma unroll
        for (int e = 0; e < kFew; ++e) {
            gone[e] = n;
            if (e >= gone_max) continue;
            uint64_t least = ~0ull;
            __syncthreads();
            for (int32_t i = tid; i < n; i += kSelectBlock) {
                const uint64_t x = uint64_t(key_of(i)) << 32 | uint32_t(n - 1 - i);
                if ((e == 0 || x > above) && x < least) least = x;
            }
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const uint64_t y = __shfl_xor((unsigned long long)least, d);
                least = y < least ? y : least;
            }
            if (lane == 0) wave_least[wave] = least;
            __syncthreads();
#pragma unroll
            for (int x = 0; x < kSelectWaves; ++x) least = wave_least[x] < least ? wave_least[x] : least;
            above = least;
            gone[e] = n - 1 - int32_t(uint32_t(least));
        }
        // free slots, and the kept ones behind `keep`, both ascending; the same in every thread
        n_moves = 0;
        int32_t last_to = -1, last_from = keep - 1;
#pragma unroll
        for (int e = 0; e < kFew; ++e) {
            int32_t to = n, from = n;
#pragma unroll
            for (int x = 0; x < kFew; ++x)
                if (gone[x] > last_to && gone[x] < to) to = gone[x];
            if (to >= keep) break;
            for (int32_t i = last_from + 1; i < n; ++i) {
                bool stays = true;
#pragma unroll
                for (int x = 0; x < kFew; ++x) stays = stays && gone[x] != i;
                if (stays) {
                    from = i;
                    break;
                }
            }
            if (tid == 0) {
                few[2 * e] = to;
                few[2 * e + 1] = from;
            }
            last_to = to;
            last_from = from;
            ++n_moves;
        }
        n_moves = n_moves < uint32_t(a.max_moves) ? n_moves : uint32_t(a.max_moves);
        __syncthreads();
        if (!a.fused && tid < int32_t(2 * n_moves)) moves[tid] = few[tid];
        if (!in_place)
            for (int32_t i = tid; i < keep; i += kSelectBlock) {
                uint32_t from = i;
                for (uint32_t x = 0; x < n_moves; ++x)
                    if (few[2 * x] == uint32_t(i)) from = few[2 * x + 1];
                ow[i] = w[from];
                op[i] = p[from];
            }
        else if (tid < int32_t(n_moves)) {
            ow[few[2 * tid]] = w[few[2 * tid + 1]];
            op[few[2 * tid]] = p[few[2 * tid + 1]];
        }
    } else {
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

        // a run of slots a thread (an odd number of them: its keys lie in other banks than its neighbours'); what stays,
        // and the moves by rank
        const int32_t run = ((n + kSelectBlock - 1) / kSelectBlock) | 1;
        const int32_t i0 = tid * run < n ? tid * run : n, i1 = i0 + run < n ? i0 + run : n;
        uint32_t my_ties = 0;
        for (int32_t i = i0; i < i1; ++i) my_ties += key_of(i) == border_key;
        uint32_t total;
        const uint32_t ties0 = block_scan(my_ties, wave_sums, total);
        auto stays_from = [&](int32_t i, uint32_t& ties) {
            const uint32_t key = key_of(i);
            const bool tie = key == border_key, stays = key > border_key || (tie && ties < uint32_t(want));
            ties += tie;
            return stays;
        };
        uint32_t holes = 0, sources = 0, ties = ties0;
        for (int32_t i = i0; i < i1; ++i) {
            const bool stays = stays_from(i, ties);
            holes += i < keep && !stays;
            sources += i >= keep && stays;
        }
        uint32_t to = block_scan(holes, wave_sums, n_moves), from = block_scan(sources, wave_sums, total);
        n_moves = n_moves < uint32_t(a.max_moves) ? n_moves : uint32_t(a.max_moves);
        ties = ties0;
        for (int32_t i = i0; i < i1; ++i) {
            const bool stays = stays_from(i, ties);
            if (i < keep && !stays && to < n_moves) {
                moves[2 * to++] = i;
                if (to <= kFusedMoves) few[2 * to - 2] = i;
            }
            if (i >= keep && stays && from < n_moves) {
                moves[2 * from++ + 1] = i;
                if (from <= kFusedMoves) few[2 * from - 1] = i;
            }
        }
        if (!in_place)                         // every slot; those that fall free are overwritten after the barrier
            for (int32_t i = tid; i < keep; i += kSelectBlock) {
                ow[i] = w[i];
                op[i] = p[i];
            }
        __threadfence_block();
        __syncthreads();
        for (uint32_t x = tid; x < n_moves; x += kSelectBlock) {
            const uint32_t t = moves[2 * x], f = moves[2 * x + 1];
            ow[t] = w[f];
            op[t] = p[f];
        }
    }
    if (!a.fused) {
        if (tid == 0) gptr<gu32>(a.counts)[job] = n_moves;
        return;
    }
    bool ok;
    const RowMover mover = row_mover(a, job, ok);
    const uint32_t total = n_moves * a.vecs;
    if (ok)
        for (uint32_t x = 0; x < total; x += kSelectBlock * kMoveRowsPer)
            mover.run<kSelectBlock>([&](uint32_t i) { return few[i]; }, x, total);
}

// blockIdx.x: (layer, sequence, head); blockIdx.y: a share of its moves.
__global__ __launch_bounds__(kMoveRowsBlock) void evict_move(EvictArgs a)
{
    const int32_t job = blockIdx.x;
    // counts and slots come from the caller's workspace: cut to their bounds, so that calls that wrongly share one
    // cannot send an access outside
    uint32_t n = gptr<const gu32>(a.counts)[job];
    n = n < uint32_t(a.max_moves) ? n : uint32_t(a.max_moves);
    const gu32* moves = gptr<const gu32>(a.moves) + int64_t(job) * a.max_moves * 2;
    if (n == 0) return;
    bool ok;
    const RowMover mover = row_mover(a, job, ok);
    if (!ok) return;
    const uint32_t total = n * a.vecs;
    for (uint32_t x = blockIdx.y * kMoveRowsBlock * kMoveRowsPer; x < total;
         x += gridDim.y * kMoveRowsBlock * kMoveRowsPer)
        mover.run<kMoveRowsBlock>([&](uint32_t i) { return moves[i]; }, x, total);
}

}  // namespace kvmove
