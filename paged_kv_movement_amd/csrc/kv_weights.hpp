// kv_weights.hpp -- the attention weight of every cached token, added to its
// running sum (what an eviction ranks the tokens by).
//
//   out[t] = in[t] + sum over the rows that see t, and over the query heads
//            of the KV head, of exp(scale q.k_t - lse[row])
//
// with the lse of a finished attention, so no maximum is searched.  A wave
// keeps its tokens' K in registers as the left operand of S^T = K Q^T and
// walks the rows, 16 at a time, the next ones' q already on its way: K is
// read once whatever the number of rows.  With few rows the four waves of a
// workgroup take different tokens; with many rows they take the same tokens
// and every fourth block of rows (kSplitRows), and their sums meet in LDS.
// Each token's sum has one owner and one order, so the same call gives the
// same bits.
//
// Bound: for single tokens the read of K, half of what the attention reads;
// for prompts one exponential (a quarter-rate instruction), one fused product
// and one sum per (row, token): 24 cycles a wave for 64 of them beside 16 of
// matrix products.
#pragma once

#include "kv_attend.hpp"

namespace kvmove {

struct WeightsArgs {
    PoolArg pool;
    StepArg step;
    uint64_t q, lse;               // bf16 rows with strides, float32 [n_rows][q_heads]
    int64_t q_row, q_head;
    int32_t q_heads, rep;
    uint32_t rep_magic, rep_shift;
    float scale_log2;
    uint64_t own_in, own_out;      // float32 [own.n][heads][own_cap]; in may be 0 (zeros) or out
    uint64_t prefix_in, prefix_out;// float32 [prefix.n][heads][prefix_cap]
    int64_t own_cap, prefix_cap;
    int32_t own_blocks, prefix_blocks;      // workgroups for the tokens of a row of the tables
    uint32_t prefix_items;
};

// Tiles of 16 tokens a wave holds: four where many rows pass by, so that a
// row's q serves more products; two otherwise, for more waves in flight.
template <int DP, bool kSplitRows>
constexpr int kWeightsTiles = DP <= 128 && kSplitRows ? 4 : 2;

template <int DP, bool kSplitRows>
constexpr int kWeightsTokens = 16 * kWeightsTiles<DP, kSplitRows> * (kSplitRows ? 1 : kAttendWaves);   // of a workgroup

struct WeightsPiece {
    uint64_t kh;                   // this KV head's K pool
    uint64_t in, out;              // sums of (table row, KV head)
    const TablesArg& tab;
    int32_t table_row, h, len, first_row, count;
    bool prefix;
};

// Column r of a block of 16 rows.
template <int DP>
struct WeightsColumn {
    u32x4 q[DP / 32];
    float lse;
    int32_t vis;
    bool live;
};

// No load stands behind a branch, so that the compiler counts which of them a
// wait is for: columns past the last row read it again and add nothing.
template <int DP>
__device__ __forceinline__ void load_column(const WeightsArgs& a, const WeightsPiece& w, int32_t x,
                                            WeightsColumn<DP>& c)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, dim = a.pool.dim;
    const int32_t n = w.count * a.rep, f = x * 16 + r < n ? x * 16 + r : n - 1;
    const int32_t i = new_token(a, f), head = w.h * a.rep + (f - i * a.rep);
    const int64_t qr = w.first_row + i;
    c.vis = w.prefix ? w.len : clamp_i32(w.len - w.count + i + 1, 0, w.len);
    c.live = x * 16 + r < n;
    c.lse = gptr<const gf32>(a.lse)[qr * a.q_heads + head];
    load_row<DP>(c.q, a.q + (qr * a.q_row + head * a.q_head) * 2, g, dim);
}

// Adds the weights of row block x for the wave's tokens from t.
template <int DP, int NT>
__device__ __forceinline__ void add_block(const WeightsArgs& a, const WeightsPiece& w, int32_t x, int32_t t,
                                          const u32x4 (&k)[NT][DP / 32], WeightsColumn<DP>& c,
                                          f32x4 (&sum)[NT])
{
    const int g = (threadIdx.x & 63) >> 4;
    if (int(a.pool.dim) < DP) clear_past<DP>(c.q, g, a.pool.dim);
    f32x4 s[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        s[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) s[i] = mfma16(k[i][j], c.q[j], s[i]);
    }
    // minus lse in log2 units; a row that saw nothing adds nothing: exp2(-infinity)
    const float neg = !c.live || c.lse == -__builtin_inff() ? -__builtin_inff() : -c.lse * kLog2e;
    // the block's first row sees the least
    if (!w.prefix && w.len - w.count + new_token(a, x * 16) + 1 < t + 16 * NT) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n], a.scale_log2, neg));
                sum[i][n] += t + 16 * i + 4 * g + n < c.vis ? p : 0.0f;
            }
    } else {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                sum[i][n] += __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n], a.scale_log2, neg));
    }
}

// The tokens' K, from the rows that lane y holds for token y; of row 0 where
// there is none (what comes of it is not used).
template <int DP, int NT>
__device__ __forceinline__ void load_keys(const WeightsArgs& a, const WeightsPiece& w, int32_t row,
                                          u32x4 (&k)[NT][DP / 32])
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, dim = a.pool.dim;
    const uint32_t row_bytes = a.pool.heads * dim * 2;
    row = row < 0 ? 0 : row;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const uint32_t kr = uint32_t(__shfl(row, 16 * i + r));
        load_row<DP>(k[i], w.kh + uint64_t(kr) * row_bytes, g, dim);
    }
    if (dim < DP)
#pragma unroll
        for (int i = 0; i < NT; ++i) clear_past<DP>(k[i], g, dim);
}

// The sums over the 16 columns, token y's to part[y].
template <int NT>
__device__ __forceinline__ void fold_columns(const f32x4 (&sum)[NT], float* part)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float v = sum[i][n];
            v += __shfl_xor(v, 1);
            v += __shfl_xor(v, 2);
            v += __shfl_xor(v, 4);
            v += __shfl_xor(v, 8);
            if (r == 0) part[16 * i + 4 * g + n] = v;
        }
}

// Many rows: the four waves hold the same tokens [t, t + 16 NT) and take every
// fourth block of rows, the q of the next two on their way.
template <int DP>
__device__ __forceinline__ void weights_by_rows(const WeightsArgs& a, const WeightsPiece& w, int32_t t, bool pool_ok,
                                                float (&part)[kAttendWaves][64])
{
    constexpr int NT = kWeightsTiles<DP, true>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool here = pool_ok && lane < 16 * NT && lane < w.len - t;
    const int32_t row = here ? token_row(a.pool, w.tab, w.table_row, t + lane) : -1;
    u32x4 k[NT][DP / 32];
    if (pool_ok) load_keys<DP, NT>(a, w, row, k);
    f32x4 sum[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) sum[i] = f32x4{0, 0, 0, 0};
    // token t is first seen by new token t - (len - count): blocks of rows before it see none of these tokens
    const int32_t before = w.prefix ? 0 : t - (w.len - w.count);
    const int32_t n_blocks = (w.count * a.rep + 15) / 16;
    int32_t x = (before > 0 ? before * a.rep / 16 : 0) + wave;
    WeightsColumn<DP> c0, c1, c2;
    if (!pool_ok) x = n_blocks;
    if (x < n_blocks) {
        load_column<DP>(a, w, x, c0);
        load_column<DP>(a, w, x + kAttendWaves, c1);
    }
    // three columns by name: to move one on would wait for its loads
#pragma unroll 1
    while (x < n_blocks) {
        load_column<DP>(a, w, x + 2 * kAttendWaves, c2);
        add_block<DP, NT>(a, w, x, t, k, c0, sum);
        if ((x += kAttendWaves) >= n_blocks) break;
        load_column<DP>(a, w, x + 2 * kAttendWaves, c0);
        add_block<DP, NT>(a, w, x, t, k, c1, sum);
        if ((x += kAttendWaves) >= n_blocks) break;
        load_column<DP>(a, w, x + 2 * kAttendWaves, c1);
        add_block<DP, NT>(a, w, x, t, k, c2, sum);
        x += kAttendWaves;
    }
    fold_columns<NT>(sum, part[wave]);
    __syncthreads();
    if (wave == 0 && lane < 16 * NT && lane < w.len - t) {
        float v = part[0][lane];
#pragma unroll
        for (int y = 1; y < kAttendWaves; ++y) v += part[y][lane];
        const float old = w.in != 0 ? gptr<const gf32>(w.in)[t + lane] : 0.0f;
        gptr<gf32>(w.out)[t + lane] = old + (row >= 0 ? v : 0.0f);
    }
}

// Few rows: each wave has its own tokens [t, t + 16 NT), one group of them:
// many short waves hide their three rounds of loads (lengths and pages; K and
// q; the sums out) behind each other, which measured better than fewer waves
// that walk through the tokens with the next K on its way (30 us against 36
// to 46 for 32 sequences behind an 8192-token prefix).
template <int DP>
__device__ __forceinline__ void weights_by_tokens(const WeightsArgs& a, const WeightsPiece& w, int32_t t, int32_t page,
                                                  float old, bool pool_ok, float (&part)[kAttendWaves][64])
{
    constexpr int NT = kWeightsTiles<DP, false>, T = 16 * NT;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool here = pool_ok && lane < T && lane < w.len - t;
    const int32_t row = here ? row_in_page(a.pool, page, t + lane) : -1;
    const int32_t n_blocks = pool_ok ? (w.count * a.rep + 15) / 16 : 0;
    u32x4 k[NT][DP / 32];
    WeightsColumn<DP> c0, c1;
    if (n_blocks > 0) {
        load_keys<DP, NT>(a, w, row, k);
        load_column<DP>(a, w, 0, c0);
    }
    f32x4 sum[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) sum[i] = f32x4{0, 0, 0, 0};
    // two columns by name: to move one on would wait for its loads
#pragma unroll 1
    for (int32_t x = 0; x < n_blocks; x += 2) {
        load_column<DP>(a, w, x + 1, c1);
        add_block<DP, NT>(a, w, x, t, k, c0, sum);
        if (x + 1 >= n_blocks) break;
        load_column<DP>(a, w, x + 2, c0);
        add_block<DP, NT>(a, w, x + 1, t, k, c1, sum);
    }
    fold_columns<NT>(sum, part[wave]);
    __builtin_amdgcn_wave_barrier();
    if (lane < T && lane < w.len - t) gptr<gf32>(w.out)[t + lane] = old + (row >= 0 ? part[wave][lane] : 0.0f);
}

template <int DP, bool kSplitRows>
__global__ __launch_bounds__(kAttendBlock, kSplitRows || DP > 128 ? 2 : 4) void add_weights(WeightsArgs a)
{
    __shared__ float part[kAttendWaves][64];
    uint32_t b = blockIdx.x;
    const bool prefix = b < a.prefix_items;
    if (!prefix) b -= a.prefix_items;
    const int32_t heads = a.pool.heads;
    const int32_t h = b % heads;
    b /= heads;
    const int32_t blocks = prefix ? a.prefix_blocks : a.own_blocks;
    const int32_t table_row = b / blocks, t0 = (b - table_row * blocks) * kWeightsTokens<DP, kSplitRows>;
    const TablesArg& tab = prefix ? a.step.prefix : a.step.own;
    const int64_t cap = prefix ? a.prefix_cap : a.own_cap, at = (int64_t(table_row) * heads + h) * cap;
    const uint64_t in = prefix ? a.prefix_in : a.own_in, out = prefix ? a.prefix_out : a.own_out;
    // page ids and old sums are asked for together with the lengths: within the bounds, and not used behind the end
    const int32_t t = t0 + (kSplitRows ? 0 : int(threadIdx.x >> 6) * 16 * kWeightsTiles<DP, false>);
    const int lane = threadIdx.x & 63;
    int32_t page = -1;
    float old = 0.0f;
    if constexpr (!kSplitRows) {
        if (t >= tab.max_len) return;
        const int32_t tok = lane < tab.max_len - t ? t + lane : tab.max_len - 1;
        page = token_page(a.pool, tab, table_row, tok);
        if (in != 0) old = gptr<const gf32>(in)[at + tok];
    }
    const uint64_t kb = wave_uniform(gptr<const gu64>(a.pool.k_pages)[a.pool.layer]);
    const int32_t len = __builtin_amdgcn_readfirstlane(table_len(tab, table_row));
    const Rows rows = prefix ? group_rows(a.step, table_row) : seq_rows(a.step, table_row);
    if (t >= len) return;
    const WeightsPiece w = {kb + uint64_t(h) * a.pool.dim * 2, in != 0 ? in + at * 4 : 0, out + at * 4, tab, table_row,
                            h, len, __builtin_amdgcn_readfirstlane(rows.first),
                            __builtin_amdgcn_readfirstlane(rows.count), prefix};
    const bool pool_ok = !bad_addr(kb);
    if (!pool_ok && lane == 0) raise_fault_lane(kFaultPool);
    if constexpr (kSplitRows)
        weights_by_rows<DP>(a, w, t, pool_ok, part);
    else
        weights_by_tokens<DP>(a, w, __builtin_amdgcn_readfirstlane(t), page, old, pool_ok, part);
}

}  // namespace kvmove
