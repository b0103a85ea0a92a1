// kv_weights.hpp -- the attention weight of every cached token, added to its
// running sum (what an eviction ranks the tokens by).
//
//   out[t] = in[t] + sum over the rows that see t, and over the query heads
//            of the KV head, of exp(scale q.k_t - lse[row])
//
// with the lse of a finished attention, so no maximum is searched.  A wave
// keeps its tokens' K in registers as the left operand of S^T = K Q^T and
// walks the rows, 16 at a time: K is read once whatever the number of rows.
//
// add_weights        few rows: each of a workgroup's four waves has its own
//                    tokens, and the next rows' q on its way to registers;
// add_weights_rows   many rows: eight waves, two groups of tokens by four
//                    shares of the rows, whose q comes through LDS for all of
//                    them, a stage ahead; the four sums of a token meet there.
//
// Each token's sum has one owner and one order, so the same call gives the
// same bits.
//
// Bound: for single tokens the read of K, half of what the attention reads, in
// three waits a wave, and behind a large group's prefix the rows' q, which each
// wave reads for itself (32 rows of 4 heads: four times its K): 31 to 34 us for
// 32 sequences of up to 2000 tokens behind an 8192-token prefix, 92 MB, 2.7 to
// 2.9 TB/s.  For prompts, instructions and waits: the formula needs three
// vector instructions per 64 scores (exponential, fused product, sum: 16
// cycles of a wave) beside 16 cycles of matrix products, the kernel issues 6.8.
// The vector units are busy 43 % of the cycles, the matrix cores 22 %
// (counters, at 2.3 GHz).  Four prompts of 1000 to 1300 tokens, 32 heads of
// 128: 83 to 87 us, 540 to 560 TFLOP/s.
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

constexpr int kWeightsTiles = 2;                                        // tiles of 16 tokens a wave holds
constexpr int kWeightsTokens = 16 * kWeightsTiles * kAttendWaves;       // of a workgroup
// add_weights_rows: groups of tokens by shares of the rows, and the rows whose
// q is in LDS at a time.  Two tiles a wave and short stages leave room for two
// workgroups a CU, which counts for more than a q read by fewer of them (four
// prompts of 1000 to 1300 tokens: 87 us, with four tiles and 128 rows 116, with
// either alone 86; four tiles cost the form for few rows 68 us instead of 34).
constexpr int kRowsGroups = 2, kRowsShares = 4, kRowsWaves = kRowsGroups * kRowsShares;
constexpr int kRowsTokens = 16 * kWeightsTiles * kRowsGroups;
constexpr int kStageRows = 64;
constexpr int kStageBlocks = kStageRows / 16 / kRowsShares;             // blocks of 16 rows of a wave in a stage

struct WeightsPiece {
    uint64_t kh;                   // this KV head's K pool
    uint64_t in, out;              // sums of (table row, KV head)
    int32_t h, len, first_row, count;
    bool prefix;
};

// Column r of a block of 16 rows.
template <int DP>
struct WeightsColumn {
    u32x4 q[DP / 32];
    float lse;
    int32_t f;             // flattened row
    bool live;             // else it repeats the last one and sees nothing
};

// No load stands behind a branch, so that the compiler counts which of them a
// wait is for: columns past the last row read it again and see nothing.
template <int DP>
__device__ __forceinline__ void load_column(const WeightsArgs& a, const WeightsPiece& w, int32_t x,
                                            WeightsColumn<DP>& c)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, dim = a.pool.dim;
    const int32_t n = w.count * a.rep, f = x * 16 + r < n ? x * 16 + r : n - 1;
    const int32_t i = new_token(a, f), head = w.h * a.rep + (f - i * a.rep);
    const int64_t qr = w.first_row + i;
    c.f = f;
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
    for (int i = 0; i < NT; ++i) s[i] = f32x4{0, 0, 0, 0};
    // the sums in turn: a product waits for the one before it on the same sum
#pragma unroll
    for (int j = 0; j < DP / 32; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i] = mfma16(k[i][j], c.q[j], s[i]);
    __builtin_amdgcn_sched_group_barrier(0x008, NT * (DP / 32), 0);
    // minus lse in log2 units; a row that saw nothing adds nothing: exp2(-infinity)
    const float neg = c.lse == -__builtin_inff() ? -__builtin_inff() : -c.lse * kLog2e;
    // the block's first row sees the least; a column past the last row sees nothing
    const bool whole = (x + 1) * 16 <= w.count * a.rep;
    if (!whole || (!w.prefix && w.len - w.count + new_token(a, x * 16) + 1 < t + 16 * NT)) {
        const int32_t vis = !c.live ? 0 : w.prefix ? w.len : w.len - w.count + new_token(a, c.f) + 1;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n], a.scale_log2, neg));
                sum[i][n] += t + 16 * i + 4 * g + n < vis ? p : 0.0f;
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

// The sums over the 16 columns, token y's to part[y].  Each step adds across a
// distance and halves what a lane still holds: 4 NT - 1 exchanges, not 16 NT.
template <int NT>
__device__ __forceinline__ void fold_columns(const f32x4 (&sum)[NT], float* part)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    float v[4 * NT];
#pragma unroll
    for (int x = 0; x < 4 * NT; ++x) v[x] = sum[x / 4][x % 4];
    int which = 0;                       // the value that this lane ends with
#pragma unroll
    for (int n = 4 * NT, d = 8; d > 0; d /= 2) {
        const bool up = (r & d) != 0;
        if (n > 1) {
            n /= 2;
#pragma unroll
            for (int x = 0; x < n; ++x) {
                const float mine = up ? v[x + n] : v[x], other = up ? v[x] : v[x + n];
                v[x] = mine + __shfl_xor(other, d);
            }
            which += up ? n : 0;
        } else {
            v[0] += __shfl_xor(v[0], d);
        }
    }
    const bool first = (4 * NT == 16) || (r & 1) == 0;
    if (first) part[16 * (which / 4) + 4 * g + which % 4] = v[0];
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
    constexpr int NT = kWeightsTiles, T = 16 * NT;
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

// What the workgroup at b works on; tokens: of a workgroup.
struct WeightsItem {
    bool prefix;
    int32_t h, table_row, t0;
    int64_t at;            // first sum of (table row, KV head)
    uint64_t in, out;
};

template <bool kByTokens>
__device__ __forceinline__ WeightsItem weights_item(const WeightsArgs& a, uint32_t b, int tokens)
{
    WeightsItem it;
    it.prefix = b < a.prefix_items;
    if (!it.prefix) b -= a.prefix_items;
    it.h = b % a.pool.heads;
    b /= a.pool.heads;
    if (kByTokens) {
        // every sequence's first tokens, which the most rows see, before the later ones
        const int32_t n = it.prefix ? a.step.prefix.n : a.step.own.n;
        it.t0 = b / n * tokens;
        it.table_row = b % n;
    } else {
        const int32_t blocks = it.prefix ? a.prefix_blocks : a.own_blocks;
        it.table_row = b / blocks;
        it.t0 = (b - it.table_row * blocks) * tokens;
    }
    it.at = (int64_t(it.table_row) * a.pool.heads + it.h) * (it.prefix ? a.prefix_cap : a.own_cap);
    it.in = it.prefix ? a.prefix_in : a.own_in;
    it.out = it.prefix ? a.prefix_out : a.own_out;
    return it;
}

__device__ __forceinline__ WeightsPiece weights_piece(const WeightsArgs& a, const WeightsItem& it, uint64_t kb,
                                                      int32_t len)
{
    const Rows rows = it.prefix ? group_rows(a.step, it.table_row) : seq_rows(a.step, it.table_row);
    return {kb + uint64_t(it.h) * a.pool.dim * 2,
            it.in != 0 ? it.in + it.at * 4 : 0,
            it.out + it.at * 4,
            it.h,
            len,
            __builtin_amdgcn_readfirstlane(rows.first),
            __builtin_amdgcn_readfirstlane(rows.count),
            it.prefix};
}

template <int DP>
__global__ __launch_bounds__(kAttendBlock, DP > 128 ? 2 : 4) void add_weights(WeightsArgs a)
{
    __shared__ float part[kAttendWaves][64];
    const WeightsItem it = weights_item<false>(a, blockIdx.x, kWeightsTokens);
    const TablesArg& tab = it.prefix ? a.step.prefix : a.step.own;
    const int lane = threadIdx.x & 63;
    const int32_t t = it.t0 + int(threadIdx.x >> 6) * 16 * kWeightsTiles;
    if (t >= tab.max_len) return;
    // page ids and old sums are asked for together with the lengths: within the bounds, and not used behind the end
    const int32_t tok = lane < tab.max_len - t ? t + lane : tab.max_len - 1;
    const int32_t page = token_page(a.pool, tab, it.table_row, tok);
    float old = 0.0f;
    if (it.in != 0) old = gptr<const gf32>(it.in)[it.at + tok];
    const uint64_t kb = wave_uniform(gptr<const gu64>(a.pool.k_pages)[a.pool.layer]);
    const int32_t len = __builtin_amdgcn_readfirstlane(table_len(tab, it.table_row));
    const WeightsPiece w = weights_piece(a, it, kb, len);
    if (t >= len) return;
    const bool pool_ok = !bad_addr(kb);
    if (!pool_ok && lane == 0) raise_fault_lane(kFaultPool);
    weights_by_tokens<DP>(a, w, __builtin_amdgcn_readfirstlane(t), page, old, pool_ok, part);
}

// Where a lane's share of a stage is in memory: the q vectors that it brings
// into LDS (a row's at chunk ^ wide_swizzle(row), as in the attention's tiles;
// rows past the last one repeat it, elements past dim are 0) and the lse of
// its columns.  Where a stage holds whole tokens, the next stage's addresses
// follow by a step; they are worked out anew for the last stage, and
// everywhere for other numbers of heads.
template <int DP>
struct StageCursor {
    static constexpr int V = DP / 8, kPer = 64 / V, kLoads = kStageRows / kPer / kRowsWaves;
    static constexpr int Y = kStageBlocks;
    uint64_t q[kLoads], lse[Y];

    __device__ __forceinline__ void place(const WeightsArgs& a, const WeightsPiece& w, int32_t f0)
    {
        const int lane = anew(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int32_t n = w.count * a.rep;
        const uint64_t zero = reinterpret_cast<uint64_t>(&g_zero_vector);
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            const int y = (wave * kLoads + x) * kPer + lane / V;
            const int chunk = lane % V ^ wide_swizzle<DP>(y);
            const int32_t f = f0 + y < n ? f0 + y : n - 1;
            const int32_t i = new_token(a, f), head = w.h * a.rep + (f - i * a.rep);
            const uint64_t at = a.q + (int64_t(w.first_row + i) * a.q_row + head * a.q_head) * 2 + chunk * 16;
            q[x] = chunk * 8 < int(a.pool.dim) ? at : zero;
        }
#pragma unroll
        for (int y = 0; y < Y; ++y) {
            const int32_t g = f0 + (y * kRowsShares + wave % kRowsShares) * 16 + lane % 16, f = g < n ? g : n - 1;
            const int32_t i = new_token(a, f);
            lse[y] = a.lse + (int64_t(w.first_row + i) * a.q_heads + w.h * a.rep + (f - i * a.rep)) * 4;
        }
    }

    // The stage from flattened row f0 on, and the cursor to the next one.
    __device__ __forceinline__ void load(const WeightsArgs& a, const WeightsPiece& w, int32_t f0, bool steps,
                                         u32x4* stage, float (&to)[Y])
    {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if (!steps || f0 + kStageRows > w.count * a.rep) place(a, w, f0);
        const int64_t tokens = kStageRows / a.rep;
#pragma unroll
        for (int y = 0; y < Y; ++y) {
            to[y] = *gptr<const gf32>(lse[y]);
            lse[y] += tokens * a.q_heads * 4;
        }
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            __builtin_amdgcn_global_load_lds(gptr<const gvec4>(q[x]),
                                             (__attribute__((address_space(3))) void*)&stage[(wave * kLoads + x) * 64],
                                             16, 0, 0);
            q[x] += tokens * a.q_row * 2;
        }
    }
};

// The blocks of rows that this wave has in a stage.
template <int DP>
__device__ __forceinline__ void add_stage(const WeightsArgs& a, const WeightsPiece& w, int32_t f0, int32_t t,
                                          const u32x4* stage, const float (&lse)[kStageBlocks],
                                          const u32x4 (&k)[kWeightsTiles][DP / 32], f32x4 (&sum)[kWeightsTiles])
{
    constexpr int V = DP / 8, NT = kWeightsTiles;
    const int lane = threadIdx.x & 63, share = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kRowsShares,
              r = lane & 15, g = lane >> 4;
    const int32_t n = w.count * a.rep;
#pragma unroll
    for (int y = 0; y < kStageBlocks; ++y) {
        const int block = y * kRowsShares + share;
        const int32_t f = f0 + block * 16 + r;
        if (f0 + block * 16 >= n) break;
        WeightsColumn<DP> c;
        c.live = f < n;
        c.f = c.live ? f : n - 1;
        c.lse = lse[y];
#pragma unroll
        for (int j = 0; j < DP / 32; ++j)
            c.q[j] = stage[(block * 16 + r) * V + ((4 * j + g) ^ wide_swizzle<DP>(r))];
        add_block<DP, NT>(a, w, f0 / 16 + block, t, k, c, sum);
    }
}

template <int DP>
__global__ __launch_bounds__(kRowsWaves * 64, DP > 128 ? 2 : 4) void add_weights_rows(WeightsArgs a)
{
    constexpr int NT = kWeightsTiles, V = DP / 8, S = kStageRows;
    __shared__ u32x4 stage0[S * V];
    __shared__ u32x4 stage1[S * V];
    __shared__ float part[kRowsWaves][64];
    const WeightsItem it = weights_item<true>(a, blockIdx.x, kRowsTokens);
    const TablesArg& tab = it.prefix ? a.step.prefix : a.step.own;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6),
              share = wave % kRowsShares;
    const uint64_t kb = wave_uniform(gptr<const gu64>(a.pool.k_pages)[a.pool.layer]);
    const int32_t len = __builtin_amdgcn_readfirstlane(table_len(tab, it.table_row));
    const WeightsPiece w = weights_piece(a, it, kb, len);
    if (it.t0 >= len) return;
    const bool pool_ok = !bad_addr(kb);
    if (!pool_ok) raise_fault(kFaultPool);
    const int32_t t = it.t0 + wave / kRowsShares * 16 * NT;
    const bool here = pool_ok && lane < 16 * NT && lane < len - t;
    const int32_t row = here ? token_row(a.pool, tab, it.table_row, t + lane) : -1;
    u32x4 k[NT][DP / 32];
    if (pool_ok) load_keys<DP, NT>(a, w, row, k);
    f32x4 sum[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) sum[i] = f32x4{0, 0, 0, 0};
    // token t0 is first seen by new token t0 - (len - count): stages of rows before it see none of these tokens
    const int32_t before = w.prefix ? 0 : it.t0 - (len - w.count), n = pool_ok ? w.count * a.rep : 0;
    int32_t f0 = before > 0 ? before * a.rep / S * S : 0;
    const bool steps = S % a.rep == 0 && int(a.pool.dim) == DP;
    StageCursor<DP> cursor;
    float lse0[kStageBlocks], lse1[kStageBlocks];
    if (f0 < n) {
        cursor.place(a, w, f0);
        cursor.load(a, w, f0, steps, stage0, lse0);
    }
#pragma unroll 1
    for (; f0 < n; f0 += 2 * S) {
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (f0 + S < n) cursor.load(a, w, f0 + S, steps, stage1, lse1);
        add_stage<DP>(a, w, f0, t, stage0, lse0, k, sum);
        if (f0 + S >= n) break;
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (f0 + 2 * S < n) cursor.load(a, w, f0 + 2 * S, steps, stage0, lse0);
        add_stage<DP>(a, w, f0 + S, t, stage1, lse1, k, sum);
    }
    fold_columns<NT>(sum, part[wave]);
    __syncthreads();
    if (share == 0 && lane < 16 * NT && lane < len - t) {
        float v = part[wave][lane];
#pragma unroll
        for (int y = 1; y < kRowsShares; ++y) v += part[wave + y][lane];
        const float old = w.in != 0 ? gptr<const gf32>(w.in)[t + lane] : 0.0f;
        gptr<gf32>(w.out)[t + lane] = old + (row >= 0 ? v : 0.0f);
    }
}

}  // namespace kvmove
