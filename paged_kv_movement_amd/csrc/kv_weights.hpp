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
    int32_t own_blocks, prefix_blocks;
    uint32_t prefix_items;
};

// Tiles of 16 tokens a wave holds: four where many rows pass by, so that a
// row's q serves more products; two otherwise, for more waves in flight.
template <int DP, bool kSplitRows>
constexpr int kWeightsTiles = DP <= 128 && kSplitRows ? 4 : 2;

template <int DP, bool kSplitRows>
constexpr int kWeightsTokens = 16 * kWeightsTiles<DP, kSplitRows> * (kSplitRows ? 1 : kAttendWaves);   // of a workgroup

template <int DP, bool kSplitRows>
__global__ __launch_bounds__(kAttendBlock) void add_weights(WeightsArgs a)
{
    constexpr int J = DP / 32, NT = kWeightsTiles<DP, kSplitRows>;
    __shared__ float part[kAttendWaves][16 * NT];
    uint32_t b = blockIdx.x;
    const bool prefix = b < a.prefix_items;
    if (!prefix) b -= a.prefix_items;
    const int32_t heads = a.pool.heads, dim = a.pool.dim;
    const int32_t h = b % heads;
    b /= heads;
    const int32_t blocks = prefix ? a.prefix_blocks : a.own_blocks;
    const int32_t table_row = b / blocks, block = b - table_row * blocks;
    const TablesArg& tab = prefix ? a.step.prefix : a.step.own;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15,
              g = lane >> 4;
    const int32_t t = block * kWeightsTokens<DP, kSplitRows> + (kSplitRows ? 0 : wave * 16 * NT);
    if (t >= tab.max_len) return;
    // lengths, rows, page ids and old sums are asked for together; the page of a token behind the end is not used
    const int32_t tok = lane < tab.max_len - t ? t + lane : tab.max_len - 1;
    const int32_t page = token_page(a.pool, tab, table_row, tok);
    const int64_t cap = prefix ? a.prefix_cap : a.own_cap;
    const int64_t at = (int64_t(table_row) * heads + h) * cap + t;
    const uint64_t in = prefix ? a.prefix_in : a.own_in, out = prefix ? a.prefix_out : a.own_out;
    float old = 0.0f;
    if (in != 0 && lane < 16 * NT && lane < tab.max_len - t) old = gptr<const gf32>(in)[at + lane];
    const uint64_t kb = wave_uniform(gptr<const gu64>(a.pool.k_pages)[a.pool.layer]);
    const int32_t len = __builtin_amdgcn_readfirstlane(table_len(tab, table_row));
    const Rows rw = prefix ? group_rows(a.step, table_row) : seq_rows(a.step, table_row);
    const int32_t first_row = __builtin_amdgcn_readfirstlane(rw.first),
                  count = __builtin_amdgcn_readfirstlane(rw.count);
    if (t >= len) return;
    const bool pool_ok = !bad_addr(kb);
    if (!pool_ok && lane == 0) raise_fault_lane(kFaultPool);
    const int32_t row = pool_ok && lane < 16 * NT && t + lane < len ? row_in_page(a.pool, page, t + lane) : -1;
    const uint64_t valid = __ballot(row >= 0);
    const uint32_t row_bytes = heads * dim * 2;
    const uint64_t kh = kb + uint64_t(h) * dim * 2;
    u32x4 k[NT][J];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int32_t kr = __shfl(row, 16 * i + r);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            k[i][j] = u32x4{0, 0, 0, 0};
            if (kr >= 0) k[i][j] = load_k8(kh + uint64_t(uint32_t(kr)) * row_bytes, j * 32 + g * 8, dim);
        }
    }
    f32x4 sum[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) sum[i] = f32x4{0, 0, 0, 0};
    const int32_t flat_n = count * a.rep;
    // token t is first seen by new token t - (len - count): rows before its first head see none of these tokens
    const int32_t before = prefix ? 0 : t - (len - count);
    const int32_t skip = before > 0 ? before * a.rep / 16 : 0;
    constexpr int kStep = kSplitRows ? kAttendWaves : 1;

    // column r of row block x: its q and lse (-infinity for no row)
    struct Column {
        u32x4 q[J];
        float lse;
        int32_t vis;
    };
    auto load_column = [&](int32_t x, Column& c) {
        const int32_t f = x * 16 + r;
        const bool live = f < flat_n;
        const int32_t i = live ? new_token(a, f) : 0, head = h * a.rep + (live ? f - i * a.rep : 0);
        const int64_t qr = first_row + i;
        c.vis = prefix ? len : clamp_i32(len - count + i + 1, 0, len);
        c.lse = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < J; ++j) c.q[j] = u32x4{0, 0, 0, 0};
        if (!live) return;
        c.lse = gptr<const gf32>(a.lse)[qr * a.q_heads + head];
#pragma unroll
        for (int j = 0; j < J; ++j)
            c.q[j] = load_k8(a.q + (qr * a.q_row + head * a.q_head) * 2, j * 32 + g * 8, dim);
    };
    const int32_t n_blocks = (flat_n + 15) / 16;
    int32_t x = skip + (kSplitRows ? wave : 0);
    Column now;
    if (x < n_blocks) load_column(x, now);
#pragma unroll 1
    for (; x < n_blocks; x += kStep) {
        Column next;
        load_column(x + kStep, next);
        f32x4 s[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            s[i] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < J; ++j) s[i] = mfma16(k[i][j], now.q[j], s[i]);
        }
        // minus lse in log2 units; a row that saw nothing adds nothing: exp2(-infinity)
        const float neg = now.lse == -__builtin_inff() ? now.lse : -now.lse * kLog2e;
        // the block's first row sees the least
        const bool masked = !prefix && len - count + new_token(a, x * 16) + 1 < t + 16 * NT;
        if (masked) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n], a.scale_log2, neg));
                    sum[i][n] += t + 16 * i + 4 * g + n < now.vis ? p : 0.0f;
                }
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    sum[i][n] += __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n], a.scale_log2, neg));
        }
        now = next;
    }
    // over the 16 columns; then lane y of the wave has token y
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float v = sum[i][n];
            v += __shfl_xor(v, 1);
            v += __shfl_xor(v, 2);
            v += __shfl_xor(v, 4);
            v += __shfl_xor(v, 8);
            if (r == 0) part[wave][16 * i + 4 * g + n] = v;
        }
    if (kSplitRows) __syncthreads();
    else __builtin_amdgcn_wave_barrier();
    if (kSplitRows && wave != 0) return;
    if (lane < 16 * NT && lane < len - t) {
        float v = part[kSplitRows ? 0 : wave][lane];
        if (kSplitRows)
#pragma unroll
            for (int w = 1; w < kAttendWaves; ++w) v += part[w][lane];
        gptr<gf32>(out)[at + lane] = old + (((valid >> lane) & 1) ? v : 0.0f);
    }
}

}  // namespace kvmove
