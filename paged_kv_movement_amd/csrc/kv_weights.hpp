// kv_weights.hpp -- the attention weight of every cached token, added to its
// running sum (what an eviction ranks the tokens by).
//
//   out[t] = in[t] + sum over the rows that see t, and over the query heads
//            of the KV head, of exp(scale q.k_t - lse[row])
//
// with the lse of a finished attention, so no maximum is searched.  A wave
// keeps its tokens' K in registers and walks the rows, so K is read once
// whatever the number of rows, each token's sum has one owner, and its order
// (rows ascending, then the 16 columns of the product) is fixed: no atomics.
//
// Bound: for single tokens the read of K, half of what the attention reads;
// for prompts the products S^T = K Q^T and one exponential for each.
#pragma once

#include "kv_attend.hpp"

namespace kvmove {

struct WeightsArgs {
    PoolArg pool;
    StepArg step;
    uint64_t q, lse;               // bf16 rows with strides, float32 [n_rows][q_heads]
    int64_t q_row, q_head;
    int32_t q_heads, rep;
    float scale_log2;
    uint64_t own_in, own_out;      // float32 [own.n][heads][own_cap]; in may be 0 (zeros) or out
    uint64_t prefix_in, prefix_out;// float32 [prefix.n][heads][prefix_cap]
    int64_t own_cap, prefix_cap;
    int32_t own_blocks, prefix_blocks;
    uint32_t prefix_items;
};

constexpr int kWeightsTokens = kAttendWaves * kAttendTile;     // tokens of a workgroup

template <int DP>
__global__ __launch_bounds__(kAttendBlock) void add_weights(WeightsArgs a)
{
    constexpr int J = DP / 32;
    uint32_t b = blockIdx.x;
    const bool prefix = b < a.prefix_items;
    if (!prefix) b -= a.prefix_items;
    const int32_t heads = a.pool.heads, dim = a.pool.dim;
    const int32_t h = b % heads;
    b /= heads;
    const int32_t blocks = prefix ? a.prefix_blocks : a.own_blocks;
    const int32_t block = b % blocks, table_row = b / blocks;
    const TablesArg& tab = prefix ? a.step.prefix : a.step.own;
    const int32_t len = table_len(tab, table_row);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int32_t t = block * kWeightsTokens + wave * kAttendTile;
    if (t >= len) return;
    const Rows rows = prefix ? group_rows(a.step, table_row) : seq_rows(a.step, table_row);
    const uint64_t kb = wave_uniform(gptr<const gu64>(a.pool.k_pages)[a.pool.layer]);
    const bool pool_ok = !bad_addr(kb);
    if (!pool_ok && lane == 0) raise_fault_lane(kFaultPool);

    int32_t row = -1;
    if (pool_ok && lane < kAttendTile && t + lane < len) row = token_row(a.pool, tab, table_row, t + lane);
    const uint32_t valid = uint32_t(__ballot(row >= 0));
    const int64_t row_bytes = int64_t(heads) * dim * 2;
    const uint64_t kh = kb + uint64_t(h) * dim * 2;
    u32x4 k[2][J];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t kr = __shfl(row, 16 * i + r);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            k[i][j] = u32x4{0, 0, 0, 0};
            if (kr >= 0) k[i][j] = load_k8(kh + kr * row_bytes, j * 32 + g * 8, dim);
        }
    }
    f32x4 sum[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    const int32_t flat_n = rows.count * a.rep;
    // rows before `skip` see none of these tokens
    int32_t skip = 0;
    if (!prefix) {
        const int32_t first = t - (len - rows.count);          // first new token that sees token t
        skip = first > 0 ? first * a.rep / 16 * 16 : 0;
    }
    for (int32_t f0 = skip; f0 < flat_n; f0 += 16) {
        const int32_t f = f0 + r;
        const bool live = f < flat_n;
        const int32_t i = (live ? f : 0) / a.rep, head = h * a.rep + (live ? f : 0) % a.rep;
        const int64_t qr = rows.first + i;
        const int32_t vis = prefix ? len : clamp_i32(len - rows.count + i + 1, 0, len);
        float lse2 = -__builtin_inff();
        if (live) lse2 = gptr<const gf32>(a.lse)[qr * a.q_heads + head] * kLog2e;
        f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            u32x4 q = {0, 0, 0, 0};
            if (live) q = load_k8(a.q + (qr * a.q_row + head * a.q_head) * 2, j * 32 + g * 8, dim);
            s[0] = mfma16(k[0][j], q, s[0]);
            s[1] = mfma16(k[1][j], q, s[1]);
        }
        const bool counts = live && lse2 != -__builtin_inff();     // a row that sees nothing adds nothing
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int32_t tok = 16 * x + 4 * g + n;
                const bool sees = counts && t + tok < vis && ((valid >> tok) & 1);
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][n], a.scale_log2, -lse2));
                sum[x][n] += sees ? p : 0.0f;
            }
    }
    const int64_t cap = prefix ? a.prefix_cap : a.own_cap;
    const int64_t at = (int64_t(table_row) * heads + h) * cap + t;
    const uint64_t in = prefix ? a.prefix_in : a.own_in, out = prefix ? a.prefix_out : a.own_out;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float v = sum[x][n];
            v += __shfl_xor(v, 1);
            v += __shfl_xor(v, 2);
            v += __shfl_xor(v, 4);
            v += __shfl_xor(v, 8);
            const int32_t tok = 16 * x + 4 * g + n;
            if (r == 0 && t + tok < len) {
                if (in != 0) v += gptr<const gf32>(in)[at + tok];
                gptr<gf32>(out)[at + tok] = v;
            }
        }
}

}  // namespace kvmove
