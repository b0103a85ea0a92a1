// kv_attend.hpp -- attention of a step's new tokens over the paged cache: a
// prefix that the sequences of a group share, then each sequence's own pages.
//
// For a row (new token, query head) and the tokens t that it sees,
//   s_t = scale q.k_t,  lse = log sum exp s_t,  o = sum exp(s_t - lse) v_t.
// Any cut of the tokens into pieces gives the same sums: a piece keeps its
// maximum m, l = sum exp(s_t - m) and acc = sum exp(s_t - m) v_t, and pieces
// join as sum exp(m_i - m) l_i and sum exp(m_i - m) acc_i.  The prefix is one
// such cut, so the rows of ALL sequences of a group go through its pages
// together (its K and V are read once for the group), and the own pages of
// each sequence are the rest.  Both are cut further along the tokens so that
// a few rows over a long context fill the GPU.
//
// attend_pieces   one workgroup per (row tile, KV head, piece of the tokens);
// attend_join     joins the pieces of a row, in the order of their tokens
//                 (no atomics: the same call gives the same bits).
//
// Sums, maxima and accumulators are float32.  The products run on the matrix
// cores with the cache's own bf16: S^T = K Q^T, exact products of bf16 in
// float32 sums, and O^T = V^T P^T.  P is the one value that has to be bf16
// there; it goes in as two bf16 (p and what rounding p left), so that the
// output's error stays that of its own final rounding.
#pragma once

#include "kv_step.hpp"

namespace kvmove {

constexpr int kAttendWaves = 4;
constexpr int kAttendBlock = kAttendWaves * 64;
constexpr int kAttendTile = 32;        // tokens a wave takes at a time
constexpr int kAttendRows = 16;        // rows of a tile: columns of one matrix product
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttendArgs {
    PoolArg pool;
    StepArg step;
    uint64_t q, out, lse;          // bf16 rows [n_rows][q_heads][dim] with strides, bf16, float32 [n_rows][q_heads]
    int64_t q_row, q_head;         // strides in elements
    int64_t o_row, o_head;
    uint64_t part_ml;              // float2 [n_rows * q_heads][slots]: maximum (log2 units) and sum of a piece
    uint64_t part_acc;             // float32 [n_rows * q_heads][slots][dim]
    int32_t q_heads, rep;          // rep = q_heads / KV heads
    float scale_log2;              // scale * log2(e)
    int32_t prefix_tiles, prefix_pieces, prefix_tokens;   // row tiles of a group, pieces, tokens of a piece
    int32_t own_tiles, own_pieces, own_tokens;
    int32_t slots;                 // prefix_pieces + own_pieces
    uint32_t prefix_items;         // workgroups [0, prefix_items) take prefix pieces
};

// What one workgroup does: rows [row0, row0 + n_rows) of the flattened (new
// token, head of the KV head's group), against tokens [t0, t1) of a table.
struct AttendItem {
    int32_t h;            // KV head
    int32_t table_row;
    bool prefix;
    Rows rows;            // the new tokens of the sequence or group
    int32_t flat0, flat_n;// rows of this tile in the flattened order
    int32_t t0, t1;       // tokens of the piece, t1 cut to the length
    int32_t len;          // tokens of the table's row
    int32_t slot;
};

__device__ __forceinline__ AttendItem attend_item(const AttendArgs& a, uint32_t b, int tile_rows)
{
    AttendItem it;
    it.prefix = b < a.prefix_items;
    if (!it.prefix) b -= a.prefix_items;
    const uint32_t heads = a.pool.heads;
    it.h = b % heads;
    b /= heads;
    const int32_t tiles = it.prefix ? a.prefix_tiles : a.own_tiles;
    const int32_t pieces = it.prefix ? a.prefix_pieces : a.own_pieces;
    const int32_t tokens = it.prefix ? a.prefix_tokens : a.own_tokens;
    const int32_t tile = b % tiles;
    b /= tiles;
    const int32_t piece = b % pieces;
    it.table_row = b / pieces;
    it.rows = it.prefix ? group_rows(a.step, it.table_row) : seq_rows(a.step, it.table_row);
    it.len = table_len(it.prefix ? a.step.prefix : a.step.own, it.table_row);
    it.flat0 = tile * tile_rows;
    it.flat_n = it.rows.count * a.rep - it.flat0;
    it.flat_n = it.flat_n < tile_rows ? it.flat_n : tile_rows;
    it.t0 = piece * tokens;
    it.t1 = it.len - it.t0 < tokens ? it.len : it.t0 + tokens;
    it.slot = it.prefix ? piece : a.prefix_pieces + piece;
    return it;
}

// Tokens that the flattened row f sees of the table's row: all of a prefix,
// own tokens up to itself.
__device__ __forceinline__ int32_t visible_end(const AttendArgs& a, const AttendItem& it, int32_t f)
{
    if (it.prefix) return it.len;
    return clamp_i32(it.len - it.rows.count + (it.flat0 + f) / a.rep + 1, 0, it.len);
}

// Row of a layer's [num_pages * page_size] that token t is in, or -1 for a
// bad page id.
__device__ __forceinline__ int32_t token_row(const PoolArg& p, const TablesArg& t, int32_t table_row, int32_t tok)
{
    const uint32_t pi = page_of(p, uint32_t(tok));
    const int32_t page = gptr<const gi32>(t.table)[table_row * t.stride + pi];
    if (page < 0 || uint32_t(page) >= p.num_pages) {
        raise_fault_lane(kFaultPage);
        return -1;
    }
    return page * int32_t(p.page_size) + int32_t(uint32_t(tok) - pi * p.page_size);
}

// Two float32 -> two bf16 in one word, and the two bf16 of what that rounding
// left.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo)
{
    hi = bf16x2_rne(a, b);
    const float ra = __builtin_bit_cast(float, hi << 16), rb = __builtin_bit_cast(float, hi & 0xFFFF0000u);
    lo = bf16x2_rne(a - ra, b - rb);
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

__device__ __forceinline__ bool has_nonfinite(uint32_t x)
{
    return (x & 0x7F800000u) == 0x7F800000u || (x & 0x7F80u) == 0x7F80u;
}

// A wave's registers of the online softmax over 16 rows (matrix columns):
// lane l holds column l % 16 and, of every 16 matrix rows, the four from
// 4 * (l / 16).
template <int DP>
struct RowState {
    static constexpr int E = DP / 16;
    f32x4 acc[E];          // acc[m][i]: element d = (4 * (l / 16) + i) * E + m
    float m, l;            // maximum (log2 units); this lane's share of the sum
};

// One tile of 32 tokens.  k[i][j]: token 16 i + l % 16, elements 32 j + 8 (l / 16) ..+8.
// v[4 i + n]: token 16 i + 4 (l / 16) + n, elements (l % 16) * E ..+E.  The
// tile's matrix rows are the tokens in their order, so P^T comes out of the
// first product in the layout that the second one takes, and the second one's
// left operand is v transposed in registers, two elements an instruction.
// With kMasked, token t + x counts for this lane's row if t + x < vis and bit
// x of valid is set.
template <int DP, bool kMasked>
__device__ __forceinline__ void tile_step(RowState<DP>& st, const u32x4 (&q)[DP / 32], const u32x4 (&k)[2][DP / 32],
                                          const uint32_t (&v)[8][DP / 32], float c, int32_t t, int32_t vis,
                                          uint32_t valid)
{
    constexpr int E = DP / 16;
    const int g = (threadIdx.x & 63) >> 4;
    f32x4 s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) s[i] = mfma16(k[i][j], q[j], s[i]);
    }
    if (kMasked) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (t + 16 * i + 4 * g + n >= vis || !((valid >> (16 * i + 4 * g + n)) & 1))
                    s[i][n] = -__builtin_inff();
    }
    float mx = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) mx = __builtin_fmaxf(mx, s[i][n]);
    mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16));
    mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32));
    const float m_new = __builtin_fmaxf(st.m, mx * c);
    const float base = m_new == -__builtin_inff() ? 0.0f : m_new;     // a row that has seen nothing yet
    if (__any(m_new > st.m)) {
        const float alpha = __builtin_amdgcn_exp2f(st.m - base);
        st.l *= alpha;
#pragma unroll
        for (int m = 0; m < E; ++m) st.acc[m] *= alpha;
        st.m = m_new;
    }
    u32x4 ph, pl;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 4; n += 2) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n], c, -base));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n + 1], c, -base));
            st.l += p0 + p1;
            uint32_t hi, lo;
            split_bf16(p0, p1, hi, lo);
            ph[2 * i + n / 2] = hi;
            pl[2 * i + n / 2] = lo;
        }
    bool odd = false;
    if (kMasked) {
        // a token that some rows do not see must not reach them through 0 * inf or 0 * NaN
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < DP / 32; ++y) odd |= has_nonfinite(v[x][y]);
    }
    if (kMasked && __any(odd)) {
        // token by token, each row taking only what it sees
#pragma unroll 1
        for (int x = 0; x < 32; ++x) {
            const bool mine = g == ((x & 15) >> 2);
            const int word = 2 * (x >> 4) + ((x & 3) >> 1);
            u32x4 keep;
#pragma unroll
            for (int w = 0; w < 4; ++w) keep[w] = mine && w == word ? ((x & 1) ? 0xFFFF0000u : 0xFFFFu) : 0u;
            const bool sees = t + x < vis && ((valid >> x) & 1);
#pragma unroll
            for (int m = 0; m < E; ++m) {
                u32x4 vt;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    vt[w] = __builtin_amdgcn_perm(v[2 * w + 1][m / 2], v[2 * w][m / 2],
                                                  m % 2 ? 0x07060302u : 0x05040100u) & keep[w];
                f32x4 o = mfma16(vt, ph & keep, f32x4{0, 0, 0, 0});
                o = mfma16(vt, pl & keep, o);
                if (sees) st.acc[m] += o;
            }
        }
        return;
    }
#pragma unroll
    for (int m = 0; m < E; ++m) {
        u32x4 vt;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            vt[w] = __builtin_amdgcn_perm(v[2 * w + 1][m / 2], v[2 * w][m / 2], m % 2 ? 0x07060302u : 0x05040100u);
        st.acc[m] = mfma16(vt, ph, st.acc[m]);
        st.acc[m] = mfma16(vt, pl, st.acc[m]);
    }
}

// Elements [d, d + 8) of a row at `base` (byte address), 0 at and past dim.
template <int DP>
__device__ __forceinline__ u32x4 load_k8(uint64_t base, int d, int dim)
{
    if (d < dim) return *gptr<const gvec4>(base + d * 2);
    return u32x4{0, 0, 0, 0};
}

// Elements [r * E, r * E + E) of a row at `base`, 0 at and past dim.
template <int DP>
__device__ __forceinline__ void load_v(uint32_t (&v)[DP / 32], uint64_t base, int r, int dim)
{
    constexpr int E = DP / 16;
    if constexpr (E == 4) {
        u32x2 x = {0, 0};
        if (r * E < dim) x = *gptr<const gvec2>(base + r * E * 2);
        v[0] = x[0];
        v[1] = x[1];
    } else {
#pragma unroll
        for (int y = 0; y < E / 8; ++y) {
            const u32x4 x = load_k8<DP>(base, r * E + 8 * y, dim);
#pragma unroll
            for (int w = 0; w < 4; ++w) v[4 * y + w] = x[w];
        }
    }
}

template <int DP>
__global__ __launch_bounds__(kAttendBlock) void attend_pieces(AttendArgs a)
{
    constexpr int E = DP / 16, J = DP / 32;
    __shared__ float sm[kAttendWaves][kAttendRows], sl[kAttendWaves][kAttendRows];
    __shared__ float sacc[kAttendWaves][kAttendRows][DP + 4];
    const AttendItem it = attend_item(a, blockIdx.x, kAttendRows);
    if (it.flat_n <= 0) return;
    // the last row sees the most: no later token is needed
    const int32_t end_all = visible_end(a, it, it.flat_n - 1);
    if (it.t0 >= (it.t1 < end_all ? it.t1 : end_all)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int dim = a.pool.dim, heads = a.pool.heads;
    const uint64_t kb = wave_uniform(gptr<const gu64>(a.pool.k_pages)[a.pool.layer]);
    const uint64_t vb = wave_uniform(gptr<const gu64>(a.pool.v_pages)[a.pool.layer]);
    const bool pool_ok = !bad_addr(kb) && !bad_addr(vb);
    if (!pool_ok) raise_fault(kFaultPool);

    const int32_t t1 = pool_ok ? (it.t1 < end_all ? it.t1 : end_all) : it.t0;
    const int32_t all_see = visible_end(a, it, 0);          // tokens below it are seen by every row
    const bool live = r < it.flat_n;
    const int32_t vis = live ? visible_end(a, it, r) : 0;

    const int32_t f = it.flat0 + (live ? r : 0);
    const int32_t q_row = it.rows.first + f / a.rep, head = it.h * a.rep + f % a.rep;
    u32x4 q[J];
    const uint64_t qb = a.q + (q_row * a.q_row + head * a.q_head) * 2;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        q[j] = u32x4{0, 0, 0, 0};
        if (live) q[j] = load_k8<DP>(qb, j * 32 + g * 8, dim);
    }

    RowState<DP> st;
    st.m = -__builtin_inff();
    st.l = 0.0f;
#pragma unroll
    for (int m = 0; m < E; ++m) st.acc[m] = f32x4{0, 0, 0, 0};

    const TablesArg& tab = it.prefix ? a.step.prefix : a.step.own;
    const int64_t row_bytes = int64_t(heads) * dim * 2;
    const uint64_t kh = kb + uint64_t(it.h) * dim * 2, vh = vb + uint64_t(it.h) * dim * 2;
    for (int32_t t = it.t0 + wave * kAttendTile; t < t1; t += kAttendWaves * kAttendTile) {
        // lane l < 32 looks up token t + l; the others take it from there
        int32_t row = -1;
        if (lane < kAttendTile && t + lane < t1) row = token_row(a.pool, tab, it.table_row, t + lane);
        const uint32_t valid = uint32_t(__ballot(row >= 0));
        u32x4 k[2][J];
        uint32_t v[8][J];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int32_t kr = __shfl(row, 16 * i + r);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                k[i][j] = u32x4{0, 0, 0, 0};
                if (kr >= 0) k[i][j] = load_k8<DP>(kh + kr * row_bytes, j * 32 + g * 8, dim);
            }
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int32_t vr = __shfl(row, 16 * (x / 4) + 4 * g + x % 4);
            if (vr >= 0) {
                load_v<DP>(v[x], vh + vr * row_bytes, r, dim);
            } else {
#pragma unroll
                for (int y = 0; y < J; ++y) v[x][y] = 0;
            }
        }
        if (valid == ~0u && t + kAttendTile <= all_see)
            tile_step<DP, false>(st, q, k, v, a.scale_log2, t, vis, valid);
        else
            tile_step<DP, true>(st, q, k, v, a.scale_log2, t, vis, valid);
    }
    st.l += __shfl_xor(st.l, 16);
    st.l += __shfl_xor(st.l, 32);

    // the waves' pieces joined
    if (g == 0) {
        sm[wave][r] = st.m;
        sl[wave][r] = st.l;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < E; ++m) sacc[wave][r][(4 * g + i) * E + m] = st.acc[m][i];
    __syncthreads();
    for (int x = threadIdx.x; x < it.flat_n * (dim / 4); x += kAttendBlock) {
        const int row = x / (dim / 4), d = 4 * (x - row * (dim / 4));
        float m = sm[0][row];
#pragma unroll
        for (int w = 1; w < kAttendWaves; ++w) m = __builtin_fmaxf(m, sm[w][row]);
        const float base = m == -__builtin_inff() ? 0.0f : m;
        float l = 0.0f;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) {
            const float e = __builtin_amdgcn_exp2f(sm[w][row] - base);
            l += e * sl[w][row];
            o += *reinterpret_cast<const f32x4*>(&sacc[w][row][d]) * e;
        }
        const int32_t fr = it.flat0 + row;
        const int64_t at = (int64_t(it.rows.first + fr / a.rep) * a.q_heads + it.h * a.rep + fr % a.rep) * a.slots + it.slot;
        *gptr<gf32x4>(a.part_acc + (at * dim + d) * 4) = o;
        if (d == 0) {
            gptr<gf32>(a.part_ml)[2 * at] = m;
            gptr<gf32>(a.part_ml)[2 * at + 1] = l;
        }
    }
}

// One workgroup per (row, query head): its valid pieces, prefix first.
template <int DP>
__global__ __launch_bounds__(256) void attend_join(AttendArgs a)
{
    constexpr int L = DP / 4, G = 256 / L;
    __shared__ f32x4 so[G][L];
    const int32_t r = blockIdx.x / a.q_heads, head = blockIdx.x - r * a.q_heads;
    const int32_t s = wave_find(a.step.q_start, a.step.own.n, r);
    if (s < 0) return;
    const Rows rows = seq_rows(a.step, s);
    const int32_t i = r - rows.first;
    if (i >= rows.count) return;
    const int32_t len = table_len(a.step.own, s);
    const int32_t own = clamp_i32(len - rows.count + i + 1, 0, len);
    int32_t n_pre = 0;
    if (a.step.prefix.n > 0) {
        const int32_t g = wave_find(a.step.group_start, a.step.prefix.n, s);
        if (g >= 0) {
            const Rows gr = group_rows(a.step, g);
            if (r - gr.first < gr.count)
                n_pre = (table_len(a.step.prefix, g) + a.prefix_tokens - 1) / a.prefix_tokens;
        }
    }
    const int32_t n_own = (own + a.own_tokens - 1) / a.own_tokens, n = n_pre + n_own;
    const int64_t at = (int64_t(r) * a.q_heads + head) * a.slots;
    const int lane = threadIdx.x & 63;
    float m = -__builtin_inff();
    for (int x = lane; x < n; x += 64) {
        const int slot = x < n_pre ? x : a.prefix_pieces + x - n_pre;
        m = __builtin_fmaxf(m, gptr<const gf32>(a.part_ml)[2 * (at + slot)]);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = __builtin_fmaxf(m, __shfl_xor(m, d));
    const float base = m == -__builtin_inff() ? 0.0f : m;
    float l = 0.0f;
    for (int x = lane; x < n; x += 64) {
        const int slot = x < n_pre ? x : a.prefix_pieces + x - n_pre;
        const float e = __builtin_amdgcn_exp2f(gptr<const gf32>(a.part_ml)[2 * (at + slot)] - base);
        l += e * gptr<const gf32>(a.part_ml)[2 * (at + slot) + 1];
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) l += __shfl_xor(l, d);
    const int dim = a.pool.dim, c = threadIdx.x % L, grp = threadIdx.x / L;
    f32x4 o = {0, 0, 0, 0};
    if (c * 4 < dim)
        for (int x = grp; x < n; x += G) {
            const int slot = x < n_pre ? x : a.prefix_pieces + x - n_pre;
            const float e = __builtin_amdgcn_exp2f(gptr<const gf32>(a.part_ml)[2 * (at + slot)] - base);
            o += *gptr<const gf32x4>(a.part_acc + ((at + slot) * dim + c * 4) * 4) * e;
        }
    so[grp][c] = o;
    __syncthreads();
    if (grp == 0 && c * 4 < dim) {
#pragma unroll
        for (int x = 1; x < G; ++x) o += so[x][c];
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);       // NaN stays
        const u32x2 y = {bf16x2_rne(o[0] * inv, o[1] * inv), bf16x2_rne(o[2] * inv, o[3] * inv)};
        *gptr<gvec2>(a.out + (r * a.o_row + head * a.o_head + c * 4) * 2) = y;
        if (c == 0) gptr<gf32>(a.lse)[int64_t(r) * a.q_heads + head] = (m + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

}  // namespace kvmove
