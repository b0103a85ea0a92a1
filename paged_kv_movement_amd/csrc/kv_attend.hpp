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
// there; it goes in as two bf16, p and what rounding p left (at most 2^-8 of
// it), so that at most 2^-16 of a weight is lost and the output's error stays
// that of its own final rounding, at most 2^-8.  Over 10000 tokens: 1.1e-6
// before that rounding, float32 weights 0.5e-6, and 1.677e-3 after it either
// way; one bf16 output in a thousand differs from that of float32 sums in
// another order, by its last bit, and one in two thousand does with float32
// weights.  A third part would keep all 24 bits for a third more products.
#pragma once

#include "kv_pool8.hpp"

namespace kvmove {

constexpr int kAttendWaves = 4;
constexpr int kAttendBlock = kAttendWaves * 64;
constexpr int kAttendTile = 32;        // tokens a wave of the narrow form takes at a time
constexpr int kAttendRows = 16;        // columns of one matrix product: the narrow form's rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What the kernels are made for besides a head's size: a pool of bytes with
// scales, and a window.
template <bool kBytePool, bool kWindow>
struct Form {
    static constexpr bool byte = kBytePool, win = kWindow;
};

struct AttendArgs {
    PoolArg pool;
    StepArg step;
    ScalesArg scales;              // of an 8-bit pool
    int32_t window, sinks;         // a windowed form's
    uint64_t q, out, lse;          // bf16 rows [n_rows][q_heads][dim] with strides, bf16, float32 [n_rows][q_heads]
    int64_t q_row, q_head;         // strides in elements
    int64_t o_row, o_head;
    uint64_t part_ml;              // float2 [n_rows * q_heads][slots]: maximum (log2 units) and sum of a piece
    uint64_t part_acc;             // float32 [n_rows * q_heads][slots][dim]
    int32_t q_heads, rep;          // rep = q_heads / KV heads
    uint32_t rep_magic, rep_shift; // f / rep = (f * rep_magic) >> rep_shift for f < 2^31
    float scale_log2;              // scale * log2(e)
    int32_t prefix_tiles, prefix_pieces, prefix_tokens;   // row tiles of a group, pieces, tokens of a piece
    int32_t own_tiles, own_pieces, own_tokens;
    int32_t slots;                 // prefix_pieces + own_pieces
    uint32_t prefix_items;         // workgroups [0, prefix_items) take prefix pieces
    int32_t prefix_wide, own_wide; // which form a piece takes
    int32_t own_tile_rows;         // rows of an own item, a power of two
    int32_t direct;                // one slot in all: out and lse are written at once, nothing is left to join
};

// With a window a row at position p (its own token counted from the start of
// the prefix) sees the tokens t <= p with t > p - window or t < sinks.  What
// some row of an item sees of a table is then a head [0, sink) and a run that
// begins at the first row's window.  A span numbers the two without the gap
// between them, whole 64s left out, so that no tile lies in both: pieces are cut
// from what is seen, wherever in the table it lies.
struct Span {
    int32_t head, gap, n; // token u is u < head ? u : u + gap; n in all
};

constexpr int kSpanTile = 64;

// Tokens [0, sink) and [lo, end) of a table.
__device__ __forceinline__ Span make_span(int32_t sink, int32_t lo, int32_t end)
{
    const int32_t head = int32_t((uint32_t(sink) + kSpanTile - 1) & ~uint32_t(kSpanTile - 1));
    const int32_t begin = lo & ~(kSpanTile - 1);
    const bool apart = lo < end && begin > head;
    const int32_t gap = apart ? begin - head : 0;
    const int32_t n = lo < end ? end - gap : sink < end ? sink : end;
    return {apart ? head : 0, gap, n};
}

template <class F>
__device__ __forceinline__ int32_t token_at(const Span& s, int32_t u)
{
    if constexpr (!F::win) return u;
    return u < s.head ? u : u + s.gap;
}

// Tokens that a row sees of a table: [0, end), and with a window of those the ones from lo on or below sink.
struct Seen {
    int32_t end, lo, sink;
};

template <class F>
__device__ __forceinline__ bool sees(const Seen& s, int32_t t)
{
    if constexpr (F::win) return t < s.end && (t >= s.lo || t < s.sink);
    return t < s.end;
}

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
    // with a window: t0 and t1 count the tokens of `span`, not those of the table
    Span span;
    int32_t sink;         // the table's tokens [0, sink) are seen by every row that comes after them
    int32_t seq0, seqs;   // the sequences of a prefix's group
    int32_t start, past;  // of up to 64 of them, in lane i the i-th's: first row, tokens ahead of it
};

__device__ __forceinline__ AttendItem attend_item(const AttendArgs& a, uint32_t b, int wide_rows)
{
    AttendItem it;
    it.prefix = b < a.prefix_items;
    if (!it.prefix) b -= a.prefix_items;
    const uint32_t heads = a.pool.heads;
    const int32_t tokens = it.prefix ? a.prefix_tokens : a.own_tokens;
    const int32_t tiles = it.prefix ? a.prefix_tiles : a.own_tiles;
    it.h = b % heads;
    b /= heads;
    const int32_t pieces = it.prefix ? a.prefix_pieces : a.own_pieces;
    // the last rows of a prompt see the most: they start first
    const int32_t tile = it.prefix ? b % tiles : tiles - 1 - b % tiles;
    b /= tiles;
    const int32_t piece = b % pieces;
    it.table_row = b / pieces;
    const Rows rows = it.prefix ? group_rows(a.step, it.table_row) : seq_rows(a.step, it.table_row);
    it.rows = {__builtin_amdgcn_readfirstlane(rows.first), __builtin_amdgcn_readfirstlane(rows.count)};
    it.len = __builtin_amdgcn_readfirstlane(table_len(it.prefix ? a.step.prefix : a.step.own, it.table_row));
    const int32_t tile_rows = (it.prefix ? a.prefix_wide : a.own_wide) ? wide_rows : kAttendRows;
    it.flat0 = tile * tile_rows;
    it.flat_n = it.rows.count * a.rep - it.flat0;
    it.flat_n = it.flat_n < tile_rows ? it.flat_n : tile_rows;
    it.t0 = piece * tokens;
    it.t1 = it.len - it.t0 < tokens ? it.len : it.t0 + tokens;
    it.slot = it.prefix ? piece : a.prefix_pieces + piece;
    it.sink = 0;
    return it;
}

// New token of the flattened row f, counted from the first.
template <class Args>
__device__ __forceinline__ int32_t new_token(const Args& a, int32_t f)
{
    return int32_t((uint64_t(uint32_t(f)) * a.rep_magic) >> a.rep_shift);
}

// Tokens that the flattened row f sees of the table's row: all of a prefix,
// own tokens up to itself.
__device__ __forceinline__ int32_t visible_end(const AttendArgs& a, const AttendItem& it, int32_t f)
{
    if (it.prefix) return it.len;
    return clamp_i32(it.len - it.rows.count + new_token(a, it.flat0 + f) + 1, 0, it.len);
}

// First token that is inside the window of a row at position p.
__device__ __forceinline__ int32_t window_begin(const AttendArgs& a, int32_t p)
{
    return p < a.window ? 0 : p - a.window + 1;
}

// Own tokens that are among the first `sinks`, behind a prefix of `ahead`; no table holds more than 2^30.
__device__ __forceinline__ int32_t own_sink(const AttendArgs& a, int32_t ahead)
{
    return clamp_i32(a.sinks - ahead, 0, 1 << 30);
}

// Prefix tokens ahead of sequence s.
__device__ __forceinline__ int32_t prefix_ahead(const StepArg& a, int32_t s)
{
    if (a.prefix.n == 0) return 0;
    const int32_t i0 = ranges_around(a.group_start, a.prefix.n, s), i = i0 + int32_t(threadIdx.x & 63);
    int32_t b = 0, e = 0, n = 0;
    if (i < a.prefix.n) {
        b = gptr<const gi32>(a.group_start)[i];
        e = gptr<const gi32>(a.group_start)[i + 1];
        n = table_len(a.prefix, i);
    }
    const uint64_t m = __ballot(b <= s && s < e);
    return m == 0 ? 0 : __builtin_amdgcn_readlane(n, __builtin_ctzll(m));
}

// Position in its own pages of a sequence's i-th new token, the first being at
// `first`; one that the lengths leave no slot for counts as standing on the
// prefix's last token.
__device__ __forceinline__ int32_t row_position(int32_t first, int32_t i) { return first + i < -1 ? -1 : first + i; }

// What a group's rows see of a prefix of len tokens: the sinks, and all from
// the first window of its sequences on.  Lane i gets the i-th of the first 64
// sequences.
struct GroupWindow {
    Span span;
    int32_t seq0, seqs, start, past;
};

__device__ __forceinline__ GroupWindow group_window(const AttendArgs& a, int32_t g, int32_t len)
{
    const StepArg& st = a.step;
    const int32_t lane = threadIdx.x & 63;
    GroupWindow w;
    w.seq0 = clamp_i32(__builtin_amdgcn_readfirstlane(gptr<const gi32>(st.group_start)[g]), 0, st.own.n);
    w.seqs = clamp_i32(__builtin_amdgcn_readfirstlane(gptr<const gi32>(st.group_start)[g + 1]), w.seq0, st.own.n) - w.seq0;
    int32_t least = 0x7FFFFFFF;                                // first position of the group's new tokens
    w.start = 0x7FFFFFFF;
    w.past = 0;
    for (int32_t i = lane; i < w.seqs; i += 64) {
        const Rows r = seq_rows(st, w.seq0 + i);
        const int32_t p = table_len(st.own, w.seq0 + i) - r.count;
        if (i == lane) {
            w.start = r.first;
            w.past = p;
        }
        if (r.count > 0 && p < least) least = p;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t x = __shfl_xor(least, d);
        least = x < least ? x : least;
    }
    least = __builtin_amdgcn_readfirstlane(least);
    // 2^30 tokens of each table at most: no sum passes 31 bits
    const int32_t lo = least == 0x7FFFFFFF ? len : window_begin(a, len + row_position(least, 0));
    w.span = make_span(a.sinks < len ? a.sinks : len, lo, len);
    return w;
}

// Position in its own pages of row `row` of a group.  A row of a sequence that
// has fewer rows than counted is never read.
__device__ __forceinline__ int32_t group_row_position(const AttendArgs& a, const AttendItem& it, int32_t row)
{
    int32_t at = 0, start, past;                               // the last sequence that starts at or before it
    if (it.seqs <= 64) {
        for (int32_t step = 32; step > 0; step >>= 1) {
            const int32_t b = __shfl(it.start, at + step);
            if (at + step < it.seqs && b <= row) at += step;
        }
        start = __shfl(it.start, at);
        past = __shfl(it.past, at);
    } else {
        int32_t n = it.seqs;                                   // among [at, at + n)
        while (n > 1) {
            const int32_t half = n / 2;
            if (clamp_i32(gptr<const gi32>(a.step.q_start)[it.seq0 + at + half], 0, a.step.n_rows) <= row) {
                at += half;
                n -= half;
            } else {
                n = half;
            }
        }
        const Rows r = seq_rows(a.step, it.seq0 + at);
        start = r.first;
        past = table_len(a.step.own, it.seq0 + at) - r.count;
    }
    return row_position(past, row - start);
}

// Tokens that the flattened row f sees of the item's table.  All lanes of a wave together.
template <class F>
__device__ __forceinline__ Seen seen_by(const AttendArgs& a, const AttendItem& it, int32_t f)
{
    Seen s{visible_end(a, it, f), 0, it.sink};
    if constexpr (F::win) {
        const int32_t i = new_token(a, it.flat0 + f);
        if (it.prefix)
            s.lo = window_begin(a, it.len + group_row_position(a, it, it.rows.first + i));
        else
            s.lo = window_begin(a, row_position(it.len - it.rows.count, i));
    }
    return s;
}

// The item's piece of what its rows see.
__device__ __forceinline__ void window_item(const AttendArgs& a, AttendItem& it)
{
    GroupWindow w{};
    int32_t sink;
    if (it.prefix) {
        sink = a.sinks < it.len ? a.sinks : it.len;
        w = group_window(a, it.table_row, it.len);
    } else {
        sink = own_sink(a, a.sinks > 0 ? prefix_ahead(a.step, it.table_row) : 0);
        const int32_t first = row_position(it.len - it.rows.count, new_token(a, it.flat0));
        w.span = make_span(sink, window_begin(a, first), visible_end(a, it, it.flat_n - 1));
    }
    it.sink = __builtin_amdgcn_readfirstlane(sink);
    it.span = {__builtin_amdgcn_readfirstlane(w.span.head), __builtin_amdgcn_readfirstlane(w.span.gap),
               __builtin_amdgcn_readfirstlane(w.span.n)};
    it.seq0 = w.seq0;
    it.seqs = w.seqs;
    it.start = w.start;
    it.past = w.past;
    const int32_t tokens = it.prefix ? a.prefix_tokens : a.own_tokens;
    it.t1 = it.span.n - it.t0 < tokens ? it.span.n : it.t0 + tokens;
}

// Page id of token tok; the load is started here, what waits for it is
// row_in_page.
__device__ __forceinline__ int32_t token_page(const PoolArg& p, const TablesArg& t, int32_t table_row, int32_t tok)
{
    return gptr<const gi32>(t.table)[table_row * t.stride + page_of(p, uint32_t(tok))];
}

// Row of a layer's [num_pages * page_size] that token tok, on that page, is
// in; -1 for a page outside the pool.
__device__ __forceinline__ int32_t row_in_page(const PoolArg& p, int32_t page, int32_t tok)
{
    if (uint32_t(page) >= p.num_pages) {
        raise_fault_lane(kFaultPage);
        return -1;
    }
    return page * int32_t(p.page_size) + int32_t(uint32_t(tok) - page_of(p, uint32_t(tok)) * p.page_size);
}

__device__ __forceinline__ int32_t token_row(const PoolArg& p, const TablesArg& t, int32_t table_row, int32_t tok)
{
    return row_in_page(p, token_page(p, t, table_row, tok), tok);
}

// Two float32 -> two bf16 in one word, and the two bf16 of what that rounding
// left.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo)
{
    hi = bf16x2_rne(a, b);
    const float ra = __builtin_bit_cast(float, hi << 16), rb = __builtin_bit_cast(float, hi & 0xFFFF0000u);
    lo = bf16x2_rne(a - ra, b - rb);
}

// x, formed anew where this stands: what is made of it is not kept in registers over a loop.
__device__ __forceinline__ int anew(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// One instruction (v_maximum3_f32).  Not by inline assembly: the compiler does
// not count the wait states that a product's result needs before it is read
// there.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// Maximum over the four lanes l % 16, + 16, + 32, + 48, without LDS: a swap of
// a value with itself leaves the two halves side by side in every lane.
__device__ __forceinline__ float max_over_groups(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t p0 = p[0], p1 = p[1];
    const float y = max3(__builtin_bit_cast(float, p0), __builtin_bit_cast(float, p1), __builtin_bit_cast(float, p1));
    const uint32_t w = __builtin_bit_cast(uint32_t, y);
    const auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    const uint32_t q0 = q[0], q1 = q[1];
    return max3(__builtin_bit_cast(float, q0), __builtin_bit_cast(float, q1), __builtin_bit_cast(float, q1));
}

// Maximum over the 16 rows of a wave: of lane l % 16, the same in every group.
__device__ __forceinline__ int32_t max_of_rows(int32_t x)
{
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
        const int32_t y = __shfl_xor(x, d);
        x = y > x ? y : x;
    }
    return x;
}

__device__ __forceinline__ int32_t min_of_rows(int32_t x) { return -max_of_rows(-x); }

// A wave's registers of the online softmax over 16 rows (matrix columns):
// lane l holds column l % 16 and, of every 16 matrix rows, the four from
// 4 * (l / 16).
template <int DP>
struct RowState {
    f32x4 acc[DP / 16];    // acc[m][i]: element acc_element(4 * (l / 16) + i, m)
    float m, l;            // the exponents' base (log2 units); this lane's share of the sum
};

template <int DP>
__device__ __forceinline__ void clear(RowState<DP>& st)
{
    st.m = -__builtin_inff();
    st.l = 0.0f;
#pragma unroll
    for (int m = 0; m < DP / 16; ++m) st.acc[m] = f32x4{0, 0, 0, 0};
}

// Elements of a token's V that lane r of 16 holds: 8 from 8 r, and for
// 256-wide heads 8 more from 128 + 8 r; for 64-wide ones 4 from 4 r.
template <int DP>
__device__ __forceinline__ constexpr int acc_element(int r, int m)
{
    return DP == 64 ? r * 4 + m : (m / 8) * 128 + r * 8 + m % 8;
}

// How far the running maximum may lag behind: exponentials stay below 2^8,
// and the accumulators are rescaled only when a row's maximum rises by more.
constexpr float kLag = 8.0f;

// Scores of 32 tokens that this lane's row does not see to -infinity: token
// t + x counts if the row sees it and bit x of valid is set.
template <class F>
__device__ __forceinline__ void mask_scores(f32x4 (&s)[2], int32_t t, const Seen& vis, uint32_t valid)
{
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (F::win) {
        // counted from the lane's first token, so that a score's place is a constant; two comparisons a score
        const int32_t first = t + 4 * g, lo = vis.lo - first, n_lo = vis.end - vis.lo;
        const int32_t sink = (vis.sink < vis.end ? vis.sink : vis.end) - first;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int x = 16 * i + n;
                const bool in_window = n_lo > 0 && uint32_t(x - lo) < uint32_t(n_lo);
                if (!(in_window || x < sink)) s[i][n] = -__builtin_inff();
            }
        if (valid == ~0u) return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (!((valid >> (16 * i + 4 * g + n)) & 1)) s[i][n] = -__builtin_inff();
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int x = 16 * i + 4 * g + n;
            if (!sees<F>(vis, t + x) || !((valid >> x) & 1)) s[i][n] = -__builtin_inff();
        }
}

__device__ __forceinline__ float max_of(const f32x4 (&s)[2])
{
    return max3(max3(max3(s[0][0], s[0][1], s[0][2]), s[0][3], s[1][0]), max3(s[1][1], s[1][2], s[1][3]), s[1][3]);
}

// Raises the state's base to a row's new maximum `top` (log2 units) where it
// has risen by more than kLag, and what it holds with it.  The base stays
// finite: a score of +infinity then weighs infinity, l is infinite and so is
// the lse (less an infinite base it would be NaN), and a NaN beside it still
// makes l NaN; the row's out is NaN, its weights' second part being
// infinity less infinity.
template <int DP>
__device__ __forceinline__ void raise_base(RowState<DP>& st, float top)
{
    if (__any(top > st.m + kLag)) {
        const float m_new = __builtin_fminf(__builtin_fmaxf(st.m, top), __FLT_MAX__);
        const float alpha = m_new == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(st.m - m_new);
        st.l *= alpha;
#pragma unroll
        for (int m = 0; m < DP / 16; ++m) st.acc[m] *= alpha;
        st.m = m_new;
    }
}

// Softmax weights of 32 tokens for one block of rows, as two bf16 parts in the
// layout of the next product's right operand; their sum goes to the state.
template <int DP>
__device__ __forceinline__ void weights_of(RowState<DP>& st, const f32x4 (&s)[2], u32x4& ph, u32x4& pl, float c)
{
    const float base = st.m == -__builtin_inff() ? 0.0f : st.m;       // a row that has seen nothing yet
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 4; n += 2) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n], c, -base));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][n + 1], c, -base));
            sum += p0 + p1;
            uint32_t hi, lo;
            split_bf16(p0, p1, hi, lo);
            ph[2 * i + n / 2] = hi;
            pl[2 * i + n / 2] = lo;
        }
    st.l += sum;
}

// Left operand of O^T = V^T P^T for accumulator m: the lane's element m of
// its eight tokens (v[x]: token 16 (x / 4) + 4 (l / 16) + x % 4), two tokens
// an instruction.
template <int DP>
__device__ __forceinline__ u32x4 v_column(const uint32_t (&v)[8][DP / 32], int m)
{
    u32x4 vt;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        vt[w] = __builtin_amdgcn_perm(v[2 * w + 1][m / 2], v[2 * w][m / 2], m % 2 ? 0x07060302u : 0x05040100u);
    return vt;
}

// Adds 32 tokens' weighted V to NB blocks of rows.
template <int DP, int NB>
__device__ __forceinline__ void add_v(RowState<DP> (&st)[NB], const uint32_t (&v)[8][DP / 32], const u32x4 (&ph)[NB],
                                      const u32x4 (&pl)[NB])
{
#pragma unroll
    for (int m = 0; m < DP / 16; ++m) {
        const u32x4 vt = v_column<DP>(v, m);
#pragma unroll
        for (int b = 0; b < NB; ++b) st[b].acc[m] = mfma16(vt, ph[b], st[b].acc[m]);
#pragma unroll
        for (int b = 0; b < NB; ++b) st[b].acc[m] = mfma16(vt, pl[b], st[b].acc[m]);
    }
}

// A V that is not finite does not go through add_v: 0 times it is NaN, for a
// row that does not see its token and for the second part of a weight alike.
// A piece is therefore done without a thought of it, and if a result is not
// finite it is done again with care: take_nonfinite sets such elements to 0
// for add_v, add_nonfinite adds them as the formula has it, token by token,
// each row what it sees.
template <int DP>
__device__ __forceinline__ void take_nonfinite(uint32_t (&v)[8][DP / 32])
{
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) {
            uint32_t u = v[x][y];
            if ((u & 0x7F80u) == 0x7F80u) u &= 0xFFFF0000u;
            if ((u & 0x7F800000u) == 0x7F800000u) u &= 0x0000FFFFu;
            v[x][y] = u;
        }
}

// row_of(x): LDS address of the 32 tokens' V row x, as it came from the pool;
// at(d): where its elements [d, d + 4) are in the row, in bf16 elements.
template <int DP, class F, class RowOf, class At>
__device__ __forceinline__ void add_nonfinite(RowState<DP>& st, u32x4 ph, u32x4 pl, int32_t t, const Seen& vis,
                                              uint32_t valid, RowOf&& row_of, At&& at)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll 1
    for (int x = 0; x < 32; ++x) {
        const int word = 2 * (x >> 4) + ((x & 3) >> 1), shift = (x & 1) ? 0 : 16;
        const uint32_t hi = word == 0 ? ph[0] : word == 1 ? ph[1] : word == 2 ? ph[2] : ph[3];
        const uint32_t lo = word == 0 ? pl[0] : word == 1 ? pl[1] : word == 2 ? pl[2] : pl[3];
        const int from = ((x & 15) >> 2) * 16 + r;                   // the lane that holds this weight
        const uint32_t h = uint32_t(__shfl(int(hi), from)) << shift, l = uint32_t(__shfl(int(lo), from)) << shift;
        const float p = __builtin_bit_cast(float, h & 0xFFFF0000u) + __builtin_bit_cast(float, l & 0xFFFF0000u);
        if (!sees<F>(vis, t + x) || !((valid >> x) & 1)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < DP / 16; m += 4) {
                const u32x2 w = *reinterpret_cast<const u32x2*>(row_of(x) + at(x, acc_element<DP>(4 * g + i, m)));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t bits = e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16;
                    if ((bits & 0x7F800000u) == 0x7F800000u) st.acc[m + e][i] += p * __builtin_bit_cast(float, bits);
                }
            }
    }
}

template <int DP>
__device__ __forceinline__ bool all_finite(const RowState<DP>& st)
{
    float sum = 0.0f;                     // x - x is 0 for what is finite, else NaN
#pragma unroll
    for (int m = 0; m < DP / 16; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += st.acc[m][i] - st.acc[m][i];
    return sum == 0.0f;
}

// Elements [d, d + 8) of a row at `base` (byte address), 0 at and past dim.
__device__ __forceinline__ u32x4 load_k8(uint64_t base, int d, int dim)
{
    if (d < dim) return *gptr<const gvec4>(base + d * 2);
    return u32x4{0, 0, 0, 0};
}

// A token's (or a row's) elements 32 j + 8 g ..+8, without a branch: past dim
// the first ones are read instead, for clear_past to set to 0.
template <int DP>
__device__ __forceinline__ void load_row(u32x4 (&x)[DP / 32], uint64_t base, int g, int dim)
{
#pragma unroll
    for (int j = 0; j < DP / 32; ++j) {
        const int d = j * 32 + g * 8;
        x[j] = *gptr<const gvec4>(base + (d < dim ? d : 0) * 2);
    }
}

// q of one block of 16 rows in the layout of the first product's right
// operand: column r, elements q_element(j, g) ..+8.  The order of a head's
// elements does not matter to q.k: where K's bytes are a left operand straight
// from memory, a lane's 16 of them serve two products.
template <bool kBytes>
__device__ __forceinline__ constexpr int q_element(int j, int g)
{
    return kBytes ? j / 2 * 64 + g * 16 + j % 2 * 8 : j * 32 + g * 8;
}

template <int DP, bool kBytes = false>
__device__ __forceinline__ void clear_past(u32x4 (&x)[DP / 32], int g, int dim)
{
#pragma unroll
    for (int j = 0; j < DP / 32; ++j)
        if (q_element<kBytes>(j, g) >= dim) x[j] = u32x4{0, 0, 0, 0};
}

// The same of an 8-bit row: elements 64 j + 16 g ..+16.
template <int DP>
__device__ __forceinline__ void load_row8(u32x4 (&x)[DP / 64], uint64_t base, int g, int dim)
{
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
        const int d = j * 64 + g * 16;
        x[j] = *gptr<const gvec4>(base + (d < dim ? d : 0));
    }
}

template <int DP>
__device__ __forceinline__ void widen_row(u32x4 (&x)[DP / 32], const u32x4 (&b)[DP / 64], float scale)
{
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
        x[2 * j] = bf16_of_bytes8(b[j][0], b[j][1], scale);
        x[2 * j + 1] = bf16_of_bytes8(b[j][2], b[j][3], scale);
    }
}

// Lane r's elements of a V row at `base`; past dim the first ones.
template <int DP>
__device__ __forceinline__ void load_v(uint32_t (&v)[DP / 32], uint64_t base, int r, int dim)
{
    if constexpr (DP == 64) {
        const u32x2 x = *gptr<const gvec2>(base + (r * 4 < dim ? r * 8 : 0));
        v[0] = x[0];
        v[1] = x[1];
    } else {
#pragma unroll
        for (int y = 0; y < DP / 128; ++y) {
            const int d = y * 128 + r * 8;
            const u32x4 x = *gptr<const gvec4>(base + (d < dim ? d : 0) * 2);
#pragma unroll
            for (int w = 0; w < 4; ++w) v[4 * y + w] = x[w];
        }
    }
}

// The same of an 8-bit row, as bytes.
template <int DP>
__device__ __forceinline__ void load_v8(uint32_t (&v)[DP / 64], uint64_t base, int r, int dim)
{
    if constexpr (DP == 64) {
        v[0] = *gptr<const gu32>(base + (r * 4 < dim ? r * 4 : 0));
    } else {
#pragma unroll
        for (int y = 0; y < DP / 128; ++y) {
            const int d = y * 128 + r * 8;
            const u32x2 x = *gptr<const gvec2>(base + (d < dim ? d : 0));
            v[2 * y] = x[0];
            v[2 * y + 1] = x[1];
        }
    }
}

template <int DP>
__device__ __forceinline__ void widen_v(uint32_t (&v)[DP / 32], const uint32_t (&b)[DP / 64], float scale)
{
#pragma unroll
    for (int y = 0; y < DP / 64; ++y) {
        const u32x2 x = bf16_of_bytes(b[y], scale);
        v[2 * y] = x[0];
        v[2 * y + 1] = x[1];
    }
}

// q of one block of 16 rows: column r of the first product's right operand.
template <int DP, bool kBytes>
__device__ __forceinline__ void load_q(u32x4 (&q)[DP / 32], const AttendArgs& a, const AttendItem& it, int32_t f,
                                       bool live)
{
    const int g = (threadIdx.x & 63) >> 4;
    const int32_t flat = it.flat0 + (live ? f : 0);
    const int32_t i = new_token(a, flat);
    const int64_t row = it.rows.first + i, head = it.h * a.rep + (flat - i * a.rep);
    const uint64_t qb = a.q + (row * a.q_row + head * a.q_head) * 2;
#pragma unroll
    for (int j = 0; j < DP / 32; ++j) {
        q[j] = u32x4{0, 0, 0, 0};
        if (live) q[j] = load_k8(qb, q_element<kBytes>(j, g), a.pool.dim);
    }
}

__device__ __forceinline__ float log_sum(float m, float l) { return (m + __builtin_amdgcn_logf(l)) * kLn2; }

// 1 / l; 0 for a row that saw nothing, NaN stays.
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l); }

// Where row f of a piece goes: its part of the workspace, or with `direct`
// the result itself.
struct RowSink {
    uint64_t at;           // bf16 out or float32 acc
    float inv;             // 1 / l with `direct`
};

// The sink of row f; `first` (one lane of the row) writes its maximum and sum, or its lse.
__device__ __forceinline__ RowSink open_row(const AttendArgs& a, const AttendItem& it, int32_t f, float m, float l,
                                            bool first)
{
    const int32_t flat = it.flat0 + f, i = new_token(a, flat);
    const int64_t row = it.rows.first + i, head = it.h * a.rep + (flat - i * a.rep);
    if (a.direct) {
        if (first) gptr<gf32>(a.lse)[row * a.q_heads + head] = log_sum(m, l);
        return {a.out + (row * a.o_row + head * a.o_head) * 2, inverse_sum(l)};
    }
    const int64_t part = (row * a.q_heads + head) * a.slots + it.slot;
    if (first) {
        gptr<gf32>(a.part_ml)[2 * part] = m;
        gptr<gf32>(a.part_ml)[2 * part + 1] = l;
    }
    return {a.part_acc + part * a.pool.dim * 4, 1.0f};
}

__device__ __forceinline__ void put4(const AttendArgs& a, const RowSink& to, int d, f32x4 o)
{
    if (a.direct) {
        const u32x2 y = {bf16x2_rne(o[0] * to.inv, o[1] * to.inv), bf16x2_rne(o[2] * to.inv, o[3] * to.inv)};
        *gptr<gvec2>(to.at + d * 2) = y;
    } else {
        *gptr<gf32x4>(to.at + d * 4) = o;
    }
}

// 32 tokens of an 8-bit pool on their way into a wave's registers.
template <int DP>
struct NarrowBytes {
    u32x4 k[2][DP / 64];
    uint32_t v[8][DP / 64];
    float ks, vs;              // scales, lane x's of token x
    int32_t page;
    uint32_t valid;

    // row: lane x's is token x's; those of no token read row 0
    __device__ __forceinline__ void load(const LayerAt& l, const PoolArg& p, int32_t h, uint64_t kh, uint64_t vh,
                                         uint32_t row_bytes, int32_t row)
    {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
        const int32_t some = row < 0 ? 0 : row;
        const uint64_t at = (uint64_t(row < 0 ? 0 : page) * p.heads + h) * 4;
        valid = uint32_t(__ballot(row >= 0));
        ks = *gptr<const gf32>(l.k_scales + at);
        vs = *gptr<const gf32>(l.v_scales + at);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load_row8<DP>(k[i], kh + uint64_t(uint32_t(__shfl(some, 16 * i + r))) * row_bytes, g, p.dim);
#pragma unroll
        for (int x = 0; x < 8; ++x)
            load_v8<DP>(v[x], vh + uint64_t(uint32_t(__shfl(some, 16 * (x / 4) + 4 * g + x % 4))) * row_bytes, r, p.dim);
    }

    __device__ __forceinline__ void keys(u32x4 (&to)[2][DP / 32]) const
    {
        const int r = threadIdx.x & 15;
#pragma unroll
        for (int i = 0; i < 2; ++i) widen_row<DP>(to[i], k[i], __shfl(ks, 16 * i + r));
    }

    __device__ __forceinline__ void values(uint32_t (&to)[8][DP / 32]) const
    {
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int x = 0; x < 8; ++x) widen_v<DP>(to[x], v[x], __shfl(vs, 16 * (x / 4) + 4 * g + x % 4));
    }
};

template <int DP>
struct NarrowShared {
    float m[kAttendWaves][kAttendRows], l[kAttendWaves][kAttendRows];
    union {
        float acc[kAttendWaves][kAttendRows][DP + 4];
        u32x2 v[kAttendWaves][kAttendTile][DP / 4];          // a wave's V, for add_nonfinite
    };
};

// A piece with at most 16 rows: the waves take its tokens in turn, 32 at a
// time, each with K and V straight from memory in its registers (K rows as
// they lie are the first product's left operand), and join at the end.
//
// Bound: the read of K and V.  16 KiB a wave are in flight, two waves a SIMD:
// 64 sequences of 9000 to 10000 tokens, 8 KV heads of 128, in 454 us, 5.5 TB/s.
// One such sequence is 27 pieces a head and the waits from page id to K and V,
// three rounds of them, and the waves' join: 11.8 us for 41 MB.  In 8 bits the 64
// take 262 to 268 us, 4.7 TB/s, which is what 128-byte rows 1 KiB apart can be read at;
// the one 9.3.  A window of 4096 of 32768 tokens 9.5, in 8 bits 8.3; of 4096 of the
// 64 sequences' 202 and 121.
template <int DP, class F>
__device__ __forceinline__ void narrow_piece(const AttendArgs& a, const AttendItem& it, const LayerAt& l, int32_t t1,
                                             NarrowShared<DP>& sh)
{
    constexpr int J = DP / 32;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int dim = a.pool.dim;
    const int32_t all_see = visible_end(a, it, 0);          // tokens below it are seen by every row
    const bool live = r < it.flat_n;
    Seen vis[1] = {seen_by<F>(a, it, live ? r : 0)};
    const int32_t all_from = F::win ? max_of_rows(vis[0].lo) : 0;            // and from here on, or below vis.sink
    if (!live) vis[0].end = 0;
    u32x4 q[J];
    load_q<DP, F::byte>(q, a, it, r, live);
    RowState<DP> st[1];

    const TablesArg& tab = it.prefix ? a.step.prefix : a.step.own;
    constexpr int kSize = F::byte ? 1 : 2;
    const uint32_t row_bytes = a.pool.heads * dim * kSize;
    const uint64_t kh = l.k + uint64_t(it.h) * dim * kSize, vh = l.v + uint64_t(it.h) * dim * kSize;
    // lane l < 32 looks up token t + l, its page a round ahead; the others take it from there
    auto mine = [&](int32_t t) { return lane < kAttendTile && lane < t1 - t; };
    auto page_at = [&](int32_t t) {                // of the last token where there is no such one: no branch to wait at
        return token_page(a.pool, tab, it.table_row, token_at<F>(it.span, lane < t1 - t ? t + lane : t1 - 1));
    };
    const int32_t first = it.t0 + wave * kAttendTile;
    constexpr int32_t kRound = kAttendWaves * kAttendTile;
    clear<DP>(st[0]);
    // K, V where there is no element (of V no token either): 0
    auto clean_k = [&](u32x4 (&k)[2][J]) {
        if (dim < DP)
#pragma unroll
            for (int i = 0; i < 2; ++i) clear_past<DP, F::byte>(k[i], g, dim);
    };
    auto clean_v = [&](uint32_t valid, uint32_t (&v)[8][J]) {
        if (dim < DP)
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
                for (int y = 0; y < J; ++y)
                    if (acc_element<DP>(r, DP == 64 ? 2 * y : 8 * (y / 4)) >= dim) v[x][y] = 0;
        if (valid != ~0u) {               // a token that is not there weighs 0, and 0 times what was read may be NaN
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
                for (int y = 0; y < J; ++y)
                    if (!((valid >> (16 * (x / 4) + 4 * g + x % 4)) & 1)) v[x][y] = 0;
        }
    };
    // 32 tokens' scores, and with them what they add to the state
    auto scores = [&](f32x4 (&s)[2], const u32x4 (&k)[2][J]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[i] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < J; ++j) s[i] = mfma16(k[i][j], q[j], s[i]);
        }
    };
    auto take = [&](int32_t t, uint32_t valid, f32x4 (&s)[2], uint32_t (&v)[8][J], bool care) {
        u32x4 ph[1], pl[1];
        bool masked = valid != ~0u || t + kAttendTile > all_see;
        if constexpr (F::win) masked = masked || (t < all_from && t + kAttendTile > it.sink);
        if (masked) mask_scores<F>(s, t, vis[0], valid);
        raise_base<DP>(st[0], max_over_groups(max_of(s)) * a.scale_log2);
        weights_of<DP>(st[0], s, ph[0], pl[0], a.scale_log2);
        if (care) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
                for (int y = 0; y < J / 2; ++y) {
                    const int chunk = DP == 64 ? r : (y / 2) * 32 + 2 * r + y % 2;
                    sh.v[wave][16 * (x / 4) + 4 * g + x % 4][chunk] = u32x2{v[x][2 * y], v[x][2 * y + 1]};
                }
            __builtin_amdgcn_s_waitcnt(0);
            __builtin_amdgcn_wave_barrier();
            take_nonfinite<DP>(v);
            add_nonfinite<DP, F>(st[0], ph[0], pl[0], t, vis[0], valid,
                              [&](int x) { return reinterpret_cast<const uint16_t*>(&sh.v[wave][x][0]); },
                              [](int, int d) { return d; });
            __builtin_amdgcn_wave_barrier();
        }
        add_v<DP, 1>(st, v, ph, pl);
    };
    if constexpr (F::byte) {
        // Bytes take half the registers, so those of a round are on their way while the one before is computed: one
        // token over 10000 13.9 us, without 14.7; with two rounds on their way 14.5.
        NarrowBytes<DP> b;
        auto ask = [&](int32_t u) {                          // b.page: lane x's is that of token x of the round
            const int32_t row = mine(u) ? row_in_page(a.pool, b.page, token_at<F>(it.span, u) + lane) : -1;
            b.load(l, a.pool, it.h, kh, vh, row_bytes, row);
            b.page = page_at(u + kRound);
        };
        auto round = [&](int32_t u, bool care) {
            u32x4 k[2][J];
            uint32_t v[8][J];
            f32x4 s[2];
            b.keys(k);
            clean_k(k);
            scores(s, k);
            b.values(v);
            const uint32_t valid = b.valid;
            if (!care) ask(u + kRound);
            clean_v(valid, v);
            take(token_at<F>(it.span, u), valid, s, v, care);
        };
        if (it.t0 < t1) {
            b.page = page_at(first);
            ask(first);
        }
#pragma unroll 1
        for (int32_t u = first; u < t1; u += kRound) round(u, false);
        if (__any(!all_finite<DP>(st[0]))) {                 // a loop of its own: its care leaves no registers for rounds
            clear<DP>(st[0]);
#pragma unroll 1
            for (int32_t u = first; u < t1; u += kRound) {
                b.page = page_at(u);
                ask(u);
                round(u, true);
            }
        }
    } else {
        bool care = false;
      again:
        int32_t page = it.t0 < t1 ? page_at(first) : -1;
#pragma unroll 1
        for (int32_t u = first; u < t1; u += kRound) {
            const int32_t t = token_at<F>(it.span, u);
            const int32_t row = mine(u) ? row_in_page(a.pool, page, t + lane) : -1;
            page = page_at(u + kRound);
            const uint32_t valid = uint32_t(__ballot(row >= 0));
            u32x4 k[2][J];
            uint32_t v[8][J];
            f32x4 s[2];
            // no load behind a branch (row 0 for a token that has none), so that the waits for K leave V in flight
            const int32_t some = row < 0 ? 0 : row;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t kr = uint32_t(__shfl(some, 16 * i + r));
                load_row<DP>(k[i], kh + uint64_t(kr) * row_bytes, g, dim);
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint32_t vr = uint32_t(__shfl(some, 16 * (x / 4) + 4 * g + x % 4));
                load_v<DP>(v[x], vh + uint64_t(vr) * row_bytes, r, dim);
            }
            // V's zeros before the scores: behind them the compiler waits for all of V ahead of K's second product (one
            // token over 10000 16.3 us, so 15.5; eight on one KV head 15.9 and 15.0; 24 ragged sequences 150 and 156)
            clean_k(k);
            clean_v(valid, v);
            scores(s, k);
            take(t, valid, s, v, care);
        }
        if (!care && __any(!all_finite<DP>(st[0]))) {
            care = true;
            clear<DP>(st[0]);
            goto again;
        }
    }
    __syncthreads();                       // sh.v and sh.acc are one memory
    st[0].l += __shfl_xor(st[0].l, 16);
    st[0].l += __shfl_xor(st[0].l, 32);

    // the waves' shares joined
    if (g == 0) {
        sh.m[wave][r] = st[0].m;
        sh.l[wave][r] = st[0].l;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < DP / 16; ++m) sh.acc[wave][r][acc_element<DP>(4 * g + i, m)] = st[0].acc[m][i];
    __syncthreads();
    for (int x = threadIdx.x; x < it.flat_n * (dim / 4); x += kAttendBlock) {
        const int row = x / (dim / 4), d = 4 * (x - row * (dim / 4));
        float m = sh.m[0][row];
#pragma unroll
        for (int w = 1; w < kAttendWaves; ++w) m = __builtin_fmaxf(m, sh.m[w][row]);
        const float base = m == -__builtin_inff() ? 0.0f : m;
        float l = 0.0f;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) {
            const float e = __builtin_amdgcn_exp2f(sh.m[w][row] - base);
            l += e * sh.l[w][row];
            o += *reinterpret_cast<const f32x4*>(&sh.acc[w][row][d]) * e;
        }
        put4(a, open_row(a, it, row, m, l, d == 0), d, o);
    }
}

// Zeros in device memory: where a lane of a direct-to-LDS load has no token or
// no element to fetch, it fetches these.
__device__ u32x4 g_zero_vector;

template <int DP>
constexpr int kWideTile = DP <= 128 ? 64 : 32;       // tokens of a tile

template <int DP>
struct WideTile {
    u32x4 k[kWideTile<DP> * DP / 8];
    u32x4 v[kWideTile<DP> * DP / 8];
};

// Vectors of a token's row are stored at chunk ^ wide_swizzle(token): the 16
// tokens that a K operand reads at one chunk then lie in different banks.
template <int DP>
__device__ __forceinline__ int wide_swizzle(int token)
{
    return DP == 64 ? (token >> 1) & 7 : token & 15;
}

// One tile of tokens into LDS, this wave's share of it: kWideTile / 4 tokens.
// rows: lane x's is the pool row of the tile's token x (-1: none); valid: its
// ballot.  `flat`: a wave's tokens always lie in one page and heads fill DP,
// so that its rows follow one another and need one address.
template <int DP>
__device__ __forceinline__ void wide_load(uint64_t kh, uint64_t vh, uint32_t row_bytes, int dim, bool flat,
                                          int32_t rows, uint64_t valid, WideTile<DP>& tile)
{
    constexpr int V = DP / 8, kPer = 64 / V;                             // vectors of a row, rows of a load
    constexpr int kLoads = kWideTile<DP> / kPer / kAttendWaves, kTokens = kLoads * kPer;
    const int lane = anew(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t all = ((1ull << kTokens) - 1) << (wave * kTokens);
    if (flat && (valid & all) == all) {
        const uint64_t at = uint64_t(uint32_t(__builtin_amdgcn_readlane(rows, wave * kTokens))) * row_bytes;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int first = (wave * kLoads + i) * kPer;
            const int chunk = lane % V ^ wide_swizzle<DP>(first + lane / V);
            const uint32_t off = uint32_t(i * kPer + lane / V) * row_bytes + chunk * 16;
            __builtin_amdgcn_global_load_lds(gptr<const gvec4>(kh + at + off),
                                             (__attribute__((address_space(3))) void*)&tile.k[first * V], 16, 0, 0);
            __builtin_amdgcn_global_load_lds(gptr<const gvec4>(vh + at + off),
                                             (__attribute__((address_space(3))) void*)&tile.v[first * V], 16, 0, 0);
        }
        return;
    }
    const uint64_t zero = reinterpret_cast<uint64_t>(&g_zero_vector);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int first = (wave * kLoads + i) * kPer;
        const int tok = first + lane / V, chunk = lane % V ^ wide_swizzle<DP>(tok);
        const int32_t row = __shfl(rows, tok);
        const bool there = row >= 0 && chunk * 8 < dim;
        const uint64_t at = uint64_t(uint32_t(row)) * row_bytes + chunk * 16;
        __builtin_amdgcn_global_load_lds(gptr<const gvec4>(there ? kh + at : zero),
                                         (__attribute__((address_space(3))) void*)&tile.k[first * V], 16, 0, 0);
        __builtin_amdgcn_global_load_lds(gptr<const gvec4>(there ? vh + at : zero),
                                         (__attribute__((address_space(3))) void*)&tile.v[first * V], 16, 0, 0);
    }
}

// A wave's share of a tile of an 8-bit pool on its way: 16 bytes a lane and
// load, and the scales of the tile's tokens, lane x's of token x.
template <int DP>
struct Stage8 {
    static constexpr int V = DP / 16;                                    // vectors of a row
    static constexpr int kTokens = kWideTile<DP> / kAttendWaves, kLoads = kTokens * V / 64;
    u32x4 k[kLoads], v[kLoads];
    float ks, vs;
    uint64_t there;

    static __device__ __forceinline__ int token(int i)
    {
        const int lane = anew(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        return wave * kTokens + i * (64 / V) + lane / V;
    }

    // rows, page: lane x's are token x's
    __device__ __forceinline__ void load(const LayerAt& l, const PoolArg& p, int32_t h, uint64_t kh, uint64_t vh,
                                         uint32_t row_bytes, int32_t rows, int32_t page)
    {
        const int chunk = anew(threadIdx.x & 63) % V;
        const uint32_t off = chunk * 16 < int(p.dim) ? chunk * 16 : 0;
        const uint64_t at = (uint64_t(rows < 0 ? 0 : page) * p.heads + h) * 4;
        ks = *gptr<const gf32>(l.k_scales + at);
        vs = *gptr<const gf32>(l.v_scales + at);
        there = __ballot(rows >= 0);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int32_t row = __shfl(rows, token(i));
            const uint64_t from = uint64_t(uint32_t(row < 0 ? 0 : row)) * row_bytes + off;
            k[i] = *gptr<const gvec4>(kh + from);
            v[i] = *gptr<const gvec4>(vh + from);
        }
    }

    // as bf16, in the places that wide_load would have put them; 0 where there is no token or no element, and no scale
    // either: the one that was read in its place may be NaN, and 0 times it would be
    __device__ __forceinline__ void put(WideTile<DP>& tile, int dim) const
    {
        const int lane = anew(threadIdx.x & 63), chunk = lane % V;
        const bool mine = (there >> lane) & 1;
        const float ks1 = mine ? ks : 1.0f, vs1 = mine ? vs : 1.0f;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int tok = token(i), at = tok * (DP / 8), swz = wide_swizzle<DP>(tok);
            const bool live = ((there >> tok) & 1) && chunk * 16 < dim;
            const float sk = __shfl(ks1, tok), sv = __shfl(vs1, tok);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t none = 0;
                const int to = at + ((2 * chunk + e) ^ swz);
                tile.k[to] = bf16_of_bytes8(live ? k[i][2 * e] : none, live ? k[i][2 * e + 1] : none, sk);
                tile.v[to] = bf16_of_bytes8(live ? v[i][2 * e] : none, live ? v[i][2 * e + 1] : none, sv);
            }
        }
    }
};

// Scores of 32 tokens (half h of a tile) for this wave's NB blocks of rows.
template <int DP, int NB>
__device__ __forceinline__ void wide_scores(f32x4 (&s)[NB][2], const u32x4 (&q)[NB][DP / 32],
                                            const WideTile<DP>& tile, int h)
{
    constexpr int V = DP / 8;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) s[b][i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < DP / 32; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 k = tile.k[(32 * h + 16 * i + r) * V + ((4 * j + g) ^ wide_swizzle<DP>(r))];
#pragma unroll
            for (int b = 0; b < NB; ++b) s[b][i] = mfma16(k, q[b][j], s[b][i]);
        }
}

// V of those tokens as add_v takes it.
template <int DP>
__device__ __forceinline__ void wide_values(uint32_t (&v)[8][DP / 32], const WideTile<DP>& tile, int h)
{
    constexpr int V = DP / 8;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const int tok = 32 * h + 16 * (x / 4) + 4 * g + x % 4, swz = wide_swizzle<DP>(4 * g + x % 4);
        if constexpr (DP == 64) {
            const u32x2 y = reinterpret_cast<const u32x2*>(&tile.v[tok * V + (r / 2 ^ swz)])[r & 1];
            v[x][0] = y[0];
            v[x][1] = y[1];
        } else {
#pragma unroll
            for (int y = 0; y < DP / 128; ++y) {
                const u32x4 z = tile.v[tok * V + ((16 * y + r) ^ swz)];
#pragma unroll
                for (int w = 0; w < 4; ++w) v[x][4 * y + w] = z[w];
            }
        }
    }
}

// The products and the softmax of a tile for this wave's NB blocks of rows.
// One maximum and one look at the base for the whole tile; the first half's
// second product runs beside the second half's exponentials.
template <int DP, int NB, class F>
__device__ __forceinline__ void wide_tile(RowState<DP> (&st)[NB], const u32x4 (&q)[NB][DP / 32],
                                          const WideTile<DP>& tile, float c, bool masked, int32_t t,
                                          const Seen (&vis)[NB], uint64_t valid)
{
    constexpr int H = kWideTile<DP> / 32;
    f32x4 s[H][NB][2];
#pragma unroll
    for (int h = 0; h < H; ++h) wide_scores<DP, NB>(s[h], q, tile, h);
    if (masked)
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int b = 0; b < NB; ++b) mask_scores<F>(s[h][b], t + 32 * h, vis[b], uint32_t(valid >> (32 * h)));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float mx = max_of(s[0][b]);
        if (H > 1) {
            const float m1 = max_of(s[H - 1][b]);
            mx = max3(mx, m1, m1);
        }
        raise_base<DP>(st[b], max_over_groups(mx) * c);
    }
    u32x4 ph[NB], pl[NB];
    uint32_t v[8][DP / 32];
#pragma unroll
    for (int b = 0; b < NB; ++b) weights_of<DP>(st[b], s[0][b], ph[b], pl[b], c);
    wide_values<DP>(v, tile, 0);
    if (H > 1) {
        u32x4 ph1[NB], pl1[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) weights_of<DP>(st[b], s[H - 1][b], ph1[b], pl1[b], c);
        add_v<DP, NB>(st, v, ph, pl);
        wide_values<DP>(v, tile, H - 1);
        add_v<DP, NB>(st, v, ph1, pl1);
    } else {
        add_v<DP, NB>(st, v, ph, pl);
    }
}

// The same for a piece that is done again with care: half by half.
template <int DP, int NB, class F>
__device__ __forceinline__ void wide_half_with_care(RowState<DP> (&st)[NB], const u32x4 (&q)[NB][DP / 32],
                                                    const WideTile<DP>& tile, int h, float c, int32_t t,
                                                    const Seen (&vis)[NB], uint32_t valid)
{
    f32x4 s[NB][2];
    u32x4 ph[NB], pl[NB];
    wide_scores<DP, NB>(s, q, tile, h);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        mask_scores<F>(s[b], t, vis[b], valid);
        raise_base<DP>(st[b], max_over_groups(max_of(s[b])) * c);
        weights_of<DP>(st[b], s[b], ph[b], pl[b], c);
        add_nonfinite<DP, F>(
            st[b], ph[b], pl[b], t, vis[b], valid,
            [&](int x) { return reinterpret_cast<const uint16_t*>(&tile.v[(32 * h + x) * (DP / 8)]); },
            [](int x, int d) { return ((d / 8) ^ wide_swizzle<DP>(x)) * 8 + d % 8; });
    }
    uint32_t v[8][DP / 32];
    wide_values<DP>(v, tile, h);
    take_nonfinite<DP>(v);
    add_v<DP, NB>(st, v, ph, pl);
}

// A piece with many rows: each wave has 16 NB rows, and all of them go through
// the tokens together, kWideTile at a time, K and V brought into LDS once for
// the four waves while the tile before is computed.
//
// Bound: the vector and the matrix units, which mostly take turns.  Per 64
// scores there are 11.8 vector instructions (the exponential, the splitting of
// P, the maximum, the transposition of V) and three products: the vector units
// are busy 45 % of the cycles and the matrix cores 41 % (counters, at 2.2 GHz,
// four prompts of up to 1024 tokens behind 4096).  An 8192-token prompt, 32
// heads of 128: 742 us, 741 TFLOP/s of the formula's products; the second part
// of P makes them half as many again.  Without it 14 % shorter and an error 1.4
// times the output's own rounding.  128 rows a workgroup and two workgroups a
// CU; with 64 rows K and V come through LDS twice as often.  A window costs what
// its rows see and the tiles at its two edges: 16262 new tokens of two prompts
// under a window of 1024 in 519 to 530 us, of 128 in 224.
//
// Over bytes the same two parts, and every byte is widened by each workgroup that
// takes it: four ragged prompts behind a prefix 431 us (bf16 383), an 8192-token
// prompt 823, the window of 1024 590; the vector units are busy 60 %.  One fp16
// part takes 378, but its range ends 2^-25 below the heaviest weight of a piece,
// and what it drops is still in l: where a few tokens draw the attention and their
// V is small, the output is the sum of the light ones.  V's scales had to be near
// one another for it, too: with pages of zeros in between it was 10.7 ms.
template <int DP, int NB, class F>
__device__ __forceinline__ void wide_piece(const AttendArgs& a, const AttendItem& it, const LayerAt& l, int32_t t1,
                                           WideTile<DP>& tile0, WideTile<DP>& tile1)
{
    constexpr int T = kWideTile<DP>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15,
              g = lane >> 4;
    const int dim = a.pool.dim;
    const TablesArg& tab = it.prefix ? a.step.prefix : a.step.own;
    constexpr int kSize = F::byte ? 1 : 2;
    const uint32_t row_bytes = a.pool.heads * dim * kSize;
    const uint64_t kh = l.k + uint64_t(it.h) * dim * kSize, vh = l.v + uint64_t(it.h) * dim * kSize;
    // lane x looks up token x of a tile, its page two tiles ahead
    auto page_at = [&](int32_t t) {                // of the last token where there is no such one: no branch to wait at
        const int x = anew(lane);
        return token_page(a.pool, tab, it.table_row, token_at<F>(it.span, x < t1 - t ? t + x : t1 - 1));
    };
    auto row_at = [&](int32_t t, int32_t page) {
        const int x = anew(lane);
        return x < T && x < t1 - t ? row_in_page(a.pool, page, token_at<F>(it.span, t + x)) : -1;
    };

    const int32_t f0 = wave * 16 * NB;                       // the wave's first row in the tile
    u32x4 q[NB][DP / 32];
    RowState<DP> st[NB];
    Seen vis[NB];
    int32_t all_from = 0, some_from = 0;                     // from here on (or below the sinks) every row, some row sees
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int32_t f = f0 + 16 * b + r;
        vis[b] = seen_by<F>(a, it, f < it.flat_n ? f : 0);
        if constexpr (F::win) {
            const int32_t first = min_of_rows(f < it.flat_n ? vis[b].lo : 0x7FFFFFFF);
            const int32_t last = max_of_rows(f < it.flat_n ? vis[b].lo : 0);
            all_from = b == 0 || last > all_from ? last : all_from;
            some_from = b == 0 || first < some_from ? first : some_from;
        }
        if (f >= it.flat_n) vis[b].end = 0;
        load_q<DP, false>(q[b], a, it, f, f < it.flat_n);
    }
    const bool busy = f0 < it.flat_n;
    const int32_t all_see = busy ? visible_end(a, it, f0) : 0;
    const int32_t last = f0 + 16 * NB < it.flat_n ? f0 + 16 * NB - 1 : it.flat_n - 1;
    const int32_t end = busy ? visible_end(a, it, last) : 0; // the wave's rows see nothing from here on

    const bool flat = dim == DP && a.pool.page_size % (T / kAttendWaves) == 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) clear<DP>(st[b]);
    int32_t page = -1, rows = -1;
    uint64_t valid = 0;
    constexpr uint64_t full = T == 64 ? ~0ull : (1ull << (T & 63)) - 1;
    // the wave's part of a tile in LDS, at token u of the piece
    auto compute = [&](int32_t u, uint64_t seen, WideTile<DP>& now) {
        const int32_t t = token_at<F>(it.span, u);
        bool masked = seen != full || t + T > all_see, any = t < end;
        if constexpr (F::win) {
            masked = masked || (t < all_from && t + T > it.sink);
            any = any && (t + T > some_from || t < it.sink);
        }
        if (any) wide_tile<DP, NB, F>(st, q, now, a.scale_log2, masked, t, vis, seen);
    };
    if constexpr (F::byte) {
        // bytes come through registers, which is where they are widened: those of a tile are asked for while the one
        // before the one before it is computed, and put into LDS when that is done
        Stage8<DP> stage;
        uint64_t staged = 0;
        auto ask = [&](int32_t u) {
            rows = row_at(u, page);
            stage.load(l, a.pool, it.h, kh, vh, row_bytes, rows, page);
            staged = __ballot(rows >= 0);
            page = page_at(u + T);
        };
        if (it.t0 < t1) {
            page = page_at(it.t0);
            ask(it.t0);
            stage.put(tile0, dim);
            valid = staged;
            ask(it.t0 + T);
        }
        auto one = [&](int32_t u, WideTile<DP>& now, WideTile<DP>& next) {
            __syncthreads();                                 // now is whole, and next is done with
            const uint64_t seen = valid;
            if (u + T < t1) {
                stage.put(next, dim);
                valid = staged;
                ask(u + 2 * T);
            }
            compute(u, seen, now);
        };
#pragma unroll 1
        for (int32_t u = it.t0; u < t1; u += 2 * T) {
            one(u, tile0, tile1);
            if (u + T >= t1) break;
            one(u + T, tile1, tile0);
        }
    } else {
        if (it.t0 < t1) {
            page = page_at(it.t0);
            rows = row_at(it.t0, page);
            page = page_at(it.t0 + T);
            valid = __ballot(rows >= 0);
            wide_load<DP>(kh, vh, row_bytes, dim, flat, rows, valid, tile0);
            rows = row_at(it.t0 + T, page);
            page = page_at(it.t0 + 2 * T);
        }
        // the loads of a tile are waited for one tile after they were issued; the barrier says both that every wave's
        // share has landed and that the other tile is free again
        auto one = [&](int32_t u, WideTile<DP>& now, WideTile<DP>& next) {
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
            const uint64_t seen = valid;
            if (u + T < t1) {
                valid = __ballot(rows >= 0);
                wide_load<DP>(kh, vh, row_bytes, dim, flat, rows, valid, next);
            }
            rows = row_at(u + 2 * T, page);
            page = page_at(u + 3 * T);
            compute(u, seen, now);
        };
        // two tiles by name: with an index between them the reads of one would wait for the loads of the other
#pragma unroll 1
        for (int32_t u = it.t0; u < t1; u += 2 * T) {
            one(u, tile0, tile1);
            if (u + T >= t1) break;
            one(u + T, tile1, tile0);
        }
    }
    bool finite = true;
#pragma unroll
    for (int b = 0; b < NB; ++b) finite = finite && all_finite<DP>(st[b]);
    if (__syncthreads_or(!finite)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) clear<DP>(st[b]);
#pragma unroll 1
        for (int32_t u = it.t0; u < t1; u += T) {
            const int32_t t = token_at<F>(it.span, u);
            page = page_at(u);
            rows = row_at(u, page);
            valid = __ballot(rows >= 0);
            __syncthreads();                               // the tile before is done with
            if constexpr (F::byte) {
                Stage8<DP> stage;
                stage.load(l, a.pool, it.h, kh, vh, row_bytes, rows, page);
                stage.put(tile0, dim);
            } else {
                wide_load<DP>(kh, vh, row_bytes, dim, flat, rows, valid, tile0);
                __builtin_amdgcn_s_waitcnt(0);
            }
            __syncthreads();
#pragma unroll 1
            for (int h = 0; h < T / 32; ++h)
                if (t + 32 * h < end)
                    wide_half_with_care<DP, NB, F>(st, q, tile0, h, a.scale_log2, t + 32 * h, vis,
                                                   uint32_t(valid >> (32 * h)));
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float sum = st[b].l;
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        const int32_t f = f0 + 16 * b + anew(r);
        if (f >= it.flat_n) continue;
        const RowSink to = open_row(a, it, f, st[b].m, sum, g == 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < DP / 16; m += 4) {
                const int d = acc_element<DP>(4 * g + i, m);
                if (d < dim)
                    put4(a, to, d,
                         f32x4{st[b].acc[m][i], st[b].acc[m + 1][i], st[b].acc[m + 2][i], st[b].acc[m + 3][i]});
            }
    }
}

// NB: blocks of 16 rows a wave of the wide form takes; 0: only the narrow form.
template <int DP, int NB, class F>
__global__ __launch_bounds__(kAttendBlock, DP <= 128 ? 2 : 1) void attend_pieces(AttendArgs a)
{
    AttendItem it = attend_item(a, blockIdx.x, kAttendWaves * 16 * NB);
    if (it.flat_n <= 0) return;
    int32_t t1;
    if constexpr (F::win) {
        window_item(a, it);
        t1 = it.t1;
    } else {
        // the last row sees the most: no later token is needed
        const int32_t end_all = visible_end(a, it, it.flat_n - 1);
        t1 = it.t1 < end_all ? it.t1 : end_all;
    }
    if (it.t0 >= t1) {
        if (!a.direct) return;                              // nothing seen: the join takes no such piece
        t1 = it.t0;
    }
    const LayerAt l = layer_at<F::byte>(a.pool, a.scales);
    if (bad_layer<F::byte>(l)) {
        raise_fault(kFaultPool);
        t1 = it.t0;
    }
    if constexpr (NB > 0) {
        __shared__ union { WideTile<DP> tile; NarrowShared<DP> narrow; } sh;
        __shared__ WideTile<DP> other;
        if (it.prefix ? a.prefix_wide : a.own_wide)
            wide_piece<DP, NB, F>(a, it, l, t1, sh.tile, other);
        else
            narrow_piece<DP, F>(a, it, l, t1, sh.narrow);
    } else {
        __shared__ NarrowShared<DP> sh;
        narrow_piece<DP, F>(a, it, l, t1, sh);
    }
}

// What a join needs of row r: how many pieces each side has.  One round of
// loads for its sequence and one for its group, and one more only where a
// group may be larger than its bound.
struct RowPieces {
    int32_t prefix, own;       // pieces; own < 0: a row of no sequence
    int32_t i, first, end, sink;   // with a window: new token, the first one's position, tokens seen up to, sinks
};

// Own pieces of a row's head, the h-th of its KV head: they are cut from what the row's tile sees.
__device__ __forceinline__ int32_t window_pieces(const AttendArgs& a, const RowPieces& n, int32_t h)
{
    const int32_t flat = n.i * a.rep + h, tile = flat & ~(a.own_tile_rows - 1);
    const Span s = make_span(n.sink, window_begin(a, row_position(n.first, new_token(a, tile))), n.end);
    return int32_t((uint32_t(s.n) + a.own_tokens - 1) / uint32_t(a.own_tokens));
}

template <bool kWindow>
__device__ __forceinline__ RowPieces row_pieces(const AttendArgs& a, int32_t r)
{
    const StepArg& st = a.step;
    const int32_t lane = threadIdx.x & 63;
    const RowOwner o = row_owner(st, r);
    if (o.s < 0) return {0, -1, 0, 0, 0, 0};
    int32_t prefix = 0, ahead = 0;
    if (st.prefix.n > 0) {
        const int32_t i0 = ranges_around(st.group_start, st.prefix.n, o.s), i = i0 + lane;
        int32_t b = 0, e = 0, n = 0;
        if (i < st.prefix.n) {
            b = gptr<const gi32>(st.group_start)[i];
            e = gptr<const gi32>(st.group_start)[i + 1];
            n = table_len(st.prefix, i);
        }
        const uint64_t m = __ballot(b <= o.s && o.s < e);
        if (m != 0) {
            const int j = __builtin_ctzll(m);
            prefix = __builtin_amdgcn_readlane(n, j);
            ahead = prefix;
            if constexpr (kWindow) prefix = group_window(a, i0 + j, prefix).span.n;
            if (st.max_group_rows < st.n_rows) {               // else no group can be cut
                const Rows gr = group_rows(st, i0 + j);
                if (r - gr.first >= gr.count) prefix = 0;
            }
        }
    }
    const int32_t own = clamp_i32(o.len - o.count + (r - o.first) + 1, 0, o.len);
    return {int32_t((uint32_t(prefix) + a.prefix_tokens - 1) / uint32_t(a.prefix_tokens)),
            int32_t((uint32_t(own) + a.own_tokens - 1) / uint32_t(a.own_tokens)), r - o.first, o.len - o.count, own,
            kWindow ? own_sink(a, ahead) : 0};
}

// Bound: a row's waits -- its sequence, its group, its parts -- and for many
// rows the read of the parts: 3.9 us for one token, 5.0 for 32, 28 for 2862 tokens
// of 32 heads and two pieces each (119 MB, 4.2 TB/s).
constexpr int kJoinAhead = 4;      // pieces of a lane whose sums are on their way at once

// Joins the pieces of (row, query head), G lanes' worth of slots at a time:
// lane group `grp` of `groups` takes pieces grp, grp + groups, ...  Returns
// this lane's elements [4 c, 4 c + 4), summed over its own group only, and
// the row's maximum and sum.
template <int DP>
__device__ __forceinline__ f32x4 join_row(const AttendArgs& a, int64_t at, RowPieces n, int c, int grp, int groups,
                                          float& m, float& l)
{
    const int lane = threadIdx.x & 63, dim = a.pool.dim, total = n.prefix + n.own;
    auto slot_of = [&](int x) { return x < n.prefix ? x : a.prefix_pieces + x - n.prefix; };
    m = -__builtin_inff();
    l = 0.0f;
    if (total == 0) return f32x4{0, 0, 0, 0};
    auto part_of = [&](int x) {
        return *gptr<const gf32x4>(a.part_acc + ((at + slot_of(x)) * dim + (c * 4 < dim ? c * 4 : 0)) * 4);
    };
    // the first pieces' sums are asked for together with their maxima: the last piece again where there are fewer
    f32x4 first[kJoinAhead];
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u) first[u] = part_of(grp + u * groups < total ? grp + u * groups : total - 1);
    float pm = -__builtin_inff(), pl = 0.0f;                   // this lane's piece of the first 64
    if (lane < total) {
        const int64_t p = at + slot_of(lane);
        pm = gptr<const gf32>(a.part_ml)[2 * p];
        pl = gptr<const gf32>(a.part_ml)[2 * p + 1];
    }
    m = pm;
    for (int x = lane + 64; x < total; x += 64)
        m = __builtin_fmaxf(m, gptr<const gf32>(a.part_ml)[2 * (at + slot_of(x))]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = __builtin_fmaxf(m, __shfl_xor(m, d));
    const float base = m == -__builtin_inff() ? 0.0f : m;
    const float w = __builtin_amdgcn_exp2f(pm - base);         // weight of this lane's piece
    l = lane < total ? w * pl : 0.0f;
    for (int x = lane + 64; x < total; x += 64) {
        const int64_t p = at + slot_of(x);
        l += __builtin_amdgcn_exp2f(gptr<const gf32>(a.part_ml)[2 * p] - base) * gptr<const gf32>(a.part_ml)[2 * p + 1];
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) l += __shfl_xor(l, d);
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u) {
        const int x = grp + u * groups;                        // below 64
        const float e = __shfl(w, x);
        if (x < total) o += first[u] * e;
    }
    for (int x0 = kJoinAhead * groups; x0 < total; x0 += groups) {   // the same rounds in every lane
        const int x = x0 + grp;
        float e = __shfl(w, x & 63);
        if (x >= 64 && x < total)
            e = __builtin_amdgcn_exp2f(gptr<const gf32>(a.part_ml)[2 * (at + slot_of(x))] - base);
        if (x < total) o += part_of(x) * e;
    }
    return o;
}

__device__ __forceinline__ void put_joined(const AttendArgs& a, int32_t r, int32_t head, int c, f32x4 o, float m,
                                           float l)
{
    const float inv = inverse_sum(l);
    const u32x2 y = {bf16x2_rne(o[0] * inv, o[1] * inv), bf16x2_rne(o[2] * inv, o[3] * inv)};
    *gptr<gvec2>(a.out + (r * a.o_row + head * a.o_head + c * 4) * 2) = y;
    if (c == 0) gptr<gf32>(a.lse)[int64_t(r) * a.q_heads + head] = log_sum(m, l);
}

// Few rows, many pieces: a workgroup per (row, query head).
template <int DP, bool kWindow>
__global__ __launch_bounds__(256) void attend_join(AttendArgs a)
{
    constexpr int L = DP / 4, G = 256 / L;
    __shared__ f32x4 so[G][L];
    const int32_t r = blockIdx.x / a.q_heads, head = blockIdx.x - r * a.q_heads;
    RowPieces n = row_pieces<kWindow>(a, r);
    if (n.own < 0) return;
    if constexpr (kWindow) n.own = window_pieces(a, n, head - new_token(a, head) * a.rep);
    const int c = threadIdx.x % L, grp = threadIdx.x / L;
    float m, l;
    f32x4 o = join_row<DP>(a, (int64_t(r) * a.q_heads + head) * a.slots, n, c, grp, G, m, l);
    so[grp][c] = o;
    __syncthreads();
    if (grp == 0 && c * 4 < int(a.pool.dim)) {
#pragma unroll
        for (int x = 1; x < G; ++x) o += so[x][c];
        put_joined(a, r, head, c, o, m, l);
    }
}

// Many rows: a workgroup per row, a wave per query head at a time, so that a
// row's lookups are made once for its heads.
template <int DP, bool kWindow>
__global__ __launch_bounds__(256) void attend_join_rows(AttendArgs a)
{
    constexpr int L = DP / 4, G = 64 / L;
    const int32_t r = blockIdx.x;
    RowPieces n = row_pieces<kWindow>(a, r);
    if (n.own < 0) return;
    const int lane = threadIdx.x & 63, c = lane % L, grp = lane / L;
#pragma unroll 1
    for (int32_t head = blockIdx.y * 4 + (threadIdx.x >> 6); head < a.q_heads; head += 4 * gridDim.y) {
        float m, l;
        if constexpr (kWindow) n.own = window_pieces(a, n, head - new_token(a, head) * a.rep);
        f32x4 o = join_row<DP>(a, (int64_t(r) * a.q_heads + head) * a.slots, n, c, grp, G, m, l);
#pragma unroll
        for (int d = L; d < 64; d *= 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], d);
        if (grp == 0 && c * 4 < int(a.pool.dim)) put_joined(a, r, head, c, o, m, l);
    }
}

}  // namespace kvmove
