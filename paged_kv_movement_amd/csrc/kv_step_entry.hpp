// kv_step_entry.hpp -- host side of the model-step entry points (append,
// attend, weights, evict): argument checks, launch shapes, workspaces.
// Included by kvmove.hip, whose helpers (fail, ok, check_paged, ceil_div,
// max_blocks) it uses.
#pragma once

namespace {

int check_tables(const kv_paged* p, const kv_tables* t, const char* what)
{
    if (t->n < 0 || t->n > (1 << 24)) return fail(KV_EINVAL, "%s: %d sequences outside [0, 2^24]", what, t->n);
    if (t->max_len < 0 || t->max_len > (1 << 30))
        return fail(KV_EINVAL, "%s: max_len %d outside [0, 2^30]", what, t->max_len);
    if (t->n == 0) return KV_OK;
    if (t->lens == nullptr) return fail(KV_EINVAL, "%s: lens is NULL", what);
    if (t->max_len > 0 && t->table == nullptr) return fail(KV_EINVAL, "%s: table is NULL", what);
    if (t->stride < 0 || t->stride > INT32_MAX)
        return fail(KV_EINVAL, "%s: stride %lld outside [0, 2^31)", what, (long long)t->stride);
    if (t->max_len > t->stride * p->page_size)
        return fail(KV_ERANGE, "%s: max_len %d beyond the block table (%lld pages of %d)", what, t->max_len,
                    (long long)t->stride, p->page_size);
    return KV_OK;
}

// No slot is ever read or written: then its arrays may be NULL, as an empty tensor's address is.
bool holds_nothing(const kv_tables& t) { return t.n == 0 || t.max_len == 0; }

// The pool as the step kernels take it: rows of a layer are numbered in 31 bits.
int check_step_pool(const kv_paged* p, int32_t layer_begin, int32_t layer_end)
{
    int rc = check_paged(p);
    if (rc != KV_OK) return rc;
    if (layer_begin < 0 || layer_end <= layer_begin || layer_end > p->num_layers)
        return fail(KV_EINVAL, "layers [%d, %d) are not a non-empty range inside [0, %d)", layer_begin, layer_end,
                    p->num_layers);
    if (p->num_pages > INT32_MAX / p->page_size)
        return fail(KV_EINVAL, "num_pages * page_size = %lld * %d rows: must stay below 2^31",
                    (long long)p->num_pages, p->page_size);
    return KV_OK;
}

int check_step(const kv_paged* p, const kv_step* s)
{
    if (s == nullptr) return fail(KV_EINVAL, "step is NULL");
    int rc = check_tables(p, &s->own, "own");
    if (rc == KV_OK) rc = check_tables(p, &s->prefix, "prefix");
    if (rc != KV_OK) return rc;
    if (s->n_rows < 0 || s->max_new < 0 || s->max_group_rows < 0)
        return fail(KV_EINVAL, "n_rows, max_new and max_group_rows must be >= 0");
    // a group of no sequences reads q_start[0]
    if ((s->own.n > 0 || s->prefix.n > 0) && s->q_start == nullptr) return fail(KV_EINVAL, "q_start is NULL");
    if (s->prefix.n > 0 && s->group_start == nullptr) return fail(KV_EINVAL, "group_start is NULL");
    return KV_OK;
}

// The calls launch on the current device, and so must their stream.
int check_stream(hipStream_t stream)
{
    if (stream == nullptr) return KV_OK;
    int dev = -1, sdev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipStreamGetDevice(stream, &sdev);
    if (e != hipSuccess) return fail(KV_EHIP, "reading the device failed: %s", hipGetErrorString(e));
    if (sdev != dev) return fail(KV_EINVAL, "the stream belongs to device %d, the current device is %d", sdev, dev);
    return KV_OK;
}

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// [n_rows][heads][dim] with strides in elements of `size` bytes: vectors of
// 16 bytes can be used.
bool rows_vectors(const kv_rows& x, int64_t size)
{
    return !misaligned(x.data, 16) && x.row_stride * size % 16 == 0 && x.head_stride * size % 16 == 0;
}

// Two of the [n_rows][heads] runs of dim elements have an element in common.
bool rows_overlap(const kv_rows& x, int64_t n_rows, int64_t heads, int64_t dim)
{
    using Wide = __int128;
    const Wide row = x.row_stride < 0 ? -Wide(x.row_stride) : x.row_stride;
    const Wide head = x.head_stride < 0 ? -Wide(x.head_stride) : x.head_stride;
    if ((n_rows > 1 && row < dim) || (heads > 1 && head < dim)) return true;
    if (n_rows <= 1 || heads <= 1) return false;
    // one dimension lies wholly within a step of the other: nearly every layout
    if (row >= (heads - 1) * head + dim || head >= (n_rows - 1) * row + dim) return false;
    for (int64_t h = 1; h < heads; ++h)        // the two rows nearest to h heads on (signs do not matter: all h and rows)
        for (Wide r = h * head / row; r <= h * head / row + 1; ++r) {
            const Wide apart = h * head - r * row;
            if (r >= 1 && r < n_rows && (apart < 0 ? -apart : apart) < dim) return true;
        }
    return false;
}

// x / d = (x * magic) >> shift for x < 2^31: with 2^s >= d, magic = floor(2^(31 + s) / d) + 1 is too large by at most
// 2^s / 2^(31 + s) of itself, which stays below one over the whole range.
void magic_of(int32_t d, uint32_t* magic, uint32_t* shift)
{
    uint32_t s = 0;
    while ((int64_t(1) << s) < d) ++s;
    *magic = uint32_t((uint64_t(1) << (31 + s)) / uint64_t(d) + 1);
    *shift = 31 + s;
}

PoolArg pool_arg(const kv_paged* p, int32_t layer)
{
    PoolArg a{};
    a.k_pages = reinterpret_cast<uint64_t>(p->k_pages);
    a.v_pages = reinterpret_cast<uint64_t>(p->v_pages);
    a.num_pages = uint32_t(p->num_pages);
    a.page_size = uint32_t(p->page_size);
    magic_of(p->page_size, &a.page_magic, &a.page_shift);
    a.heads = uint32_t(p->num_kv_heads);
    a.dim = uint32_t(p->head_dim);
    a.layer = layer;
    return a;
}

TablesArg tables_arg(const kv_tables* t)
{
    return {reinterpret_cast<uint64_t>(t->table), reinterpret_cast<uint64_t>(t->lens), t->stride, t->n, t->max_len};
}

StepArg step_arg(const kv_step* s)
{
    StepArg a{};
    a.own = tables_arg(&s->own);
    a.prefix = tables_arg(&s->prefix);
    a.q_start = reinterpret_cast<uint64_t>(s->q_start);
    a.group_start = reinterpret_cast<uint64_t>(s->group_start);
    a.n_rows = s->n_rows;
    a.max_new = s->max_new;
    a.max_group_rows = s->max_group_rows;
    return a;
}

int launch(KernelFn k, int64_t grid, int block, void* arg, hipStream_t stream, unsigned grid_y = 1)
{
    if (grid <= 0) return KV_OK;
    if (grid > max_blocks(block)) return fail(KV_EINVAL, "%lld workgroups exceed one launch", (long long)grid);
    void* args[] = {arg};
    const hipError_t e = hipLaunchKernel(k, dim3(unsigned(grid), grid_y), dim3(block), args, 0, stream);
    if (e != hipSuccess) return fail(KV_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return KV_OK;
}

template <class TI, class TO>
KernelFn append_kernel(bool vectors)
{
    return vectors ? reinterpret_cast<KernelFn>(&append_rows<TI, TO, 8>)
                   : reinterpret_cast<KernelFn>(&append_rows<TI, TO, 1>);
}

int append(const kv_paged* paged, const kv_step* step, int32_t layer, const kv_rows* q, const kv_rows* k,
           const kv_rows* v, const kv_rows* q_out, int32_t q_heads, kv_type type, kv_type q_out_type,
           const int32_t* positions, const kv_rope* rope, const kv_slots* slots, hipStream_t stream)
{
    int rc = check_step_pool(paged, layer, layer + 1);
    if (rc == KV_OK) rc = check_step(paged, step);
    if (rc != KV_OK) return rc;
    if (rope == nullptr || k == nullptr || v == nullptr) return fail(KV_EINVAL, "k, v or rope is NULL");
    if ((q == nullptr) != (q_out == nullptr)) return fail(KV_EINVAL, "q and q_out are given together or not at all");
    if (type != KV_TYPE_BF16 && type != KV_TYPE_FP16 && type != KV_TYPE_FP32)
        return fail(KV_EINVAL, "unknown type %d", int(type));
    if (q != nullptr && q_out_type != type && q_out_type != KV_TYPE_BF16)
        return fail(KV_EINVAL, "q_out's type must be q's or bf16");
    if (q != nullptr && q_heads <= 0) return fail(KV_EINVAL, "q_heads must be > 0");
    if (rope->rot < 0 || rope->rot % 2 != 0 || rope->rot > paged->head_dim || rope->rot > kMaxRot)
        return fail(KV_EINVAL, "rot = %d must be even and within head_dim = %d and %d", rope->rot, paged->head_dim,
                    kMaxRot);
    if (rope->rot > 0 && rope->freqs == nullptr) return fail(KV_EINVAL, "freqs is NULL");
    if (slots != nullptr) {
        if ((slots->weights == nullptr || slots->positions == nullptr) && !holds_nothing(step->own))
            return fail(KV_EINVAL, "slots: weights and positions must both be given");
        if (slots->heads != 1 && slots->heads != paged->num_kv_heads)
            return fail(KV_EINVAL, "slots: heads must be 1 or num_kv_heads (got %d)", slots->heads);
        if (slots->cap < step->own.max_len)
            return fail(KV_ERANGE, "slots: cap %lld below max_len %d", (long long)slots->cap, step->own.max_len);
    }
    if (step->n_rows == 0) return ok();
    if (q_out != nullptr && rows_overlap(*q_out, step->n_rows, q_heads, paged->head_dim))
        return fail(KV_EINVAL, "q_out's rows overlap");
    if (k->data == nullptr || v->data == nullptr || positions == nullptr || (q != nullptr && (q->data == nullptr || q_out->data == nullptr)))
        return fail(KV_EINVAL, "q, k, v, q_out or positions is NULL");
    const int64_t size = type == KV_TYPE_FP32 ? 4 : 2, out_size = q_out_type == KV_TYPE_FP32 ? 4 : 2;
    // 16-byte vectors where every address, stride and the pairs' distance allow them, else element by element
    const int dim = paged->head_dim, unit = rope->interleaved ? 8 : 16;
    bool vectors = dim % 8 == 0 && rope->rot % unit == 0 && rows_vectors(*k, size) && rows_vectors(*v, size);
    if (q != nullptr) vectors = vectors && rows_vectors(*q, size) && rows_vectors(*q_out, out_size);
    for (const kv_rows* x : {k, v, q})
        if (x != nullptr && misaligned(x->data, size)) return fail(KV_EINVAL, "q, k or v is not aligned to its type");
    if (q != nullptr && misaligned(q_out->data, out_size)) return fail(KV_EINVAL, "q_out is not aligned to its type");
    rc = check_stream(stream);
    if (rc != KV_OK) return rc;
    AppendArgs a{};
    a.pool = pool_arg(paged, layer);
    a.step = step_arg(step);
    auto at = [](const kv_rows* x, uint64_t& data, int64_t& row, int64_t& head) {
        if (x == nullptr) return;
        data = reinterpret_cast<uint64_t>(x->data);
        row = x->row_stride;
        head = x->head_stride;
    };
    at(q, a.q, a.q_row, a.q_head);
    at(k, a.k, a.k_row, a.k_head);
    at(v, a.v, a.v_row, a.v_head);
    at(q_out, a.q_out, a.o_row, a.o_head);
    a.positions = reinterpret_cast<uint64_t>(positions);
    a.freqs = reinterpret_cast<uint64_t>(rope->freqs);
    if (slots != nullptr) {
        a.weights = reinterpret_cast<uint64_t>(slots->weights);
        a.slot_positions = reinterpret_cast<uint64_t>(slots->positions);
        a.w_cap = slots->cap;
        a.w_heads = slots->heads;
    }
    a.rot = rope->rot;
    a.q_heads = q != nullptr ? q_heads : 0;
    a.interleaved = rope->interleaved;
    const int vec = vectors ? 8 : 1;
    a.units = head_units(a.rot, dim, a.interleaved != 0, vec);
    magic_of(a.units, &a.unit_magic, &a.unit_shift);
    magic_of(dim / vec, &a.vec_magic, &a.vec_shift);
    if (int64_t(a.q_heads + 2 * int64_t(paged->num_kv_heads)) * dim > INT32_MAX / 2)
        return fail(KV_EINVAL, "a token's heads are too large for one workgroup");
    a.gain = rope->gain;
    KernelFn f;
    if (type == KV_TYPE_BF16)
        f = append_kernel<__bf16, __bf16>(vectors);
    else if (type == KV_TYPE_FP16)
        f = q == nullptr || q_out_type == type ? append_kernel<_Float16, _Float16>(vectors)
                                               : append_kernel<_Float16, __bf16>(vectors);
    else
        f = q == nullptr || q_out_type == type ? append_kernel<float, float>(vectors)
                                               : append_kernel<float, __bf16>(vectors);
    rc = launch(f, step->n_rows, kAppendBlock, &a, stream);
    return rc == KV_OK ? ok() : rc;
}

// ---- attend

// The launch of an attention: how many row tiles and pieces, from the bounds
// that the host knows.
struct AttendShape {
    int32_t prefix_tiles, prefix_pieces, prefix_tokens;
    int32_t own_tiles, own_pieces, own_tokens;
    int32_t slots;
    int32_t blocks;                // blocks of 16 rows of a wave of the wide form, 0: narrow only
    bool prefix_wide, own_wide, direct;
    int64_t prefix_items, own_items;
    int64_t ml_bytes, bytes;
};

int check_heads(const kv_paged* p, int32_t q_heads)
{
    if (q_heads <= 0 || q_heads % p->num_kv_heads != 0)
        return fail(KV_EINVAL, "q_heads = %d must be a multiple of num_kv_heads = %d", q_heads, p->num_kv_heads);
    if (p->head_dim % 8 != 0 || p->head_dim > 256)
        return fail(KV_EINVAL, "head_dim = %d must be a multiple of 8 and at most 256 here", p->head_dim);
    return KV_OK;
}

// Tokens of a piece: as many pieces as make `room` workgroups (what runs at
// once) of all pairs of (row tile, KV head) together, in whole rounds of a
// workgroup's waves.
void cut_tokens(int64_t pairs, int32_t max_len, int64_t room, int32_t* tokens, int32_t* pieces)
{
    constexpr int64_t kRound = kAttendWaves * kAttendTile;
    const int64_t want = std::max<int64_t>(1, room / std::max<int64_t>(1, pairs));
    const int64_t t = ceil_div(ceil_div(std::max(max_len, 1), want), kRound) * kRound;
    *tokens = int32_t(t);
    *pieces = int32_t(ceil_div(max_len, t));
}

// Cuts of a table's tokens into pieces of whole tiles that cut_wide chooses
// from: each number of pieces up to eight, then every half as many more.
struct WideCuts {
    static constexpr int kMost = 24;
    int32_t pieces[kMost], tokens[kMost];
    int n = 0;

    WideCuts(int64_t pairs, int32_t len)
    {
        constexpr int32_t kTile = 64;
        if (len == 0) {
            pieces[0] = 0;
            tokens[0] = kTile;
            n = 1;
        }
        // no more than four rounds of 512 items, none below a tile
        for (int32_t x = 1; len > 0 && n < kMost && (x == 1 || pairs * x <= 2048); x += x < 8 ? 1 : x / 2) {
            const int32_t t = int32_t(ceil_div(ceil_div(len, x), kTile) * kTile);
            if (n == 0 || tokens[n - 1] != t) {
                tokens[n] = t;
                pieces[n++] = int32_t(ceil_div(len, t));
            }
            if (t == kTile) break;
        }
    }
};

// Pieces of a prefix and of own pages that both go through the wide form: the
// cheapest numbers of them by what an item and a join cost, in us for heads of
// 128 elements.  An item costs 8 and, for every 64 tokens, 2.0 where it has a
// CU to itself and 2.9 beside another; 512 run at once.  With more than one
// piece a row there is a join: 6, and the parts' way to memory and back.
// As many pieces as fill the GPU, whatever they cost to join, measured longer:
// 512 new tokens behind 2048 (32 query heads) 103 us, so 53; 1024 new ones 109
// and 91; 700 and no prefix 33 and 29; 512 at the end of 16384 own ones the
// same, 213.  Every row tile counts as if each sequence had max_new rows, so a
// prompt beside single tokens is cut less than alone.
void cut_wide(const kv_paged* p, const kv_step* s, int32_t q_heads, int64_t pre, int64_t own, AttendShape* a)
{
    const double wide = std::max(1.0, p->head_dim / 128.0), tile = wide / 64;
    const int32_t pl = s->prefix.n > 0 ? s->prefix.max_len : 0, ol = std::max(s->own.max_len, 1);
    const double seen = std::max(ol - s->max_new / 2.0, ol / 2.0) / ol;      // of the own tokens, by a row on average
    const WideCuts pc(pre, pl), oc(own, ol);
    double best = 0;
    for (int x = 0; x < pc.n; ++x)
        for (int y = 0; y < oc.n; ++y) {
            const int32_t pp = pc.pieces[x], op = oc.pieces[y];
            const double live = std::min<double>(op, std::max(1.0, op * seen + 0.5));   // own pieces of a tile
            const double pi = double(pre) * pp, oi = double(own) * live;
            const double sum = (8 * (pi + oi) + 2.9 * tile * (double(pre) * pl + double(own) * seen * ol)) / 512;
            // the longest items: beside one another where there are more of them than CUs
            const double last = 8 + tile * std::max((pi > 256 ? 2.9 : 2.0) * (pp > 0 ? pc.tokens[x] : 0),
                                                    (oi * seen > 256 ? 2.9 : 2.0) * oc.tokens[y]);
            double cost = pi + oi <= 512 ? std::max(last, sum) : std::max(last, sum + 0.15 * last);
            if (pp + op > 1) cost += 6 + 2.5e-4 * wide * double(s->n_rows) * q_heads * (pp + op);
            if (best == 0 || cost < best) {
                best = cost;
                a->prefix_pieces = pp;
                a->prefix_tokens = pc.tokens[x];
                a->own_pieces = op;
                a->own_tokens = oc.tokens[y];
            }
        }
}

int attend_shape(const kv_paged* p, const kv_step* s, int32_t q_heads, AttendShape* out)
{
    const int64_t heads = p->num_kv_heads, rep = q_heads / heads;
    AttendShape a{};
    const int64_t pr = s->prefix.n > 0 ? int64_t(s->max_group_rows) * rep : 0, orows = int64_t(s->max_new) * rep;
    a.prefix_wide = pr > kAttendRows;
    a.own_wide = orows > kAttendRows;
    if (a.prefix_wide || a.own_wide) a.blocks = std::max(pr, orows) > 64 && p->head_dim <= 128 ? 2 : 1;
    const int64_t wide_rows = kAttendWaves * 16 * a.blocks;
    const int64_t pt = ceil_div(pr, a.prefix_wide ? wide_rows : kAttendRows);
    const int64_t ot = ceil_div(orows, a.own_wide ? wide_rows : kAttendRows);
    const int64_t most = max_blocks(kAttendBlock);
    if (pt > most || ot > most || s->prefix.n * heads > most || s->own.n * heads > most ||
        s->prefix.n * heads * pt > most || s->own.n * heads * ot > most)
        return fail(KV_EINVAL, "too many row tiles for one launch");
    a.prefix_tiles = int32_t(pt);
    a.own_tiles = int32_t(ot);
    const int64_t pre = s->prefix.n * heads * pt, own = s->own.n * heads * ot;
    // Two workgroups fit a CU, so 512 pieces run at once.  Narrow own pieces alone are cut into 256: a CU's loads in
    // flight are enough from one of them, and there is half as much to join (one 10000-token sequence: 15.1 us, with 128
    // pieces 17.0, with 512 16.7; 24 of them 190, 190, 210).  A wide prefix beside narrow own pieces
    // takes its share of them, so that its pieces, which start first, last as long as the own ones take on the rest of
    // the GPU: the ones wait for the matrix cores, the others for memory.  A token of a narrow piece costs what one of a
    // wide tile does; the own lengths are taken to be a little over half their bound, which holds for ragged batches under
    // an exact bound and is a guess for others.  (32 sequences behind an 8192-token prefix: 58 us, with 256 wide pieces
    // 67, with 512 79; 64 behind two 32768-token ones: 200, 210, 226; inputs not in a cache.)  The own pieces are then cut
    // once more, as sequences of different lengths end at different times (24 ragged ones of up to 10000 tokens 144 us,
    // not cut 177; the 32 sequences 67; but the two documents 183).
    // All pieces are cut by the bounds: lengths far below them leave most pieces empty (10000 tokens under a bound of
    // 10000 15 us, of 32768 20, of 131072 45; eight such sequences 67, 124 and 146).
    const int64_t room = 512, narrow_room = 256;
    const int64_t prefix_work = pre * s->prefix.max_len, own_work = own * s->own.max_len * 6 / 10;
    const bool wide = a.own_wide && (a.prefix_wide || prefix_work == 0);
    const bool beside = a.prefix_wide && !a.own_wide && prefix_work > 0 && own_work > 0;
    const int64_t wide_room =
        beside ? std::max<int64_t>(room / 8, int64_t(double(room) * prefix_work / (double(prefix_work) + own_work)))
               : room;
    cut_tokens(pre, s->prefix.n > 0 ? s->prefix.max_len : 0, wide_room, &a.prefix_tokens, &a.prefix_pieces);
    cut_tokens(own, s->own.n > 0 ? s->own.max_len : 0, beside ? 2 * room : narrow_room, &a.own_tokens, &a.own_pieces);
    if (wide) cut_wide(p, s, q_heads, pre, own, &a);
    a.own_pieces = std::max(1, a.own_pieces);
    a.slots = a.prefix_pieces + a.own_pieces;
    a.direct = a.slots == 1;
    if (pre * a.prefix_pieces + own * a.own_pieces > most)
        return fail(KV_EINVAL, "too many row tiles and pieces for one launch");
    a.prefix_items = pre * a.prefix_pieces;
    a.own_items = own * a.own_pieces;
    const int64_t parts = int64_t(s->n_rows) * q_heads;
    if (parts > (int64_t(1) << 31) / 8) return fail(KV_EINVAL, "too many rows for one launch");
    a.ml_bytes = ceil_div(parts * a.slots * 8, 256) * 256;
    a.bytes = a.ml_bytes + ceil_div(parts * a.slots * p->head_dim * 4, 256) * 256;
    *out = a;
    return KV_OK;
}

int attend_checks(const kv_paged* paged, const kv_step* step, int32_t layer, int32_t q_heads)
{
    int rc = check_step_pool(paged, layer, layer + 1);
    if (rc == KV_OK) rc = check_step(paged, step);
    if (rc == KV_OK) rc = check_heads(paged, q_heads);
    return rc;
}

int check_q(const kv_rows* q, float scale)
{
    if (q == nullptr || q->data == nullptr) return fail(KV_EINVAL, "q is NULL");
    if (!rows_vectors(*q, 2)) return fail(KV_EINVAL, "q's address and strides must be multiples of 16 bytes");
    if (!(scale > 0.0f) || scale > 1e30f) return fail(KV_EINVAL, "scale must be finite and > 0");
    return KV_OK;
}

template <int DP>
KernelFn attend_kernel(int blocks)
{
    if constexpr (DP <= 128)
        if (blocks == 2) return reinterpret_cast<KernelFn>(&attend_pieces<DP, 2>);
    return blocks == 0 ? reinterpret_cast<KernelFn>(&attend_pieces<DP, 0>)
                       : reinterpret_cast<KernelFn>(&attend_pieces<DP, 1>);
}

template <int DP>
KernelFn join_kernel(bool by_row)
{
    return by_row ? reinterpret_cast<KernelFn>(&attend_join_rows<DP>) : reinterpret_cast<KernelFn>(&attend_join<DP>);
}

int attend(const kv_paged* paged, const kv_step* step, int32_t layer, const kv_rows* q, int32_t q_heads, float scale,
           const kv_rows* out, float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    int rc = attend_checks(paged, step, layer, q_heads);
    if (rc != KV_OK) return rc;
    AttendShape sh;
    rc = attend_shape(paged, step, q_heads, &sh);
    if (rc != KV_OK) return rc;
    if (step->n_rows == 0 || step->own.n == 0) return ok();
    rc = check_q(q, scale);
    if (rc != KV_OK) return rc;
    if (out == nullptr || out->data == nullptr || lse == nullptr) return fail(KV_EINVAL, "out or lse is NULL");
    if (misaligned(out->data, 8) || out->row_stride % 4 != 0 || out->head_stride % 4 != 0)
        return fail(KV_EINVAL, "out's address and strides must be multiples of 8 bytes");
    if (rows_overlap(*out, step->n_rows, q_heads, paged->head_dim)) return fail(KV_EINVAL, "out's rows overlap");
    if (workspace == nullptr || workspace_bytes < size_t(sh.bytes) || misaligned(workspace, 256))
        return fail(KV_EINVAL, "workspace of %lld bytes, 256-byte aligned, needed (got %zu at %p)",
                    (long long)sh.bytes, workspace_bytes, workspace);
    if (out->data == q->data) return fail(KV_EINVAL, "out must not be q");
    rc = check_stream(stream);
    if (rc != KV_OK) return rc;
    AttendArgs a{};
    a.pool = pool_arg(paged, layer);
    a.step = step_arg(step);
    a.q = reinterpret_cast<uint64_t>(q->data);
    a.q_row = q->row_stride;
    a.q_head = q->head_stride;
    a.out = reinterpret_cast<uint64_t>(out->data);
    a.o_row = out->row_stride;
    a.o_head = out->head_stride;
    a.lse = reinterpret_cast<uint64_t>(lse);
    a.part_ml = reinterpret_cast<uint64_t>(workspace);
    a.part_acc = a.part_ml + uint64_t(sh.ml_bytes);
    a.q_heads = q_heads;
    a.rep = q_heads / paged->num_kv_heads;
    magic_of(a.rep, &a.rep_magic, &a.rep_shift);
    a.scale_log2 = float(double(scale) * 1.4426950408889634);
    a.prefix_tiles = sh.prefix_tiles;
    a.prefix_pieces = sh.prefix_pieces;
    a.prefix_tokens = sh.prefix_tokens;
    a.own_tiles = sh.own_tiles;
    a.own_pieces = sh.own_pieces;
    a.own_tokens = sh.own_tokens;
    a.slots = sh.slots;
    a.prefix_items = uint32_t(sh.prefix_items);
    a.prefix_wide = sh.prefix_wide;
    a.own_wide = sh.own_wide;
    a.direct = sh.direct;
    const int dim = paged->head_dim;
    KernelFn pieces = dim <= 64    ? attend_kernel<64>(sh.blocks)
                      : dim <= 128 ? attend_kernel<128>(sh.blocks)
                                   : attend_kernel<256>(sh.blocks);
    // Rows enough to fill the GPU: a workgroup a row and some of its heads, so that 4096 of them make up for the
    // shared look-ups' wait.  (512 new tokens behind 2048: by row 53 us, by row and head 72; one token over 10000: 19 and 15.)
    const bool by_row = step->n_rows >= 128;
    KernelFn join = dim <= 64    ? join_kernel<64>(by_row)
                    : dim <= 128 ? join_kernel<128>(by_row)
                                 : join_kernel<256>(by_row);
    rc = launch(pieces, sh.prefix_items + sh.own_items, kAttendBlock, &a, stream);
    if (rc == KV_OK && !sh.direct)
        rc = launch(join, by_row ? step->n_rows : int64_t(step->n_rows) * q_heads, 256, &a, stream,
                    by_row ? unsigned(std::clamp<int64_t>(4096 / step->n_rows, 1, ceil_div(q_heads, 4))) : 1u);
    return rc == KV_OK ? ok() : rc;
}

// ---- weights

template <int DP>
KernelFn weights_kernel(bool rows, int32_t* tokens, int* block)
{
    *tokens = rows ? kRowsTokens : kWeightsTokens;
    *block = rows ? kRowsWaves * 64 : kAttendBlock;
    return rows ? reinterpret_cast<KernelFn>(&add_weights_rows<DP>) : reinterpret_cast<KernelFn>(&add_weights<DP>);
}

int add_weights_call(const kv_paged* paged, const kv_step* step, int32_t layer, const kv_rows* q, const float* lse,
                     int32_t q_heads, float scale, const kv_sums* own, const kv_sums* prefix, hipStream_t stream)
{
    int rc = attend_checks(paged, step, layer, q_heads);
    if (rc != KV_OK) return rc;
    if (own == nullptr && prefix == nullptr) return fail(KV_EINVAL, "own or prefix sums are needed");
    auto check_sums = [](const kv_sums* x, const kv_tables& t, bool may_be_null, const char* what) {
        if (x == nullptr) return int(KV_OK);
        if (x->out == nullptr && !may_be_null) return fail(KV_EINVAL, "%s sums: out is NULL", what);
        if (x->cap < t.max_len)
            return fail(KV_ERANGE, "%s sums: cap %lld below max_len %d", what, (long long)x->cap, t.max_len);
        return int(KV_OK);
    };
    rc = check_sums(own, step->own, holds_nothing(step->own), "own");
    // prefix sums of a step without prefixes stay a mistake
    if (rc == KV_OK) rc = check_sums(prefix, step->prefix, step->prefix.n > 0 && step->prefix.max_len == 0, "prefix");
    if (rc != KV_OK) return rc;
    if (step->n_rows > 0) {
        rc = check_q(q, scale);
        if (rc != KV_OK) return rc;
        if (lse == nullptr) return fail(KV_EINVAL, "lse is NULL");
    }
    rc = check_stream(stream);
    if (rc != KV_OK) return rc;
    WeightsArgs a{};
    a.pool = pool_arg(paged, layer);
    a.step = step_arg(step);
    if (q != nullptr) {
        a.q = reinterpret_cast<uint64_t>(q->data);
        a.q_row = q->row_stride;
        a.q_head = q->head_stride;
    }
    a.lse = reinterpret_cast<uint64_t>(lse);
    a.q_heads = q_heads;
    a.rep = q_heads / paged->num_kv_heads;
    magic_of(a.rep, &a.rep_magic, &a.rep_shift);
    a.scale_log2 = float(double(scale) * 1.4426950408889634);
    // Many rows: the waves share a workgroup's tokens and split the rows.  (4 sequences of 4000 tokens, 4 heads a KV
    // head: 32 new tokens 23 us, split 30; 64 new ones 38 and 34; 256 126 and 65.)
    const int64_t rows = std::max(own != nullptr ? step->max_new : 0, prefix != nullptr ? step->max_group_rows : 0);
    if (rows * a.rep > INT32_MAX - 2 * kStageRows) return fail(KV_EINVAL, "too many rows for one launch");
    const bool split = rows * a.rep > 192;
    const int dim = paged->head_dim;
    int32_t tokens = 0;
    int block = 0;
    KernelFn f = dim <= 64    ? weights_kernel<64>(split, &tokens, &block)
                 : dim <= 128 ? weights_kernel<128>(split, &tokens, &block)
                              : weights_kernel<256>(split, &tokens, &block);
    int64_t own_items = 0, prefix_items = 0;
    if (own != nullptr) {
        a.own_in = reinterpret_cast<uint64_t>(own->in);
        a.own_out = reinterpret_cast<uint64_t>(own->out);
        a.own_cap = own->cap;
        a.own_blocks = int32_t(ceil_div(step->own.max_len, tokens));
        own_items = int64_t(step->own.n) * paged->num_kv_heads * a.own_blocks;
    }
    if (prefix != nullptr) {
        a.prefix_in = reinterpret_cast<uint64_t>(prefix->in);
        a.prefix_out = reinterpret_cast<uint64_t>(prefix->out);
        a.prefix_cap = prefix->cap;
        a.prefix_blocks = int32_t(ceil_div(step->prefix.max_len, tokens));
        prefix_items = int64_t(step->prefix.n) * paged->num_kv_heads * a.prefix_blocks;
    }
    const int64_t most = max_blocks(block);
    if (own_items > most || prefix_items > most) return fail(KV_EINVAL, "too many tokens for one launch");
    a.prefix_items = uint32_t(prefix_items);
    rc = launch(f, prefix_items + own_items, block, &a, stream);
    return rc == KV_OK ? ok() : rc;
}

// ---- evict

struct EvictShape {
    int64_t jobs, max_moves, count_bytes, bytes;
};

int evict_shape(const kv_paged* p, const kv_tables* t, int32_t n_layers, int32_t heads, int32_t keep, EvictShape* out)
{
    if (t == nullptr) return fail(KV_EINVAL, "tables is NULL");
    int rc = check_tables(p, t, "tables");
    if (rc != KV_OK) return rc;
    if (heads != 1 && heads != p->num_kv_heads)
        return fail(KV_EINVAL, "heads must be 1 or num_kv_heads (got %d)", heads);
    if (int64_t(p->num_kv_heads) * p->head_dim / heads % 8 != 0)
        return fail(KV_EINVAL, "head_dim = %d must be a multiple of 8 to evict by head", p->head_dim);
    if (keep < 0) return fail(KV_EINVAL, "keep < 0");
    out->jobs = int64_t(n_layers) * t->n * heads;
    if (out->jobs > max_blocks(kSelectBlock)) return fail(KV_EINVAL, "too many (layer, sequence, head) for one launch");
    out->max_moves = std::min<int64_t>(keep, std::max(0, t->max_len - keep));
    // vectors of a row's moves are numbered in 31 bits
    const int64_t vecs = int64_t(p->num_kv_heads) * p->head_dim / heads / 8;
    if (out->max_moves * vecs > INT32_MAX - kSelectBlock * kMoveRowsPer)
        return fail(KV_EINVAL, "%lld moves of %lld bytes: too many for one call", (long long)out->max_moves,
                    (long long)(vecs * 16));
    out->count_bytes = ceil_div(out->jobs * 4, 256) * 256;
    out->bytes = out->count_bytes + ceil_div(out->jobs * out->max_moves * 8, 256) * 256;
    return KV_OK;
}

int evict(const kv_paged* paged, const kv_tables* tables, int32_t layer_begin, int32_t layer_end, const kv_slots* in,
          const kv_slots* out, int32_t keep, int32_t recent, int32_t* out_lens, void* workspace,
          size_t workspace_bytes, hipStream_t stream)
{
    int rc = check_step_pool(paged, layer_begin, layer_end);
    if (rc != KV_OK) return rc;
    if (in == nullptr || out == nullptr) return fail(KV_EINVAL, "in or out is NULL");
    EvictShape sh;
    rc = evict_shape(paged, tables, layer_end - layer_begin, in->heads, keep, &sh);
    if (rc != KV_OK) return rc;
    if (recent < 0 || recent > keep) return fail(KV_EINVAL, "need 0 <= recent <= keep (got %d, %d)", recent, keep);
    if (out->heads != in->heads) return fail(KV_EINVAL, "in and out must have the same heads");
    if (tables->n == 0) return ok();
    const int32_t kept = std::min(keep, tables->max_len);
    if (out_lens == nullptr || (tables->max_len > 0 && (in->weights == nullptr || in->positions == nullptr)) ||
        (kept > 0 && (out->weights == nullptr || out->positions == nullptr)))
        return fail(KV_EINVAL, "weights, positions or out_lens is NULL");
    if (out_lens == tables->lens) return fail(KV_EINVAL, "out_lens must not be the lengths that are read");
    if ((in->weights == out->weights) != (in->positions == out->positions))
        return fail(KV_EINVAL, "weights and positions are both updated in place or both written elsewhere");
    if (in->weights == out->weights && in->cap != out->cap)
        return fail(KV_EINVAL, "in place, in and out must have the same cap");
    if (in->cap < tables->max_len)
        return fail(KV_ERANGE, "cap %lld below max_len %d", (long long)in->cap, tables->max_len);
    if (out->cap < kept)
        return fail(KV_ERANGE, "out's cap %lld below the %d slots kept", (long long)out->cap, kept);
    if (workspace == nullptr || workspace_bytes < size_t(sh.bytes) || misaligned(workspace, 256))
        return fail(KV_EINVAL, "workspace of %lld bytes, 256-byte aligned, needed (got %zu at %p)",
                    (long long)sh.bytes, workspace_bytes, workspace);
    rc = check_stream(stream);
    if (rc != KV_OK) return rc;
    EvictArgs a{};
    a.pool = pool_arg(paged, layer_begin);
    a.tab = tables_arg(tables);
    a.weights = reinterpret_cast<uint64_t>(in->weights);
    a.positions = reinterpret_cast<uint64_t>(in->positions);
    a.out_weights = reinterpret_cast<uint64_t>(out->weights);
    a.out_positions = reinterpret_cast<uint64_t>(out->positions);
    a.cap = in->cap;
    a.out_cap = out->cap;
    a.out_lens = reinterpret_cast<uint64_t>(out_lens);
    a.counts = reinterpret_cast<uint64_t>(workspace);
    a.moves = a.counts + uint64_t(sh.count_bytes);
    a.heads = in->heads;
    a.n_layers = layer_end - layer_begin;
    a.keep = keep;
    a.recent = recent;
    a.max_moves = int32_t(sh.max_moves);
    a.vecs = uint32_t(int64_t(paged->num_kv_heads) * paged->head_dim / in->heads / 8);
    magic_of(int32_t(a.vecs), &a.vec_magic, &a.vec_shift);
    a.fused = sh.max_moves <= kFusedMoves;
    // keys in LDS: as little of it as the bound needs, so that several workgroups fit a CU
    const int32_t len = tables->max_len;
    const KernelFn select = len <= 4096    ? reinterpret_cast<KernelFn>(&evict_select<4096>)
                            : len <= 12288 ? reinterpret_cast<KernelFn>(&evict_select<12288>)
                                           : reinterpret_cast<KernelFn>(&evict_select<32768>);
    rc = launch(select, sh.jobs, kSelectBlock, &a, stream);
    if (rc == KV_OK && sh.max_moves > 0 && !a.fused) {
        const int64_t shares = ceil_div(sh.max_moves * a.vecs, kMoveRowsBlock * kMoveRowsPer);
        rc = launch(reinterpret_cast<KernelFn>(&evict_move), sh.jobs, kMoveRowsBlock, &a, stream,
                    unsigned(std::min<int64_t>(shares, 256)));
    }
    return rc == KV_OK ? ok() : rc;
}

}  // namespace

extern "C" {

int kv_append(const kv_paged* paged, const kv_step* step, int32_t layer, const kv_rows* q, const kv_rows* k,
              const kv_rows* v, const kv_rows* q_out, int32_t q_heads, kv_type type, kv_type q_out_type,
              const int32_t* positions, const kv_rope* rope, const kv_slots* slots, hipStream_t stream)
{
    return append(paged, step, layer, q, k, v, q_out, q_heads, type, q_out_type, positions, rope, slots, stream);
}

size_t kv_attend_workspace_bytes(const kv_paged* paged, const kv_step* step, int32_t q_heads)
{
    AttendShape sh;
    if (attend_checks(paged, step, 0, q_heads) != KV_OK || attend_shape(paged, step, q_heads, &sh) != KV_OK) return 0;
    ok();
    return size_t(std::max<int64_t>(sh.bytes, 256));
}

int kv_attend(const kv_paged* paged, const kv_step* step, int32_t layer, const kv_rows* q, int32_t q_heads,
              float scale, const kv_rows* out, float* lse, void* workspace, size_t workspace_bytes,
              hipStream_t stream)
{
    return attend(paged, step, layer, q, q_heads, scale, out, lse, workspace, workspace_bytes, stream);
}

int kv_add_weights(const kv_paged* paged, const kv_step* step, int32_t layer, const kv_rows* q, const float* lse,
                   int32_t q_heads, float scale, const kv_sums* own, const kv_sums* prefix, hipStream_t stream)
{
    return add_weights_call(paged, step, layer, q, lse, q_heads, scale, own, prefix, stream);
}

size_t kv_evict_workspace_bytes(const kv_paged* paged, const kv_tables* tables, int32_t n_layers, int32_t heads,
                                int32_t keep)
{
    EvictShape sh;
    if (check_paged(paged) != KV_OK) return 0;
    if (n_layers <= 0 || n_layers > paged->num_layers) {
        fail(KV_EINVAL, "n_layers = %d outside [1, %d]", n_layers, paged->num_layers);
        return 0;
    }
    if (evict_shape(paged, tables, n_layers, heads, keep, &sh) != KV_OK) return 0;
    ok();
    return size_t(std::max<int64_t>(sh.bytes, 256));
}

int kv_evict(const kv_paged* paged, const kv_tables* tables, int32_t layer_begin, int32_t layer_end,
             const kv_slots* in, const kv_slots* out, int32_t keep, int32_t recent, int32_t* out_lens,
             void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return evict(paged, tables, layer_begin, layer_end, in, out, keep, recent, out_lens, workspace, workspace_bytes,
                 stream);
}

}  // extern "C"
