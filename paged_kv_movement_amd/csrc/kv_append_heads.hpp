// kv_append_heads.hpp -- append with each head of q and k normalised before it
// is rotated, and append into an 8-bit pool.
//
// Norm: y = (x - c) / sqrt(mean((x - c)^2) + eps) * w over a head's elements,
// c = 0 or their mean.  The sums are float32, two passes over registers for the
// centered form (mean of squares less square of mean would cancel); where the
// squares leave float32's range the head is first scaled by a power of two.
// Then the rotation of kv_append.hpp, and one rounding.  Keys on their way into
// 8 bits go through all of it in 64 bits (see above wide_norm).
//
// A head lies in a group of G lanes, the next power of two to its units, so
// that its sums are exchanges within a wave and no head waits for another.
//
// append_heads_rows   one workgroup per token, for q (and, into a bf16 pool, k
//                     and v).  Bound: memory, as append_rows: 45116 tokens of
//                     32 query heads and 8 KV heads of 128 in 222 us, 5.0 TB/s
//                     (without a norm 200; fp16 251, float32, nearly twice the
//                     bytes, 381); one token in 5.7 us, of which 1.9 are the
//                     weights and the two sums.  Element by element (rot 20 of
//                     128) 1025 us.
// append8_rows        those workgroups for q, and behind them one per (sequence,
//                     page, some of the heads) for k and v: a wave takes one
//                     head's K or V of the page, all its new tokens, finds the
//                     block's scale and writes the bytes.
#pragma once

#include "kv_append.hpp"
#include "kv_pool8.hpp"

namespace kvmove {

enum : int { kNormNone = 0, kNormRms = 1, kNormCentered = 2 };

constexpr int kMaxShared = 512;        // weights of a head kept in LDS where all heads share them

struct NormArg {
    uint64_t q_weight, k_weight;       // float32 [heads][dim], or 0: ones
    int64_t q_stride, k_stride;        // elements from head to head
    int32_t kind;
    float eps;
};

struct AppendHeadsArgs {
    AppendArgs a;
    NormArg norm;
    ScalesArg scales;                  // of an 8-bit pool
    int32_t lanes_log2, per;           // lanes G of a head of q or k, its units of a lane: one with vectors
    int32_t v_units, v_lanes_log2, v_per;   // append8: the same for a head of v, in units of two vectors
    uint32_t token_items;              // append8: workgroups [0, token_items) take a token's q
    int32_t pages, splits;             // append8: pages of a sequence, workgroups that share a page's heads
    int32_t angles;                    // append8: angles that LDS has room for, a token's at least
};

__device__ __forceinline__ float sum_over(float x, int lanes)
{
    for (int d = 1; d < lanes; d *= 2) x += __shfl_xor(x, d);
    return x;
}

__device__ __forceinline__ float max_over(float x, int lanes)
{
    for (int d = 1; d < lanes; d *= 2) x = __builtin_fmaxf(x, __shfl_xor(x, d));
    return x;
}

// A unit's two vectors as they lie in memory; without a second one, the first again.
template <class TI, int kVec>
struct RawUnit {
    Vec<TI, kVec> x, y;
};

template <class TI, int kVec>
__device__ __forceinline__ RawUnit<TI, kVec> load_raw(const TI* head, const Unit& u)
{
    return {*reinterpret_cast<const Vec<TI, kVec>*>(head + u.d0), *reinterpret_cast<const Vec<TI, kVec>*>(head + u.d1)};
}

// The same as float32; n of the 2 kVec elements count, the others are 0.
template <int kVec>
struct Values {
    float x[2 * kVec];
};

template <class TI, int kVec>
__device__ __forceinline__ Values<kVec> values_of(const RawUnit<TI, kVec>& r, const Unit& u, bool live)
{
    Values<kVec> v;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        v.x[i] = live ? float(r.x.x[i]) : 0.0f;
        v.x[kVec + i] = live && u.kind == kUnitPairs ? float(r.y.x[i]) : 0.0f;
    }
    return v;
}

__device__ __forceinline__ int values_in(const Unit& u, int vec, bool live)
{
    return !live ? 0 : u.kind == kUnitPairs ? 2 * vec : vec;
}

// What a head is normalised with: x * r - c.
struct HeadNorm {
    float r, c;
};

// Of a group of lanes: each(f) calls f with every (values, number of them that
// count) of the lane's units.  v: its first unit's.  Squares that leave float32
// are rare, and looked for in their sum: such a head is done again, its values
// brought near 1 by a power of two, v's too (below 1 only where eps does not
// outweigh the squares anyway, and no further than eps stays finite).  A head
// with an infinity or a NaN takes the formula as it is.
template <int kVec, class Each>
__device__ __forceinline__ HeadNorm head_norm(const NormArg& n, int dim, int lanes, Values<kVec>& v, float& scale,
                                              Each&& each)
{
    const float inv_dim = 1.0f / float(dim);
    auto sums = [&](float s, float& mean, float& squares) {
        mean = 0.0f;
        if (n.kind == kNormCentered) {
            each([&](const Values<kVec>& x, int count) {
#pragma unroll
                for (int i = 0; i < 2 * kVec; ++i) mean = __builtin_fmaf(x.x[i], s, mean);
            });
            mean = sum_over(mean, lanes) * inv_dim;
        }
        squares = 0.0f;
        each([&](const Values<kVec>& x, int count) {
            if (n.kind == kNormCentered) {
#pragma unroll
                for (int i = 0; i < 2 * kVec; ++i) {
                    const float d = i < count ? __builtin_fmaf(x.x[i], s, -mean) : 0.0f;
                    squares = __builtin_fmaf(d, d, squares);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2 * kVec; ++i) {
                    const float d = x.x[i] * s;
                    squares = __builtin_fmaf(d, d, squares);
                }
            }
        });
        squares = sum_over(squares, lanes);
    };
    float mean, squares;
    sums(1.0f, mean, squares);
    scale = 1.0f;
    const bool far = !(squares < 0x1p120f) || (squares < 0x1p-90f && n.eps < 0x1p-96f);
    if (__any(far)) {
        float big = 0.0f;
        bool odd = false;
        each([&](const Values<kVec>& x, int count) {
#pragma unroll
            for (int i = 0; i < 2 * kVec; ++i) {
                const float a = __builtin_fabsf(x.x[i]);
                odd = odd || !(a < __builtin_inff());
                big = __builtin_fmaxf(big, a);
            }
        });
        big = max_over(odd ? __builtin_inff() : big, lanes);
        if (far && big < __builtin_inff())
            scale = exp2_int(clamp_i32(127 - int(__float_as_uint(big) >> 23), -126, n.eps == 0.0f ? 126 : 60));
        sums(scale, mean, squares);
#pragma unroll
        for (int i = 0; i < 2 * kVec; ++i) v.x[i] *= scale;
    }
    const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(squares, inv_dim, n.eps * scale * scale));
    return {r, mean * r};
}

// Weights that all heads of q, all heads of k share, in LDS (ones where there are none).
struct SharedWeights {
    alignas(16) float w[2][kMaxShared];
};

__device__ __forceinline__ bool weights_shared(const NormArg& n, bool k, int dim)
{
    return ((k ? n.k_weight : n.q_weight) == 0 || (k ? n.k_stride : n.q_stride) == 0) && dim <= kMaxShared;
}

// For all threads; a barrier has to follow.
__device__ __forceinline__ void share_weights(const NormArg& n, int dim, SharedWeights& sh)
{
    if (n.kind == kNormNone) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint64_t base = k ? n.k_weight : n.q_weight;
        if (weights_shared(n, k != 0, dim))
            for (int d = threadIdx.x; d < dim; d += kAppendBlock) sh.w[k][d] = base == 0 ? 1.0f : gptr<const gf32>(base)[d];
    }
}

// Weights of a unit of head `head` of q or k.
template <int kVec>
__device__ __forceinline__ RawUnit<float, kVec> weights_of_unit(const NormArg& n, bool k, int head, const Unit& u,
                                                                int dim, const SharedWeights& sh)
{
    RawUnit<float, kVec> w;
    if (weights_shared(n, k, dim))
        w = load_raw<float, kVec>(sh.w[k ? 1 : 0], u);
    else if ((k ? n.k_weight : n.q_weight) != 0)
        w = load_raw<float, kVec>(reinterpret_cast<const float*>(k ? n.k_weight : n.q_weight) +
                                      head * (k ? n.k_stride : n.q_stride), u);
    else
#pragma unroll
        for (int i = 0; i < kVec; ++i) w.x.x[i] = w.y.x[i] = 1.0f;
    return w;
}

// The unit of head `head` of q or k, its values scaled as head_norm says, normalised.
template <int kVec>
__device__ __forceinline__ void normalise(Values<kVec>& v, const HeadNorm& h, const NormArg& n, bool k, int head,
                                          const Unit& u, int dim, const SharedWeights& sh)
{
    const RawUnit<float, kVec> w = weights_of_unit<kVec>(n, k, head, u, dim, sh);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        v.x[i] = __builtin_fmaf(v.x[i], h.r, -h.c) * w.x.x[i];
        v.x[kVec + i] = __builtin_fmaf(v.x[kVec + i], h.r, -h.c) * w.y.x[i];
    }
}

// The unit rotated; angle(i): cosine and sine of its i-th pair, 1 and 0 for a
// unit that passes.  Not in place: the compiler would keep the values in memory.
template <int kVec, bool kInterleaved, class Angle>
__device__ __forceinline__ Values<kVec> rotated(const Values<kVec>& v, const Unit& u, int rot, Angle&& angle)
{
    Values<kVec> o = v;
    if constexpr (kVec == 1 || !kInterleaved) {              // one that passes has no second vector: 0
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const float2 c = angle(i);
            o.x[i] = __builtin_fmaf(v.x[i], c.x, -(v.x[kVec + i] * c.y));
            o.x[kVec + i] = __builtin_fmaf(v.x[kVec + i], c.x, v.x[i] * c.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
            // the vector may lie across the end of what turns; there an infinity's pair would get its product with 0
            const bool turns = u.d0 + i < rot;
            const float2 c = angle(i / 2);
            const float a = __builtin_fmaf(v.x[i], c.x, -(v.x[i + 1] * c.y));
            const float b = __builtin_fmaf(v.x[i + 1], c.x, v.x[i] * c.y);
            o.x[i] = turns ? a : v.x[i];
            o.x[i + 1] = turns ? b : v.x[i + 1];
        }
    }
    return o;
}

template <int kVec, class Angle>
__device__ __forceinline__ Values<kVec> rotated(const AppendArgs& a, const Values<kVec>& v, const Unit& u, Angle&& angle)
{
    return a.interleaved != 0 ? rotated<kVec, true>(v, u, a.rot, angle) : rotated<kVec, false>(v, u, a.rot, angle);
}

// LDS for angles begins with the ones of a unit that passes, and ends with room
// for a vector's that lies across the end of what turns.
constexpr int kPassAngles = 8, kAngleRoom = kPassAngles + 4;

__device__ __forceinline__ void put_pass_angles(float2* cs)
{
    if (threadIdx.x < kPassAngles) cs[threadIdx.x] = {1.0f, 0.0f};
}

__device__ __forceinline__ const float2* angles_at(const float2* cs, const Unit& u, int first)
{
    return u.kind == kUnitPass ? cs : cs + kPassAngles + first + u.pair;
}

// Cosine and sine of pair j at a position, formed as kv_append.hpp says.
__device__ __forceinline__ float2 angle_of(const AppendArgs& a, int32_t pos, int j)
{
    const double turns_per_radian = 0.15915494309189533577;
    const double f = gptr<const __attribute__((address_space(1))) double>(a.freqs)[j];
    const double turns = double(pos) * (f * turns_per_radian);
    const float frac = float(turns - __builtin_rint(turns));
    float sn, cn;
    sincospif(2.0f * frac, &sn, &cn);
    return {cn * a.gain, sn * a.gain};
}

template <class TO, int kVec>
__device__ __forceinline__ void put_values(TO* head, const Unit& u, const Values<kVec>& v)
{
    Vec<TO, kVec> x, y;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        x.x[i] = TO(v.x[i]);
        y.x[i] = TO(v.x[kVec + i]);
    }
    *reinterpret_cast<Vec<TO, kVec>*>(head + u.d0) = x;
    if (u.kind == kUnitPairs) *reinterpret_cast<Vec<TO, kVec>*>(head + u.d1) = y;
}

// One token: its heads of q, and with kKv those of k and its v, into a bf16
// pool.  cs: room for its angles.  As in append_rows, the first heads' values
// are asked for before the owner, the page and the angles are known.
template <class TI, class TO, int kVec, bool kKv>
__device__ __forceinline__ void token_heads(const AppendHeadsArgs& h, int32_t r, float2* cs, SharedWeights& sh)
{
    constexpr int kAhead = 2;                      // heads of a lane in flight
    const AppendArgs& a = h.a;
    const int32_t tid = threadIdx.x;
    const int dim = a.pool.dim, kv_heads = kKv ? a.pool.heads : 0, lanes = 1 << h.lanes_log2;
    const int heads = a.q_heads + kv_heads, stride = kAppendBlock >> h.lanes_log2;
    const int first = tid >> h.lanes_log2, lane = tid & (lanes - 1);
    auto source = [&](int head) {
        const bool k = head >= a.q_heads;
        return reinterpret_cast<const TI*>(k ? a.k : a.q) + r * (k ? a.k_row : a.q_row) +
               (k ? head - a.q_heads : head) * (k ? a.k_head : a.q_head);
    };
    auto unit = [&](int i) { return head_unit<kVec>(i < a.units ? i : 0, a.rot, a.interleaved != 0); };
    auto norm = [&](Values<kVec>& v, const HeadNorm& n, int head, const Unit& u) {
        const bool k = head >= a.q_heads;
        normalise<kVec>(v, n, h.norm, k, k ? head - a.q_heads : head, u, dim, sh);
    };
    const Unit u0 = unit(lane);
    RawUnit<TI, kVec> raw[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
        const int head = first + x * stride;
        if (head >= heads) continue;
        raw[x] = load_raw<TI, kVec>(source(head), u0);
    }
    Vec<TI, kVec> v{};
    const int v_vectors = kv_heads * (dim / kVec);
    auto v_at = [&](int i) {
        const int head = int((uint64_t(uint32_t(i)) * a.vec_magic) >> a.vec_shift);
        return reinterpret_cast<const TI*>(a.v) + r * a.v_row + head * a.v_head + (i - head * (dim / kVec)) * kVec;
    };
    if (tid < v_vectors) v = *reinterpret_cast<const Vec<TI, kVec>*>(v_at(tid));
    const int32_t pos = gptr<const gi32>(a.positions)[r];
    uint64_t kd = 0, vd = 0;
    int32_t slot = 0, s = -1;
    if constexpr (kKv) {
        // where k and v go; 0: nowhere (a row of no sequence, no slot left, a bad page)
        const uint64_t kb = gptr<const gu64>(a.pool.k_pages)[a.pool.layer];
        const uint64_t vb = gptr<const gu64>(a.pool.v_pages)[a.pool.layer];
        const RowOwner o = row_owner(a.step, r);
        s = o.s;
        slot = o.len - o.count + (r - o.first);
        if (o.s >= 0 && slot >= 0) {
            const uint32_t pi = page_of(a.pool, uint32_t(slot));
            const int32_t page = gptr<const gi32>(a.step.own.table)[o.s * a.step.own.stride + pi];
            if (uint32_t(page) >= a.pool.num_pages) {
                raise_fault(kFaultPage);
            } else if (bad_addr(kb) || bad_addr(vb)) {
                raise_fault(kFaultPool);
            } else {
                const int64_t row = int64_t(page) * a.pool.page_size + (uint32_t(slot) - pi * a.pool.page_size);
                kd = kb + uint64_t(row) * a.pool.heads * dim * 2;
                vd = vb + uint64_t(row) * a.pool.heads * dim * 2;
            }
        }
    }
    share_weights(h.norm, dim, sh);
    put_pass_angles(cs);
    for (int j = tid; j < a.rot / 2; j += kAppendBlock) cs[kPassAngles + j] = angle_of(a, pos, j);
    __syncthreads();
    auto finish = [&](int head, const RawUnit<TI, kVec>& r0) {
        const TI* src = source(head);
        const bool live = lane < a.units;
        auto put = [&](const Unit& u, const Values<kVec>& y) {
            const float2* angles = angles_at(cs, u, 0);
            const Values<kVec> x = rotated<kVec>(a, y, u, [&](int j) { return angles[j]; });
            if (head < a.q_heads)
                put_values<TO, kVec>(reinterpret_cast<TO*>(a.q_out) + r * a.o_row + head * a.o_head, u, x);
            else if (kd != 0)
                put_values<__bf16, kVec>(reinterpret_cast<__bf16*>(kd) + (head - a.q_heads) * dim, u, x);
        };
        Values<kVec> x0 = values_of<TI, kVec>(r0, u0, live);
        HeadNorm n{};
        float scale = 1.0f;
        if (h.norm.kind != kNormNone) {
            n = head_norm<kVec>(h.norm, dim, lanes, x0, scale, [&](auto&& f) {
                f(x0, values_in(u0, kVec, live));
                if constexpr (kVec > 1) return;
                for (int i = lane + lanes; i < h.per * lanes; i += lanes) {
                    const Unit u = unit(i);
                    f(values_of<TI, kVec>(load_raw<TI, kVec>(src, u), u, i < a.units), values_in(u, kVec, i < a.units));
                }
            });
            norm(x0, n, head, u0);
        }
        if (live) put(u0, x0);
        if constexpr (kVec > 1) return;
        for (int i = lane + lanes; i < a.units; i += lanes) {
            const Unit u = unit(i);
            Values<kVec> x = values_of<TI, kVec>(load_raw<TI, kVec>(src, u), u, true);
            if (h.norm.kind != kNormNone) {
#pragma unroll
                for (int e = 0; e < 2 * kVec; ++e) x.x[e] *= scale;
                norm(x, n, head, u);
            }
            put(u, x);
        }
    };
    // the lanes of a head go through this together, whatever the wave's other heads do
    for (int base = 0; base < heads; base += kAhead * stride) {
        if (base > 0)
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int head = base + first + x * stride;
                if (head >= heads) continue;
                raw[x] = load_raw<TI, kVec>(source(head), u0);
            }
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
            if (base + first + x * stride < heads) finish(base + first + x * stride, raw[x]);
    }
    if (kd == 0) return;
    for (int i = tid; i < v_vectors; i += kAppendBlock) {
        if (i != tid) v = *reinterpret_cast<const Vec<TI, kVec>*>(v_at(i));
        Vec<__bf16, kVec> o;
#pragma unroll
        for (int e = 0; e < kVec; ++e) o.x[e] = __bf16(float(v.x[e]));
        *reinterpret_cast<Vec<__bf16, kVec>*>(reinterpret_cast<__bf16*>(vd) + i * kVec) = o;
    }
    if (a.weights != 0)
        for (int x = tid; x < a.w_heads; x += kAppendBlock) {
            const int64_t at = (int64_t(s) * a.w_heads + x) * a.w_cap + slot;
            gptr<gf32>(a.weights)[at] = 0.0f;
            gptr<gi32>(a.slot_positions)[at] = pos;
        }
}

template <class TI, class TO, int kVec, bool kKv>
__global__ __launch_bounds__(kAppendBlock) void append_heads_rows(AppendHeadsArgs h)
{
    __shared__ float2 cs[kAngleRoom + kMaxRot / 2];
    __shared__ SharedWeights sh;
    token_heads<TI, TO, kVec, kKv>(h, blockIdx.x, cs, sh);
}

// ---- keys and values of an 8-bit pool
//
// A byte keeps four bits, so a key that is off by the last bit of a float32
// falls on the other side of a border, a 16th of it away, once in 10^6; a
// block's scale does so by a factor of two.  k is therefore normalised and
// rotated in 64 bits, and becomes a float32 only by rounding to odd, which
// leaves it on its own side of every border of fewer bits: the bytes and
// scales are those of the formula.  (v is what it was.)  Of 45116 tokens the
// pages' part takes 115 us so and took 90 with keys in float32.

template <int kVec>
struct WideValues {
    double x[2 * kVec];
};

template <class TI, int kVec>
__device__ __forceinline__ WideValues<kVec> wide_values_of(const RawUnit<TI, kVec>& r, const Unit& u, bool live)
{
    const Values<kVec> v = values_of<TI, kVec>(r, u, live);
    WideValues<kVec> w;
#pragma unroll
    for (int i = 0; i < 2 * kVec; ++i) w.x[i] = double(v.x[i]);
    return w;
}

__device__ __forceinline__ double sum_over(double x, int lanes)
{
    for (int d = 1; d < lanes; d *= 2) x += __shfl_xor(x, d);
    return x;
}

// (mean, 1 / sqrt(mean square + eps)) of a head; each as for head_norm.  No square of a float32 leaves 64 bits.
template <int kVec, class Each>
__device__ __forceinline__ double2 wide_norm(const NormArg& n, int dim, int lanes, Each&& each)
{
    double mean = 0.0, squares = 0.0;
    if (n.kind == kNormCentered) {
        each([&](const WideValues<kVec>& x, int count) {
#pragma unroll
            for (int i = 0; i < 2 * kVec; ++i) mean += x.x[i];
        });
        mean = sum_over(mean, lanes) / double(dim);
    }
    each([&](const WideValues<kVec>& x, int count) {
#pragma unroll
        for (int i = 0; i < 2 * kVec; ++i) {
            const double d = i < count ? x.x[i] - mean : 0.0;
            squares = __builtin_fma(d, d, squares);
        }
    });
    return {mean, 1.0 / __builtin_sqrt(sum_over(squares, lanes) / double(dim) + double(n.eps))};
}

// Cosine and sine of an angle in turns.
__device__ __forceinline__ double2 wide_angle(double turns)
{
    double sn, cn;
    sincospi(2.0 * (turns - __builtin_rint(turns)), &sn, &cn);
    return {cn, sn};
}

// float32 by rounding to odd: towards 0, and the last bit set where that lost
// something.  What is beyond float32 becomes its largest value (infinity's bits
// less one); NaN and infinities stay.
__device__ __forceinline__ float to_odd(double x)
{
    const float f = float(x);
    const double back = double(f);
    const uint32_t u = __float_as_uint(f), down = __builtin_fabs(back) > __builtin_fabs(x) ? u - 1u : u;
    return __uint_as_float(back != x ? down | 1u : u);
}

constexpr int kPageAngles = 4096;      // angles of a page's new tokens in LDS at once, 16 bytes each
constexpr int kChunkHeads = 64;        // heads of a workgroup at most where that is not all of them
constexpr int kHeldUnits = 2;          // units of a lane kept between the look for the scale and the bytes

// New tokens of one page of a sequence, some of its heads: a wave takes one head's K or V at a time.
//
// Bound: 64-bit arithmetic, and waits.  The vector units work 63 % of the cycles, and with 163 registers there are three
// waves a SIMD to hide the rest, which wait 48 % of their time: 45116 tokens of 8 KV heads of 128 (277 MB) in 115 us,
// 2.4 TB/s; one token of each of 64 sequences 8.3 us with its q.  Asking for the next task's values while one is worked on,
// or for the first ahead of the angles, took as long, as did angles without bank conflicts; rounding to odd is 7 us of it
// and the sines 1.5.  The whole call takes 232 us with pages of 16 tokens, 255 of 32, 270 of 64, 421 of 128 (whose angles
// do not fit and are made twice); in float32 392.
template <class TI, int kVec>
__device__ __forceinline__ void page_heads(const AppendHeadsArgs& h, uint32_t item, double2* cs, SharedWeights& sh)
{
    __shared__ float found_by[2][kAppendBlock / 64];
    const AppendArgs& a = h.a;
    const PoolArg& p = a.pool;
    const int dim = p.dim, half = a.rot / 2, lane = threadIdx.x & 63;
    const int split = int(item % uint32_t(h.splits)), at = int(item / uint32_t(h.splits));
    const int32_t s = at / h.pages;
    const Rows rows = seq_rows(a.step, s);
    const int32_t len = table_len(a.step.own, s);
    const int32_t ahead = len - rows.count, begin = ahead < 0 ? 0 : ahead;       // slots before the new tokens
    const int32_t pi = int32_t(page_of(p, uint32_t(begin))) + (at - s * h.pages);
    const int64_t slot0 = int64_t(pi) * p.page_size;                             // may be far past len
    if (rows.count == 0 || slot0 >= len) return;
    const int32_t lo = slot0 > begin ? int32_t(slot0) : begin;
    const int32_t hi = len - slot0 < p.page_size ? len : int32_t(slot0) + int32_t(p.page_size);
    const int n = hi - lo, old = lo - int32_t(slot0);
    const int64_t row0 = rows.first + int64_t(lo - ahead);
    const int32_t page = __builtin_amdgcn_readfirstlane(gptr<const gi32>(a.step.own.table)[s * a.step.own.stride + pi]);
    const LayerAt l = layer_at<true>(p, h.scales);
    if (uint32_t(page) >= p.num_pages) {
        raise_fault(kFaultPage);
        return;
    }
    if (bad_layer<true>(l)) {
        raise_fault(kFaultPool);
        return;
    }
    const int heads = (int(p.heads) + h.splits - 1) / h.splits, h0 = split * heads;
    const int h1 = h0 + heads < int(p.heads) ? h0 + heads : int(p.heads);
    // Angles of new tokens [c0, c0 + count), times the gain: a thread takes a pair over a run of tokens, and where their
    // positions follow one another it turns on by one position's angle, which is 4 operations for the 100 of a new one.
    auto fill = [&](int c0, int count) {
        if (half == 0) return;
        const double turns_per_radian = 0.15915494309189533577, gain = double(a.gain);
        const int shares = kAppendBlock / half < 1 ? 1 : kAppendBlock / half < count ? kAppendBlock / half : count;
        const int run = (count + shares - 1) / shares, share = int(threadIdx.x) / half;
        const int t0 = share * run, t1 = t0 + run < count ? t0 + run : count;
        if (share >= shares) return;
        const int j = int(threadIdx.x) - share * half;
        const double f = gptr<const __attribute__((address_space(1))) double>(a.freqs)[j] * turns_per_radian;
        const double2 step = wide_angle(f);
        double2 c{};
        int32_t last = 0;
        for (int t = t0; t < t1; ++t) {
            const int32_t pos = gptr<const gi32>(a.positions)[row0 + c0 + t];
            if (t > t0 && int64_t(pos) == int64_t(last) + 1)
                c = {__builtin_fma(c.x, step.x, -(c.y * step.y)), __builtin_fma(c.y, step.x, c.x * step.y)};
            else
                c = wide_angle(double(pos) * f);
            last = pos;
            cs[t * half + j] = {c.x * gain, c.y * gain};
        }
    };
    // a task's work on those tokens: kFind looks for the largest magnitude, kPut writes; kBoth does both, with what
    // join(largest) makes of it between them.  lead: the wave that sees to the tokens that were there and the scale.
    enum { kFind, kPut, kBoth };
    auto work = [&](int task, int c0, int count, int what, float found, bool lead, auto&& join) {
        const int head = __builtin_amdgcn_readfirstlane(task >> 1);
        const bool is_v = __builtin_amdgcn_readfirstlane(task & 1) != 0;
        const int lg = is_v ? h.v_lanes_log2 : h.lanes_log2, lanes = 1 << lg;
        const int per = kVec > 1 ? 1 : is_v ? h.v_per : h.per;
        const int units = is_v ? h.v_units : a.units, steps = ((count + (64 >> lg) - 1) >> (6 - lg)) * per;
        const uint64_t scale_at = (is_v ? l.v_scales : l.k_scales) + (uint64_t(page) * p.heads + head) * 4;
        const uint64_t dst = (is_v ? l.v : l.k) + (uint64_t(page) * p.page_size * p.heads + head) * dim;
        const uint64_t row_bytes = uint64_t(p.heads) * dim;
        const float was = *gptr<const gf32>(scale_at);
        const int in_lds = what == kBoth ? c0 : 0;              // the first of them among the angles
        const int64_t row = is_v ? a.v_row : a.k_row;
        const TI* base = reinterpret_cast<const TI*>(is_v ? a.v : a.k) + (row0 + c0) * row +
                         head * (is_v ? a.v_head : a.k_head);
        struct Place {
            int tok, i;
            bool live;
        };
        auto place = [&](int step) {
            const int round = per == 1 ? step : step / per;
            Place x;
            x.tok = (round << (6 - lg)) + (lane >> lg);
            x.i = (lane & (lanes - 1)) + ((step - round * per) << lg);
            x.live = x.tok < count && x.i < units;
            return x;
        };
        auto unit = [&](const Place& x) {
            const int i = x.i < units ? x.i : 0;
            return is_v ? Unit{kUnitPairs, i * kVec, dim / 2 + i * kVec, 0}
                        : head_unit<kVec>(i, a.rot, a.interleaved != 0);
        };
        auto load = [&](const Place& x, const Unit& u) {
            return load_raw<TI, kVec>(base + int64_t(x.tok < count ? x.tok : 0) * row, u);
        };
        // a step's values as they are to be cached; all lanes together
        auto ready = [&](const Place& x, const Unit& u, const RawUnit<TI, kVec>& raw) {
            if (is_v) return values_of<TI, kVec>(raw, u, x.live);
            WideValues<kVec> v = wide_values_of<TI, kVec>(raw, u, x.live);
            if (h.norm.kind != kNormNone) {
                const double2 m = wide_norm<kVec>(h.norm, dim, lanes, [&](auto&& f) {
                    f(v, values_in(u, kVec, x.live));
                    if constexpr (kVec > 1) return;
                    for (int k = 1; k < per; ++k) {             // the head's other units, in whatever order
                        Place y = x;
                        y.i = x.i + (k << lg);
                        if (y.i >= per << lg) y.i -= per << lg;
                        y.live = y.tok < count && y.i < units;
                        const Unit w = unit(y);
                        f(wide_values_of<TI, kVec>(load(y, w), w, y.live), values_in(w, kVec, y.live));
                    }
                });
                const RawUnit<float, kVec> w = weights_of_unit<kVec>(h.norm, true, head, u, dim, sh);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    v.x[i] = (v.x[i] - m.x) * m.y * double(w.x.x[i]);
                    v.x[kVec + i] = (v.x[kVec + i] - m.x) * m.y * double(w.y.x[i]);
                }
            }
            const double2* angles = cs + (in_lds + (x.tok < count ? x.tok : 0)) * half + u.pair;
            Values<kVec> o;
            if (kVec == 1 || a.interleaved == 0) {
                const bool turns = u.kind == kUnitPairs;
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const double2 c = turns ? angles[i] : double2{1.0, 0.0};
                    const double b = turns ? v.x[kVec + i] : 0.0;
                    o.x[i] = to_odd(__builtin_fma(v.x[i], c.x, -(b * c.y)));
                    o.x[kVec + i] = to_odd(__builtin_fma(b, c.x, v.x[i] * c.y));
                }
            } else {
#pragma unroll
                for (int i = 0; i < kVec; i += 2) {
                    // as for q: the vector may lie across the end of what turns
                    const bool turns = u.d0 + i < a.rot;
                    const double2 c = turns ? angles[i / 2] : double2{1.0, 0.0};
                    const double x0 = __builtin_fma(v.x[i], c.x, -(v.x[i + 1] * c.y));
                    const double x1 = __builtin_fma(v.x[i + 1], c.x, v.x[i] * c.y);
                    o.x[i] = to_odd(turns ? x0 : v.x[i]);
                    o.x[i + 1] = to_odd(turns ? x1 : v.x[i + 1]);
                    o.x[kVec + i] = o.x[kVec + i + 1] = 0.0f;
                }
            }
            return o;
        };
        auto largest = [&](const Place& x, const Unit& u, const Values<kVec>& v, float m) {
            const int count = values_in(u, kVec, x.live);
#pragma unroll
            for (int i = 0; i < 2 * kVec; ++i)
                if (i < count) m = __builtin_fmaxf(m, finite_magnitude(v.x[i]));
            return m;
        };
        Values<kVec> held[kHeldUnits];
        if (what != kPut) {
            RawUnit<TI, kVec> raw[kHeldUnits];
#pragma unroll
            for (int i = 0; i < kHeldUnits; ++i) {
                const Place x = place(i);
                raw[i] = load(x, unit(x));
            }
#pragma unroll
            for (int i = 0; i < kHeldUnits; ++i) {
                if (i >= steps) break;
                const Place x = place(i);
                const Unit u = unit(x);
                held[i] = ready(x, u, raw[i]);
                found = largest(x, u, held[i], found);
            }
#pragma unroll 1
            for (int i = kHeldUnits; i < steps; ++i) {
                const Place x = place(i);
                const Unit u = unit(x);
                found = largest(x, u, ready(x, u, load(x, u)), found);
            }
            found = wave_max(found);
        }
        if (what == kFind) return found;
        if (what == kBoth) found = join(found);
        int e = scale_exponent(found);
        const int e_was = stored_exponent(was);
        if (old > 0 && e_was > e) e = e_was;
        if (lead && old > 0 && e > e_was) {                  // the tokens that are there, held anew
            const float factor = exp2_int(e - e_was > 30 ? -30 : e_was - e);     // 448 2^-30 is below the least byte
            const int vectors = dim / 16;
            for (int i = lane; i < old * vectors; i += 64) {
                const int tok = i / vectors;
                const uint64_t at16 = dst + tok * row_bytes + (i - tok * vectors) * 16;
                u32x4 b = *gptr<const gvec4>(at16);
#pragma unroll
                for (int w = 0; w < 4; ++w) b[w] = bytes_under(b[w], factor);
                *gptr<gvec4>(at16) = b;
            }
        }
        const float inv = exp2_int(-e);
        auto put = [&](const Place& x, const Unit& u, const Values<kVec>& v) {
            if (!x.live) return;
            const uint64_t to = dst + (old + c0 + x.tok) * row_bytes;
            float y[2 * kVec];
#pragma unroll
            for (int i = 0; i < 2 * kVec; ++i) y[i] = for_byte(v.x[i], inv);
            if constexpr (kVec == 8) {
                *gptr<gvec2>(to + u.d0) = u32x2{bytes_of(y[0], y[1], y[2], y[3]), bytes_of(y[4], y[5], y[6], y[7])};
                if (u.kind == kUnitPairs)
                    *gptr<gvec2>(to + u.d1) =
                        u32x2{bytes_of(y[8], y[9], y[10], y[11]), bytes_of(y[12], y[13], y[14], y[15])};
            } else {
                const uint32_t b = bytes_of(y[0], y[1], 0.0f, 0.0f);
                *gptr<gbyte>(to + u.d0) = uint8_t(b);
                if (u.kind == kUnitPairs) *gptr<gbyte>(to + u.d1) = uint8_t(b >> 8);
            }
        };
        int from = 0;
        if (what == kBoth) {
#pragma unroll
            for (int i = 0; i < kHeldUnits; ++i) {
                if (i >= steps) break;
                const Place x = place(i);
                put(x, unit(x), held[i]);
            }
            from = kHeldUnits;
        }
#pragma unroll 1
        for (int i = from; i < steps; ++i) {
            const Place x = place(i);
            const Unit u = unit(x);
            put(x, u, ready(x, u, load(x, u)));
        }
        if (lead && lane == 0) *gptr<gf32>(scale_at) = exp2_int(e);
        return found;
    };
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = kAppendBlock / 64;
    const int first = 2 * h0 + wave, last = 2 * h1;
    auto alone = [](float x) { return x; };
    share_weights(h.norm, dim, sh);
    if (int64_t(n) * half <= h.angles) {
        fill(0, n);
        __syncthreads();
        if (n <= kHeldUnits * (64 >> h.lanes_log2)) {
#pragma unroll 1
            for (int task = first; task < last; task += waves) work(task, 0, n, kBoth, 0.0f, true, alone);
            return;
        }
        // Pages of more tokens than a wave keeps: the waves share a task's.  What they found lies in LDS twice over, so
        // that one barrier a task keeps the next one's from this one's.
        const int share = (n + waves - 1) / waves, c0 = wave * share < n ? wave * share : n - 1;
        const int count = n - wave * share < 0 ? 0 : n - wave * share < share ? n - wave * share : share;
#pragma unroll 1
        for (int task = 2 * h0; task < last; ++task)
            work(task, c0, count, kBoth, 0.0f, wave == 0, [&](float x) {
                float* f = found_by[task & 1];
                if (lane == 0) f[wave] = x;
                __syncthreads();
                float m = f[0];
#pragma unroll
                for (int w = 1; w < waves; ++w) m = __builtin_fmaxf(m, f[w]);
                return m;
            });
        return;
    }
    // More angles than fit: some tokens at a time, first for the scales, then for the bytes; a block's largest magnitude
    // waits behind the angles, where only its own wave looks.
    float* most = reinterpret_cast<float*>(cs + h.angles);
    const int chunk = h.angles / half;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass)
#pragma unroll 1
        for (int c0 = 0; c0 < n; c0 += chunk) {
            const int count = n - c0 < chunk ? n - c0 : chunk;
            __syncthreads();
            fill(c0, count);
            __syncthreads();
#pragma unroll 1
            for (int task = first; task < last; task += kAppendBlock / 64) {
                float& m = most[task - 2 * h0];
                // in the second pass the first tokens' call holds the old ones anew and writes the scale; the later calls
                // read that scale, which is the largest of what they found and what was there, and come to it again
                const float found = work(task, c0, count, pass == 0 ? kFind : kPut, pass == 0 && c0 == 0 ? 0.0f : m,
                                         pass == 1 && c0 == 0, alone);
                if (pass == 0) m = found;
            }
        }
}

template <class TI, class TO, int kVec>
__global__ __launch_bounds__(kAppendBlock, 3) void append8_rows(AppendHeadsArgs h)
{
    extern __shared__ double2 cs[];
    __shared__ SharedWeights sh;
    if (blockIdx.x < h.token_items)
        token_heads<TI, TO, kVec, false>(h, blockIdx.x, reinterpret_cast<float2*>(cs), sh);
    else
        page_heads<TI, kVec>(h, blockIdx.x - h.token_items, cs, sh);
}

}  // namespace kvmove
