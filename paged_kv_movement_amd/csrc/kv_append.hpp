// kv_append.hpp -- new tokens' q and k rotated by their positions, k and v
// written into their page rows.
//
// Rotary positions: pair j of a head, (x, y), at position p turns by
// a = p * f[j]: (x cos a - y sin a, y cos a + x sin a), times a gain (1, or
// the attention factor of a scaled rotation).  A pair is (j, j + R/2) or
// (2j, 2j + 1) of the head's first R elements; the others pass.  The angle is
// formed in 64 bits as turns (p * f / 2 pi) and its whole turns dropped
// before it becomes a float: in 32 bits a position of 10^6 would already be
// off by 0.03 rad.  The rotation is float32 and each result is rounded once.
//
// Bound: memory, q, k and v read once, q', k', v' written once.  One workgroup
// per token, so that the R/2 angles are formed once for all its heads, and two
// units a thread in flight before anything is waited for.  45116 tokens of 32
// query heads and 8 KV heads of 128 (1.1 GB): 200 us, 5.5 TB/s, where a plain
// copy reaches 6.8; with the units asked for after the angles 237, and no
// better with 128 or 512 threads, four units or streaming loads.  One token:
// 3.8 us, 64 tokens 5.3, the wait for owner, page and stores in turn.
#pragma once

#include "kv_step.hpp"

namespace kvmove {

constexpr int kAppendBlock = 256;
constexpr int kMaxRot = 512;           // angles of a token kept in LDS: R/2 pairs

struct AppendArgs {
    PoolArg pool;
    StepArg step;
    uint64_t q, k, v, q_out;           // q 0: only k and v
    int64_t q_row, q_head;             // strides in elements
    int64_t k_row, k_head;
    int64_t v_row, v_head;
    int64_t o_row, o_head;
    uint64_t positions;                // int32[n_rows]
    uint64_t freqs;                    // float64[rot / 2], radians per position
    uint64_t weights, slot_positions;  // float32 / int32 [own.n][w_heads][w_cap], or 0
    int64_t w_cap;
    int32_t w_heads;
    int32_t rot;
    int32_t units;                     // units of a head of q or k
    uint32_t unit_magic, unit_shift;   // i / units
    uint32_t vec_magic, vec_shift;     // i / (vectors of a head)
    int32_t q_heads;
    int32_t interleaved;
    float gain;
};

template <class T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Vec {
    T x[N];
};

// A token's heads are cut into units of one or two vectors of kVec elements:
// two halves of kVec pairs (half layout; interleaved pairs element by element
// for kVec = 1), one vector of interleaved pairs, or one vector that passes.
enum : int { kUnitPairs = 0, kUnitInterleaved = 1, kUnitPass = 2 };

struct Unit {
    int kind;
    int d0, d1;           // elements of the head where its vectors begin
    int pair;             // first pair's angle
};

template <int kVec>
__device__ __forceinline__ Unit head_unit(int u, int rot, bool interleaved)
{
    if (interleaved) {
        if (kVec == 1) {
            if (u < rot / 2) return {kUnitPairs, 2 * u, 2 * u + 1, u};
            return {kUnitPass, u + rot / 2, u + rot / 2, 0};
        }
        const int d = u * kVec;
        return {d < rot ? kUnitInterleaved : kUnitPass, d, d, d / 2};
    }
    const int pairs = rot / (2 * kVec);
    if (u < pairs) return {kUnitPairs, u * kVec, rot / 2 + u * kVec, u * kVec};
    const int d = rot + (u - pairs) * kVec;
    return {kUnitPass, d, d, 0};
}

// Units a head has.
__host__ __device__ __forceinline__ int head_units(int rot, int dim, bool interleaved, int vec)
{
    if (!interleaved) return rot / (2 * vec) + (dim - rot) / vec;
    return vec == 1 ? rot / 2 + (dim - rot) : dim / vec;
}

// Writes a unit: x and y are its vectors, cs the token's cosines and sines.
template <class TI, class TO, int kVec>
__device__ __forceinline__ void put_unit(const Unit& u, const Vec<TI, kVec>& x, const Vec<TI, kVec>& y, TO* dst,
                                         const float2* cs)
{
    Vec<TO, kVec> ox, oy;
    if (u.kind == kUnitPairs) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const float2 c = cs[u.pair + i];
            const float a = float(x.x[i]), b = float(y.x[i]);
            ox.x[i] = TO(__builtin_fmaf(a, c.x, -(b * c.y)));
            oy.x[i] = TO(__builtin_fmaf(b, c.x, a * c.y));
        }
        *reinterpret_cast<Vec<TO, kVec>*>(dst + u.d1) = oy;
    } else if (kVec > 1 && u.kind == kUnitInterleaved) {
#pragma unroll
        for (int i = 0; i + 1 < kVec; i += 2) {
            const float2 c = cs[u.pair + i / 2];
            const float a = float(x.x[i]), b = float(x.x[i + 1]);
            ox.x[i] = TO(__builtin_fmaf(a, c.x, -(b * c.y)));
            ox.x[i + 1] = TO(__builtin_fmaf(b, c.x, a * c.y));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) ox.x[i] = TO(float(x.x[i]));
    }
    *reinterpret_cast<Vec<TO, kVec>*>(dst + u.d0) = ox;
}

// Unit i of a token: of q's heads, then k's, then v's.
template <class TI, int kVec>
struct TokenUnit {
    Vec<TI, kVec> x, y;
    Unit u;
    int head;             // of its array
    int array;            // 0: q, 1: k, 2: v
};

template <class TI, int kVec>
__device__ __forceinline__ void load_unit(const AppendArgs& a, int32_t r, int i, TokenUnit<TI, kVec>& t)
{
    const int nq = a.q_heads * a.units, nk = a.pool.heads * a.units;
    const bool v = i >= nq + nk;
    t.array = v ? 2 : i >= nq ? 1 : 0;
    i -= v ? nq + nk : t.array == 1 ? nq : 0;
    int u;
    if (v) {
        const int per = a.pool.dim / kVec;
        t.head = int((uint64_t(uint32_t(i)) * a.vec_magic) >> a.vec_shift);
        u = i - t.head * per;
        t.u = {kUnitPass, u * kVec, u * kVec, 0};
    } else {
        t.head = int((uint64_t(uint32_t(i)) * a.unit_magic) >> a.unit_shift);
        u = i - t.head * a.units;
        t.u = head_unit<kVec>(u, a.rot, a.interleaved != 0);
    }
    const uint64_t base = t.array == 0 ? a.q : t.array == 1 ? a.k : a.v;
    const int64_t row = t.array == 0 ? a.q_row : t.array == 1 ? a.k_row : a.v_row;
    const int64_t head = t.array == 0 ? a.q_head : t.array == 1 ? a.k_head : a.v_head;
    const TI* src = reinterpret_cast<const TI*>(base) + r * row + t.head * head;
    t.x = *reinterpret_cast<const Vec<TI, kVec>*>(src + t.u.d0);
    if (t.u.kind == kUnitPairs) t.y = *reinterpret_cast<const Vec<TI, kVec>*>(src + t.u.d1);
}

// One workgroup per token.  What does not depend on each other is asked for
// at once: the first units' values, the token's owner and length, the
// frequencies; the angles are formed while these are on their way.
template <class TI, class TO, int kVec>
__global__ __launch_bounds__(kAppendBlock) void append_rows(AppendArgs a)
{
    constexpr int kUnits = kVec == 1 ? 4 : 2;      // units of a thread in flight
    __shared__ float2 cs[kMaxRot / 2];
    const int32_t r = blockIdx.x, tid = threadIdx.x;
    const int dim = a.pool.dim, kv_heads = a.pool.heads;
    const int total = (a.q_heads + kv_heads) * a.units + kv_heads * (dim / kVec);
    TokenUnit<TI, kVec> t[kUnits];
#pragma unroll
    for (int x = 0; x < kUnits; ++x)
        if (tid + x * kAppendBlock < total) load_unit<TI, kVec>(a, r, tid + x * kAppendBlock, t[x]);
    const int32_t pos = gptr<const gi32>(a.positions)[r];
    const uint64_t kb = gptr<const gu64>(a.pool.k_pages)[a.pool.layer];
    const uint64_t vb = gptr<const gu64>(a.pool.v_pages)[a.pool.layer];
    const RowOwner o = row_owner(a.step, r);
    const double turns_per_radian = 0.15915494309189533577;
    for (int j = tid; j < a.rot / 2; j += kAppendBlock) {
        const double f = gptr<const __attribute__((address_space(1))) double>(a.freqs)[j];
        const double turns = double(pos) * (f * turns_per_radian);
        const float frac = float(turns - __builtin_rint(turns));
        float sn, cn;
        sincospif(2.0f * frac, &sn, &cn);
        cs[j] = {cn * a.gain, sn * a.gain};
    }
    // where k and v go; 0: nowhere (a row of no sequence, no slot left, a bad page)
    uint64_t kd = 0, vd = 0;
    const int32_t slot = o.len - o.count + (r - o.first);
    if (o.s >= 0 && slot >= 0) {
        const uint32_t pi = page_of(a.pool, uint32_t(slot));
        const int32_t page = gptr<const gi32>(a.step.own.table)[o.s * a.step.own.stride + pi];
        if (uint32_t(page) >= a.pool.num_pages) {
            raise_fault(kFaultPage);
        } else if (bad_addr(kb) || bad_addr(vb)) {
            raise_fault(kFaultPool);
        } else {
            const int64_t row = int64_t(page) * a.pool.page_size + (uint32_t(slot) - pi * a.pool.page_size);
            kd = kb + uint64_t(row) * kv_heads * dim * 2;
            vd = vb + uint64_t(row) * kv_heads * dim * 2;
        }
    }
    __syncthreads();
    for (int i = tid; i < total; i += kUnits * kAppendBlock) {
        if (i != tid)
#pragma unroll
            for (int x = 0; x < kUnits; ++x)
                if (i + x * kAppendBlock < total) load_unit<TI, kVec>(a, r, i + x * kAppendBlock, t[x]);
#pragma unroll
        for (int x = 0; x < kUnits; ++x) {
            if (i + x * kAppendBlock >= total) continue;
            if (t[x].array == 0) {
                TO* dst = reinterpret_cast<TO*>(a.q_out) + r * a.o_row + t[x].head * a.o_head;
                put_unit<TI, TO, kVec>(t[x].u, t[x].x, t[x].y, dst, cs);
            } else if (kd != 0) {
                __bf16* dst = reinterpret_cast<__bf16*>(t[x].array == 1 ? kd : vd) + t[x].head * dim;
                put_unit<TI, __bf16, kVec>(t[x].u, t[x].x, t[x].y, dst, cs);
            }
        }
    }
    if (a.weights != 0 && kd != 0)
        for (int h = tid; h < a.w_heads; h += kAppendBlock) {
            const int64_t at = (int64_t(o.s) * a.w_heads + h) * a.w_cap + slot;
            gptr<gf32>(a.weights)[at] = 0.0f;
            gptr<gi32>(a.slot_positions)[at] = pos;
        }
}

}  // namespace kvmove
