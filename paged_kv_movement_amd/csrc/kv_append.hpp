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
// Bound: memory, q, k and v read once, q', k', v' written once; one workgroup
// per token, so that the R/2 angles are formed once for all its heads.
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
    int32_t q_heads;
    int32_t interleaved;
    float gain;
};

template <class T>
__device__ __forceinline__ float to_float(T x)
{
    return float(x);
}

template <class T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Vec {
    T x[N];
};

template <class T>
__device__ __forceinline__ T from_float(float x)
{
    return T(x);
}

// One head's unit u of kVec-wide vectors, rotated or passed on.  Units of a
// head: half layout, rot / (2 kVec) pairs of vectors, then the vectors behind
// the rotated part; interleaved, dim / kVec vectors (pairs of elements for
// kVec = 1).
template <class TI, class TO, int kVec>
__device__ __forceinline__ void rotate_unit(const TI* src, TO* dst, int u, int rot, bool interleaved,
                                            const float2* cs)
{
    using VI = Vec<TI, kVec>;
    using VO = Vec<TO, kVec>;
    if (!interleaved) {
        const int half = rot / 2, pairs = half / kVec;
        if (u < pairs) {
            const int d = u * kVec;
            const VI x = *reinterpret_cast<const VI*>(src + d), y = *reinterpret_cast<const VI*>(src + half + d);
            VO ox, oy;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float2 c = cs[d + i];
                const float a = to_float(x.x[i]), b = to_float(y.x[i]);
                ox.x[i] = from_float<TO>(__builtin_fmaf(a, c.x, -(b * c.y)));
                oy.x[i] = from_float<TO>(__builtin_fmaf(b, c.x, a * c.y));
            }
            *reinterpret_cast<VO*>(dst + d) = ox;
            *reinterpret_cast<VO*>(dst + half + d) = oy;
            return;
        }
        const int d = rot + (u - pairs) * kVec;
        const VI x = *reinterpret_cast<const VI*>(src + d);
        VO o;
#pragma unroll
        for (int i = 0; i < kVec; ++i) o.x[i] = from_float<TO>(to_float(x.x[i]));
        *reinterpret_cast<VO*>(dst + d) = o;
        return;
    }
    if constexpr (kVec == 1) {
        if (u < rot / 2) {
            const float a = to_float(src[2 * u]), b = to_float(src[2 * u + 1]);
            const float2 c = cs[u];
            dst[2 * u] = from_float<TO>(__builtin_fmaf(a, c.x, -(b * c.y)));
            dst[2 * u + 1] = from_float<TO>(__builtin_fmaf(b, c.x, a * c.y));
        } else {
            const int d = u + rot / 2;
            dst[d] = from_float<TO>(to_float(src[d]));
        }
    } else {
        const int d = u * kVec;
        const VI x = *reinterpret_cast<const VI*>(src + d);
        VO o;
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
            float a = to_float(x.x[i]), b = to_float(x.x[i + 1]);
            if (d < rot) {
                const float2 c = cs[(d + i) / 2];
                const float r = __builtin_fmaf(a, c.x, -(b * c.y));
                b = __builtin_fmaf(b, c.x, a * c.y);
                a = r;
            }
            o.x[i] = from_float<TO>(a);
            o.x[i + 1] = from_float<TO>(b);
        }
        *reinterpret_cast<VO*>(dst + d) = o;
    }
}

// Units a head has under rotate_unit.
__device__ __forceinline__ int head_units(int rot, int dim, bool interleaved, int vec)
{
    if (!interleaved) return rot / (2 * vec) + (dim - rot) / vec;
    return vec == 1 ? rot / 2 + (dim - rot) : dim / vec;
}

template <class TI, class TO, int kVec>
__global__ __launch_bounds__(kAppendBlock) void append_rows(AppendArgs a)
{
    __shared__ float2 cs[kMaxRot / 2];
    const int32_t r = blockIdx.x, tid = threadIdx.x;
    const int32_t pos = gptr<const gi32>(a.positions)[r];
    const double turns_per_radian = 0.15915494309189533577;
    for (int j = tid; j < a.rot / 2; j += kAppendBlock) {
        const double f = gptr<const __attribute__((address_space(1))) double>(a.freqs)[j];
        const double t = double(pos) * (f * turns_per_radian);
        const float frac = float(t - __builtin_rint(t));
        float sn, cn;
        sincospif(2.0f * frac, &sn, &cn);
        cs[j] = {cn * a.gain, sn * a.gain};
    }
    const int32_t s = wave_find(a.step.q_start, a.step.own.n, r);

    const int dim = a.pool.dim, rot = a.rot;
    const bool il = a.interleaved != 0;
    const int per = head_units(rot, dim, il, kVec);
    const int vper = dim / kVec;
    const int kv_heads = a.pool.heads;
    __syncthreads();
    if (a.q != 0) {
        const TI* q = reinterpret_cast<const TI*>(a.q) + int64_t(r) * a.q_row;
        TO* o = reinterpret_cast<TO*>(a.q_out) + int64_t(r) * a.o_row;
        for (int i = tid; i < a.q_heads * per; i += kAppendBlock) {
            const int h = i / per, u = i - h * per;
            rotate_unit<TI, TO, kVec>(q + h * a.q_head, o + h * a.o_head, u, rot, il, cs);
        }
    }
    if (s < 0) return;                             // a row of no sequence: nothing is cached
    const Rows rows = seq_rows(a.step, s);
    const int32_t i = r - rows.first;
    const int32_t slot = table_len(a.step.own, s) - rows.count + i;
    if (i >= rows.count || slot < 0) return;
    const uint32_t pi = page_of(a.pool, uint32_t(slot));
    const int32_t page = gptr<const gi32>(a.step.own.table)[s * a.step.own.stride + pi];
    const uint64_t kb = gptr<const gu64>(a.pool.k_pages)[a.pool.layer];
    const uint64_t vb = gptr<const gu64>(a.pool.v_pages)[a.pool.layer];
    if (page < 0 || uint32_t(page) >= a.pool.num_pages) {
        raise_fault(kFaultPage);
        return;
    }
    if (bad_addr(kb) || bad_addr(vb)) {
        raise_fault(kFaultPool);
        return;
    }
    const int64_t row = int64_t(page) * a.pool.page_size + (uint32_t(slot) - pi * a.pool.page_size);
    __bf16* kd = reinterpret_cast<__bf16*>(kb) + row * kv_heads * dim;
    __bf16* vd = reinterpret_cast<__bf16*>(vb) + row * kv_heads * dim;
    const TI* k = reinterpret_cast<const TI*>(a.k) + int64_t(r) * a.k_row;
    const TI* v = reinterpret_cast<const TI*>(a.v) + int64_t(r) * a.v_row;
    for (int i = tid; i < kv_heads * per; i += kAppendBlock) {
        const int h = i / per, u = i - h * per;
        rotate_unit<TI, __bf16, kVec>(k + h * a.k_head, kd + h * dim, u, rot, il, cs);
    }
    for (int i = tid; i < kv_heads * vper; i += kAppendBlock) {
        const int h = i / vper, u = i - h * vper;
        const Vec<TI, kVec> x = *reinterpret_cast<const Vec<TI, kVec>*>(v + h * a.v_head + u * kVec);
        Vec<__bf16, kVec> o;
#pragma unroll
        for (int e = 0; e < kVec; ++e) o.x[e] = from_float<__bf16>(to_float(x.x[e]));
        *reinterpret_cast<Vec<__bf16, kVec>*>(vd + h * dim + u * kVec) = o;
    }
    if (a.weights != 0)
        for (int h = tid; h < a.w_heads; h += kAppendBlock) {
            const int64_t at = (int64_t(s) * a.w_heads + h) * a.w_cap + slot;
            gptr<gf32>(a.weights)[at] = 0.0f;
            gptr<gi32>(a.slot_positions)[at] = pos;
        }
}

}  // namespace kvmove
