// kv_pack8.hpp -- cached tokens from bf16 pages into 8-bit ones and back.
//
// pack8_pages    a wave per (layer, sequence, page, head, K or V): the block's
//                largest magnitude, its scale, its bytes (kv_pool8.hpp);
// unpack8_pages  byte * scale, which bf16 holds exactly; a workgroup per
//                (layer, sequence, page, K or V).
//
// Bound: memory, 3 bytes an element either way.
#pragma once

#include "kv_pool8.hpp"

namespace kvmove {

constexpr int kPackBlock = 256;
constexpr int kPackHeld = 4;           // vectors of 16 elements of a lane kept between the scale and the bytes

struct PackArgs {
    PoolArg from, to;                  // one page size, heads and head size
    ScalesArg scales;                  // of the 8-bit one
    TablesArg tables;                  // of `from`
    uint64_t to_table;                 // int32[n][to_stride]
    int64_t to_stride;
    int32_t pages;                     // of a sequence
    int32_t head_groups;               // pack8: workgroups of a page
    uint32_t vec_magic, vec_shift;     // i / (vectors of 16 elements of a head)
    uint32_t row_magic, row_shift;     // i / (of a row)
};

// The page that workgroup b works on; n: its tokens.  n <= 0: none.
struct PackPage {
    int32_t n, from, to;
};

__device__ __forceinline__ PackPage pack_page(const PackArgs& a, uint32_t b, bool bad)
{
    const int32_t s = int32_t(b / uint32_t(a.pages)), pi = int32_t(b % uint32_t(a.pages));
    const int64_t left = table_len(a.tables, s) - int64_t(pi) * a.from.page_size;
    PackPage p{0, 0, 0};
    if (left <= 0) return p;
    p.from = __builtin_amdgcn_readfirstlane(gptr<const gi32>(a.tables.table)[s * a.tables.stride + pi]);
    p.to = __builtin_amdgcn_readfirstlane(gptr<const gi32>(a.to_table)[s * a.to_stride + pi]);
    if (uint32_t(p.from) >= a.from.num_pages || uint32_t(p.to) >= a.to.num_pages) {
        raise_fault(kFaultPage);
        return p;
    }
    if (bad) {
        raise_fault(kFaultPool);
        return p;
    }
    p.n = left < a.from.page_size ? int32_t(left) : int32_t(a.from.page_size);
    return p;
}

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float largest_of(u32x4 x, float m)
{
#pragma unroll
    for (int w = 0; w < 4; ++w)
        m = __builtin_fmaxf(m, __builtin_fmaxf(finite_magnitude(bf16_low(x[w])), finite_magnitude(bf16_high(x[w]))));
    return m;
}

__device__ __forceinline__ u32x2 bytes_of_bf16(u32x4 x, float inv)
{
    u32x2 b;
#pragma unroll
    for (int w = 0; w < 2; ++w)
        b[w] = bytes_of(for_byte(bf16_low(x[2 * w]), inv), for_byte(bf16_high(x[2 * w]), inv),
                        for_byte(bf16_low(x[2 * w + 1]), inv), for_byte(bf16_high(x[2 * w + 1]), inv));
    return b;
}

// grid: (pages of all sequences * head groups, K and V of every layer)
__global__ __launch_bounds__(kPackBlock) void pack8_pages(PackArgs a)
{
    a.from.layer += blockIdx.y / 2;
    a.to.layer += blockIdx.y / 2;
    const LayerAt from = layer_at<false>(a.from, a.scales), to = layer_at<true>(a.to, a.scales);
    const uint32_t group = blockIdx.x % uint32_t(a.head_groups);
    const PackPage p = pack_page(a, blockIdx.x / uint32_t(a.head_groups), bad_layer<false>(from) || bad_layer<true>(to));
    const int32_t head = int32_t(group) * (kPackBlock / 64) + (threadIdx.x >> 6);
    if (p.n <= 0 || head >= int32_t(a.from.heads)) return;
    const bool v = blockIdx.y % 2 != 0;
    const int lane = threadIdx.x & 63, dim = a.from.dim, vectors = dim / 16, total = p.n * vectors;
    const uint32_t row = a.from.heads * dim;                             // elements
    const uint64_t src = (v ? from.v : from.k) + (uint64_t(p.from) * a.from.page_size * row + head * dim) * 2;
    const uint64_t dst = (v ? to.v : to.k) + (uint64_t(p.to) * a.to.page_size * row + head * dim);
    auto element = [&](int i) {                                          // where vector i begins
        const int tok = int((uint64_t(uint32_t(i)) * a.vec_magic) >> a.vec_shift);
        return uint32_t(tok) * row + uint32_t(i - tok * vectors) * 16;
    };
    u32x4 x[kPackHeld][2];
#pragma unroll
    for (int k = 0; k < kPackHeld; ++k) {
        const int i = lane + 64 * k;
        const uint64_t at = src + uint64_t(element(i < total ? i : 0)) * 2;   // the first again where there is no more
        x[k][0] = *gptr<const gvec4>(at);
        x[k][1] = *gptr<const gvec4>(at + 16);
    }
    float most = 0.0f;
#pragma unroll
    for (int k = 0; k < kPackHeld; ++k) most = largest_of(x[k][1], largest_of(x[k][0], most));
    for (int i = lane + 64 * kPackHeld; i < total; i += 64) {
        const uint64_t at = src + uint64_t(element(i)) * 2;
        most = largest_of(*gptr<const gvec4>(at + 16), largest_of(*gptr<const gvec4>(at), most));
    }
    const int e = scale_exponent(wave_max(most));
    const float inv = exp2_int(-e);
    auto put = [&](int i, u32x4 y, u32x4 z) {
        const u32x2 b = bytes_of_bf16(y, inv), c = bytes_of_bf16(z, inv);
        *gptr<gvec4>(dst + element(i)) = u32x4{b[0], b[1], c[0], c[1]};
    };
#pragma unroll
    for (int k = 0; k < kPackHeld; ++k)
        if (lane + 64 * k < total) put(lane + 64 * k, x[k][0], x[k][1]);
    for (int i = lane + 64 * kPackHeld; i < total; i += 64) {
        const uint64_t at = src + uint64_t(element(i)) * 2;
        put(i, *gptr<const gvec4>(at), *gptr<const gvec4>(at + 16));
    }
    if (lane == 0)
        gptr<gf32>(v ? to.v_scales : to.k_scales)[uint64_t(p.to) * a.to.heads + head] = exp2_int(e);
}

// grid: (pages of all sequences, K and V of every layer)
__global__ __launch_bounds__(kPackBlock) void unpack8_pages(PackArgs a)
{
    a.from.layer += blockIdx.y / 2;
    a.to.layer += blockIdx.y / 2;
    const LayerAt from = layer_at<true>(a.from, a.scales), to = layer_at<false>(a.to, a.scales);
    const PackPage p = pack_page(a, blockIdx.x, bad_layer<true>(from) || bad_layer<false>(to));
    if (p.n <= 0) return;
    const bool v = blockIdx.y % 2 != 0;
    const int vectors = a.from.dim / 16, row = a.from.heads * vectors;   // vectors of 16 elements
    const uint64_t bytes = uint64_t(a.from.page_size) * row * 16;
    const uint64_t src = (v ? from.v : from.k) + p.from * bytes, dst = (v ? to.v : to.k) + p.to * bytes * 2;
    const uint64_t scales = (v ? from.v_scales : from.k_scales) + uint64_t(p.from) * a.from.heads * 4;
    for (int64_t i = threadIdx.x; i < int64_t(p.n) * row; i += kPackBlock) {
        const uint32_t in_row = uint32_t(i) - uint32_t((uint64_t(i) * a.row_magic) >> a.row_shift) * uint32_t(row);
        const uint32_t head = uint32_t((uint64_t(in_row) * a.vec_magic) >> a.vec_shift);
        const u32x4 b = *gptr<const gvec4>(src + i * 16);
        const float s = gptr<const gf32>(scales)[head];
        *gptr<gvec4>(dst + i * 32) = bf16_of_bytes8(b[0], b[1], s);
        *gptr<gvec4>(dst + i * 32 + 16) = bf16_of_bytes8(b[2], b[3], s);
    }
}

}  // namespace kvmove
