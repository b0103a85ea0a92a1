// kv_pack8.hpp -- cached tokens from bf16 pages into 8-bit ones and back.
//
// pack8_pages    a workgroup per (layer, sequence, page, group of heads, K or
//                V): a thread always sees the same head, so that a block's
//                largest magnitude is the maximum of some threads' own; then
//                the scale and the bytes (kv_pool8.hpp).
// unpack8_pages  byte * scale, which bf16 holds exactly; a wave per 4 KiB of
//                the page's bf16.
//
// Bound: memory, 3 bytes an element either way.  4 layers of 77482 tokens of 8 KV
// heads of 128 (1.9 GB) in 355 us and back in 365, 5.4 and 5.2 TB/s, where a
// large copy reaches 6.7; one layer of 4 x 256 tokens in 5.7 and 4.3.
#pragma once

#include "kv_pool8.hpp"

namespace kvmove {

constexpr int kPackBlock = 256;
constexpr int kPackHeld = 8;           // vectors of a thread kept between the scale and the bytes
constexpr int kUnpackVectors = 4;      // vectors of a lane

struct PackArgs {
    PoolArg from, to;                  // one page size, heads and head size
    ScalesArg scales;                  // of the 8-bit one
    TablesArg tables;                  // of `from`
    uint64_t to_table;                 // int32[n][to_stride]
    int64_t to_stride;
    int32_t pages;                     // of a sequence
    int32_t parts;                     // workgroups of a page: head groups (pack8), tiles (unpack8)
    int32_t group;                     // pack8: heads of a workgroup
    int32_t cols;                      // pack8: their vectors of 8 elements in a row, at most a thread each
    uint32_t vec_magic, vec_shift;     // i / (vectors of a head)
    uint32_t row_magic, row_shift;     // i / cols (pack8), i / (vectors of a row) (unpack8)
};

// The page that workgroup b works on; n: its tokens.  n <= 0: none.
struct PackPage {
    int32_t n, from, to;
};

__device__ __forceinline__ PackPage pack_page(const PackArgs& a, uint32_t b, bool bad)
{
    const int32_t s = __builtin_amdgcn_readfirstlane(b / uint32_t(a.pages)), pi = int32_t(b - uint32_t(s) * a.pages);
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
    __shared__ unsigned int largest[kPackBlock / 2];         // of a head of the group, as bits: order of magnitudes
    a.from.layer += blockIdx.y / 2;
    a.to.layer += blockIdx.y / 2;
    const LayerAt from = layer_at<false>(a.from, a.scales), to = layer_at<true>(a.to, a.scales);
    const uint32_t b = xcd_contiguous(blockIdx.x, gridDim.x), at = b / uint32_t(a.parts);
    const PackPage p = pack_page(a, at, bad_layer<false>(from) || bad_layer<true>(to));
    if (p.n <= 0) return;
    const bool v = blockIdx.y % 2 != 0;
    const int32_t h0 = int32_t(b - at * uint32_t(a.parts)) * a.group;
    const int dim = a.from.dim, tid = threadIdx.x;
    const int heads = a.group < int(a.from.heads) - h0 ? a.group : int(a.from.heads) - h0;
    const uint32_t row = a.from.heads * dim;                             // elements
    // thread: vector `col` of the group's row, tokens first, first + step, ...
    const int first = int((uint64_t(uint32_t(tid)) * a.row_magic) >> a.row_shift), col = tid - first * a.cols;
    const int step = kPackBlock / a.cols, head = int((uint64_t(uint32_t(col)) * a.vec_magic) >> a.vec_shift);
    const bool live = first < step && head < heads;
    const uint32_t offset = first * row + h0 * dim + col * 8, stride = step * row;
    const uint64_t page = uint64_t(a.from.page_size) * row;
    const __amdgpu_buffer_rsrc_t src = byte_range((v ? from.v : from.k) + p.from * page * 2, p.n * row * 2);
    const __amdgpu_buffer_rsrc_t dst = byte_range((v ? to.v : to.k) + p.to * page, p.n * row);
    auto has = [&](int k) { return live && first + k * step < p.n; };
    auto load = [&](int k) {
        return has(k) ? __builtin_amdgcn_raw_buffer_load_b128(src, (offset + k * stride) * 2, 0, kCpolNt | kCpolSc1)
                      : u32x4{0, 0, 0, 0};
    };
    if (tid < kPackBlock / 2) largest[tid] = 0;
    u32x4 x[kPackHeld];
#pragma unroll
    for (int k = 0; k < kPackHeld; ++k) x[k] = load(k);
    __syncthreads();
    float most = 0.0f;
#pragma unroll
    for (int k = 0; k < kPackHeld; ++k) most = largest_of(x[k], most);
    const int rounds = (p.n + step - 1) / step;
    for (int k = kPackHeld; k < rounds; ++k) most = largest_of(load(k), most);
    if (live) atomicMax(&largest[head], __float_as_uint(most));          // a maximum does not depend on the order
    __syncthreads();
    const int e = scale_exponent(__uint_as_float(largest[live ? head : 0]));
    const float inv = exp2_int(-e);
    auto put = [&](int k, u32x4 y) {
        if (has(k))
            __builtin_amdgcn_raw_buffer_store_b64(bytes_of_bf16(y, inv), dst, offset + k * stride, 0, kCpolNt | kCpolSc1);
    };
#pragma unroll
    for (int k = 0; k < kPackHeld; ++k) put(k, x[k]);
    for (int k = kPackHeld; k < rounds; ++k) put(k, load(k));
    if (tid < heads)
        gptr<gf32>(v ? to.v_scales : to.k_scales)[uint64_t(p.to) * a.to.heads + h0 + tid] =
            exp2_int(scale_exponent(__uint_as_float(largest[tid])));
}

// grid: (pages of all sequences * tiles, K and V of every layer)
__global__ __launch_bounds__(64) void unpack8_pages(PackArgs a)
{
    a.from.layer += blockIdx.y / 2;
    a.to.layer += blockIdx.y / 2;
    const LayerAt from = layer_at<true>(a.from, a.scales), to = layer_at<false>(a.to, a.scales);
    const uint32_t b = xcd_contiguous(blockIdx.x, gridDim.x), at = b / uint32_t(a.parts);
    const PackPage p = pack_page(a, at, bad_layer<true>(from) || bad_layer<false>(to));
    const bool v = blockIdx.y % 2 != 0;
    const uint32_t dim = a.from.dim, row = a.from.heads * dim / 8;       // vectors of 8 elements
    const uint32_t first = (b - at * uint32_t(a.parts)) * (64 * kUnpackVectors) + threadIdx.x;
    if (p.n <= 0 || first - threadIdx.x >= p.n * row) return;
    const uint64_t page = uint64_t(a.from.page_size) * row * 8;
    const __amdgpu_buffer_rsrc_t src = byte_range((v ? from.v : from.k) + p.from * page, p.n * row * 8);
    const __amdgpu_buffer_rsrc_t dst = byte_range((v ? to.v : to.k) + p.to * page * 2, p.n * row * 16);
    const uint64_t scales = (v ? from.v_scales : from.k_scales) + uint64_t(p.from) * a.from.heads * 4;
    u32x2 x[kUnpackVectors];
    float s[kUnpackVectors];
#pragma unroll
    for (int k = 0; k < kUnpackVectors; ++k) {
        const uint32_t i = first + 64 * k, r = uint32_t((uint64_t(i) * a.row_magic) >> a.row_shift);
        const uint32_t head = uint32_t((uint64_t(i - r * row) * a.vec_magic) >> a.vec_shift);
        x[k] = __builtin_amdgcn_raw_buffer_load_b64(src, i * 8, 0, kCpolNt | kCpolSc1);
        s[k] = gptr<const gf32>(scales)[head];
    }
#pragma unroll
    for (int k = 0; k < kUnpackVectors; ++k)
        __builtin_amdgcn_raw_buffer_store_b128(bf16_of_bytes8(x[k][0], x[k][1], s[k]), dst, (first + 64 * k) * 16, 0,
                                               kCpolNt | kCpolSc1);
}

}  // namespace kvmove
