// tp_w4.cu -- 4-bit weights with group scales: quantising, the layout that the
// products read, and the products of few tokens with such weights.
//
// A group of `group` consecutive columns of a row has the scale s (bf16), its
// elements are (code - 8) s with codes 0..15.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "tc_ptx.cuh"
#include "tp_act.cuh"
#include "tp_internal.h"
#include "tpffn.h"

namespace tpffn {
namespace w4 {

__device__ __forceinline__ float bf16_at(uint32_t w, int half) {
  return __uint_as_float(half ? w & 0xffff0000u : w << 16);
}

// ================================================================ quantising
// s = bf16(max |w| / 7), code = rint(w / s) + 8, ties to even.
// A group with an infinity or NaN has that for its scale.  With s = 0 (all
// zero, or too small for bf16) every code is 8.
__device__ __forceinline__ float group_scale(float amax) { return __bfloat162float(__float2bfloat16_rn(amax / 7.f)); }

// code - 8 as a float: w / s rounded to a whole number, ties to even, for w of
// eight bits and finite s > 0 with |w| <= 7.03 s.  w * inv is within 2^-22 of the
// quotient, which lies at least 2^-18 from a tie unless it is one; ties are told
// by the remainder, which is exact.
__device__ __forceinline__ float steps_of(float w, float s, float inv) {
  const float magic = 12582912.f;  // 1.5 2^23: the sum's last bit is worth 1
  const float u = fmaf(w, inv, magic);
  float q = u - magic;
  const float r = fmaf(-q, s, w);
  if (fabsf(r + r) == s && (__float_as_uint(u) & 1u)) q += copysignf(1.f, r);
  return q;
}
__device__ __forceinline__ uint32_t code_of(float w, float s, float inv) {
  if (!(s > 0.f) || !(s < INFINITY)) return 8u;
  return static_cast<uint32_t>(static_cast<int>(steps_of(w, s, inv)) + 8);
}
// 1 / s overflows for the smallest scales: s and w are brought up by 2^64 first.
__device__ __forceinline__ void ready(float& s, float& inv, float& up) {
  up = s < 1e-30f ? 18446744073709551616.f : 1.f;
  s *= up;
  inv = 1.f / s;
}

// 16 elements to a lane, group / 16 lanes to a group.
__global__ void __launch_bounds__(256) quantize16_kernel(const uint4* __restrict__ W, long long pieces, int row_pieces,
                                                         int seg_pieces, int lanes, int seg_groups, int segs,
                                                         uint2* __restrict__ codes, __nv_bfloat16* __restrict__ scales) {
  // places: the pieces of a row, each segment's rounded up to whole groups
  const long long row_places = static_cast<long long>(segs) * seg_groups * lanes;
  const long long rows = pieces / row_pieces, total = rows * row_places;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i0 = static_cast<long long>(blockIdx.x) * blockDim.x; i0 < total; i0 += stride) {
    const long long i = i0 + threadIdx.x;
    const long long row = i / row_places;
    const int place = static_cast<int>(i - row * row_places), per = seg_groups * lanes;
    const int seg = place / per, in = place - seg * per;
    const bool ok = i < total && in < seg_pieces;
    const long long at = row * row_pieces + static_cast<long long>(seg) * seg_pieces + in;
    uint32_t v[8] = {};
    if (ok) {
      const uint4 a = W[2 * at], b = W[2 * at + 1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __nv_bfloat162 m = __habs2(*reinterpret_cast<__nv_bfloat162*>(&v[0]));
#pragma unroll
    for (int j = 1; j < 8; ++j) m = __hmax2_nan(m, __habs2(*reinterpret_cast<__nv_bfloat162*>(&v[j])));
    for (int d = 1; d < lanes; d <<= 1) m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    const __nv_bfloat16 top = __hmax_nan(m.x, m.y);
    float s = group_scale(__bfloat162float(top)), inv, up;
    if (ok && in % lanes == 0) scales[(row * segs + seg) * seg_groups + in / lanes] = __float2bfloat16_rn(s);
    ready(s, inv, up);
    uint32_t word[2] = {};
#pragma unroll
    for (int j = 0; j < 16; ++j)
      word[j >> 3] |= code_of(bf16_at(v[j >> 1], j & 1) * up, s, inv) << (4 * (j & 7));
    if (ok) codes[at] = make_uint2(word[0], word[1]);
  }
}

// Widths that 16-element pieces do not fit: the scales, a warp to a group, then
// the codes, a thread to a byte (whose two columns may belong to two segments).
__global__ void __launch_bounds__(256) scales_kernel(const __nv_bfloat16* __restrict__ W, long long rows, long long cols,
                                                     int segs, long long seg, int group, long long seg_groups,
                                                     __nv_bfloat16* __restrict__ scales) {
  const long long row_groups = segs * seg_groups, total = rows * row_groups;
  const int lane = threadIdx.x & 31;
  for (long long g = blockIdx.x * 8ll + (threadIdx.x >> 5); g < total; g += gridDim.x * 8ll) {
    const long long row = g / row_groups, in = g - row * row_groups, e = in / seg_groups, first = (in - e * seg_groups) * group;
    const __nv_bfloat16* src = W + row * cols + e * seg;
    __nv_bfloat16 m = __float2bfloat16_rn(0.f);
    for (int j = lane; j < group && first + j < seg; j += 32) m = __hmax_nan(m, __habs(src[first + j]));
#pragma unroll
    for (int d = 16; d; d >>= 1) m = __hmax_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) scales[g] = __float2bfloat16_rn(group_scale(__bfloat162float(m)));
  }
}
__global__ void __launch_bounds__(256) codes_kernel(const __nv_bfloat16* __restrict__ W, long long rows, long long cols,
                                                    int segs, long long seg, int group, long long seg_groups,
                                                    const __nv_bfloat16* __restrict__ scales, uint8_t* __restrict__ codes) {
  const long long row_bytes = (cols + 1) / 2, total = rows * row_bytes;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long row = i / row_bytes, c0 = (i - row * row_bytes) * 2;
    uint32_t byte = 0x88;  // a column behind the last: zero
    for (int h = 0; h < 2 && c0 + h < cols; ++h) {
      const long long c = c0 + h, e = c / seg, g = (c - e * seg) / group;
      float s = __bfloat162float(scales[(row * segs + e) * seg_groups + g]), inv, up;
      ready(s, inv, up);
      const uint32_t q = code_of(__bfloat162float(W[row * cols + c]) * up, s, inv);
      byte = h ? (byte & 0x0fu) | (q << 4) : (byte & 0xf0u) | q;
    }
    codes[i] = static_cast<uint8_t>(byte);
  }
}

__device__ __forceinline__ float value_of(uint32_t word, int j, float s) {
  return (static_cast<float>((word >> (4 * j)) & 15u) - 8.f) * s;
}
__global__ void __launch_bounds__(256) dequantize16_kernel(const uint2* __restrict__ codes,
                                                           const __nv_bfloat16* __restrict__ scales, long long pieces,
                                                           int row_pieces, int seg_pieces, int lanes, int seg_groups,
                                                           int segs, uint4* __restrict__ W) {
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < pieces; i += stride) {
    const long long row = i / row_pieces;
    const int in_row = static_cast<int>(i - row * row_pieces), e = in_row / seg_pieces, in = in_row - e * seg_pieces;
    const uint2 q = codes[i];
    const float s = __bfloat162float(scales[(row * segs + e) * seg_groups + in / lanes]);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = tc::pack_bf16x2(value_of(j < 4 ? q.x : q.y, 2 * (j & 3), s), value_of(j < 4 ? q.x : q.y, 2 * (j & 3) + 1, s));
    W[2 * i] = make_uint4(w[0], w[1], w[2], w[3]);
    W[2 * i + 1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                         const __nv_bfloat16* __restrict__ scales, long long rows,
                                                         long long cols, int segs, long long seg, int group,
                                                         long long seg_groups, __nv_bfloat16* __restrict__ W) {
  const long long row_bytes = (cols + 1) / 2, total = rows * cols;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long row = i / cols, c = i - row * cols, e = c / seg, g = (c - e * seg) / group;
    const float s = __bfloat162float(scales[(row * segs + e) * seg_groups + g]);
    W[i] = __float2bfloat16_rn(value_of(codes[row * row_bytes + c / 2], static_cast<int>(c & 1), s));
  }
}

// ================================================================ packing
// Eight codes in column order as a packed word (even columns in the low half).
__device__ __forceinline__ uint32_t half_of(uint32_t w) {  // nibbles 0, 2, 4, 6
  w &= 0x0f0f0f0fu;
  w = (w | (w >> 4)) & 0x00ff00ffu;
  return (w | (w >> 8)) & 0xffffu;
}
__device__ __forceinline__ uint32_t to_packed(uint32_t w) { return half_of(w) | (half_of(w >> 4) << 16); }

// A block of the packed layout to a thread block.
__global__ void __launch_bounds__(256) pack_kernel(W4Shape m, W4Codes c, uint8_t* packed, int unpack) {
  const long long chunks = m.chunks(), seg_chunks = m.seg_chunks(), cols = m.cols(), row_bytes = (cols + 1) / 2;
  const long long blocks = m.units() * chunks, groups = m.segs * m.seg_groups();
  for (long long b = blockIdx.x; b < blocks; b += gridDim.x) {
    const long long unit = b / chunks, chunk = b - unit * chunks, e = chunk / seg_chunks, in = (chunk - e * seg_chunks) * 128;
    uint8_t* blk = packed + b * m.block_bytes();
    for (int i = threadIdx.x; i < 1024 && !unpack; i += 256) {
      const int piece = i & 3, r = (i >> 2) & 127, tile = i >> 9;
      const W4Tile t = w4_tile(m, unit * 2 + tile);
      const uint8_t* src = static_cast<const uint8_t*>(c.codes[t.mat]) + (t.row0 + r) * row_bytes;
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const long long col = in + 32 * q + 8 * piece, from = e * m.seg + col;  // within the segment, the row
        const int live = r >= t.n || col >= m.seg ? 0 : (m.seg - col < 8 ? static_cast<int>(m.seg - col) : 8);
        uint32_t v = 0x88888888u;
        for (int j = 0; j < live; ++j) {
          const uint32_t code = (src[(from + j) >> 1] >> (4 * ((from + j) & 1))) & 15u;
          v = (v & ~(15u << (4 * j))) | (code << (4 * j));
        }
        w[q] = to_packed(v);
      }
      *reinterpret_cast<uint4*>(blk + tile * 8192 + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    for (int i = threadIdx.x; i < 256 * (128 / m.group); i += 256) {
      const int r = i & 127, tile = (i >> 7) & 1, sub = i >> 8;
      const W4Tile t = w4_tile(m, unit * 2 + tile);
      const long long g = in / m.group + sub;
      const bool ok = r < t.n && g < m.seg_groups();
      __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(blk + 16384) + i;
      __nv_bfloat16* src = static_cast<__nv_bfloat16*>(c.scales[t.mat]) + (t.row0 + r) * groups + e * m.seg_groups() + g;
      if (!unpack)
        *at = ok ? *src : __float2bfloat16_rn(0.f);
      else if (ok)
        *src = *at;
    }
  }
}
// The codes back: a thread to a byte of the natural layout.
__global__ void __launch_bounds__(256) unpack_codes_kernel(W4Shape m, W4Codes c, const uint8_t* packed) {
  const long long cols = m.cols(), row_bytes = (cols + 1) / 2, chunks = m.chunks(), seg_chunks = m.seg_chunks();
  for (long long ti = blockIdx.x; ti < m.tiles(); ti += gridDim.x) {
    const W4Tile t = w4_tile(m, ti);
    const uint8_t* from = packed + (ti >> 1) * chunks * m.block_bytes() + (ti & 1) * 8192;
    for (long long i = threadIdx.x; i < t.n * row_bytes; i += 256) {
      const long long r = i / row_bytes, c0 = (i - r * row_bytes) * 2;
      uint32_t byte = 0x88;
      for (int h = 0; h < 2 && c0 + h < cols; ++h) {
        const long long e = (c0 + h) / m.seg, in = c0 + h - e * m.seg, chunk = e * seg_chunks + in / 128;
        const int k = static_cast<int>(in & 127);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(from + chunk * m.block_bytes() + r * 64 +
                                                              ((((k >> 3) & 3) ^ ((r >> 1) & 3)) << 4) + (k >> 5) * 4);
        const uint32_t q = (w >> (16 * (k & 1) + 4 * ((k & 7) >> 1))) & 15u;
        byte = h ? (byte & 0x0fu) | (q << 4) : (byte & 0xf0u) | q;
      }
      static_cast<uint8_t*>(c.codes[t.mat])[(t.row0 + r) * row_bytes + c0 / 2] = static_cast<uint8_t>(byte);
    }
  }
}

// ================================================================ products
// y[token][row] = sum_g s[row][g] sum_{k in g} (code - 8) x[token][k], for up to
// 64 tokens at a time.  Bound by the one read of the codes.
//
// What is left to count are the instructions that make operands of codes.  A code
// in the low bits of a floating number with few exponent bits is a subnormal, code
// times its least number, and takes no addition or conversion:
//  * fp16 (up to 16 tokens): code * 2^-24, and four bits higher code * 2^-20.  A word's
//    eight codes are four operand registers after one shift and four masks.
//  * e4m3 (more tokens): code * 2^-9.  A word's eight codes are two registers after
//    one shift and two masks, and a product takes 32 columns instead of 16.
// (Codes made into bf16 take 11 instructions a word: 102 us instead of 68 for one
// token of the 70B feed-forward.)  For that
//  * the tokens are of the same type: a block of 128 columns of a token times a power
//    of two.  fp16: its largest element comes to 2^14..2^15, so that bf16's eight bits
//    are kept down to 2^-25 of it and what is smaller is rounded to 2^-40 of it; columns
//    2, 3, 6, 7 of each eight are times 2^-4 besides, for their codes' place.  e4m3: its
//    largest element comes to 2^7..2^8, and an element is the sum of two numbers of
//    four bits, the second times 2^-4: eight bits as bf16 down to 2^-13 of the largest, what is
//    smaller is rounded to 2^-21 of it.
//  * the codes' offset of 8 is taken off as the block's sum, -8 times the sum of the
//    group's 32, 64 or 128 columns: product * down + sum, times the row's scale.
// A group's product is scaled in 32 bits, so a result is as exact as the sums in 32
// bits.  (A scaled weight would have to be rounded.)  A token with an infinity or a
// NaN gets those throughout.
//
// A block takes a run of chunks (128 columns of a unit's 256 rows) of the list of
// all units' chunks, the same number as the others, whatever units they belong to;
// a run of chunks of one unit is a segment.  A unit that several blocks share is
// joined by the last of them to come, in the order of the columns.
using namespace tc;

// A block of tokens as the kernels keep it ("image"), for NT tokens: fp16 [2][NT][64],
// 64 columns each, or e4m3 [2][NT][128], the elements' first and second numbers, in
// rows of 128 bytes whose 16-byte pieces are swizzled by the token (piece i at i ^
// (token & 7)); e4m3 columns 0, 4, 1, 5, 2, 6, 3, 7 of each eight in this order, as a
// word's codes come apart.  Then float [8][NT]: -8 times the sums of its four 32-column
// parts, its two halves and the whole, in units of a code's 2^-24 or 2^-9, and the power
// of two that undoes the block's and is in the sums already.
__host__ __device__ constexpr int image_bytes(int nt) { return nt * 288; }
__host__ __device__ constexpr bool image_f8(int nt) { return nt > 16; }
constexpr int SUM_OF = 0, SUM_OF_HALF = 4, SUM_OF_ALL = 6, DOWN = 7;

struct ProductParams {
  W4Shape m;
  const uint8_t* packed;
  long long total;  // chunks of all units
  int chunks, block_bytes, units;
  long long n, out_rs;
  int epi;
  const __nv_bfloat16* bias;
  __nv_bfloat16* out;
  const uint8_t* image;  // [token tiles][chunks]
  uint8_t* image_out;    // the hidden activations', likewise
  int out_chunks;
  float* parts;   // [token tiles][blocks][2][NT][256]
  int* counters;  // [token tiles][units]
  int* err;
  int skip_load;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3),
                 hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float4 from_e4m3x4(uint32_t v) {
  const __half2 lo(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xffffu), __NV_E4M3)),
      hi(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v >> 16), __NV_E4M3));
  const float2 a = __half22float2(lo), b = __half22float2(hi);
  return make_float4(a.x, a.y, b.x, b.y);
}

// Columns 4 lane .. 4 lane + 3 of a token's block, by a warp, into an image.
template <bool F8>
__device__ __forceinline__ void store_block(uint8_t* image, int nt, int token, int lane, const float (&v)[4]) {
  const float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));  // without NaN
  const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu);
  // most * 2^e in 2^14..2^15, or 2^7..2^8
  const int e = min((F8 ? 134 : 141) - static_cast<int>(min(most >> 23, 254u)), 126);
  const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  float sum;
  if (F8) {
    const uint32_t first = e4m3x4(v[0] * up, v[1] * up, v[2] * up, v[3] * up);
    const float4 f = from_e4m3x4(first);
    const uint32_t second = e4m3x4(16.f * fmaf(v[0], up, -f.x), 16.f * fmaf(v[1], up, -f.y), 16.f * fmaf(v[2], up, -f.z),
                                   16.f * fmaf(v[3], up, -f.w));
    const float4 g = from_e4m3x4(second);
    sum = ((f.x + f.y) + (f.z + f.w)) + 0.0625f * ((g.x + g.y) + (g.z + g.w));
    // (infinities are cut to the largest number: the sum tells of them, and of NaN)
    if (most >= 0x7f800000u || !(v[0] + v[1] + v[2] + v[3] == v[0] + v[1] + v[2] + v[3])) sum = __uint_as_float(0x7fc00000u);
    const bool odd = lane & 1;
    const uint32_t first2 = __shfl_xor_sync(0xffffffffu, first, 1), second2 = __shfl_xor_sync(0xffffffffu, second, 1);
    uint8_t* at = image + token * 128 + (((lane >> 2) ^ (token & 7)) << 4) + (lane & 3) * 4;
    *reinterpret_cast<uint32_t*>(at) = odd ? __byte_perm(first2, first, 0x7362) : __byte_perm(first, first2, 0x5140);
    *reinterpret_cast<uint32_t*>(at + nt * 128) = odd ? __byte_perm(second2, second, 0x7362) : __byte_perm(second, second2, 0x5140);
  } else {
    const __half2 lo = __floats2half2_rn(v[0] * up, v[1] * up), hi = __floats2half2_rn(v[2] * up * 0.0625f, v[3] * up * 0.0625f);
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    sum = (a.x + a.y) + 16.f * (b.x + b.y);
    uint8_t* at = image + (lane >> 4) * (nt * 128) + token * 128 + ((((lane & 15) >> 1) ^ (token & 7)) << 4) + (lane & 1) * 8;
    *reinterpret_cast<uint2*>(at) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  sum *= (F8 ? -0.015625f : -4.76837158203125e-7f) * down;  // -8 * 2^-9, -8 * 2^-24
  const float two = sum + __shfl_xor_sync(0xffffffffu, sum, 8), all = two + __shfl_xor_sync(0xffffffffu, two, 16);
  float* tail = reinterpret_cast<float*>(image + nt * 256) + token;
  if ((lane & 7) == 0) tail[(SUM_OF + (lane >> 3)) * nt] = sum;
  if ((lane & 15) == 0) tail[(SUM_OF_HALF + (lane >> 4)) * nt] = two;
  if (lane == 0) tail[SUM_OF_ALL * nt] = all;
  if (lane == 0) tail[DOWN * nt] = down;
}

struct PrepareParams {
  const __nv_bfloat16* x;
  long long x_seg, x_rs, seg, seg_chunks, chunks, n;
  int nt, tiles;
  uint8_t* image;  // [tiles][chunks]
  int *err, *counters, n_counters;
};
// The kernel before a call's first product: the tokens' blocks, a warp to a token's;
// clears what the call counts in.  It lets others start when everything before it
// on the stream is done: the products behind it read their weights without a further wait.
__global__ void __launch_bounds__(256) prepare_kernel(const __grid_constant__ PrepareParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.err) *p.err = 0;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < p.n_counters; i += gridDim.x * 256) p.counters[i] = 0;
  for (long long i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < p.tiles * p.chunks * p.nt; i += gridDim.x * 8ll) {
    const long long block = i / p.nt, tile = block / p.chunks, chunk = block - tile * p.chunks;
    const long long e = chunk / p.seg_chunks, col = (chunk - e * p.seg_chunks) * 128 + lane * 4;
    const int in = static_cast<int>(i - block * p.nt);
    const long long token = tile * p.nt + in;
    float v[4] = {};
    if (token < p.n && col < p.seg) {  // segments end at multiples of 8
      const uint2 w = *reinterpret_cast<const uint2*>(p.x + token * p.x_rs + e * p.x_seg + col);
      v[0] = bf16_at(w.x, 0), v[1] = bf16_at(w.x, 1), v[2] = bf16_at(w.y, 0), v[3] = bf16_at(w.y, 1);
    }
    if (image_f8(p.nt))
      store_block<true>(p.image + block * image_bytes(p.nt), p.nt, in, lane, v);
    else
      store_block<false>(p.image + block * image_bytes(p.nt), p.nt, in, lane, v);
  }
}

// Bounded wait on an mbarrier phase, as tc::Waiter's, for waits that mostly last
// some hundred cycles: the clock, which takes longer than that to read, is looked
// at only after many tries.
struct Wait {
  volatile int* abort_flag;
  int* err;
  unsigned long long timeout_ns;
  __device__ __noinline__ bool slow(uint64_t* bar, uint32_t parity, bool honour_abort) const {
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
      if (mbar_try_wait(bar, parity)) return true;
      if (n & 63u) continue;
      if (honour_abort && *abort_flag) return false;
      const uint64_t t = global_timer();
      if (!t0) t0 = t;
      if (t - t0 > timeout_ns) {
        *abort_flag = 1;
        atomicOr(err, DEV_ERR_TIMEOUT);
        __threadfence();
        return false;
      }
    }
  }
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    return mbar_try_wait(bar, parity) || slow(bar, parity, true);
  }
  __device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) const {
    if (!mbar_try_wait(bar, parity)) slow(bar, parity, false);
  }
  // of a whole warp
  __device__ __forceinline__ void warp(uint64_t* bar, uint32_t parity) const {
    if (!mbar_try_wait(bar, parity)) slow(bar, parity, true);
    __syncwarp();
  }
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float ld_shared_f(uint32_t addr) { return __uint_as_float(ld_shared(addr)); }
__device__ __forceinline__ float ld_shared_scale(uint32_t addr) {  // a bf16
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr));
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// The codes at bits 0-3 and 16-19 as two fp16 numbers, and those at bits 4-7 and 20-23.
__device__ __forceinline__ uint32_t low(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t high(uint32_t w) { return w & 0x00f000f0u; }
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// The run of chunks of a block.
struct Run {
  long long first;
  int count;
  __device__ __forceinline__ explicit Run(const ProductParams& p) {
    first = p.total * blockIdx.x / gridDim.x;
    count = static_cast<int>(p.total * (blockIdx.x + 1) / gridDim.x - first);
  }
};

// The copying thread: chunks of weights (the packed block as it lies) and of tokens
// (the image) into a ring of stages, tokens first.
template <typename R>
__device__ __forceinline__ void copy_chunks(const ProductParams& p, const Run& run, uint8_t* ring, uint64_t* full,
                                            uint64_t* empty, const Wait& W) {
  // A single token tile reads the weights once.
  const uint64_t often = l2_policy_evict_normal(), once = gridDim.y == 1 ? l2_policy_evict_first() : often;
  const uint8_t* src = p.packed + run.first * p.block_bytes;
  const uint8_t* image = p.image + static_cast<long long>(blockIdx.y) * p.chunks * image_bytes(R::NT);
  int c = static_cast<int>(run.first % p.chunks);
  auto weights = [&](int stage) {
    mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(p.block_bytes + image_bytes(R::NT)));
    bulk_load(ring + stage * R::STAGE + R::X_BYTES, src, static_cast<uint32_t>(p.block_bytes), &full[stage], once);
    src += p.block_bytes;
  };
  auto tokens = [&](int stage) {
    bulk_load(ring + stage * R::STAGE, image + static_cast<long long>(c) * image_bytes(R::NT), image_bytes(R::NT),
              &full[stage], often);
    if (++c == p.chunks) c = 0;
  };
  // The weights are not the previous kernel's to write (what wrote them is done
  // before the call's first kernel lets others start); the tokens are.
  const int ahead = run.count < R::STAGES ? run.count : R::STAGES;
  for (int i = 0; i < ahead; ++i) weights(i);
  grid_dep_wait();
  for (int i = p.skip_load ? 1 : 0; i < ahead; ++i) tokens(i);
  int issued = ahead, stage = 0;
  uint32_t phase = 0;
  for (int i = ahead; i < run.count; ++i, ++issued) {
    if (!W(&empty[stage], phase)) break;
    weights(stage);
    tokens(stage);
    if (++stage == R::STAGES) {
      stage = 0;
      phase ^= 1;
    }
  }
  // every issued copy lands before the block may exit
  for (int i = issued > R::STAGES ? issued - R::STAGES : 0; i < issued; ++i) W.drain(&full[i % R::STAGES], (i / R::STAGES) & 1);
}

// Four neighbouring rows of a token, by a warp that has 128: bias or activation, and out.
template <int NT>
__device__ __forceinline__ void write4(const ProductParams& p, int in_tile, long long row, int lane, float4 v) {
  float a[4] = {v.x, v.y, v.z, v.w};
  if (p.epi == W4_OUT) {
    const long long token = static_cast<long long>(blockIdx.y) * NT + in_tile;
    if (token >= p.n || row >= p.m.rows) return;  // rows are a multiple of 8
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] += __bfloat162float(p.bias[row + i]);
    }
    *reinterpret_cast<uint2*>(p.out + token * p.out_rs + row) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
    return;
  }
  const int chunk = static_cast<int>(row >> 7);
  if (chunk >= p.out_chunks) return;
  if (p.epi == W4_GELU) {
    const long long t = row / p.m.sp, in = row - t * p.m.sp;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = gelu_tanh_f(a[i] + (p.bias && in + i < p.m.s ? __bfloat162float(p.bias[t * p.m.s + in + i]) : 0.f));
  }
  store_block<image_f8(NT)>(p.image_out + (static_cast<long long>(blockIdx.y) * p.out_chunks + chunk) * image_bytes(NT), NT, in_tile, lane, a);
}

// The end of a segment of `unit`, whose sums lie in shared memory, [token][row], 256
// rows and a few of padding: out if the segment is the whole unit, else as a part,
// and the last block of the unit joins the parts.  By the WARPS warps from FIRST on,
// which then may write the sums anew.
constexpr int SUM_PITCH = 256 + 8;
template <int NT, int WARPS, int FIRST>
__device__ __forceinline__ void finish_segment(const ProductParams& p, long long unit, const float* sum, int* s_last,
                                               const Wait& W) {
  // a thread: rows 4 q .. 4 q + 3 of tile 0 and of tile 1, of a token of every WARPS
  const int warp = (threadIdx.x >> 5) - FIRST, lane = threadIdx.x & 31, q4 = lane * 4;
  const long long u0 = unit * p.chunks, u1 = u0 + p.chunks - 1;
  const int C = gridDim.x;
  const int c0 = static_cast<int>(((u0 + 1) * C - 1) / p.total), c1 = static_cast<int>(((u1 + 1) * C - 1) / p.total);
  bool store = true;
  float* parts = p.parts + static_cast<long long>(blockIdx.y) * C * 2 * (NT * 256) + q4;
  auto slot = [&](int b) { return static_cast<long long>(2 * b + (b == c0)) * (NT * 256); };
  if (c0 != c1) {
    float* to = parts + slot(blockIdx.x);
#pragma unroll
    for (int token = warp; token < NT; token += WARPS) {
      __stcg(reinterpret_cast<float4*>(to + token * 256), *reinterpret_cast<const float4*>(sum + token * SUM_PITCH + q4));
      __stcg(reinterpret_cast<float4*>(to + token * 256 + 128), *reinterpret_cast<const float4*>(sum + token * SUM_PITCH + 128 + q4));
    }
    __threadfence();
    bar_sync(1, WARPS * 32);
    if (threadIdx.x == FIRST * 32) {
      __threadfence();
      *s_last = atomicAdd(p.counters + static_cast<long long>(blockIdx.y) * p.units + unit, 1) == c1 - c0;
      __threadfence();
    }
    bar_sync(1, WARPS * 32);
    store = *s_last;
  }
  if (store && *W.abort_flag == 0) {
#pragma unroll 1
    for (int token = warp; token < NT; token += WARPS) {
      float4 v0, v1;
      if (c0 == c1) {
        v0 = *reinterpret_cast<const float4*>(sum + token * SUM_PITCH + q4);
        v1 = *reinterpret_cast<const float4*>(sum + token * SUM_PITCH + 128 + q4);
      } else {
        v0 = v1 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int b = c0; b <= c1; ++b) {
          const float* from = parts + slot(b) + token * 256;
          v0 = add4(v0, __ldcg(reinterpret_cast<const float4*>(from)));
          v1 = add4(v1, __ldcg(reinterpret_cast<const float4*>(from + 128)));
        }
      }
      const float one = image_f8(NT) ? 512.f : 16777216.f;  // 2^9, 2^24: a code's unit
      v0 = make_float4(v0.x * one, v0.y * one, v0.z * one, v0.w * one);
      v1 = make_float4(v1.x * one, v1.y * one, v1.z * one, v1.w * one);
      if (p.epi == W4_SWIGLU) {  // tile 1 has the second matrix's rows of the same hidden slots
        v0.x *= sigmoid_f(v0.x) * v1.x;
        v0.y *= sigmoid_f(v0.y) * v1.y;
        v0.z *= sigmoid_f(v0.z) * v1.z;
        v0.w *= sigmoid_f(v0.w) * v1.w;
        write4<NT>(p, token, unit * 128 + q4, lane, v0);
      } else {
        write4<NT>(p, token, unit * 256 + q4, lane, v0);
        write4<NT>(p, token, unit * 256 + 128 + q4, lane, v1);
      }
    }
  }
  bar_sync(1, WARPS * 32);
}

// ---------------------------------------------------------------- few tokens
// Up to 16 tokens: m16n8k16 matrix instructions on registers.  They take 2.05 cycles
// an SM (measured), 8 tokens of a chunk 262 of the some 720 that its bytes take, 16
// tokens 525; the tensor-memory products take 768 whatever the number of tokens,
// besides the way of the weights into tensor memory.
//
// The order of a product's columns is free as long as both operands have it: lane
// t of a row's four takes the 32-bit words of codes 8 t .. 8 t + 7 of 32 columns, their
// pairs as the halves of two k16 steps, and so reads the same 8 columns of a token
// in one piece.  Token t of eight stands in column 2 t, token t + 4 in column 2 t +
// 1 of the product, so that the two tokens of an eighth of a warp lie in different
// halves of the swizzled rows.
// 8 warps, 32 rows of the unit each, two blocks per SM.
template <int NT_>
struct Few {
  static constexpr int NT = NT_, X_BYTES = image_bytes(NT), STAGE = X_BYTES + 18432;
  static constexpr int STAGES = NT == 8 ? 5 : 4;
  static constexpr int M_SUM = STAGES * STAGE, SMEM = M_SUM + NT * SUM_PITCH * 4 + 128;
  static_assert(2 * (SMEM + 2048) <= 233472, "two blocks per SM");
};
constexpr int FEW_WARPS = 8, FEW_THREADS = (FEW_WARPS + 1) * 32;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// SUBS: groups of a chunk.
template <int NT, int SUBS>
__global__ void __launch_bounds__(FEW_THREADS, 2) few_kernel(const __grid_constant__ ProductParams p) {
  using F = Few<NT>;
  constexpr int NB = NT / 8;  // products of eight tokens
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  __shared__ uint64_t full[F::STAGES], empty[F::STAGES];
  __shared__ int s_abort, s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < F::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], FEW_WARPS);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  __syncthreads();
  grid_dep_launch();
  const Wait W{&s_abort, p.err, p.timeout_ns};
  const Run run(p);
  if (warp == FEW_WARPS) {
    if (lane == 0) copy_chunks<F>(p, run, smem, full, empty, W);
    return;
  }
  const int t = lane & 3, i8 = lane >> 2;
  const int row0 = warp * 32 + i8;  // of the unit; the warp's rows: + 0, 8, 16, 24
  const int tok0 = (i8 & 1) * 4 + (i8 >> 1);
  // bytes from a stage's start
  const uint32_t at_x = tok0 * 128, swz = tok0 & 7;
  const uint32_t at_w = F::X_BYTES + row0 * 64 + ((t ^ ((i8 >> 1) & 3)) << 4), at_s = F::X_BYTES + 16384 + row0 * 2;
  const uint32_t at_tail = NT * 256 + t * 4;  // of token t
  float* sum = reinterpret_cast<float*>(smem + F::M_SUM);
  uint64_t acc[2][NB][2] = {};  // rows row0 + 16 m + 8 h, tokens 8 b + t and 8 b + t + 4
  grid_dep_wait();  // the counters are clear, and nobody reads the outputs or parts of before
  int stage = 0;
  uint32_t phase = 0;
  long long unit = run.first / p.chunks;
  int chunk = static_cast<int>(run.first - unit * p.chunks);
#pragma unroll 1
  for (int i = 0; i < run.count; ++i) {
    const uint32_t st = smem_u32(smem) + stage * F::STAGE;
    W.warp(&full[stage], phase);
    uint4 w[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[m][h] = ld_shared_v4(st + at_w + m * 1024 + h * 512);
    uint64_t down[NB], sums[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t at = st + at_tail + DOWN * NT * 4 + b * 32;
      down[b] = pack2(ld_shared_f(at), ld_shared_f(at + 16));
    }
    float c[2][NB][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      constexpr int PER = 4 / SUBS;
      if (q % PER == 0) {
        constexpr int FIRST = SUBS == 1 ? SUM_OF_ALL : SUBS == 2 ? SUM_OF_HALF : SUM_OF;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t at = st + at_tail + (FIRST + q / PER) * NT * 4 + b * 32;
          sums[b] = pack2(ld_shared_f(at), ld_shared_f(at + 16));
#pragma unroll
          for (int m = 0; m < 2; ++m) c[m][b][0] = c[m][b][1] = c[m][b][2] = c[m][b][3] = 0.f;
        }
      }
      uint4 x[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        x[b] = ld_shared_v4(st + at_x + (q >> 1) * (NT * 128) + b * 1024 + ((((q & 1) * 4 + t) ^ swz) << 4));
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t w0 = q == 0 ? w[m][0].x : q == 1 ? w[m][0].y : q == 2 ? w[m][0].z : w[m][0].w;
        uint32_t w1 = q == 0 ? w[m][1].x : q == 1 ? w[m][1].y : q == 2 ? w[m][1].z : w[m][1].w;
#pragma unroll
        for (int b = 0; b < NB; ++b) mma(c[m][b], low(w0), low(w1), high(w0), high(w1), x[b].x, x[b].y);
        w0 >>= 8;
        w1 >>= 8;
#pragma unroll
        for (int b = 0; b < NB; ++b) mma(c[m][b], low(w0), low(w1), high(w0), high(w1), x[b].z, x[b].w);
      }
      if (q % PER != PER - 1) continue;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float s = ld_shared_scale(st + at_s + (q / PER) * 512 + (16 * m + 8 * h) * 2);
          const uint64_t s2 = pack2(s, s);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[m][b][h] = fma2(s2, fma2(pack2(c[m][b][2 * h], c[m][b][2 * h + 1]), down[b], sums[b]), acc[m][b][h]);
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[stage]);
    if (++stage == F::STAGES) {
      stage = 0;
      phase ^= 1;
    }
    if (++chunk < p.chunks && i + 1 < run.count) continue;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 v = unpack2(acc[m][b][h]);
          sum[(8 * b + t) * SUM_PITCH + row0 + 16 * m + 8 * h] = v.x;
          sum[(8 * b + t + 4) * SUM_PITCH + row0 + 16 * m + 8 * h] = v.y;
          acc[m][b][h] = 0;
        }
    bar_sync(1, FEW_WARPS * 32);
    finish_segment<NT, FEW_WARPS, 0>(p, unit, sum, &s_last, W);
    chunk = 0;
    ++unit;
  }
}

// ---------------------------------------------------------------- more tokens
// 32 tokens to a block, several token tiles side by side (the weights come from L2
// for all but the first).  The weights are the A operand of tcgen05.mma, 128 rows at
// a time, in tensor memory (in shared memory they would be written and read once
// more), the tokens its N: 64 columns, both numbers of 32 tokens.  A product (M 128, K
// 32) takes 46 cycles whatever N up to 64 is, as one of fp16 with K 16 does (measured,
// from tensor or shared memory).  One block per SM, a step being a group's columns:
//  * two groups of four warps, a row of tile 0 or 1 to a thread, write the row's
//    codes to tensor memory as operands, a step ahead of the products;
//  * two groups of four warps, a row of either tile and 16 tokens to a thread, read a
//    step's products back while the next's run, scale and add them (a token's two
//    numbers are loaded once for both rows: shared memory's loads are what the time
//    goes by, 109 us with a row and all tokens to a thread);
//  * a warp copies, a warp issues the products.
// (With fp16 operands a step has 16 products, and the writes of the maker warps on the
// issuing warp's scheduler wait behind them: 113 us for 32 tokens of the 70B
// feed-forward.  One thread after the other making operands, waiting and reading
// back: 116 us.)
// Every wait is bounded (abort flag and error word); after an abort the warps run
// on without waiting, so that they meet at the block's barriers.
template <int NT_>
struct Ring {
  static constexpr int NT = NT_, X_BYTES = (image_bytes(NT) + 1023) / 1024 * 1024, STAGE = X_BYTES + 18432;
  static constexpr int STAGES = 6;
  static constexpr int M_SUM = STAGES * STAGE, SMEM = M_SUM + NT * SUM_PITCH * 4 + 1024;
  static constexpr int MAKERS = 8, READERS = 8, WARPS = MAKERS + READERS + 2, THREADS = WARPS * 32;
  static_assert(SMEM <= 232448 - 1024, "shared memory per block");
};

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void tmem_load8(uint32_t at, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(at));
}
// Waits for loads and names their registers, so that no use of them moves before the wait.
__device__ __forceinline__ void tmem_loaded(uint32_t (&a)[8], uint32_t (&b)[8], uint32_t (&c)[8], uint32_t (&d)[8]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    asm volatile("" : "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(b[i]), "+r"(b[i + 1]), "+r"(b[i + 2]), "+r"(b[i + 3]));
    asm volatile("" : "+r"(c[i]), "+r"(c[i + 1]), "+r"(c[i + 2]), "+r"(c[i + 3]), "+r"(d[i]), "+r"(d[i + 1]), "+r"(d[i + 2]), "+r"(d[i + 3]));
  }
}
__device__ __forceinline__ void tmem_store8(uint32_t at, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// A in tensor memory, four consecutive columns of a row to a 32-bit cell.
__device__ __forceinline__ void umma_f8_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int NT, int SUBS>
__global__ void __launch_bounds__(Ring<NT>::THREADS, 1) product_kernel(const __grid_constant__ ProductParams p) {
  using R = Ring<NT>;
  constexpr int KSTEPS = 4 / SUBS;  // K = 32 steps of a group
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // of a buffer: operands written, products done, products read
  __shared__ uint64_t full[R::STAGES], empty[R::STAGES], a_full[2], d_full[2], d_free[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort, s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], R::MAKERS + R::READERS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], R::MAKERS);
      mbar_init(&d_full[i], 1);
      mbar_init(&d_free[i], R::READERS);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == R::WARPS - 1) tmem_alloc(&tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  // operands of a tile's buffer at 128 tile + 64 buffer (32 columns), products 256 columns on
  const uint32_t tmem = tmem_slot;
  const Wait W{&s_abort, p.err, p.timeout_ns};
  const Run run(p);

  if (warp == R::WARPS - 2) {
    if (lane == 0) copy_chunks<R>(p, run, smem, full, empty, W);
    __syncwarp();
  } else if (warp == R::WARPS - 1) {
    // ------------------------------------------------ products
    // The warp stays together and one lane waits and issues: what a product is told is
    // the same for all lanes, else it takes three times as long to issue.  One wait
    // a step beside the chunk's, for both tiles: a wait takes 150 cycles even where
    // it finds what it waits for.
    const bool leader = elect_one();
    constexpr uint32_t ID = (1u << 4) | (static_cast<uint32_t>(2 * NT >> 3) << 17) | (8u << 24);  // e4m3 x e4m3 -> fp32, M = 128
    const uint64_t x_desc = sw128_desc(smem_u32(smem), 16);
    int stage = 0;
    uint32_t phase = 0, step = 0;
#pragma unroll 1
    for (int i = 0; i < run.count; ++i) {
      if (leader) W(&full[stage], phase);
      const uint64_t xd = x_desc + static_cast<uint64_t>(stage * (R::STAGE >> 4));
#pragma unroll
      for (int sub = 0; sub < SUBS; ++sub, ++step) {
        const uint32_t buf = step & 1, at = tmem + buf * 64;
        if (leader) W(&a_full[buf], (step >> 1) & 1);
        __syncwarp();
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int tile = 0; tile < 2; ++tile)
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) {
              const int ks = sub * KSTEPS + k;
              umma_f8_ta(at + 256 + tile * 128, at + tile * 128 + k * 8, xd + static_cast<uint64_t>(ks * 32 >> 4), ID, k > 0);
            }
          umma_commit(&d_full[buf]);
        }
        __syncwarp();
      }
      if (++stage == R::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (leader) {
      umma_commit(&drain);
      W.drain(&drain, 0);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int stage = 0;
    uint32_t phase = 0, step = 0;
    if (warp < R::MAKERS) {
      // ------------------------------------------------ operands
      const int tile = warp >> 2;
      const uint32_t at_w = R::X_BYTES + tile * 8192 + r * 64, swz = (r >> 1) & 3;
      constexpr int PIECES = 4 / SUBS;
#pragma unroll 1
      for (int i = 0; i < run.count; ++i) {
        const uint32_t st = smem_u32(smem) + stage * R::STAGE;
        W.warp(&full[stage], phase);
        uint4 v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = ld_shared_v4(st + at_w + ((t ^ swz) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub, ++step) {
          const uint32_t buf = step & 1, uses = step >> 1, at = lanes + tile * 128 + buf * 64;
          W.warp(&d_full[buf], (uses & 1) ^ 1);  // the products that had the buffer are done
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < PIECES; ++q) {
            const int word = sub * PIECES + q;
            uint32_t o[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t w = word == 0 ? v[t].x : word == 1 ? v[t].y : word == 2 ? v[t].z : v[t].w;
              o[2 * t] = w & 0x0f0f0f0fu;
              o[2 * t + 1] = (w >> 4) & 0x0f0f0f0fu;
            }
            tmem_store8(at + q * 8, o);
          }
          tmem_wait_st();
          W.warp(&d_free[buf], (uses & 1) ^ 1);  // and read
          tc_fence_before();
          if (lane == 0) mbar_arrive(&a_full[buf]);
        }
        if (++stage == R::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    } else {
      // ------------------------------------------------ products back, sums
      const int token0 = ((warp - R::MAKERS) >> 2) * (NT / 2);
      const uint32_t at_s = R::X_BYTES + 16384 + r * 2;
      float* sum = reinterpret_cast<float*>(smem + R::M_SUM);
      grid_dep_wait();  // the counters are clear, and nobody reads the outputs or parts of before
      uint64_t acc[2][NT / 4] = {};  // rows r and 128 + r
      const uint64_t second = pack2(0.0625f, 0.0625f);
      long long unit = run.first / p.chunks;
      int chunk = static_cast<int>(run.first - unit * p.chunks);
#pragma unroll 1
      for (int i = 0; i < run.count; ++i) {
        const uint32_t st = smem_u32(smem) + stage * R::STAGE;
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub, ++step) {
          const uint32_t buf = step & 1, at = lanes + 256 + buf * 64 + token0;
          W.warp(&d_full[buf], (step >> 1) & 1);  // (the chunk has landed, else there were no products)
          tc_fence_after();
          constexpr int FIRST = SUBS == 1 ? SUM_OF_ALL : SUBS == 2 ? SUM_OF_HALF : SUM_OF;
          const uint32_t at_sum = st + NT * 256 + ((FIRST + sub) * NT + token0) * 4, at_down = st + NT * 256 + (DOWN * NT + token0) * 4;
          const float s0 = ld_shared_scale(st + at_s + sub * 512), s1 = ld_shared_scale(st + at_s + sub * 512 + 256);
          const uint64_t s2[2] = {pack2(s0, s0), pack2(s1, s1)};
#pragma unroll
          for (int c = 0; c < NT / 2; c += 8) {  // eight tokens
            uint32_t d[2][2][8];  // [tile][number]
#pragma unroll
            for (int m = 0; m < 4; ++m) tmem_load8(at + (m >> 1) * 128 + (m & 1) * NT + c, d[m >> 1][m & 1]);
            uint64_t sums[4], down[4];
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(sums[j]), "=l"(sums[j + 1]) : "r"(at_sum + (c + 2 * j) * 4));
              asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(down[j]), "=l"(down[j + 1]) : "r"(at_down + (c + 2 * j) * 4));
            }
            tmem_loaded(d[0][0], d[0][1], d[1][0], d[1][1]);
            if (c + 8 == NT / 2) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&d_free[buf]);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                auto two = [&](int k) { return pack2(__uint_as_float(d[m][k][2 * j]), __uint_as_float(d[m][k][2 * j + 1])); };
                uint64_t& a = acc[m][c / 2 + j];
                a = fma2(s2[m], fma2(fma2(second, two(1), two(0)), down[j], sums[j]), a);
              }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == R::STAGES) {
          stage = 0;
          phase ^= 1;
        }
        if (++chunk < p.chunks && i + 1 < run.count) continue;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < NT / 4; ++j) {
            const float2 v = unpack2(acc[m][j]);
            float* to = sum + (token0 + 2 * j) * SUM_PITCH + m * 128 + r;
            to[0] = v.x;
            to[SUM_PITCH] = v.y;
            acc[m][j] = 0;
          }
        bar_sync(1, R::READERS * 32);
        finish_segment<NT, R::READERS, R::MAKERS>(p, unit, sum, &s_last, W);
        chunk = 0;
        ++unit;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == R::WARPS - 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename... KArgs, typename... Args>
void launch_dep(void (*kern)(KArgs...), dim3 grid, int block, int smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kern, args...);
}

// Launches an instance of a product's kernel, after raising its shared-memory limit
// on a device where that is not done.
template <auto KERNEL, int BLOCK, int SMEM, typename... Args>
int launch_inst(dim3 grid, cudaStream_t st, const Args&... args) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TP_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) return TP_ERR_CUDA;
    done.fetch_or(bit);
  }
  launch_dep(KERNEL, grid, BLOCK, SMEM, st, args...);
  return TP_OK;
}
template <int NT>
int launch_few(const ProductParams& p, dim3 grid, cudaStream_t st) {
  constexpr int SMEM = Few<NT>::SMEM;
  if (p.m.group == 128) return launch_inst<few_kernel<NT, 1>, FEW_THREADS, SMEM>(grid, st, p);
  if (p.m.group == 64) return launch_inst<few_kernel<NT, 2>, FEW_THREADS, SMEM>(grid, st, p);
  return launch_inst<few_kernel<NT, 4>, FEW_THREADS, SMEM>(grid, st, p);
}
template <int NT>
int launch_product(const ProductParams& p, dim3 grid, cudaStream_t st) {
  constexpr int SMEM = Ring<NT>::SMEM;
  if (p.m.group == 128) return launch_inst<product_kernel<NT, 1>, Ring<NT>::THREADS, SMEM>(grid, st, p);
  if (p.m.group == 64) return launch_inst<product_kernel<NT, 2>, Ring<NT>::THREADS, SMEM>(grid, st, p);
  return launch_inst<product_kernel<NT, 4>, Ring<NT>::THREADS, SMEM>(grid, st, p);
}

// How a product of n tokens is cut: NT tokens to a block, `tiles` of them, `blocks`
// runs of chunks.
struct Cut {
  int nt, tiles, blocks;
};
Cut cut_of(const W4Shape& m, int64_t n, int num_sms) {
  Cut c;
  c.nt = n <= 8 ? 8 : n <= 16 ? 16 : 32;
  c.tiles = static_cast<int>((n + c.nt - 1) / c.nt);
  const int64_t most = c.nt <= 16 ? 2 * num_sms : std::max(num_sms / c.tiles, 1), total = m.units() * m.chunks();
  c.blocks = static_cast<int>(std::min<int64_t>(most, total));
  return c;
}

// A grid of at most 32 blocks per SM.
unsigned grid_of(long long blocks) { return static_cast<unsigned>(std::min<long long>(std::max<long long>(blocks, 1), 32 * 152)); }
int launched() { return cudaPeekAtLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA; }

}  // namespace w4

int launch_w4_quantize(const void* W, int64_t rows, int64_t cols, int64_t segs, int group, void* codes, void* scales,
                       cudaStream_t st) {
  using namespace w4;
  const int64_t seg = cols / segs, seg_groups = (seg + group - 1) / group;
  auto* sc = static_cast<__nv_bfloat16*>(scales);
  if (seg % 16 == 0) {
    const int lanes = group / 16;
    const long long places = rows * segs * seg_groups * lanes;
    quantize16_kernel<<<grid_of((places + 255) / 256), 256, 0, st>>>(
        static_cast<const uint4*>(W), rows * (cols / 16), static_cast<int>(cols / 16), static_cast<int>(seg / 16), lanes,
        static_cast<int>(seg_groups), static_cast<int>(segs), static_cast<uint2*>(codes), sc);
    return launched();
  }
  const auto* w = static_cast<const __nv_bfloat16*>(W);
  scales_kernel<<<grid_of((rows * segs * seg_groups + 7) / 8), 256, 0, st>>>(w, rows, cols, static_cast<int>(segs), seg,
                                                                             group, seg_groups, sc);
  codes_kernel<<<grid_of((rows * ((cols + 1) / 2) + 255) / 256), 256, 0, st>>>(
      w, rows, cols, static_cast<int>(segs), seg, group, seg_groups, sc, static_cast<uint8_t*>(codes));
  return launched();
}

int launch_w4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, int64_t segs, int group,
                         void* W, cudaStream_t st) {
  using namespace w4;
  const int64_t seg = cols / segs, seg_groups = (seg + group - 1) / group;
  const auto* sc = static_cast<const __nv_bfloat16*>(scales);
  if (seg % 16 == 0) {
    const long long pieces = rows * (cols / 16);
    dequantize16_kernel<<<grid_of((pieces + 255) / 256), 256, 0, st>>>(
        static_cast<const uint2*>(codes), sc, pieces, static_cast<int>(cols / 16), static_cast<int>(seg / 16), group / 16,
        static_cast<int>(seg_groups), static_cast<int>(segs), static_cast<uint4*>(W));
  } else {
    dequantize_kernel<<<grid_of((rows * cols + 255) / 256), 256, 0, st>>>(
        static_cast<const uint8_t*>(codes), sc, rows, cols, static_cast<int>(segs), seg, group, seg_groups,
        static_cast<__nv_bfloat16*>(W));
  }
  return launched();
}

int launch_w4_pack(const W4Shape& m, const W4Codes& c, void* packed, int unpack, cudaStream_t st) {
  using namespace w4;
  pack_kernel<<<grid_of(m.units() * m.chunks()), 256, 0, st>>>(m, c, static_cast<uint8_t*>(packed), unpack);
  if (unpack)
    unpack_codes_kernel<<<grid_of(m.tiles()), 256, 0, st>>>(m, c, static_cast<const uint8_t*>(packed));
  return launched();
}

size_t w4_product_scratch(const W4Shape& m, int64_t n, int num_sms) {
  const w4::Cut c = w4::cut_of(m, n, num_sms);
  return static_cast<size_t>(c.blocks) * c.tiles * 2 * 256 * c.nt * sizeof(float);
}
int64_t w4_product_counters(const W4Shape& m, int64_t n) { return m.units() * ((n + 15) / 16); }

size_t w4_image_bytes(const W4Shape& m, int64_t n) {
  const w4::Cut c = w4::cut_of(m, n, 1);
  return static_cast<size_t>(m.chunks()) * c.tiles * w4::image_bytes(c.nt);
}

int launch_w4_prepare(const W4Product& a, int* err, int64_t n_counters, LaunchCtx& ctx) {
  using namespace w4;
  const Cut c = cut_of(a.m, a.n, ctx.num_sms);
  PrepareParams p{};
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.x_seg = a.x_seg;
  p.x_rs = a.x_rs;
  p.seg = a.m.seg;
  p.seg_chunks = a.m.seg_chunks();
  p.chunks = a.m.chunks();
  p.n = a.n;
  p.nt = c.nt;
  p.tiles = c.tiles;
  p.image = static_cast<uint8_t*>(a.image);
  p.err = err;
  p.counters = a.counters;
  p.n_counters = static_cast<int>(n_counters);
  const int64_t warps = p.tiles * p.chunks * p.nt;
  if (ctx.before) ctx.before(ctx.user, "prepare4", ctx.stream);
  launch_dep(prepare_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((warps + 7) / 8, 8 * ctx.num_sms))), 256, 0,
             ctx.stream, p);
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  return launched();
}

int launch_w4_product(const W4Product& a, LaunchCtx& ctx) {
  using namespace w4;
  const Cut c = cut_of(a.m, a.n, ctx.num_sms);
  ProductParams p{};
  p.m = a.m;
  p.packed = static_cast<const uint8_t*>(a.packed);
  p.chunks = static_cast<int>(a.m.chunks());
  p.total = a.m.units() * a.m.chunks();
  p.block_bytes = a.m.block_bytes();
  p.units = static_cast<int>(a.m.units());
  p.n = a.n;
  p.out_rs = a.out_rs;
  p.epi = a.epi;
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.image = static_cast<const uint8_t*>(a.image);
  p.image_out = static_cast<uint8_t*>(a.image_out);
  p.out_chunks = a.epi == W4_OUT ? 0 : static_cast<int>(a.m.T * a.m.sp / 128);
  p.parts = static_cast<float*>(a.scratch);
  p.counters = a.counters;
  p.err = ctx.err;
  p.skip_load = ctx.debug_skip_load;
  p.timeout_ns = ctx.timeout_ns;
  ctx.debug_skip_load = 0;
  const dim3 grid(static_cast<unsigned>(c.blocks), static_cast<unsigned>(c.tiles));
  if (ctx.before) ctx.before(ctx.user, a.name, ctx.stream);
  int rc;
  if (c.nt == 8)
    rc = launch_few<8>(p, grid, ctx.stream);
  else if (c.nt == 16)
    rc = launch_few<16>(p, grid, ctx.stream);
  else
    rc = launch_product<32>(p, grid, ctx.stream);
  if (rc) return rc;
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  return launched();
}

}  // namespace tpffn
