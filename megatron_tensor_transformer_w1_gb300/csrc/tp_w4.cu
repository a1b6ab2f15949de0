// tp_w4.cu -- 4-bit weights with group scales: quantising, the layout that the
// products read, and the products of few tokens with such weights.
//
// A group of `group` consecutive columns of a row has the scale s (bf16), its
// elements are (code - 8) s with codes 0..15.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
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
// Eight codes in column order <-> a packed word (even columns in the low half).
__device__ __forceinline__ uint32_t half_of(uint32_t w) {  // nibbles 0, 2, 4, 6
  w &= 0x0f0f0f0fu;
  w = (w | (w >> 4)) & 0x00ff00ffu;
  return (w | (w >> 8)) & 0xffffu;
}
__device__ __forceinline__ uint32_t spread(uint32_t h) {
  h = (h | (h << 8)) & 0x00ff00ffu;
  return (h | (h << 4)) & 0x0f0f0f0fu;
}
__device__ __forceinline__ uint32_t to_packed(uint32_t w) { return half_of(w) | (half_of(w >> 4) << 16); }
__device__ __forceinline__ uint32_t to_natural(uint32_t p) { return spread(p & 0xffffu) | (spread(p >> 16) << 4); }

// A block of the packed layout to a thread block.
__global__ void __launch_bounds__(256) pack_kernel(W4Shape m, W4Codes c, uint8_t* packed, int unpack) {
  const long long chunks = m.chunks(), seg_chunks = m.seg_chunks(), cols = m.cols(), row_bytes = (cols + 1) / 2;
  const long long blocks = m.units() * chunks, groups = m.segs * m.seg_groups();
  for (long long b = blockIdx.x; b < blocks; b += gridDim.x) {
    const long long unit = b / chunks, chunk = b - unit * chunks, e = chunk / seg_chunks, in = (chunk - e * seg_chunks) * 128;
    uint8_t* blk = packed + b * m.block_bytes();
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int piece = i & 3, r = (i >> 2) & 127, tile = i >> 9;
      const W4Tile t = w4_tile(m, unit * 2 + tile);
      const long long col0 = in + piece * 32;  // within the segment
      const bool row_ok = r < t.n;
      const int live = !row_ok || col0 >= m.seg ? 0 : (m.seg - col0 < 32 ? static_cast<int>(m.seg - col0) : 32);
      uint4* at = reinterpret_cast<uint4*>(blk + tile * 8192 + piece * 2048 + r * 16);
      uint8_t* src = static_cast<uint8_t*>(c.codes[t.mat]) + (t.row0 + r) * row_bytes;
      const long long from = e * m.seg + col0;
      uint32_t w[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
      if (!unpack) {
        for (int j = 0; j < live; ++j) {
          const uint32_t q = (src[(from + j) >> 1] >> (4 * ((from + j) & 1))) & 15u;
          w[j >> 3] = (w[j >> 3] & ~(15u << (4 * (j & 7)))) | (q << (4 * (j & 7)));
        }
        *at = make_uint4(to_packed(w[0]), to_packed(w[1]), to_packed(w[2]), to_packed(w[3]));
      }
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
        const uint32_t w = *reinterpret_cast<const uint32_t*>(from + chunk * m.block_bytes() + (k >> 5) * 2048 + r * 16 +
                                                              ((k >> 3) & 3) * 4);
        const uint32_t q = (w >> (16 * (k & 1) + 4 * ((k & 7) >> 1))) & 15u;
        byte = h ? (byte & 0x0fu) | (q << 4) : (byte & 0xf0u) | q;
      }
      static_cast<uint8_t*>(c.codes[t.mat])[(t.row0 + r) * row_bytes + c0 / 2] = static_cast<uint8_t>(byte);
    }
  }
}

// ================================================================ products
// The simplest form: a thread to a row of a unit, eight tokens at a time, the
// group's sum in 32 bits times its scale.
struct ProductParams {
  W4Shape m;
  const uint8_t* packed;
  const __nv_bfloat16* x;
  long long n, x_seg, x_rs, out_rs;
  int epi;
  const __nv_bfloat16* bias;
  __nv_bfloat16* out;
};
constexpr int TOK = 8;

__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ ProductParams p) {
  __shared__ float sx[128][TOK];
  __shared__ float sg[128][TOK];
  const W4Shape& m = p.m;
  const long long unit = blockIdx.x, n0 = static_cast<long long>(blockIdx.y) * TOK;
  const int tile = threadIdx.x >> 7, r = threadIdx.x & 127;
  const long long chunks = m.chunks(), seg_chunks = m.seg_chunks();
  float acc[TOK] = {};
  for (long long chunk = 0; chunk < chunks; ++chunk) {
    const long long e = chunk / seg_chunks, in = (chunk - e * seg_chunks) * 128;
    __syncthreads();
    for (int i = threadIdx.x; i < 128 * TOK; i += 256) {
      const int k = i & 127, j = i >> 7;
      const bool ok = n0 + j < p.n && in + k < m.seg;
      sx[k][j] = ok ? __bfloat162float(p.x[(n0 + j) * p.x_rs + e * p.x_seg + in + k]) : 0.f;
    }
    __syncthreads();
    const uint8_t* blk = p.packed + (unit * chunks + chunk) * m.block_bytes();
    for (int sub = 0; sub < 128 / m.group; ++sub) {
      float part[TOK] = {};
      for (int k = sub * m.group; k < (sub + 1) * m.group; k += 8) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + tile * 8192 + (k >> 5) * 2048 + r * 16 + ((k >> 3) & 3) * 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = static_cast<float>((w >> (16 * (i & 1) + 4 * (i >> 1))) & 15u) - 8.f;
#pragma unroll
          for (int j = 0; j < TOK; ++j) part[j] += q * sx[k + i][j];
        }
      }
      const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(blk + 16384)[sub * 256 + threadIdx.x]);
#pragma unroll
      for (int j = 0; j < TOK; ++j) acc[j] += s * part[j];
    }
  }
  long long row = unit * 256 + threadIdx.x;
  if (p.epi == W4_SWIGLU) {
    __syncthreads();
    if (tile == 1)
      for (int j = 0; j < TOK; ++j) sg[r][j] = acc[j];
    __syncthreads();
    if (tile == 1) return;
    row = unit * 128 + r;
    for (int j = 0; j < TOK; ++j) acc[j] = acc[j] * sigmoid_f(acc[j]) * sg[r][j];
  } else if (p.epi == W4_GELU) {
    const long long t = row / m.sp, in = row - t * m.sp;
    const float b = p.bias && in < m.s && t < m.T ? __bfloat162float(p.bias[t * m.s + in]) : 0.f;
    for (int j = 0; j < TOK; ++j) acc[j] = gelu_tanh_f(acc[j] + b);
  } else if (p.bias && row < m.rows) {
    const float b = __bfloat162float(p.bias[row]);
    for (int j = 0; j < TOK; ++j) acc[j] += b;
  }
  if (row >= (p.epi == W4_OUT ? m.rows : m.T * m.sp)) return;
  for (int j = 0; j < TOK && n0 + j < p.n; ++j) p.out[(n0 + j) * p.out_rs + row] = __float2bfloat16_rn(acc[j]);
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

int launch_w4_product(const W4Product& a, LaunchCtx& ctx) {
  using namespace w4;
  ProductParams p{};
  p.m = a.m;
  p.packed = static_cast<const uint8_t*>(a.packed);
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.n = a.n;
  p.x_seg = a.x_seg;
  p.x_rs = a.x_rs;
  p.out_rs = a.out_rs;
  p.epi = a.epi;
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  if (ctx.before) ctx.before(ctx.user, a.name, ctx.stream);
  product_kernel<<<dim3(static_cast<unsigned>(a.m.units()), static_cast<unsigned>((a.n + TOK - 1) / TOK)), 256, 0,
                   ctx.stream>>>(p);
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  return launched();
}

}  // namespace tpffn
