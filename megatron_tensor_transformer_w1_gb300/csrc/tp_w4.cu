// tp_w4.cu -- 4-bit weights with group scales: quantising, the layout that the
// products read, and the products with such weights.
//
// A group of `group` consecutive columns of a row has the scale s (bf16), its
// elements are (code - 8) s with codes 0..15.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 2^e, e brought into a range where 2^-e is a normal number too.
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(static_cast<uint32_t>(min(max(e, -126), 126) + 127) << 23);
}

// ================================================================ quantising
// s = bf16(max |w| / 7), code = rint(w / s) + 8, ties to even, limited to 0..15: only a scale
// that is a subnormal is more than 2^-9 off max |w| / 7, so that |w| > 7.03 s.
// A group with an infinity or NaN has that for its scale.  With s = 0 (all
// zero, or too small for bf16) every code is 8.
// The quotient by a product with 1 / 7 and its remainder, which is exact.
__device__ __forceinline__ float group_scale(float amax) {
  const float seventh = 1.f / 7.f, q = amax * seventh;
  return __bfloat162float(__float2bfloat16_rn(amax < INFINITY ? fmaf(fmaf(-7.f, q, amax), seventh, q) : amax));
}

// 1 / s overflows for the smallest scales: s and w are brought up by 2^64 first.
__device__ __forceinline__ void ready(float& s, float& inv, float& up) {
  up = s < 1e-30f ? 18446744073709551616.f : 1.f;
  s *= up;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));  // (to 2^-22; s is below 2^126)
}
// What `ready` asks for besides, which is where |w| may be above 7.03 s: w between -8 s and 7 s, for
// the same codes.
__device__ __forceinline__ float limited(float w, float s) { return fminf(fmaxf(w, -8.f * s), 7.f * s); }
// The codes of two elements, in the low bytes, for finite s > 0 and w in -8 s .. 7.03 s.  The
// quotient in two steps: q = w inv, then q + (w - q s) inv, whose remainder is exact and
// which is the quotient to 2^-43 before its last rounding: a tie, which 32 bits hold,
// comes out exactly, and others lie at least 2^-18 from one.  The sum with 1.5 2^23 + 8
// has a last bit worth 1: ties go to the even code.
__device__ __forceinline__ uint2 codes_of(uint64_t w, uint64_t less_s, uint64_t inv) {
  const uint64_t q = mul2(w, inv), magic = pack2(12582920.f, 12582920.f);
  const float2 u = unpack2(add2(fma2(fma2(q, less_s, w), inv, q), magic));
  return make_uint2(__float_as_uint(u.x), __float_as_uint(u.y));
}
__device__ __forceinline__ bool has_codes(float s) { return s > 0.f && s < INFINITY; }

// A thread's row and place in it, of `width` places each, over a grid's strides: the
// division of 64 bits once.
struct Walk {
  long long row, rows_on;
  unsigned place, places_on, width;
  __device__ __forceinline__ Walk(long long first, long long stride, unsigned w) : width(w) {
    row = first / w;
    place = static_cast<unsigned>(first - row * w);
    rows_on = stride / w;
    places_on = static_cast<unsigned>(stride - rows_on * w);
  }
  __device__ __forceinline__ void next() {
    row += rows_on;
    place += places_on;
    if (place >= width) {
      place -= width;
      ++row;
    }
  }
};
// 16 elements to a lane, 1 << lanes of them to a group.  Bound by memory and, nearly as
// much, by its instructions (76 % of the issue slots): 28672 x 8192 in 104 us, 5.8 TB/s.
__global__ void __launch_bounds__(256) quantize16_kernel(const uint4* __restrict__ W, long long pieces, int row_pieces,
                                                         int seg_pieces, int lanes, int seg_groups, int segs,
                                                         uint2* __restrict__ codes, __nv_bfloat16* __restrict__ scales) {
  // places: the pieces of a row, each segment's rounded up to whole groups
  const unsigned per = static_cast<unsigned>(seg_groups) << lanes;
  const long long rows = pieces / row_pieces, total = rows * (static_cast<long long>(segs) * per);
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x, first = static_cast<long long>(blockIdx.x) * blockDim.x;
  Walk at_row(first + threadIdx.x, stride, segs * per);
  for (long long i0 = first; i0 < total; i0 += stride, at_row.next()) {
    const long long row = at_row.row;
    const int seg = segs == 1 ? 0 : static_cast<int>(at_row.place / per), in = static_cast<int>(at_row.place - seg * per);
    const bool ok = row < rows && in < seg_pieces;
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
    for (int d = 1; d < 1 << lanes; d <<= 1) m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    const __nv_bfloat16 top = __hmax_nan(m.x, m.y);
    float s = group_scale(__bfloat162float(top)), inv, up;
    if (ok && (in & ((1 << lanes) - 1)) == 0) scales[(row * segs + seg) * seg_groups + (in >> lanes)] = __float2bfloat16_rn(s);
    const bool any = has_codes(s);
    ready(s, inv, up);
    if (up != 1.f) {
      const uint32_t most = tc::pack_bf16x2(7.f * s, 7.f * s), least = tc::pack_bf16x2(-8.f * s, -8.f * s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // limited(w 2^64, s)
        asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v[j]) : "r"(0x5f805f80u));
        asm("min.bf16x2 %0, %0, %1;" : "+r"(v[j]) : "r"(most));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(v[j]) : "r"(least));
      }
    }
    const uint64_t less2 = pack2(-s, -s), inv2 = pack2(inv, inv);
    uint32_t word[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = codes_of(pack2(bf16_at(v[4 * h + j], 0), bf16_at(v[4 * h + j], 1)), less2, inv2);
      const uint32_t even = __byte_perm(__byte_perm(c[0].x, c[1].x, 0x0040), __byte_perm(c[2].x, c[3].x, 0x0040), 0x5410),
                     odd = __byte_perm(__byte_perm(c[0].y, c[1].y, 0x0040), __byte_perm(c[2].y, c[3].y, 0x0040), 0x5410);
      word[h] = any ? even + 16 * odd : 0x88888888u;
    }
    if (ok) codes[at] = make_uint2(word[0], word[1]);
  }
}

// The groups of eight columns from c on, of segments of at least eight: up to `first` the
// scale at `at`, up to `second` the next (a segment's last group may be of one column),
// then the one behind it.
struct Groups {
  int at, first, second;
  __device__ __forceinline__ Groups(int c, int segs, int seg, int group, int seg_groups) {
    const int e = segs == 1 ? 0 : c / seg, in = c - e * seg, g = group == 32 ? in >> 5 : group == 64 ? in >> 6 : in >> 7;
    const int end = min((g + 1) * group, seg);
    at = e * seg_groups + g;
    first = end - in;
    second = first + (end == seg ? 8 : min(group, seg - end));
  }
  template <typename V>
  __device__ __forceinline__ V of(int j, V a, V b, V c) const {
    return j < first ? a : j < second ? b : c;
  }
};
// Eight columns from any even address on, in the largest pieces that it allows.  Columns
// behind `live` are zeros, or are not written.
__device__ __forceinline__ void load8(uint32_t (&v)[4], const __nv_bfloat16* src, int live) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
  const int low = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
  if (live < 8) {
    v[0] = v[1] = v[2] = v[3] = 0;
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < live) v[j >> 1] |= static_cast<uint32_t>(h[j]) << (16 * (j & 1));
  } else if (low == 0) {
    const uint4 a = *reinterpret_cast<const uint4*>(src);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else if ((low & 3) == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = reinterpret_cast<const uint32_t*>(src)[j];
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(h + 1);
    const uint32_t a = h[0], b = w[0], c = w[1], d = w[2], e = h[7];
    v[0] = a | b << 16, v[1] = b >> 16 | c << 16, v[2] = c >> 16 | d << 16, v[3] = d >> 16 | e << 16;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* to, const uint32_t (&v)[4], int live) {
  uint16_t* h = reinterpret_cast<uint16_t*>(to);
  const int low = static_cast<int>(reinterpret_cast<uintptr_t>(to) & 15);
  if (live < 8) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < live) h[j] = static_cast<uint16_t>(v[j >> 1] >> (16 * (j & 1)));
  } else if (low == 0) {
    *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
  } else if ((low & 3) == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(to)[j] = v[j];
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(h + 1);
    h[0] = static_cast<uint16_t>(v[0]);
    w[0] = v[0] >> 16 | v[1] << 16, w[1] = v[1] >> 16 | v[2] << 16, w[2] = v[2] >> 16 | v[3] << 16;
    h[7] = static_cast<uint16_t>(v[3] >> 16);
  }
}
// Four bytes from any address on, of which `live` are there.
__device__ __forceinline__ uint32_t load4(const uint8_t* src, int live) {
  const int low = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 3);
  uint32_t w = 0;
  if (live < 4) {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < live) w |= static_cast<uint32_t>(src[j]) << (8 * j);
  } else if (low == 0) {
    w = *reinterpret_cast<const uint32_t*>(src);
  } else if (low == 2) {
    w = reinterpret_cast<const uint16_t*>(src)[0] | static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(src)[1]) << 16;
  } else {
    w = src[0] | static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(src + 1)) << 8 | static_cast<uint32_t>(src[3]) << 24;
  }
  return w;
}
__device__ __forceinline__ void store4(uint8_t* to, uint32_t w, int live) {
  const int low = static_cast<int>(reinterpret_cast<uintptr_t>(to) & 3);
  if (live < 4) {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < live) to[j] = static_cast<uint8_t>(w >> (8 * j));
  } else if (low == 0) {
    *reinterpret_cast<uint32_t*>(to) = w;
  } else if (low == 2) {
    reinterpret_cast<uint16_t*>(to)[0] = static_cast<uint16_t>(w);
    reinterpret_cast<uint16_t*>(to)[1] = static_cast<uint16_t>(w >> 16);
  } else {
    to[0] = static_cast<uint8_t>(w);
    *reinterpret_cast<uint16_t*>(to + 1) = static_cast<uint16_t>(w >> 8);
    to[3] = static_cast<uint8_t>(w >> 24);
  }
}
// Widths that 16-element pieces do not fit: the scales, a thread to eight columns of a
// group, then the codes, a thread to eight columns of a row (or, with segments of less
// than eight, to a byte, whose two columns may belong to two segments).  Pieces of 16
// are the faster way (28672 x 8192: 104 us), but rows that begin at any even address and
// groups that begin in any column do not have them.  Bound by instructions, 270 to
// eight columns: 28672 x 8190 in 416 us (the scales 129 of it), back in 174.
// 8 << lanes columns to a group.
__global__ void __launch_bounds__(256) scales_kernel(const __nv_bfloat16* __restrict__ W, long long rows, long long cols,
                                                     int segs, int seg, int lanes, int seg_groups,
                                                     __nv_bfloat16* __restrict__ scales) {
  const int per = 256 >> lanes, lane = threadIdx.x & ((1 << lanes) - 1), group = 8 << lanes;
  const long long stride = static_cast<long long>(gridDim.x) * per, first = static_cast<long long>(blockIdx.x) * per;
  Walk at(first + (threadIdx.x >> lanes), stride, static_cast<unsigned>(segs) * seg_groups);
  for (long long g0 = first; g0 < rows * (static_cast<long long>(segs) * seg_groups); g0 += stride, at.next()) {
    const int e = segs == 1 ? 0 : static_cast<int>(at.place) / seg_groups, g = static_cast<int>(at.place) - e * seg_groups;
    const int in = g * group + lane * 8, live = at.row < rows ? min(seg - in, 8) : 0;
    uint32_t v[4] = {};
    if (live > 0) load8(v, W + at.row * cols + static_cast<long long>(e) * seg + in, live);
    __nv_bfloat162 m = __habs2(*reinterpret_cast<__nv_bfloat162*>(&v[0]));
#pragma unroll
    for (int j = 1; j < 4; ++j) m = __hmax2_nan(m, __habs2(*reinterpret_cast<__nv_bfloat162*>(&v[j])));
    for (int d = 1; d < 1 << lanes; d <<= 1) m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0 && live > 0)
      scales[at.row * at.width + at.place] = __float2bfloat16_rn(group_scale(__bfloat162float(__hmax_nan(m.x, m.y))));
  }
}
__global__ void __launch_bounds__(256) codes8_kernel(const __nv_bfloat16* __restrict__ W, long long rows, int cols, int segs,
                                                     int seg, int group, int seg_groups,
                                                     const __nv_bfloat16* __restrict__ scales, uint8_t* __restrict__ codes) {
  const long long row_bytes = (cols + 1) / 2, stride = gridDim.x * 256ll;
  for (Walk at(blockIdx.x * 256ll + threadIdx.x, stride, (cols + 7) / 8); at.row < rows; at.next()) {
    const int c = static_cast<int>(at.place) * 8, live = min(cols - c, 8);
    const Groups of(c, segs, seg, group, seg_groups);
    const __nv_bfloat16* sc = scales + at.row * (static_cast<long long>(segs) * seg_groups) + of.at;
    uint32_t v[4];
    load8(v, W + at.row * cols + c, live);
    float sg[3], inv[3], up[3];
    uint32_t any[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      sg[k] = k == 0 || (k == 1 ? of.first : of.second) < live ? __bfloat162float(sc[k]) : sg[0];
      any[k] = has_codes(sg[k]) ? 15u : 0u;
      ready(sg[k], inv[k], up[k]);
    }
    auto pick = [&](int i, auto& a) { return of.of(i, a[0], a[1], a[2]); };
    if (up[0] != 1.f || up[1] != 1.f || up[2] != 1.f) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = tc::pack_bf16x2(limited(bf16_at(v[j], 0) * pick(2 * j, up), pick(2 * j, sg)),
                               limited(bf16_at(v[j], 1) * pick(2 * j + 1, up), pick(2 * j + 1, sg)));
    }
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int a = 2 * j, b = a + 1;
      const uint2 q = codes_of(pack2(bf16_at(v[j], 0), bf16_at(v[j], 1)), pack2(-pick(a, sg), -pick(b, sg)), pack2(pick(a, inv), pick(b, inv)));
      word |= (q.x & 15u) << (8 * j) | (q.y & 15u) << (8 * j + 4);
    }
    if (!(any[0] & any[1] & any[2]) || live < 8) {  // codes of 8 in the place of some
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!pick(j, any) || j >= live) word = (word & ~(15u << (4 * j))) | 8u << (4 * j);
    }
    store4(codes + at.row * row_bytes + c / 2, word, (live + 1) / 2);
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
      const bool any = has_codes(s);
      ready(s, inv, up);
      const float w = limited(__bfloat162float(W[row * cols + c]) * up, s);
      const uint32_t q = any ? codes_of(pack2(w, w), pack2(-s, -s), pack2(inv, inv)).x & 15u : 8u;
      byte = h ? (byte & 0x0fu) | (q << 4) : (byte & 0xf0u) | q;
    }
    codes[i] = static_cast<uint8_t>(byte);
  }
}

__device__ __forceinline__ float value_of(uint32_t word, int j, float s) {
  return (static_cast<float>((word >> (4 * j)) & 15u) - 8.f) * s;
}
// (code - 8) s as bf16, for the codes at bits 0-3 and 16-19: 128 + code less 136 is exact,
// and the product is rounded once.
__device__ __forceinline__ uint32_t two_values(uint32_t c, uint32_t s) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(c), "r"(0x000f000fu), "r"(0x43004300u));
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0x43084308u));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(s));
  return v;
}
// Bound by memory: 28672 x 8192 in 104 us, 5.7 TB/s, two pieces to a thread on their way
// (one: 123 us).
__global__ void __launch_bounds__(256) dequantize16_kernel(const uint2* __restrict__ codes,
                                                           const __nv_bfloat16* __restrict__ scales, long long pieces,
                                                           int row_pieces, int seg_pieces, int lanes, int seg_groups,
                                                           int segs, uint4* __restrict__ W) {
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  Walk at_row(i, stride, row_pieces);
  auto scale_of = [&] {
    const int e = segs == 1 ? 0 : static_cast<int>(at_row.place) / seg_pieces, in = static_cast<int>(at_row.place) - e * seg_pieces;
    return reinterpret_cast<const uint16_t*>(scales)[(at_row.row * segs + e) * seg_groups + (in >> lanes)];
  };
  auto write = [&](uint4* to, uint2 q, uint32_t s) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      // four codes: the second of either pair 12 bits up, in the upper half
      const uint32_t four = (j < 4 ? q.x : q.y) >> (16 * ((j >> 1) & 1)) & 0xffffu, c = four | four << 12;
      w[j] = two_values(c, s);
      w[j + 1] = two_values(c >> 8, s);
    }
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  };
  for (; i < pieces; i += 2 * stride) {  // two at a time, both loads on their way
    const bool more = i + stride < pieces;
    const uint2 q0 = codes[i], q1 = more ? codes[i + stride] : q0;
    const uint32_t s0 = scale_of();
    at_row.next();
    const uint32_t s1 = more ? scale_of() : s0;
    at_row.next();
    write(W + 2 * i, q0, s0 * 0x10001u);
    if (more) write(W + 2 * (i + stride), q1, s1 * 0x10001u);
  }
}
__global__ void __launch_bounds__(256) dequantize8_kernel(const uint8_t* __restrict__ codes,
                                                          const __nv_bfloat16* __restrict__ scales, long long rows, int cols,
                                                          int segs, int seg, int group, int seg_groups,
                                                          __nv_bfloat16* __restrict__ W) {
  const long long row_bytes = (cols + 1) / 2, stride = gridDim.x * 256ll;
  for (Walk at(blockIdx.x * 256ll + threadIdx.x, stride, (cols + 7) / 8); at.row < rows; at.next()) {
    const int c = static_cast<int>(at.place) * 8, live = min(cols - c, 8);
    const Groups of(c, segs, seg, group, seg_groups);
    const uint16_t* sc = reinterpret_cast<const uint16_t*>(scales) + at.row * (static_cast<long long>(segs) * seg_groups) + of.at;
    const uint32_t word = load4(codes + at.row * row_bytes + c / 2, (live + 1) / 2);
    const uint32_t s0 = sc[0], s1 = of.first < live ? sc[1] : s0, s2 = of.second < live ? sc[2] : s0;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t byte = word >> (8 * j) & 0xffu;
      w[j] = two_values(byte | byte << 12, of.of(2 * j, s0, s1, s2) | of.of(2 * j + 1, s0, s1, s2) << 16);
    }
    store8(W + at.row * cols + c, w, live);
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

// The factors of the rows (see W4Shape::row_up): a block to a unit, a thread to a row.
__global__ void __launch_bounds__(256) row_up_kernel(W4Shape m, uint8_t* packed) {
  const long long chunks = m.chunks(), unit = blockIdx.x;
  const int r = threadIdx.x, subs = 128 / m.group;
  uint32_t top = 0;  // the largest |scale|, as bits: infinities and NaN are largest
  for (long long c = 0; c < chunks; ++c) {
    const auto* at = reinterpret_cast<const uint16_t*>(packed + (unit * chunks + c) * m.block_bytes() + 16384) + r;
    for (int i = 0; i < subs; ++i) top = max(top, at[i * 256] & 0x7fffu);
  }
  const int e = min(static_cast<int>(top >> 7), 254) - 127;  // top < 2^(e + 1)
  m.row_up(packed)[unit * 256 + r] = pow2(top ? 11 - e : 0);
}

// ================================================================ products
// y[token][row] = sum_g s[row][g] sum_{k in g} (code - 8) x[token][k].
//
// A block takes a run of chunks (128 columns of a unit's 256 rows) of the list of
// all units' chunks, the same number as the others, whatever units they belong to;
// a run of chunks of one unit is a segment.  A unit that several blocks share is
// joined by the last of them to come, in the order of the columns.
//
// Two kernels: few tokens (up to 8) on registers, more on tensor memory.  Both sum in 32
// bits.  Tokens are fp16 numbers times a power of two, which holds bf16's eight bits.
// Hidden activations are rounded to it, to 11 bits: beside y's own rounding to bf16, 2^-9, that
// is 2^-12 (0.00167 -> 0.00168 in root mean square against 64 bits for the 70B
// feed-forward).  In two fp16 numbers each they would have 22, and the second
// product twice the matrix instructions, whose time a prompt's is.  The scaled weights
// of the second kernel are rounded where a scale is below 2^-12 of its row's largest.
using namespace tc;

// A block of tokens as the kernels keep it ("image"), for NT tokens: fp16 [2][NT][64],
// 64 columns each, in rows of 128 bytes whose 16-byte pieces are swizzled by the token
// (piece i at i ^ (token & 7)).
//  * Few tokens: every token's 128 columns have their own power of two, and behind
//    them lies float [NT], the powers that undo it.  A block's largest element comes to
//    2^14..2^15, so that bf16's eight bits are kept down to 2^-31 of it and what is
//    smaller is rounded to 2^-39 of it.
//  * More: the power of two is the token's, for all columns.  Behind the images of
//    all tokens lies int [tokens][APART], in the first the exponent e: |x| < 2^e, kept as
//    x 2^(15 - e) (every block's maximum for a token goes there: thousands that
//    met in a line took 4 us for 32 tokens of the 70B feed-forward).  For hidden
//    activations int [chunks][tokens] behind that, those of each block of columns, with
//    which they are written before the token's is known (see fit_kernel).
constexpr int FEW = 8;  // tokens
__host__ __device__ constexpr int image_bytes(int nt) { return nt * 256 + (nt <= FEW ? 128 : 0); }  // (copied to multiples of 128)
constexpr int APART = 32;
constexpr int LEAST = -111;  // an exponent: 2^(15 - e) is a number
__device__ __forceinline__ int exponent(uint32_t bits) {  // |v| < 2^it, from v's bits (infinities, NaN: the largest)
  return max(static_cast<int>(bits >> 23 & 255u) - 126, LEAST);
}

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
  int nt, stages, stage_bytes, bufs;  // more than a few tokens
  const float* row_up;
  const int* e_in;          // the tokens' exponents, by token
  int *e_out, *e_chunk;     // those of the hidden activations, of all columns and by chunk and token
  int padded;               // tokens of all tiles
  int blocks;               // runs of chunks
  // few tokens: [blocks][2][NT][256], else [token tiles][blocks + units - 1][NT][256]
  float* parts;
  int* counters;  // few tokens: [units]
  int* err;
  int skip_load;
  unsigned long long timeout_ns;
};

// Columns 4 lane .. 4 lane + 3 of a token's block, by a warp, into an image of few tokens.
__device__ __forceinline__ void store_block(uint8_t* image, int nt, int token, int lane, const float (&v)[4]) {
  const float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));  // without NaN
  const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu);
  const int e = min(141 - static_cast<int>(min(most >> 23, 254u)), 126);  // most * 2^e in 2^14..2^15
  const float up = pow2(e), down = pow2(-e);
  const __half2 lo = __floats2half2_rn(v[0] * up, v[1] * up), hi = __floats2half2_rn(v[2] * up, v[3] * up);
  uint8_t* at = image + (lane >> 4) * (nt * 128) + token * 128 + ((((lane & 15) >> 1) ^ (token & 7)) << 4) + (lane & 1) * 8;
  *reinterpret_cast<uint2*>(at) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (lane == 0) reinterpret_cast<float*>(image + nt * 256)[token] = down;
}

struct PrepareParams {
  const __nv_bfloat16* x;
  long long x_seg, x_rs, seg, seg_chunks, chunks, n;
  int nt, tiles;
  uint8_t* image;  // [tiles][chunks]
  int *err, *counters, n_counters;
  int *e_in, *e_out;  // more than a few tokens: exponents; those of hidden activations to come are cleared
};
// The kernel before a call's first product: the tokens' blocks, a warp to a token's;
// clears what the call counts in.  It lets others start when everything before it
// on the stream is done: the products behind it read their weights without a further wait.
__device__ __forceinline__ void prepare_call(const PrepareParams& p) {
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.err) *p.err = 0;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.n_counters; i += gridDim.x * blockDim.x) p.counters[i] = 0;
}
__global__ void __launch_bounds__(256) prepare_few_kernel(const __grid_constant__ PrepareParams p) {
  prepare_call(p);
  const int lane = threadIdx.x & 31;
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
    store_block(p.image + block * image_bytes(p.nt), p.nt, in, lane, v);
  }
}
// More tokens: a block to a token (some 4 us, most of it its start), whose largest element it needs before the first
// is written.
constexpr int PREPARE_THREADS = 512;
__global__ void __launch_bounds__(PREPARE_THREADS) prepare_kernel(const __grid_constant__ PrepareParams p) {
  prepare_call(p);
  __shared__ uint32_t s_most[PREPARE_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pieces = static_cast<int>(p.chunks) * 16;
  const int padded = p.tiles * p.nt;
  for (int token = blockIdx.x; token < padded; token += gridDim.x) {
    const int tile = token / p.nt, in = token - tile * p.nt;
    auto piece = [&](int i) {  // eight columns
      const int chunk = i >> 4, e = chunk / static_cast<int>(p.seg_chunks);
      const long long col = (chunk - e * p.seg_chunks) * 128 + (i & 15) * 8;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (token < p.n && col < p.seg) w = *reinterpret_cast<const uint4*>(p.x + token * p.x_rs + e * p.x_seg + col);
      return w;
    };
    uint32_t most = 0;
    for (int i = threadIdx.x; i < pieces; i += PREPARE_THREADS) {
      const uint4 w = piece(i);
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) most = max(most, max(v[j] & 0x7fff0000u, (v[j] << 16) & 0x7fff0000u));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s_most[warp] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, s_most[lane & (PREPARE_THREADS / 32 - 1)]);
    __syncthreads();
    const int e_x = exponent(most);
    const float up = pow2(15 - e_x);
    uint8_t* image = p.image + static_cast<long long>(tile) * p.chunks * image_bytes(p.nt) + in * 128;
    for (int i = threadIdx.x; i < pieces; i += PREPARE_THREADS) {
      const uint4 w = piece(i);
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(bf16_at(v[j], 0) * up, bf16_at(v[j], 1) * up);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(image + static_cast<long long>(i >> 4) * image_bytes(p.nt) + ((i >> 3) & 1) * (p.nt * 128) +
                                (((i & 7) ^ (in & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (threadIdx.x == 0) {
      p.e_in[token * APART] = e_x;
      if (p.e_out) p.e_out[token * APART] = LEAST;
    }
  }
}

// Bounded wait on an mbarrier phase, as tc::Waiter's, for waits that mostly last
// some hundred cycles: the clock, which takes longer than that to read, is looked
// at only after many tries.
struct Wait {
  volatile int* abort_flag;
  int* err;
  unsigned long long timeout_ns;
  __device__ __noinline__ bool slow(uint64_t* bar, uint32_t parity, bool honour_abort, bool sleep) const {
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
      if (mbar_try_wait(bar, parity)) return true;
      if (sleep) __nanosleep(256);
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
    return mbar_try_wait(bar, parity) || slow(bar, parity, true, false);
  }
  __device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) const {
    if (!mbar_try_wait(bar, parity)) slow(bar, parity, false, false);
  }
  // of a whole warp
  __device__ __forceinline__ void warp(uint64_t* bar, uint32_t parity) const {
    if (!mbar_try_wait(bar, parity)) slow(bar, parity, true, false);
    __syncwarp();
  }
  // and for what lasts some microseconds: the tries would take the others' issue slots
  __device__ __forceinline__ void warp_long(uint64_t* bar, uint32_t parity) const {
    if (!mbar_try_wait(bar, parity)) slow(bar, parity, true, true);
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
// (code - 8) 2^-14 for the codes at bits 0-3 and 16-19, which are code * 2^-24 as fp16 subnormals,
// and for those at bits 4-7 and 20-23, code * 2^-20: times 2^10 or 2^6, less 2^-11.  Exact
// and no subnormals (but 0); with larger ones, sums times a token's largest power overflow.
__device__ __forceinline__ uint32_t low(uint32_t w) {
  uint32_t v = w & 0x000f000fu;
  asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(v) : "r"(0x64006400u), "r"(0x90009000u));
  return v;
}
__device__ __forceinline__ uint32_t high(uint32_t w) {
  uint32_t v = w & 0x00f000f0u;
  asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(v) : "r"(0x54005400u), "r"(0x90009000u));
  return v;
}
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
struct Ring {
  int stages, x_bytes, stage_bytes;
};
__device__ __forceinline__ void copy_chunks(const ProductParams& p, const Run& run, const Ring& r, uint8_t* ring,
                                            uint64_t* full, uint64_t* empty, const Wait& W) {
  // A single token tile reads the weights once.
  const uint64_t often = l2_policy_evict_normal(), once = gridDim.y == 1 ? l2_policy_evict_first() : often;
  const uint8_t* src = p.packed + run.first * p.block_bytes;
  const uint8_t* image = p.image + static_cast<long long>(blockIdx.y) * p.chunks * r.x_bytes;
  int c = static_cast<int>(run.first % p.chunks);
  auto weights = [&](int stage) {
    mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(p.block_bytes + r.x_bytes));
    bulk_load(ring + stage * r.stage_bytes + r.x_bytes, src, static_cast<uint32_t>(p.block_bytes), &full[stage], once);
    src += p.block_bytes;
  };
  auto tokens = [&](int stage) {
    bulk_load(ring + stage * r.stage_bytes, image + static_cast<long long>(c) * r.x_bytes, r.x_bytes, &full[stage], often);
    if (++c == p.chunks) c = 0;
  };
  // The weights are not the previous kernel's to write (what wrote them is done
  // before the call's first kernel lets others start); the tokens are.
  const int ahead = run.count < r.stages ? run.count : r.stages;
  for (int i = 0; i < ahead; ++i) weights(i);
  grid_dep_wait();
  for (int i = p.skip_load ? 1 : 0; i < ahead; ++i) tokens(i);
  int issued = ahead, stage = 0;
  uint32_t phase = 0;
  for (int i = ahead; i < run.count; ++i, ++issued) {
    if (!W(&empty[stage], phase)) break;
    weights(stage);
    tokens(stage);
    if (++stage == r.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // every issued copy lands before the block may exit
  for (int i = issued > r.stages ? issued - r.stages : 0; i < issued; ++i) W.drain(&full[i % r.stages], (i / r.stages) & 1);
}

// Four neighbouring rows of a token, by a warp that has 128: bias or activation, and
// out.  FEW_TOKENS: into an image of few tokens.
template <bool FEW_TOKENS>
__device__ __forceinline__ void write4(const ProductParams& p, int nt, int tile, int in_tile, long long row, int lane, float4 v) {
  float a[4] = {v.x, v.y, v.z, v.w};
  if (p.epi == W4_OUT) {
    const long long token = static_cast<long long>(tile) * nt + in_tile;
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
  uint8_t* image = p.image_out + (static_cast<long long>(tile) * p.out_chunks + chunk) * image_bytes(nt);
  if (FEW_TOKENS) {
    store_block(image, nt, in_tile, lane, a);
  } else {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = max(most, __float_as_uint(a[i]) & 0x7fffffffu);
    const int e = exponent(__reduce_max_sync(0xffffffffu, most));
    const float up = pow2(15 - e);
    if (lane == 0) {
      const int token = tile * nt + in_tile;
      p.e_chunk[static_cast<long long>(chunk) * p.padded + token] = e;
      atomicMax(p.e_out + token * APART, e);
    }
    const __half2 lo = __floats2half2_rn(a[0] * up, a[1] * up), hi = __floats2half2_rn(a[2] * up, a[3] * up);
    uint8_t* at = image + (lane >> 4) * (nt * 128) + in_tile * 128 + ((((lane & 15) >> 1) ^ (in_tile & 7)) << 4) + (lane & 1) * 8;
    *reinterpret_cast<uint2*>(at) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// The end of a segment of `unit`, whose sums lie in shared memory, [token][row], 256
// rows and a few of padding: out if the segment is the whole unit, else as a part,
// and the last block of the unit joins the parts.  By the block's first
// FEW_WARPS warps, which then may write the sums anew.
constexpr int SUM_PITCH = 256 + 8, FEW_WARPS = 8;
__device__ __forceinline__ void finish_segment(const ProductParams& p, long long unit, const float* sum, int* s_last,
                                               const Wait& W) {
  // a thread: rows 4 q .. 4 q + 3 of tile 0 and of tile 1, of a warp's token
  static_assert(FEW == FEW_WARPS, "a token to a warp");
  const int token = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = lane * 4;
  const long long u0 = unit * p.chunks, u1 = u0 + p.chunks - 1;
  const int C = gridDim.x;
  const int c0 = static_cast<int>(((u0 + 1) * C - 1) / p.total), c1 = static_cast<int>(((u1 + 1) * C - 1) / p.total);
  float4 v0 = *reinterpret_cast<const float4*>(sum + token * SUM_PITCH + q4), v1 = *reinterpret_cast<const float4*>(sum + token * SUM_PITCH + 128 + q4);
  bool store = true;
  if (c0 != c1) {
    float* parts = p.parts + token * 256 + q4;
    auto slot = [&](int b) { return static_cast<long long>(2 * b + (b == c0)) * (FEW * 256); };
    float* to = parts + slot(blockIdx.x);
    __stcg(reinterpret_cast<float4*>(to), v0);
    __stcg(reinterpret_cast<float4*>(to + 128), v1);
    __threadfence();
    bar_sync(1, FEW_WARPS * 32);
    if (threadIdx.x == 0) {
      __threadfence();
      *s_last = atomicAdd(p.counters + unit, 1) == c1 - c0;
      __threadfence();
    }
    bar_sync(1, FEW_WARPS * 32);
    store = *s_last;
    if (store) {
      v0 = v1 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int b = c0; b <= c1; ++b) {
        const float* from = parts + slot(b);
        v0 = add4(v0, __ldcg(reinterpret_cast<const float4*>(from)));
        v1 = add4(v1, __ldcg(reinterpret_cast<const float4*>(from + 128)));
      }
    }
  }
  if (store && *W.abort_flag == 0) {
    const float one = 16384.f;  // 2^14: a code's unit
    v0 = make_float4(v0.x * one, v0.y * one, v0.z * one, v0.w * one);
    v1 = make_float4(v1.x * one, v1.y * one, v1.z * one, v1.w * one);
    if (p.epi == W4_SWIGLU) {  // tile 1 has the second matrix's rows of the same hidden slots
      v0.x *= sigmoid_f(v0.x) * v1.x;
      v0.y *= sigmoid_f(v0.y) * v1.y;
      v0.z *= sigmoid_f(v0.z) * v1.z;
      v0.w *= sigmoid_f(v0.w) * v1.w;
      write4<true>(p, FEW, 0, token, unit * 128 + q4, lane, v0);
    } else {
      write4<true>(p, FEW, 0, token, unit * 256 + q4, lane, v0);
      write4<true>(p, FEW, 0, token, unit * 256 + 128 + q4, lane, v1);
    }
  }
  bar_sync(1, FEW_WARPS * 32);
}

// ---------------------------------------------------------------- few tokens
// Up to 8 tokens, bound by the one read of the codes: m16n8k16 matrix instructions on
// registers.  What is left to count are the instructions that make operands of
// codes.  A code in the low bits of an fp16 number is a subnormal, code * 2^-24, and four
// bits higher code * 2^-20: a word's eight codes are four operand registers after one
// shift, four masks and four multiply-adds, which take the offset of 8 off.  (Codes made
// into bf16 take 11 instructions a word: 102 us for one token of the 70B feed-forward, for 72.
// The codes as they lie and the offset taken off as -8 times the columns' sum: 68 us, but
// an infinity less an infinity, and sums short by some 2^-17 of 8 times the block's
// largest element, as the unit aligns products by exponents that a subnormal does not
// fill: an element 2^12 above the others left them an error of 2^-9.  The codes
// shifted to the top of the mantissa, with that sum: 73 to 76 us and still short.)
// Sums are products times the block's power of two and the row's scale, in 32 bits.
//
// The matrix instructions take 2.05 cycles an SM (measured), those of a chunk 262 of
// the some 720 that its bytes take; the tensor-memory products take 768 whatever the
// number of tokens.  One token of the 70B feed-forward (363 MB)
// takes 72 us, 5.0 TB/s; what is beyond the copy rate is the start and the end of its two
// products and the kernel before them.  (Two instructions for 9 to 16 tokens: 88.5 us for the 70B feed-forward
// as the other kernel, but 26 us against 19 for a block of d 768 and 16 against 14 for
// an output projection of d 4096.)
//
// The order of a product's columns is free as long as both operands have it: lane
// t of a row's four takes the 32-bit words of codes 8 t .. 8 t + 7 of 32 columns, their
// pairs as the halves of two k16 steps, and so reads the same 8 columns of a token
// in one piece.  Token t stands in column 2 t, token t + 4 in column 2 t +
// 1 of the product, so that the two tokens of an eighth of a warp lie in different
// halves of the swizzled rows.
// 8 warps, 32 rows of the unit each, two blocks per SM.
struct Few {
  static constexpr int X_BYTES = image_bytes(FEW), STAGE = X_BYTES + 18432, STAGES = 5;
  static constexpr int M_SUM = STAGES * STAGE, SMEM = M_SUM + FEW * SUM_PITCH * 4 + 128;
  static_assert(2 * (SMEM + 2048) <= 233472, "two blocks per SM");
};
constexpr int FEW_THREADS = (FEW_WARPS + 1) * 32;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// SUBS: groups of a chunk.
template <int SUBS>
__global__ void __launch_bounds__(FEW_THREADS, 2) few_kernel(const __grid_constant__ ProductParams p) {
  using F = Few;
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
    if (lane == 0) copy_chunks(p, run, Ring{F::STAGES, F::X_BYTES, F::STAGE}, smem, full, empty, W);
    return;
  }
  const int t = lane & 3, i8 = lane >> 2;
  const int row0 = warp * 32 + i8;  // of the unit; the warp's rows: + 0, 8, 16, 24
  const int tok0 = (i8 & 1) * 4 + (i8 >> 1);
  // bytes from a stage's start
  const uint32_t at_x = tok0 * 128, swz = tok0 & 7;
  const uint32_t at_w = F::X_BYTES + row0 * 64 + ((t ^ ((i8 >> 1) & 3)) << 4), at_s = F::X_BYTES + 16384 + row0 * 2;
  const uint32_t at_down = FEW * 256 + t * 4;  // of token t
  float* sum = reinterpret_cast<float*>(smem + F::M_SUM);
  uint64_t acc[2][2] = {};  // rows row0 + 16 m + 8 h, tokens t and t + 4
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
    const uint64_t down = pack2(ld_shared_f(st + at_down), ld_shared_f(st + at_down + 16));  // of tokens t and t + 4
    float c[2][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      constexpr int PER = 4 / SUBS;
      if (q % PER == 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m) c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
      }
      const uint4 x = ld_shared_v4(st + at_x + (q >> 1) * (FEW * 128) + ((((q & 1) * 4 + t) ^ swz) << 4));
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t w0 = q == 0 ? w[m][0].x : q == 1 ? w[m][0].y : q == 2 ? w[m][0].z : w[m][0].w;
        const uint32_t w1 = q == 0 ? w[m][1].x : q == 1 ? w[m][1].y : q == 2 ? w[m][1].z : w[m][1].w;
        mma(c[m], low(w0), low(w1), high(w0), high(w1), x.x, x.y);
        mma(c[m], low(w0 >> 8), low(w1 >> 8), high(w0 >> 8), high(w1 >> 8), x.z, x.w);
      }
      if (q % PER != PER - 1) continue;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float s = ld_shared_scale(st + at_s + (q / PER) * 512 + (16 * m + 8 * h) * 2);
          acc[m][h] = fma2(pack2(s, s), mul2(pack2(c[m][2 * h], c[m][2 * h + 1]), down), acc[m][h]);
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
      for (int h = 0; h < 2; ++h) {
        const float2 v = unpack2(acc[m][h]);
        sum[t * SUM_PITCH + row0 + 16 * m + 8 * h] = v.x;
        sum[(t + 4) * SUM_PITCH + row0 + 16 * m + 8 * h] = v.y;
        acc[m][h] = 0;
      }
    bar_sync(1, FEW_WARPS * 32);
    finish_segment(p, unit, sum, &s_last, W);
    chunk = 0;
    ++unit;
  }
}

// ---------------------------------------------------------------- more tokens
// Up to 128 tokens to a block, several token tiles side by side (the weights come
// from L2 for all but the first).  The weights are the A operand of tcgen05.mma, 128
// rows at a time, in tensor memory (in shared memory they would be written and read
// once more), the tokens its N.  A product (M 128, K 16) takes 47 cycles for N up to 64
// and 65 for N = 128 (measured).
//
// The weights are scaled before the products, so that a product's sums run on over
// all columns and are read back once a segment: (code - 8) s in fp16, the row's largest
// scale brought to 2^-5..2^-4.  It has at most 11 significant bits, as many as fp16 keeps:
// the weights are exact where s is at least 2^-12 of the row's largest, smaller ones are
// rounded to 2^-19 of it.  One block per SM:
//  * up to three groups of eight warps, each for every second or third chunk, a row of
//    tile 0 or 1 to a thread, make the row's operands, and bring a segment's sums out
//    behind its last chunk.  A group takes some 2200 cycles to a chunk: 330 instructions a
//    warp, the six warps of a scheduler in turn, which is what the time goes by.  The
//    writes of the warps on an issuing warp's scheduler moreover wait behind the
//    products that were issued before.
//  * a warp copies, two warps issue the products, one a tile's.
// Every wait is bounded (abort flag and error word); after an abort the warps run
// on without waiting, so that they meet at the block's barriers.
//
// 70B feed-forward: 32 tokens 82 us, 64 tokens 98, 128 tokens 140; 389 tokens of the 8B
// one 139 us, 0.99 PFLOP/s.  Up to 64 tokens a chunk takes some 1000 cycles, of which
// its bytes take 720 and its products 750.  Tried:
//  * e4m3 operands as subnormals, group sums read back and scaled in 32 bits: 32 tokens
//    100 us, 64 tokens (two tiles) 170;
//  * half a chunk to a step: 107 us (for 97), an issuing warp waits twice as often;
//  * two groups instead of three where there are three buffers: 95 us (for 91).
// Operands in shared memory would be written and read once more there, some 1500 cycles
// a chunk.
constexpr int MOST = 128;  // tokens of a tile
__host__ __device__ constexpr int sum_columns(int nt) { return (nt + 31) / 32 * 32; }
constexpr int GROUP = 8, GROUPS = 3, MANY_WARPS = GROUP * GROUPS + 3, COPIER = GROUP * GROUPS, ISSUERS = COPIER + 1, MANY_THREADS = MANY_WARPS * 32;
constexpr int MANY_STAGES = 8, MANY_BUFS = 3, MANY_SMEM = 224 * 1024 + 1024;
static_assert(MANY_SMEM + 1024 <= 232448, "shared memory per block, what the kernel declares itself counted in");

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
__device__ __forceinline__ void tmem_loaded(uint32_t (&a)[8], uint32_t (&b)[8]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 8; i += 4)
    asm volatile("" : "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(b[i]), "+r"(b[i + 1]), "+r"(b[i + 2]), "+r"(b[i + 3]));
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// A in tensor memory, two consecutive columns of a row to a 32-bit cell.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// (code - 8) * s for the codes of two columns at bits 4-7 and 20-23, which are code * 2^-20
// as fp16 subnormals, with m = s 2^20 and c = -8 s.  (Codes made into numbers of ordinary
// size, less 8, times s: two instructions for this one, 87 us for 82.)
__device__ __forceinline__ uint32_t weights_of(uint32_t w, uint32_t m, uint32_t c) {
  uint32_t v = w & 0x00f000f0u;
  asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(v) : "r"(m), "r"(c));
  return v;
}

template <int SUBS>
__global__ void __launch_bounds__(MANY_THREADS, 1) product_kernel(const __grid_constant__ ProductParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // of a chunk: copied, its products done; of a buffer of operands: written; of the sums: read
  __shared__ uint64_t full[MANY_STAGES], done[MANY_STAGES], a_full[2][MANY_BUFS], d_free, drain[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < MANY_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&done[i], 2);
    }
    for (int i = 0; i < 2 * MANY_BUFS; ++i) mbar_init(&a_full[0][i], GROUP / 2);
    mbar_init(&d_free, GROUP);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == COPIER) tmem_alloc(&tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  // the sums of tile 0 and of tile 1, then the buffers, 64 columns for either tile.  All of
  // tensor memory is the block's: it starts at 0 (and that the compiler knows it makes
  // issuing products cheaper).
  const uint32_t d_cols = sum_columns(p.nt), a_tmem = 2 * d_cols;
  const Wait W{&s_abort, p.err, p.timeout_ns};
  const Run run(p);
  const int x_bytes = p.nt * 256;

  if (warp == COPIER) {
    if (lane == 0) copy_chunks(p, run, Ring{p.stages, x_bytes, p.stage_bytes}, smem, full, done, W);
    __syncwarp();
  } else if (warp >= ISSUERS) {
    const int tile = warp - ISSUERS;
    // ------------------------------------------------ products
    // A warp to a tile (one for both: 91 us for 32 tokens of the 70B feed-forward).  It
    // stays together and one lane waits and issues: what a product is told is
    // the same for all lanes, else it takes three times as long to issue.
    const bool leader = elect_one();
    const uint32_t id = (1u << 4) | (static_cast<uint32_t>(p.nt >> 3) << 17) | (8u << 24);  // fp16 x fp16 -> fp32, M = 128
    const uint64_t x_desc = sw128_desc(smem_u32(smem), 16);
    int stage = 0, buf = 0, chunk = static_cast<int>(run.first % p.chunks);
    uint32_t a_phase = 0, d_phase = 1;
    bool fresh = true;  // of a unit's sums
#pragma unroll 1
    for (int i = 0; i < run.count; ++i) {
      const uint64_t xd = x_desc + static_cast<uint64_t>(stage * (p.stage_bytes >> 4));
      if (leader) {
        if (fresh) W(&d_free, d_phase);
        W(&a_full[tile][buf], a_phase);  // (the tokens have landed, else there were no operands)
      }
      __syncwarp();
      tc_fence_after();
      if (leader) {
        const uint32_t at = a_tmem + buf * 128 + tile * 64;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_f16_ta(tile * d_cols, at + k * 8, xd + static_cast<uint64_t>((k >> 2) * (p.nt * 128 >> 4) + ((k & 3) * 32 >> 4)), id,
                      k > 0 || !fresh);
        umma_commit(&done[stage]);
      }
      __syncwarp();
      if (++buf == p.bufs) {
        buf = 0;
        a_phase ^= 1;
      }
      if (fresh) d_phase ^= 1;
      fresh = ++chunk == p.chunks;
      if (fresh) chunk = 0;
      if (++stage == p.stages) stage = 0;
    }
    if (leader) {
      umma_commit(&drain[tile]);
      W.drain(&drain[tile], 0);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    // ------------------------------------------------ operands, and the sums back
    const int tile = (warp >> 2) & 1, group = warp / GROUP;
    const uint32_t at_w = x_bytes + tile * 8192 + r * 64, swz = (r >> 1) & 3;
    const uint32_t at_s = x_bytes + 16384 + (tile * 128 + r) * 2;
    // Chunk i goes to buffer i mod bufs, whose products before are chunk i - bufs's.  A
    // group that comes to chunk i knows chunk i - groups - bufs done.  So no wait here
    // may pass for a phase two before the one it means: there are as many groups as
    // buffers at most, and stages for both together (see launch_w4_product).
    const int groups = p.bufs < GROUPS ? p.bufs : GROUPS;
    int stage = group, buf = group, before = group - p.bufs;  // of chunk i - bufs
    uint32_t phase = 0, before_phase = 0;
    int unit = static_cast<int>(run.first / p.chunks), chunk = static_cast<int>(run.first - static_cast<long long>(unit) * p.chunks) + group;
    for (; chunk >= p.chunks; chunk -= p.chunks) ++unit;
    const float* up_at = p.row_up + tile * 128 + r;
    float up = unit < p.units ? up_at[unit * 256] : 0.f, next = unit + 1 < p.units ? up_at[(unit + 1) * 256] : 0.f;
    float* parts = p.parts + (static_cast<long long>(blockIdx.y) * (p.blocks + p.units - 1) + blockIdx.x) * (p.nt * 256) + tile * 128 + r;
    bool waited = false;
#pragma unroll 1
    for (int i = group < groups ? group : run.count; i < run.count; i += groups) {
      const uint32_t st = smem_u32(smem) + stage * p.stage_bytes;
      W.warp(&full[stage], phase);
      uint4 v[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = ld_shared_v4(st + at_w + ((t ^ swz) << 4));
      uint32_t m[SUBS], c[SUBS];
#pragma unroll
      for (int j = 0; j < SUBS; ++j) {
        const float s = ld_shared_scale(st + at_s + j * 512) * up;
        asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(m[j]) : "f"(s * 16.f));
        asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(c[j]) : "f"(s * -1.220703125e-4f));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // 32 columns
        uint32_t o[16];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t w = q == 0 ? v[t].x : q == 1 ? v[t].y : q == 2 ? v[t].z : v[t].w;
          const uint32_t mq = m[q * SUBS / 4], cq = c[q * SUBS / 4];
          o[4 * t] = weights_of(w << 4, mq, cq);
          o[4 * t + 1] = weights_of(w, mq, cq);
          o[4 * t + 2] = weights_of(w >> 4, mq, cq);
          o[4 * t + 3] = weights_of(w >> 8, mq, cq);
        }
        if (q == 0) {
          if (i >= p.bufs) W.warp(&done[before], before_phase);
          tc_fence_after();
        }
        tmem_store16(a_tmem + lanes + buf * 128 + tile * 64 + q * 16, o);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_full[tile][buf]);
      if (chunk + 1 == p.chunks || i + 1 == run.count) {
        // a segment's last chunk: the sums back, a row of one tile to a thread
        W.warp_long(&done[stage], phase);  // its products are done, so all are
        tc_fence_after();
        if (!waited) grid_dep_wait();  // nobody reads the parts of before
        waited = true;
        float* to = parts + static_cast<long long>(unit) * (p.nt * 256);
        const uint32_t from = lanes + tile * d_cols;
#pragma unroll 1
        for (int c = 0; c < p.nt; c += 16) {
          uint32_t a[8], b[8];
          tmem_load8(from + c, a);
          tmem_load8(from + c + 8, b);
          tmem_loaded(a, b);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            __stcg(to + (c + j) * 256, __uint_as_float(a[j]));
            __stcg(to + (c + j + 8) * 256, __uint_as_float(b[j]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_free);
      }
      buf += groups;
      if (buf >= p.bufs) buf -= p.bufs;
      stage += groups;
      if (stage >= p.stages) {
        stage -= p.stages;
        phase ^= 1;
      }
      before += groups;
      if (before >= p.stages) {
        before -= p.stages;
        before_phase ^= 1;
      }
      chunk += groups;
      if (chunk >= p.chunks) {
        const int units = chunk / p.chunks;  // more than one where units are short
        chunk -= units * p.chunks;
        unit += units;
        up = units == 1 ? next : unit < p.units ? up_at[unit * 256] : 0.f;
        next = unit + 1 < p.units ? up_at[(unit + 1) * 256] : 0.f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == COPIER) {
    tc_fence_after();
    tmem_dealloc(tmem_slot, 512);
  }
}

// The parts of a unit's sums, in the order of the columns, to outputs or hidden
// activations: a warp to a token, four rows of tile 0 and four of tile 1 to a thread.
// Its own kernel, as then all of the device takes part; the block that came last
// doing it cost 8 us for 64 tokens of an output projection and 14 for 128 of the 70B
// feed-forward, this costs some 3.
constexpr int FINISH_TOKENS = 8;
__global__ void __launch_bounds__(FINISH_TOKENS * 32) finish_kernel(const __grid_constant__ ProductParams p) {
  grid_dep_launch();
  const int unit = blockIdx.x, tile = blockIdx.z, in_tile = blockIdx.y * FINISH_TOKENS + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, q4 = lane * 4;
  const long long token = static_cast<long long>(tile) * p.nt + in_tile;
  auto block_of = [&](long long chunk) {  // (a division of 64 bits takes as long as the rest)
    const long long a = (chunk + 1) * p.blocks - 1;
    return a >> 32 ? static_cast<int>(a / p.total) : static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(p.total));
  };
  const long long u0 = static_cast<long long>(unit) * p.chunks;
  const int c0 = block_of(u0), c1 = block_of(u0 + p.chunks - 1);
  const float* from = p.parts + ((static_cast<long long>(tile) * (p.blocks + p.units - 1) + c0 + unit) * p.nt + in_tile) * 256 + q4;
  const float4 up0 = *reinterpret_cast<const float4*>(p.row_up + unit * 256 + q4),
               up1 = *reinterpret_cast<const float4*>(p.row_up + unit * 256 + 128 + q4);
  grid_dep_wait();
  if (token >= p.n) return;
  const int down = p.e_in[token * APART] - 15;
  float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
#pragma unroll 4
  for (int b = c0; b <= c1; ++b, from += p.nt * 256) {
    v0 = add4(v0, __ldcg(reinterpret_cast<const float4*>(from)));
    v1 = add4(v1, __ldcg(reinterpret_cast<const float4*>(from + 128)));
  }
  auto scaled = [&](float4 v, float4 u) {  // by 2^(16 + down) over the row's factor
    auto one = [&](float x, float f) {
      const int e = down + 16 + 127 - static_cast<int>(__float_as_uint(f) >> 23);
      if (e >= -126 && e <= 127) return x * __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      return x * pow2(e / 2) * pow2(e - e / 2);  // (a tiny token and a huge row, or the other way round)
    };
    return make_float4(one(v.x, u.x), one(v.y, u.y), one(v.z, u.z), one(v.w, u.w));
  };
  v0 = scaled(v0, up0);
  v1 = scaled(v1, up1);
  if (p.epi == W4_SWIGLU) {  // tile 1 has the second matrix's rows of the same hidden slots
    v0.x *= sigmoid_f(v0.x) * v1.x;
    v0.y *= sigmoid_f(v0.y) * v1.y;
    v0.z *= sigmoid_f(v0.z) * v1.z;
    v0.w *= sigmoid_f(v0.w) * v1.w;
    write4<false>(p, p.nt, tile, in_tile, unit * 128ll + q4, lane, v0);
  } else {
    write4<false>(p, p.nt, tile, in_tile, unit * 256ll + q4, lane, v0);
    write4<false>(p, p.nt, tile, in_tile, unit * 256ll + 128 + q4, lane, v1);
  }
}

// The hidden activations of a token, whose blocks of 128 columns finish_kernel has written
// with powers of two of their own, brought to the token's: its largest is known when all
// of them are written.  What it rounds are elements below 2^-28 of that, by 2^-39 of it.
// (A bound from the token's absolute sum and the largest scales needs no kernel, but lies
// as far above the hidden activations as one scale lies above the others: with one
// group in either matrix 2^10 times the others, results were off by up to 0.016 for 0.0017.)
// A block to 16 tokens of a block of columns, a thread to eight columns: 2 us of the
// pass for 32 tokens of the 70B feed-forward, 5 for 128.
constexpr int FIT_TOKENS = 16;
__global__ void __launch_bounds__(FIT_TOKENS * 16) fit_kernel(const __grid_constant__ ProductParams p) {
  grid_dep_launch();
  const int chunk = blockIdx.x, tile = blockIdx.z, i = threadIdx.x & 127, in = blockIdx.y * FIT_TOKENS + (i >> 3);
  const int token = tile * p.nt + in;
  uint4* at = reinterpret_cast<uint4*>(p.image_out + (static_cast<long long>(tile) * p.out_chunks + chunk) * image_bytes(p.nt)) +
              (threadIdx.x >> 7) * (p.nt * 8) + in * 8 + (i & 7);
  grid_dep_wait();
  if (token >= p.n) return;
  const uint4 v = *at;
  const float f = pow2(p.e_chunk[static_cast<long long>(chunk) * p.padded + token] - p.e_out[token * APART]);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    const __half2 h = __floats2half2_rn(a.x * f, a.y * f);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *at = make_uint4(w[0], w[1], w[2], w[3]);
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
int launch_few(const ProductParams& p, dim3 grid, cudaStream_t st) {
  if (p.m.group == 128) return launch_inst<few_kernel<1>, FEW_THREADS, Few::SMEM>(grid, st, p);
  if (p.m.group == 64) return launch_inst<few_kernel<2>, FEW_THREADS, Few::SMEM>(grid, st, p);
  return launch_inst<few_kernel<4>, FEW_THREADS, Few::SMEM>(grid, st, p);
}
int launch_product(const ProductParams& p, dim3 grid, cudaStream_t st) {
  if (p.m.group == 128) return launch_inst<product_kernel<1>, MANY_THREADS, MANY_SMEM>(grid, st, p);
  if (p.m.group == 64) return launch_inst<product_kernel<2>, MANY_THREADS, MANY_SMEM>(grid, st, p);
  return launch_inst<product_kernel<4>, MANY_THREADS, MANY_SMEM>(grid, st, p);
}

// How a product of n tokens is cut: NT tokens to a block, `tiles` of them, `blocks`
// runs of chunks.
struct Cut {
  int nt, tiles, blocks;
};
Cut cut_of(const W4Shape& m, int64_t n, int num_sms) {
  Cut c;
  if (n <= FEW) {
    c.nt = FEW;
    c.tiles = 1;
    c.blocks = 2 * num_sms;
  } else {
    c.tiles = static_cast<int>((n + MOST - 1) / MOST);
    c.nt = static_cast<int>(((n + c.tiles - 1) / c.tiles + 15) / 16 * 16);
    c.blocks = std::max(num_sms / c.tiles, 1);  // a wave: a call has four tiles at most
  }
  c.blocks = static_cast<int>(std::min<int64_t>(c.blocks, m.units() * m.chunks()));
  return c;
}
// Where the exponents of an image of n tokens lie.
int64_t image_end(const W4Shape& m, const Cut& c) { return m.chunks() * c.tiles * image_bytes(c.nt); }

int64_t hidden_chunks(const W4Shape& m) { return m.T * m.sp / 128; }
int* hidden_exponents(const W4Product& a, const Cut& c) {
  return reinterpret_cast<int*>(static_cast<uint8_t*>(a.image_out) + hidden_chunks(a.m) * c.tiles * image_bytes(c.nt));
}
// A grid of at most 32 blocks per SM.
unsigned grid_of(long long blocks, int num_sms) { return static_cast<unsigned>(std::min<long long>(std::max<long long>(blocks, 1), 32 * num_sms)); }
int launched() { return cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA; }  // (an error is not left for the next call)

}  // namespace w4

int launch_w4_quantize(const void* W, int64_t rows, int64_t cols, int64_t segs, int group, void* codes, void* scales,
                       int num_sms, cudaStream_t st) {
  using namespace w4;
  const int64_t seg = cols / segs, seg_groups = (seg + group - 1) / group;
  auto* sc = static_cast<__nv_bfloat16*>(scales);
  if (seg % 16 == 0) {
    const int lanes = group == 32 ? 1 : group == 64 ? 2 : 3;
    const long long places = rows * segs * (seg_groups << lanes);
    quantize16_kernel<<<grid_of((places + 255) / 256, num_sms), 256, 0, st>>>(
        static_cast<const uint4*>(W), rows * (cols / 16), static_cast<int>(cols / 16), static_cast<int>(seg / 16), lanes,
        static_cast<int>(seg_groups), static_cast<int>(segs), static_cast<uint2*>(codes), sc);
    return launched();
  }
  const auto* w = static_cast<const __nv_bfloat16*>(W);
  const int n_segs = static_cast<int>(segs), width = static_cast<int>(seg), groups = static_cast<int>(seg_groups);
  const int lanes = group == 32 ? 2 : group == 64 ? 3 : 4;
  scales_kernel<<<grid_of((((rows * segs * seg_groups) << lanes) + 255) / 256, num_sms), 256, 0, st>>>(w, rows, cols, n_segs, width,
                                                                                              lanes, groups, sc);
  if (seg >= 8)
    codes8_kernel<<<grid_of((rows * ((cols + 7) / 8) + 255) / 256, num_sms), 256, 0, st>>>(
        w, rows, static_cast<int>(cols), n_segs, width, group, groups, sc, static_cast<uint8_t*>(codes));
  else
    codes_kernel<<<grid_of((rows * ((cols + 1) / 2) + 255) / 256, num_sms), 256, 0, st>>>(
      w, rows, cols, static_cast<int>(segs), seg, group, seg_groups, sc, static_cast<uint8_t*>(codes));
  return launched();
}

int launch_w4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, int64_t segs, int group,
                         void* W, int num_sms, cudaStream_t st) {
  using namespace w4;
  const int64_t seg = cols / segs, seg_groups = (seg + group - 1) / group;
  const auto* sc = static_cast<const __nv_bfloat16*>(scales);
  if (seg % 16 == 0) {
    const long long pieces = rows * (cols / 16);
    dequantize16_kernel<<<grid_of((pieces + 255) / 256, num_sms), 256, 0, st>>>(
        static_cast<const uint2*>(codes), sc, pieces, static_cast<int>(cols / 16), static_cast<int>(seg / 16),
        group == 32 ? 1 : group == 64 ? 2 : 3, static_cast<int>(seg_groups), static_cast<int>(segs), static_cast<uint4*>(W));
  } else if (seg >= 8) {
    dequantize8_kernel<<<grid_of((rows * ((cols + 7) / 8) + 255) / 256, num_sms), 256, 0, st>>>(
        static_cast<const uint8_t*>(codes), sc, rows, static_cast<int>(cols), static_cast<int>(segs), static_cast<int>(seg),
        group, static_cast<int>(seg_groups), static_cast<__nv_bfloat16*>(W));
  } else {
    dequantize_kernel<<<grid_of((rows * cols + 255) / 256, num_sms), 256, 0, st>>>(
        static_cast<const uint8_t*>(codes), sc, rows, cols, static_cast<int>(segs), seg, group, seg_groups,
        static_cast<__nv_bfloat16*>(W));
  }
  return launched();
}

int launch_w4_pack(const W4Shape& m, const W4Codes& c, void* packed, int unpack, int num_sms, cudaStream_t st) {
  using namespace w4;
  auto* to = static_cast<uint8_t*>(packed);
  pack_kernel<<<grid_of(m.units() * m.chunks(), num_sms), 256, 0, st>>>(m, c, to, unpack);
  if (unpack) {
    unpack_codes_kernel<<<grid_of(m.tiles(), num_sms), 256, 0, st>>>(m, c, to);
  } else {
    row_up_kernel<<<static_cast<unsigned>(m.units()), 256, 0, st>>>(m, to);
  }
  return launched();
}

size_t w4_product_scratch(const W4Shape& m, int64_t n, int num_sms) {
  const w4::Cut c = w4::cut_of(m, n, num_sms);
  const size_t places = c.nt <= w4::FEW ? 2 * c.blocks : c.tiles * (c.blocks + m.units() - 1);
  return places * 256 * c.nt * sizeof(float);
}
int64_t w4_product_counters(const W4Shape& m, int64_t n) { return n <= w4::FEW ? m.units() : 0; }

size_t w4_image_bytes(const W4Shape& m, int64_t n, bool hidden) {
  const w4::Cut c = w4::cut_of(m, n, 1);
  const int64_t exponents = c.nt <= w4::FEW ? 0 : c.tiles * c.nt * (w4::APART + (hidden ? m.chunks() : 0));
  return static_cast<size_t>(w4::image_end(m, c)) + static_cast<size_t>(exponents) * sizeof(int);
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
  const bool few = c.nt <= FEW;
  unsigned blocks;
  if (few) {
    blocks = static_cast<unsigned>(std::min<int64_t>((p.tiles * p.chunks * p.nt + 7) / 8, 8 * ctx.num_sms));
  } else {
    p.e_in = reinterpret_cast<int*>(p.image + image_end(a.m, c));
    if (a.epi != W4_OUT) p.e_out = hidden_exponents(a, c);
    blocks = static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(p.tiles) * p.nt, 4 * ctx.num_sms));
  }
  if (ctx.before) ctx.before(ctx.user, "prepare4", ctx.stream);
  if (few)
    launch_dep(prepare_few_kernel, dim3(blocks), 256, 0, ctx.stream, p);
  else
    launch_dep(prepare_kernel, dim3(blocks), PREPARE_THREADS, 0, ctx.stream, p);
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
  p.out_chunks = a.epi == W4_OUT ? 0 : static_cast<int>(hidden_chunks(a.m));
  p.parts = static_cast<float*>(a.scratch);
  p.counters = a.counters;
  p.err = ctx.err;
  p.skip_load = ctx.debug_skip_load;
  p.timeout_ns = ctx.timeout_ns;
  ctx.debug_skip_load = 0;
  const dim3 grid(static_cast<unsigned>(c.blocks), static_cast<unsigned>(c.tiles));
  if (ctx.before) ctx.before(ctx.user, a.name, ctx.stream);
  int rc;
  if (c.nt == FEW) {
    rc = launch_few(p, grid, ctx.stream);
  } else {
    p.nt = c.nt;
    p.stage_bytes = image_bytes(c.nt) + (p.block_bytes + 1023) / 1024 * 1024;
    // bufs + groups <= stages: 3 + 3 of at least 6 up to 64 tokens, 2 + 2 of at least 4 above
    p.stages = std::min((MANY_SMEM - 1024) / p.stage_bytes, MANY_STAGES);
    p.bufs = std::min((512 - 2 * sum_columns(c.nt)) / 128, MANY_BUFS);
    if (p.stages < p.bufs + std::min(p.bufs, GROUPS)) return TP_ERR_INVALID;
    p.row_up = a.m.row_up(const_cast<void*>(a.packed));
    p.padded = c.tiles * c.nt;
    p.e_in = reinterpret_cast<const int*>(p.image + image_end(a.m, c));
    if (a.epi != W4_OUT) {
      p.e_out = hidden_exponents(a, c);
      p.e_chunk = p.e_out + p.padded * APART;
    }
    p.blocks = c.blocks;
    rc = launch_product(p, grid, ctx.stream);
  }
  if (rc) return rc;
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  if (c.nt > FEW) {
    if (ctx.before) ctx.before(ctx.user, "finish4", ctx.stream);
    launch_dep(finish_kernel, dim3(static_cast<unsigned>(p.units), static_cast<unsigned>(c.nt / FINISH_TOKENS), static_cast<unsigned>(c.tiles)),
               FINISH_TOKENS * 32, 0, ctx.stream, p);
    ctx.launches++;
    if (a.epi != W4_OUT) {  // (timed as one with it)
      launch_dep(fit_kernel, dim3(static_cast<unsigned>(p.out_chunks), static_cast<unsigned>(c.nt / FIT_TOKENS), static_cast<unsigned>(c.tiles)),
                 FIT_TOKENS * 16, 0, ctx.stream, p);
      ctx.launches++;
    }
    if (ctx.after) ctx.after(ctx.user, ctx.stream);
  }
  return launched();
}

}  // namespace tpffn
