// tp_w4.cu -- 4-bit weights with group scales: quantising, the layout that the
// products read, and the products of few tokens with such weights.
//
// A group of `group` consecutive columns of a row has the scale s (bf16), its
// elements are (code - 8) s with codes 0..15.
#include <cuda.h>
#include <cuda_bf16.h>
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
// y[token][row] = sum_g s[row][g] sum_{k in g} (code - 8) x[token][k], for up to
// 64 tokens at a time.
//
// Bound by the one read of the codes for few tokens.  The weights are the matrix
// unit's A operand, 128 rows at a time, the tokens its N: code - 8 is a bf16
// number without rounding, and the product of a group is scaled in 32 bits when
// it is read back, so a result is as exact as the sums in 32 bits.  (A scaled
// weight would have to be rounded to bf16.)
//
// A block takes a run of chunks (128 columns of a unit's 256 rows) of the list of
// all units' chunks, the same number as the others, whatever units they belong to;
// a run of chunks of one unit is a segment.  One block has
//  * warp 16: copies of the chunks into a ring: the packed block (codes, scales) in
//    one piece, as it lies, the tokens' 128 columns by two TMA boxes;
//  * warps 0-15, in four groups of 128 threads, a row to a thread: tile 0 and 1 of
//    the unit, the even and the odd steps (a step: a group's columns).  A thread
//    turns its row's codes into bf16 and writes them to tensor memory, where the
//    matrix unit takes them from (shared memory would be written and read once
//    more), then reads the step's product back, scales and adds it.  Four groups,
//    so that one's products run while others turn codes;
//  * warp 17: issues tcgen05.mma.
// At a segment's end the groups' sums meet in tensor memory (all four have row r in
// lane r).  A unit that several blocks share is joined by the last of them to
// come, in the order of the columns.
//
// Every wait is bounded (abort flag and error word); after an abort the warps run
// on without waiting, so that they meet at the block's barriers.
using namespace tc;

constexpr int GROUPS_OF_WARPS = 4, WORK_WARPS = 16, THREADS = (WORK_WARPS + 2) * 32;
constexpr int T_COLS = 64;  // columns of tensor memory for a group's weights, and for its products

struct ProductParams {
  W4Shape m;
  const uint8_t* packed;
  long long total;  // chunks of all units
  int chunks, seg_chunks, block_bytes, units;
  long long n, out_rs;
  int epi;
  const __nv_bfloat16* bias;
  __nv_bfloat16* out;
  float* parts;   // [blocks][2][2 tiles][NT][128]
  int* counters;  // [token tiles][units]
  int* err;
  int skip_load;
  unsigned long long timeout_ns;
};

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
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) ok = slow(bar, parity, true);
    return __all_sync(0xffffffffu, ok) != 0;
  }
};

// NT: tokens of a product (N); NC: those that are read back.
template <int NT>
struct Ring {
  static constexpr int X_BYTES = NT * 256, CODES = 18432, STAGE = X_BYTES + CODES;
  static constexpr int STAGES = NT <= 16 ? 8 : (NT <= 32 ? 7 : 6);
  static constexpr int SMEM = STAGES * STAGE + 1024;
  static_assert(SMEM <= 232448 - 1024, "shared memory per block");
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
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Two codes (bits 0-3 of each half) as bf16: 128 + code by its bits, less 136.
__device__ __forceinline__ uint32_t two_weights(uint32_t w) {
  uint32_t d, r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(d) : "r"(w));  // (w & mask) | bits
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(d), "r"(0x43084308u));
  return r;
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[N]) {
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
  }
  tmem_wait_ld();
  // names the registers, so that no use of them moves before the wait
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_store8(uint32_t at, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// SUBS: groups of a chunk.
template <int NT, int NC, int SUBS>
__global__ void __launch_bounds__(THREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ ProductParams p) {
  using R = Ring<NT>;
  constexpr int LD = NC < 16 ? NC : 16;  // columns read back at a time
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[R::STAGES], empty[R::STAGES], a_full[GROUPS_OF_WARPS], d_full[GROUPS_OF_WARPS], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort, s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], SUBS == 1 ? WORK_WARPS / 2 : WORK_WARPS);  // the warps that have a step of the chunk
    }
    for (int i = 0; i < GROUPS_OF_WARPS; ++i) {
      mbar_init(&a_full[i], 4);
      mbar_init(&d_full[i], 1);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == WORK_WARPS && lane == 0) prefetch_tmap(&tx);
  if (warp == WORK_WARPS + 1) tmem_alloc(&tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;  // group g's weights at T_COLS g, its products at 256 + T_COLS g
  const Wait W{&s_abort, p.err, p.timeout_ns};
  const long long first = p.total * blockIdx.x / gridDim.x, last = p.total * (blockIdx.x + 1) / gridDim.x;
  const int count = static_cast<int>(last - first);  // chunks
  constexpr int KSTEPS = 8 / SUBS;  // K = 16 steps of a group
  const long long n0 = static_cast<long long>(blockIdx.y) * NT;

  if (warp == WORK_WARPS) {
    // ------------------------------------------------ copies
    // The weights are not the previous kernel's to write (what wrote them is done
    // before the call's first kernel lets others start); the tokens may be.
    if (lane == 0) {
      const uint64_t policy = gridDim.y == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
      const uint8_t* src = p.packed + first * p.block_bytes;
      auto weights = [&](int i) {
        uint8_t* st = smem + (i % R::STAGES) * R::STAGE;
        mbar_arrive_expect_tx(&full[i % R::STAGES], static_cast<uint32_t>(p.block_bytes + R::X_BYTES));
        if (!(p.skip_load && i == 0)) bulk_load(st + R::X_BYTES, src + static_cast<long long>(i) * p.block_bytes,
                                                static_cast<uint32_t>(p.block_bytes), &full[i % R::STAGES], policy);
      };
      int c = static_cast<int>(first % p.chunks), e = c / p.seg_chunks, in = c - e * p.seg_chunks;
      auto tokens = [&](int i) {
        uint8_t* st = smem + (i % R::STAGES) * R::STAGE;
        uint64_t* bar = &full[i % R::STAGES];
        tma_load_3d(st, &tx, bar, in * 128, e, static_cast<int>(n0));
        tma_load_3d(st + NT * 128, &tx, bar, in * 128 + 64, e, static_cast<int>(n0));
        if (++in == p.seg_chunks) {
          in = 0;
          if (++e * p.seg_chunks == p.chunks) e = 0;
        }
      };
      const int ahead = count < R::STAGES ? count : R::STAGES;
      for (int i = 0; i < ahead; ++i) weights(i);
      grid_dep_wait();
      for (int i = 0; i < ahead; ++i) tokens(i);
      int issued = ahead;
      for (int i = ahead; i < count; ++i) {
        if (!W(&empty[i % R::STAGES], ((i / R::STAGES) & 1) ^ 1)) break;
        weights(i);
        tokens(i);
        ++issued;
      }
      // every issued copy lands before the block may exit
      for (int i = issued > R::STAGES ? issued - R::STAGES : 0; i < issued; ++i)
        W.drain(&full[i % R::STAGES], (i / R::STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == WORK_WARPS + 1) {
    // ------------------------------------------------ products
    // A product takes 48 cycles, whatever N up to 64 is (measured; M 128, K 16, from
    // tensor or shared memory): few instructions may lie between two.
    const bool leader = elect_one();
    constexpr uint32_t ID = idesc(NT, 0, 0);
    const uint64_t x_desc = kdesc(smem_u32(smem), NT, 0);
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0, step = 0;
#pragma unroll 1
    for (int i = 0; i < count && ok; ++i) {
      ok = W.warp(&full[stage], phase);
      const uint64_t xd = x_desc + static_cast<uint64_t>(stage * (R::STAGE >> 4));
#pragma unroll
      for (int sub = 0; sub < SUBS; ++sub, ++step) {
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          const uint32_t g = 2 * tile + (step & 1);
          ok = ok && W.warp(&a_full[g], (step >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ad = tmem + g * T_COLS;
          if (leader) {
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) {
              const int ks = sub * KSTEPS + k;
              umma_bf16_ta(ad + 256, ad + k * 8, xd + static_cast<uint64_t>(((ks >> 2) * NT * 128 + (ks & 3) * 32) >> 4), ID,
                           k > 0);
            }
            umma_commit(&d_full[g]);
          }
          __syncwarp();
        }
      }
      if (++stage == R::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (leader) umma_commit(&drain);
    __syncwarp();
    W.drain(&drain, 0);
    __syncwarp();
  } else {
    // ------------------------------------------------ weights to bf16, products back, sums
    const int g = warp >> 2, tile = g >> 1, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t at_a = tmem + lane_base + g * T_COLS, at_d = tmem + lane_base + 256 + g * T_COLS;
    constexpr int PIECES = 4 / SUBS;
    grid_dep_wait();  // the counters are clear, and nobody reads the outputs or parts of before
    float acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = 0.f;
    uint32_t mine = 0;  // steps of this group so far
    int stage = 0;
    uint32_t phase = 0;
    long long unit = first / p.chunks;
    int chunk = static_cast<int>(first - unit * p.chunks);
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      if (SUBS > 1 || (i & 1) == (g & 1)) {
        const uint8_t* st = smem + stage * R::STAGE + R::X_BYTES;
        const uint32_t codes = smem_u32(st) + tile * 8192 + r * 16;
        W.warp(&full[stage], phase);
#pragma unroll 1
        for (int sub = SUBS > 1 ? g & 1 : 0; sub < SUBS; sub += 2) {
#pragma unroll
          for (int q = 0; q < PIECES; ++q) {
            const uint4 v = ld_shared_v4(codes + (sub * PIECES + q) * 2048);
            uint32_t a[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              a[j] = two_weights(v.x >> (4 * j));
              a[4 + j] = two_weights(v.y >> (4 * j));
              a[8 + j] = two_weights(v.z >> (4 * j));
              a[12 + j] = two_weights(v.w >> (4 * j));
            }
            tmem_st16(at_a + q * 16, a);
          }
          const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(st + 16384)[sub * 256 + tile * 128 + r]);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&a_full[g]);
          W.warp(&d_full[g], mine & 1);
          ++mine;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < NC; c += LD) {
            uint32_t d[LD];
            tmem_load<LD>(at_d + c, d);
#pragma unroll
            for (int j = 0; j < LD; ++j) acc[c + j] = fmaf(s, __uint_as_float(d[j]), acc[c + j]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
      }
      if (++stage == R::STAGES) {
        stage = 0;
        phase ^= 1;
      }
      if (++chunk < p.chunks && i + 1 < count) continue;

      // ---- end of a segment of `unit`: the odd steps' sums to the even ones'
      const int odd = g & 1;
      if (odd) {
#pragma unroll
        for (int c = 0; c < NC; c += 8) tmem_store8(at_d + c, acc + c);
        tmem_wait_st();
        tc_fence_before();
      }
      bar_sync(1 + tile, 256);
      if (!odd) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NC; c += LD) {
          uint32_t d[LD];
          tmem_load<LD>(at_d + T_COLS + c, d);
#pragma unroll
          for (int j = 0; j < LD; ++j) acc[c + j] += __uint_as_float(d[j]);
        }
        tc_fence_before();
      }
      bar_sync(1 + tile, 256);  // read: the odd group's next products may come
      if (!odd) {
        const long long u0 = unit * p.chunks, u1 = u0 + p.chunks - 1;
        const int C = gridDim.x;
        const int c0 = static_cast<int>(((u0 + 1) * C - 1) / p.total), c1 = static_cast<int>(((u1 + 1) * C - 1) / p.total);
        bool write = true;
        if (c0 != c1) {
          // a part: [tile][token][row]
          const long long slot = NT * 256;
          float* parts = p.parts + static_cast<long long>(blockIdx.y) * C * 2 * slot + tile * (NT * 128) + r;
          float* to = parts + (2 * blockIdx.x + (blockIdx.x == c0)) * slot;
#pragma unroll
          for (int c = 0; c < NC; ++c) __stcg(to + c * 128, acc[c]);
          __threadfence();
          bar_sync(3, 256);
          if (threadIdx.x == 0) {
            int* counter = p.counters + blockIdx.y * p.units + unit;
            s_last = atomicAdd(counter, 1) == c1 - c0;
          }
          bar_sync(3, 256);
          write = s_last != 0;
          if (write) {
            __threadfence();
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[c] = 0.f;
            for (int b = c0; b <= c1; ++b) {
              const float* from = parts + (2 * b + (b == c0)) * slot;
#pragma unroll
              for (int c = 0; c < NC; ++c) acc[c] += __ldcg(from + c * 128);
            }
          }
        }
        long long row = unit * 256 + tile * 128 + r;
        bool store = write && *W.abort_flag == 0;
        if (p.epi == W4_SWIGLU) {
          // tile 1 has the second matrix's rows of the same hidden slots
          if (tile) {
#pragma unroll
            for (int c = 0; c < NC; c += 8) tmem_store8(at_d + c, acc + c);
            tmem_wait_st();
            tc_fence_before();
          }
          bar_sync(3, 256);
          if (!tile) {
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < NC; c += LD) {
              uint32_t d[LD];
              tmem_load<LD>(at_d + 2 * T_COLS + c, d);
#pragma unroll
              for (int j = 0; j < LD; ++j) acc[c + j] = acc[c + j] * sigmoid_f(acc[c + j]) * __uint_as_float(d[j]);
            }
            tc_fence_before();
          }
          bar_sync(3, 256);
          row = unit * 128 + r;
          store = store && !tile && row < p.m.T * p.m.sp;
        } else if (p.epi == W4_GELU) {
          const long long t = row / p.m.sp, in = row - t * p.m.sp;
          const float b = p.bias && in < p.m.s && t < p.m.T ? __bfloat162float(p.bias[t * p.m.s + in]) : 0.f;
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[c] = gelu_tanh_f(acc[c] + b);
          store = store && row < p.m.T * p.m.sp;
        } else {
          store = store && row < p.m.rows;
          if (p.bias && store) {
            const float b = __bfloat162float(p.bias[row]);
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[c] += b;
          }
        }
        if (store) {
          __nv_bfloat16* to = p.out + n0 * p.out_rs + row;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (n0 + c < p.n) to[c * p.out_rs] = __float2bfloat16_rn(acc[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] = 0.f;
      chunk = 0;
      ++unit;
    }
  }
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  if (warp == WORK_WARPS + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Clears what a call counts in, when everything before it on the stream is done;
// the products behind it read their weights without a further wait.
__global__ void __launch_bounds__(256) reset_kernel(int* err, int* counters, int n) {
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x == 0 && blockIdx.x == 0) *err = 0;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) counters[i] = 0;
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

template <int NT, int NC, int SUBS>
int launch_product_inst(const CUtensorMap& tx, const ProductParams& p, dim3 grid, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TP_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    if (cudaFuncSetAttribute(product_kernel<NT, NC, SUBS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<NT>::SMEM) != cudaSuccess)
      return TP_ERR_CUDA;
    done.fetch_or(bit);
  }
  launch_dep(product_kernel<NT, NC, SUBS>, grid, THREADS, Ring<NT>::SMEM, st, tx, p);
  return TP_OK;
}

template <int NT, int NC>
int launch_product(const CUtensorMap& tx, const ProductParams& p, dim3 grid, cudaStream_t st) {
  if (p.m.group == 128) return launch_product_inst<NT, NC, 1>(tx, p, grid, st);
  if (p.m.group == 64) return launch_product_inst<NT, NC, 2>(tx, p, grid, st);
  return launch_product_inst<NT, NC, 4>(tx, p, grid, st);
}

// How a product of n tokens is cut: NT tokens to a block, `tiles` of them, `blocks`
// runs of chunks.
struct Cut {
  int nt, tiles, blocks;
};
Cut cut_of(const W4Shape& m, int64_t n, int num_sms) {
  Cut c;
  c.nt = n <= 16 ? 16 : (n <= 32 ? 32 : 64);
  c.tiles = static_cast<int>((n + c.nt - 1) / c.nt);
  const int64_t most = std::max(num_sms / c.tiles, 1), total = m.units() * m.chunks();
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

int launch_w4_reset(int* err, int* counters, int64_t n, LaunchCtx& ctx) {
  w4::launch_dep(w4::reset_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 8) + (n == 0))), 256, 0,
                 ctx.stream, err, counters, static_cast<int>(n));
  ctx.launches++;
  return w4::launched();
}

int launch_w4_product(const W4Product& a, LaunchCtx& ctx) {
  using namespace w4;
  const Cut c = cut_of(a.m, a.n, ctx.num_sms);
  ProductParams p{};
  p.m = a.m;
  p.packed = static_cast<const uint8_t*>(a.packed);
  p.chunks = static_cast<int>(a.m.chunks());
  p.seg_chunks = static_cast<int>(a.m.seg_chunks());
  p.total = a.m.units() * a.m.chunks();
  p.block_bytes = a.m.block_bytes();
  p.units = static_cast<int>(a.m.units());
  p.n = a.n;
  p.out_rs = a.out_rs;
  p.epi = a.epi;
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.parts = static_cast<float*>(a.scratch);
  p.counters = a.counters;
  p.err = ctx.err;
  p.skip_load = ctx.debug_skip_load;
  p.timeout_ns = ctx.timeout_ns;
  ctx.debug_skip_load = 0;
  const uint64_t dims[3] = {static_cast<uint64_t>(a.m.seg), static_cast<uint64_t>(a.m.segs), static_cast<uint64_t>(a.n)};
  const uint64_t str[2] = {static_cast<uint64_t>(a.m.segs > 1 ? a.x_seg : a.x_rs) * 2, static_cast<uint64_t>(a.x_rs) * 2};
  const uint32_t box[3] = {64, 1, static_cast<uint32_t>(c.nt)};
  CUtensorMap tx;
  if (int rc = encode_map_3d_bf16(&tx, a.x, dims, str, box)) return rc;
  const dim3 grid(static_cast<unsigned>(c.blocks), static_cast<unsigned>(c.tiles));
  if (ctx.before) ctx.before(ctx.user, a.name, ctx.stream);
  int rc;
  if (a.n <= 8)
    rc = launch_product<16, 8>(tx, p, grid, ctx.stream);
  else if (c.nt == 16)
    rc = launch_product<16, 16>(tx, p, grid, ctx.stream);
  else if (c.nt == 32)
    rc = launch_product<32, 32>(tx, p, grid, ctx.stream);
  else
    rc = launch_product<64, 64>(tx, p, grid, ctx.stream);
  if (rc) return rc;
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  return launched();
}

}  // namespace tpffn
