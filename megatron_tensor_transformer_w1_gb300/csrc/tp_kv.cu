// tp_kv.cu -- the serving operators of the head-sharded attention sublayer:
// appending the new tokens' keys and values to a paged cache, with the
// rotation by position, and attention of few query rows over that cache.
//
// Sequence b of a batch has new tokens in rows cu[b] .. cu[b+1] - 1 and
// kv_len[b] keys, the new tokens' included; key j lies in page
// page_table[b][j / page_size], slot j % page_size.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "tc_ptx.cuh"
#include "tp_internal.h"
#include "tp_kv.cuh"
#include "tpffn.h"

namespace tpffn {
namespace kv {
using tc::grid_dep_launch;
using tc::grid_dep_wait;
using tc::ex2;
using tc::pack_bf16x2;
using tc::smem_u32;

// ================================================================ append
// A token at position t turns the pairs (x_j, y_j) of each of its query and
// key heads by the angle t * inv_freq[j]:
//   x' = (x cos - y sin) scale,  y' = (y cos + x sin) scale,
// pairs (j, j + r/2) or, interleaved, (2j, 2j + 1), for the first r columns.
// The angle is formed in turns, modulo one, in 64-bit fixed point: t times
// the fraction inv_freq / 2 pi, which is found once per thread (a float
// product t * f loses the angle of far positions, and 64-bit floating point is
// slow here); what sincospi gets is rounded to 24 bits of half a turn.
//
// Bound by memory: every element is read once and written once.  A warp takes
// 4 IT heads of a token, a lane 8 pairs of a head: its 8 angles are the same
// for all heads, so four lanes find two each and pass them around.  The
// elements are on their way before the token's sequence and page are looked
// up.  IT = 2 makes that and the angles cheaper per head (12604 tokens of 48
// heads, 310 MB: 53 us, IT = 4 60 us); IT = 1 spreads few tokens over more
// warps.
struct AppendParams {
  Batch b;
  const __nv_bfloat16* qkv;
  __nv_bfloat16* q;
  const float* inv_freq;
  float scale;
  int rot, interleaved;
  int hq_per, hk_per;  // query / key heads per shard
  int* header;         // see kKvHeaderBytes
  int alone;
};

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
// (x, y) = (low, high) halves of two words' pairs: the pairs (a.lo, b.lo), (a.hi, b.hi)
__device__ __forceinline__ void turn_across(uint32_t& wa, uint32_t& wb, float2 c0, float2 c1) {
  const float2 a = unpack_bf16x2(wa), b = unpack_bf16x2(wb);
  wa = pack_bf16x2(a.x * c0.x - b.x * c0.y, a.y * c1.x - b.y * c1.y);
  wb = pack_bf16x2(b.x * c0.x + a.x * c0.y, b.y * c1.x + a.y * c1.y);
}
// the pair within a word
__device__ __forceinline__ void turn_within(uint32_t& w, float2 c) {
  const float2 x = unpack_bf16x2(w);
  w = pack_bf16x2(x.x * c.x - x.y * c.y, x.y * c.x + x.x * c.y);
}

constexpr int APPEND_THREADS = 256;

template <int IT>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int s_err;
  const Batch& B = p.b;
  const int lane = threadIdx.x & 31, k = lane & 7, sub = lane >> 3;
  const int per = p.hq_per + 2 * p.hk_per, heads = B.H + 2 * B.Hkv;
  const int half = p.rot / 16;  // 16-byte chunks of half the rotated columns
  const bool turns = k < half;  // lane k of a head has the pairs 8 k .. 8 k + 7
  // two 16-byte chunks of a head: eight pairs' halves, or neighbours
  const int ca = !p.interleaved && turns ? k : 2 * k, cb = !p.interleaved && turns ? k + half : 2 * k + 1;
  if (threadIdx.x == 0) s_err = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  unsigned long long freq[2] = {0, 0};  // turns per position of pairs 8 k + 2 sub, + 1, in 2^-64
  if (turns) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const double f = static_cast<double>(p.inv_freq[8 * k + 2 * sub + e]) * 0.15915494309189533577;  // 1 / (2 pi)
      freq[e] = static_cast<unsigned long long>(__double2ll_rn((f - rint(f)) * 9223372036854775808.0)) << 1;
    }
  }
  const int chunks = (heads + 4 * IT - 1) / (4 * IT);
  const long long units = static_cast<long long>(B.n_tokens) * chunks;
  const int warps = gridDim.x * (APPEND_THREADS / 32);
  int err = 0;
  for (long long u = blockIdx.x * (APPEND_THREADS / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const int row = static_cast<int>(u / chunks), h0 = static_cast<int>(u - static_cast<long long>(row) * chunks) * 4 * IT;
    const uint4* src = reinterpret_cast<const uint4*>(p.qkv + static_cast<long long>(row) * heads * HD);
    uint4 a[IT], c[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int hh = h0 + 4 * i + sub;
      if (hh < heads) {
        a[i] = src[hh * 16 + ca];
        c[i] = src[hh * 16 + cb];
      }
    }
    const int b = find_seq_warp(B.cu, B.B, row);
    if (b >= B.B) continue;
    const int first = B.cu[b], end = B.cu[b + 1];
    if (first > row || first < 0) {  // no sequence's row: left as it is
      if (first < 0) err = DEV_ERR_BATCH;
      continue;
    }
    const int pos = B.kv_len[b] - (end - row);
    long long page = -1;
    if (pos >= 0 && pos < B.cap) {
      page = B.table[static_cast<long long>(b) * B.max_pages + (pos >> B.page_shift)];
      if (page >= B.n_pages) page = -1;
    }
    if (page < 0 || end > B.n_tokens) err = DEV_ERR_BATCH;
    float2 cs[8];
    if (half) {
      float2 mine[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int turn = static_cast<int>((static_cast<unsigned long long>(static_cast<long long>(pos)) * freq[e]) >> 32);
        float s, co;
        sincospif(static_cast<float>(turn) * 4.656612873077392578125e-10f, &s, &co);  // 2^-31: half turns
        mine[e] = make_float2(co * p.scale, s * p.scale);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i].x = __shfl_sync(0xffffffffu, mine[i & 1].x, k + 8 * (i >> 1));
        cs[i].y = __shfl_sync(0xffffffffu, mine[i & 1].y, k + 8 * (i >> 1));
      }
    }
    const int slot = pos & ((1 << B.page_shift) - 1);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int hh = h0 + 4 * i + sub;
      if (hh >= heads) continue;
      const int t = hh / per, w = hh - t * per;
      if (turns && w < p.hq_per + p.hk_per) {
        if (p.interleaved) {
          turn_within(a[i].x, cs[0]);
          turn_within(a[i].y, cs[1]);
          turn_within(a[i].z, cs[2]);
          turn_within(a[i].w, cs[3]);
          turn_within(c[i].x, cs[4]);
          turn_within(c[i].y, cs[5]);
          turn_within(c[i].z, cs[6]);
          turn_within(c[i].w, cs[7]);
        } else {
          turn_across(a[i].x, c[i].x, cs[0], cs[1]);
          turn_across(a[i].y, c[i].y, cs[2], cs[3]);
          turn_across(a[i].z, c[i].z, cs[4], cs[5]);
          turn_across(a[i].w, c[i].w, cs[6], cs[7]);
        }
      }
      __nv_bfloat16* dst;
      if (w < p.hq_per) {
        dst = p.q + (static_cast<long long>(row) * B.H + t * p.hq_per + w) * HD;
        if (pos < 0) a[i] = c[i] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        if (page < 0) continue;
        const bool is_k = w < p.hq_per + p.hk_per;
        const int h = t * p.hk_per + (is_k ? w - p.hq_per : w - p.hq_per - p.hk_per);
        dst = (is_k ? B.k : B.v) + ((((page * B.Hkv + h) << B.page_shift) + slot) * HD);
      }
      reinterpret_cast<uint4*>(dst)[ca] = a[i];
      reinterpret_cast<uint4*>(dst)[cb] = c[i];
    }
  }
  if (err) atomicOr(&s_err, err);
  __syncthreads();
  if (threadIdx.x == 0) {
    p.header[kKvHeaderWords + blockIdx.x] = s_err;
    if (blockIdx.x == 0) {
      p.header[1] = gridDim.x;
      if (p.alone) p.header[0] = p.header[2] = 0;
    }
  }
}

// ================================================================ few rows
// Attention of at most 16 WR query rows per item over the cache.  An item is
// a key/value head of a sequence, its rows the sequence's new tokens times
// the G query heads of the group (so K and V are read once for the group);
// or, for the shared keys, a key/value head with the rows of every sequence.
// Its floor is the one read of K and V from memory, 512 bytes per key.
//
// Work is cut in tiles of 64 keys and every block takes the same number of
// consecutive ones of the whole batch (see Cut), however the lengths differ; a block
// starts and ends inside an item, and the parts of an item (its running
// maximum, sum and unnormalised output) are joined by kv_combine_kernel.
//
// One block: 4 warps, stages of a tile's K and V (32 KB) filled by 16-byte
// asynchronous copies, so that two blocks per SM keep some 128 KB in flight.
// 4 / WR key groups of warps: a warp takes 16 query rows and 16 WR keys of a
// tile with its own running maximum and sum (no exchange per tile); the groups
// meet at the end of a segment, where few instructions count: with a warp or
// two per scheduler each takes some four cycles, and short sequences end a
// segment every few tiles (a row to a warp, no division, absent rows left out:
// 3900 -> 2000 cycles a segment; 7 sequences of 100 to 5000 keys 19 -> 17 us).
// The products are m16n8k16 matrix instructions on registers: for so few rows
// they take less time than the bytes do, and the 128-row tensor-memory products
// would be mostly empty.
// WR = 2 has two stages: three would leave room for one block per SM (32
// sequences of 4000 keys, 32 rows, 531 MB: 150 us; with two 97 us).
// Measured: one sequence of 131072 keys, 537 MB, 84 us with the join (6.4
// TB/s); 32 sequences of 64 to 16384 keys, 390 MB, 67 us.
// A segment costs about a tile's time besides its tiles, and counts for one more
// when work is dealt (64 sequences of 16 to 1024 keys 28 -> 26 us, 32 of 64 to
// 16384 keys 68 -> 67 us).
constexpr int FEW_START = 1;
template <int WR>
struct Few {
  static constexpr int WK = 4 / WR;           // key groups
  static constexpr int ROWS = 16 * WR;
  static constexpr int NB = WR;               // 16-key blocks of a warp per tile
  static constexpr int STAGES = WR == 1 ? 3 : 2;  // two blocks per SM
  static constexpr int KV_BYTES = KT * HD * 2;
  static constexpr int Q_BYTES = ROWS * HD * 2;
  static constexpr int STAGE = 2 * KV_BYTES + Q_BYTES;
  static constexpr int SMEM = STAGES * STAGE + 1024;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// 16-byte chunk c of row r of a tile with 256-byte rows: eight rows' chunks
// of one column fall into different banks
__device__ __forceinline__ uint32_t tile_chunk(uint32_t tile, int r, int c) {
  return tile + static_cast<uint32_t>(r * 256 + ((c ^ (r & 7)) << 4));
}

template <int WR, bool PREFIX>
__global__ void __launch_bounds__(128, 2) kv_few_kernel(const __grid_constant__ AttendParams p) {
  using F = Few<WR>;
  using C = Cut<PREFIX, KT, 0, PREFIX ? 0 : FEW_START>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ float2 s_ml[4][16];
  __shared__ Cursor s_cur[F::STAGES];
  __shared__ int s_err;
  const Batch& B = p.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rg = warp / F::WK, kg = warp % F::WK;
  // row / G for rows below 32, without a division (some thirty instructions)
  const uint32_t g_inv = (65536u + B.G - 1) / B.G;
  auto token_of = [&](int r) { return static_cast<int>(r * g_inv >> 16); };
  if (tid == 0) s_err = 0;
  if (!p.beside && !p.behind_append) grid_dep_wait();
  if (!p.behind_append) grid_dep_launch();
  int err = 0;
  Cursor c;
  const Sched S = schedule<C, PREFIX>(B, p.part.sched, reinterpret_cast<SchedScratch*>(smem), c, &err, p.part.early,
                                      p.part.lead);
  if (p.behind_append) {
    grid_dep_wait();
    grid_dep_launch();
  }
  __syncthreads();
  const int t0 = C::t0(B), lo = C::first_key(B);
  int left = S.left;
  int n_tiles = left;  // at most; known when the copies have come to the end
  if (left <= 0) {
    if (!PREFIX && S.some_empty && B.shared == 0) write_empty_rows<C>(p, 0);
    if (tid == 0 && p.part.split) p.part.split[blockIdx.x] = Split{};
    if (p.beside) grid_dep_wait();
    if (err) atomicOr(&s_err, err);
    __syncthreads();
    if (tid == 0) p.status[blockIdx.x] = s_err;
    return;
  }

  // The page of each 8-key group of four tiles of the cursor's item from its
  // tile on, a lane to a group; checked when it is used, a tile later: behind
  // the copies under way a load takes long.
  auto look_up = [&](const Cursor& x) -> int {
    const int key = (t0 + x.t) * KT + lane * 8;
    if (key >= x.s.kv) return -1;
    const int row = PREFIX ? S.table_row : x.b;
    return B.table[static_cast<long long>(row) * B.max_pages + (key >> B.page_shift)];
  };
  // Copies of tile x, whose groups' pages are in lanes `from` on.  What this
  // takes to issue is felt in the stream of bytes: a whole tile within a page
  // (pages of 64 keys or more) finds its place once.
  const int ch = tid & 15, r0 = tid >> 4, mask = (1 << B.page_shift) - 1;
  const long long page_stride = (static_cast<long long>(B.Hkv) << B.page_shift) * HD;
  auto issue = [&](int stage, const Cursor& x, int pages, int from, bool new_item) {
    if (pages < 0 || pages >= B.n_pages) {
      // (a lane without a key has -1)
      if ((t0 + x.t) * KT + (lane - from) * 8 < x.s.kv && lane >= from && lane < from + 8) err = DEV_ERR_BATCH;
      pages = -1;
    }
    const uint32_t ks = smem_u32(smem + stage * F::STAGE), vs = ks + F::KV_BYTES, qs = vs + F::KV_BYTES;
    const int first = (t0 + x.t) * KT;
    const int page = __shfl_sync(0xffffffffu, pages, from);
    if (B.page_shift >= 6 && page >= 0 && first >= lo && first + KT <= x.s.kv) {
      const long long off =
          (((static_cast<long long>(page) * B.Hkv + x.h) << B.page_shift) + (first & mask) + r0) * HD + ch * 8;
      const __nv_bfloat16 *k = B.k + off, *v = B.v + off;
      const uint32_t at = tile_chunk(0, r0, ch);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cp_async16(ks + at + i * 2048, k + i * 8 * HD);
        cp_async16(vs + at + i * 2048, v + i * 8 * HD);
      }
    } else if (B.page_shift >= 6) {
      const long long off =
          (((static_cast<long long>(max(page, 0)) * B.Hkv + x.h) << B.page_shift) + (first & mask) + r0) * HD + ch * 8;
      const __nv_bfloat16 *k = B.k + off, *v = B.v + off;
      const uint32_t at = tile_chunk(0, r0, ch);
      const int from = lo - first - r0, to = page >= 0 ? x.s.kv - first - r0 : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cp_async16(ks + at + i * 2048, k + i * 8 * HD, 8 * i >= from && 8 * i < to);
        cp_async16(vs + at + i * 2048, v + i * 8 * HD, 8 * i >= from && 8 * i < to);
      }
    } else {
      const long long head = (static_cast<long long>(x.h) << B.page_shift) * HD + ch * 8;
      const uint32_t at = tile_chunk(0, r0, ch);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = first + r0 + 8 * i;
        const int page = __shfl_sync(0xffffffffu, pages, from + i);
        const bool ok = page >= 0 && key >= lo && key < x.s.kv;
        const long long off = ok ? page * page_stride + head + (key & mask) * HD : 0;
        cp_async16(ks + at + i * 2048, B.k + off, ok);
        cp_async16(vs + at + i * 2048, B.v + off, ok);
      }
    }
    if (new_item) {
      const int rows = x.s.qn * B.G;
#pragma unroll
      for (int i = 0; i < 2 * WR; ++i) {
        const int r = r0 + 8 * i;
        const bool ok = r < rows;
        const int tok = ok ? token_of(r) : 0, g = ok ? r - tok * B.G : 0;
        const long long off =
            ok ? (static_cast<long long>(x.s.q0 + tok) * B.H + x.h * B.G + g) * HD + ch * 8 : 0;
        cp_async16(tile_chunk(qs, r, ch), p.q + off, ok);
      }
    }
    if (tid == 0) s_cur[stage] = x;
  };

  int issued = 0, looked_at = c.t;  // tiles copied so far; the tile that `pages` begins with
  int pages = look_up(c);

  float o[16][4];
  float m[2], l[2];
  uint32_t qf[8][4];
  int limit[2] = {0, 0};
  bool fresh = true;         // the next tile starts a segment
  int seg_t = 0;             // its first tile within the item
  // (The copies run STAGES - 1 tiles ahead.  They begin in the same loop: the
  // code for them is long, and a second copy of it is fetched for nothing.)
#pragma unroll 1
  for (int i = 1 - F::STAGES; i < n_tiles; ++i) {
    if (i >= 0) {
      cp_async_wait<F::STAGES - 2>();
      __syncthreads();  // tile i has landed for everybody; tile i - 1 has been used by everybody
    }
    if (issued < n_tiles) {
      issue(issued % F::STAGES, c, pages, 8 * (c.t - looked_at), issued == 0 || c.t == 0);
      ++issued;
      left = left_behind<C>(B, c, left);
      if (left <= 0) {
        n_tiles = issued;
      } else {
        advance<C, PREFIX>(B, c);
        if (c.t == 0 || c.t == looked_at + 4) {
          looked_at = c.t;
          pages = look_up(c);
        }
      }
    }
    cp_async_commit();
    if (i < 0) continue;
    const int stage = i % F::STAGES;
    const Cursor x = s_cur[stage];
    const uint32_t ks = smem_u32(smem + stage * F::STAGE), vs = ks + F::KV_BYTES, qs = vs + F::KV_BYTES;
    const int rows = x.s.qn * B.G;
    if (fresh) {
      seg_t = x.t;
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        ldsm4(qf[k], tile_chunk(qs, rg * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)));
      // how many of the sequence's keys this thread's two rows see
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rg * 16 + (lane >> 2) + 8 * e;
        limit[e] = 0;
        if (r < rows) {
          const int tok = token_of(r);
          if (PREFIX && S.all_see) {
            limit[e] = x.s.kv;
          } else if (PREFIX) {
            const int b = find_seq(B.cu, B.B, tok);
            if (b < B.B) {
              const Seq s = load_seq(B, b);
              if (tok >= s.q0 && tok < s.q0 + s.qn) limit[e] = min(s.visible(tok - s.q0, B.causal), x.s.kv);
            }
          } else {
            limit[e] = x.s.visible(tok, B.causal);
          }
        }
      }
      fresh = false;
    }
    if (rg * 16 < rows) {
      const int key0 = kg * 16 * F::NB;  // this warp's keys of the tile
      const int base = (t0 + x.t) * KT + key0;
      float s[F::NB][2][4];
#pragma unroll
      for (int nb = 0; nb < F::NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nb][0][e] = s[nb][1][e] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t kf[4];
          ldsm4(kf, tile_chunk(ks, key0 + nb * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
          mma16816(s[nb][0], qf[k], kf[0], kf[1]);
          mma16816(s[nb][1], qf[k], kf[2], kf[3]);
        }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nb = 0; nb < F::NB; ++nb)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = base + nb * 16 + n * 8 + (lane & 3) * 2 + (e & 1);
            if (key < lo || key >= limit[e >> 1]) s[nb][n][e] = -INFINITY;
            mx[e >> 1] = fmaxf(mx[e >> 1], s[nb][n][e]);
          }
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2)) * p.scale_log2;
        // the maximum moves only when it grew by more than 2^8
        alpha[e] = 1.f;
        if (mx[e] > m[e] + 8.f || m[e] == -INFINITY) {
          if (mx[e] > m[e]) {
            alpha[e] = ex2(m[e] - mx[e]);
            m[e] = mx[e];
          }
        }
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= alpha[e >> 1];
        l[0] *= alpha[0];
        l[1] *= alpha[1];
      }
      const float nm[2] = {m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]};
#pragma unroll
      for (int nb = 0; nb < F::NB; ++nb) {
        uint32_t pf[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            e4[e] = ex2(fmaf(s[nb][n][e], p.scale_log2, nm[e >> 1]));
            l[e >> 1] += e4[e];
          }
          // the probabilities are rounded to bf16 for the second product, as
          // its operand has to be; their sum is taken before that
          pf[2 * n] = pack_bf16x2(e4[0], e4[1]);
          pf[2 * n + 1] = pack_bf16x2(e4[2], e4[3]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t vf[4];
          ldsm4t(vf, tile_chunk(vs, key0 + nb * 16 + (lane & 15), 2 * j + (lane >> 4)));
          mma16816(o[2 * j], pf, vf[0], vf[1]);
          mma16816(o[2 * j + 1], pf, vf[2], vf[3]);
        }
      }
    }
    if (x.t + 1 < x.nt && i + 1 < n_tiles) continue;

    // ---- end of a segment: the key groups of the rows meet
    fresh = true;
    if (tid == 0 && i + 1 == n_tiles && p.part.split)
      p.part.split[blockIdx.x] = split_of<C>(B, S, x, seg_t, S.first + S.places - 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if ((lane & 3) == 0) s_ml[warp][(lane >> 2) + 8 * e] = make_float2(m[e], l[e]);
    }
    __syncthreads();  // everybody is done with this tile's K and V: they become the meeting place
    const uint32_t meet = smem_u32(smem + stage * F::STAGE);  // [4 warps][16 rows][HD]
    {
      // a row's groups of 8 columns are exchanged by the row, so that a store's
      // eight rows use different banks; rows behind the last are not read
      const uint32_t at = meet + (warp * 16 + (lane >> 2)) * (HD * 4) + ((lane >> 2) << 5) + ((lane & 3) << 3);
      if (rg * 16 < rows) {
#pragma unroll
        for (int j = 0; j < 16; ++j) st_shared_v2(at ^ (j << 5), o[j][0], o[j][1]);
      }
      if (rg * 16 + 8 < rows) {
#pragma unroll
        for (int j = 0; j < 16; ++j) st_shared_v2((at + 8 * HD * 4) ^ (j << 5), o[j][2], o[j][3]);
      }
    }
    __syncthreads();
    const bool whole = seg_t == 0 && x.t + 1 == x.nt;
    const bool direct = whole && !PREFIX && B.shared == 0;
    const long long slot = 2ll * blockIdx.x + (seg_t ? 0 : 1);
    // a warp takes a row, a lane four columns
#pragma unroll 2
    for (int r = warp; r < rows; r += 4) {
      const int r16 = r & 15, w0 = (r >> 4) * F::WK, tok = token_of(r);
      float2 ml[F::WK];
      float mr = -INFINITY, lr = 0.f;
#pragma unroll
      for (int g = 0; g < F::WK; ++g) {
        ml[g] = s_ml[w0 + g][r16];
        mr = fmaxf(mr, ml[g].x);
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < F::WK; ++g) {
        const float f = mr == -INFINITY ? 0.f : ex2(ml[g].x - mr);
        lr += ml[g].y * f;
        const float4 w = ld_shared_f4(meet + ((w0 + g) * 16 + r16) * (HD * 4) + ((lane << 4) ^ ((r16 & 7) << 5)));
        v.x += w.x * f;
        v.y += w.y * f;
        v.z += w.z * f;
        v.w += w.w * f;
      }
      const long long row = static_cast<long long>(x.s.q0 + tok) * B.H + x.h * B.G + (r - tok * B.G);
      if (direct) {
        const float inv = inverse_sum(lr, x.s.visible(tok, B.causal) > 0);
        reinterpret_cast<uint2*>(p.o + row * HD)[lane] =
            make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        if (p.lse && lane == 0) p.lse[row] = log2_sum_exp(mr, lr);
      } else {
        float* dst = whole ? p.part.row_o + row * HD + lane * 4 : p.part.slot_o + slot_chunk(p.part, slot, r, lane);
        *reinterpret_cast<float4*>(dst) = v;
        if (lane == 0) (whole ? p.part.row_ml[row] : p.part.slot_ml[slot * p.part.slot_rows + r]) = make_float2(mr, lr);
      }
    }
  }
  cp_async_wait<0>();
  if (!PREFIX && S.some_empty && B.shared == 0) write_empty_rows<C>(p, 0);
  if (p.beside) grid_dep_wait();
  if (err) atomicOr(&s_err, err);
  __syncthreads();
  if (tid == 0) p.status[blockIdx.x] = s_err;
}

// ================================================================ combine
// Joins the parts of a row: with (m_i, l_i, O_i) the running maximum, sum and
// unnormalised output of part i, m = max m_i, l = sum l_i 2^(m_i - m),
// o = sum O_i 2^(m_i - m) / l, always in the order of the parts, so that a
// result does not change from run to run.  A row without any key gets zeros; one
// with NaN or +inf among its scores has NaN for its sum, and gets NaN.
// Bound by latency: the parts lie in L2.  A warp takes a row, a lane
// four columns; several warps share a row where there are few rows in all, so
// that the many parts of a long sequence are read at once.
struct CombineParams {
  Batch b;
  Parts own, shared;
  __nv_bfloat16* o;
  float* lse;
  int rows_per_pass;     // that a block's eight warps take: 1, 2, 4 or 8
  int* header;           // see kKvHeaderBytes
  int alone, status_words;
};

// The parts of an item's rows: block c's slot of rows for c of [c0, c0 + n),
// or, n = 1, the rows' own places.
struct ItemParts {
  int n = 0;
  long long c0 = 0;
  // its first and last tile's places
  __device__ __forceinline__ void set(const Parts& P, long long first, long long last, long long total, int least) {
    if (first < 0 || first > last || last >= total) return;  // no list that the kernels cut: no parts
    const Deal D(total, P.grid, P.early, P.lead, least);
    c0 = D.block_of(first);
    n = static_cast<int>(D.block_of(last) - c0) + 1;
  }
  // the slot of part i: the first begins the item, the others go on
  __device__ __forceinline__ long long slot(int i) const { return 2 * (c0 + i) + (i == 0); }
};

__device__ __forceinline__ void scale4(float4& a, float f) {
  a.x *= f;
  a.y *= f;
  a.z *= f;
  a.w *= f;
}
__device__ __forceinline__ void add4(float4& a, float f, const float4& v) {
  a.x += f * v.x;
  a.y += f * v.y;
  a.z += f * v.z;
  a.w += f * v.w;
}

// A block takes rows of one item.  SHARED: any item, blockIdx.x being its
// number, with the parts of its own keys and of the shared ones.  Otherwise
// the item that block blockIdx.x of the attention began and others ended.
template <bool SHARED>
__global__ void __launch_bounds__(256) kv_combine_kernel(const __grid_constant__ CombineParams p) {
  __shared__ float4 s_acc[8][32];
  __shared__ float2 s_ml[8];
  grid_dep_wait();
  grid_dep_launch();
  const Batch& B = p.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    p.header[2] = p.status_words;
    if (p.alone) p.header[0] = p.header[1] = 0;
  }
  ItemParts own, sh;
  Seq s{};  // the item's sequence
  int h, rt = 0, rows = 0;  // rows: of this row tile
  long long nt_sh = 0, n_rt_sh = 0;
  int srt = 0;  // row tile of the shared keys' that `sh` is of
  auto shared_parts = [&](int row_tile) {
    srt = row_tile;
    sh.n = 0;
    const long long at = (h * n_rt_sh + srt) * nt_sh;
    if (nt_sh > 0) sh.set(p.shared, at, at + nt_sh - 1, nt_sh * n_rt_sh * B.Hkv, 1);
  };
  auto shared_tile = [&](int row) { return p.shared.rt ? row / RT_MANY : 0; };
  if (SHARED) {
    // The first warp looks the item up for all: eight times its divisions are
    // most of what the kernel would issue.
    __shared__ ItemParts s_own, s_sh;
    __shared__ int s_item[3];
    __shared__ Seq s_seq;
    __shared__ long long s_tiles[2];
    h = blockIdx.x % B.Hkv;
    if (warp == 0) {
      const int u = blockIdx.x / B.Hkv;
      int b = u;
      if (p.own.rt) {
        // sequence b's row tiles start at cu[b] G / RT + b: the last b with
        // first(b) <= u, 32 places to a round
        auto first = [&](int x) {
          return min(max(B.cu[x], 0), B.n_tokens) * static_cast<long long>(B.G) / RT_MANY + x;
        };
        int n = B.B;  // b lies in [lo, lo + n)
        b = 0;
        while (n > 1) {
          const int step = (n + 31) >> 5, at = lane * step;
          const int cnt = __popc(__ballot_sync(0xffffffffu, at < n && first(b + at) <= u));
          const int skip = max(cnt - 1, 0) * step;
          b += skip;
          n = min(step, n - skip);
        }
        rt = static_cast<int>(u - first(b));
      }
      s = load_seq(B, b);
      const long long before = p.own.sched[b], per_head = p.own.sched[b + 1] - before, total = p.own.sched[B.B];
      nt_sh = p.shared.sched[0];
      n_rt_sh = p.shared.sched[1];
      rows = rt < 0 ? 0 : min(s.qn * B.G - rt * p.own.rt, p.own.slot_rows);
      long long at = before * B.Hkv + h * per_head;  // the item's places
      if (p.own.rt) {
        using C = Many<false>;
        int sum = 0;
        for (int i = lane; i < rt; i += 32) sum += C::places(B, s, i);
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        at += sum + C::START;
        const int nt = rows > 0 ? C::tiles(B, s, rt) : 0;
        if (nt > 0) own.set(p.own, at, at + (nt - 1) * C::width(B, s, rt), total * B.Hkv, C::LEAST);
      } else if (per_head > 0) {
        own.set(p.own, at + FEW_START, at + per_head - 1, total * B.Hkv, 1);
      }
      shared_parts(shared_tile(s.q0 * B.G + max(rt, 0) * p.own.rt));
      if (lane == 0) {
        s_own = own;
        s_sh = sh;
        s_seq = s;
        s_item[0] = rt;
        s_item[1] = rows;
        s_item[2] = srt;
        s_tiles[0] = nt_sh;
        s_tiles[1] = n_rt_sh;
      }
    }
    __syncthreads();
    own = s_own;
    sh = s_sh;
    s = s_seq;
    rt = s_item[0];
    rows = s_item[1];
    srt = s_item[2];
    nt_sh = s_tiles[0];
    n_rt_sh = s_tiles[1];
  } else {
    const Split x = p.own.split[blockIdx.x];
    if (x.parts == 0) return;
    s = x.s;
    h = x.h;
    rt = x.rt;
    rows = min(s.qn * B.G - rt * p.own.rt, p.own.slot_rows);
    own.n = x.parts;
    own.c0 = blockIdx.x;
  }
  const int share = 8 / p.rows_per_pass;  // warps to a row
  const int wr = warp / share, wp = warp - wr * share;
  for (int row0 = blockIdx.y * p.rows_per_pass; row0 < rows; row0 += gridDim.y * p.rows_per_pass) {
    const int r = row0 + wr;
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    long long at = 0;
    bool sees = false;
    if (r < rows) {
      const int item_row = rt * p.own.rt + r, i_tok = item_row / B.G, tok = s.q0 + i_tok, g = item_row - i_tok * B.G;
      sees = s.visible(i_tok, B.causal) > 0;
      at = static_cast<long long>(tok) * B.H + h * B.G + g;
      int r_sh = 0;
      if (SHARED) {
        const int all = tok * B.G + g, tile = shared_tile(all);
        if (tile != srt) shared_parts(tile);
        r_sh = all - tile * RT_MANY;
      }
      const int n = own.n + sh.n;
      // this warp's parts wp, wp + share, ..., four at a time: all loads of the
      // four are on their way at once
      for (int i0 = wp; i0 < n; i0 += 4 * share) {
        float2 x[4];
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + j * share;
          x[j] = make_float2(-INFINITY, 0.f);
          v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < n) {
            const bool mine = !SHARED || i < own.n;
            const Parts& P = mine ? p.own : p.shared;
            const ItemParts& I = mine ? own : sh;
            const int row = mine ? r : r_sh;
            if (SHARED && I.n == 1) {
              x[j] = P.row_ml[at];
              v[j] = reinterpret_cast<const float4*>(P.row_o + at * HD)[lane];
            } else {
              const long long slot = I.slot(mine ? i : i - own.n);
              x[j] = P.slot_ml[slot * P.slot_rows + row];
              v[j] = *reinterpret_cast<const float4*>(P.slot_o + slot_chunk(P, slot, row, lane));
            }
          }
        }
        const float top = fmaxf(m, fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)));
        // No maximum yet: the sums are 0, or NaN where scores are (a maximum drops
        // NaN), and are added with a weight of 0.
        const float base = top == -INFINITY ? 0.f : top;
        const float f = ex2(m - base);
        m = top;
        l *= f;
        scale4(a, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float w = ex2(x[j].x - base);
          l += w * x[j].y;
          add4(a, w, v[j]);
        }
      }
    }
    if (share > 1) {
      s_acc[warp][lane] = a;
      if (lane == 0) s_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (wp == 0) {
        float top = m;
        for (int w = 1; w < share; ++w) top = fmaxf(top, s_ml[warp + w].x);
        const float f = top == -INFINITY ? 0.f : ex2(m - top);
        m = top;
        l *= f;
        scale4(a, f);
        for (int w = 1; w < share; ++w) {
          const float2 y = s_ml[warp + w];
          const float g = top == -INFINITY ? 0.f : ex2(y.x - top);
          l += g * y.y;
          add4(a, g, s_acc[warp + w][lane]);
        }
      }
      __syncthreads();
    }
    if (r >= rows || wp) continue;
    const float inv = inverse_sum(l, sees);
    reinterpret_cast<uint2*>(p.o + at * HD)[lane] =
        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    if (p.lse && lane == 0) p.lse[at] = log2_sum_exp(m, l);
  }
}

// ================================================================ host
Batch make_batch(const KvSpec& a) {
  Batch b{};
  b.k = static_cast<__nv_bfloat16*>(a.k);
  b.v = static_cast<__nv_bfloat16*>(a.v);
  b.n_pages = a.n_pages;
  b.max_pages = a.max_pages;
  while ((1 << b.page_shift) < a.page_size) ++b.page_shift;
  b.B = a.n_seqs;
  b.n_tokens = a.n_tokens;
  b.max_new = a.max_new;
  b.H = a.H;
  b.Hkv = a.Hkv;
  b.G = a.H / a.Hkv;
  b.causal = a.causal;
  b.cap = kv_cap(a);
  b.shared = a.shared_len;
  b.cu = a.cu;
  b.kv_len = a.kv_len;
  b.table = a.table;
  return b;
}

int few_blocks(int num_sms) { return 2 * num_sms; }

template <int WR, bool PREFIX>
int launch_few_inst(const AttendParams& p, LaunchCtx& ctx, const char* name) {
  static std::atomic<uint64_t> done{0};
  if (int rc = set_smem_once(kv_few_kernel<WR, PREFIX>, Few<WR>::SMEM, done)) return rc;
  if (ctx.before) ctx.before(ctx.user, name, ctx.stream);
  launch_dep(kv_few_kernel<WR, PREFIX>, dim3(p.part.grid), 128, Few<WR>::SMEM, ctx.stream, p);
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  return cudaPeekAtLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}
template <bool PREFIX>
int launch_few(const AttendParams& p, LaunchCtx& ctx, const char* name) {
  if (p.part.slot_rows <= 16) return launch_few_inst<1, PREFIX>(p, ctx, name);
  return launch_few_inst<2, PREFIX>(p, ctx, name);
}

}  // namespace kv

int kv_cap(const KvSpec& a) {
  const long long keys = static_cast<long long>(a.max_pages) * a.page_size;
  return keys < (1 << 30) ? static_cast<int>(keys) : (1 << 30);
}

int launch_kv_append(const KvSpec& a, const KvRotation& r, const void* qkv, void* q, int* header, bool alone,
                     LaunchCtx& ctx) {
  kv::AppendParams p{};
  p.b = kv::make_batch(a);
  p.qkv = static_cast<const __nv_bfloat16*>(qkv);
  p.q = static_cast<__nv_bfloat16*>(q);
  p.inv_freq = r.inv_freq;
  p.scale = r.scale;
  p.rot = r.rotary_dim;
  p.interleaved = r.interleaved;
  p.hq_per = a.H / a.T_p;
  p.hk_per = a.Hkv / a.T_p;
  p.header = header;
  p.alone = alone;
  // 8 heads to a warp where that still gives every SM 32 warps
  const int heads = a.H + 2 * a.Hkv, warps = kv::APPEND_THREADS / 32;
  const bool wide = static_cast<int64_t>(a.n_tokens) * ((heads + 7) / 8) >= 32 * ctx.num_sms;
  const int64_t units = static_cast<int64_t>(a.n_tokens) * (wide ? (heads + 7) / 8 : (heads + 3) / 4);
  const int64_t most = 8 * ctx.num_sms < kKvStatusWords ? 8 * ctx.num_sms : kKvStatusWords;
  const int64_t blocks = (units + warps - 1) / warps;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
  if (ctx.before) ctx.before(ctx.user, "kv_append", ctx.stream);
  if (wide)
    kv::launch_dep(kv::kv_append_kernel<2>, grid, kv::APPEND_THREADS, 0, ctx.stream, p);
  else
    kv::launch_dep(kv::kv_append_kernel<1>, grid, kv::APPEND_THREADS, 0, ctx.stream, p);
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  return cudaPeekAtLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

namespace {
size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// How a call's attention is launched, and its scratch.
// At most so many rows to a key/value head: the few-rows kernel.  32 sequences
// of 4000 keys (8 heads, 531 MB): 16 rows 89 us, 32 rows 97 us against 101 us
// of the many-rows kernel; 64 sequences of 300 keys, 32 rows: 27 against 36.  A
// form of it for 64 rows took 140 against 103 us on the long sequences; where
// only starting the kernel counts it was the faster one (4 sequences of 300 keys,
// 17 against 21 us), which was not worth a third form.
constexpr int kFewRows = 32;
// At most so many rows to a key/value head, on average over the sequences, for
// the shared keys to be taken together: with more, a sequence's products against
// them take longer than their reads.  Of 300 random batches of 40 to 500 rows 38 of
// more than 64 pass the bound below; together they are 0.67 to 2.0 times as fast
// (median 1.07; 27 sequences of 67 tokens, 8 key heads, behind 21184 keys 181 / 366
// us, 13 of 96 rows of one key head behind 16576, with 2000 own keys, 58 / 39 us),
// the faster ones behind some 20000 keys and without own ones.
constexpr int kShareRows = 64;
// At least so many bytes of shared keys and values that would be read again: what
// a kernel and the join cost (12 us of reads), and for each row its parts.  Both
// ways were timed for 1400 random batches (1 to 16 key heads, groups of 1 to 8, 1
// to 32 new tokens, 2 to 256 sequences, 14 MB to 1 GB saved, no to 4096 own keys),
// with the caches flushed and with the keys left in L2 where they fit: these two
// numbers have the times within 1 % of the better way's on average both times, and
// within 33 % at most; without the rows' share, from 96 MiB on, 2 % and 139 %.
// Together / each on its own, 8 key heads, 300 own keys: 64 single tokens (4 query
// heads to a key head) behind 512 keys (132 MB saved, 105 asked for) 30 / 32 us,
// behind 256 (66 MB) 28 / 25 us, 16 behind 1600 (98 MB, 89) 24 / 27 us, behind 1088
// (67 MB) 21.5 / 22.5 us; 64 of 4 tokens behind 512 (132 MB, 166) 32 / 35 us, behind
// 384 31 - 36 / 31 us; 128 of 16 tokens behind 256 (133 MB, 740) 108 / 66 us.
constexpr double kShareBytes = 80 << 20, kShareRowBytes = 10000;
struct AttendPlan {
  bool share = false;
  kv::Parts own, shared;      // the pointers as offsets from the scratch's start
  int items = 0;              // that the combine kernel looks at
  size_t bytes = 0;
};
// The shared keys' kernel of many rows and the own keys' of few rows, side by
// side: the first on just so many SMs that both end together, by what they were
// measured to take.  The own keys' lengths are the device's to know: short
// items, of two tiles, are assumed; of longer ones the blocks that start at once
// take what they can in the meantime (Deal).  In turn / side by side: 64
// sequences of one token, 4 rows to a key head, 8 key heads, 8192 shared keys
// and 16 to 1024 own ones 48 / 38 us, 4000 own 188 / 178, none 34 / 35, 1024
// shared and 300 own 35 / 26; 128 sequences, 2048 shared and 100 own 40 / 36.
void split_sms(const KvSpec& a, int num_sms, AttendPlan& P) {
  const int64_t rows = static_cast<int64_t>(a.n_tokens) * (a.H / a.Hkv);
  const int64_t tiles = a.Hkv * ((rows + kv::RT_MANY - 1) / kv::RT_MANY) * ((a.shared_len + 127) / 128);
  const double step = rows > 128 ? 1.8 : 1.2;  // us per 128 keys, with two row tiles or one
  auto shared_us = [&](int64_t sms) { return 9.0 + step * ((tiles + sms - 1) / sms); };
  auto own_us = [&](int64_t sms) { return 8.0 + 4.0 * a.n_seqs * a.Hkv / kv::few_blocks(static_cast<int>(sms)); };
  double best = shared_us(num_sms) + own_us(num_sms) - 6.0;  // in turn; the second's start is hidden
  for (int64_t n = 1; n <= 64; ++n) {
    const int64_t sms = (tiles + n - 1) / n;  // with n tiles each
    if (sms >= num_sms) continue;
    const double s = shared_us(sms), o = own_us(num_sms - sms), us = s > o ? s : o;
    if (us >= best) continue;
    best = us;
    P.shared.grid = static_cast<int>(sms);
    P.own.early = kv::few_blocks(static_cast<int>(num_sms - sms));
    P.own.lead = static_cast<int>(s / 1.2);  // 64 keys of an item take a block that long
  }
}
AttendPlan attend_plan(const KvSpec& a, int num_sms, char* ws) {
  AttendPlan P;
  const int64_t G = a.H / a.Hkv, rows = static_cast<int64_t>(a.n_tokens) * a.H;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* at = ws + off;
    off += align256(bytes);
    return at;
  };
  auto part = [&](kv::Parts& p, int64_t item_rows, size_t sched) {
    const bool many = item_rows > kFewRows;
    p.rt = many ? kv::RT_MANY : 0;
    p.slot_rows = static_cast<int>(many ? kv::RT_MANY : item_rows);
    p.grid = many ? num_sms : kv::few_blocks(num_sms);
    const size_t slots = 2 * static_cast<size_t>(p.grid) * p.slot_rows;
    if (P.share)
      p.sched = reinterpret_cast<long long*>(take(sched * 8));
    else
      p.split = reinterpret_cast<kv::Split*>(take(p.grid * sizeof(kv::Split)));
    p.slot_o = reinterpret_cast<float*>(take(slots * kv::HD * 4));
    p.slot_ml = reinterpret_cast<float2*>(take(slots * 8));
    if (P.share) {
      p.row_o = reinterpret_cast<float*>(take(rows * kv::HD * 4));
      p.row_ml = reinterpret_cast<float2*>(take(rows * 8));
    }
  };
  // Where the sequences bring many rows each, their products bound the time,
  // not the reads of the shared keys.
  // Taking the shared keys together pays where it saves enough reads.
  const double saved = (a.n_seqs - 1.0) * a.shared_len * a.Hkv * (kv::HD * 4);
  P.share = saved >= kShareBytes + kShareRowBytes * rows && a.n_tokens * G <= static_cast<int64_t>(kShareRows) * a.n_seqs;
  part(P.own, a.max_new * G, static_cast<size_t>(a.n_seqs) + 1);
  if (P.share) part(P.shared, a.n_tokens * G, 2);
  if (P.share && P.shared.rt && !P.own.rt) split_sms(a, num_sms, P);
  const int64_t units = P.own.rt ? a.n_tokens * G / kv::RT_MANY + a.n_seqs : a.n_seqs;
  P.items = P.share ? static_cast<int>(units * a.Hkv) : P.own.grid;
  P.bytes = off;
  return P;
}
}  // namespace

size_t kv_attend_scratch_bytes(const KvSpec& a, int num_sms) { return attend_plan(a, num_sms, nullptr).bytes; }

int launch_kv_attend(const KvSpec& a, const void* q, void* o, float* lse, int* header, bool alone, void* scratch,
                     LaunchCtx& ctx) {
  const AttendPlan P = attend_plan(a, ctx.num_sms, static_cast<char*>(scratch));
  int* status = header + kKvHeaderWords + kKvStatusWords;
  kv::CombineParams c{};
  kv::AttendParams p{};
  p.b = kv::make_batch(a);
  if (!P.share) p.b.shared = 0;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(kv::HD)));
  p.timeout_ns = ctx.timeout_ns;
  p.skip_load = ctx.debug_skip_load;
  p.behind_append = !alone;
  int rc = TP_OK;
  if (P.share) {
    p.part = c.shared = P.shared;
    p.status = status;
    c.status_words += P.shared.grid;
    rc = P.shared.rt ? kv::launch_many(p, true, ctx, "kv_attend_shared_many")
                     : kv::launch_few<true>(p, ctx, "kv_attend_shared_few");
    if (rc) return rc;
  }
  p.part = c.own = P.own;
  p.beside = P.share;
  p.behind_append = !alone && !P.share;
  p.status = status + c.status_words;
  c.status_words += P.own.grid;
  rc = P.own.rt ? kv::launch_many(p, false, ctx, "kv_attend_many") : kv::launch_few<false>(p, ctx, "kv_attend_few");
  if (rc) return rc;
  c.b = p.b;
  c.o = p.o;
  c.lse = lse;
  c.header = header;
  c.alone = alone;
  // All eight warps of a block at work, and few rows on more blocks than one:
  // at most two blocks of 256 threads per SM before a warp has a row to itself.
  // A block goes through the rows of an item in strides: 16 blocks per SM are
  // enough, and blocks that find nothing to do cost a launch each (39000 of
  // them 30 us).
  const int64_t item_rows = static_cast<int64_t>(a.max_new) * (a.H / a.Hkv);
  const int rows = static_cast<int>(item_rows < P.own.slot_rows ? item_rows : P.own.slot_rows);
  const int64_t all = static_cast<int64_t>(a.n_tokens) * a.H;
  c.rows_per_pass = 8;
  while (c.rows_per_pass > 1 && (c.rows_per_pass >= 2 * rows || all < 2 * c.rows_per_pass * ctx.num_sms))
    c.rows_per_pass /= 2;
  const int passes = (rows + c.rows_per_pass - 1) / c.rows_per_pass, most = 16 * ctx.num_sms / P.items;
  const dim3 grid(P.items, most < 1 ? 1 : (passes < most ? passes : most));
  if (ctx.before) ctx.before(ctx.user, "kv_combine", ctx.stream);
  if (P.share)
    kv::launch_dep(kv::kv_combine_kernel<true>, grid, 256, 0, ctx.stream, c);
  else
    kv::launch_dep(kv::kv_combine_kernel<false>, grid, 256, 0, ctx.stream, c);
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  return cudaPeekAtLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

}  // namespace tpffn
