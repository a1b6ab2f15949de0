// tp_norm.cu -- what stands between two sublayers of a block: the norm of the
// sublayer's output, its gate and residual scale, the residual sum, and the norm
// before the next sublayer; forward and backward.
//
//   u = after(b),  r = x + scale gate u,  out = before(r)
// Both norms are y = (v - m) f, times w, plus c: RMS m = 0, f = 1 / sqrt(mean v^2 +
// eps); layer m = mean v, f = 1 / sqrt(mean (v - m)^2 + eps), the deviations taken
// from the mean in a second pass over the registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "tc_ptx.cuh"
#include "tp_internal.h"
#include "tpffn.h"

namespace tpffn {
namespace norm {
using tc::grid_dep_launch;
using tc::grid_dep_wait;

// Eight columns of a row.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, long long at) { v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at); }
  __device__ __forceinline__ void load(const uint4* slot) { v = slot[0]; }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ void store(void* p, long long at, const float (&a)[8]) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at) =
        make_uint4(tc::pack_bf16x2(a[0], a[1]), tc::pack_bf16x2(a[2], a[3]), tc::pack_bf16x2(a[4], a[5]), tc::pack_bf16x2(a[6], a[7]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, long long at) {
    a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
  }
  __device__ __forceinline__ void load(const uint4* slot) {
    a = *reinterpret_cast<const float4*>(slot);
    b = *reinterpret_cast<const float4*>(slot + blockDim.x);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float operator[](int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
  static __device__ __forceinline__ void store(void* p, long long at, const float (&v)[8]) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// A row belongs to `tpr` threads, a multiple of 32, thread t of them having the
// columns 8 t .. 8 t + 7; a block has blockDim / tpr row groups with R rows each.
// A thread copies its columns of the next rows into slots of its own in shared memory
// while it works on these: it waits for nobody, and no registers are held for them.
struct NormParams {
  long long n, d, per;  // per: tokens of a gate
  int tpr, after, before;
  float eps, scale, inv_d;
  const void *x, *b, *w_after, *c_after, *gate, *w_before, *c_before;
  void *r, *out;
  float4* stats;
  // backward
  const void *dr, *dout;
  void *dx, *db, *dgate;
  int want_sums;          // bit k: sums[k] is wanted: w_before, c_before, w_after, c_after
  int gate_each;          // a gate for each token: its gradient is written as it comes
  long long chunks;       // of each gate's tokens
  long long units;        // gates times chunks
  float* sums;            // [4][gridDim.x][d]
  float* gate_sums;       // [gates][chunks][d]
};

template <typename T>
__device__ __forceinline__ void fetch(uint4* slot, const void* p, long long at) {
  const T* src = static_cast<const T*>(p) + at;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(slot + i * blockDim.x)),
                 "l"(reinterpret_cast<const uint4*>(src) + i)
                 : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
// 16-byte slots of an array's row: one to a thread (bf16), or two.
template <typename T>
__host__ __device__ constexpr int slots(int threads) {
  return threads * static_cast<int>(sizeof(T)) / 2;
}

// Sums of N values over a row's threads.  `turn` alternates between two buffers, so
// that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int tpr, float (*s)[32][N], int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int d = 16; d; d >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  if (tpr == 32) return;
  const int warp = threadIdx.x >> 5, warps = tpr >> 5, first = warp / warps * warps;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) s[turn][warp][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
#pragma unroll 8
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += s[turn][first + w][k];
  turn ^= 1;
}

// The mean and factor of R rows' norms.
template <bool LAYER, int R>
__device__ __forceinline__ void row_stats(const float (&v)[R][8], bool ok, const NormParams& p, float (*s)[32][R], int& turn,
                                          float2 (&st)[R]) {
  float sum[R] = {};
#pragma unroll
  for (int k = 0; k < R; ++k) st[k].x = 0.f;
  if (LAYER) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[k] += v[k][i];
    row_sums<R>(sum, p.tpr, s, turn);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      st[k].x = sum[k] * p.inv_d;
      sum[k] = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = ok ? v[k][i] - st[k].x : 0.f;
      sum[k] = fmaf(a, a, sum[k]);
    }
  row_sums<R>(sum, p.tpr, s, turn);
#pragma unroll
  for (int k = 0; k < R; ++k) st[k].y = 1.f / sqrtf(fmaf(sum[k], p.inv_d, p.eps));
}

template <typename T, bool LAYER, int R>
__global__ void __launch_bounds__(R == 2 ? 512 : 1024) forward_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s_sum[2][32][R];
  extern __shared__ uint4 s_slots[];  // [2][x, b][R] of slots
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, groups = blockDim.x / p.tpr;
  const long long col = 8ll * t, step = static_cast<long long>(gridDim.x) * groups * R;
  const bool ok = col < p.d;
  int turn = 0, stage = 0;
  auto slot = [&](int st, int array, int k) { return s_slots + ((st * 2 + array) * R + k) * slots<T>(blockDim.x) + threadIdx.x; };
  auto fetch_rows = [&](long long row0, int st) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + group + k * groups;
      if (!ok || row >= p.n) continue;
      fetch<T>(slot(st, 0, k), p.x, row * p.d + col);
      if (p.b) fetch<T>(slot(st, 1, k), p.b, row * p.d + col);
    }
    fetch_commit();
  };
  long long row0 = static_cast<long long>(blockIdx.x) * groups * R;
  fetch_rows(row0, 0);
  Eight<T> wa, ca, wb, cb;
  if (ok && p.w_after) wa.load(p.w_after, col);
  if (ok && p.c_after) ca.load(p.c_after, col);
  if (ok && p.w_before) wb.load(p.w_before, col);
  if (ok && p.c_before) cb.load(p.c_before, col);
  for (; row0 < p.n; row0 += step, stage ^= 1) {
    float v[R][8], u[R][8];
    float2 sa[R] = {}, sb[R] = {};
    fetch_wait();
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool live = ok && row0 + group + k * groups < p.n;
      Eight<T> x, b;
      x.zero();
      b.zero();
      if (live) {
        x.load(slot(stage, 0, k));
        if (p.b) b.load(slot(stage, 1, k));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[k][i] = x[i];
        u[k][i] = b[i];
      }
    }
    if (row0 + step < p.n) fetch_rows(row0 + step, stage ^ 1);
    if (p.after) {
      row_stats<LAYER, R>(u, ok, p, s_sum, turn, sa);
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[k][i] = (u[k][i] - sa[k].x) * sa[k].y;
          if (p.w_after) u[k][i] *= wa[i];
          if (p.c_after) u[k][i] += ca[i];
        }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + group + k * groups;
      if (!ok || row >= p.n) continue;  // (columns and rows that there are not stay zero)
      if (p.b) {
        Eight<T> g;
        if (p.gate) g.load(p.gate, row / p.per * p.d + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = fmaf(p.gate ? p.scale * g[i] : p.scale, u[k][i], v[k][i]);
      }
      Eight<T>::store(p.r, row * p.d + col, v[k]);
    }
    if (p.before) row_stats<LAYER, R>(v, ok, p, s_sum, turn, sb);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + group + k * groups;
      if (!ok || row >= p.n) continue;
      if (p.before) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[k][i] = (v[k][i] - sb[k].x) * sb[k].y;
          if (p.w_before) v[k][i] *= wb[i];
          if (p.c_before) v[k][i] += cb[i];
        }
        Eight<T>::store(p.out, row * p.d + col, v[k]);
      }
      if (p.stats && t == 0) {
        float2* st = reinterpret_cast<float2*>(p.stats + row);
        if (p.after) st[0] = sa[k];
        if (p.before) st[1] = sb[k];
      }
    }
  }
}

// The tokens are cut into units, each of one gate's; a block goes through units
// and keeps the sums over its tokens of the weights' gradients, a column's in the
// registers of the thread that has the column.  SHIFT: those of the shifts too.
enum { S_WB = 0, S_CB = 1, S_WA = 2, S_CA = 3 };
enum { A_DR = 0, A_DOUT = 1, A_R = 2, A_B = 3, A_GATE = 4 };  // slots; the last with a gate for each token
// Rows of a row group at a time, and whether the next ones fit beside them.
template <typename T, int MAX_THREADS>
struct Back {
  static constexpr int R = sizeof(T) == 2 && MAX_THREADS == 512 ? 2 : 1, STAGES = sizeof(T) == 4 && MAX_THREADS == 1024 ? 1 : 2;
  static int smem(int threads, bool gate_each) { return STAGES * (gate_each ? 5 : 4) * R * slots<T>(threads) * 16; }
};
template <typename T, bool LAYER, bool SHIFT, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) backward_kernel(const __grid_constant__ NormParams p) {
  using B = Back<T, MAX_THREADS>;
  constexpr int R = B::R;
  __shared__ float s_sum[2][32][2 * R];
  extern __shared__ uint4 s_slots[];  // [STAGES][arrays][R] of slots; at the end [threads][8] floats
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, groups = blockDim.x / p.tpr;
  const long long col = 8ll * t;
  const bool ok = col < p.d;
  const int arrays = p.gate_each ? 5 : 4;
  int turn = 0, stage = 0;
  auto slot = [&](int st, int array, int k) { return s_slots + ((st * arrays + array) * R + k) * slots<T>(blockDim.x) + threadIdx.x; };
  // Rows of the block's units, a few at a time.
  struct Place {
    long long unit, row, to;
  };
  auto enter = [&](Place& at) {
    if (at.unit >= p.units) return;
    const long long gi = at.unit / p.chunks, c = at.unit - gi * p.chunks;
    at.row = gi * p.per + c * p.per / p.chunks;
    at.to = gi * p.per + (c + 1) * p.per / p.chunks;
  };
  auto fetch_rows = [&](const Place& at, int st) {
    if (at.unit < p.units) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const long long row = at.row + group + k * groups, from = row * p.d + col;
        if (!ok || row >= at.to) continue;
        if (p.dr) fetch<T>(slot(st, A_DR, k), p.dr, from);
        if (p.before) {
          fetch<T>(slot(st, A_DOUT, k), p.dout, from);
          fetch<T>(slot(st, A_R, k), p.r, from);
        }
        if (p.b) fetch<T>(slot(st, A_B, k), p.b, from);
        if (p.gate_each) fetch<T>(slot(st, A_GATE, k), p.gate, from);
      }
    }
    fetch_commit();
  };
  Place here{blockIdx.x, 0, 0};
  enter(here);
  if (B::STAGES == 2) fetch_rows(here, 0);
  Eight<T> wa, ca, wb, gate;
  wa.zero();
  ca.zero();
  wb.zero();
  gate.zero();
  if (ok && p.w_after) wa.load(p.w_after, col);
  if (ok && p.c_after) ca.load(p.c_after, col);
  if (ok && p.w_before) wb.load(p.w_before, col);
  if (ok && p.gate && !p.gate_each && here.unit < p.units) gate.load(p.gate, here.unit / p.chunks * p.d + col);
  float sums[4][8] = {}, gsum[8] = {};
  // A column sum over the block's row groups, then to `write`.
  auto flush = [&](float (&a)[8], float* s_cols, auto&& write) {
    if (groups > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) s_cols[threadIdx.x * 8 + i] = a[i];
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < groups; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] += s_cols[(g * p.tpr + t) * 8 + i];
    }
    if (group == 0 && ok) write(a);
  };
  float* s_cols = reinterpret_cast<float*>(s_slots + B::STAGES * arrays * R * slots<T>(blockDim.x));
  auto to_floats = [](float* at, const float (&a)[8]) {
    reinterpret_cast<float4*>(at)[0] = make_float4(a[0], a[1], a[2], a[3]);
    reinterpret_cast<float4*>(at)[1] = make_float4(a[4], a[5], a[6], a[7]);
  };
  while (here.unit < p.units) {
    Place next = here;
    next.row += groups * R;
    const bool ends = next.row >= next.to;
    if (ends) {
      next.unit += gridDim.x;
      enter(next);
    }
    if (B::STAGES == 1) fetch_rows(here, 0);
    fetch_wait();
    if (B::STAGES == 2) fetch_rows(next, stage ^ 1);
    float g[R][8], s[2 * R];
    float4 st[R];
    bool live[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = here.row + group + k * groups;
      live[k] = ok && row < here.to;
      st[k] = live[k] && p.stats ? p.stats[row] : make_float4(0.f, 0.f, 0.f, 0.f);
      Eight<T> dr;
      dr.zero();
      if (live[k] && p.dr) dr.load(slot(stage, A_DR, k));
#pragma unroll
      for (int i = 0; i < 8; ++i) g[k][i] = dr[i];
      s[2 * k] = s[2 * k + 1] = 0.f;
    }
    if (p.before) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (!live[k]) continue;
        Eight<T> r, dout;
        r.load(slot(stage, A_R, k));
        dout.load(slot(stage, A_DOUT, k));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = (r[i] - st[k].z) * st[k].w, d = dout[i], dy = p.w_before ? d * wb[i] : d;
          s[2 * k] = fmaf(dy, y, s[2 * k]);
          s[2 * k + 1] += dy;
          sums[S_WB][i] = fmaf(d, y, sums[S_WB][i]);
          if (SHIFT) sums[S_CB][i] += d;
        }
      }
      row_sums<2 * R>(s, p.tpr, s_sum, turn);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (!live[k]) continue;
        const float m1 = s[2 * k] * p.inv_d, m0 = LAYER ? s[2 * k + 1] * p.inv_d : 0.f;
        Eight<T> r, dout;
        r.load(slot(stage, A_R, k));
        dout.load(slot(stage, A_DOUT, k));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = (r[i] - st[k].z) * st[k].w, d = dout[i], dy = p.w_before ? d * wb[i] : d;
          g[k][i] = fmaf(st[k].w, dy - fmaf(y, m1, m0), g[k][i]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long at = (here.row + group + k * groups) * p.d + col;
      s[2 * k] = s[2 * k + 1] = 0.f;
      if (!live[k]) continue;
      if (p.dx) Eight<T>::store(p.dx, at, g[k]);
      Eight<T> b, ge = gate;
      b.zero();
      if (p.b) b.load(slot(stage, A_B, k));
      if (p.gate_each) ge.load(slot(stage, A_GATE, k));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = p.after ? (b[i] - st[k].x) * st[k].y : b[i], sg = p.scale * g[k][i];
        if (p.dgate) {
          const float dg = sg * fmaf(y, p.w_after ? wa[i] : 1.f, ca[i]);
          gsum[i] = p.gate_each ? dg : gsum[i] + dg;
        }
        float du = p.gate ? sg * ge[i] : sg;
        if (p.after) {
          sums[S_WA][i] = fmaf(du, y, sums[S_WA][i]);
          if (SHIFT) sums[S_CA][i] += du;
          if (p.w_after) du *= wa[i];
          s[2 * k] = fmaf(du, y, s[2 * k]);
          s[2 * k + 1] += du;
        }
        g[k][i] = du;
      }
      if (p.gate_each && p.dgate) Eight<T>::store(p.dgate, at, gsum);
    }
    if (p.after) {
      row_sums<2 * R>(s, p.tpr, s_sum, turn);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (!live[k]) continue;
        const float m1 = s[2 * k] * p.inv_d, m0 = LAYER ? s[2 * k + 1] * p.inv_d : 0.f;
        Eight<T> b;
        b.load(slot(stage, A_B, k));
#pragma unroll
        for (int i = 0; i < 8; ++i) g[k][i] = st[k].y * (g[k][i] - fmaf((b[i] - st[k].x) * st[k].y, m1, m0));
      }
    }
    if (p.db)
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (live[k]) Eight<T>::store(p.db, (here.row + group + k * groups) * p.d + col, g[k]);
    if (ends && p.gate && !p.gate_each) {
      const long long gi = here.unit / p.chunks;
      if (p.dgate) {
        flush(gsum, s_cols, [&](const float (&a)[8]) {
          if (p.chunks == 1)
            Eight<T>::store(p.dgate, gi * p.d + col, a);
          else
            to_floats(p.gate_sums + here.unit * p.d + col, a);
        });
#pragma unroll
        for (int i = 0; i < 8; ++i) gsum[i] = 0.f;
      }
      if (ok && next.unit < p.units) gate.load(p.gate, next.unit / p.chunks * p.d + col);
    }
    here = next;
    if (B::STAGES == 2) stage ^= 1;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (p.want_sums >> k & 1)
      flush(sums[k], s_cols, [&](const float (&a)[8]) {
        to_floats(p.sums + (static_cast<long long>(k) * gridDim.x + blockIdx.x) * p.d + col, a);
      });
}

// Column sums of up to four [parts][d] and, beside them, of [gates] of them; a block
// takes 32 columns of four and its eight warps every eighth part.
struct SumParams {
  const float* from[5];
  void* to[5];
  long long parts[5], d, gates;
};
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const __grid_constant__ SumParams p) {
  __shared__ float4 s[8][32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long which = blockIdx.y < 4 ? blockIdx.y : 4, gate = blockIdx.y < 4 ? 0 : blockIdx.y - 4;
  if (!p.to[which]) return;
  const long long parts = p.parts[which], at = (static_cast<long long>(blockIdx.x) * 32 + lane) * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at < p.d) {
    const float* from = p.from[which] + gate * parts * p.d + at;
#pragma unroll 4
    for (long long i = warp; i < parts; i += 8) {
      const float4 v = *reinterpret_cast<const float4*>(from + i * p.d);
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp || at >= p.d) return;
  for (int w = 1; w < 8; ++w) {
    a.x += s[w][lane].x;
    a.y += s[w][lane].y;
    a.z += s[w][lane].z;
    a.w += s[w][lane].w;
  }
  T* to = static_cast<T*>(p.to[which]) + gate * p.d + at;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(to) = make_uint2(tc::pack_bf16x2(a.x, a.y), tc::pack_bf16x2(a.z, a.w));
  else
    *reinterpret_cast<float4*>(to) = a;
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
int launched() { return cudaPeekAtLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA; }

// Threads to a row, row groups and threads of a block.
struct Shape {
  int tpr, groups, threads;
};
Shape shape_of(int64_t d, int64_t n, int num_sms) {
  Shape s;
  s.tpr = static_cast<int>((d / 8 + 31) / 32 * 32);
  s.groups = std::max(512 / s.tpr, 1);
  while (s.groups > 1 && (n + s.groups - 1) / s.groups < num_sms) s.groups /= 2;  // few tokens: on all SMs
  s.threads = s.groups * s.tpr;
  return s;
}

// How the backward's tokens are cut: `blocks` blocks, `chunks` of each gate's tokens.
struct Plan {
  int64_t blocks, chunks, gates, per, units;
  bool each;
};
Plan plan_of(const NormSpec& a, int num_sms) {
  Plan p;
  p.each = a.n_gates == a.n && a.n > 1;
  p.gates = a.n_gates && !p.each ? a.n_gates : 1;
  p.per = a.n / p.gates;
  const Shape s = shape_of(a.d, a.n, num_sms);
  const int64_t most = num_sms * std::max(1, 512 / s.threads);
  p.chunks = std::min<int64_t>(std::max<int64_t>(most / p.gates, 1), (p.per + s.groups - 1) / s.groups);
  p.units = p.gates * p.chunks;
  p.blocks = std::min<int64_t>(p.units, most);
  return p;
}

NormParams params_of(const NormSpec& a, const Shape& s) {
  NormParams p{};
  p.n = a.n;
  p.d = a.d;
  p.per = a.n_gates ? a.n / a.n_gates : a.n;
  p.tpr = s.tpr;
  p.after = a.after;
  p.before = a.before;
  p.eps = a.eps;
  p.scale = a.scale;
  p.inv_d = 1.f / static_cast<float>(a.d);
  p.b = a.b;
  p.w_after = a.w_after;
  p.c_after = a.c_after;
  p.gate = a.gate;
  p.w_before = a.w_before;
  p.c_before = a.c_before;
  p.stats = reinterpret_cast<float4*>(a.stats);
  return p;
}

// Raises a kernel's shared-memory limit, once for a device.
template <auto KERNEL>
int allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TP_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (bytes > 48 * 1024 && !(done.load() & bit)) {
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess) return TP_ERR_CUDA;
    done.fetch_or(bit);
  }
  return TP_OK;
}

template <typename T, bool LAYER, int R>
int launch_forward_inst(const NormParams& p, const Shape& s, int num_sms, cudaStream_t st) {
  const int smem = 2 * 2 * R * slots<T>(s.threads) * 16, rows = s.groups * R;
  if (int rc = allow_smem<forward_kernel<T, LAYER, R>>(smem)) return rc;
  const int64_t blocks = (p.n + rows - 1) / rows, most = static_cast<int64_t>(num_sms) * std::max(1, 1024 / s.threads);
  launch_dep(forward_kernel<T, LAYER, R>, dim3(static_cast<unsigned>(std::min(blocks, most))), s.threads, smem, st, p);
  return launched();
}
// Two rows to a thread at a time where there are enough for all SMs.
template <typename T, bool LAYER>
int launch_forward(const NormParams& p, const Shape& s, int num_sms, cudaStream_t st) {
  if (p.n >= 4ll * num_sms * s.groups && s.threads <= 512) return launch_forward_inst<T, LAYER, 2>(p, s, num_sms, st);
  return launch_forward_inst<T, LAYER, 1>(p, s, num_sms, st);
}
template <typename T, bool LAYER, bool SHIFT, int MAX_THREADS>
int launch_backward_inst(const NormParams& p, const Shape& s, unsigned grid, cudaStream_t st) {
  const int smem = Back<T, MAX_THREADS>::smem(s.threads, p.gate_each) + (s.groups > 1 ? s.threads * 32 : 0);
  if (int rc = allow_smem<backward_kernel<T, LAYER, SHIFT, MAX_THREADS>>(smem)) return rc;
  launch_dep(backward_kernel<T, LAYER, SHIFT, MAX_THREADS>, dim3(grid), s.threads, smem, st, p);
  return launched();
}
// Up to 512 threads a thread may have 128 registers, which the sums need.
template <typename T, bool LAYER>
int launch_backward(const NormParams& p, const Shape& s, unsigned grid, cudaStream_t st) {
  const bool shift = p.want_sums & (1 << S_CB | 1 << S_CA);
  if (s.threads <= 512)
    return shift ? launch_backward_inst<T, LAYER, true, 512>(p, s, grid, st) : launch_backward_inst<T, LAYER, false, 512>(p, s, grid, st);
  return shift ? launch_backward_inst<T, LAYER, true, 1024>(p, s, grid, st) : launch_backward_inst<T, LAYER, false, 1024>(p, s, grid, st);
}
}  // namespace norm

int launch_norm_fwd(const NormSpec& a, int num_sms, cudaStream_t st) {
  using namespace norm;
  const Shape s = shape_of(a.d, a.n, num_sms);
  NormParams p = params_of(a, s);
  p.x = a.x;
  p.r = a.r;
  p.out = a.out;
  if (a.f32) return a.layer ? launch_forward<float, true>(p, s, num_sms, st) : launch_forward<float, false>(p, s, num_sms, st);
  return a.layer ? launch_forward<__nv_bfloat16, true>(p, s, num_sms, st) : launch_forward<__nv_bfloat16, false>(p, s, num_sms, st);
}

size_t norm_workspace_bytes(const NormSpec& a, int num_sms) {
  const norm::Plan p = norm::plan_of(a, num_sms);
  return static_cast<size_t>(a.d) * sizeof(float) * (4 * p.blocks + (p.chunks > 1 && a.n_gates && !p.each ? p.units : 0));
}

int launch_norm_bwd(const NormSpec& a, void* workspace, int num_sms, cudaStream_t st) {
  using namespace norm;
  const Shape s = shape_of(a.d, a.n, num_sms);
  const Plan c = plan_of(a, num_sms);
  NormParams p = params_of(a, s);
  p.r = const_cast<void*>(a.r_in);
  p.per = c.per;
  p.dr = a.dr;
  p.dout = a.dout;
  p.dx = a.dx;
  p.db = a.db;
  p.dgate = a.dgate;
  p.gate_each = c.each;
  p.chunks = c.chunks;
  p.units = c.units;
  p.sums = static_cast<float*>(workspace);
  p.gate_sums = p.sums + 4 * c.blocks * a.d;
  void* const to[4] = {a.dw_before, a.dc_before, a.dw_after, a.dc_after};
  SumParams q{};
  for (int k = 0; k < 4; ++k) {
    p.want_sums |= (to[k] != nullptr) << k;
    q.from[k] = p.sums + k * c.blocks * a.d;
    q.to[k] = to[k];
    q.parts[k] = c.blocks;
  }
  const unsigned grid = static_cast<unsigned>(c.blocks);
  const int rc = a.f32 ? (a.layer ? launch_backward<float, true>(p, s, grid, st) : launch_backward<float, false>(p, s, grid, st))
                       : (a.layer ? launch_backward<__nv_bfloat16, true>(p, s, grid, st)
                                  : launch_backward<__nv_bfloat16, false>(p, s, grid, st));
  if (rc) return rc;
  q.d = a.d;
  if (a.dgate && !c.each && c.chunks > 1) {
    q.from[4] = p.gate_sums;
    q.to[4] = a.dgate;
    q.parts[4] = c.chunks;
    q.gates = c.gates;
  }
  if (p.want_sums || q.gates) {
    const dim3 blocks(static_cast<unsigned>((a.d + 127) / 128), static_cast<unsigned>(4 + q.gates));
    if (a.f32)
      launch_dep(sum_parts_kernel<float>, blocks, 256, 0, st, q);
    else
      launch_dep(sum_parts_kernel<__nv_bfloat16>, blocks, 256, 0, st, q);
  }
  return launched();
}

}  // namespace tpffn
