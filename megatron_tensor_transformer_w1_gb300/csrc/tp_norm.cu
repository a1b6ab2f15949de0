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

// Pairs of 32-bit numbers, two operations to an instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint64_t both(float v) { return pair(v, v); }
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float total(uint64_t v) {
  const float2 r = halves(v);
  return r.x + r.y;
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

// Eight columns of a row, as four pairs.
using Pairs = uint64_t[4];
__device__ __forceinline__ void fill(Pairs& a, float v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = both(v);
}
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  static __device__ __forceinline__ void open(Pairs& a, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ void load(Pairs& a, const void* p, long long at, int) {
    open(a, *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at));
  }
  static __device__ __forceinline__ void load_slot(Pairs& a, uint32_t slot) { open(a, ld_shared(slot)); }
  static __device__ __forceinline__ void store(void* p, long long bytes, const Pairs& a, int) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = halves(a[i]);
      w[i] = tc::pack_bf16x2(v.x, v.y);
    }
    *reinterpret_cast<uint4*>(static_cast<char*>(p) + bytes) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Eight<float> {
  static __device__ __forceinline__ void open(Pairs& a, float4 v, float4 w) {
    a[0] = pair(v.x, v.y);
    a[1] = pair(v.z, v.w);
    a[2] = pair(w.x, w.y);
    a[3] = pair(w.z, w.w);
  }
  static __device__ __forceinline__ void load(Pairs& a, const void* p, long long at, int apart) {
    const float* src = static_cast<const float*>(p) + at;
    open(a, *reinterpret_cast<const float4*>(src), *reinterpret_cast<const float4*>(src + apart));
  }
  static __device__ __forceinline__ void load_slot(Pairs& a, uint32_t slot) {
    const uint4 v = ld_shared(slot), w = ld_shared(slot + blockDim.x * 16);
    open(a, make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)),
         make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)));
  }
  static __device__ __forceinline__ void store(void* p, long long bytes, const Pairs& a, int apart) {
    float* to = reinterpret_cast<float*>(static_cast<char*>(p) + bytes);
    const float2 v = halves(a[0]), w = halves(a[1]), x = halves(a[2]), y = halves(a[3]);
    *reinterpret_cast<float4*>(to) = make_float4(v.x, v.y, w.x, w.y);
    *reinterpret_cast<float4*>(to + apart) = make_float4(x.x, x.y, y.x, y.y);
  }
};

// A row belongs to `tpr` threads, a multiple of 32, a thread having eight of the
// 256 columns of its warp: in bf16 one behind the other, in 32 bits two fours of which a
// warp's lie one behind the other (a warp's 16-byte pieces side by side: with eight
// columns in a row a store fills half of every sector, and the backward pass of 4104
// tokens of 1160 took 44 us); a block has blockDim / tpr row groups.  A thread copies its
// columns of the next rows into slots of its own in shared memory while it works on
// this one (`stages` rows in all): it waits for nobody, and no registers are held for
// them.
template <typename T>
__device__ __forceinline__ int columns_apart(int t, int d) {  // from a thread's first four to its second
  const int left = d - (t >> 5) * 256;
  return sizeof(T) == 2 || left <= 0 ? 4 : min(left, 256) / 2;
}
template <typename T>
__device__ __forceinline__ int first_column(int t) {
  return sizeof(T) == 2 ? 8 * t : (t >> 5) * 256 + (t & 31) * 4;
}
struct NormParams {
  int n, d, per;          // per: tokens of a gate
  int tpr, after, before, stages;
  float eps, scale, inv_d;
  const void *x, *b, *w_after, *c_after, *gate, *w_before, *c_before;
  void *r, *out;
  float4* stats;
  // backward
  const void *dr, *dout;
  void *dx, *db, *dgate;
  int want_sums;          // bit k: sums[k] is wanted: w_before, c_before, w_after, c_after
  int gate_each;          // a gate for each token: its gradient is written as it comes
  int chunks;             // of each gate's tokens
  int units;              // gates times chunks
  float* sums;            // [4][gridDim.x][d]
  float* gate_sums;       // [gates][chunks][d]
};

// Not `valid`: the slot gets zeros, nothing is read.
template <typename T>
__device__ __forceinline__ void fetch(uint32_t slot, const void* p, long long bytes, int apart, bool valid = true) {
  const char* src = static_cast<const char*>(p) + bytes;
  const int n = valid ? 16 : 0;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + i * blockDim.x * 16), "l"(src + i * apart * 4), "r"(n) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The oldest of stages - 1 groups, one for each row ahead, has landed (or, of one
// stage, all have).
__device__ __forceinline__ void fetch_wait(int stages) {
  if (stages >= 4)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (stages == 3)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}
// 16-byte slots of an array's row: one to a thread (bf16), or two.
template <typename T>
__host__ __device__ constexpr int slots(int threads) {
  return threads * static_cast<int>(sizeof(T)) / 2;
}

// Eight columns of a weight for all rows: as pairs, or, where registers are short, as
// they lie.
template <typename T, bool SHORT>
struct Held {
  Pairs a;
  __device__ __forceinline__ void set(float v) { fill(a, v); }
  __device__ __forceinline__ void load(const void* p, long long at, int apart) { Eight<T>::load(a, p, at, apart); }
  __device__ __forceinline__ void load_slot(uint32_t slot) { Eight<T>::load_slot(a, slot); }
  __device__ __forceinline__ uint64_t operator[](int i) const { return a[i]; }
};
template <>
struct Held<__nv_bfloat16, true> {
  uint32_t w[4];
  __device__ __forceinline__ void set(float v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = tc::pack_bf16x2(v, v);
  }
  __device__ __forceinline__ void put(uint4 v) {
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
  __device__ __forceinline__ void load(const void* p, long long at, int) { put(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at)); }
  __device__ __forceinline__ void load_slot(uint32_t slot) { put(ld_shared(slot)); }
  __device__ __forceinline__ uint64_t operator[](int i) const { return pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)); }
};

// Sums of N values over a row's threads.  `turn` alternates between two buffers, so
// that one barrier a sum is enough.
struct Group {
  int warps, first;  // of a row, the first of this thread's row
  __device__ __forceinline__ explicit Group(int tpr) : warps(tpr >> 5), first((threadIdx.x >> 5) / (tpr >> 5) * (tpr >> 5)) {}
};
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], const Group& G, float (*s)[32][N], int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int d = 16; d; d >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  if (G.warps == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) s[turn][warp][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    // (up to 16 warps: both halves of a warp have the same)
    const int at = G.warps > 16 ? lane : lane & 15;
    v[k] = at < G.warps ? s[turn][G.first + at][k] : 0.f;
    if (G.warps > 16) v[k] += __shfl_xor_sync(0xffffffffu, v[k], 16);
#pragma unroll
    for (int d = 8; d; d >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  }
  turn ^= 1;
}

// The mean and factor of a row's norm.
template <bool LAYER>
__device__ __forceinline__ float2 row_stats(const Pairs& v, bool ok, const NormParams& p, const Group& G, float (*s)[32][1], int& turn) {
  float2 st = make_float2(0.f, 0.f);
  float sum[1];
  if (LAYER) {
    sum[0] = total(add2(add2(v[0], v[1]), add2(v[2], v[3])));
    row_sums<1>(sum, G, s, turn);
    st.x = sum[0] * p.inv_d;
  }
  uint64_t q = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t a = LAYER ? add2(v[i], both(-st.x)) : v[i];
    q = fma2(a, a, q);
  }
  sum[0] = ok ? total(q) : 0.f;
  row_sums<1>(sum, G, s, turn);
  st.y = rsqrtf(fmaf(sum[0], p.inv_d, p.eps));
  return st;
}
// (v - mean) * factor
template <bool LAYER>
__device__ __forceinline__ uint64_t unit(uint64_t v, uint64_t mean, uint64_t factor) {
  return mul2(LAYER ? add2(v, mean) : v, factor);  // (mean: its negative)
}

// Bound by memory: 8192 tokens of 4096 in bf16 with both norms and a gate, 268 MB, in 44
// us, 6.1 TB/s (without the copies ahead 84).  SHIFT: there are shifts.
template <typename T, bool LAYER, bool SHIFT>
__global__ void __launch_bounds__(1024) forward_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s_sum[2][32][1];
  extern __shared__ uint4 s_slots[];  // [stages][x, b] of slots
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, groups = blockDim.x / p.tpr;
  const Group G(p.tpr);
  const bool ok = 8 * t < p.d;
  const int apart = columns_apart<T>(t, p.d), col = first_column<T>(t), step = gridDim.x * groups;
  const long long step_bytes = static_cast<long long>(step) * p.d * sizeof(T);
  const uint32_t array = slots<T>(blockDim.x) * 16, ring = tc::smem_u32(s_slots) + threadIdx.x * 16;
  int turn = 0, row = blockIdx.x * groups + group, gate_until = 0, ahead = row;
  long long bytes = (static_cast<long long>(row) * p.d + col) * sizeof(T), ahead_bytes = bytes;
  uint32_t stage = ring, ahead_stage = ring;
  const uint32_t ring_end = ring + p.stages * 2 * array;
  auto fetch_row = [&] {
    if (ok && ahead < p.n) {
      fetch<T>(ahead_stage, p.x, ahead_bytes, apart);
      if (p.b) fetch<T>(ahead_stage + array, p.b, ahead_bytes, apart);
    }
    fetch_commit();
    ahead += step;
    ahead_bytes += step_bytes;
    ahead_stage += 2 * array;
    if (ahead_stage == ring_end) ahead_stage = ring;
  };
  for (int i = 1; i < p.stages; ++i) fetch_row();
  Pairs k1, k0, w, c;  // scale gate w_after, scale gate c_after, w_before, c_before
  fill(k1, 0.f);
  fill(k0, 0.f);
  fill(w, 1.f);
  fill(c, 0.f);
  if (ok && p.w_before) Eight<T>::load(w, p.w_before, col, apart);
  if (SHIFT && ok && p.c_before) Eight<T>::load(c, p.c_before, col, apart);
  for (; row - group < p.n; row += step, bytes += step_bytes) {
    const bool live = ok && row < p.n;
    if (p.b && live && row >= gate_until) {
      const int gate_at = p.gate ? row / p.per : 0;
      gate_until = p.gate ? (gate_at + 1) * p.per : p.n;
      fill(k1, 1.f);
      if (p.gate) Eight<T>::load(k1, p.gate, static_cast<long long>(gate_at) * p.d + col, apart);
#pragma unroll
      for (int i = 0; i < 4; ++i) k1[i] = mul2(k1[i], both(p.scale));
      if (SHIFT && p.c_after) {
        Eight<T>::load(k0, p.c_after, col, apart);
#pragma unroll
        for (int i = 0; i < 4; ++i) k0[i] = mul2(k0[i], k1[i]);
      }
      if (p.w_after) {
        Pairs wa;
        Eight<T>::load(wa, p.w_after, col, apart);
#pragma unroll
        for (int i = 0; i < 4; ++i) k1[i] = mul2(k1[i], wa[i]);
      }
    }
    Pairs v, u;
    fill(v, 0.f);
    fill(u, 0.f);
    fetch_wait(p.stages);
    if (live) {
      Eight<T>::load_slot(v, stage);
      if (p.b) Eight<T>::load_slot(u, stage + array);
    }
    stage += 2 * array;
    if (stage == ring_end) stage = ring;
    fetch_row();  // (into the slots of the row before)
    float2 sa = make_float2(0.f, 1.f), sb = make_float2(0.f, 0.f);
    if (p.after) sa = row_stats<LAYER>(u, ok, p, G, s_sum, turn);
    if (live && p.b) {  // (columns and rows that there are not stay zero)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fma2(unit<LAYER>(u[i], both(-sa.x), both(sa.y)), k1[i], SHIFT ? add2(v[i], k0[i]) : v[i]);
    }
    if (live) Eight<T>::store(p.r, bytes, v, apart);
    if (p.before) {
      sb = row_stats<LAYER>(v, ok, p, G, s_sum, turn);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t y = unit<LAYER>(v[i], both(-sb.x), both(sb.y));
        v[i] = SHIFT ? fma2(y, w[i], c[i]) : mul2(y, w[i]);
      }
      if (live) Eight<T>::store(p.out, bytes, v, apart);
    }
    if (p.stats && live && t == 0) {
      float2* st = reinterpret_cast<float2*>(p.stats + row);
      if (p.after) st[0] = sa;
      if (p.before) st[1] = sb;
    }
  }
}

// The tokens are cut into units, each of one gate's; a block goes through units
// and keeps the sums over its tokens of the weights' gradients, a column's in the
// registers of the thread that has the column.  SHIFT: those of the shifts too.
// Eight columns' sums, weights and values take 128 registers, which leaves 512 threads
// to an SM: in bf16 8192 tokens of 4096, 403 MB, take 92 us, 4.4 TB/s, the issue slots 54 %
// full, a row's two sums over its threads one behind the other; 4104 tokens of 1160 in
// 32 bits with layer norms, 114 MB, 40 us.  (Two columns to a thread more: spills, 145 us; its
// own instance for every combination of norms and gates: no faster.)
// Rows of more than 4096 columns need more than 512 threads and have 64 registers
// each, so that sums, weights and values are spilled (590 to 1380 bytes a thread; the other
// instances with shifts 20 to 40): 8192 tokens of 5120 in bf16, 503 MB, 263 us, of 8192, 805 MB,
// 334 us, 2.4 TB/s.
enum { S_WB = 0, S_CB = 1, S_WA = 2, S_CA = 3 };
enum { A_DR = 0, A_DOUT = 1, A_R = 2, A_B = 3, A_GATE = 4 };  // slots; the last with a gate for each token
template <typename T, bool LAYER, bool SHIFT, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) backward_kernel(const __grid_constant__ NormParams p) {
  constexpr int N = LAYER ? 2 : 1;  // sums of a row
  __shared__ float s_sum[2][32][N];
  extern __shared__ uint4 s_slots[];  // [stages][arrays] of slots; at the end [threads][8] floats
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, groups = blockDim.x / p.tpr;
  const Group G(p.tpr);
  const bool ok = 8 * t < p.d;
  const int apart = columns_apart<T>(t, p.d), col = first_column<T>(t);
  const long long step_bytes = static_cast<long long>(groups) * p.d * sizeof(T);
  const uint32_t array = slots<T>(blockDim.x) * 16, row_slots = (p.gate_each ? 5 : 4) * array;
  const uint32_t ring = tc::smem_u32(s_slots) + threadIdx.x * 16, ring_end = ring + p.stages * row_slots;
  int turn = 0;
  // Rows of the block's units, one to a row group at a time.
  struct Place {
    int unit, row, to;
    long long bytes;
    uint32_t slot;
  };
  auto enter = [&](Place& at) {
    if (at.unit >= p.units) return;
    const int gi = at.unit / p.chunks, c = at.unit - gi * p.chunks;
    at.row = gi * p.per + static_cast<int>(static_cast<long long>(c) * p.per / p.chunks) + group;
    at.to = gi * p.per + static_cast<int>(static_cast<long long>(c + 1) * p.per / p.chunks);
    at.bytes = (static_cast<long long>(at.row) * p.d + col) * sizeof(T);
  };
  auto go_on = [&](Place& at) {  // whether that ended a unit
    at.slot += row_slots;
    if (at.slot == ring_end) at.slot = ring;
    at.row += groups;
    at.bytes += step_bytes;
    if (at.row - group < at.to) return false;
    at.unit += gridDim.x;
    enter(at);
    return true;
  };
  // What there is not is zeros in the slots, columns and rows among it: they add
  // nothing to any sum.
  const void* some = p.r ? p.r : p.stats ? static_cast<const void*>(p.stats) : p.sums;
  auto fetch_row = [&](const Place& at) {
    const bool there = ok && at.unit < p.units && at.row < at.to;
    auto array_of = [&](int a, const void* from) {
      const bool valid = there && from;
      fetch<T>(at.slot + a * array, valid ? from : some, valid ? at.bytes : 0, apart, valid);
    };
    array_of(A_DR, p.dr);
    if (p.before) {
      array_of(A_DOUT, p.dout);
      array_of(A_R, p.r);
    }
    array_of(A_B, p.b);
    if (p.gate_each) array_of(A_GATE, p.gate);
    fetch_commit();
  };
  Place here{static_cast<int>(blockIdx.x), 0, 0, 0, ring};
  enter(here);
  Place ahead = here;
  for (int i = 1; i < p.stages; ++i) {
    fetch_row(ahead);
    if (ahead.unit < p.units) go_on(ahead);
  }
  Held<T, MAX_THREADS == 1024> wa, ca, wb, gate;
  wa.set(1.f);
  ca.set(0.f);
  wb.set(1.f);
  gate.set(1.f);
  if (ok && p.w_after) wa.load(p.w_after, col, apart);
  if (ok && p.c_after) ca.load(p.c_after, col, apart);
  if (ok && p.w_before) wb.load(p.w_before, col, apart);
  if (ok && p.gate && !p.gate_each && here.unit < p.units) gate.load(p.gate, static_cast<long long>(here.unit / p.chunks) * p.d + col, apart);
  Pairs sums[4] = {}, gsum = {};
  // A column sum over the block's row groups, then to `write`.
  auto flush = [&](Pairs& a, float* s_cols, auto&& write) {
    if (groups > 1) {
      float4* mine = reinterpret_cast<float4*>(s_cols) + threadIdx.x * 2;
      __syncthreads();
      const float2 v = halves(a[0]), w = halves(a[1]), x = halves(a[2]), y = halves(a[3]);
      mine[0] = make_float4(v.x, v.y, w.x, w.y);
      mine[1] = make_float4(x.x, x.y, y.x, y.y);
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < groups; ++g) {
          const float4 lo = mine[g * p.tpr * 2], hi = mine[g * p.tpr * 2 + 1];
          a[0] = add2(a[0], pair(lo.x, lo.y));
          a[1] = add2(a[1], pair(lo.z, lo.w));
          a[2] = add2(a[2], pair(hi.x, hi.y));
          a[3] = add2(a[3], pair(hi.z, hi.w));
        }
    }
    if (group == 0 && ok) write(a);
  };
  float* s_cols = reinterpret_cast<float*>(reinterpret_cast<char*>(s_slots) + p.stages * row_slots);
  // A row's statistics are on their way while the row before it is worked on.
  auto stats_of = [&](const Place& at) {
    return ok && p.stats && at.unit < p.units && at.row < at.to ? p.stats[at.row] : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 st_next = stats_of(here);
  while (here.unit < p.units) {
    Place next = here;
    const bool ends = go_on(next);
    if (p.stages == 1) fetch_row(here);
    const bool live = ok && here.row < here.to;
    const float4 st = st_next;
    st_next = stats_of(next);
    fetch_wait(p.stages);
    if (p.stages > 1) {  // (into the slots of the row before)
      fetch_row(ahead);
      if (ahead.unit < p.units) go_on(ahead);
    }
    Pairs g;
    Eight<T>::load_slot(g, here.slot + A_DR * array);
    if (p.before) {
      Pairs y, dy;
      Eight<T>::load_slot(y, here.slot + A_R * array);
      Eight<T>::load_slot(dy, here.slot + A_DOUT * array);
      uint64_t s0 = 0, s1 = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = unit<LAYER>(y[i], both(-st.z), both(st.w));
        sums[S_WB][i] = fma2(dy[i], y[i], sums[S_WB][i]);
        if (SHIFT) sums[S_CB][i] = add2(sums[S_CB][i], dy[i]);
        dy[i] = mul2(dy[i], wb[i]);
        s0 = fma2(dy[i], y[i], s0);
        if (LAYER) s1 = add2(s1, dy[i]);
      }
      float s[N];
      s[0] = total(s0);
      if (LAYER) s[N - 1] = total(s1);
      row_sums<N>(s, G, s_sum, turn);
      const uint64_t m1 = both(-s[0] * p.inv_d), m0 = both(-s[N - 1] * p.inv_d);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = fma2(fma2(y[i], m1, LAYER ? add2(dy[i], m0) : dy[i]), both(st.w), g[i]);
    }
    if (p.dx && live) Eight<T>::store(p.dx, here.bytes, g, apart);
    if (p.b || p.db) {  // (of all threads)
      Pairs y;
      Eight<T>::load_slot(y, here.slot + A_B * array);
      if (p.gate_each) gate.load_slot(here.slot + A_GATE * array);
      uint64_t s0 = 0, s1 = 0;
      if (p.after)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = unit<LAYER>(y[i], both(-st.x), both(st.y));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t sg = mul2(ok ? g[i] : 0, both(p.scale));  // (a layer norm's gradient is not zero behind the last column)
        const uint64_t u = SHIFT ? fma2(y[i], wa[i], ca[i]) : mul2(y[i], wa[i]);
        gsum[i] = p.gate_each ? mul2(sg, u) : fma2(sg, u, gsum[i]);
        g[i] = mul2(sg, gate[i]);
        sums[S_WA][i] = fma2(g[i], y[i], sums[S_WA][i]);
        if (SHIFT) sums[S_CA][i] = add2(sums[S_CA][i], g[i]);
        g[i] = mul2(g[i], wa[i]);
        s0 = fma2(g[i], y[i], s0);
        if (LAYER) s1 = add2(s1, g[i]);
      }
      if (p.gate_each && p.dgate && live) Eight<T>::store(p.dgate, here.bytes, gsum, apart);
      if (p.after) {
        float s[N];
        s[0] = total(s0);
        if (LAYER) s[N - 1] = total(s1);
        row_sums<N>(s, G, s_sum, turn);
        const uint64_t m1 = both(-s[0] * p.inv_d), m0 = both(-s[N - 1] * p.inv_d);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = mul2(fma2(y[i], m1, LAYER ? add2(g[i], m0) : g[i]), both(st.y));
      }
      if (p.db && live) Eight<T>::store(p.db, here.bytes, g, apart);
    }
    if (ends && p.gate && !p.gate_each) {
      const long long gi = here.unit / p.chunks;
      if (p.dgate) {
        flush(gsum, s_cols, [&](const Pairs& a) {
          if (p.chunks == 1)
            Eight<T>::store(p.dgate, (gi * p.d + col) * sizeof(T), a, apart);
          else
            Eight<float>::store(p.gate_sums, (static_cast<long long>(here.unit) * p.d + col) * 4, a, apart);
        });
        fill(gsum, 0.f);
      }
      if (ok && next.unit < p.units) gate.load(p.gate, static_cast<long long>(next.unit / p.chunks) * p.d + col, apart);
    }
    here = next;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (p.want_sums >> k & 1)
      flush(sums[k], s_cols, [&](const Pairs& a) {
        Eight<float>::store(p.sums, ((static_cast<long long>(k) * gridDim.x + blockIdx.x) * p.d + col) * 4, a, apart);
      });
}

// Column sums of up to four [parts][d] and, beside them, of [gates] of them; a block
// takes 32 columns of four and its 32 warps every 32nd part (with eight warps, the
// backward pass of 4104 tokens of 1160 takes 3 us more).
struct SumParams {
  const float* from[5];
  void* to[5];
  long long parts[5], d, gates;
};
constexpr int SUM_WARPS = 32;
template <typename T>
__global__ void __launch_bounds__(SUM_WARPS * 32) sum_parts_kernel(const __grid_constant__ SumParams p) {
  __shared__ float4 s[SUM_WARPS][32];
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
    for (long long i = warp; i < parts; i += SUM_WARPS) {
      const float4 v = *reinterpret_cast<const float4*>(from + i * p.d);
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
  }
  s[warp][lane] = a;
  __syncthreads();
  const long long col = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x;
  if (threadIdx.x >= 128 || col >= p.d) return;
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < SUM_WARPS; ++w) sum += reinterpret_cast<const float*>(s[w])[threadIdx.x];
  T* to = static_cast<T*>(p.to[which]) + gate * p.d + col;
  if constexpr (sizeof(T) == 2)
    *to = __float2bfloat16_rn(sum);
  else
    *to = sum;
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
int launched() { return cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA; }  // (an error is not left for the next call)

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
  p.n = static_cast<int>(a.n);
  p.d = static_cast<int>(a.d);
  p.per = static_cast<int>(a.n_gates ? a.n / a.n_gates : a.n);
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

// Raises a kernel's shared-memory limit, once for a device.  Up to 48 KiB need no raising,
// what the kernel declares itself (2 KiB at most) counted in.
template <auto KERNEL>
int allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TP_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (bytes > 46 * 1024 && !(done.load() & bit)) {
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess) return TP_ERR_CUDA;
    done.fetch_or(bit);
  }
  return TP_OK;
}

// Up to four rows' slots in `room` bytes.
int stages_in(int room, int row) { return std::max(1, std::min(4, room / row)); }

template <typename T, bool LAYER, bool SHIFT>
int launch_forward_inst(NormParams p, const Shape& s, int num_sms, cudaStream_t st) {
  const int64_t blocks = (p.n + s.groups - 1) / s.groups, most = static_cast<int64_t>(num_sms) * std::max(1, 1024 / s.threads);
  const int row = 2 * slots<T>(s.threads) * 16, per_sm = std::max(1, 1024 / s.threads);
  p.stages = blocks <= most ? 2 : std::max(2, stages_in(200 * 1024 / per_sm, row));
  const int smem = p.stages * row;
  if (int rc = allow_smem<forward_kernel<T, LAYER, SHIFT>>(smem)) return rc;
  launch_dep(forward_kernel<T, LAYER, SHIFT>, dim3(static_cast<unsigned>(std::min(blocks, most))), s.threads, smem, st, p);
  return launched();
}
template <typename T, bool LAYER>
int launch_forward(const NormParams& p, const Shape& s, int num_sms, cudaStream_t st) {
  if (p.c_after || p.c_before) return launch_forward_inst<T, LAYER, true>(p, s, num_sms, st);
  return launch_forward_inst<T, LAYER, false>(p, s, num_sms, st);
}
template <typename T, bool LAYER, bool SHIFT, int MAX_THREADS>
int launch_backward_inst(NormParams p, const Shape& s, unsigned grid, cudaStream_t st) {
  const int row = (p.gate_each ? 5 : 4) * slots<T>(s.threads) * 16, columns = s.groups > 1 ? s.threads * 32 : 0;
  p.stages = stages_in((200 * 1024 - columns * std::max(1, 512 / s.threads)) / std::max(1, 512 / s.threads), row);
  const int smem = p.stages * row + columns;
  if (int rc = allow_smem<backward_kernel<T, LAYER, SHIFT, MAX_THREADS>>(smem)) return rc;
  launch_dep(backward_kernel<T, LAYER, SHIFT, MAX_THREADS>, dim3(grid), s.threads, smem, st, p);
  return launched();
}
// Up to 512 threads a thread may have 128 registers, which the sums need.
template <typename T, bool LAYER>
int launch_backward(const NormParams& p, const Shape& s, unsigned grid, cudaStream_t st) {
  const bool shift = p.c_after || (p.want_sums & (1 << S_CB | 1 << S_CA));
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
  p.per = static_cast<int>(c.per);
  p.dr = a.dr;
  p.dout = a.dout;
  p.dx = a.dx;
  p.db = a.db;
  p.dgate = a.dgate;
  p.gate_each = c.each;
  p.chunks = static_cast<int>(c.chunks);
  p.units = static_cast<int>(c.units);
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
      launch_dep(sum_parts_kernel<float>, blocks, SUM_WARPS * 32, 0, st, q);
    else
      launch_dep(sum_parts_kernel<__nv_bfloat16>, blocks, SUM_WARPS * 32, 0, st, q);
  }
  return launched();
}

}  // namespace tpffn
