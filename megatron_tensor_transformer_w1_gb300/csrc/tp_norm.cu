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
// columns 8 t .. 8 t + 7; a block has blockDim / tpr rows at a time.
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
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += s[turn][first + w][k];
  turn ^= 1;
}

// The mean and factor of a row's norm.
template <bool LAYER>
__device__ __forceinline__ float2 row_stats(const float (&v)[8], bool ok, const NormParams& p, float (*s)[32][1], int& turn) {
  float mean = 0.f, sum[1] = {0.f};
  if (LAYER) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[0] += v[i];
    row_sums<1>(sum, p.tpr, s, turn);
    mean = sum[0] * p.inv_d;
    sum[0] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = ok ? v[i] - mean : 0.f;
    sum[0] = fmaf(a, a, sum[0]);
  }
  row_sums<1>(sum, p.tpr, s, turn);
  return make_float2(mean, 1.f / sqrtf(fmaf(sum[0], p.inv_d, p.eps)));
}

template <typename T, bool LAYER>
__global__ void __launch_bounds__(1024) forward_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s_sum[2][32][1];
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x % p.tpr, rows = blockDim.x / p.tpr;
  int turn = 0;
  const long long col = 8ll * t;
  const bool ok = col < p.d;
  Eight<T> wa, ca, wb, cb;
  if (ok && p.w_after) wa.load(p.w_after, col);
  if (ok && p.c_after) ca.load(p.c_after, col);
  if (ok && p.w_before) wb.load(p.w_before, col);
  if (ok && p.c_before) cb.load(p.c_before, col);
  for (long long row0 = static_cast<long long>(blockIdx.x) * rows; row0 < p.n; row0 += static_cast<long long>(gridDim.x) * rows) {
    const long long row = row0 + threadIdx.x / p.tpr, at = row * p.d + col;
    const bool live = ok && row < p.n;
    Eight<T> x, b, g;
    x.zero();
    b.zero();
    g.zero();
    if (live) {
      x.load(p.x, at);
      if (p.b) b.load(p.b, at);
      if (p.gate) g.load(p.gate, row / p.per * p.d + col);
    }
    float v[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = x[i];
      u[i] = b[i];
    }
    float2 sa{}, sb{};
    if (p.after) {
      sa = row_stats<LAYER>(u, ok, p, s_sum, turn);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = (u[i] - sa.x) * sa.y;
        if (p.w_after) u[i] *= wa[i];
        if (p.c_after) u[i] += ca[i];
      }
    }
    if (live && p.b) {  // (columns that there are not stay zero)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(p.gate ? p.scale * g[i] : p.scale, u[i], v[i]);
    }
    if (live) Eight<T>::store(p.r, at, v);
    if (p.before) {
      sb = row_stats<LAYER>(v, ok, p, s_sum, turn);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = (v[i] - sb.x) * sb.y;
        if (p.w_before) v[i] *= wb[i];
        if (p.c_before) v[i] += cb[i];
      }
      if (live) Eight<T>::store(p.out, at, v);
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
enum { S_WB = 0, S_CB = 1, S_WA = 2, S_CA = 3 };
template <typename T, bool LAYER, bool SHIFT, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) backward_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s_sum[2][32][2];
  extern __shared__ float s_cols[];  // [rows of a block][tpr * 8]
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, rows = blockDim.x / p.tpr;
  int turn = 0;
  const long long col = 8ll * t;
  const bool ok = col < p.d;
  Eight<T> wa, ca, wb, gate;
  wa.zero();
  ca.zero();
  wb.zero();
  gate.zero();
  if (ok && p.w_after) wa.load(p.w_after, col);
  if (ok && p.c_after) ca.load(p.c_after, col);
  if (ok && p.w_before) wb.load(p.w_before, col);
  float sums[4][8] = {}, gsum[8] = {};
  // A column sum over the block's row groups, then to `write`.
  auto flush = [&](float (&a)[8], auto&& write) {
    if (rows > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) s_cols[threadIdx.x * 8 + i] = a[i];
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < rows; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] += s_cols[(g * p.tpr + t) * 8 + i];
    }
    if (group == 0 && ok) write(a);
  };
  auto to_floats = [](float* at, const float (&a)[8]) {
    reinterpret_cast<float4*>(at)[0] = make_float4(a[0], a[1], a[2], a[3]);
    reinterpret_cast<float4*>(at)[1] = make_float4(a[4], a[5], a[6], a[7]);
  };
  for (long long unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
    const long long gi = unit / p.chunks, c = unit - gi * p.chunks;
    const long long from = gi * p.per + c * p.per / p.chunks, to = gi * p.per + (c + 1) * p.per / p.chunks;
    if (ok && p.gate && !p.gate_each) gate.load(p.gate, gi * p.d + col);
    for (long long row0 = from; row0 < to; row0 += rows) {
      const long long row = row0 + group, at = row * p.d + col;
      const bool live = ok && row < to;
      Eight<T> b, r, dout, dr;
      b.zero();
      r.zero();
      dout.zero();
      dr.zero();
      float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
      if (live) {
        if (p.before) {
          dout.load(p.dout, at);
          r.load(p.r, at);
        }
        if (p.b) b.load(p.b, at);
        if (p.dr) dr.load(p.dr, at);
        if (p.gate_each) gate.load(p.gate, at);
        if (p.stats) st = p.stats[row];
      }
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = dr[i];
      if (p.before) {
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = (r[i] - st.z) * st.w, d = dout[i], dy = p.w_before ? d * wb[i] : d;
          s[0] = fmaf(dy, y, s[0]);
          s[1] += dy;
          sums[S_WB][i] = fmaf(d, y, sums[S_WB][i]);
          if (SHIFT) sums[S_CB][i] += d;
        }
        row_sums<2>(s, p.tpr, s_sum, turn);
        const float m1 = s[0] * p.inv_d, m0 = LAYER ? s[1] * p.inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = (r[i] - st.z) * st.w, d = dout[i], dy = p.w_before ? d * wb[i] : d;
          g[i] = fmaf(st.w, dy - fmaf(y, m1, m0), g[i]);
        }
      }
      if (p.dx && live) Eight<T>::store(p.dx, at, g);
      if (!p.b && !p.db) continue;  // (of all threads)
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = p.after ? (b[i] - st.x) * st.y : b[i], sg = live ? p.scale * g[i] : 0.f;
        if (p.dgate) {
          const float dg = sg * fmaf(y, p.w_after ? wa[i] : 1.f, ca[i]);
          gsum[i] = p.gate_each ? dg : gsum[i] + dg;
        }
        float du = p.gate ? sg * gate[i] : sg;
        if (p.after) {
          sums[S_WA][i] = fmaf(du, y, sums[S_WA][i]);
          if (SHIFT) sums[S_CA][i] += du;
          if (p.w_after) du *= wa[i];
          s[0] = fmaf(du, y, s[0]);
          s[1] += du;
        }
        g[i] = du;
      }
      if (p.gate_each && p.dgate && live) Eight<T>::store(p.dgate, at, gsum);
      if (p.after) {
        row_sums<2>(s, p.tpr, s_sum, turn);
        const float m1 = s[0] * p.inv_d, m0 = LAYER ? s[1] * p.inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = st.y * (g[i] - fmaf((b[i] - st.x) * st.y, m1, m0));
      }
      if (p.db && live) Eight<T>::store(p.db, at, g);
    }
    if (p.dgate && !p.gate_each) {
      flush(gsum, [&](const float (&a)[8]) {
        if (p.chunks == 1)
          Eight<T>::store(p.dgate, gi * p.d + col, a);
        else
          to_floats(p.gate_sums + unit * p.d + col, a);
      });
#pragma unroll
      for (int i = 0; i < 8; ++i) gsum[i] = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (p.want_sums >> k & 1)
      flush(sums[k], [&](const float (&a)[8]) {
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

// Threads to a row, rows and threads of a block.
struct Shape {
  int tpr, rows, threads;
};
Shape shape_of(int64_t d, int64_t n, int num_sms) {
  Shape s;
  s.tpr = static_cast<int>((d / 8 + 31) / 32 * 32);
  s.rows = std::max(512 / s.tpr, 1);
  while (s.rows > 1 && (n + s.rows - 1) / s.rows < num_sms) s.rows /= 2;  // few tokens: on all SMs
  s.threads = s.rows * s.tpr;
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
  p.chunks = std::min<int64_t>(std::max<int64_t>(most / p.gates, 1), (p.per + s.rows - 1) / s.rows);
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

template <typename T, bool LAYER>
void launch_forward(const NormParams& p, const Shape& s, unsigned grid, cudaStream_t st) {
  launch_dep(forward_kernel<T, LAYER>, dim3(grid), s.threads, 0, st, p);
}
// Up to 512 threads a thread may have 128 registers, which the sums need.
template <typename T, bool LAYER, bool SHIFT>
void launch_backward_inst(const NormParams& p, const Shape& s, unsigned grid, cudaStream_t st) {
  const int smem = s.rows > 1 ? s.threads * 8 * 4 : 0;
  if (s.threads <= 512)
    launch_dep(backward_kernel<T, LAYER, SHIFT, 512>, dim3(grid), s.threads, smem, st, p);
  else
    launch_dep(backward_kernel<T, LAYER, SHIFT, 1024>, dim3(grid), s.threads, smem, st, p);
}
template <typename T, bool LAYER>
void launch_backward(const NormParams& p, const Shape& s, unsigned grid, cudaStream_t st) {
  if (p.want_sums & (1 << S_CB | 1 << S_CA))
    launch_backward_inst<T, LAYER, true>(p, s, grid, st);
  else
    launch_backward_inst<T, LAYER, false>(p, s, grid, st);
}
}  // namespace norm

int launch_norm_fwd(const NormSpec& a, int num_sms, cudaStream_t st) {
  using namespace norm;
  const Shape s = shape_of(a.d, a.n, num_sms);
  NormParams p = params_of(a, s);
  p.x = a.x;
  p.r = a.r;
  p.out = a.out;
  const int64_t blocks = (a.n + s.rows - 1) / s.rows, most = static_cast<int64_t>(num_sms) * std::max(1, 2048 / s.threads);
  const unsigned grid = static_cast<unsigned>(std::min(blocks, most));
  if (a.f32)
    a.layer ? launch_forward<float, true>(p, s, grid, st) : launch_forward<float, false>(p, s, grid, st);
  else
    a.layer ? launch_forward<__nv_bfloat16, true>(p, s, grid, st) : launch_forward<__nv_bfloat16, false>(p, s, grid, st);
  return launched();
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
  if (a.f32)
    a.layer ? launch_backward<float, true>(p, s, grid, st) : launch_backward<float, false>(p, s, grid, st);
  else
    a.layer ? launch_backward<__nv_bfloat16, true>(p, s, grid, st) : launch_backward<__nv_bfloat16, false>(p, s, grid, st);
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
