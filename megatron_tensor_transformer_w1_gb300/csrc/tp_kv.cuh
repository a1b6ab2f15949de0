// tp_kv.cuh -- what the kernels over the paged key/value cache share: the
// batch they are given, its bounds checks, and how work is cut into segments.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tp_internal.h"

namespace tpffn {
namespace kv {

constexpr int HD = 128;  // head width
constexpr int KT = 64;   // keys per tile of the few-rows kernel

// A batch over the cache as the kernels see it (see KvSpec).  Every value
// read from a device array is brought into range here, so that no batch
// makes a kernel read or write outside its buffers; what was out of range is
// reported in the block's status word.
struct Batch {
  __nv_bfloat16 *k, *v;   // [n_pages][Hkv][page_size][HD]
  long long n_pages, max_pages;
  int page_shift;
  int B, n_tokens, max_new;
  int H, Hkv, G, causal;
  int cap;                // keys that a row of the page table can hold
  int shared;             // leading keys of every sequence that live in the same pages
  const int *cu, *kv_len, *table;
};

struct Seq {
  int q0, qn;  // first row and number of new tokens
  int kv;      // keys, the new tokens' included
  int err;
  // keys that new token i sees: a prefix of the sequence
  __device__ __forceinline__ int visible(int i, int causal) const {
    if (!causal) return kv;
    const int v = kv - qn + i + 1;
    return v > 0 ? v : 0;
  }
};

__device__ __forceinline__ Seq load_seq(const Batch& p, int b) {
  Seq s;
  const int a = p.cu[b], e = p.cu[b + 1], len = p.kv_len[b];
  s.q0 = min(max(a, 0), p.n_tokens);
  const int q1 = min(max(e, s.q0), p.n_tokens);
  s.qn = min(q1 - s.q0, p.max_new);
  s.kv = min(max(len, 0), p.cap);
  s.err = (s.q0 != a || q1 != e || s.qn != q1 - s.q0 || s.kv != len) ? DEV_ERR_BATCH : 0;
  return s;
}

// The sequence whose rows hold `row`: the first b with cu[b + 1] > row, or B.
// Called by a whole warp: 32 places are looked at per round.
__device__ __forceinline__ int find_seq_warp(const int* cu, int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) >> 5;
    const int at = lo + min((lane + 1) * step, n) - 1;
    const unsigned past = __ballot_sync(0xffffffffu, cu[at + 1] <= row);
    const int cnt = __popc(past);  // a prefix of the lanes, cu being ascending
    if (cnt == 32) return lo + n;
    lo += min(cnt * step, n);
    n = min(step, B - lo);
    if (step == 1) return lo;
    --n;  // the place at the end of the step is past the row
  }
  return lo;
}
// The same for one thread.
__device__ __forceinline__ int find_seq(const int* cu, int B, int row) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] <= row) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// 2^x by the SFU instruction; 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Work is a list of tiles, in the order of the items they belong to.  Block c
// of C takes the tiles [c T / C, (c + 1) T / C); a run of tiles of one item
// in one block is a segment.
__host__ __device__ __forceinline__ long long first_tile(long long c, long long T, long long C) { return c * T / C; }
__host__ __device__ __forceinline__ long long block_of_tile(long long t, long long T, long long C) {
  return ((t + 1) * C - 1) / T;
}

}  // namespace kv
}  // namespace tpffn
