// tp_kv.cuh -- what the kernels over the paged key/value cache share: the
// batch they are given, its bounds checks, and how work is cut into segments.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "tp_internal.h"
#include "tpffn.h"

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

// Work is a list of tiles of KTILE keys, in the order of the items they belong
// to: sequence by sequence, its key/value heads, their row tiles of RT rows
// (RT = 0: all rows of the item in one).  The rows of a sequence and a key/value
// head are its new tokens times the G query heads of the group, row r being
// token r / G, head h G + r % G.  Prefix items (PREFIX) take the rows of all
// sequences together against the shared keys.
//
// A tile takes one or more places of the list (see Cut).  Block c of C takes the
// places [c T / C, (c + 1) T / C) and the tiles that begin there, whatever items
// they belong to; a run of tiles of one item in one block is a segment.  Every
// block gets the same number of places however the lengths differ (but see
// Deal).

// (A 64-bit division takes some hundred cycles, and several in a row are felt.)
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<unsigned>(a) / static_cast<unsigned>(b) : a / b;
}
__device__ __forceinline__ long long first_tile(long long c, long long T, long long C) { return quotient(c * T, C); }
__device__ __forceinline__ long long block_of_tile(long long t, long long T, long long C) {
  return quotient((t + 1) * C - 1, T);
}

// How T places fall to `grid` blocks: the first E share Te of them evenly, the L
// behind them the rest.  Where the first `early` blocks start while the SMs of
// the others are still busy, for as long as a block takes for `lead` places,
// they get so many more; otherwise (early = 0) all get the same.  A block has
// `least` of them, the most that a tile takes, so that no block inside an item is
// without a tile.  (Where blocks do not start in that order it takes longer.)
struct Deal {
  long long T, Te;
  int E, L;
  __device__ __forceinline__ Deal(long long T_, int grid, int early, int lead, int least) : T(T_), Te(T_), L(0) {
    const long long ahead = static_cast<long long>(early) * lead;
    E = early && T <= ahead ? early : grid;
    if (early && T > ahead) {
      const long long late = quotient((T - ahead) * (grid - early), grid);
      Te = T - late;
      E = early;
      L = static_cast<int>(late < grid - early ? late : grid - early);
    }
    const long long most = least > 1 ? quotient(T, least) : T;
    if (most < E) E = most > 1 ? static_cast<int>(most) : 1;
  }
  __device__ __forceinline__ long long first(long long c) const {
    return c <= E ? first_tile(c, Te, E) : Te + first_tile(c - E, T - Te, L);
  }
  __device__ __forceinline__ long long block_of(long long t) const {
    return t < Te ? block_of_tile(t, Te, E) : E + block_of_tile(t - Te, T - Te, L);
  }
};

// An item takes START places of the list before its first tile, for what a block
// spends on a segment besides its tiles, and a tile ONE places, or TWO if it has
// more than half of RT rows.  A tile is the block's that has its first place.
template <bool PREFIX, int KTILE, int RT, int START_ = 0, int ONE = 1, int TWO = 1>
struct Cut {
  static constexpr int START = START_, LEAST = TWO;
  static __device__ __forceinline__ int width(const Batch& p, const Seq& s, int rt) {
    return ONE == TWO || s.qn * p.G - rt * RT <= RT / 2 ? ONE : TWO;
  }
  static __device__ __forceinline__ int row_tiles(const Batch& p, const Seq& s) {
    const int rows = s.qn * p.G;
    return RT ? (rows + RT - 1) / (RT ? RT : 1) : (rows > 0);
  }
  static __device__ __forceinline__ int first_key(const Batch& p) { return PREFIX ? 0 : p.shared; }
  static __device__ __forceinline__ int t0(const Batch& p) { return first_key(p) / KTILE; }
  // tiles of one row tile: up to the last key that any of its rows sees
  static __device__ __forceinline__ int tiles(const Batch& p, const Seq& s, int rt) {
    int hi = s.kv;
    if (RT && !PREFIX) {
      const int tok = min((rt * RT + RT - 1) / p.G, s.qn - 1);
      hi = s.visible(tok, p.causal);
    }
    return (s.qn > 0 && hi > first_key(p)) ? (hi + KTILE - 1) / KTILE - t0(p) : 0;
  }
  // places in the list
  static __device__ __forceinline__ int places(const Batch& p, const Seq& s, int rt) {
    const int n = tiles(p, s, rt);
    return n * width(p, s, rt) + (n > 0 ? START : 0);
  }
  static __device__ __forceinline__ long long places_per_head(const Batch& p, const Seq& s) {
    const int n = row_tiles(p, s);
    if (!RT || PREFIX) return static_cast<long long>(n) * places(p, s, 0);
    long long sum = 0;
    for (int rt = 0; rt < n; ++rt) sum += places(p, s, rt);
    return sum;
  }
};

// Where a block stands in the list: tile t of the nt of a row tile.
struct Cursor {
  int b, h, rt, t, nt;
  Seq s;
};

// The next tile; past an item's end the next one that has tiles.  The caller
// knows that there is one; should the arrays have changed meanwhile, the walk
// ends at the last sequence with an item of no rows and no keys.
template <typename C, bool PREFIX>
__device__ __forceinline__ void advance(const Batch& p, Cursor& c) {
  if (++c.t < c.nt) return;
  c.t = 0;
  do {
    if (++c.rt >= C::row_tiles(p, c.s)) {
      c.rt = 0;
      if (++c.h >= p.Hkv) {
        c.h = 0;
        if constexpr (!PREFIX) {
          if (++c.b >= p.B) {
            c.b = p.B - 1;
            c.s.qn = c.s.kv = 0;
            c.nt = 1;
            return;
          }
          c.s = load_seq(p, c.b);
        }
      }
    }
    c.nt = C::tiles(p, c.s, c.rt);
  } while (c.nt == 0);
}

// Places left behind the tile at the cursor, up to the block's last; the block
// has another tile where they are more than none.  `left`: from the tile's first.
template <typename C>
__device__ __forceinline__ int left_behind(const Batch& p, const Cursor& c, int left) {
  return left - C::width(p, c.s, c.rt) - (c.t + 1 == c.nt ? C::START : 0);
}

struct SchedScratch {
  long long sums[4];
  unsigned long long longest[4];
  int least[4];
  Cursor start;
  int gone;
};
struct Sched {
  int places = 0;          // of this block
  int left = 0;            // from its first tile's on; none: no tile
  int table_row = 0;       // whose page table leads to the shared pages
  bool all_see = false;    // every row sees every shared key
  bool some_empty = false; // there are rows of sequences that belong to no tile
  long long first = 0, total = 0, blocks = 0;
  // this block's share of `total_` tiles; false: none
  __device__ __forceinline__ bool set(long long total_, int early, int lead, int least) {
    if (total_ == 0) return false;
    const Deal D(total_, gridDim.x, early, lead, least);
    total = total_;
    blocks = D.E + D.L;
    if (blockIdx.x >= blocks) return false;
    first = D.first(blockIdx.x);
    left = places = static_cast<int>(D.first(blockIdx.x + 1) - first);
    return true;
  }
};

// The first tile from place `at` of a sequence's (x.b, x.s) places on; returns how
// many places lie before it.  x.t = x.nt: the next item's first.
template <typename C>
__device__ __forceinline__ int locate(const Batch& p, Cursor& x, long long at, long long per_head) {
  x.h = static_cast<int>(quotient(at, per_head));
  at -= x.h * per_head;
  for (x.rt = 0;; ++x.rt) {
    x.nt = C::tiles(p, x.s, x.rt);
    const int n = C::places(p, x.s, x.rt);
    if (at < n) break;
    at -= n;
  }
  const int w = C::width(p, x.s, x.rt), in = static_cast<int>(at) - C::START;
  x.t = in > 0 ? (in + w - 1) / w : 0;
  return x.t * w - in;
}

// Called by every thread of a block (at least 128): sums the tiles of all
// sequences and finds the block's first tile.  Block 0 leaves the prefix sums
// for the combine kernel where that asks for them: `sched` [B + 1] places per
// key/value head before sequence b, or for prefix items {tiles of a row tile,
// row tiles}.  Up to 32 sequences every warp does it for itself, a lane to a
// sequence, without meeting the others: a call of few tokens waits for this
// before its first copy.
template <typename C, bool PREFIX>
__device__ __forceinline__ Sched schedule(const Batch& p, long long* sched, SchedScratch* w, Cursor& c, int* err,
                                          int early = 0, int lead = 0) {
  const int tid = threadIdx.x, lane = tid & 31;
  const bool small = p.B <= 32;
  Sched S;
  if constexpr (PREFIX) {
    // the longest sequence's table covers the shared pages if any does
    unsigned long long longest = 0;
    int least = INT_MAX;
    if (small || tid < 128) {
      for (int b = small ? lane : tid; b < p.B; b += 128) {
        const Seq s = load_seq(p, b);
        const unsigned long long key = (static_cast<unsigned long long>(s.kv) << 32) | (0xffffffffu - b);
        longest = key > longest ? key : longest;
        if (s.qn > 0) least = min(least, s.visible(0, p.causal));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, longest, d);
        longest = o > longest ? o : longest;
        least = min(least, __shfl_xor_sync(0xffffffffu, least, d));
      }
    }
    if (!small) {
      if (tid < 128 && lane == 0) {
        w->longest[tid >> 5] = longest;
        w->least[tid >> 5] = least;
      }
      __syncthreads();
      longest = 0;
      for (int i = 0; i < 4; ++i) {
        longest = w->longest[i] > longest ? w->longest[i] : longest;
        least = min(least, w->least[i]);
      }
    }
    S.table_row = static_cast<int>(0xffffffffu - static_cast<unsigned>(longest));
    c.b = 0;
    c.s.q0 = 0;
    c.s.qn = min(max(p.cu[p.B], 0), p.n_tokens);
    c.s.kv = min(p.shared, static_cast<int>(longest >> 32));
    c.s.err = 0;
    S.all_see = least >= c.s.kv;
    const int n_rt = C::row_tiles(p, c.s);
    c.nt = C::tiles(p, c.s, 0);
    if (blockIdx.x == 0 && tid == 0) {
      sched[0] = c.nt;
      sched[1] = n_rt;
    }
    if (!S.set(static_cast<long long>(n_rt) * c.nt * p.Hkv, 0, 0, 1)) return S;
    const long long item = quotient(S.first, c.nt);
    c.t = static_cast<int>(S.first - item * c.nt);
    c.h = static_cast<int>(quotient(item, n_rt));
    c.rt = static_cast<int>(item - static_cast<long long>(c.h) * n_rt);
  } else {
    const int per = small ? 1 : (p.B + 127) / 128;
    const int b0 = small ? min(lane, p.B) : min(tid * per, p.B), b1 = small || tid < 128 ? min(b0 + per, p.B) : b0;
    long long sum = 0;
    int empty = 0;
    Cursor x{};
    for (int b = b0; b < b1; ++b) {
      x.s = load_seq(p, b);
      *err |= x.s.err;
      sum += C::places_per_head(p, x.s);
      empty |= x.s.qn > 0 && C::tiles(p, x.s, 0) == 0;
    }
    long long before = sum;  // inclusive sums within the warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    long long total = 0;
    if (small) {
      S.some_empty = __any_sync(0xffffffffu, empty);
      total = __shfl_sync(0xffffffffu, before, 31);
    } else {
      if (tid < 128 && lane == 31) w->sums[tid >> 5] = before;
      S.some_empty = __syncthreads_or(empty) != 0;
      for (int i = 0; i < 4; ++i) {
        if (i < (tid >> 5)) before += w->sums[i];
        total += w->sums[i];
      }
    }
    before -= sum;
    if (sched && blockIdx.x == 0 && tid < (small ? 32 : 128)) {
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        sched[b] = at;
        at += C::places_per_head(p, load_seq(p, b));
      }
      if (tid == 0) sched[p.B] = total;
    }
    if (!S.set(total * p.Hkv, early, lead, C::LEAST)) return S;
    const bool mine = (small || tid < 128) && S.first >= before * p.Hkv && S.first < (before + sum) * p.Hkv;
    if (small) {
      const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      c.b = src;
      c.s.q0 = __shfl_sync(0xffffffffu, x.s.q0, src);
      c.s.qn = __shfl_sync(0xffffffffu, x.s.qn, src);
      c.s.kv = __shfl_sync(0xffffffffu, x.s.kv, src);
      c.s.err = 0;
      sum = __shfl_sync(0xffffffffu, sum, src);
      before = __shfl_sync(0xffffffffu, before, src);
      S.left -= locate<C>(p, c, S.first - before * p.Hkv, sum);
    } else {
      if (mine) {
        w->start = Cursor{p.B - 1, 0, 0, 0, 1, Seq{}};  // see advance()
        w->gone = 0;
        long long at = S.first - before * p.Hkv;
        for (int b = b0; b < b1; ++b) {
          x.b = b;
          x.s = load_seq(p, b);
          const long long per_head = C::places_per_head(p, x.s);
          if (at < per_head * p.Hkv) {
            w->gone = locate<C>(p, x, at, per_head);
            w->start = x;
            break;
          }
          at -= per_head * p.Hkv;
        }
      }
      __syncthreads();
      c = w->start;
      S.left -= w->gone;
    }
    if (c.t == c.nt) {  // behind an item's last tile
      S.left -= C::START;
      --c.t;
      if (S.left > 0) advance<C, PREFIX>(p, c);
    }
  }
  return S;
}

// An item cut between blocks, noted by the block that has its first tile.
struct Split {
  Seq s;
  int h, rt;
  int parts;  // 0: the block's last segment is none
  int pad;
};

// What a segment leaves for the combine kernel: the running maximum (in log2
// units) and sum of each row, and its unnormalised output in 32 bits.  A
// segment that is a whole item goes to its rows' own places ([token][head],
// used only where other keys are still to be joined); the others, of which a
// block has at most two, go to its two slots: one that goes on with an item to
// the first, one that begins an item to the second.
// A slot's outputs lie in four parts of 32 columns, [4][slot_rows][32], the
// 16-byte chunks of a row's 128 bytes swizzled by the row (chunk k at k ^ (r &
// 7)): so the many-rows kernel, a row to a thread, can stage a warp's 32 rows
// free of bank conflicts and write them as they lie, 512 bytes in a row per
// store, and the combine kernel reads whole lines.
struct Parts {
  float* slot_o = nullptr;    // [2 blocks][4][slot_rows][32]
  float2* slot_ml = nullptr;  // [2 blocks][slot_rows]
  float* row_o = nullptr;     // [n_tokens * H][HD]
  float2* row_ml = nullptr;
  long long* sched = nullptr; // null: the splits say all
  Split* split = nullptr;     // [blocks]
  int slot_rows = 0, grid = 0, rt = 0;  // rt: rows of a row tile, 0: all
  int early = 0, lead = 0;              // see Deal
};

// Chunk c (of 32, four columns each) of row r of a slot.
__device__ __forceinline__ long long slot_chunk(const Parts& P, long long slot, int r, int c) {
  return ((slot * 4 + (c >> 3)) * P.slot_rows + r) * 32 + (((c & 7) ^ (r & 7)) << 2);
}

// The note on a block's last segment, whose last tile is x at place `at` of the
// list.  (Where all blocks get the same number of places.)
template <typename C>
__device__ __forceinline__ Split split_of(const Batch& p, const Sched& S, const Cursor& x, int seg_t, long long at) {
  Split r{};
  if (seg_t == 0 && x.t + 1 < x.nt) {
    const long long end = at + (x.nt - 1 - x.t) * C::width(p, x.s, x.rt);  // the item's last tile
    r.s = x.s;
    r.h = x.h;
    r.rt = x.rt;
    r.parts = static_cast<int>(block_of_tile(end, S.total, S.blocks) - blockIdx.x) + 1;
  }
  return r;
}

// 1 / l and the log2-sum-exp of a row with running maximum m and sum l.  l is NaN
// where a score was NaN or +inf (the maximum drops NaN): that is what the row
// gets.  It is 0 where the row sees no key, for an output of 0, and where all
// scores that it sees are -inf, for one of 0 / 0.
__device__ __forceinline__ float inverse_sum(float l, bool sees) { return l == 0.f && !sees ? 0.f : 1.f / l; }
__device__ __forceinline__ float log2_sum_exp(float m, float l) { return l == 0.f ? -INFINITY : m + log2f(l); }

struct AttendParams {
  Batch b;
  const __nv_bfloat16* q;  // [n_tokens][H * HD]
  __nv_bfloat16* o;        // [n_tokens][H * HD]
  float* lse;              // [n_tokens][H] or null
  Parts part;
  float scale_log2;
  int* status;             // a word per block
  // The kernel before it on the stream is the shared keys' of the same call:
  // nothing that it writes is read here, and it lets its successor start only
  // when the call's inputs are there.  This kernel starts without waiting for
  // it, and waits before its blocks end.
  int beside;
  // The kernel before it is the same call's append, which lets its successor
  // start only when the call's inputs are there: the place in the list is looked
  // for while that runs, and waited for before anything else is read.
  int behind_append;
  int skip_load;           // test hook: no block issues its first copy
  unsigned long long timeout_ns;
};

constexpr int RT_MANY = 256;  // rows of an item of the many-rows kernel
// A segment costs it about a tile, a tile of one row tile little less than one of
// two (its softmax waits for its own products).  All tiles alike and segments for
// nothing / these weights: 4 prompt chunks 373 / 365 us, 16 prompts behind 4096
// shared keys 215 / 208 us, 86 sequences of 40 rows 109 / 93 us; one row tile for
// two thirds of two 374 / 219 / 94 us.
template <bool PREFIX>
using Many = Cut<PREFIX, 128, RT_MANY, PREFIX ? 0 : 6, PREFIX ? 1 : 6, PREFIX ? 1 : 7>;
// The many-rows kernel (tp_kv_tc.cu).
int launch_many(const AttendParams& p, bool prefix, LaunchCtx& ctx, const char* name);

// Rows that see no key at all and belong to no tile: zeros.  By all threads;
// block c takes the sequences c, c + grid, ...
template <typename C>
__device__ __forceinline__ void write_empty_rows(const AttendParams& p, int rt_rows) {
  const Batch& B = p.b;
  for (int b = blockIdx.x; b < B.B; b += gridDim.x) {
    const Seq s = load_seq(B, b);
    const int rows = s.qn * B.G, n_rt = C::row_tiles(B, s);
    for (int rt = 0; rt < n_rt && C::tiles(B, s, rt) == 0; ++rt) {
      const int r0 = rt * rt_rows, n = rt_rows ? min(rt_rows, rows - r0) : rows;
      for (int i = threadIdx.x; i < n * B.Hkv * 16; i += blockDim.x) {
        const int r = r0 + i / (16 * B.Hkv), h = (i >> 4) % B.Hkv;
        const long long row = static_cast<long long>(s.q0 + r / B.G) * B.H + h * B.G + r % B.G;
        reinterpret_cast<uint4*>(p.o + row * HD)[i & 15] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse && (i & 15) == 0) p.lse[row] = -INFINITY;
      }
    }
  }
}

// Launch as a programmatic dependent of the stream's previous kernel.
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

// Whether a kernel's shared-memory limit has been raised on the current device.
template <typename K>
int set_smem_once(K kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TP_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return TP_ERR_CUDA;
    done.fetch_or(bit);
  }
  return TP_OK;
}

}  // namespace kv
}  // namespace tpffn
