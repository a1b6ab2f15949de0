// tp_kv_tc.cu -- attention of many query rows over the paged key/value cache:
// prompts and chunks of prompts, and the rows of a whole batch against the
// keys that its sequences share.
//
// An item is a key/value head with 256 of a sequence's rows (new tokens times
// the G query heads of the group; of all sequences' rows for the shared
// keys), in two tiles of 128; its keys come in tiles of 128.  One persistent
// block per SM takes an equal share of the batch's key tiles by cost (Cut in
// tp_kv.cuh) and leaves the parts of items that it shares with its
// neighbours to kv_combine_kernel.
//
// With R rows a key takes 256 R multiply-adds for its 512 bytes, R flops a byte:
// at 1898 TFLOP/s and 6773 GB/s the products bound the time of own keys from
// some 280 rows on (fewer rows of a tile of 128 cost as much as a full one, and
// keys that lie in L2 or are shared cost less to read).  A step of two row tiles
// has 4 x 128^3 multiply-adds, 2048 cycles at 4096 a cycle.  The two row tiles
// take turns: while one tile's scores go through the softmax, the products of
// the other run.  A block has
//  * warp 0: copies K and V tiles by TMA, a copy for each page (or 128 keys of
//    a longer one), into a ring of four 32 KB slots;
//  * warps 1 and 2: a lane of each issues tcgen05.mma for row tile t = 0, 1:
//    S_t = Q_t K^T into tensor memory, then O_t += P_t V with P_t, in bf16,
//    over the S_t it came from.  Products run in the order of issue, so the
//    S_t that is issued behind O_t += P_t V into the same buffer finds P_t
//    read.  Two warps, because one spends a third of a step between products;
//  * warps 4-7 and 8-11: the softmax of row tiles 0 and 1, a row per thread,
//    with a maximum that moves only when it grew by more than 2^8, so that
//    O_t is rarely rescaled; they write the rows out at the end of a segment;
//  * warp 3: gathers the query rows of the next segment meanwhile (of the
//    block's first, the softmax warps do).
// S_t comes in halves of 64 keys into two buffers, so that the softmax of one
// half finds the next one's scores done: with one buffer of 128 keys a row
// tile waits for its two products in every step.
// Values of slots behind a sequence's last key may be anything, also NaN, and
// 0 x NaN would spoil a row: the rows of V behind the last key are zeroed up
// to the 16 that a product step takes, and the steps behind are left out.
//
// Every wait is bounded (status word and block-wide abort flag; copies and
// products in flight are drained and tensor memory freed).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "tc_ptx.cuh"
#include "tp_internal.h"
#include "tp_kv.cuh"
#include "tpffn.h"

namespace tpffn {
namespace kv {
using namespace tc;

constexpr int BK = 128;                 // keys of a tile
constexpr int TILE_BYTES = 128 * HD * 2;
constexpr int SLOTS = 4;                // K and V tiles in flight
constexpr int SK = 64;                  // keys of a product's half tile
constexpr int MANY_THREADS = 384;
constexpr int M_Q = 0;                             // two row tiles
constexpr int M_RING = M_Q + 2 * TILE_BYTES;
constexpr int M_OUT = M_RING + SLOTS * TILE_BYTES; // 4 KB per softmax warp
constexpr int M_BAR = M_OUT + 8 * 4096;
constexpr int M_SMEM = M_BAR + 512 + 1024;
static_assert(M_SMEM <= 232448, "shared memory per block");
static_assert(sizeof(SchedScratch) <= 8 * 4096, "the schedule's scratch lies where the output is staged");

// A K or V tile in shared memory: groups of 8 keys, 2 KB each, the columns
// 0-63 of the group's keys and then 64-127 in 128-byte swizzled rows.  So a
// page of any size is one box of the tensor map {64 columns, 8 keys, 2 column
// halves, groups of a page, heads and pages}; with the column halves 16 KB
// apart a page takes two.
constexpr uint32_t GROUP = 2048, COL_HALF = 1024;
// The products' operands: K, keys by columns (step ks: columns 16 ks ..), and
// V, its columns along N (step ks: keys 16 ks ..).
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lbo) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(GROUP >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// 16-byte chunk c (of 16) of key r.
__device__ __forceinline__ uint32_t key_chunk(uint32_t tile, int r, int c) {
  return tile + (r >> 3) * GROUP + (c >> 3) * COL_HALF + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// A tile, to the issuing warp: product steps of 16 keys, whether it ends a
// segment, whether the second row tile has rows, whether it is the block's last.
constexpr uint32_t I_STEPS = 15, I_LAST = 16, I_TWO = 32, I_END = 64;

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* tm, uint64_t* bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Waits for tensor-memory loads; the second statement names their registers,
// so that no use of them moves before the wait.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7]));
}
// Two 32-bit operations per instruction, and a maximum of three: with two
// softmax warps per scheduler their instructions are what the time goes by.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Hides the columns outside [from, to) of 32.
__device__ __forceinline__ void hide(uint32_t (&r)[32], int from, int to) {
  const uint32_t below = to >= 32 ? 0xffffffffu : (to <= 0 ? 0u : (1u << to) - 1u);
  const uint32_t seen = below & (from <= 0 ? 0xffffffffu : (from >= 32 ? 0u : 0xffffffffu << from));
#pragma unroll
  for (int k = 0; k < 32; ++k) r[k] = (seen >> k) & 1u ? r[k] : __float_as_uint(-INFINITY);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <bool PREFIX>
__global__ void __launch_bounds__(MANY_THREADS, 1)
    kv_many_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ AttendParams p) {
  using C = Many<PREFIX>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + M_BAR);
  uint64_t* full = bar;         // [SLOTS] a K or V tile has landed
  uint64_t* empty = bar + 4;    // [SLOTS] its products are done
  uint64_t* q_full = bar + 8;   // [2]
  uint64_t* q_empty = bar + 10; // [2] a segment's last S_t is done
  uint64_t* s_full = bar + 12;  // [2][2] S_t of a half tile is done
  uint64_t* p_full = bar + 16;  // [2][2] P_t written (a warp each)
  uint64_t* pv_done = bar + 20; // [2][2] O_t has its product
  uint64_t* drain = bar + 24;   // [2]
  volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(bar + 26);  // [2] of the tiles in the ring
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 27);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + 27) + 1;
  const Batch& B = p.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = p.status + blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);  // both row tiles
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 4);
      mbar_init(&q_empty[t], 1);
      mbar_init(&drain[t], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  if (!p.beside && !p.behind_append) grid_dep_wait();
  if (!p.behind_append) grid_dep_launch();
  if (threadIdx.x == 0) {
    *status = 0;
    if (p.part.split) p.part.split[blockIdx.x] = Split{};
  }
  int err = 0;
  Cursor c;
  const Sched S = schedule<C, PREFIX>(B, p.part.sched, reinterpret_cast<SchedScratch*>(smem + M_OUT), c, &err);
  if (p.behind_append) {
    grid_dep_wait();
    grid_dep_launch();
  }
  tc_fence_before();
  __syncthreads();  // (also: the status word is clear, the scratch has been read)
  tc_fence_after();
  if (err) atomicOr(status, err);
  const uint32_t tmem = *tmem_slot;  // S_t at columns 128 t and 128 t + 64, O_t at 256 + 128 t
  const Waiter W{abort_flag, status, p.timeout_ns};
  const int t0 = C::t0(B), lo = C::first_key(B);
  const bool some = S.left > 0;
  int left = S.left;  // of each role, with its cursor
  auto ring = [&](uint32_t i) { return smem + M_RING + (i & (SLOTS - 1)) * TILE_BYTES; };
  auto rows_of = [&](const Cursor& x) { return x.s.qn * B.G - x.rt * RT_MANY; };  // > 128: both row tiles

  // Query rows [first, first + n) of row tile t of a segment, into the swizzled
  // layout of the products: 16 lanes to a row, two rows of 256 bytes to a warp's
  // copy.
  const int dtok = 2 / B.G, dg = 2 - dtok * B.G;
  auto fetch_q = [&](const Cursor& x, int t, int first, int n) {
    const int rows = rows_of(x) - t * 128, r0 = first + (lane >> 4);
    const int item_row = x.rt * RT_MANY + t * 128 + r0, tok = item_row / B.G;
    int g = item_row - tok * B.G;
    const uint32_t qs = smem_u32(smem + M_Q + t * TILE_BYTES);
    const __nv_bfloat16* src =
        p.q + ((static_cast<long long>(x.s.q0) + tok) * B.H + static_cast<long long>(x.h) * B.G + g) * HD +
        (lane & 15) * 8;
    const int step = (dtok * B.H + dg) * HD, wrap = (B.H - B.G) * HD;  // two rows on; past a token's last head
#pragma unroll 4
    for (int i = 0; i < n; i += 2) {
      const bool valid = r0 + i < rows;
      cp_async16z(sw_chunk(qs, 128, r0 + i, lane & 15), valid ? src : p.q, valid);
      src += step;
      g += dg;
      if (g >= B.G) {
        g -= B.G;
        src += wrap;
      }
    }
  };
  // `arrivals` of the four that a row tile's rows take
  auto publish_q = [&](int t, int arrivals) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane < arrivals) mbar_arrive(&q_full[t]);
  };
  if (warp == 0) {
    // ------------------------------------------------ copies: K_0, V_0, K_1, V_1, ...
    const int page_keys = 1 << B.page_shift, box = page_keys < BK ? page_keys : BK;
    const int groups = BK / box;  // at most 16
    int last_phase[SLOTS] = {-1, -1, -1, -1};
    bool ok = true;
    // the page of this lane's group of tile x, looked up a tile ahead
    auto look_up = [&](const Cursor& x) -> int {
      const int key = (t0 + x.t) * BK + lane * box;
      if (lane >= groups || key >= x.s.kv) return -1;
      const int row = PREFIX ? S.table_row : x.b;
      return B.table[static_cast<long long>(row) * B.max_pages + (key >> B.page_shift)];
    };
    int next = some ? look_up(c) : -1;
    for (int n = 0; left > 0 && ok; ++n) {
      const int base = (t0 + c.t) * BK;
      const int live = max(min(groups, (c.s.kv - base + box - 1) / box), 0);  // groups that hold keys
      const int key = base + lane * box, h = c.h;
      // what the issuing warp has to know of the tile; published with its K
      left = left_behind<C>(B, c, left);
      const uint32_t what = static_cast<uint32_t>((max(min(BK, c.s.kv - base), 0) + 15) / 16) |
                            (c.t + 1 == c.nt || left <= 0 ? I_LAST : 0u) | (rows_of(c) > 128 ? I_TWO : 0u) |
                            (left <= 0 ? I_END : 0u);
      int page = next;
      if (left > 0) {
        advance<C, PREFIX>(B, c);
        next = look_up(c);
      }
      if (lane < live && (page < 0 || page >= B.n_pages)) {
        page = static_cast<int>(B.n_pages);  // past the end: the copy fills with zeros
        atomicOr(status, DEV_ERR_BATCH);
      }
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t i = 2u * n + kv;
        const int slot = i & (SLOTS - 1);
        const uint32_t ph = (i / SLOTS) & 1u;
        if (!W.warp(&empty[slot], ph ^ 1u)) { ok = false; break; }
        if (p.skip_load && i == 0) continue;
        if (lane == 0) {
          if (kv == 0) info[n & 1] = what;
          mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(live * box) * HD * 2);
        }
        __syncwarp();
        last_phase[slot] = static_cast<int>(ph);
        if (lane < live) {
          tma_load_5d(ring(i) + lane * box * (HD * 2), kv ? &tv : &tk, &full[slot], 0, 0, 0,
                      (key & (page_keys - 1)) >> 3, page * B.Hkv + h);
        }
      }
    }
    // every issued copy lands before the block may exit
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (last_phase[i] >= 0) W.drain(&full[i], static_cast<uint32_t>(last_phase[i]));
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------ products of row tile t
    if (some) {
      constexpr uint32_t ID_S = idesc(SK, 0, 0);    // S = Q K^T
      constexpr uint32_t ID_PV = idesc(128, 0, 1);  // O += P V (V: N = hd contiguous)
      const int t = warp - 1;
      uint32_t q_uses = 0, s_cnt = 0, p_cnt = 0;    // half tiles so far: buffer and phase
      // The warp stays together and one lane issues: what a product is told
      // (descriptors: one of each kind, then steps in units of 16 bytes) is the
      // same for all lanes.  The few instructions between two products count:
      // a product takes 32 to 64 cycles.
      const bool leader = elect_one();
      const uint64_t q_desc = kdesc(smem_u32(smem + M_Q + t * TILE_BYTES), 128, 0),
                     k_desc = tile_desc(smem_u32(smem + M_RING), 16), v_desc = tile_desc(smem_u32(smem + M_RING), COL_HALF);
      // S_t of half j of the n-th tile
      auto issue_s = [&](int n, int j, bool seg_ends) {
        const uint32_t buf = s_cnt++ & 1u;
        const uint64_t kd = k_desc + static_cast<uint64_t>(((2u * n) & (SLOTS - 1)) * (TILE_BYTES >> 4) + j * (SK / 8 * GROUP >> 4));
        const uint32_t sd = tmem + t * 128 + buf * SK;
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint64_t q_step = ((ks >> 2) * 128 * 128 + (ks & 3) * 32) >> 4,
                           k_step = ((ks >> 2) * COL_HALF + (ks & 3) * 32) >> 4;
            umma_bf16(sd, q_desc + q_step, kd + k_step, ID_S, ks > 0 ? 1u : 0u);
          }
          umma_commit(&s_full[2 * t + buf]);
          if (seg_ends) umma_commit(&q_empty[t]);
        }
        __syncwarp();
      };
      // O_t += P_t V of half j of the n-th tile
      auto issue_pv = [&](int n, int j, bool first, int steps) -> bool {
        const uint32_t buf = p_cnt & 1u;
        if (!W.warp(&p_full[2 * t + buf], (p_cnt >> 1) & 1u)) return false;
        ++p_cnt;
        tc_fence_after();
        const uint64_t vd = v_desc + static_cast<uint64_t>(((2u * n + 1) & (SLOTS - 1)) * (TILE_BYTES >> 4) + j * (SK / 8 * GROUP >> 4));
        const uint32_t od = tmem + 256 + t * 128, pd = tmem + t * 128 + buf * SK;
        if (leader) {
          if (steps == 4) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_bf16_ta(od, pd + ks * 8, vd + static_cast<uint64_t>(ks * (2 * GROUP >> 4)), ID_PV, ks > 0 ? 1u : (first ? 0u : 1u));
          } else {
#pragma unroll 1
            for (int ks = 0; ks < steps; ++ks)
              umma_bf16_ta(od, pd + ks * 8, vd + static_cast<uint64_t>(ks * (2 * GROUP >> 4)), ID_PV, ks > 0 ? 1u : (first ? 0u : 1u));
          }
          umma_commit(&pv_done[2 * t + buf]);
        }
        __syncwarp();
        return true;
      };
      // row tile t is done with ring entry i: when its products are, or at once
      auto release = [&](uint32_t i, bool active) {
        if (leader) {
          if (active)
            umma_commit(&empty[i & (SLOTS - 1)]);
          else
            mbar_arrive(&empty[i & (SLOTS - 1)]);
        }
        __syncwarp();
      };
      auto wait_tile = [&](uint32_t i) { return W.warp(&full[i & (SLOTS - 1)], (i / SLOTS) & 1u); };
      auto halves = [](uint32_t what) { return (what & I_STEPS) > 4 ? 2 : 1; };
      bool ok = true, first = true;
      uint32_t cur = 0;
      for (int n = 0; ok; ++n) {
        if (first) {
          // a segment begins: both halves of its first S
          if (!(ok = wait_tile(2u * n))) break;
          cur = info[n & 1];
          const bool active = t == 0 || (cur & I_TWO);
          if (active) {
            if (!(ok = W.warp(&q_full[t], q_uses++ & 1u))) break;
            tc_fence_after();
            for (int j = 0; j < halves(cur); ++j) issue_s(n, j, (cur & I_LAST) && j + 1 == halves(cur));
          }
          release(2u * n, active);
        }
        const bool last = cur & I_LAST, active = t == 0 || (cur & I_TWO);
        const int steps = cur & I_STEPS;
        if (!(ok = wait_tile(2u * n + 1))) break;
        uint32_t next = 0;
        if (active) {
          int n_next = 0;
#pragma unroll 1
          for (int j = 0; j < halves(cur); ++j) {
            if (!(ok = issue_pv(n, j, first && j == 0, min(4, steps - 4 * j)))) break;
            if (j == 0 && !last) {
              if (!(ok = wait_tile(2u * n + 2))) break;
              next = info[(n + 1) & 1];
              n_next = halves(next);
            }
            if (j < n_next) issue_s(n + 1, j, (next & I_LAST) && j + 1 == n_next);
          }
          if (!ok) break;
        } else if (!last) {
          if (!(ok = wait_tile(2u * n + 2))) break;
          next = info[(n + 1) & 1];
        }
        release(2u * n + 1, active);
        if (!last) release(2u * n + 2, active);
        if (cur & I_END) break;
        first = last;
        cur = next;
      }
      // all issued products complete before tensor memory is released
      if (leader) umma_commit(&drain[t]);
      __syncwarp();
      W.drain(&drain[t], 0u);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------ query rows of all segments but the first
    uint32_t uses[2] = {0, 0};
    bool fresh = true, ok = true;
    for (int n = 0; left > 0 && ok; ++n) {
      for (int t = 0; fresh && t < 2 && rows_of(c) > t * 128; ++t) {
        // S_t of the segment before that had this row tile is done
        if (n > 0) {
          if (uses[t] && !(ok = W.warp(&q_empty[t], (uses[t] - 1) & 1u))) break;
          fetch_q(c, t, 0, 128);
          publish_q(t, 4);
        }
        ++uses[t];
      }
      fresh = c.t + 1 == c.nt;
      left = left_behind<C>(B, c, left);
      if (left > 0) advance<C, PREFIX>(B, c);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax of row tile t
    const int t = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t sbuf = smem_u32(smem + M_OUT + (warp - 4) * 4096);
    uint32_t cnt = 0;  // half tiles so far: buffer and phase
    if (some && rows_of(c) > t * 128) {
      fetch_q(c, t, quarter * 32, 32);
      publish_q(t, 1);
    }
    const uint64_t scale2 = pack2(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
    bool fresh = true;
    int seg_t = 0, limit = 0;
    int at = -1;  // token * H + head of this thread's row, -1: none
    float m = -INFINITY, l = 0.f;
    for (int n = 0; left > 0; ++n) {
      const int rows = rows_of(c), behind = left_behind<C>(B, c, left);
      const bool last = c.t + 1 == c.nt || behind <= 0;
      if (rows > t * 128) {
        if (fresh) {
          seg_t = c.t;
          m = -INFINITY;
          l = 0.f;
          limit = 0;
          at = -1;
          const int r = t * 128 + quarter * 32 + lane;
          if (r < rows) {
            const int item_row = c.rt * RT_MANY + r, tok = item_row / B.G;
            at = (c.s.q0 + tok) * B.H + c.h * B.G + (item_row - tok * B.G);
            if (PREFIX && S.all_see) {
              limit = c.s.kv;
            } else if (PREFIX) {
              const int b = find_seq(B.cu, B.B, tok);
              if (b < B.B) {
                const Seq s = load_seq(B, b);
                if (tok >= s.q0 && tok < s.q0 + s.qn) limit = min(s.visible(tok - s.q0, B.causal), c.s.kv);
              }
            } else {
              limit = c.s.visible(tok, B.causal);
            }
          }
        }
        const int base0 = (t0 + c.t) * BK, keys = min(BK, c.s.kv - base0);  // V behind them may be anything
        bool ok = true;
#pragma unroll 1
        for (int j = 0; j * SK < keys; ++j, ++cnt) {
          const uint32_t buf = cnt & 1u;
          if (!W.warp(&s_full[2 * t + buf], (cnt >> 1) & 1u)) { ok = false; break; }
          tc_fence_after();
          const uint32_t ts = tl + t * 128 + buf * SK;
          uint32_t ra[32], rb[32];
          tmem_ld32(ts, ra);
          tmem_ld32(ts + 32, rb);
          const int base = base0 + j * SK, from = lo - base, to = limit - base;
          tmem_wait_ld32(ra);
          tmem_wait_ld32(rb);
          if (__any_sync(0xffffffffu, from > 0 || to < SK)) {
            hide(ra, from, to);
            hide(rb, from - 32, to - 32);
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            m4[k & 2] = max3(m4[k & 2], __uint_as_float(ra[k]), __uint_as_float(ra[k + 1]));
            m4[(k & 2) + 1] = max3(m4[(k & 2) + 1], __uint_as_float(rb[k]), __uint_as_float(rb[k + 1]));
          }
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2;
          float alpha = 1.f;
          bool rescale = false;
          if (m == -INFINITY) {
            m = mx;  // the first key that this row sees: O_t and l are still zero (or NaN, from scores that are)
          } else if (mx > m + 8.f) {
            alpha = ex2(m - mx);
            m = mx;
            rescale = true;
          }
          if (__any_sync(0xffffffffu, rescale)) {
            // O_t has to hold the sum up to the half tile before
            const uint32_t was = cnt - 1;
            if (!W.warp(&pv_done[2 * t + (was & 1u)], (was >> 1) & 1u)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < HD; k += 16) {
              uint32_t o[16];
              tmem_ld16(tl + 256 + t * 128 + k, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tl + 256 + t * 128 + k, o);
            }
            tmem_wait_st();
          }
          const float neg_m = m == -INFINITY ? 0.f : -m;  // no key yet: every p is 0
          const uint64_t neg_m2 = pack2(__float_as_uint(neg_m), __float_as_uint(neg_m));
          uint64_t l2[4] = {0, 0, 0, 0};
          // P (two to a cell) goes over the first half of the S it comes from
          auto exponentials = [&](const uint32_t (&r)[32], uint32_t dst) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float e0, e1;
              unpack2(fma2(pack2(r[2 * k], r[2 * k + 1]), scale2, neg_m2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              l2[k & 3] = add2(l2[k & 3], pack2(__float_as_uint(e0), __float_as_uint(e1)));
              // rounded to bf16 for the second product; the sum is taken before
              pk[k] = pack_bf16x2(e0, e1);
            }
            tmem_st16(dst, pk);
          };
          exponentials(ra, ts);
          exponentials(rb, ts + 16);
          tmem_wait_st();
          float la, lb;
          unpack2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])), la, lb);
          l = l * alpha + (la + lb);
          if ((keys & 15) && keys - j * SK <= SK) {
            // (both row tiles' warps: the products of neither wait for the other's)
            const uint32_t i = 2u * n + 1;
            if (!W.warp(&full[i & (SLOTS - 1)], (i / SLOTS) & 1u)) { ok = false; break; }
            const uint32_t vs = smem_u32(ring(i));
            const int tid = threadIdx.x & 127, bad = 16 - (keys & 15);
            for (int k = tid; k < bad * 16; k += 128) st_shared_v4(key_chunk(vs, keys + (k >> 4), k & 15), 0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          tc_fence_before();
          arrive_warp(&p_full[2 * t + buf]);
        }
        if (!ok) break;
        if (last) {
          if (threadIdx.x == 128 && behind <= 0 && p.part.split)
            p.part.split[blockIdx.x] = split_of<C>(B, S, c, seg_t, S.first + S.places - left);
          // ---- the segment's rows: to o, to their own places, or to a slot
          const uint32_t was = cnt - 1;
          if (!W.warp(&pv_done[2 * t + (was & 1u)], (was >> 1) & 1u)) break;
          tc_fence_after();
          const bool whole = seg_t == 0 && c.t + 1 == c.nt;
          const bool direct = whole && !PREFIX && B.shared == 0;
          const long long slot = 2ll * blockIdx.x + (seg_t ? 0 : 1);
          const int row0 = t * 128 + quarter * 32;  // of the warp, in the item
          const float inv = inverse_sum(l, limit > 0);
          // 128 bytes of each of the warp's 32 rows, staged so that eight lanes
          // write a row's together: dst(row of the warp, row among all)
          auto write_rows = [&](auto dst) {
            __syncwarp();
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3), k = lane & 7;
              const uint4 v = ld_shared_v4(sbuf + rr * 128 + ((k ^ (rr & 7)) << 4));
              const int row = __shfl_sync(0xffffffffu, at, rr);
              if (row >= 0) reinterpret_cast<uint4*>(dst(rr, row))[k] = v;
            }
            __syncwarp();
          };
          auto stage = [&](int k, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
            st_shared_v4(sbuf + lane * 128 + ((k ^ (lane & 7)) << 4), a, b, c, d);
          };
#pragma unroll 1
          for (int col = 0; col < HD; col += 16) {
            uint32_t o[16];
            tmem_ld16(tl + 256 + t * 128 + col, o);
            tmem_wait_ld16(o);
            if (direct) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = pack_bf16x2(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
                stage((col & 48) / 8 + k, w[0], w[1], w[2], w[3]);
              }
              if ((col & 48) == 48) write_rows([&](int, int row) { return p.o + static_cast<long long>(row) * HD + col - 48; });
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) stage((col & 16) / 4 + k, o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
              if (col & 16) {
                if (whole) {
                  write_rows([&](int, int row) { return p.part.row_o + static_cast<long long>(row) * HD + col - 16; });
                } else {
                  __syncwarp();
                  uint4* dst = reinterpret_cast<uint4*>(p.part.slot_o) +
                               ((slot * 4 + (col >> 5)) * p.part.slot_rows + row0) * 8 + lane;
#pragma unroll
                  for (int i = 0; i < 8; ++i) dst[32 * i] = ld_shared_v4(sbuf + (32 * i + lane) * 16);
                  __syncwarp();
                }
              }
            }
          }
          if (at >= 0) {
            if (!direct)
              (whole ? p.part.row_ml[at] : p.part.slot_ml[slot * p.part.slot_rows + row0 + lane]) = make_float2(m, l);
            else if (p.lse)
              p.lse[at] = log2_sum_exp(m, l);
          }
          tc_fence_before();
        }
      }
      fresh = last;
      left = behind;
      if (left > 0) advance<C, PREFIX>(B, c);
    }
    __syncwarp();
  }

  if (!PREFIX && S.some_empty && B.shared == 0) write_empty_rows<C>(p, RT_MANY);
  if (p.beside) grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {
int map_pages(CUtensorMap* m, const void* ptr, const Batch& b) {
  const uint64_t page = 1ull << b.page_shift;
  const uint64_t dims[5] = {64, 8, 2, page / 8, static_cast<uint64_t>(b.Hkv) * static_cast<uint64_t>(b.n_pages)};
  const uint64_t str[4] = {HD * 2, 128, 8 * HD * 2, page * HD * 2};
  const uint32_t box[5] = {64, 8, 2, static_cast<uint32_t>((page < BK ? page : BK) / 8), 1};
  return encode_map_5d_bf16(m, ptr, dims, str, box);
}

template <bool PREFIX>
int launch_many_inst(const AttendParams& p, LaunchCtx& ctx, const char* name) {
  CUtensorMap tk, tv;
  int rc;
  if ((rc = map_pages(&tk, p.b.k, p.b)) || (rc = map_pages(&tv, p.b.v, p.b))) return rc;
  static std::atomic<uint64_t> done{0};
  if ((rc = set_smem_once(kv_many_kernel<PREFIX>, M_SMEM, done))) return rc;
  if (ctx.before) ctx.before(ctx.user, name, ctx.stream);
  launch_dep(kv_many_kernel<PREFIX>, dim3(p.part.grid), MANY_THREADS, M_SMEM, ctx.stream, tk, tv, p);
  if (ctx.after) ctx.after(ctx.user, ctx.stream);
  ctx.launches++;
  return cudaPeekAtLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}
}  // namespace

int launch_many(const AttendParams& p, bool prefix, LaunchCtx& ctx, const char* name) {
  return prefix ? launch_many_inst<true>(p, ctx, name) : launch_many_inst<false>(p, ctx, name);
}

}  // namespace kv
}  // namespace tpffn
