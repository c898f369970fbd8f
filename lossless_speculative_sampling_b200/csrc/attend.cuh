// attend.cuh -- attention of a batch of tries (or drafted chains) over a shared prefix, each
// request's own context and the ancestors of each node, on the 5th-generation tensor cores.
//
// out = sum_k exp(s_k - m) v_k / sum_k exp(s_k - m), s = scale q k, in one pass over the keys with
// the running maximum m and sum. attend_plan.cuh says how rows and keys are cut into tiles and
// the tiles shared out. A persistent CTA per SM works on its segments:
//   warp 10     finds the segments, checks their pages and hands them to the others in a ring,
//   warp 11     finds every node's ancestors ahead of the tiles of nodes (a chain of dependent loads,
//               microseconds that no softmax warp has),
//   warp 9      loads: query tiles and 128-token key and value tiles by TMA into a ring of stages
//               (a page of the cache is a box; 32 lanes issue the boxes of a tile side by side),
//   warp 8      issues the matrix products: S = Q K^T and O += P V, both with fp32 accumulators in
//               tensor memory, P read from tensor memory and K, V from shared memory,
//   warps 0-3   the softmax of stream 0, one row per thread, warps 4-7 that of stream 1.
// The two streams keep the tensor cores busy: while one stream's scores become weights, the other
// stream's products run. A pair of query tiles gives each stream a tile of its own, and both read
// the same keys; a single tile (short drafts, single tokens) goes to both streams, whose key tiles
// alternate, and their two results are combined like those of two CTAs.
//
// The running maximum is only raised when a row's scores pass it by more than 2^8 in weight: the
// output accumulated so far is then read from tensor memory, scaled and written back, which most
// tiles skip. Weights and sums stay relative to that maximum, so the result is the same; weights
// are at most 2^8, far inside fp16. They are rounded to the inputs' type for the product with V
// (the tensor cores take 16-bit operands); the sum is of the unrounded ones, in fp32.
//
// Keys that a row does not see get the score -inf; rows of V behind a length are zeroed in shared
// memory before they are multiplied, since their weight of 0 would not silence a NaN.
//
// Measured on a B200 (device time): 16 tries of 61 nodes behind 2K shared and 1K own tokens (32 heads of 128) 77 us,
// 64 tries behind 8K 547-640 us (0.47 to 0.55 of the burst rate of products); 64 single tokens over 8K own
// tokens 232-259 us (0.87 to 0.98 of the copy rate), where nothing but memory counts. In the steady state
// a pair of 128-key tiles takes 3975 cycles: 1576 of exponentials, 1290 until the scores are there,
// 367 for the maximum; the products of both streams need about 2050 and the exponentials 2048, so
// each unit idles half the time, and what bounds it is that a stream has one score tile: its next
// product waits for its weights. Tensor memory holds no third tile beside two outputs of 128
// columns, and more or smaller tiles on more warps were slower.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "attend_plan.cuh"
#include "common.cuh"
#include "psispec.h"
#include "stats.cuh"

namespace psi {

constexpr int kAttendThreads = 384;
// Registers per thread: the softmax warps take what the third warpgroup gives back (168 x 384 at
// launch = 208 x 256 + 88 x 128).
constexpr int kSoftmaxRegs = 208, kHelperRegs = 88;
constexpr float kRaise = 8.0f;  // log2 of how far weights may pass 1 before the maximum is raised

// What a wait inside the kernel is given (about a second), and whether the ancestors of node tiles are handed
// over: a build for tests lowers the one and leaves out the other, so that waits run out.
#ifndef PSISPEC_ATTEND_WAIT_CYCLES
#define PSISPEC_ATTEND_WAIT_CYCLES (1ll << 31)
#endif
#ifndef PSISPEC_ATTEND_HAND_OVER
#define PSISPEC_ATTEND_HAND_OVER 1
#endif
// What the warps that run segments ahead are given besides, for every unit of a CTA's work (which takes up to 2000
// cycles): they wait while whole segments are worked on, which may take longer than a second. The sizes bound
// the units. The other roles' waits are over within a tile's time (with this limit chains took 2% longer).
constexpr long long kUnitCycles = 1 << 14;
// The most ancestors of a node: they are followed one by one, for 32 nodes at a time, so up to four times for a
// query tile and eight for a pair, and the wait for them has to see their end (8 x 2^17 steps of up to 2000
// cycles, several times what a load takes). Lower in a build for tests.
#ifndef PSISPEC_ATTEND_MAX_DEPTH
#define PSISPEC_ATTEND_MAX_DEPTH (1 << 17)
#endif

template <int DP>
struct AttendCfg {
  static constexpr int kHalves = DP / 64;                          // 64-column (128-byte) swizzled blocks of a tile
  static constexpr int kTileBytes = kHalves * kTileKeys * 128;     // a query, key or value tile
  static constexpr int kStages = DP == 128 ? 5 : 10;               // 160 KB of keys and values in flight
  static constexpr int kTiles = 2 + kStages;
  static constexpr int kO = 256;                                   // tensor memory columns: S0, S1, O0, O1
};

struct AttendParams {
  CUtensorMap q, kn, vn, kc, vc;
  AttendShape shape;
  int B, N, Hq, D;
  int pages, page_size, max_pages, prefix_pages;
  int box_log2;      // tokens of a page that one copy loads
  int tile_pages, tile_rest;  // 128 / page_size, 128 % page_size
  int ctas;
  long long wait_cycles;  // the limit of a wait for whole segments
  float scale_log2;  // scale * log2(e)
  const int32_t* node_offsets;
  const int32_t* parent;
  const int32_t* page_table;
  const int32_t* context_len;
  const int32_t* prefix_table;
  const int32_t* prefix_len;
  // workspace
  int4* plan;      // {error, whether the prefix is a group of its own, nodes, gave up}
  int4* info;      // per item: R, first and last CTA, rows of a pair of one tile (0: two tiles)
  int2* node_map;  // per node: its pair's item of key head 0, its place in the pair
  float2* ml;      // per partial row: maximum (log2 units) and sum
  float* part;     // per partial row: D columns
  uint4* seen;     // per CTA, stream and buffer: 128 nodes' ancestors in a node tile
  void* out;
  float* lse;
};

// A segment as the roles read it, from shared memory: they hold only the score tile in registers.
struct AttendWork {
  int last;                      // no segment: the end
  int lo, n, len, ctx_tiles;     // the group
  int pre_tiles, pre_len;        // prefix tiles that the request reads itself
  int req, kvh, item;
  int wide;                      // two query tiles
  int first_node;                // of the pair
  int t0, tiles;                 // key tiles t0 .. t0 + tiles - 1
  int row;                       // of the first partial row here
  int rows[2];                   // partial rows of each stream
  int bad;                       // a length or page out of range: NaN
  int direct;                    // the only piece of its rows: the output itself is written
  int ring;                      // ring slots used before
};
constexpr int kWorkRing = 4;

template <int DP>
struct AttendShared {
  uint64_t q_full[2], q_empty[2], kv_full[AttendCfg<DP>::kStages], kv_empty[AttendCfg<DP>::kStages];
  uint64_t s_full[2], p_full[2], o_full[2], n_full[2][2], n_empty[2][2], v_both, v_one[2], w_full[kWorkRing], w_empty[kWorkRing], done;
  int64_t scan_units[kAttendThreads / 32], scan_joined[kAttendThreads / 32], scan_rows[kAttendThreads / 32];
  int scan_items[kAttendThreads / 32], scan_flags[kAttendThreads / 32];
  int64_t units, start_units, start_rows;
  int start_req, start_items, shared;
  AttendWork work[kWorkRing];
  uint32_t bad_node[2][2][4];    // per stream, alternating: nodes of the query tile with a parent out of range
  uint32_t not_finite[2][2][2][4];  // per width of the pair and stream, alternating: value rows of a node tile
                                    // that are not finite
  uint32_t tmem;
  volatile int dead;
};

template <int DP>
constexpr int attend_smem() {
  return 1024 + AttendCfg<DP>::kTiles * AttendCfg<DP>::kTileBytes + static_cast<int>(sizeof(AttendShared<DP>));
}

// --- tensor core and copy instructions -----------------------------------------------------

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// Shared-memory matrix descriptor: 128-byte swizzle, groups of eight 128-byte rows 1024 bytes
// apart; `lead`: bytes between 64-column blocks (of the value tile, whose columns are contiguous).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return uint64_t((addr >> 4) & 0x3FFF) | (uint64_t((lead >> 4) & 0x3FFF) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// One lane of a converged warp: the compiler then keeps the operands of what it guards in uniform
// registers (behind a lane test each product cost about 150 cycles of issue).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
  return yes != 0;
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}

// One 32-byte store (a whole sector: rows of partial results are far apart within a warp).
__device__ __forceinline__ void store8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
template <bool F16>
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t d;
  if constexpr (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Bounded wait: gives up after the limit, or as soon as another role has given up. A role that gives up
// leaves its loop; copies and products that were issued are waited for (with a limit) by the warps that issued them,
// and the second kernel makes all rows NaN.
__device__ __forceinline__ bool attend_wait(uint64_t* bar, uint32_t parity, volatile int* dead,
                                            long long limit = PSISPEC_ATTEND_WAIT_CYCLES) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > limit) {
      *dead = 1;
      return false;
    }
  }
  return true;
}

// Ring slots of a segment's n key tiles, in the order in which the products use them: a wide pair
// uses a tile's keys and values for both streams before the next tile's; with one query tile the
// streams alternate, so the next tile's keys come before this tile's values.
__device__ __forceinline__ int k_slot(bool wide, int t) { return wide ? 2 * t : (t == 0 ? 0 : 2 * t - 1); }
__device__ __forceinline__ int v_slot(bool wide, int t, int n) { return wide ? 2 * t + 1 : (t < n - 1 ? 2 * t + 2 : 2 * n - 1); }

struct AttendLoad {
  const AttendParams& p;
  int pre_len;  // tokens of the prefix that every request reads itself
  __device__ __forceinline__ AttendGroup operator()(int req) const {
    if (req < 0) {
      if (p.prefix_pages == 0) return make_group(0, 0, 0, 0, true);
      const int nodes = __ldg(p.node_offsets + p.B);
      return make_group(0, nodes, __ldg(p.prefix_len), int64_t(p.prefix_pages) * p.page_size, true);
    }
    const int lo = __ldg(p.node_offsets + req);
    return make_group(lo, __ldg(p.node_offsets + req + 1) - lo, __ldg(p.context_len + req),
                      int64_t(p.max_pages) * p.page_size, false, pre_len);
  }
};

// Finds the CTA's place on the line of units: every CTA adds up all groups (a thread takes
// consecutive requests), with the prefix as a group of its own and as every request's first tiles,
// and the way of fewer units is taken. False if offsets or the prefix's length are out of range, or
// there is nothing for this CTA; CTA 0 notes for the second kernel what it needs.
template <int DP>
__device__ bool attend_place(const AttendParams& p, AttendShared<DP>& sh, AttendLoad& load, AttendWalk& walk,
                             int* active) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kAttendThreads / 32;
  const int per = (p.B + kAttendThreads - 1) / kAttendThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int flags = 0;  // 1: bad offsets, 2: a pair of two tiles, 4: a bad length of the prefix
  AttendSize pre{0, 0, 0};
  int pre_len = 0;
  if (p.prefix_pages > 0) {
    const int nodes = __ldg(p.node_offsets + p.B);
    const AttendGroup g = load(-1);
    if (nodes < 0 || nodes > p.N) {
      flags |= 1;
    } else if (g.bad) {
      flags |= 4;
    } else {
      pre = group_size(g, p.shape);
      pre_len = g.len;
      if (g.query_tiles(p.shape) > 1) flags |= 2;
    }
  }
  AttendSize sum{0, 0, 0};
  int64_t joined = 0;
  for (int b = b0; b < b1; ++b) {
    const int lo = __ldg(p.node_offsets + b), hi = __ldg(p.node_offsets + b + 1), len = __ldg(p.context_len + b);
    if (lo > hi || lo < 0 || hi > p.N || (b == 0 && lo != 0)) {
      flags |= 1;
      continue;
    }
    AttendGroup g = make_group(lo, hi - lo, len, int64_t(p.max_pages) * p.page_size, false);
    const AttendSize z = group_size(g, p.shape);
    sum.units += z.units;
    sum.rows += z.rows;
    sum.items += z.items;
    if (g.query_tiles(p.shape) > 1) flags |= 2;
    g.ctx_tiles += (pre_len + kTileKeys - 1) / kTileKeys;
    joined += group_size(g, p.shape).units;
  }
  AttendSize inc = sum;
  int64_t inc_joined = joined;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, inc.units, o), r = __shfl_up_sync(0xffffffffu, inc.rows, o);
    const int64_t j = __shfl_up_sync(0xffffffffu, inc_joined, o);
    const int i = __shfl_up_sync(0xffffffffu, inc.items, o);
    if (lane >= o) {
      inc.units += u;
      inc.rows += r;
      inc.items += i;
      inc_joined += j;
    }
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 31) {
    sh.scan_units[warp] = inc.units;
    sh.scan_joined[warp] = inc_joined;
    sh.scan_rows[warp] = inc.rows;
    sh.scan_items[warp] = inc.items;
    sh.scan_flags[warp] = flags;
  }
  __syncthreads();
  AttendSize base{0, 0, 0};  // before this thread's requests
  int64_t base_joined = 0, units = 0, all_joined = 0;
  flags = 0;
  const int used = min(kWarps, (p.B + 32 * per - 1) / (32 * per));  // warps that have requests
  for (int w = 0; w < used; ++w) {
    if (w < warp) {
      base.units += sh.scan_units[w];
      base_joined += sh.scan_joined[w];
      base.rows += sh.scan_rows[w];
      base.items += sh.scan_items[w];
    }
    units += sh.scan_units[w];
    all_joined += sh.scan_joined[w];
  }
#pragma unroll
  for (int w = 0; w < kWarps; ++w) flags |= sh.scan_flags[w];
  base.units += inc.units - sum.units;
  base_joined += inc_joined - joined;
  base.rows += inc.rows - sum.rows;
  base.items += inc.items - sum.items;
  // (a row's partial results of the prefix, written and added again, cost a sixteenth of a unit.) Measured,
  // as a group of its own against in every request: 32 chains of 9 rows behind 16K 101 us against 437,
  // 16 tries of 244 rows behind 2K 103 against 80; near the bound the two are equal
  const bool shared = pre.units > 0 && all_joined > pre.units + units + pre.rows / 16;
  if (shared) {
    units += pre.units;
    base.units += pre.units;
    base.rows += pre.rows;
    base.items += pre.items;
  } else {
    pre.units = 0;
    units = all_joined;
    sum.units = joined;
    base.units = base_joined;
    load.pre_len = pre_len;
  }
  // (bad offsets tell no rows apart: all N become NaN; of a bad prefix those of the requests)
  const bool err = (flags & 5) != 0;
  if (blockIdx.x == 0 && tid == 0)
    *p.plan = make_int4(err, shared, flags & 1 ? p.N : __ldg(p.node_offsets + p.B), 0);
  const int C = active_ctas(units, (flags & 2) != 0, p.ctas);
  *active = C;
  if (err || static_cast<int>(blockIdx.x) >= C) return false;
  const int64_t w0 = cta_first_unit(units, blockIdx.x, C), w1 = cta_first_unit(units, blockIdx.x + 1, C);
  if (tid == 0) {
    sh.units = units;
    sh.shared = shared;
    if (w0 < pre.units) {
      sh.start_req = -1;
      sh.start_units = sh.start_rows = 0;
      sh.start_items = 0;
    }
  }
  if (w0 >= base.units && w0 < base.units + sum.units) {  // the thread whose requests hold the first unit
    int b = b0;
    for (; b + 1 < b1; ++b) {  // (the last one needs no look)
      const AttendSize z = group_size(load(b), p.shape);
      if (w0 < base.units + z.units) break;
      base.units += z.units;
      base.rows += z.rows;
      base.items += z.items;
    }
    sh.start_req = b;
    sh.start_units = base.units;
    sh.start_rows = base.rows;
    sh.start_items = base.items;
  }
  __syncthreads();
  walk.start(p.shape, p.B, w0, w1, sh.start_req, sh.start_units, sh.start_rows, sh.start_items, load);
  return true;
}

// Bits of the nodes of key tile `base` (request-local nodes base .. base + 127) that node i sees:
// itself and its ancestors. False if a parent is out of range or there are too many.
__device__ __forceinline__ bool ancestor_bits(const int32_t* parent, int i, int base, uint32_t (&bits)[4]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) bits[w] = 0;
  if (parent == nullptr) {  // a chain
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int n = i - (base + 32 * w);
      bits[w] = n < 0 ? 0u : (n >= 31 ? 0xffffffffu : (2u << n) - 1u);
    }
    return true;
  }
  for (int steps = 0; i >= base; ++steps) {
    const int k = i - base;
    if (k < kTileKeys) {
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if ((k >> 5) == w) bits[w] |= 1u << (k & 31);
    }
    const int up = __ldg(parent + i);
    if (up < -1 || up >= i || (up >= 0 && steps == PSISPEC_ATTEND_MAX_DEPTH)) return false;
    i = up;
  }
  return true;
}

// A softmax warp: rows 32 wq .. 32 wq + 31 of stream s, one per lane.
template <int DP, bool F16>
__device__ __forceinline__ void attend_softmax(const AttendParams& p, AttendShared<DP>& sh, uint8_t* tiles, uint32_t tmem,
                                               volatile int* dead) {
  using Cfg = AttendCfg<DP>;
  const int G = p.shape.G, npt = p.shape.npt;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
  const int node_in = r / G, head_in = r % G;
  const uint32_t lanes = uint32_t(wq * 32) << 16;
  const uint32_t t_s = tmem + lanes + s * 128, t_o = tmem + lanes + Cfg::kO + s * DP;
  const float c = p.scale_log2;
  const f32x2 cc = pack2(c, c);
  uint32_t s_uses = 0, o_uses = 0, n_uses = 0, v_uses[2] = {0, 0};
  bool ok = true;
  for (int at = 0;; ++at) {
    const AttendWork& w = sh.work[at % kWorkRing];
    ok = __all_sync(0xffffffffu, attend_wait(&sh.w_full[at % kWorkRing], (at / kWorkRing) & 1, dead));
    if (!ok || w.last) break;
    const bool wide = w.wide;
    const int n = w.tiles, steps = wide ? n : (n + 1 - s) / 2;
    const int rows = w.rows[s];
    const bool valid = r < rows, live = wq * 32 < rows;
    const int node = w.first_node + (wide ? s * npt : 0) + node_in;  // of the group
    bool bad = w.bad;
    if (w.t0 == 0 && w.req >= 0 && w.kvh == 0 && valid && head_in == 0 && (wide || s == 0))
      p.node_map[w.lo + node] = make_int2(w.item, (wide ? s * npt : 0) + node_in);
    float m = -INFINITY, l = 0.0f;
    for (int i = 0; i < steps; ++i) {
      const int tt = wide ? i : 2 * i + s, t = w.t0 + tt;
      const bool is_node = t >= w.ctx_tiles;
      const bool is_pre = t < w.pre_tiles;
      const int base = (is_node ? t - w.ctx_tiles : is_pre ? t : t - w.pre_tiles) * kTileKeys;
      const int count = (is_node ? w.n : is_pre ? w.pre_len : w.len) - base;  // keys of the tile, if below 128
      uint32_t bits[4];
      if (is_node) {
        const int buf = n_uses & 1;
        ok = __all_sync(0xffffffffu, attend_wait(&sh.n_full[s][buf], (n_uses >> 1) & 1, dead));
        if (!ok) break;
        ++n_uses;
        const uint4 x4 = p.seen[((blockIdx.x * 2 + s) * 2 + buf) * kTileRows + node_in];
        const uint32_t wrong = *const_cast<volatile uint32_t*>(&sh.bad_node[s][buf][node_in >> 5]);
        bits[0] = x4.x, bits[1] = x4.y, bits[2] = x4.z, bits[3] = x4.w;
        if (valid && ((wrong >> (node_in & 31)) & 1u)) bad = true;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.n_empty[s][buf]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = count - 32 * j;
          bits[j] = k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u);
        }
      }
      ok = __all_sync(0xffffffffu, attend_wait(&sh.s_full[s], s_uses & 1, dead));
      if (!ok) break;
      ++s_uses;
      tmem_fence_after();
      if (live) {
        float x[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(t_s + 32 * k, x + 32 * k);
        tmem_wait_ld();
        if (is_node || count < kTileKeys) {
#pragma unroll
          for (int k = 0; k < 128; ++k) x[k] = (bits[k >> 5] >> (k & 31)) & 1u ? x[k] : -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 8) {
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = max3(mx[j], x[k + 2 * j], x[k + 2 * j + 1]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        const bool raise = valid && (m == -INFINITY ? top > -INFINITY : top > m + kRaise);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2(m - top) : 1.0f;  // (0 for the first keys)
          if (raise) {
            m = top;
            l *= f;
          }
          if (i > 0) {
#pragma unroll 1
            for (int k = 0; k < DP; k += 32) {
              float o[32];
              tmem_ld32(t_o + k, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= f;
              tmem_st32(t_o + k, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
        const float mu = m == -INFINITY ? 0.0f : m;
        const f32x2 neg = pack2(-mu, -mu);
        f32x2 sum[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float a, b;
            unpack2(fma2(pack2(x[64 * h + 2 * k], x[64 * h + 2 * k + 1]), cc, neg), a, b);
            a = ex2(a);
            b = ex2(b);
            sum[k & 1] = add2(sum[k & 1], pack2(a, b));
            pk[k] = pack_half<F16>(a, b);
          }
          tmem_st32(t_s + 32 * h, pk);
        }
        float a, b;
        unpack2(add2(sum[0], sum[1]), a, b);
        l += a + b;
        tmem_wait_st();
      }
      if (is_node || count < kTileKeys) {  // rows of V that must not be multiplied
        const int slot = w.ring + v_slot(wide, tt, n), st = slot % Cfg::kStages;
        ok = __all_sync(0xffffffffu, attend_wait(&sh.kv_full[st], (slot / Cfg::kStages) & 1, dead));
        if (!ok) break;
        uint8_t* const row = tiles + (2 + st) * Cfg::kTileBytes + r * 128;
        bool drop = r >= count;
        if (is_node) {
          // Values that are not finite: a thread looks through its row, in a pair of two tiles each
          // stream through half of it. All warps that use the tile meet before one zeroes a row (their
          // words alternate between two places, so one that is ahead writes none that another reads).
          constexpr int kUnits = 8 * Cfg::kHalves;
          const int use = v_uses[wide], buf = use & 1;
          const int u0 = wide ? s * (kUnits / 2) : 0, u1 = wide ? u0 + kUnits / 2 : kUnits;
          uint32_t most = 0;  // two largest magnitudes, as bits
          for (int k = u0; k < u1; ++k) {
            const uint4 y = *reinterpret_cast<const uint4*>(row + (k >> 3) * kTileKeys * 128 + ((k + r) & 7) * 16);
            most = __vmaxu2(__vmaxu2(most, y.x & 0x7FFF7FFFu), __vmaxu2(y.y & 0x7FFF7FFFu, y.z & 0x7FFF7FFFu));
            most = __vmaxu2(most, y.w & 0x7FFF7FFFu);
          }
          constexpr uint32_t inf = F16 ? 0x7C00u : 0x7F80u;
          const bool nf = !drop && ((most & 0xFFFFu) >= inf || (most >> 16) >= inf);
          const uint32_t word = __ballot_sync(0xffffffffu, nf);
          uint64_t* const met = wide ? &sh.v_both : &sh.v_one[s];
          if (lane == 0) {
            sh.not_finite[wide][s][buf][wq] = word;
            mbar_arrive(met);
          }
          ok = __all_sync(0xffffffffu, attend_wait(met, use & 1, dead));
          if (!ok) break;
          ++v_uses[wide];
          const volatile uint32_t* mine = sh.not_finite[wide][s][buf];
          const volatile uint32_t* other = wide ? sh.not_finite[wide][s ^ 1][buf] : mine;
          uint32_t seen = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) seen |= bits[k] & (mine[k] | other[k]);
          if (valid && seen) bad = true;
          drop = drop || (((mine[wq] | other[wq]) >> lane) & 1u);
        }
        if (drop) {
#pragma unroll
          for (int h = 0; h < Cfg::kHalves; ++h)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(row + h * kTileKeys * 128 + ((k + r) & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[s]);
    }
    if (!ok) break;
    const int64_t slot_row = w.row + (s ? w.rows[0] : 0) + r;
    const int64_t out_row = int64_t(w.lo + node) * p.Hq + w.kvh * G + head_in;  // of a wide pair
    if (steps > 0) {
      ok = __all_sync(0xffffffffu, attend_wait(&sh.o_full[s], o_uses & 1, dead));
      if (!ok) break;
      ++o_uses;
      tmem_fence_after();
      if (live && w.direct) {
        const float inv = bad ? NAN : 1.0f / l;
        const bool none = !bad && l == 0.0f;  // no key has weight: 0, whatever the products left
        uint16_t* dst = static_cast<uint16_t*>(p.out) + out_row * p.D;
#pragma unroll 1
        for (int k = 0; k < DP; k += 32) {
          float o[32];
          tmem_ld32(t_o + k, o);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              if (k + j >= p.D) break;
#pragma unroll
              for (int i = j; i < j + 8; ++i) o[i] = none ? 0.0f : o[i] * inv;
              uint4 v;
              v.x = pack_half<F16>(o[j], o[j + 1]);
              v.y = pack_half<F16>(o[j + 2], o[j + 3]);
              v.z = pack_half<F16>(o[j + 4], o[j + 5]);
              v.w = pack_half<F16>(o[j + 6], o[j + 7]);
              *reinterpret_cast<uint4*>(dst + k + j) = v;
            }
          }
        }
      } else if (live) {
        float* dst = p.part + slot_row * p.D;
#pragma unroll 1
        for (int k = 0; k < DP; k += 32) {
          float o[32];
          tmem_ld32(t_o + k, o);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              if (k + j < p.D) store8(dst + k + j, o + j);
          }
        }
      }
    }
    if (valid && w.direct) {
      if (p.lse) p.lse[out_row] = bad ? NAN : (m + log2f(l)) * 0.6931471805599453f;
    } else if (valid) {
      p.ml[slot_row] = make_float2(bad ? 0.0f : m, bad ? NAN : l);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.w_empty[at % kWorkRing]);
  }
}

template <int DP, bool F16>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_tree_kernel(const __grid_constant__ AttendParams p) {
  using Cfg = AttendCfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  AttendShared<DP>& sh = *reinterpret_cast<AttendShared<DP>*>(tiles + Cfg::kTiles * Cfg::kTileBytes);
  const uint32_t q_addr = smem_u32(tiles), kv_addr = q_addr + 2 * Cfg::kTileBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* dead = &sh.dead;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_full[i], 1);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&sh.n_full[i][j], 1);
        mbar_init(&sh.n_empty[i][j], 4);
      }
    }
    for (int i = 0; i < Cfg::kStages; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 1);
    }
    for (int i = 0; i < kWorkRing; ++i) {
      mbar_init(&sh.w_full[i], 1);
      mbar_init(&sh.w_empty[i], 11);  // 8 softmax warps, products, loads, nodes
    }
    mbar_init(&sh.v_both, 8);
    mbar_init(&sh.v_one[0], 4);
    mbar_init(&sh.v_one[1], 4);
    mbar_init(&sh.done, 1);
    sh.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the second kernel waits for this one's end
  AttendLoad load{p, 0};
  AttendWalk walk;
  int C = 0;
  if (!attend_place<DP>(p, sh, load, walk, &C)) return;  // the same in every thread
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;
  const int G = p.shape.G, npt = p.shape.npt;
  int at = 0;          // segments taken
  bool ok = true;
  // the next segment, null at the end
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, attend_wait(bar, parity, dead)) != 0;
  };
  auto wait_segments = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, attend_wait(bar, parity, dead, p.wait_cycles)) != 0;
  };
  auto take = [&](bool ahead = false) -> const AttendWork* {
    const int i = at % kWorkRing;
    ok = ahead ? wait_segments(&sh.w_full[i], (at / kWorkRing) & 1) : wait_all(&sh.w_full[i], (at / kWorkRing) & 1);
    return ok && !sh.work[i].last ? &sh.work[i] : nullptr;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kHelperRegs));
    if (warp == 10) {
      // ----- segments -----
      AttendSegment seg;
      int ring = 0;
      for (bool more = true; more && ok; ++at) {
        more = walk.next(seg, load);
        const int i = at % kWorkRing;
        ok = wait_segments(&sh.w_empty[i], ((at / kWorkRing) & 1) ^ 1);
        if (!ok) break;
        bool off = more && seg.g.bad;
        const int pre_tiles = more ? seg.g.pre_tiles : 0;
        auto check = [&](const int32_t* table, int t0, int t1, int len) {  // the pages that the segment reads
          const int64_t from = int64_t(t0) * kTileKeys, end = min(int64_t(len), int64_t(t1) * kTileKeys);
#pragma unroll 4
          for (int64_t k = from / p.page_size + lane; k * p.page_size < end; k += 32) {
            const int page = __ldg(table + k);
            off |= page < 0 || page >= p.pages;
          }
        };
        if (more && seg.t0 < pre_tiles) check(p.prefix_table, seg.t0, min(seg.t1, pre_tiles), load.pre_len);
        if (more && seg.t1 > pre_tiles && seg.t0 < seg.g.ctx_tiles)
          check(seg.req < 0 ? p.prefix_table : p.page_table + int64_t(seg.req) * p.max_pages,
                max(seg.t0 - pre_tiles, 0), seg.t1 - pre_tiles, seg.g.len);
        off = __any_sync(0xffffffffu, off);
        if (lane == 0) {
          AttendWork& w = sh.work[i];
          w.last = !more;
          if (more) {
            const int rest = seg.g.n - seg.first_node;
            w.lo = seg.g.lo;
            w.n = seg.g.n;
            w.len = seg.g.len;
            w.ctx_tiles = seg.g.ctx_tiles;
            w.pre_tiles = pre_tiles;
            w.pre_len = load.pre_len;
            w.req = seg.req;
            w.kvh = seg.kvh;
            w.item = seg.item;
            w.wide = seg.q_tiles == 2;
            w.first_node = seg.first_node;
            w.t0 = seg.t0;
            w.tiles = seg.t1 - seg.t0;
            w.row = static_cast<int>(seg.row) + kItemRows * blockIdx.x;
            w.rows[0] = min(npt, rest) * G;
            w.rows[1] = (seg.q_tiles == 2 ? min(npt, rest - npt) : min(npt, rest)) * G;
            w.bad = off;
            w.direct = !sh.shared && w.wide && seg.t0 == 0 && seg.t1 == seg.g.key_tiles();
            w.ring = ring;
          }
          mbar_arrive(&sh.w_full[i]);
          if (more && seg.t0 == 0) {
            const int64_t units = sh.units;
            p.info[seg.item] = make_int4(static_cast<int>(seg.row), cta_of_unit(units, seg.u0, C),
                                         cta_of_unit(units, seg.u0 + int64_t(seg.g.key_tiles() - 1) * seg.q_tiles, C),
                                         seg.q_tiles == 2 ? 0 : min(npt, seg.g.n - seg.first_node) * G);
          }
        }
        __syncwarp();
        ring += more ? 2 * (seg.t1 - seg.t0) : 0;
      }
    } else if (warp == 11) {
      // ----- nodes -----
      uint32_t uses[2] = {0, 0};
      while (const AttendWork* w = take(true)) {
        const int lo = w->lo, n = w->n, first = w->first_node, t0 = w->t0, end = t0 + w->tiles;
        const bool wide = w->wide;
        const int32_t* parent = p.parent ? p.parent + lo : nullptr;
        for (int t = max(t0, w->ctx_tiles); t < end && ok; ++t) {
          const int base = (t - w->ctx_tiles) * kTileKeys;
          for (int s = wide ? 0 : (t - t0) & 1; s <= (wide ? 1 : (t - t0) & 1); ++s) {
            const int buf = uses[s] & 1, from = first + (wide ? s * npt : 0), nodes = min(npt, n - from);
            ok = wait_segments(&sh.n_empty[s][buf], ((uses[s] >> 1) & 1) ^ 1);
            if (!ok) break;
            ++uses[s];
            for (int k = 0; 32 * k < nodes; ++k) {
              const int i = 32 * k + lane;
              uint32_t bits[4];
              bool wrong = false;
              if (i < nodes) {
                wrong = !ancestor_bits(parent, from + i, base, bits);
                p.seen[((blockIdx.x * 2 + s) * 2 + buf) * kTileRows + i] = make_uint4(bits[0], bits[1], bits[2], bits[3]);
              }
              const uint32_t word = __ballot_sync(0xffffffffu, wrong);
              if (lane == 0) sh.bad_node[s][buf][k] = word;
            }
            __syncwarp();
            if (PSISPEC_ATTEND_HAND_OVER && lane == 0) mbar_arrive(&sh.n_full[s][buf]);
          }
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&sh.w_empty[at % kWorkRing]);
        ++at;
      }
    } else if (warp == 9) {
      // ----- loads -----
      int slots = 0, st = 0;  // ring slots that were loaded, and the stage and turn of the next one
      uint32_t turn = 0;
      uint32_t q_uses[2] = {0, 0};
      int narrow = 0;  // query buffer of the next single tile (they alternate)
      const int half = lane % Cfg::kHalves, in_tile = (lane / Cfg::kHalves) << p.box_log2;
      while (const AttendWork* w = take()) {
        const bool wide = w->wide;
        const int n = w->tiles, kvh = w->kvh;
        for (int i = 0; i < (wide ? 2 : 1) && ok; ++i) {
          const int buf = wide ? i : narrow;
          ok = wait_all(&sh.q_empty[buf], (q_uses[buf] & 1) ^ 1);
          if (!ok) break;
          ++q_uses[buf];
          const uint32_t dst = q_addr + buf * Cfg::kTileBytes;
          if (lane == 0) mbar_expect_tx(&sh.q_full[buf], Cfg::kHalves * npt * G * 128);
          __syncwarp();
          if (lane < Cfg::kHalves)
            tma_3d(dst + lane * kTileKeys * 128, &p.q, lane * 64, kvh * G, w->lo + w->first_node + i * npt,
                   &sh.q_full[buf]);
        }
        if (!wide) narrow ^= 1;
        const int32_t* const own = w->req < 0 ? p.prefix_table : p.page_table + int64_t(w->req) * p.max_pages;
        const int ctx_tiles = w->ctx_tiles, len = w->len, t0 = w->t0, lo = w->lo;
        const int pre_tiles = w->pre_tiles, pre_len = w->pre_len;
        // each lane loads one box of 64 columns of a tile of the cache; its page and its token in the
        // page move on tile by tile, and pages are looked up a tile ahead
        const int32_t* table = t0 < pre_tiles ? p.prefix_table : own;
        int token = (t0 < pre_tiles ? t0 : t0 - pre_tiles) * kTileKeys + in_tile;  // of the next tile
        int entry = token / p.page_size, in_page = token - entry * p.page_size;
        auto look_up = [&](int t) {
          return t < ctx_tiles && in_tile < kTileKeys && token < (t < pre_tiles ? pre_len : len) ? __ldg(table + entry) : 0;
        };
        // one tile of keys or values into the next stage: `left` tokens of the cache, none: nodes
        auto put = [&](const CUtensorMap* cache, const CUtensorMap* nodes, int t, int left, int page, int at_page) {
          uint64_t* const bar = &sh.kv_full[st];
          const uint32_t dst = kv_addr + st * Cfg::kTileBytes + half * kTileKeys * 128;
          if (!wait_all(&sh.kv_empty[st], turn ^ 1)) return false;
          if (lane == 0)
            mbar_expect_tx(bar, left == 0 || left >= kTileKeys
                                    ? Cfg::kTileBytes
                                    : (Cfg::kHalves * ((left + (1 << p.box_log2) - 1) >> p.box_log2)) << (p.box_log2 + 7));
          __syncwarp();
          if (left > 0) {
            if (in_tile < min(left, kTileKeys)) tma_4d(dst + in_tile * 128, cache, half * 64, at_page, kvh, page, bar);
          } else if (lane < Cfg::kHalves) {
            tma_3d(dst, nodes, half * 64, kvh, lo + (t - ctx_tiles) * kTileKeys, bar);
          }
          ++slots;
          if (++st == Cfg::kStages) {
            st = 0;
            turn ^= 1;
          }
          return true;
        };
        // in the order of use: K0 V0 K1 V1 ..., or K0 K1 V0 K2 V1 ... with one query tile
        int page_next = look_up(t0), page = 0, at_page = 0, left = 0;
        const int end = t0 + n;
        for (int t = t0; t <= end; ++t) {
          const int page_before = page, at_before = at_page, left_before = left;
          if (t < end) {
            page = page_next < 0 || page_next >= p.pages ? 0 : page_next;  // (a bad page's rows become NaN)
            at_page = in_page;
            left = t < pre_tiles ? pre_len - t * kTileKeys : t < ctx_tiles ? len - (t - pre_tiles) * kTileKeys : 0;
            token += kTileKeys;
            entry += p.tile_pages;
            in_page += p.tile_rest;
            if (in_page >= p.page_size) {
              in_page -= p.page_size;
              ++entry;
            }
            if (t + 1 == pre_tiles) {  // from the prefix's last tile to the first of its own
              table = own;
              token = in_tile;
              entry = in_tile / p.page_size;
              in_page = in_tile - entry * p.page_size;
            }
            if (t + 1 < end) page_next = look_up(t + 1);
            ok = put(&p.kc, &p.kn, t, left, page, at_page);
          }
          if (wide ? t < end : t > t0)
            ok = ok && (wide ? put(&p.vc, &p.vn, t, left, page, at_page)
                             : put(&p.vc, &p.vn, t - 1, left_before, page_before, at_before));
          if (!ok) break;
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&sh.w_empty[at % kWorkRing]);
        ++at;
      }
      // no copy may still land when the CTA leaves; where another role gives up, even later than here, nobody
      // else has waited for the last ones
      for (int i = 0; i < 2; ++i)
        if (q_uses[i]) mbar_wait_bounded(&sh.q_full[i], (q_uses[i] - 1) & 1);
      for (int i = max(slots - Cfg::kStages, 0); i < slots; ++i)
        mbar_wait_bounded(&sh.kv_full[i % Cfg::kStages], (i / Cfg::kStages) & 1);
    } else if (warp == 8) {
      // ----- matrix products -----
      constexpr uint32_t fmt = F16 ? 0u : 1u;
      constexpr uint32_t common = (1u << 4) | (fmt << 7) | (fmt << 10) | ((kTileRows / 16) << 24);
      constexpr uint32_t qk_desc = common | ((kTileKeys / 8) << 17);
      constexpr uint32_t pv_desc = common | (1u << 16) | ((DP / 8) << 17);
      uint32_t p_uses[2] = {0, 0}, q_uses[2] = {0, 0};
      int narrow = 0;
      while (const AttendWork* w = take()) {
        const bool wide = w->wide;
        const int n = w->tiles, steps = wide ? 2 * n : n, ring = w->ring;
        const int qbuf = narrow;
        __syncwarp();
        if (elect_one()) mbar_arrive(&sh.w_empty[at % kWorkRing]);
        ++at;
        if (wide) {
          ok = wait_all(&sh.q_full[0], q_uses[0] & 1) && wait_all(&sh.q_full[1], q_uses[1] & 1);
          ++q_uses[0];
          ++q_uses[1];
        } else {
          ok = wait_all(&sh.q_full[qbuf], q_uses[qbuf] & 1);
          ++q_uses[qbuf];
          narrow ^= 1;
        }
        auto scores = [&](int g) {  // S of step g
          const int s = g & 1, t = wide ? g >> 1 : g;
          const int slot = ring + k_slot(wide, t), st = slot % Cfg::kStages;
          if (!wait_all(&sh.kv_full[st], (slot / Cfg::kStages) & 1)) return false;
          tmem_fence_after();
          const uint32_t a = q_addr + (wide ? s : qbuf) * Cfg::kTileBytes, b = kv_addr + st * Cfg::kTileBytes;
          const uint64_t da = smem_desc(a, 16), db = smem_desc(b, 16);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
              const uint32_t off = ((k / 4) * kTileKeys * 128 + (k % 4) * 32) >> 4;
              mma_ss(tmem + s * 128, da + off, db + off, qk_desc, k > 0);
            }
            mma_commit(&sh.s_full[s]);
            if (!wide || s == 1) mma_commit(&sh.kv_empty[st]);
            if (wide ? t == n - 1 : g == steps - 1) mma_commit(&sh.q_empty[wide ? s : qbuf]);
          }
          __syncwarp();
          return true;
        };
        ok = ok && scores(0);
        if (steps > 1) ok = ok && scores(1);
        for (int g = 0; g < steps && ok; ++g) {
          const int s = g & 1, t = wide ? g >> 1 : g;
          const int slot = ring + v_slot(wide, t, n), st = slot % Cfg::kStages;
          ok = wait_all(&sh.p_full[s], p_uses[s] & 1) && wait_all(&sh.kv_full[st], (slot / Cfg::kStages) & 1);
          ++p_uses[s];
          if (!ok) break;
          tmem_fence_after();
          const uint32_t b = kv_addr + st * Cfg::kTileBytes;
          const uint64_t db = smem_desc(b, kTileKeys * 128);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTileKeys / 16; ++k)
              mma_ts(tmem + Cfg::kO + s * DP, tmem + s * 128 + k * 8, db + ((k * 2048) >> 4), pv_desc, g >= 2 || k > 0);
            if (!wide || s == 1) mma_commit(&sh.kv_empty[st]);
            if (g + 2 >= steps) mma_commit(&sh.o_full[s]);
          }
          __syncwarp();
          if (g + 2 < steps) ok = scores(g + 2);
        }
        if (!ok) break;
      }
      if (elect_one()) mma_commit(&sh.done);  // every product has finished before the CTA leaves
      __syncwarp();
      mbar_wait_bounded(&sh.done, 0);
    }
    __syncwarp();
  } else {
    // ----- softmax -----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    attend_softmax<DP, F16>(p, sh, tiles, tmem, dead);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (tid == 0 && sh.dead) p.plan->w = 1;  // gave up: the second kernel answers NaN
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Second kernel: one warp per (node, head) combines the row's partial results, lanes over the
// columns, kBatch pieces at a time. Few rows have many pieces each, and a warp that goes through
// them a few at a time waits for memory every time; of many rows it is the blocks per SM that hide
// it. So up to one block per SM a warp takes 16 pieces at once, up to four 8, else 4 with five
// blocks per SM. Measured (us of the whole call; 16, 8, 4): one token over 4K 18.6, 20.5, 26.0; one
// trie of 33 nodes (1056 rows) 19.1, 20.2, 22.4; two of them 21.1, 20.7, 22.4; four of them 8: 22.3, 4:
// 23.2; six of them 24.9, 24.2.
constexpr int kCombineWarps = 8;

template <bool F16, int kBatch, int kBlocks>
__global__ void __launch_bounds__(kCombineWarps * 32, kBlocks) attend_combine_kernel(const __grid_constant__ AttendParams p) {
  const int64_t w = int64_t(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, Hkv = p.shape.Hkv, G = p.shape.G, npt = p.shape.npt;
  const int n = static_cast<int>(w / p.Hq), h = static_cast<int>(w % p.Hq), kvh = h / G, g = h % G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n >= p.N) return;
  // (loads that do not need each other first: the node's entry is read before it is known to exist)
  const int4 plan = *p.plan;
  const int2 map = p.node_map[n];
  if (n >= plan.z) return;  // behind the last request
  const bool err = plan.x != 0 || plan.w != 0;
  // the row's places: first the prefix's, then its request's
  int first[2] = {0, 0}, count[2] = {0, 0}, narrow[2] = {0, 0};
  if (!err) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 0 && plan.y == 0) continue;
      const int4 info = p.info[(k == 0 ? n / npt / 2 * Hkv : map.x) + kvh];
      if (k == 1 && plan.y == 0 && info.w == 0 && info.y == info.z) return;  // one piece: written already
      first[k] = info.x + kItemRows * info.y + (k == 0 ? n % (2 * npt) : map.y) * G + g;
      count[k] = (info.z - info.y + 1) * (info.w ? 2 : 1);
      narrow[k] = info.w;
    }
  }
  const int total = count[0] + count[1];
  float M = -INFINITY, L = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const bool col = lane * 4 < p.D;
  for (int i0 = 0; i0 < total; i0 += kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {  // all loads at once: none waits for a weight
      const int k = i0 + u < count[0] ? 0 : 1, i = k ? i0 + u - count[0] : i0 + u;
      const int one = k ? narrow[1] : narrow[0];
      const int row = (k ? first[1] : first[0]) + (one ? (i >> 1) * kItemRows + (i & 1) * one : i * kItemRows);
      ml[u] = make_float2(-INFINITY, 0.0f);
      x[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i0 + u < total) {
        ml[u] = p.ml[row];
        if (col) x[u] = *reinterpret_cast<const float4*>(p.part + int64_t(row) * p.D + lane * 4);
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) top = fmaxf(top, ml[u].x);
    const float mu = top == -INFINITY ? 0.0f : top, f = ex2(M - mu);
    M = top;
    L *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float e = ex2(ml[u].x - mu);
      L += ml[u].y * e;
      if (e == 0.0f) continue;  // a piece that saw no key has no output
      o.x += e * x[u].x;
      o.y += e * x[u].y;
      o.z += e * x[u].z;
      o.w += e * x[u].w;
    }
  }
  // (a sum that is NaN, of a data error, makes the whole row NaN even where o is finite)
  const float inv = err ? NAN : (L == 0.0f ? 0.0f : 1.0f / L);
  if (col) {
    uint2 v;
    v.x = pack_half<F16>(o.x * inv, o.y * inv);
    v.y = pack_half<F16>(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + w * p.D + lane * 4) = v;
  }
  if (p.lse && lane == 0) p.lse[w] = err ? NAN : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace psi
