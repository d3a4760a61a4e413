// Attention of drafted tokens, a tree or a chain, over a paged cache that holds their keys and
// values behind those of the request's earlier tokens.
//
//   o_i = sum_s p_is v_s,   p_is = exp(scale q_i k_s) / sum_s' exp(scale q_i k_s')
//
// over the slots s < length and the slots of token i's ancestors and its own.  The rows that
// share a head of keys (n tokens x q_heads / heads) are the 128 rows of a tcgen05 tile, so each
// key and value is read once for all of them; with up to about 250 rows the cache's bytes bound
// the call, not the products.
//
// A persistent CTA per SM takes an equal, contiguous share of all (request, row block, head,
// 128-slot tile) units, in that order: a piece is what it has of one (request, row block, head).
// One warp copies key and value tiles by TMA (page by page, 128-byte swizzle) into a ring of
// buffers, one issues the products S = Q K^T and O += P V, and four warps turn S into P: a thread
// a row here, a thread a slot where a key head has up to 64 rows (below).  S is double-buffered in
// tensor memory, so the next tile's S forms while this one's softmax runs.  The running maximum is
// raised only when a tile exceeds it by more than 2^8 (then O, in tensor memory, is rescaled; P <=
// 256 keeps its 16-bit rounding relative).  Pieces that hold only some of their tiles leave O,
// maximum and sum in the workspace in fp32; they are joined in tile order by the CTA that comes
// last or by a kernel of their own, so results do not depend on the order in which CTAs run.
//
// Measured on a GB300 (graphs of calls, other inputs in turn): two chains of 8 over 130,000 slots, 32
// heads on 8 of 128, 160 to 166 us, 95 to 98% of the copy bandwidth; 32 trees of up to 16 over 4000 slots in
// pages of 16 92 to 94 us, 84%; 128 chains of up to 8 over 1 to 2999 slots, 16 heads on 2 of 64, 38.1 us, 39%,
// bound by the latency of a tile's steps (1450 cycles) and of a piece's beginning and end (6000);
// one token over 1000 slots 10.1 us, launch and latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "sm100_ptx.cuh"
#include "target.cuh"

namespace dspark {
namespace {

using namespace sm100;

constexpr int kTile = 128;                 // slots of a tile, and rows of a block
constexpr int kThreads = 256;
constexpr int kProducerWarp = 0, kIssueWarp = 1, kSoftmaxWarp = 4;
constexpr float kRaise = 8.f;              // log2 of what the maximum may lag behind
constexpr int kMaxGrid = 160;              // CTAs of the persistent grid at most
constexpr int kJoinRows = 16, kJoinParts = 24;   // what one CTA joins at most
// What beginning and ending a piece costs, in tiles: with it in the shares 128 unequal chains take 39
// us, without 53, with 8 of them 41.
constexpr int kPieceUnits = 4;

// How a tile's lines lie in memory and in shared memory, in groups of 8 lines of 128 bytes.
//   kHalvesApart: a copy takes 64 elements of a page's lines; the groups of a half follow each
//                 other (the only form for heads of 64)
//   kHeadsInLine: heads of 128 side by side in a line: a copy takes both halves of a page's lines,
//                 group by group, half by half, and there are half as many copies
//   kHeadsApart:  the same where a page's heads are one after the other
enum TileForm { kHalvesApart, kHeadsInLine, kHeadsApart };

struct AttendParams {
  TileForm form;
  HeadRows q;
  char* out;
  long long out_row, out_head;
  float* lse;
  const void *k, *v;                       // the layer's, for values that are not finite
  CacheStrides cs;
  TargetRows rows;
  TargetSlots slots;
  int group;                               // query heads a key head
  float scale_log2;
  float* partial;                          // [2 CTAs][128][head_dim]
  float2* sums;                            // [2 CTAs][128] maxima (log2) and sums
  bool join_apart;                         // parts are joined by a kernel of their own
  uint32_t* arrived;                       // a byte a CTA: parts that have come of the piece it began
  int4* joins;                             // [CTAs]: of the piece it began its request's first row, its first
                                           // row of the head, rows 2^16 + head, and parts
  int* err;
};

template <int D>
struct AttendSmem {
  static constexpr int kBuf = kTile * D * 2;                 // bytes of a K or V tile
  static constexpr int kHalves = D / 64;                     // 128-byte columns of a tile
  static constexpr int kHalf = kTile * 128;
  static constexpr int kBufs = (229376 - kBuf) / kBuf;
  static constexpr int kOffQ = 0, kOffKV = kBuf, kOffBar = kBuf * (kBufs + 1);
  static constexpr int kBytes = kOffBar + 2048;
};

__host__ __device__ constexpr uint32_t idesc_16(bool bf16, int N, int b_mn_major) {
  return idesc_bf16_f32(kTile, N, 0, b_mn_major) & ~(bf16 ? 0u : (7u << 7) | (7u << 10));
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
      "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
      "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w, int v, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "l"(policy)
      : "memory");
}
// L2 policy: these lines go first (keys and values that no other CTA reads)
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A request as the kernel sees it: rows, tokens before them, slots in all and 128-slot tiles
// (0: nothing to do).  Its units are, for each (row block, head), kPieceUnits and its tiles.
struct Request {
  int row0, n, len, end, tiles, blocks, units;
};
__device__ __forceinline__ Request request_of(const AttendParams& p, int b, int block_rows) {
  Request r;
  const int length = p.slots.lengths[b];
  const RequestRows rows = request_rows(p.rows, b, p.err);
  r.row0 = rows.row0;
  r.n = rows.n;
  r.len = r.n ? checked_length(p.slots, length, r.n, p.err) : 0;
  if (r.len < 0) r.n = 0;
  r.end = r.len + r.n;
  r.tiles = r.n ? (r.end + kTile - 1) / kTile : 0;
  r.blocks = r.n ? (r.n * p.group + block_rows - 1) / block_rows : 0;
  r.units = (r.tiles + kPieceUnits) * r.blocks * p.cs.heads;
  return r;
}

// A CTA's share [lo, hi) of all `total` units, which the first G CTAs have.
struct Share {
  long long lo, hi, total, G;
  int b, off;                // the first unit's request, and its place among the request's
  Request r;
};

// The pieces of a CTA's share of the units, in order.
struct Pieces {
  long long left, unit;      // units still to come, the next one's place among all
  int b, off, block_rows;    // the next unit: `off` of request b's
  Request r;
  // the current piece
  int block, head, tile0, n_tiles;
  long long unit0;           // tile 0's place among all units
  bool whole;
  __device__ __forceinline__ void start(const AttendParams& p, int rows, const Share& s) {
    block_rows = rows;
    left = s.hi - s.lo;
    if (left <= 0) return;
    b = s.b;
    off = s.off;
    unit = s.lo;
    r = s.r;
  }
  __device__ __forceinline__ bool next(const AttendParams& p) {
    while (left > 0) {
      while (off >= r.units) {
        r = request_of(p, ++b, block_rows);
        off = 0;
      }
      const int span = r.tiles + kPieceUnits, at = off / span, from = off - at * span;
      const int take = left < span - from ? (int)left : span - from;
      block = at / p.cs.heads;
      head = at - block * p.cs.heads;
      tile0 = max(from - kPieceUnits, 0);
      n_tiles = from + take - kPieceUnits - tile0;
      whole = n_tiles == r.tiles;
      unit0 = unit - from + kPieceUnits;
      unit += take;
      off += take;
      left -= take;
      if (n_tiles > 0) return true;
    }
    return false;
  }
  __device__ __forceinline__ int rows(const AttendParams& p) const {
    return min(block_rows, r.n * p.group - block * block_rows);
  }
};

// A slot on a page that the cache does not have counts as none: the copies bring zeroes for it (and
// report it), and its scores are masked, slot by slot in what may hold such slots:
//   up to 64 rows: the pieces whose pages the loading warps found not all there, a piece ahead (a word
//     that the copying warp writes, read at each tile, cost 38.7 instead of 38.0 us for 128 chains)
//   more rows: all tiles of a CTA once the copying warp has seen such a page.  It says before it copies
//     tile t how many tiles it has looked at and whether all their pages are there, in one word; one that
//     does not yet count tile t has the tile's slots looked up, too (looked up by the softmax warps
//     with the queries: two long trees 38.6 instead of 36.9 us)
__device__ __forceinline__ bool is_page(const TargetSlots& s, int page) { return (unsigned)page < (unsigned)s.n_pages; }
__device__ __forceinline__ const int32_t* pages_of(const TargetSlots& s, int b) { return s.pages + (long long)b * s.max_pages; }

// A thread's look at every `lanes`th page of a piece, from its place `lane` on.
__device__ __forceinline__ bool lacks_pages(const TargetSlots& s, const Pieces& pc, int lane, int lanes) {
  const int32_t* table = pages_of(s, pc.b);
  const int last = (min(pc.r.end, (pc.tile0 + pc.n_tiles) * kTile) - 1) >> s.page_shift;
  int i = (pc.tile0 * kTile >> s.page_shift) + lane;
  bool lacks = i <= last && !is_page(s, table[i]);
  if (i + lanes <= last) {
#pragma unroll 4
    for (i += lanes; i <= last; i += lanes) lacks |= !is_page(s, table[i]);
  }
  return lacks;
}
__device__ __forceinline__ bool may_lack_pages(volatile uint32_t* looked_s, uint32_t t) {
  const uint32_t word = *looked_s;
  return (word & 1u) || (word >> 1) <= t;
}

// A tile's scores (of 32 rows at `scores` in tensor memory) of slots on no page or behind the last: -inf.
// A function of its own, because the softmax's registers are full and its code is read once a launch.
__device__ __noinline__ void drop_scores(const int32_t* pages, int page_shift, int n_pages, int slot0, int end, uint32_t scores) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const int slot = slot0 + 32 * c + lane;
    const uint32_t bits = __ballot_sync(0xffffffffu, slot < end && (unsigned)pages[slot >> page_shift] < (unsigned)n_pages);
    uint32_t x[32];
    tmem_ld_32x32b_sync<32>(scores + 32 * c, x);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = (bits >> e) & 1 ? x[e] : 0xff800000u;
    tmem_st_32x32b_x32(scores + 32 * c, x);
  }
  tmem_st_wait();
}

// a / b of numbers >= 0 (a 64-bit division takes some 150 cycles)
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// This CTA's share [lo, hi) of all units among the first G CTAs: a scan over the requests, each
// thread some in a row.
__device__ __forceinline__ Share share_units(const AttendParams& p, int block_rows, long long* sums_s, int* start_s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.rows.B <= 32) {
    // every warp looks at all requests, and none waits for another
    Request r = {};
    if (lane < p.rows.B) r = request_of(p, lane, block_rows);
    const long long mine = r.units;
    long long in = mine;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, in, m);
      if (lane >= m) in += y;
    }
    Share s = {};
    s.total = __shfl_sync(0xffffffffu, in, 31);
    s.G = min((long long)gridDim.x, s.total);
    if (blockIdx.x < s.G) {
      s.lo = quotient(s.total * blockIdx.x, s.G);
      s.hi = quotient(s.total * (blockIdx.x + 1), s.G);
      const int at = __ffs(__ballot_sync(0xffffffffu, s.lo < in)) - 1;
      s.b = at;
      s.off = (int)(s.lo - __shfl_sync(0xffffffffu, in - mine, at));
      s.r.row0 = __shfl_sync(0xffffffffu, r.row0, at);
      s.r.n = __shfl_sync(0xffffffffu, r.n, at);
      s.r.len = __shfl_sync(0xffffffffu, r.len, at);
      s.r.end = s.r.len + s.r.n;
      s.r.tiles = __shfl_sync(0xffffffffu, r.tiles, at);
      s.r.blocks = __shfl_sync(0xffffffffu, r.blocks, at);
      s.r.units = __shfl_sync(0xffffffffu, r.units, at);
    }
    return s;
  }
  const int each = (p.rows.B + kThreads - 1) / kThreads, b0 = tid * each, b1 = min(b0 + each, p.rows.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += request_of(p, b, block_rows).units;
  long long in = mine;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, in, m);
    if (lane >= m) in += y;
  }
  if (lane == 31) sums_s[warp] = in;
  __syncthreads();
  Share s = {};
  long long before = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sums_s[w];
    s.total += sums_s[w];
  }
  s.G = min((long long)gridDim.x, s.total);
  if (blockIdx.x < s.G) {
    s.lo = quotient(s.total * blockIdx.x, s.G);
    s.hi = quotient(s.total * (blockIdx.x + 1), s.G);
    if (before + in - mine <= s.lo && s.lo < before + in) {
      long long at = before + in - mine;
      for (int b = b0; b < b1; ++b) {
        const int u = each == 1 ? (int)mine : request_of(p, b, block_rows).units;
        if (s.lo < at + u) {
          start_s[0] = b;
          start_s[1] = (int)(s.lo - at);
          break;
        }
        at += u;
      }
    }
  }
  __syncthreads();
  if (s.hi > s.lo) {
    s.b = start_s[0];
    s.off = start_s[1];
    s.r = request_of(p, s.b, block_rows);
  }
  return s;
}

// The CTAs that share the `tiles` tiles whose units start at unit0: the first, and how many.
struct Parts {
  int first, n;
};
__device__ __forceinline__ Parts parts_of(const Share& s, long long unit0, int tiles) {
  auto cta = [&](long long unit) { return (int)quotient((unit + 1) * s.G - 1, s.total); };
  const int first = cta(unit0);
  return {first, cta(unit0 + tiles - 1) - first + 1};
}
// Where CTA `cta` leaves a part: a piece's first (its CTA's last piece) or another (its CTA's first).
__device__ __forceinline__ int part_place(int cta, bool first) { return 2 * cta + (first ? 1 : 0); }

// Bounded waits: one that runs out reports it and makes the CTA's others return too.
struct Waits {
  volatile int* abort_s;
  int* err;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = sm_cycles();
    for (;;) {
      if (mbar_try_wait_sleep(bar, parity)) return true;
      if (*abort_s) return false;
      if (sm_cycles() - t0 > kWaitCycles) {
        set_device_error(err, DSPARK_ERR_TIMEOUT);
        *abort_s = 1;
        return false;
      }
    }
  }
};

// The copying warp's side of the ring of S::kBufs buffers: tiles page by page, a lane a copy.  A
// tile's pages are looked up two tiles ahead, across pieces.
struct TileAt {
  int id, slot0, head, end;  // the page of each of its copies (lane: copy); end 0: no tile
};
template <typename S>
struct TileCopies {
  uint8_t* ring;
  uint64_t *full, *empty;
  const Waits& wait;
  const AttendParams& p;
  Pieces pc;
  uint64_t policy;
  volatile uint32_t* looked_s;   // null: nobody asks
  int left = 0, slot0 = 0;   // tiles of the piece still to come, and the next one's first slot
  uint32_t item = 0, skipped = ~0u, looked = 0;
  __device__ __forceinline__ TileAt fetch() {
    if (left == 0) {
      if (!pc.next(p)) return {0, 0, 0, 0};
      left = pc.n_tiles;
      slot0 = pc.tile0 * kTile;
    }
    const int lane = threadIdx.x & 31, box = min(1 << p.slots.page_shift, kTile);
    const int slot = slot0 + lane * box;
    const TileAt x = {lane < kTile / box && slot < pc.r.end ? slot_page(p.slots, pc.b, slot, p.err) : 0, slot0,
                      pc.head, pc.r.end};
    slot0 += kTile;
    --left;
    return x;
  }
  __device__ __forceinline__ bool copy(const CUtensorMap* map, const TileAt& x) {
    const int lane = threadIdx.x & 31, page = 1 << p.slots.page_shift, box = min(page, kTile);
    const int halves = p.form == kHalvesApart ? S::kHalves : 1;
    const int my_page = lane / halves, my_half = lane % halves;
    const uint32_t st = item % S::kBufs;
    if (!__all_sync(0xffffffffu, wait(&empty[st], ((item / S::kBufs) & 1) ^ 1))) return false;
    const int n_pages = min(kTile / box, (x.end - x.slot0 + box - 1) / box);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(n_pages * box * 128 * S::kHalves));
    __syncwarp();
    int pid = __shfl_sync(0xffffffffu, x.id, my_page);
    if (pid < 0) pid = p.slots.n_pages;        // (behind the last: zeros)
    if (my_page < n_pages) {
      uint8_t* to = ring + st * S::kBuf;
      const int line = x.slot0 & (page - 1);
      if (p.form == kHalvesApart)
        tma_load_5d(to + my_half * S::kHalf + my_page * box * 128, map, &full[st], my_half * 64, line, x.head, pid, 0, policy);
      else if (p.form == kHeadsInLine)
        tma_load_5d(to + my_page * box * 256, map, &full[st], 0, 0, 2 * x.head, line >> 3, pid, policy);
      else
        tma_load_5d(to + my_page * box * 256, map, &full[st], 0, 0, 0, line >> 3, pid * p.cs.heads + x.head, policy);
    }
    ++item;
    return true;
  }
  // K_0, K_1, V_0, K_2, V_1, .., a place left out, V_last
  __device__ __forceinline__ void run(const CUtensorMap* k_map, const CUtensorMap* v_map) {
    TileAt a = fetch(), b = fetch(), v = {0, 0, 0, 0};
    bool ok = true;
    while (ok && a.end) {
      if (looked_s) {
        looked = (looked + 2) | (__any_sync(0xffffffffu, a.id < 0) ? 1u : 0u);
        if ((threadIdx.x & 31) == 0) *looked_s = looked;
      }
      ok = copy(k_map, a);
      const TileAt c = fetch();
      if (ok && v.end) ok = copy(v_map, v);
      v = a;
      a = b;
      b = c;
    }
    if (ok && v.end) {
      skipped = item++;
      copy(v_map, v);
    }
    // every issued copy lands before the CTA may exit
    for (uint32_t i = item > (uint32_t)S::kBufs ? item - S::kBufs : 0; i < item; ++i)
      if (i != skipped) mbar_wait(&full[i % S::kBufs], (i / S::kBufs) & 1);
  }
};
// Places in the ring of a CTA's K or V tile t.
__device__ __forceinline__ uint32_t k_place(uint32_t t) { return t ? 2 * t - 1 : 0; }
__device__ __forceinline__ uint32_t v_place(uint32_t t) { return 2 * t + 2; }

// Slots behind the last hold anything, and a drafted token that some rows do not see may hold
// values that are not finite: 0 x NaN must not reach them.  Clears line r of a value tile, or
// (in_use) its values that are not finite, which are added again at the end; true if it had any.
template <typename T, int D>
__device__ __forceinline__ bool clear_line(uint8_t* tile, TileForm form, int r, bool in_use) {
  const int group = form == kHalvesApart ? 1024 : 2048, half = form == kHalvesApart ? kTile * 128 : 1024;
  uint8_t* line = tile + (r >> 3) * group + (r & 7) * 128;
  // an exponent of ones, and what carries it (and no other) into the sign's place
  constexpr uint32_t kOnes = __is_same(T, __nv_bfloat16) ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kLow = __is_same(T, __nv_bfloat16) ? 0x00800080u : 0x04000400u;
  bool bad = false;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    uint4* at = reinterpret_cast<uint4*>(line + c / 8 * half + ((c ^ r) & 7) * 16);
    if (!in_use) {
      *at = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 v = *at;
    auto carry = [](uint32_t w) { return ((w & kOnes) + kLow) & 0x80008000u; };
    if (carry(v.x) | carry(v.y) | carry(v.z) | carry(v.w)) {
      auto clear = [carry](uint32_t w) {
        const uint32_t s = carry(w);
        return w & ~((s & 0x8000u ? 0xffffu : 0u) | (s & 0x80000000u ? 0xffff0000u : 0u));
      };
      *at = make_uint4(clear(v.x), clear(v.y), clear(v.z), clear(v.w));
      bad = true;
    }
  }
  fence_proxy_async_smem();
  return bad;
}

// A barrier of the four softmax warps; true in all of them if `any` is in one.
__device__ __forceinline__ bool meet_or(bool any) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((int)any) : "memory");
  return r != 0;
}

// The four softmax warps' part of a piece is written: true in all of them if it was the last to
// come, whose CTA joins all.  The count is left at zero for the next call.  (A part that could not
// be computed is not counted: then nobody joins, and the status says why.)
__device__ __forceinline__ bool last_part(const AttendParams& p, const Parts& parts, bool ok, int* word_s) {
  if (meet_or(!ok)) return false;
  if ((threadIdx.x & 127) == 0) {
    // (bytes 64 to 127 and 132 to 255 of the workspace: another call counts at 128)
    uint32_t* word = p.arrived + (parts.first >> 2) + (parts.first >= 64 ? 1 : 0);
    const int shift = 8 * (parts.first & 3);
    __threadfence();
    const bool last = (int)(atomicAdd(word, 1u << shift) >> shift & 255) == parts.n - 1;
    __threadfence();
    if (last) atomicSub(word, (uint32_t)parts.n << shift);
    *word_s = last;
  }
  meet_or(false);
  return *word_s != 0;
}

// Joins the parts of `rows` rows of a piece, the first of which is row `first` of its request's head,
// a warp 4 of them at once: o = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k, in the parts' order.
// The parts' outputs come while their maxima do.
template <typename T, int D>
__device__ __forceinline__ void join_parts(const AttendParams& p, const Parts& parts, int row0, int first, int rows,
                                           int head0) {
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  constexpr int E = D / 32;
  auto line = [&](int k, int row) { return (long long)part_place(parts.first + k, k == 0) * kTile + row; };
  float x[4][4][E];
  auto load = [&](int k0, int r0) {        // parts k0 .. k0 + 3 of the rows r0 + 4 u
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool on = k0 + j < parts.n && r0 + 4 * u < rows;
        const float* from = p.partial + line(k0 + j, r0 + 4 * u) * D + lane * E;
        if constexpr (E == 4) {
          const float4 v = on ? __ldcg(reinterpret_cast<const float4*>(from)) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[j][u][0] = v.x;
          x[j][u][1] = v.y;
          x[j][u][2] = v.z;
          x[j][u][3] = v.w;
        } else {
          const float2 v = on ? __ldcg(reinterpret_cast<const float2*>(from)) : make_float2(0.f, 0.f);
          x[j][u][0] = v.x;
          x[j][u][1] = v.y;
        }
      }
  };
#pragma unroll 1
  for (int r0 = w4; r0 < rows; r0 += 16) {
    load(0, r0);
    // lane 8 u + k looks after row r0 + 4 u and the parts k, k + 8, ..
    const int my_row = r0 + 4 * (lane >> 3), my_k = lane & 7;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (my_k < parts.n && my_row < rows) ml = __ldcg(p.sums + line(my_k, my_row));
    float M = ml.x;
    for (int k = my_k + 8; k < parts.n; k += 8)
      if (my_row < rows) M = fmaxf(M, __ldcg(p.sums + line(k, my_row)).x);
#pragma unroll
    for (int m = 4; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    float o[4][E], l = 0.f, f = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) o[u][e] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < parts.n; k0 += 4) {
      if ((k0 & 7) == 0) {
        if (k0 > 0) {
          ml = make_float2(-INFINITY, 0.f);
          if (k0 + my_k < parts.n && my_row < rows) ml = __ldcg(p.sums + line(k0 + my_k, my_row));
        }
        f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
        l = fmaf(ml.y, f, l);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float fj = __shfl_sync(0xffffffffu, f, 8 * u + (k0 & 4) + j);
#pragma unroll
          for (int e = 0; e < E; ++e) o[u][e] = fmaf(x[j][u][e], fj, o[u][e]);
        }
      if (k0 + 4 < parts.n) load(k0 + 4, r0);
    }
#pragma unroll
    for (int m = 4; m >= 1; m >>= 1) l += __shfl_xor_sync(0xffffffffu, l, m);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + 4 * u;
      const float lu = __shfl_sync(0xffffffffu, l, 8 * u), Mu = __shfl_sync(0xffffffffu, M, 8 * u);
      if (r >= rows) continue;
      const float inv = lu > 0.f ? 1.f / lu : lu == 0.f ? 0.f : lu;       // (NaN stays)
      const int i_r = first + r, i = i_r / p.group, row = row0 + i;
      const int head = head0 * p.group + (i_r - i * p.group);
      T* dst = reinterpret_cast<T*>(p.out) + row * p.out_row + head * p.out_head + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = pack2<T>(o[u][e] * inv, o[u][e + 1] * inv);
      if (p.lse && lane == 0)
        p.lse[(long long)row * p.group * p.cs.heads + head] = lu == 0.f ? -INFINITY : (Mu + log2f(lu)) * 0.6931471805599453f;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_wide_kernel(const __grid_constant__ CUtensorMap k_map,
                                                             const __grid_constant__ CUtensorMap v_map,
                                                             const __grid_constant__ AttendParams p) {
  using S = AttendSmem<D>;
  constexpr bool kBf16 = sizeof(T) == 2 && __is_same(T, __nv_bfloat16);
  constexpr uint32_t kColO = 256, kColP = 256 + D;           // S 0 and 1 at columns 0 and 128
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t *kv_full = bars, *kv_empty = bars + S::kBufs, *s_full = bars + 2 * S::kBufs, *p_full = s_full + 2,
           *o_full = s_full + 4, *q_full = s_full + 6, *drain = s_full + 7;
  int* words = reinterpret_cast<int*>(smem + S::kOffBar + 512);
  volatile int* abort_s = words;
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(words + 1);
  int* bad_s = words + 2;                                    // by piece parity: piece + 1 with non-finite values
  int* start_s = words + 4;                                  // first request and unit of this CTA's share
  volatile uint32_t* looked_s = reinterpret_cast<uint32_t*>(words + 8);        // tiles whose pages are known
  long long* sums_s = reinterpret_cast<long long*>(smem + S::kOffBar + 640);   // [8 warps] and the total
  int* parents_s = reinterpret_cast<int*>(smem + S::kOffBar + 1024);          // [4 warps][64]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_u32(smem) & 1023u) {            // the swizzle needs it; the same for every thread
    set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < S::kBufs; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kTile);
      mbar_init(&o_full[i], 1);
      bad_s[i] = 0;
    }
    mbar_init(q_full, kTile);
    mbar_init(drain, 1);
    *abort_s = 0;
    *looked_s = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_s, 512);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_s;
  pdl_wait();
  pdl_launch_dependents();
  const Share share = share_units(p, kTile, sums_s, start_s);
  // (by the thread that may write it again)
  if (tid == 32 * kSoftmaxWarp && p.join_apart) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);

  const Waits wait{abort_s, p.err};

  Pieces pc;
  pc.left = 0;
  pc.start(p, kTile, share);

  if (warp == kProducerWarp) {
    TileCopies<S> copies{smem + S::kOffKV, kv_full, kv_empty, wait, p, pc, policy_evict_first(), looked_s};
    copies.run(&k_map, &v_map);
  } else if (warp == kIssueWarp) {
    // ----------------------------------------------------------------- products
    // The whole warp runs along and one lane issues, on values that are the same in all lanes by
    // construction: a lane on its own took 72 cycles an instruction, this 26.
    constexpr uint32_t id_s = idesc_16(kBf16, kTile, 0), id_o = idesc_16(kBf16, D, 1);
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
    const bool one = elect_one();
    const uint64_t q_desc = smem_desc(smem_u32(smem + S::kOffQ), 16u, 1024u, kSwizzle128B);
    const uint32_t group = p.form == kHalvesApart ? 1024u : 2048u, half = p.form == kHalvesApart ? S::kHalf : 1024u;
    const uint64_t k_desc = smem_desc(smem_u32(smem + S::kOffKV), 16u, group, kSwizzle128B);
    const uint64_t v_desc = smem_desc(smem_u32(smem + S::kOffKV), half, group, kSwizzle128B);
    uint32_t t = 0;
    bool ok = true;
    auto all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    // (o_full by tile parity, like S: a waiter tells a phase from its neighbours only, and the
    // softmax skips most of them; the tile's own S says that the product two before has ended)
    auto values = [&](uint32_t t, bool fresh) {      // O += P V of tile t
      const uint32_t buf = t & 1, it = v_place(t), st = it % S::kBufs;
      if (!(ok = all(&p_full[buf], (t >> 1) & 1))) return;
      if (!(ok = all(&kv_full[st], (it / S::kBufs) & 1))) return;
      tc_fence_after_sync();
      const uint64_t d = v_desc + (uint64_t)(st * (S::kBuf >> 4));
      if (one) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_ts_bf16_f32(tm + kColO, tm + kColP + 64 * buf + 8 * k, d + (uint64_t)(k * (group >> 3)), id_o,
                           !fresh || k > 0 ? 1u : 0u);
        umma_commit(&kv_empty[st]);
        umma_commit(&o_full[buf]);
      }
      __syncwarp();
    };
    for (uint32_t piece = 0; ok && pc.next(p); ++piece) {
      if (!(ok = all(q_full, piece & 1))) break;
      const int n = __reduce_max_sync(0xffffffffu, pc.n_tiles);
      for (int j = 0; j < n && ok; ++j, ++t) {
        const uint32_t it = k_place(t), st = it % S::kBufs;
        if (!(ok = all(&kv_full[st], (it / S::kBufs) & 1))) break;
        tc_fence_after_sync();
        const uint64_t d = k_desc + (uint64_t)(st * (S::kBuf >> 4));
        if (one) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_bf16_f32(tm + 128 * (t & 1), q_desc + (uint64_t)((k / 4 * S::kHalf + k % 4 * 32) >> 4),
                          d + (uint64_t)((k / 4 * half + k % 4 * 32) >> 4), id_s, k > 0 ? 1u : 0u);
          umma_commit(&kv_empty[st]);
          umma_commit(&s_full[t & 1]);
        }
        __syncwarp();
        if (j > 0) values(t - 1, j == 1);
      }
      if (ok) values(t - 1, n == 1);
    }
    if (one) umma_commit(drain);
    mbar_wait(drain, 0);
    __syncwarp();
  } else if (warp >= kSoftmaxWarp) {
    // ------------------------------------------------------------------ softmax
    const int w4 = warp - kSoftmaxWarp, r = w4 * 32 + lane;     // row of the block
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    uint32_t tc = 0, piece = 0;
    int* par = parents_s + 64 * w4;
    const float sl = p.scale_log2;
    bool ok = true;

    int row = -1, q_head = 0;                  // this thread's row of q, -1: none
    unsigned long long sees = 0;               // the tokens that it attends to
    bool busy = false;                         // the warp has a row
    auto begin = [&]() {                       // the piece's queries into shared memory
      const int i_r = pc.block * kTile + r, i = i_r / p.group;
      busy = pc.block * kTile + w4 * 32 < pc.r.n * p.group;
      row = i < pc.r.n ? pc.r.row0 + i : -1;
      q_head = pc.head * p.group + (i_r - i * p.group);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q.p) + row * p.q.row + q_head * p.q.head);
      uint4 x[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) x[c] = row >= 0 ? src[c] : make_uint4(0, 0, 0, 0);
      sees = 0;
      if (p.rows.parents) {
        __syncwarp();
        for (int a = lane; a < pc.r.n; a += 32) par[a] = parent_of(p.rows.parents, pc.r.row0 + a, a, p.err);
        __syncwarp();
        if (row >= 0)
          for (int a = i; a >= 0; a = par[a]) sees |= 1ull << a;
      } else if (row >= 0) {
        sees = (2ull << i) - 1;                // (i = 63: all)
      }
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<uint4*>(smem + S::kOffQ + c / 8 * S::kHalf + r * 128 + ((c % 8) ^ (r & 7)) * 16) = x[c];
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    };

    bool more = pc.next(p);
    if (more) begin();
    while (more) {
      const int b = pc.b, head = pc.head, block = pc.block, tile0 = pc.tile0, n = pc.n_tiles;
      const bool whole = pc.whole, my_busy = busy;
      const Request rq = pc.r;
      const int my_row = row, my_head = q_head;
      const unsigned long long my_sees = sees;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n && ok; ++j) {
        const uint32_t t = tc + j, buf = t & 1;
        const int slot0 = (tile0 + j) * kTile;
        const bool masked = slot0 + kTile > rq.len;
        ok = wait(&s_full[buf], (t >> 1) & 1);
        if (masked && ok) {
          // thread r looks after line r of the value tile
          const uint32_t it = v_place(t), st = it % S::kBufs;
          ok = wait(&kv_full[st], (it / S::kBufs) & 1);
          const int slot = slot0 + r;
          if (ok && slot >= rq.len &&
              clear_line<T, D>(smem + S::kOffKV + st * S::kBuf, p.form, r, slot < rq.end))
            bad_s[piece & 1] = (int)piece + 1;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (my_busy) {
          tc_fence_after_sync();
          if (__any_sync(0xffffffffu, may_lack_pages(looked_s, t)))
            drop_scores(pages_of(p.slots, b), p.slots.page_shift, p.slots.n_pages, slot0, rq.end,
                        tmem + lanes + 128 * buf);
          float s[kTile];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld_32x32b_sync<32>(tmem + lanes + 128 * buf + 32 * c, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[32 * c + e] = __uint_as_float(x[e]);
          }
          if (masked) {
            const int ctx = rq.len - slot0;                 // slots before the tokens (may be < 0)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              // 32 slots' bits: those before the tokens, and the tokens that this row sees
              const int a = ctx - 32 * c;                   // the first token's bit
              uint32_t bits = a >= 32 ? 0xffffffffu : a > 0 ? (1u << a) - 1 : 0u;
              if (a >= 0) bits |= a < 32 ? (uint32_t)(my_sees << a) : 0u;
              else if (a > -64) bits |= (uint32_t)(my_sees >> -a);
#pragma unroll
              for (int e = 0; e < 32; ++e) s[32 * c + e] = (bits >> e) & 1 ? s[32 * c + e] : -INFINITY;
            }
          }
          const float mx = max_of(s);
          const bool raise = (mx - m) * sl > kRaise || m == -INFINITY;
          if (__any_sync(0xffffffffu, raise)) {
            const float up = raise ? mx : m;
            if (j > 0) {
              // O of the tiles before, complete, on the new scale
              ok = __all_sync(0xffffffffu, wait(&o_full[buf ^ 1], ((t - 1) >> 1) & 1));
              if (!ok) break;
              tc_fence_after_sync();
              const float f = m == -INFINITY ? 0.f : ex2_approx((m - up) * sl);
              l *= f;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
                tmem_ld_32x32b_sync<32>(tmem + lanes + kColO + 32 * c, x);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                tmem_st_32x32b_x32(tmem + lanes + kColO + 32 * c, x);
              }
            }
            m = up;
          }
          // (a row with no slot yet: every s is -inf and every p 0)
          const float off = m == -INFINITY ? 0.f : -m * sl;
          const F2 sl2 = f2(sl, sl), off2 = f2(off, off);
          F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float a, d;
              f2_get(f2_fma(f2(s[64 * c + 2 * e], s[64 * c + 2 * e + 1]), sl2, off2), a, d);
              a = ex2_approx(a);
              d = ex2_approx(d);
              sum[e & 1] = f2_add(sum[e & 1], f2(a, d));
              x[e] = pack2<T>(a, d);
            }
            tmem_st_32x32b_x32(tmem + lanes + kColP + 64 * buf + 32 * c, x);
          }
          float even, odd;
          f2_get(f2_add(sum[0], sum[1]), even, odd);
          l += even + odd;
          tmem_st_wait();
          tc_fence_before_sync();
        }
        mbar_arrive(&p_full[buf]);
      }
      // the next piece's queries go in while this one's last product runs
      const Parts parts = whole ? Parts{0, 1} : parts_of(share, pc.unit0, rq.tiles);
      more = pc.next(p);
      if (more && ok) begin();
      const uint32_t t_last = tc + n - 1;
      ok = ok && __all_sync(0xffffffffu, wait(&o_full[t_last & 1], (t_last >> 1) & 1));
      tc_fence_after_sync();
      const bool bad = bad_s[piece & 1] == (int)piece + 1;
      if (my_busy && ok) {
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;     // (NaN stays)
        const long long line = (long long)part_place(blockIdx.x, tile0 == 0) * kTile + r;
        float* part = p.partial + line * D;
        T* dst = reinterpret_cast<T*>(p.out) + my_row * p.out_row + my_head * p.out_head;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          tmem_ld_32x32b_sync<32>(tmem + lanes + kColO + 32 * c, x);
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(x[e]);
          if (bad && my_row >= 0) {
            // the values that were left out, where this row sees their token
            for (int a = 0; a < rq.n; ++a) {
              const int slot = rq.len + a;
              if (!((my_sees >> a) & 1) || slot < tile0 * kTile || slot >= (tile0 + n) * kTile) continue;
              const int page = slot_page(p.slots, b, slot, p.err);
              if (page < 0) continue;
              const T* v = static_cast<const T*>(p.v) + page * p.cs.page +
                           (slot & ((1 << p.slots.page_shift) - 1)) * p.cs.slot + head * p.cs.head + 32 * c;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float f = elem_to_float(v[e]);
                if (!(f - f == 0.f)) o[e] += f;
              }
            }
          }
          if (my_row >= 0) {
            if (whole) {
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                uint4 y;
                y.x = pack2<T>(o[8 * g] * inv, o[8 * g + 1] * inv);
                y.y = pack2<T>(o[8 * g + 2] * inv, o[8 * g + 3] * inv);
                y.z = pack2<T>(o[8 * g + 4] * inv, o[8 * g + 5] * inv);
                y.w = pack2<T>(o[8 * g + 6] * inv, o[8 * g + 7] * inv);
                *reinterpret_cast<uint4*>(dst + 32 * c + 8 * g) = y;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(part + 32 * c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
        }
        if (my_row >= 0) {
          if (!whole) {
            p.sums[line] = make_float2(m == -INFINITY ? -INFINITY : m * sl, l);
          } else if (p.lse) {
            p.lse[(long long)my_row * p.group * p.cs.heads + my_head] =
                l == 0.f ? -INFINITY : (m * sl + log2f(l)) * 0.6931471805599453f;
          }
        }
      }
      // (a warp whose wait ran out still meets the others)
      if (!whole) {
        if (p.join_apart) {
          if (tile0 == 0 && r == 0 && ok)
            p.joins[blockIdx.x] = make_int4(rq.row0, block * kTile, min(kTile, rq.n * p.group - block * kTile) << 16 | head, parts.n);
        } else if (last_part(p, parts, ok, words + 6)) {
          join_parts<T, D>(p, parts, rq.row0, block * kTile, min(kTile, rq.n * p.group - block * kTile), head);
        }
      }
      tc_fence_before_sync();
      tc += n;
      ++piece;
    }
  }
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- up to 64 rows a head
// The same with slots and rows exchanged: S^T = K Q^T has the 128 slots on the lanes and the rows
// as columns, so that all four softmax warps are busy however few rows there are (one token of
// a group of four has 4 rows: 16 columns a thread instead of 128) and the products cost by the
// row.  P^T goes to shared memory, and O^T += V^T P^T.  A column's maximum lies across the warps: at
// each tile they agree that no score exceeds its reference by more than 2^8; where one does, and
// at a piece's first tile, they exchange maxima and rescale.  Each thread sums its own slots'
// probabilities; the sums meet at the piece's end.
//
// Two more warps bring each piece's queries and what its rows see, a piece ahead, so that products
// run on from piece to piece: S^T of the next piece's first tile forms before the last O^T.
//
// Up to 16 rows have a kernel with one chunk of 16 columns for itself: its code is read in less time
// when a launch begins (one token 10.2 instead of 10.8 us).
template <int D>
struct NarrowSmem {
  static constexpr int kRows = 64;
  static constexpr int kBuf = kTile * D * 2;                 // bytes of a K or V tile
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = kTile * 128;
  static constexpr int kQ = kRows * D * 2, kQHalf = kRows * 128, kP = kTile * 128;
  static constexpr int kOffQ = 0, kOffP = 2 * kQ, kOffSmall = kOffP + 2 * kP;
  static constexpr int kOffKV = kOffSmall + 7168;
  static constexpr int kBufs = (232448 - kOffKV) / kBuf;
  static constexpr int kBytes = kOffKV + kBufs * kBuf;
  static_assert(kOffKV % 1024 == 0 && kBufs >= 4, "layout");
};

struct PieceInfo {           // what the loading warps say of a piece; no tiles: it was the last
  int b, head, block, tile0, n_tiles, tiles, row0, n, len, end, rows;
  Parts parts;
};

// Sums over a warp's lanes of 16 columns: each exchange halves the columns that a lane looks
// after; lanes 2 c and 2 c + 1 are left with column c's.
__device__ __forceinline__ float sum_over_lanes(float (&v)[16], int lane) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float got = __shfl_xor_sync(0xffffffffu, lane & 16 ? v[e] : v[e + 8], 16);
    v[e] = (lane & 16 ? v[e + 8] : v[e]) + got;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float got = __shfl_xor_sync(0xffffffffu, lane & 8 ? v[e] : v[e + 4], 8);
    v[e] = (lane & 8 ? v[e + 4] : v[e]) + got;
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float got = __shfl_xor_sync(0xffffffffu, lane & 4 ? v[e] : v[e + 2], 4);
    v[e] = (lane & 4 ? v[e + 2] : v[e]) + got;
  }
  const float got = __shfl_xor_sync(0xffffffffu, lane & 2 ? v[0] : v[1], 2);
  const float one = (lane & 2 ? v[1] : v[0]) + got;
  return one + __shfl_xor_sync(0xffffffffu, one, 1);
}

template <typename T, int D, int kChunks>
__global__ void __launch_bounds__(kThreads, 1) attend_narrow_kernel(const __grid_constant__ CUtensorMap k_map,
                                                                    const __grid_constant__ CUtensorMap v_map,
                                                                    const __grid_constant__ AttendParams p) {
  using S = NarrowSmem<D>;
  constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
  constexpr int kRows = S::kRows, kColumns = 16 * kChunks, kLoadWarp = 2;
  constexpr uint32_t kColO = 2 * kRows;                       // S 0 and 1 at columns 0 and 64
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* small = smem + S::kOffSmall;
  uint64_t* bars = reinterpret_cast<uint64_t*>(small);
  uint64_t *kv_full = bars, *kv_empty = bars + S::kBufs, *s_full = bars + 2 * S::kBufs, *p_full = s_full + 2,
           *o_full = s_full + 4, *q_full = s_full + 6, *q_free = s_full + 8, *drain = s_full + 10;
  int* words = reinterpret_cast<int*>(small + 512);
  volatile int* abort_s = words;
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(words + 1);
  volatile int* bad_s = words + 2;                           // by piece parity: piece + 1 with values not finite
  int* start_s = words + 4;
  int* lacks_s = words + 8;                                  // [2 warps] by piece parity: it has slots on no page
  long long* sums_s = reinterpret_cast<long long*>(small + 576);
  PieceInfo* info_s = reinterpret_cast<PieceInfo*>(small + 640);                      // [2] by piece parity
  int* parents_s = reinterpret_cast<int*>(small + 768);                               // [2 warps][64]
  // [2] by piece parity [64 tokens][2]: the columns that see a token, and [64]: a column's place in out
  uint32_t* seen_s = reinterpret_cast<uint32_t*>(small + 1280);
  long long* to_s = reinterpret_cast<long long*>(small + 2304);
  float* best_s = reinterpret_cast<float*>(small + 3328);    // [64]: a column's reference (log2), -inf: none yet
  float* less_s = best_s + 64;                               // [64]: its negative, 0: none yet
  float* scale_s = best_s + 128;                             // [64]: what O and l are multiplied by
  float* down_s = best_s + 192;                              // [64]: by what the reference rose; at the end, 1 / l
  float* max_s = best_s + 256;                               // [4 warps][64]
  float* sum_s = best_s + 512;                               // [4 warps][64]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_u32(smem) & 1023u) {            // the swizzle needs it; the same for every thread
    set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < S::kBufs; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kTile);
      mbar_init(&o_full[i], 1);
      mbar_init(&q_full[i], kRows);
      mbar_init(&q_free[i], kTile);
      bad_s[i] = 0;
    }
    mbar_init(drain, 1);
    *abort_s = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_s, 256);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_s;
  pdl_wait();
  pdl_launch_dependents();
  const Share share = share_units(p, kRows, sums_s, start_s);
  // (by the thread that may write it again)
  if (tid == 32 * kSoftmaxWarp && p.join_apart) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  const Waits wait{abort_s, p.err};
  Pieces pc;
  pc.left = 0;

  if (warp == kProducerWarp) {
    pc.start(p, kRows, share);
    TileCopies<S> copies{smem + S::kOffKV, kv_full, kv_empty, wait, p, pc, policy_evict_first(), nullptr};
    copies.run(&k_map, &v_map);
  } else if (warp == kIssueWarp) {
    // ----------------------------------------------------------------- products
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
    const bool one = elect_one();
    const uint64_t q_desc = smem_desc(smem_u32(smem + S::kOffQ), 16u, 1024u, kSwizzle128B);
    const uint32_t group = p.form == kHalvesApart ? 1024u : 2048u, half = p.form == kHalvesApart ? S::kHalf : 1024u;
    const uint64_t k_desc = smem_desc(smem_u32(smem + S::kOffKV), 16u, group, kSwizzle128B);
    // (head_dim 64: rows 64 to 127 of V^T are rows 0 to 63 again)
    const uint64_t v_desc = smem_desc(smem_u32(smem + S::kOffKV), D == 128 ? half : 0u, group, kSwizzle128B);
    const uint64_t p_desc = smem_desc(smem_u32(smem + S::kOffP), (uint32_t)S::kP, 1024u, kSwizzle128B);
    bool ok = true;
    auto all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    auto values = [&](uint32_t t, int columns, bool fresh) {   // O^T += V^T P^T of tile t
      const uint32_t buf = t & 1, it = v_place(t), st = it % S::kBufs;
      const uint32_t id_p = idesc_16(kBf16, columns, 1) | (1u << 15);     // both operands along their rows
      if (!(ok = all(&p_full[buf], (t >> 1) & 1))) return;
      if (!(ok = all(&kv_full[st], (it / S::kBufs) & 1))) return;
      tc_fence_after_sync();
      const uint64_t d = v_desc + (uint64_t)(st * (S::kBuf >> 4)), b = p_desc + (uint64_t)(buf * (S::kP >> 4));
      if (one) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_bf16_f32(tm + kColO, d + (uint64_t)(k * (group >> 3)), b + (uint64_t)(k * (2048 >> 4)), id_p,
                        !fresh || k > 0 ? 1u : 0u);
        umma_commit(&kv_empty[st]);
        umma_commit(&o_full[buf]);
      }
      __syncwarp();
    };
    int columns_before = 0;
    bool fresh = false;                      // whether the tile before was its piece's first
    uint32_t t = 0;
    for (uint32_t piece = 0; ok; ++piece) {
      const uint32_t q = piece & 1;
      if (!(ok = all(&q_full[q], (piece >> 1) & 1))) break;
      const int n = __reduce_max_sync(0xffffffffu, info_s[q].n_tiles);
      const int columns = (__reduce_max_sync(0xffffffffu, info_s[q].rows) + 15) & ~15;
      if (n == 0) break;
      const uint32_t id_s = idesc_16(kBf16, columns, 0);
      for (int j = 0; j < n && ok; ++j, ++t) {
        const uint32_t it = k_place(t), st = it % S::kBufs;
        if (!(ok = all(&kv_full[st], (it / S::kBufs) & 1))) break;
        tc_fence_after_sync();
        const uint64_t d = k_desc + (uint64_t)(st * (S::kBuf >> 4)), b = q_desc + (uint64_t)(q * (S::kQ >> 4));
        if (one) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_bf16_f32(tm + kRows * (t & 1), d + (uint64_t)((k / 4 * half + k % 4 * 32) >> 4),
                          b + (uint64_t)((k / 4 * S::kQHalf + k % 4 * 32) >> 4), id_s, k > 0 ? 1u : 0u);
          umma_commit(&kv_empty[st]);
          umma_commit(&s_full[t & 1]);
        }
        __syncwarp();
        if (t > 0) values(t - 1, columns_before, fresh);
        columns_before = columns;
        fresh = j == 0;
      }
    }
    if (ok && t > 0) values(t - 1, columns_before, fresh);
    if (one) umma_commit(drain);
    mbar_wait(drain, 0);
    __syncwarp();
  } else if (warp < kSoftmaxWarp) {
    // ------------------------------------------------------------------ queries, a thread a row
    const int col = tid - 32 * kLoadWarp;
    int* par = parents_s + 64 * (warp - kLoadWarp);
    pc.start(p, kRows, share);
    for (uint32_t piece = 0;; ++piece) {
      const uint32_t q = piece & 1;
      const bool more = pc.next(p);
      if (!more) {
        if (__all_sync(0xffffffffu, wait(&q_free[q], ((piece >> 1) & 1) ^ 1))) {
          if (col == 0) info_s[q].n_tiles = 0;
          mbar_arrive(&q_full[q]);
        }
        break;
      }
      const int rows = pc.rows(p);
      const int i_r = pc.block * kRows + col, i = i_r / p.group, head = pc.head * p.group + (i_r - i * p.group);
      const bool live = col < rows;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q.p) +
                                                        (long long)(pc.r.row0 + i) * p.q.row + head * p.q.head);
      uint4 x[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) x[c] = live ? src[c] : make_uint4(0, 0, 0, 0);
      const bool lacks = lacks_pages(p.slots, pc, col, 2 * 32);
      // (while the queries come)
      const Parts parts = pc.whole ? Parts{0, 1} : parts_of(share, pc.unit0, pc.r.tiles);
      unsigned long long sees = 0;
      if (p.rows.parents) {
        __syncwarp();
        for (int a = lane; a < pc.r.n; a += 32) par[a] = parent_of(p.rows.parents, pc.r.row0 + a, a, p.err);
        __syncwarp();
        if (live)
          for (int a = i; a >= 0; a = par[a]) sees |= 1ull << a;
      }
      // the piece before the last has ended
      if (!__all_sync(0xffffffffu, wait(&q_free[q], ((piece >> 1) & 1) ^ 1))) break;
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<uint4*>(smem + S::kOffQ + q * S::kQ + c / 8 * S::kQHalf + col * 128 + ((c ^ col) & 7) * 16) = x[c];
      if (p.rows.parents) {
#pragma unroll 4
        for (int a = 0; a < pc.r.n; ++a) {
          const uint32_t who = __ballot_sync(0xffffffffu, (sees >> a) & 1);
          if (lane == (a & 31)) seen_s[128 * q + 2 * a + (warp - kLoadWarp)] = who;
        }
      } else {
        // token a of a chain: the columns from a group - first on
        for (int a = lane; a < pc.r.n; a += 32) {
          const int from = a * p.group - pc.block * kRows - 32 * (warp - kLoadWarp);
          seen_s[128 * q + 2 * a + (warp - kLoadWarp)] = from >= 32 ? 0u : ~0u << max(from, 0);
        }
      }
      to_s[64 * q + col] = (long long)(pc.r.row0 + i) * p.out_row + head * p.out_head;
      const bool any_lacks = __any_sync(0xffffffffu, lacks);
      if (lane == 0) lacks_s[2 * q + (warp - kLoadWarp)] = any_lacks;
      if (col == 0)
        info_s[q] = {pc.b, pc.head, pc.block, pc.tile0, pc.n_tiles, pc.r.tiles, pc.r.row0, pc.r.n, pc.r.len, pc.r.end, rows, parts};
      fence_proxy_async_smem();
      mbar_arrive(&q_full[q]);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    // These warps meet at barriers, so they leave together: a wait that ran out ends the others'
    // waits, and the next barrier tells all.
    const int w4 = warp - kSoftmaxWarp, r = w4 * 32 + lane;     // slot of a tile; at the end, element of a head
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const float sl = p.scale_log2;
    bool ok = true, lost = false;
    uint32_t t = 0;
    for (uint32_t piece = 0;; ++piece) {
      const uint32_t q = piece & 1;
      if (r < kRows) {
        best_s[r] = -INFINITY;
        less_s[r] = 0.f;
      }
      ok = wait(&q_full[q], (piece >> 1) & 1) && ok;
      if (meet_or(!ok)) break;
      const PieceInfo rq = info_s[q];
      const int rows = rq.rows, chunks = (rows + 15) / 16, n = rq.n_tiles, tile0 = rq.tile0;
      if (n == 0) break;
      const bool lacks = lacks_s[2 * q] | lacks_s[2 * q + 1];
      bool open = true;                        // a column has no reference yet
      F2 l[kColumns / 2];                      // this thread's slots' part of the columns' sums
#pragma unroll
      for (int e = 0; e < kColumns / 2; ++e) l[e] = f2(0.f, 0.f);
      const F2 sl2 = f2(sl, sl);
      for (int j = 0; j < n; ++j, ++t) {
        const uint32_t buf = t & 1;
        const int slot0 = (tile0 + j) * kTile, slot = slot0 + r;
        const bool masked = slot0 + kTile > rq.len || lacks;
        uint2 seen = make_uint2(~0u, ~0u);     // the columns that see this slot
        if (masked && slot >= rq.len)
          seen = slot < rq.end ? *reinterpret_cast<const uint2*>(seen_s + 128 * q + 2 * (slot - rq.len)) : make_uint2(0, 0);
        if (lacks && slot < rq.end && !is_page(p.slots, pages_of(p.slots, rq.b)[slot >> p.slots.page_shift]))
          seen = make_uint2(0, 0);
        ok = wait(&s_full[buf], (t >> 1) & 1) && ok;
        __syncwarp();
        tc_fence_after_sync();
        // the slot's scores (times scale and log2 e), less the columns' references
        float x[kColumns], mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c >= chunks) break;
          uint32_t v[16];
          tmem_ld_32x32b_sync<16>(tmem + lanes + kRows * buf + 16 * c, v);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 less = *reinterpret_cast<const float4*>(less_s + 16 * c + e);
            const F2 lo = f2_fma(f2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sl2, f2(less.x, less.y));
            const F2 hi = f2_fma(f2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), sl2, f2(less.z, less.w));
            f2_get(lo, x[16 * c + e], x[16 * c + e + 1]);
            f2_get(hi, x[16 * c + e + 2], x[16 * c + e + 3]);
          }
          if (masked) {
            const uint32_t bits = c < 2 ? seen.x : seen.y;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[16 * c + e] = bits & (1u << (16 * (c & 1) + e)) ? x[16 * c + e] : -INFINITY;
          }
          float part[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) part[e] = x[16 * c + e];
          mx = fmaxf(mx, max_of(part));
        }
        if (open || meet_or(mx > kRaise || !ok)) {
          // ---- new references from the columns' maxima over the warps
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (c >= chunks) break;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              float4 m;
              m.x = warp_max(x[16 * c + e]);     // (NaN only if every lane's is)
              m.y = warp_max(x[16 * c + e + 1]);
              m.z = warp_max(x[16 * c + e + 2]);
              m.w = warp_max(x[16 * c + e + 3]);
              if (lane == 0) *reinterpret_cast<float4*>(max_s + 64 * w4 + 16 * c + e) = m;
            }
          }
          if ((lost = meet_or(!ok))) break;
          bool none = false;
          if (r < kRows && r < 16 * chunks) {
            const float m = fmaxf(fmaxf(max_s[r], max_s[64 + r]), fmaxf(max_s[128 + r], max_s[192 + r]));
            const float old = best_s[r], ref = -less_s[r];
            const bool first = old == -INFINITY, up = first || m > kRaise;
            const float now = first ? m : up ? ref + m : old;
            const float down = first ? (m == -INFINITY ? 0.f : m) : up ? now - ref : 0.f;
            best_s[r] = now;
            less_s[r] = now == -INFINITY ? 0.f : -now;
            down_s[r] = down;
            scale_s[r] = first ? 0.f : up ? ex2_approx(-down) : 1.f;
            none = now == -INFINITY && r < rows;
          }
          open = meet_or(none);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (c >= chunks) break;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 down = *reinterpret_cast<const float4*>(down_s + 16 * c + e);
              x[16 * c + e] -= down.x;
              x[16 * c + e + 1] -= down.y;
              x[16 * c + e + 2] -= down.z;
              x[16 * c + e + 3] -= down.w;
            }
          }
          if (j > 0) {
            // O and l of the tiles before, complete, on the new scale
            ok = wait(&o_full[buf ^ 1], ((t - 1) >> 1) & 1) && ok;
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              if (c >= chunks) break;
              uint32_t v[16];
              tmem_ld_32x32b_sync<16>(tmem + lanes + kColO + 16 * c, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * scale_s[16 * c + e]);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                l[8 * c + e] = f2_mul(l[8 * c + e], f2(scale_s[16 * c + 2 * e], scale_s[16 * c + 2 * e + 1]));
              tmem_st_32x32b_x16(tmem + lanes + kColO + 16 * c, v);
            }
            tmem_st_wait();
          }
        }
        uint8_t* line = smem + S::kOffP + buf * S::kP + r * 128;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c >= chunks) break;
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = ex2_approx(x[16 * c + 2 * e]), d = ex2_approx(x[16 * c + 2 * e + 1]);
            l[8 * c + e] = f2_add(l[8 * c + e], f2(a, d));
            y[e] = pack2<T>(a, d);
          }
          *reinterpret_cast<uint4*>(line + ((2 * c ^ r) & 7) * 16) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(line + (((2 * c + 1) ^ r) & 7) * 16) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        if (masked) {
          const uint32_t it = v_place(t), st = it % S::kBufs;
          ok = wait(&kv_full[st], (it / S::kBufs) & 1) && ok;
          if (ok && slot >= rq.len &&
              clear_line<T, D>(smem + S::kOffKV + st * S::kBuf, p.form, r, slot < rq.end))
            bad_s[q] = (int)piece + 1;
          __syncwarp();
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        mbar_arrive(&p_full[buf]);
      }
      if (lost) break;
      // ---- the piece's rows: sums over the warps, then O
      const bool whole = n == rq.tiles;
      const long long line = (long long)part_place(blockIdx.x, tile0 == 0) * kTile;
      float* part = p.partial + line * D;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (c >= chunks) break;
        float v[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) f2_get(l[8 * c + e], v[2 * e], v[2 * e + 1]);
        const float s = sum_over_lanes(v, lane);
        if (!(lane & 1)) sum_s[64 * w4 + 16 * c + (lane >> 1)] = s;
      }
      if (meet_or(!ok)) break;
      if (r < rows && r < kRows) {
        const float s = (sum_s[r] + sum_s[64 + r]) + (sum_s[128 + r] + sum_s[192 + r]);
        down_s[r] = !whole ? 1.f : s > 0.f ? 1.f / s : s == 0.f ? 0.f : s;       // (NaN stays)
        if (!whole) {
          p.sums[line + r] = make_float2(best_s[r], s);
        } else if (p.lse) {
          const int i_r = rq.block * kRows + r, i = i_r / p.group;
          p.lse[(long long)(rq.row0 + i) * p.group * p.cs.heads + rq.head * p.group + (i_r - i * p.group)] =
              s == 0.f ? -INFINITY : (best_s[r] + log2f(s)) * 0.6931471805599453f;
        }
      }
      meet_or(false);
      ok = wait(&o_full[(t - 1) & 1], ((t - 1) >> 1) & 1);
      __syncwarp();
      tc_fence_after_sync();
      const bool bad = bad_s[q] == (int)piece + 1;
#pragma unroll 1
      for (int w = 0; w < (kChunks + 1) / 2; ++w) {      // 32 rows at a time
        const int left = rows - 32 * w;
        if (left <= 0) break;
        uint32_t v[32];
        tmem_ld_32x32b_sync<32>(tmem + lanes + kColO + 32 * w, v);
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(v[e]);
        if (r >= D || !ok) continue;
        if (bad) {
          // the values that were left out, where a row sees their token
          for (int a = 0; a < rq.n; ++a) {
            const int at = rq.len + a;
            if (at < tile0 * kTile || at >= (tile0 + n) * kTile) continue;
            const int page = slot_page(p.slots, rq.b, at, p.err);
            if (page < 0) continue;
            const float f = elem_to_float(static_cast<const T*>(p.v)[page * p.cs.page + (at & ((1 << p.slots.page_shift) - 1)) * p.cs.slot +
                                                                    rq.head * p.cs.head + r]);
            if (f - f == 0.f) continue;
            const uint32_t bits = seen_s[128 * q + 2 * a + w];
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((bits >> e) & 1) o[e] += f;
          }
        }
        if (whole) {
          T* out = reinterpret_cast<T*>(p.out) + r;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const longlong2 to = *reinterpret_cast<const longlong2*>(to_s + 64 * q + 32 * w + e);
            const float2 inv = *reinterpret_cast<const float2*>(down_s + 32 * w + e);
            if (e < left) out[to.x] = elem_from_float<T>(o[e] * inv.x);
            if (e + 1 < left) out[to.y] = elem_from_float<T>(o[e + 1] * inv.y);
          }
        } else {
          float* to = part + 32 * w * D + r;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < left) to[e * D] = o[e];
        }
      }
      tc_fence_before_sync();
      mbar_arrive(&q_free[q]);
      if (!whole) {
        if (p.join_apart) {
          if (tile0 == 0 && r == 0 && ok)
            p.joins[blockIdx.x] = make_int4(rq.row0, rq.block * kRows, rows << 16 | rq.head, rq.parts.n);
        } else if (last_part(p, rq.parts, ok, words + 6)) {
          join_parts<T, D>(p, rq.parts, rq.row0, rq.block * kRows, rows, rq.head);
        }
      }
    }
  }
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 256);
  }
}

// The same in a kernel of its own: CTA (c, y) the parts of the piece that CTA c began and left
// unfinished, the rows from 16 y on.
template <typename T, int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int4 join = p.joins[blockIdx.x];
  if (join.w < 2) return;
  const int n = min((join.z >> 16) - 16 * (int)blockIdx.y, 16);
  if (n <= 0) return;
  AttendParams q = p;
  q.partial += 16 * blockIdx.y * D;
  q.sums += 16 * blockIdx.y;
  join_parts<T, D>(q, {(int)blockIdx.x, join.w}, join.x, join.y + 16 * blockIdx.y, n, join.z & 0xffff);
}

// The same for pieces of many parts: the rows from 4 y on, the parts shared out over the four warps in
// order, whose sums the first warps add up in that order, a warp a row.
template <typename T, int D>
__global__ void __launch_bounds__(128) join_many_kernel(const __grid_constant__ AttendParams p) {
  constexpr int E = D / 32, kAhead = 4;
  __shared__ float o_s[4][4][D], l_s[4][4];
  pdl_wait();
  pdl_launch_dependents();
  const int4 join = p.joins[blockIdx.x];
  if (join.w < 2) return;
  const int r0 = 4 * blockIdx.y, rows = min((join.z >> 16) - r0, 4);
  if (rows <= 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto line = [&](int k, int r) { return (long long)part_place(blockIdx.x + k, k == 0) * kTile + r0 + r; };
  // every warp: the rows' maxima over all parts, lane 8 u + k those of row u and the parts k, k + 8, ..
  float M = -INFINITY;
  if ((lane >> 3) < rows)
    for (int k = lane & 7; k < join.w; k += 8) M = fmaxf(M, __ldcg(p.sums + line(k, lane >> 3)).x);
#pragma unroll
  for (int m = 4; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
  const int k_begin = join.w * warp / 4, k_end = join.w * (warp + 1) / 4;
  float o[4][E], l[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    l[u] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[u][e] = 0.f;
  }
  for (int k0 = k_begin; k0 < k_end; k0 += kAhead) {
    float x[kAhead][4][E];
    float2 ml[kAhead][4];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool on = k0 + j < k_end && u < rows;
        ml[j][u] = on ? __ldcg(p.sums + line(k0 + j, u)) : make_float2(-INFINITY, 0.f);
        const float* from = p.partial + line(k0 + j, u) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = on ? __ldcg(reinterpret_cast<const float2*>(from + e)) : make_float2(0.f, 0.f);
          x[j][u][e] = v.x;
          x[j][u][e + 1] = v.y;
        }
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = ml[j][u].x == -INFINITY ? 0.f : ex2_approx(ml[j][u].x - __shfl_sync(0xffffffffu, M, 8 * u));
        l[u] = fmaf(ml[j][u].y, f, l[u]);
#pragma unroll
        for (int e = 0; e < E; ++e) o[u][e] = fmaf(x[j][u][e], f, o[u][e]);
      }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
#pragma unroll
    for (int e = 0; e < E; ++e) o_s[warp][u][lane * E + e] = o[u][e];
    if (lane == 0) l_s[warp][u] = l[u];
  }
  __syncthreads();
  const float Mr = __shfl_sync(0xffffffffu, M, 8 * warp);
  if (warp >= rows) return;
  const float lr = (l_s[0][warp] + l_s[1][warp]) + (l_s[2][warp] + l_s[3][warp]);
  const float inv = lr > 0.f ? 1.f / lr : lr == 0.f ? 0.f : lr;         // (NaN stays)
  const int i_r = join.y + r0 + warp, i = i_r / p.group, row = join.x + i;
  const int head = (join.z & 0xffff) * p.group + (i_r - i * p.group);
  T* dst = reinterpret_cast<T*>(p.out) + row * p.out_row + head * p.out_head + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    float y[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = lane * E + e + h;
      y[h] = ((o_s[0][warp][at] + o_s[1][warp][at]) + (o_s[2][warp][at] + o_s[3][warp][at])) * inv;
    }
    *reinterpret_cast<uint32_t*>(dst + e) = pack2<T>(y[0], y[1]);
  }
  if (p.lse && lane == 0)
    p.lse[(long long)row * p.group * p.cs.heads + head] = lr == 0.f ? -INFINITY : (Mr + log2f(lr)) * 0.6931471805599453f;
}

TileForm tile_form(const CacheStrides& cs, const TargetSlots& slots) {
  if (cs.head_dim != 128) return kHalvesApart;
  if (cs.heads == 1 || cs.head == 128) return kHeadsInLine;
  return slots.n_pages == 1 || (cs.page == cs.heads * cs.head && (long long)slots.n_pages * cs.heads < (1LL << 31))
             ? kHeadsApart : kHalvesApart;
}

bool encode_cache_map(CUtensorMap* map, const void* base, bool bf16, const CacheStrides& cs,
                      const TargetSlots& slots, TileForm form) {
  EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t page = (cuuint64_t)1 << slots.page_shift, heads = (cuuint64_t)cs.heads,
                   pages = (cuuint64_t)slots.n_pages;
  const cuuint64_t slot_b = (cuuint64_t)cs.slot * 2, head_b = (cuuint64_t)cs.head * 2, page_b = (cuuint64_t)cs.page * 2;
  const cuuint32_t lines = (cuuint32_t)(page < kTile ? page : kTile);
  cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  auto encode = [&](const cuuint64_t (&dims)[5], const cuuint64_t (&strides)[4], const cuuint32_t (&box)[5]) {
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
              const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B,
              // (a head's line: more would be another's, which another CTA reads at another time)
              cs.head_dim == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (form == kHalvesApart)
    return encode({(cuuint64_t)cs.head_dim, page, heads, pages, 1}, {slot_b, head_b, page_b, 16}, {64, lines, 1, 1, 1});
  if (form == kHeadsInLine)
    return encode({64, 8, 2 * heads, page / 8, pages}, {slot_b, 128, 8 * slot_b, page_b}, {64, 8, 2, lines / 8, 1});
  return encode({64, 8, 2, page / 8, pages * heads}, {slot_b, 128, 8 * slot_b, head_b}, {64, 8, 2, lines / 8, 1});
}

static_assert(kMaxGrid <= 188, "the counts' place");

template <typename T, int D>
cudaError_t attend_for(AttendParams p, const TargetSlots& slots, bool bf16, cudaStream_t stream) {
  static std::atomic<int> cache[kMaxCachedDevices];
  int grid = per_device_grid(cache, []() {
    return cudaFuncSetAttribute(attend_wide_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttendSmem<D>::kBytes) == cudaSuccess &&
                   cudaFuncSetAttribute(attend_narrow_kernel<T, D, 4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        NarrowSmem<D>::kBytes) == cudaSuccess &&
                   cudaFuncSetAttribute(attend_narrow_kernel<T, D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        NarrowSmem<D>::kBytes) == cudaSuccess
               ? 1 : -1;
  });
  if (grid <= 0) return cudaErrorInvalidConfiguration;
  if (grid > kMaxGrid) grid = kMaxGrid;
  CUtensorMap k_map, v_map;
  p.form = tile_form(p.cs, slots);
  if (!encode_cache_map(&k_map, p.k, bf16, p.cs, slots, p.form) ||
      !encode_cache_map(&v_map, p.v, bf16, p.cs, slots, p.form))
    return cudaErrorInvalidValue;
  const int rows = p.rows.N * p.group;
  const bool narrow = rows <= NarrowSmem<D>::kRows;
  // A piece has one of its request's heads, so at most a head's share of the grid in parts and the
  // two at its ends, and a tile each.  Up to 16 rows of few parts are joined by the CTA that comes
  // last (a token of 4 rows and 8 parts: 11.3 us either way; 35 short requests without parts: 9.8
  // us, and 11.7 with a second kernel that finds nothing to do); more of them would keep that CTA
  // from its other pieces (128 rows of 6 parts: 28 us, and 14 by a kernel of their own).
  const int most_tiles = (int)((((long long)slots.max_pages << slots.page_shift) + kTile - 1) / kTile);
  const int most_parts = min(grid / p.cs.heads + 2, most_tiles);
  p.join_apart = most_parts > 1 && (rows > kJoinRows || most_parts > kJoinParts);
  const cudaError_t e =
      narrow ? launch_pdl(rows <= 16 ? attend_narrow_kernel<T, D, 1> : attend_narrow_kernel<T, D, 4>, dim3(grid), dim3(kThreads), NarrowSmem<D>::kBytes, stream, k_map,
                          v_map, p)
             : launch_pdl(attend_wide_kernel<T, D>, dim3(grid), dim3(kThreads), AttendSmem<D>::kBytes, stream, k_map,
                          v_map, p);
  if (e != cudaSuccess || !p.join_apart) return e;
  // Many parts of a piece, taking all requests to be alike, are shared out over a CTA's warps (16 parts
  // of 48 rows 14.7 to 13.9 us in all, 19 of 128 rows 38.9 to 36.9), unless the four times as many
  // CTAs that then find no rows cost more (9 parts of 128 rows 19.1 to 22.6).
  const int alike = (int)(grid / ((long long)p.rows.B * p.cs.heads * cdiv(rows, kTile))) + 2;
  const int per_cta = min(alike, most_parts) * 8 > min(rows, kTile) ? 4 : 16;
  return launch_pdl(per_cta == 4 ? join_many_kernel<T, D> : join_kernel<T, D>,
                    dim3(grid, cdiv(rows < kTile ? rows : kTile, per_cta)), dim3(128), 0, stream, p);
}

}  // namespace

size_t tree_attention_bytes(int B, int N, int q_heads, int heads, int head_dim) {
  (void)B;
  (void)N;
  (void)q_heads;
  (void)heads;
  return 256 + align_up(kMaxGrid * sizeof(int4), 256) + (size_t)2 * kMaxGrid * kTile * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_tree_attention(const HeadRows& q, int q_heads, const void* k_cache, const void* v_cache,
                                  const CacheStrides& cs, int dtype, const TargetRows& rows,
                                  const TargetSlots& slots, float scale, void* out, long long out_row,
                                  long long out_head, float* lse, int* err, void* ws, cudaStream_t stream) {
  AttendParams p = {};
  p.q = q;
  p.out = static_cast<char*>(out);
  p.out_row = out_row;
  p.out_head = out_head;
  p.lse = lse;
  p.k = k_cache;
  p.v = v_cache;
  p.cs = cs;
  p.rows = rows;
  p.slots = slots;
  p.group = q_heads / cs.heads;
  p.scale_log2 = scale * kLog2e;
  p.arrived = ws_at<uint32_t>(ws, 64);
  p.joins = ws_at<int4>(ws, 256);
  p.partial = ws_at<float>(ws, 256 + align_up(kMaxGrid * sizeof(int4), 256));
  p.sums = reinterpret_cast<float2*>(p.partial + (size_t)2 * kMaxGrid * kTile * cs.head_dim);
  p.err = err;
  const bool bf16 = dtype == DSPARK_BF16;
  if (cs.head_dim == 128)
    return bf16 ? attend_for<__nv_bfloat16, 128>(p, slots, bf16, stream) : attend_for<__half, 128>(p, slots, bf16, stream);
  return bf16 ? attend_for<__nv_bfloat16, 64>(p, slots, bf16, stream) : attend_for<__half, 64>(p, slots, bf16, stream);
}

}  // namespace dspark
