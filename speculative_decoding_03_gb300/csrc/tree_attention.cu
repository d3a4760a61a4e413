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
// buffers, one thread issues the products S = Q K^T and O += P V, and four warps, a thread a
// row, turn S into P.  S is double-buffered in tensor memory, so the next tile's S forms
// while this one's softmax runs.  The running maximum is raised only when a tile exceeds it by
// more than 2^8 (then O, in tensor memory, is rescaled; P <= 256 keeps its 16-bit rounding
// relative).  Pieces that hold only some of their tiles leave O, maximum and sum in the
// workspace in fp32, and a second kernel joins them in tile order, so results do not depend on
// the order in which CTAs run.
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

struct AttendParams {
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
  float* partial;                          // [2 CTAs][128][head_dim + 2]
  int4* joins;                             // [CTAs]: request, row block, head, parts
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

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
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
// (0: nothing to do).
struct Request {
  int row0, n, len, end, tiles, blocks, units;
};
__device__ __forceinline__ Request request_of(const AttendParams& p, int b) {
  Request r;
  const RequestRows rows = request_rows(p.rows, b, p.err);
  r.row0 = rows.row0;
  r.n = rows.n;
  r.len = r.n ? request_length(p.slots, b, r.n, p.err) : 0;
  if (r.len < 0) r.n = 0;
  r.end = r.len + r.n;
  r.tiles = r.n ? (r.end + kTile - 1) / kTile : 0;
  r.blocks = r.n ? (r.n * p.group + kTile - 1) / kTile : 0;
  r.units = r.tiles * r.blocks * p.cs.heads;
  return r;
}

// The pieces of a CTA's share [lo, hi) of the units, in order.
struct Pieces {
  long long left;            // units still to come
  int b, off;                // the next unit: `off` of request b's
  Request r;
  // the current piece
  int block, head, tile0, n_tiles;
  bool whole;
  __device__ __forceinline__ void start(const AttendParams& p, int b0, int off0, long long units) {
    b = b0;
    off = off0;
    left = units;
    if (left > 0) r = request_of(p, b);
  }
  __device__ __forceinline__ bool next(const AttendParams& p) {
    if (left <= 0) return false;
    while (off >= r.units) {
      r = request_of(p, ++b);
      off = 0;
    }
    const int at = off / r.tiles;
    block = at / p.cs.heads;
    head = at - block * p.cs.heads;
    tile0 = off - at * r.tiles;
    n_tiles = r.tiles - tile0;
    if (n_tiles > left) n_tiles = (int)left;
    whole = n_tiles == r.tiles;
    off += n_tiles;
    left -= n_tiles;
    return true;
  }
};

// Position in the ring of the K or V tile j of a piece of n tiles: K_0, K_1, V_0, K_2, V_1, ..,
// V_{n-1}, the order in which the products take them.
__device__ __forceinline__ int k_item(int j) { return j ? 2 * j - 1 : 0; }
__device__ __forceinline__ int v_item(int j, int n) { return j < n - 1 ? 2 * j + 2 : 2 * n - 1; }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ CUtensorMap k_map,
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
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's share of the units: a scan over the requests, each thread some in a row
  const int each = (p.rows.B + kThreads - 1) / kThreads, b0 = tid * each, b1 = min(b0 + each, p.rows.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += request_of(p, b).units;
  long long in = mine;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, in, m);
    if (lane >= m) in += y;
  }
  if (lane == 31) sums_s[warp] = in;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sums_s[w];
    total += sums_s[w];
  }
  const long long G = min((long long)gridDim.x, total);
  const bool working = blockIdx.x < G;
  const long long lo = working ? total * blockIdx.x / G : 0, hi = working ? total * (blockIdx.x + 1) / G : 0;
  if (working && before + in - mine <= lo && lo < before + in) {
    long long at = before + in - mine;
    for (int b = b0; b < b1; ++b) {
      const int u = request_of(p, b).units;
      if (lo < at + u) {
        start_s[0] = b;
        start_s[1] = (int)(lo - at);
        break;
      }
      at += u;
    }
  }
  if (tid == 0) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_s;

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = sm_cycles();
    for (;;) {
      if (mbar_try_wait_sleep(bar, parity)) return true;
      if (*abort_s) return false;
      if (sm_cycles() - t0 > kWaitCycles) {
        set_device_error(p.err, DSPARK_ERR_TIMEOUT);
        *abort_s = 1;
        return false;
      }
    }
  };

  Pieces pc;
  if (working) pc.start(p, start_s[0], start_s[1], hi - lo);
  else pc.left = 0;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------- copies
    const int shift = p.slots.page_shift, page = 1 << shift;
    const int box = min(page, kTile), per_tile = kTile / box;     // lines of a copy, copies of a tile
    const int my_page = lane / S::kHalves, my_half = lane % S::kHalves;
    uint32_t item = 0;
    bool ok = true;
    auto copy = [&](const CUtensorMap* map, int id, int slot0, int head, int end) {
      const uint32_t st = item % S::kBufs;
      ok = wait(&kv_empty[st], ((item / S::kBufs) & 1) ^ 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const int n_pages = min(per_tile, (end - slot0 + box - 1) / box);
      if (lane == 0) mbar_arrive_expect_tx(&kv_full[st], (uint32_t)(n_pages * box * 128 * S::kHalves));
      __syncwarp();
      const int pid = __shfl_sync(0xffffffffu, id, my_page);
      if (my_page < n_pages)
        tma_load_4d(smem + S::kOffKV + st * S::kBuf + my_half * S::kHalf + my_page * box * 128, map, &kv_full[st],
                    my_half * 64, slot0 & (page - 1), head, pid < 0 ? p.slots.n_pages : pid);
      ++item;
    };
    auto pages_of = [&](int b, int slot0, int end) {
      const int slot = slot0 + lane * box;
      return lane < per_tile && slot < end ? slot_page(p.slots, b, slot, p.err) : 0;
    };
    while (ok && pc.next(p)) {
      const int first = pc.tile0 * kTile, end = pc.r.end;
      int id = pages_of(pc.b, first, end), id_v = 0;
      for (int j = 0; j < pc.n_tiles && ok; ++j) {
        const int slot0 = first + j * kTile;
        const int id_next = j + 1 < pc.n_tiles ? pages_of(pc.b, slot0 + kTile, end) : 0;
        copy(&k_map, id, slot0, pc.head, end);
        if (ok && j > 0) copy(&v_map, id_v, slot0 - kTile, pc.head, end);
        id_v = id;
        id = id_next;
      }
      if (ok) copy(&v_map, id_v, first + (pc.n_tiles - 1) * kTile, pc.head, end);
    }
    // every issued copy lands before the CTA may exit
    for (uint32_t i = item > (uint32_t)S::kBufs ? item - S::kBufs : 0; i < item; ++i)
      mbar_wait(&kv_full[i % S::kBufs], (i / S::kBufs) & 1);
  } else if (warp == kIssueWarp) {
    // ----------------------------------------------------------------- products
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_16(kBf16, kTile, 0), id_o = idesc_16(kBf16, D, 1);
      const uint64_t q_desc = smem_desc(smem_u32(smem + S::kOffQ), 16u, 1024u, kSwizzle128B);
      const uint64_t k_desc = smem_desc(smem_u32(smem + S::kOffKV), 16u, 1024u, kSwizzle128B);
      const uint64_t v_desc = smem_desc(smem_u32(smem + S::kOffKV), (uint32_t)S::kHalf, 1024u, kSwizzle128B);
      uint32_t base = 0, tc = 0, piece = 0;
      bool ok = true;
      // (o_full by tile parity, like S: a waiter tells a phase from its neighbours only, and the
      // softmax skips most of them; the tile's own S says that the product two before has ended)
      auto values = [&](int j, int n) {              // O += P V of tile j of the piece's n
        const uint32_t t = tc + j, buf = t & 1, it = base + v_item(j, n), st = it % S::kBufs;
        if (!(ok = wait(&p_full[buf], (t >> 1) & 1))) return;
        if (!(ok = wait(&kv_full[st], (it / S::kBufs) & 1))) return;
        tc_fence_after_sync();
        const uint64_t d = v_desc + (uint64_t)(st * (S::kBuf >> 4));
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_ts_bf16_f32(tmem + kColO, tmem + kColP + 64 * buf + 8 * k, d + (uint64_t)(k * (2048 >> 4)), id_o,
                           j > 0 || k > 0 ? 1u : 0u);
        umma_commit(&kv_empty[st]);
        umma_commit(&o_full[buf]);
      };
      for (; ok && pc.next(p); ++piece) {
        if (!(ok = wait(q_full, piece & 1))) break;
        const int n = pc.n_tiles;
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t t = tc + j, it = base + k_item(j), st = it % S::kBufs;
          if (!(ok = wait(&kv_full[st], (it / S::kBufs) & 1))) break;
          tc_fence_after_sync();
          const uint64_t d = k_desc + (uint64_t)(st * (S::kBuf >> 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_bf16_f32(tmem + 128 * (t & 1), q_desc + (uint64_t)((k / 4 * S::kHalf + k % 4 * 32) >> 4),
                          d + (uint64_t)((k / 4 * S::kHalf + k % 4 * 32) >> 4), id_s, k > 0 ? 1u : 0u);
          umma_commit(&kv_empty[st]);
          umma_commit(&s_full[t & 1]);
          if (j > 0) values(j - 1, n);
        }
        if (ok) values(n - 1, n);
        base += 2 * n;
        tc += n;
      }
      umma_commit(drain);
      mbar_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp >= kSoftmaxWarp) {
    // ------------------------------------------------------------------ softmax
    const int w4 = warp - kSoftmaxWarp, r = w4 * 32 + lane;     // row of the block
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    uint32_t base = 0, tc = 0, piece = 0;
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
    while (more && ok) {
      const int b = pc.b, head = pc.head, block = pc.block, tile0 = pc.tile0, n = pc.n_tiles;
      const bool whole = pc.whole, my_busy = busy;
      const Request rq = pc.r;
      const int my_row = row, my_head = q_head;
      const unsigned long long my_sees = sees;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const uint32_t t = tc + j, buf = t & 1;
        const int slot0 = (tile0 + j) * kTile;
        const bool masked = slot0 + kTile > rq.len;
        ok = wait(&s_full[buf], (t >> 1) & 1);
        if (masked && ok) {
          // slots behind the last hold anything, and a drafted token that some rows do not see
          // may hold values that are not finite: 0 x NaN must not reach them.  Thread r clears
          // line r of the value tile, or its values that are not finite (added again at the end).
          const uint32_t it = base + v_item(j, n), st = it % S::kBufs;
          ok = wait(&kv_full[st], (it / S::kBufs) & 1);
          const int slot = slot0 + r;
          if (ok && slot >= rq.len) {
            uint8_t* line = smem + S::kOffKV + st * S::kBuf + r * 128;
            bool bad = false;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
              uint4* at = reinterpret_cast<uint4*>(line + c / 8 * S::kHalf + ((c ^ r) & 7) * 16);
              if (slot >= rq.end) {
                *at = make_uint4(0, 0, 0, 0);
              } else {
                uint4 x = *at;
                float f[8];
                unpack_chunk<T>(x, f);
                bool any = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const bool finite = f[e] - f[e] == 0.f;
                  any = any || !finite;
                  f[e] = finite ? f[e] : 0.f;
                }
                if (any) {
                  *at = pack_chunk<T>(f);
                  bad = true;
                }
              }
            }
            if (bad) bad_s[piece & 1] = (int)piece + 1;
            fence_proxy_async_smem();
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (my_busy) {
          tc_fence_after_sync();
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
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float a = ex2_approx(fmaf(s[64 * c + 2 * e], sl, off));
              const float d = ex2_approx(fmaf(s[64 * c + 2 * e + 1], sl, off));
              sum[e & 3] += a + d;
              x[e] = pack2<T>(a, d);
            }
            tmem_st_32x32b_x32(tmem + lanes + kColP + 64 * buf + 32 * c, x);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st_wait();
          tc_fence_before_sync();
        }
        mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      // the next piece's queries go in while this one's last product runs
      more = pc.next(p);
      if (more) begin();
      const uint32_t t_last = tc + n - 1;
      ok = __all_sync(0xffffffffu, wait(&o_full[t_last & 1], (t_last >> 1) & 1));
      if (!ok) break;
      tc_fence_after_sync();
      const bool bad = bad_s[piece & 1] == (int)piece + 1;
      if (my_busy) {
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;     // (NaN stays)
        const int slot_part = 2 * blockIdx.x + (tile0 == 0 ? 1 : 0);
        float* part = p.partial + ((long long)slot_part * kTile + r) * (D + 2);
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
              for (int e = 0; e < 32; e += 2)
                *reinterpret_cast<float2*>(part + 32 * c + e) = make_float2(o[e], o[e + 1]);
            }
          }
        }
        if (my_row >= 0) {
          if (!whole) {
            part[D] = m == -INFINITY ? -INFINITY : m * sl;
            part[D + 1] = l;
          } else if (p.lse) {
            p.lse[(long long)my_row * p.group * p.cs.heads + my_head] =
                l == 0.f ? -INFINITY : (m * sl + log2f(l)) * 0.6931471805599453f;
          }
        }
      }
      if (!whole && tile0 == 0 && r == 0) {
        // the first part of several: the CTA of the last tile says how many
        const long long g0 = lo + (hi - lo) - n;              // (this is the CTA's last piece)
        const long long last = ((g0 + rq.tiles) * G - 1) / total;
        p.joins[blockIdx.x] = make_int4(b, block, head, (int)(last - blockIdx.x) + 1);
      }
      tc_fence_before_sync();
      base += 2 * n;
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

// Joins the parts of a (request, row block, head) that several CTAs share: CTA (c, y) those of
// the piece that CTA c began and left unfinished, 8 rows from 8 y on, a warp a row.
template <typename T, int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x, lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int4 join = p.joins[c];
  if (join.w < 2) return;
  const RequestRows rows = request_rows(p.rows, join.x, nullptr);
  const int i_r = join.y * kTile + r, i = i_r / p.group;
  if (i >= rows.n) return;
  auto part = [&](int k) {
    return p.partial + ((long long)(2 * (c + k) + (k == 0 ? 1 : 0)) * kTile + r) * (D + 2);
  };
  float M = -INFINITY;
  for (int k = lane; k < join.w; k += 32) M = fmaxf(M, part(k)[D]);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
  constexpr int E = D / 32;
  float o[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int k0 = 0; k0 < join.w; k0 += 4) {
    float x[4][E], ml[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k0 + u < join.w) {
        const float* a = part(k0 + u);
        ml[u][0] = a[D];
        ml[u][1] = a[D + 1];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = *reinterpret_cast<const float2*>(a + lane * E + e);
          x[u][e] = v.x;
          x[u][e + 1] = v.y;
        }
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k0 + u < join.w) {
        const float f = ml[u][0] == -INFINITY ? 0.f : ex2_approx(ml[u][0] - M);
        l = fmaf(ml[u][1], f, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(x[u][e], f, o[e]);
      }
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  const int row = rows.row0 + i, head = join.z * p.group + (i_r - i * p.group);
  T* dst = reinterpret_cast<T*>(p.out) + row * p.out_row + head * p.out_head + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack2<T>(o[e] * inv, o[e + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[(long long)row * p.group * p.cs.heads + head] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

bool encode_cache_map(CUtensorMap* map, const void* base, bool bf16, const CacheStrides& cs,
                      const TargetSlots& slots) {
  EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  const int page = 1 << slots.page_shift;
  cuuint64_t dims[4] = {(cuuint64_t)cs.head_dim, (cuuint64_t)page, (cuuint64_t)cs.heads, (cuuint64_t)slots.n_pages};
  cuuint64_t strides[3] = {(cuuint64_t)cs.slot * 2, (cuuint64_t)cs.head * 2, (cuuint64_t)cs.page * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)(page < kTile ? page : kTile), 1, 1};
  cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxGrid = 160;              // CTAs of the persistent grid at most
size_t joins_bytes() { return align_up((size_t)kMaxGrid * sizeof(int4), 256); }

template <typename T, int D>
cudaError_t attend_for(AttendParams p, const TargetSlots& slots, bool bf16, cudaStream_t stream) {
  static std::atomic<int> cache[kMaxCachedDevices];
  int grid = per_device_grid(cache, []() {
    return cudaFuncSetAttribute(attend_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttendSmem<D>::kBytes) == cudaSuccess ? 1 : -1;
  });
  if (grid <= 0) return cudaErrorInvalidConfiguration;
  if (grid > kMaxGrid) grid = kMaxGrid;
  CUtensorMap k_map, v_map;
  if (!encode_cache_map(&k_map, p.k, bf16, p.cs, slots) || !encode_cache_map(&v_map, p.v, bf16, p.cs, slots))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_pdl(attend_kernel<T, D>, dim3(grid), dim3(kThreads), AttendSmem<D>::kBytes, stream, k_map,
                             v_map, p);
  if (e != cudaSuccess) return e;
  const int rows = p.rows.N * p.group < kTile ? p.rows.N * p.group : kTile;
  return launch_pdl(join_kernel<T, D>, dim3(grid, cdiv(rows, 8)), dim3(256), 0, stream, p);
}

}  // namespace

size_t tree_attention_bytes(int B, int N, int q_heads, int heads, int head_dim) {
  (void)B;
  (void)N;
  (void)q_heads;
  (void)heads;
  return 256 + joins_bytes() + (size_t)2 * kMaxGrid * kTile * (head_dim + 2) * sizeof(float);
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
  p.joins = ws_at<int4>(ws, 256);
  p.partial = ws_at<float>(ws, 256 + joins_bytes());
  p.err = err;
  const bool bf16 = dtype == DSPARK_BF16;
  if (cs.head_dim == 128)
    return bf16 ? attend_for<__nv_bfloat16, 128>(p, slots, bf16, stream) : attend_for<__half, 128>(p, slots, bf16, stream);
  return bf16 ? attend_for<__nv_bfloat16, 64>(p, slots, bf16, stream) : attend_for<__half, 64>(p, slots, bf16, stream);
}

}  // namespace dspark
