// Log probabilities of given tokens, entropy, rank and top alternatives of rows of logits,
// and the gradient of the first two.
//
// billytse.dev DSpark page, section 1: the target's distribution of a position is the
// softmax of its logits row.  With m = max_v z_v and s = sum_v exp(z_v - m):
//   logprob = z_y - m - log s,   entropy = log s - sum_v exp(z_v - m) (z_v - m) / s,
//   rank    = 1 + #{v : z_v > z_y, or z_v = z_y and v < y},
// and the K largest logits (ties to the smallest v) with their log probabilities.
//
// Bound by the one read of the row from HBM.  A row is cut into the CTAs of a cluster (1, 2,
// 4 or 8).  Clusters are persistent, so that a row's end costs no memory time: a producer
// warp streams the parts of row after row through a ring of 16 KB pieces, eight consumer
// warps keep only sums, a maximum a thread and the maximum of every 64 bytes, and four
// closing warps do what a row still needs while the consumers are in the next one.
//
// The K best without a selection in the stream: the K-th largest of G >= 2 K maxima of groups
// of threads is a lower bound of the row's K-th largest logit that only slightly more than K
// elements reach (-G log(1 - K / G) of them for random data: 89 at K = 64, G = 128).  The few
// 64-byte slots whose maximum reaches it are read again, and one CTA of the cluster (in turn)
// ranks, by counting, the elements that the others send to it.  (Few logits above -inf, or many in
// ascending order, leave more candidates than fit, and sweep() below takes the row up tile by
// tile: 1536 x 129280 in fp32 with 10 logits left take 3.9 ms, with 100 0.82, ascending 57.)  The
// rank is counted in the stream: a sampled token may have hundreds of elements before it, and
// reading those again cost more than the stream (224 against 189 us at the size below).
//
// Measured on a GB300 (copy rate 6782 GB/s): 1536 rows of 129280 in fp32, 64 alternatives,
// 152 us = 5.2 TB/s (0.77 of the copy rate; 10.1 rounds of 152 clusters take 11, and a CTA
// stands still about 1500 of 23000 cycles between rows); 256 rows of 151936, 128 with a token,
// 20 alternatives, 24 us; rows of up to 64 KB by token_logprobs_short_kernel below.
#include "internal.h"
#include "rows.cuh"

namespace dspark {
namespace {

using namespace sm100;

constexpr int kLpWarps = 8, kLpThreads = kLpWarps * 32;   // consumers
constexpr int kLpClose = 128;               // closing threads (4 warps)
constexpr int kLpBlock = kLpThreads + 32 + kLpClose;
constexpr int kLpPieceChunks = 1024;        // 16 KB: 4 chunks (64 bytes) of each consumer
constexpr int kLpRing = 4;                  // pieces in flight, two CTAs an SM
// rows announced: the producer is at most 5 rows before the consumers' (its ring holds 4
// pieces of at least a row each), and those 2 before the closing warps
constexpr int kLpRows = 8;
constexpr int kLpSlots = 12;                // maxima of a consumer thread kept for a row
constexpr int kLpCap = 768;                 // candidate keys of a CTA
constexpr int kLpList = 512;                // slots listed to be read again
constexpr int kLpTop = kMaxTop;             // most alternatives
constexpr int kLpSwept = kMaxTopLength / 8; // elements of a CTA's part where there are any
constexpr int kLpMaxima = 256;              // most groups
constexpr int kLpShortSlots = 16;
// a short row: up to 64 KB (2000 rows of 16000 in fp32: 56 us, 80 by the ring)
constexpr int kLpShortChunks = 4096;

struct LpParams {
  const void* z;
  long long ld;
  const int32_t* tokens;     // may be null: every row is used, no logprob and no rank
  int N, V, K, log_per;      // 2^log_per pieces share a consumer thread's maximum
  float* logprob;
  float* entropy;
  int32_t* rank;
  float* row_max;
  float* row_sumexp;
  int32_t* top_ids;
  float* top_logprobs;
  int* err;
};

// 1 if a > b (a >= b), else 0
__device__ __forceinline__ float one_if_gt(float a, float b) {
  float r;
  asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float one_if_ge(float a, float b) {
  float r;
  asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// larger value first, then the smaller index; never 0 for an element that is not NaN
__device__ __forceinline__ unsigned long long top_key(float z, int idx) {
  return argmax_key(z + 0.f, idx);          // -0 orders as +0
}
__device__ __forceinline__ float key_value(unsigned long long key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ int key_index(unsigned long long key) {
  return (int)(0xFFFFFFFFu - (uint32_t)key);
}

// A maximum as a whole number of the same order (-0 just below +0).
__device__ __forceinline__ uint32_t group_key(float m) {
  const uint32_t u = __float_as_uint(m);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float group_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}
// A number that at least K of the n (at most 256) keys reach: the K-th largest less 1023 at
// most (2^-13 of its value), found by quartering the keys' range.  By a whole warp.
__device__ __forceinline__ uint32_t kth_bound(const uint32_t* keys, int n, int K) {
  const int lane = threadIdx.x & 31;
  uint32_t k[8], lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    k[i] = lane + 32 * i < n ? keys[lane + 32 * i] : 0u;      // 0: below every value
    if (lane + 32 * i < n) lo = min(lo, k[i]);
    hi = max(hi, k[i]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);   // all n reach it, and n >= K
  hi = __reduce_max_sync(0xffffffffu, hi);
  while (hi - lo > 1023u) {
    // three marks at once, their counts (256 at most) in 10 bits each
    const uint32_t step = (hi - lo) / 4 + 1;
    uint32_t reach = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < n)
        reach += (uint32_t)(k[i] >= lo + step) + ((uint32_t)(k[i] >= lo + 2 * step) << 10) +
                 ((uint32_t)(k[i] >= lo + 3 * step) << 20);
    reach = __reduce_add_sync(0xffffffffu, reach);
    if ((int)(reach >> 20) >= K) {
      lo += 3 * step;
    } else if ((int)(reach >> 10 & 1023u) >= K) {
      hi = lo + 3 * step - 1;
      lo += 2 * step;
    } else if ((int)(reach & 1023u) >= K) {
      hi = lo + 2 * step - 1;
      lo += step;
    } else {
      hi = lo + step - 1;
    }
  }
  return lo;
}

struct LpShared {
  unsigned long long cand[kLpCap];
  unsigned long long best[kLpTop];                    // this CTA's K best, then 0
  unsigned long long all[8 * kLpTop];                 // every CTA's, where they are merged
  float2 counts[8];                                   // and their number (as bits)
  uint32_t gmax[2][kLpMaxima];                        // this CTA's group maxima, as keys
  uint32_t gall[2][kLpMaxima];                        // the cluster's
  float4 part[2][kLpWarps];                           // a consumer warp's m, s, t, elements before y
  float2 ms[2][8 * kLpWarps];                         // the cluster's: m, s
  float2 tb[2][8 * kLpWarps];                         // t, elements before y (as bits)
  int list[kLpList];
  int n_cand, n_list;
  float thr;
  int row[kLpRows];                                   // the producer's rows, -1 after the last
  uint64_t row_full[kLpRows];
  uint64_t full[kLpRing], empty[kLpRing];
  uint64_t stats_full[2], stats_free[2];              // consumers to closing warps and back
  uint64_t sums_full[2], merge_full;                  // messages of the cluster's CTAs
};

// The rows of a cluster, in order, for a whole warp: every step-th row that has a token, so
// that rows without one leave no cluster idle.  (It reads all the tokens for that; above
// kLpDeal rows the rows are dealt by number instead, and those without a token skipped.)
constexpr int kLpDeal = 1 << 16;
struct RowsOf {
  static constexpr int kWindows = 8;         // of 32 rows, read together
  const int32_t* tokens;
  int N, V, step, want, n, seen;
  unsigned window[kWindows];                 // rows with a token from n on
  bool deal;
  __device__ __forceinline__ void look() {
    const int lane = threadIdx.x & 31;
    int y[kWindows];
#pragma unroll
    for (int i = 0; i < kWindows; ++i) y[i] = n + 32 * i + lane < N ? tokens[n + 32 * i + lane] : -1;
#pragma unroll
    for (int i = 0; i < kWindows; ++i) window[i] = __ballot_sync(0xffffffffu, y[i] >= 0 && y[i] < V);
  }
  __device__ __forceinline__ RowsOf(const int32_t* t, int N_, int V_, int first, int step_)
      : tokens(t), N(N_), V(V_), step(step_), want(first), n(0), seen(0), deal(t && N_ <= kLpDeal) {
    if (deal) look();
  }
  // the next row, or -1
  __device__ __forceinline__ int next() {
    if (!deal) {
      while (want < N) {
        const int r = want;
        want += step;
        if (!tokens || (tokens[r] >= 0 && tokens[r] < V)) return r;
      }
      return -1;
    }
    for (; n < N; look()) {
      int left = want - seen, found = -1, all = 0;
#pragma unroll
      for (int i = 0; i < kWindows; ++i) {
        const int c = __popc(window[i]);
        if (found < 0 && left < c) {
          unsigned w = window[i];
          for (int k = left; k > 0; --k) w &= w - 1;
          found = n + 32 * i + __ffs(w) - 1;
        }
        left -= c;
        all += c;
      }
      if (found >= 0) {
        want += step;
        return found;
      }
      seen += all;
      n += 32 * kWindows;
    }
    return -1;
  }
};

__device__ __forceinline__ void close_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kLpClose) : "memory");
}
// the barrier, and whether any closing thread has `p`
__device__ __forceinline__ bool close_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(kLpClose)
      : "memory");
  return r != 0;
}

// the outputs of a row without a token, by kLpClose threads
__device__ __forceinline__ void no_token(const LpParams& a, int n, int y, int x) {
  if (x == 0) {
    if (y != -1) set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
    a.logprob[n] = 0.f;
    a.rank[n] = 0;
    if (a.entropy) a.entropy[n] = 0.f;
    if (a.row_max) a.row_max[n] = -INFINITY;
    if (a.row_sumexp) a.row_sumexp[n] = 0.f;
  }
  for (int j = x; j < a.K; j += kLpClose) {
    a.top_ids[(size_t)n * a.K + j] = -1;
    a.top_logprobs[(size_t)n * a.K + j] = -INFINITY;
  }
}
// a row's single numbers, by one thread
__device__ __forceinline__ void write_row(const LpParams& a, int n, bool bad, float M, float S, float Tm,
                                          float logs, float zy, int before) {
  const float nan = __int_as_float(0x7FC00000);
  if (a.tokens) {
    a.logprob[n] = bad ? nan : S > 0.f ? zy - M - logs : -INFINITY;
    a.rank[n] = bad ? 0 : before + 1;
  }
  if (a.entropy) a.entropy[n] = bad ? nan : S > 0.f ? logs - Tm / S : 0.f;
  if (a.row_max) a.row_max[n] = M;
  if (a.row_sumexp) a.row_sumexp[n] = bad ? nan : S;
}

// best[0 .. K) = the K largest of cand[0 .. n), descending, then 0; returns min(n, K).  All
// closing threads; up to 64 keys by two threads a key, each against half of them.
template <typename Shared>
__device__ __forceinline__ int select_top(Shared& sh, int x, int n, int K) {
  if (n <= kLpClose / 2) {
    const int i = x >> 1;
    const unsigned long long key = i < n ? sh.cand[i] : 0ull;
    int r = 0;
#pragma unroll 4
    for (int j = x & 1; j < n; j += 2) r += sh.cand[j] > key;
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    if (i < n && r < K && (x & 1) == 0) sh.best[r] = key;
  } else {
    for (int i = x; i < n; i += kLpClose) {
      const unsigned long long key = sh.cand[i];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) r += sh.cand[j] > key;
      if (r < K) sh.best[r] = key;
    }
  }
  for (int i = n + x; i < K; i += kLpClose) sh.best[i] = 0ull;
  close_sync();
  return n < K ? n : K;
}

// The same where more elements reach the bound than keys fit (equal logits, or all the large
// ones in few threads' hands): the selection goes tile by tile over the elements [from, to) and
// keeps the K best in sh.best, `got` of them so far.  A tile whose every element is better than
// all before takes up to 112000 cycles (K = 128, both CTAs of an SM at it), and the row two rows
// on waits for it: 2^23 elements a CTA take 1.5e9 cycles, a wait ends after 4e9.
template <typename Shared, typename T>
__device__ __noinline__ void sweep(Shared& sh, int x, const T* row, int from, int to, int K, int& got) {
  constexpr int kTile = (kLpCap - kLpTop) / kLpClose * kLpClose;
  for (int base = from; base < to; base += kTile) {
    close_sync();
    if (x == 0) sh.n_cand = got;
    for (int j = x; j < got; j += kLpClose) sh.cand[j] = sh.best[j];
    const unsigned long long floor_key = got == K ? sh.best[K - 1] : 0ull;
    close_sync();
    for (int v = base + x; v < min(to, base + kTile); v += kLpClose) {
      const float z = elem_to_float(row[v]);
      const unsigned long long key = top_key(z, v);
      if (z == z && key > floor_key) sh.cand[atomicAdd(&sh.n_cand, 1)] = key;
    }
    close_sync();
    if (sh.n_cand > got) got = select_top(sh, x, sh.n_cand, K);
  }
}

// Short rows: a CTA of 128 threads a row, with the same bound, re-read and ranking; many CTAs
// an SM hide a row's steps behind other rows.
struct LpShortShared {
  unsigned long long cand[kLpCap];
  unsigned long long best[kLpTop];
  uint32_t gmax[kLpMaxima];
  float4 part[kLpClose / 32];
  float slots[kLpShortSlots][kLpClose];
  int list[kLpList];
  float thr;
  int n_cand, n_list;
};
template <typename T>
__global__ void __launch_bounds__(kLpClose, 8) token_logprobs_short_kernel(LpParams a) {
  constexpr int N = Chunk<T>::N, G = 16 / N, kThreads = kLpClose, kWarps = kThreads / 32;
  __shared__ LpShortShared sh;
  const int x = threadIdx.x, lane = x & 31, warp = x >> 5;
  const int n = blockIdx.x, V = a.V, K = a.K;
  pdl_wait();
  pdl_launch_dependents();
  const float nan = __int_as_float(0x7FC00000);
  const int y = a.tokens ? a.tokens[n] : 0;
  if (y < 0 || y >= V) {
    no_token(a, n, y, x);
    return;
  }
  if (x == 0) sh.n_cand = sh.n_list = 0;
  const RowPart<T> r = row_part<T>(a.z, a.ld, n, V, 0, 0, 0x7FFFFFFF);
  const float zy = a.tokens ? elem_to_float(r.row[y]) : INFINITY;
  const int loose_n = r.rc.head + r.rc.tail;
  const int loose = x < r.rc.head ? x : V - r.rc.tail + (x - r.rc.head);
  const float zl = x < loose_n ? elem_to_float(r.row[loose]) : -INFINITY;
  RunningSoftmax rs;
  rs.init();
  float tmax[2] = {-INFINITY, -INFINITY};    // of even slots and odd ones
  int before = 0, used = 0;
  // (16 elements a slot: G chunks, kThreads apart)
  for (int i = x; i < r.held; i += G * kThreads, ++used) {
    float z[16];
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const int j = i + u * kThreads;
      float e[N];
      if (j < r.held) {
        unpack_chunk<T>(__ldg(r.body + j), e);
        const int v = r.rc.head + j * N;
        if (a.tokens) {
#pragma unroll
          for (int k = 0; k < N; ++k) before += e[k] > zy || (e[k] == zy && v + k < y);
        }
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) e[k] = -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < N; ++k) z[u * N + k] = e[k];
    }
    const float bm = max_of(z);
    rs.add(z, bm);
    sh.slots[used][x] = bm;
    const float even = tmax[0];              // (the two change places with every slot)
    tmax[0] = tmax[1];
    tmax[1] = fmaxf(even, bm);
  }
  if (x < loose_n) {
    rs.add_one(zl);
    tmax[0] = fmaxf(tmax[0], zl);
    before += zl > zy || (zl == zy && loose < y);
  }
  {
    const float m = warp_max(fmaxf(tmax[0], tmax[1]));
    float s, t;
    rs.finish(m, s, t);
    s = warp_sum(s);
    t = warp_sum(t);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) sh.part[warp] = make_float4(m, s, t, __int_as_float(before));
  }
  int groups = 32;
  while (groups < 2 * K && groups < kLpMaxima) groups <<= 1;
  if (groups == kLpMaxima) {
    sh.gmax[x] = group_key(tmax[0]);
    sh.gmax[kThreads + x] = group_key(tmax[1]);
  } else {
    float g = fmaxf(tmax[0], tmax[1]);
    for (int o = 16; o >= groups / kWarps; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (lane < groups / kWarps) sh.gmax[warp * (groups / kWarps) + lane] = group_key(g);
  }
  __syncthreads();
  float M = -INFINITY, S = 0.f, Tm = 0.f;
  before = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sh.part[i].x);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const float4 p = sh.part[i];
    before += __float_as_int(p.w);
    if (p.y != 0.f) {
      const float d = p.x - M, f = ex2_approx(d * kLog2e);
      S += p.y * f;
      if (f > 0.f) Tm += f * (p.z + d * p.y);
    }
  }
  const bool bad = !(S <= FLT_MAX);          // NaN or +inf among the logits
  const float logs = logf(S);
  if (x == 0) write_row(a, n, bad, M, S, Tm, logs, zy, before);
  if (K == 0) return;
  if (warp == 0) {
    const uint32_t key = kth_bound(sh.gmax, groups, K);
    if (lane == 0) sh.thr = group_value(key);
  }
  __syncthreads();
  const float thr = sh.thr;
  auto consider = [&](float z, int v) {
    if (z >= thr) {
      const int to = atomicAdd(&sh.n_cand, 1);
      if (to < kLpCap) sh.cand[to] = top_key(z, v);
    }
  };
  if (x < loose_n) consider(zl, loose);
  // the slots that reach the bound, listed, then their chunks dealt over all threads
  unsigned hits = 0u;
#pragma unroll
  for (int u = 0; u < kLpShortSlots; ++u) hits |= (unsigned)(u < used && sh.slots[u][x] >= thr) << u;
  if (hits) {
    int to = atomicAdd(&sh.n_list, __popc(hits));
    for (unsigned left = hits; left; left &= left - 1, ++to)
      if (to < kLpList) sh.list[to] = (__ffs(left) - 1) * kThreads + x;
  }
  __syncthreads();
  auto look = [&](int entry, int g) {        // chunk g of a slot
    const int j = (entry & (kThreads - 1)) + (entry / kThreads * G + g) * kThreads;
    if (j >= r.held) return;
    float z[N];
    unpack_chunk<T>(__ldg(r.body + j), z);
    if (max_of(z) >= thr) {
#pragma unroll
      for (int e = 0; e < N; ++e) consider(z[e], r.rc.head + j * N + e);
    }
  };
  if (sh.n_list <= kLpList) {
    for (int k = x; k < sh.n_list * G; k += kThreads) look(sh.list[k / G], k % G);
  } else {
    for (; hits; hits &= hits - 1)
      for (int g = 0; g < G; ++g) look((__ffs(hits) - 1) * kThreads + x, g);
  }
  __syncthreads();
  int got = 0;
  if (sh.n_cand <= kLpCap) {
    got = select_top(sh, x, sh.n_cand, K);
  } else {
    sweep(sh, x, r.row, 0, V, K, got);
  }
  for (int j = x; j < K; j += kThreads) {
    const unsigned long long key = j < got ? sh.best[j] : 0ull;
    const size_t o = (size_t)n * K + j;
    a.top_ids[o] = bad || j >= got ? -1 : key_index(key);
    a.top_logprobs[o] = bad ? nan : j < got && S > 0.f ? key_value(key) - M - logs : -INFINITY;
  }
}

template <typename T>
__global__ void __launch_bounds__(kLpBlock, 2) token_logprobs_kernel(LpParams a, int log_C) {
  constexpr int N = Chunk<T>::N;
  extern __shared__ __align__(128) uint4 ring_s[];    // [kLpRing][1024], then the slot maxima
  __shared__ LpShared sh;
  float* const slots_s = reinterpret_cast<float*>(ring_s + kLpRing * kLpPieceChunks);   // [2][kLpSlots][256]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = 1 << log_C;                  // CTAs of a row
  const int c = (int)(blockIdx.x & (C - 1)), first = (int)(blockIdx.x >> log_C), step = (int)(gridDim.x >> log_C);
  const int V = a.V, K = a.K;
  // groups of the cluster (at least one a warp) and of this CTA
  int log_G = log_C + 3;
  while ((1 << log_G) < 2 * K && (1 << log_G) < kLpMaxima) ++log_G;
  const int G = 1 << log_G, log_own = log_G - log_C, own = 1 << log_own;
  if (tid == 0) {
    for (int i = 0; i < kLpRing; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kLpWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.stats_full[i], kLpWarps);
      mbar_init(&sh.stats_free[i], 1);
      mbar_init(&sh.sums_full[i], 1);
    }
    for (int i = 0; i < kLpRows; ++i) mbar_init(&sh.row_full[i], 1);
    mbar_init(&sh.merge_full, 1);
    fence_mbar_init();
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  auto part_of = [&](int n) { return row_part<T>(a.z, a.ld, n, V, c, log_C, 0x7FFFFFFF); };
  bool late = false;                         // a bounded wait ran out: give up
  // the cluster's it-th row, or -1; by whole warps
  auto announced = [&](int it) {
    const bool ok = mbar_wait(&sh.row_full[it % kLpRows], (it / kLpRows) & 1);
    if (!__all_sync(0xffffffffu, ok)) {
      late = true;
      return -1;
    }
    return sh.row[it % kLpRows];
  };

  if (warp < kLpWarps) {
    // ---- consumers
    int it = 0, slot = 0;
    uint32_t phase = 0;
    while (!late) {
      const int n = announced(it);
      if (n < 0) break;
      const int y = a.tokens ? a.tokens[n] : 0;
      const int b = it & 1;
      const RowPart<T> r = part_of(n);
      const int loose_n = c == 0 ? r.rc.head + r.rc.tail : 0;   // elements outside the chunks
      const float zl = tid < loose_n
                           ? elem_to_float(r.row[tid < r.rc.head ? tid : V - r.rc.tail + (tid - r.rc.head)])
                           : -INFINITY;
      if (it >= 2 && !mbar_wait(&sh.stats_free[b], ((it >> 1) - 1) & 1)) late = true;
      RunningSoftmax rs;
      rs.init();
      float tmax = -INFINITY, smax = -INFINITY;
      // elements before y: those above its logit, and equal ones of lower index
      const float zy = a.tokens ? elem_to_float(r.row[y]) : INFINITY;
      F2 before = f2(0.f, 0.f);
      float* out = slots_s + b * kLpSlots * kLpThreads + tid;
      for (int i = 0; i < r.held; i += kLpPieceChunks) {
        if (!late && !mbar_wait(&sh.full[slot], phase)) late = true;
        // a thread's 4 chunks lie together; each group of 8 lanes reads other banks
        const uint4* piece = ring_s + slot * kLpPieceChunks + 4 * tid;
        const int turn = (tid >> 1) & 3, left = r.held - i - 4 * tid;
        // (the 64 bytes that hold y itself are counted element by element)
        const int v0 = r.rc.head + (r.c0 + i + 4 * tid) * N;
        const bool ahead = v0 + 4 * N <= y;  // all of them before y: equal ones count
        auto take = [&](const auto& q) {
          constexpr int M = sizeof(q) / sizeof(q[0]);
          float z[M * N];
#pragma unroll
          for (int g = 0; g < M; ++g) {
            float x[N];
            unpack_chunk<T>(q[g], x);
#pragma unroll
            for (int e = 0; e < N; ++e) z[g * N + e] = x[e];
          }
          const float bm = max_of(z);
          smax = fmaxf(smax, bm);
          rs.add(z, bm);
          if (a.tokens) {
            if (ahead) {
#pragma unroll
              for (int e = 0; e < M * N; e += 2)
                before = f2_add(before, f2(one_if_ge(z[e], zy), one_if_ge(z[e + 1], zy)));
            } else {
#pragma unroll
              for (int e = 0; e < M * N; e += 2)
                before = f2_add(before, f2(one_if_gt(z[e], zy), one_if_gt(z[e + 1], zy)));
            }
          }
        };
        constexpr int M = 16 / N;            // chunks of 16 elements
        if (left >= 4) {
#pragma unroll
          for (int g = 0; g < 4; g += M) {
            uint4 q[M];
#pragma unroll
            for (int u = 0; u < M; ++u) q[u] = piece[(g + u + turn) & 3];
            take(q);
          }
        } else {
          for (int g = 0; g < left; ++g) {
            const uint4 q[1] = {piece[g]};
            take(q);
          }
        }
        if (a.tokens && v0 <= y && y < v0 + 4 * N) {
          // the 64 bytes that hold y, or end before it: equal elements before it
          const T* z = reinterpret_cast<const T*>(piece);
          for (int e = 0; e < min(y - v0, left * N); ++e) before = f2_add(before, f2(elem_to_float(z[e]) == zy ? 1.f : 0.f, 0.f));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[slot]);
        if (++slot == kLpRing) {
          slot = 0;
          phase ^= 1;
        }
        const int done = i / kLpPieceChunks + 1;
        if ((done & ((1 << a.log_per) - 1)) == 0 || i + kLpPieceChunks >= r.held) {
          *out = smax;
          out += kLpThreads;
          tmax = fmaxf(tmax, smax);
          smax = -INFINITY;
        }
      }
      if (tid < loose_n) {
        rs.add_one(zl);
        tmax = fmaxf(tmax, zl);
        const int v = tid < r.rc.head ? tid : V - r.rc.tail + (tid - r.rc.head);
        if (zl > zy || (zl == zy && v < y)) before = f2_add(before, f2(1.f, 0.f));
      }
      const float m = warp_max(tmax);
      float s, t;
      rs.finish(m, s, t);
      s = warp_sum(s);
      t = warp_sum(t);
      float n0, n1;
      f2_get(before, n0, n1);                // whole numbers below 2^24: V / 512 at most
      const int n_before = __reduce_add_sync(0xffffffffu, (int)n0 + (int)n1);
      if (lane == 0) sh.part[b][warp] = make_float4(m, s, t, __int_as_float(n_before));
      float g = tmax;
      for (int o = 16; o >= own / kLpWarps; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
      if (lane < own / kLpWarps) {
        sh.gmax[b][warp * (own / kLpWarps) + lane] = group_key(g);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.stats_full[b]);
      late = __any_sync(0xffffffffu, late);
      ++it;
    }
  } else if (warp == kLpWarps) {
    // ---- producer
    int sent = 0;
    RowsOf rows(a.tokens, a.N, V, first, step);
    for (int it = 0;; ++it) {
      const int n = rows.next();
      if (lane == 0) {
        sh.row[it % kLpRows] = n;
        mbar_arrive(&sh.row_full[it % kLpRows]);
      }
      if (n < 0) break;
      if (lane == 0) {
        const RowPart<T> r = part_of(n);
        for (int i = 0; i < r.held; i += kLpPieceChunks, ++sent) {
          const int slot = sent % kLpRing, use = sent / kLpRing;
          if (use > 0 && !mbar_wait(&sh.empty[slot], (use - 1) & 1)) { late = true; break; }
          const int k = min(kLpPieceChunks, r.held - i);
          mbar_arrive_expect_tx(&sh.full[slot], (uint32_t)k * 16u);
          bulk_load(ring_s + slot * kLpPieceChunks, r.body + r.c0 + i, (uint32_t)k * 16u, &sh.full[slot]);
        }
      }
      late = __any_sync(0xffffffffu, late);
      if (late) break;
    }
    if (lane == 0) {
      // copies in flight end before the CTA does (at once, unless the consumers gave up)
      for (int j = max(0, sent - kLpRing); j < sent; ++j) mbar_wait(&sh.full[j % kLpRing], (j / kLpRing) & 1);
    }
  } else {
    // ---- closing warps
    const int x = tid - kLpThreads - 32;     // 0 .. 127
    const float nan = __int_as_float(0x7FC00000);
    // The row that this CTA has yet to merge: the other CTAs' lists are awaited only when the
    // next row's messages are sent, so that no CTA waits for a merge.
    struct {
      int n;
      uint32_t phase;
      float M, S, Tm, zy;
      int before;
    } pend = {-1, 0u, 0.f, 0.f, 0.f, 0.f, 0};
    auto merge = [&] {
      const int n = pend.n;
      pend.n = -1;
      late = close_any(late || !wait_cluster(&sh.merge_full, pend.phase));
      if (late) return;                      // (the lists' lengths are not there)
      const bool bad = !(pend.S <= FLT_MAX); // NaN or +inf among the logits
      const float logs = logf(pend.S);
      // keys of the lists up to this lane's
      int upto = lane < C ? __float_as_int(sh.counts[lane].x) : 0;
      for (int o = 1; o < 8; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const int total = __shfl_sync(0xffffffffu, upto, 7);
      if (x == 0) write_row(a, n, bad, pend.M, pend.S, pend.Tm, logs, pend.zy, pend.before);
      auto put = [&](int at, int id, float lp) {
        const size_t o = (size_t)n * K + at;
        a.top_ids[o] = bad ? -1 : id;
        a.top_logprobs[o] = bad ? nan : lp;
      };
      // a thread a key: its place is the number of keys above it
      for (int base = 0; base < total; base += kLpClose) {
        const int p = base + x;
        int list = 0, start = 0;
        for (int o = 0; o < C; ++o) {
          const int end = __shfl_sync(0xffffffffu, upto, o);
          if (p >= end) {
            list = o + 1;
            start = end;
          }
        }
        const unsigned long long key = p < total ? sh.all[list * K + p - start] : ~0ull;
        int at = 0, from = 0;
        for (int o = 0; o < C; ++o) {
          const int end = __shfl_sync(0xffffffffu, upto, o);
          const unsigned long long* other = sh.all + o * K;
#pragma unroll 4
          for (int j = 0; j < end - from; ++j) at += other[j] > key;
          from = end;
        }
        if (p < total && at < K) put(at, key_index(key), pend.S > 0.f ? key_value(key) - pend.M - logs : -INFINITY);
      }
      for (int j = total + x; j < K; j += kLpClose) put(j, -1, -INFINITY);
      late = close_any(late);                // also: all[] is free for the next row merged here
    };
    // the rows without a token
    if (a.tokens && c == 0)
      for (int n = first; n < a.N; n += step) {
        const int y = a.tokens[n];
        if (y >= 0 && y < V) continue;
        no_token(a, n, y, x);
      }
    int it = 0;
    for (;;) {
      const int n = announced(it);
      late = close_any(late);
      if (late || n < 0) break;
      const int y = a.tokens ? a.tokens[n] : 0;
      const int b = it & 1;
      const uint32_t buf_phase = (it >> 1) & 1;
      const int merger = it & (C - 1);       // the CTA that merges this row
      if (x == 0) {
        mbar_arrive_expect_tx(&sh.sums_full[b], (uint32_t)(C * kLpWarps * 16 + (K > 0 ? G * 4 : 0)));
        sh.n_cand = 0;
        sh.n_list = 0;
      }
      const RowPart<T> r = part_of(n);
      const float zy = a.tokens ? elem_to_float(r.row[y]) : INFINITY;
      const int loose_n = c == 0 ? r.rc.head + r.rc.tail : 0;
      const int loose = x < r.rc.head ? x : V - r.rc.tail + (x - r.rc.head);
      const float zl = x < loose_n ? elem_to_float(r.row[loose]) : -INFINITY;

      // ---- the row's statistics: every CTA's warps' parts to every CTA
      if (!mbar_wait(&sh.stats_full[b], buf_phase)) late = true;
      if (x < C * kLpWarps) {                // 64 at most
        const int o = x / kLpWarps, w = x % kLpWarps;
        const float4 p = sh.part[b][w];
        send_f2(&sh.ms[b][c * kLpWarps + w], &sh.sums_full[b], o, p.x, p.y);
        send_f2(&sh.tb[b][c * kLpWarps + w], &sh.sums_full[b], o, p.z, p.w);
      }
      if (K > 0)
        for (int k = x; k < G; k += kLpClose) {
          const int o = k >> log_own, j = k & (own - 1);
          send_f(reinterpret_cast<float*>(&sh.gall[b][c * own + j]), &sh.sums_full[b], o,
                 __uint_as_float(sh.gmax[b][j]));
        }
      if (pend.n >= 0) merge();
      if (c == merger && x == 0) mbar_arrive_expect_tx(&sh.merge_full, (uint32_t)(C * (8 + 8 * K)));
      if (!late && !wait_cluster(&sh.sums_full[b], buf_phase)) late = true;
      late = close_any(late);
      if (late) break;
      float M = -INFINITY, S = 0.f, Tm = 0.f;
      int before = 0;
      {
        float2 p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int w = lane + 32 * i;
          p[i] = w < C * kLpWarps ? sh.ms[b][w] : make_float2(-INFINITY, 0.f);
          M = fmaxf(M, p[i].x);
        }
        M = warp_max(M);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int w = lane + 32 * i;
          const float2 tb = w < C * kLpWarps ? sh.tb[b][w] : make_float2(0.f, 0.f);
          before += __float_as_int(tb.y);
          if (p[i].y != 0.f) {
            const float d = p[i].x - M, f = ex2_approx(d * kLog2e);
            S += p[i].y * f;
            if (f > 0.f) Tm += f * (tb.x + d * p[i].y);
          }
        }
        S = warp_sum(S);
        Tm = warp_sum(Tm);
        before = __reduce_add_sync(0xffffffffu, before);
      }

      // ---- a lower bound of the row's K-th largest element, from the maxima of its groups
      // (by one warp: four would take issue slots from the consumers)
      if (K > 0 && x < 32) {
        const uint32_t key = kth_bound(sh.gall[b], G, K);
        if (lane == 0) sh.thr = group_value(key);
      }
      close_sync();
      const float thr = K > 0 ? sh.thr : INFINITY;

      // ---- candidates for the K best: the slots that reach the bound
      int got = 0;
      if (K > 0) {
        auto consider = [&](float z, int v) {
          if (z >= thr) {
            const int to = atomicAdd(&sh.n_cand, 1);
            if (to < kLpCap) sh.cand[to] = top_key(z, v);
          }
        };
        if (x < loose_n) consider(zl, loose);
        const int pieces = (r.held + kLpPieceChunks - 1) / kLpPieceChunks;
        const int used = (pieces + (1 << a.log_per) - 1) >> a.log_per;
        const float4* maxima = reinterpret_cast<const float4*>(slots_s + b * kLpSlots * kLpThreads);
        float4 m4[kLpSlots * kLpThreads / 4 / kLpClose];
#pragma unroll
        for (int i = 0; i < kLpSlots * kLpThreads / 4 / kLpClose; ++i) {
          const int e = x + i * kLpClose;
          m4[i] = e < used * (kLpThreads / 4) ? maxima[e] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        }
#pragma unroll
        for (int i = 0; i < kLpSlots * kLpThreads / 4 / kLpClose; ++i) {
          const int e = x + i * kLpClose;
          const int hits = (m4[i].x >= thr) + 2 * (m4[i].y >= thr) + 4 * (m4[i].z >= thr) + 8 * (m4[i].w >= thr);
          if (hits && e < used * (kLpThreads / 4)) {
            int to = atomicAdd(&sh.n_list, __popc(hits));
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (hits >> u & 1) {
                if (to < kLpList) sh.list[to] = 4 * e + u;
                ++to;
              }
          }
        }
        close_sync();
        auto look = [&](int entry, int g) {  // chunk g of an entry's slot
          const int j = (((entry / kLpThreads) << a.log_per) + (g >> 2)) * kLpPieceChunks +
                        4 * (entry & (kLpThreads - 1)) + (g & 3);
          if (j >= r.held) return;
          float z[N];
          unpack_chunk<T>(__ldg(r.body + r.c0 + j), z);
          if (max_of(z) >= thr) {
            const int v = r.rc.head + (r.c0 + j) * N;
#pragma unroll
            for (int e = 0; e < N; ++e) consider(z[e], v + e);
          }
        };
        const int log_per = a.log_per + 2, n_list = sh.n_list;
        if (n_list <= kLpList) {
          for (int k = x; k < n_list << log_per; k += kLpClose) look(sh.list[k >> log_per], k & ((1 << log_per) - 1));
        } else {
          for (int e = x; e < used * kLpThreads; e += kLpClose)
            if (reinterpret_cast<const float*>(maxima)[e] >= thr)
              for (int g = 0; g < 1 << log_per; ++g) look(e, g);
        }
        close_sync();
        if (x == 0) mbar_arrive(&sh.stats_free[b]);
        const int n_cand = sh.n_cand;
        if (n_cand <= K) {                   // (the merge ranks them)
          got = n_cand;
          for (int j = x; j < K; j += kLpClose) sh.best[j] = j < n_cand ? sh.cand[j] : 0ull;
          close_sync();
        } else if (n_cand <= kLpCap) {
          got = select_top(sh, x, n_cand, K);
        } else {
          if (c == 0) sweep(sh, x, r.row, 0, r.rc.head, K, got);
          sweep(sh, x, r.row, r.rc.head + r.c0 * N, r.rc.head + r.c1 * N, K, got);
          if (c == 0) sweep(sh, x, r.row, V - r.rc.tail, V, K, got);
          if (got == 0) select_top(sh, x, 0, K);
        }
        for (int j = x; j < K; j += kLpClose) send_u64(&sh.all[c * K + j], &sh.merge_full, merger, sh.best[j]);
      } else if (x == 0) {
        mbar_arrive(&sh.stats_free[b]);
      }
      if (x == 0) send_f2(&sh.counts[c], &sh.merge_full, merger, __int_as_float(got), 0.f);

      if (c == merger) {
        pend.n = n;
        pend.phase = (it >> log_C) & 1;
        pend.M = M;
        pend.S = S;
        pend.Tm = Tm;
        pend.zy = zy;
        pend.before = before;
      }
      ++it;
    }
    if (pend.n >= 0 && !late) merge();
  }
  if (late) set_device_error(a.err, DSPARK_ERR_TIMEOUT);
  __syncwarp();
  if (C > 1) cluster_sync();                 // no CTA leaves while another may still send to it
}

// ------------------------------------------------------------------------------ gradient
// dz_v = g_lp ([v = y] - p_v) - g_H p_v (log p_v + H), p_v = exp(z_v - m) / s: one read and
// one write of the row, nothing kept between them, so a grid of independent segments of 64 KB
// (four 16-byte loads a thread in flight).  Bound by memory: 1280 rows of 129280 in bf16, 1152
// with a token, 99 us = 6.35 TB/s (0.94 of the copy rate).
constexpr int kLgThreads = 256;
constexpr int kLgBatch = 4;

struct LgParams {
  const void* z;
  long long ld;
  const int32_t* tokens;
  int V, segs;
  const float* row_max;
  const float* row_sumexp;
  const float* entropy;
  const float* d_logprob;    // may be null
  const float* d_entropy;    // may be null
  void* dz;
  long long ld_dz;
  int* err;
};

template <typename T>
__global__ void __launch_bounds__(kLgThreads) token_logprobs_grad_kernel(LgParams a) {
  constexpr int N = Chunk<T>::N;
  const int tid = threadIdx.x;
  const int n = (int)(blockIdx.x / a.segs);
  const int seg = (int)(blockIdx.x - (unsigned)n * a.segs);
  const int V = a.V;
  pdl_wait();
  pdl_launch_dependents();
  const T* row = static_cast<const T*>(a.z) + (long long)n * a.ld;
  T* out = static_cast<T*>(a.dz) + (long long)n * a.ld_dz;
  const int y = a.tokens[n];
  const float m = a.row_max[n], s = a.row_sumexp[n], H = a.entropy ? a.entropy[n] : 0.f;
  const float gl = a.d_logprob ? a.d_logprob[n] : 0.f, gh = a.d_entropy ? a.d_entropy[n] : 0.f;
  const bool in = y >= 0 && y < V;
  const bool off = !in || s == 0.f;         // no token, or no logit above -inf
  if (!in && y != -1 && tid == 0 && seg == 0) set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
  const float inv = 1.f / s, logs = logf(s), w0 = -gl - gh * H;
  // p (-g_lp - g_H (log p + H)); log p below -200 is p = 0 (and 0 * -inf is avoided)
  auto grad = [&](float z) {
    const float d = z - m;
    const float p = ex2_approx(d * kLog2e) * inv;
    return p * fmaf(-gh, fmaxf(d - logs, -200.f), w0);
  };
  const RowChunks rc = row_chunks(out, V);
  const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  if (seg == 0) {
    const int loose = tid < rc.head ? tid : V - rc.tail + (tid - rc.head);
    if (tid < rc.head + rc.tail) {
      const float g = off ? 0.f : grad(elem_to_float(row[loose])) + (loose == y ? gl : 0.f);
      out[loose] = elem_from_float<T>(g);
    }
  }
  const int c0 = (int)((long long)rc.chunks * seg / a.segs);
  const int c1 = (int)((long long)rc.chunks * (seg + 1) / a.segs);
  const uint4* in4 = reinterpret_cast<const uint4*>(row + rc.head);
  uint4* out4 = reinterpret_cast<uint4*>(out + rc.head);
  if (off) {
    for (int i = c0 + tid; i < c1; i += kLgThreads) __stcs(out4 + i, make_uint4(0u, 0u, 0u, 0u));
    return;
  }
  auto finish = [&](float (&z)[N], int i) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = grad(z[e]);
    const int ry = y - rc.head - i * N;
    if (ry >= 0 && ry < N) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e == ry) z[e] += gl;
    }
    __stcs(out4 + i, pack_chunk<T>(z));
  };
  if (same) {
    int i = c0 + tid;
    for (; i + (kLgBatch - 1) * kLgThreads < c1; i += kLgBatch * kLgThreads) {
      uint4 q[kLgBatch];
#pragma unroll
      for (int g = 0; g < kLgBatch; ++g) q[g] = __ldcs(in4 + i + g * kLgThreads);
#pragma unroll
      for (int g = 0; g < kLgBatch; ++g) {
        float z[N];
        unpack_chunk<T>(q[g], z);
        finish(z, i + g * kLgThreads);
      }
    }
    for (; i < c1; i += kLgThreads) {
      float z[N];
      unpack_chunk<T>(__ldcs(in4 + i), z);
      finish(z, i);
    }
  } else {                                  // input rows off the output rows' 16-byte grid
    const T* src = row + rc.head;
    for (int i = c0 + tid; i < c1; i += kLgThreads) {
      float z[N];
#pragma unroll
      for (int e = 0; e < N; ++e) z[e] = elem_to_float(src[(long long)i * N + e]);
      finish(z, i);
    }
  }
}

template <typename T>
cudaError_t launch_lp(LpParams p, cudaStream_t stream) {
  const int chunks = p.V / Chunk<T>::N;
  // (20 rows of 16000 in fp32, 64 KB: 15 us, 13 by the ring; of 8000 no difference)
  if (chunks <= kLpShortChunks / 2 || (chunks <= kLpShortChunks && p.N >= 304)) {
    static_assert(kLpShortChunks * Chunk<T>::N <= kLpShortSlots * kLpClose * 16, "slots of a short row");
    return launch_pdl(token_logprobs_short_kernel<T>, dim3((unsigned)p.N), dim3(kLpClose), 0, stream, p);
  }
  const size_t smem = (size_t)kLpRing * kLpPieceChunks * 16 + 2 * kLpSlots * kLpThreads * sizeof(float);
  static std::atomic<int> cache[4][kMaxCachedDevices];
  // CTAs a row is cut into: the fewest estimated cycles, a CTA streaming 12 bytes a cycle and
  // closing a row in 14000 (measured with both CTAs of an SM at work), beside the next row's
  // stream.  1536 rows of 129280 in fp32: 1, 2, 4 CTAs took 164, 152, 201 us; 256 rows
  // of 151936, half of them with a token: 1, 2, 4, 8 took 35, 24, 28, 37; 64 rows: 29, 20, 16, 20
  int log_C = 0, clusters = 0;
  long long best = 0;
  for (int i = 3; i >= 0; --i) {
    if (i > 0 && (chunks >> i) < kLpPieceChunks) continue;
    if (i < 3 && p.K > 0 && (p.V >> i) > kLpSwept) break;
    const int most = device_clusters(cache[i], token_logprobs_kernel<T>, 1 << i, kLpBlock, smem);
    if (most <= 0) return cudaErrorInvalidConfiguration;
    const long long stream_c = (long long)(chunks >> i) * 16 / 12, close_c = 14000;
    const long long rounds = cdiv(p.N, most);
    const long long cost = stream_c + (rounds - 1) * (stream_c > close_c ? stream_c : close_c) + close_c;
    if (clusters == 0 || cost < best) {
      best = cost;
      log_C = i;
      clusters = p.N < most ? p.N : most;
    }
  }
  const int pieces = cdiv((chunks >> log_C) + 1, kLpPieceChunks);
  while (pieces > kLpSlots << p.log_per) ++p.log_per;
  return launch_rows_cluster(token_logprobs_kernel<T>, (long long)clusters << log_C, 1 << log_C, kLpBlock, smem, stream,
                             p, log_C);
}

template <typename T>
cudaError_t launch_lg(LgParams p, int N, cudaStream_t stream) {
  const int chunks = p.V / Chunk<T>::N;
  // segments of about 4096 chunks (64 KB), or as many as give every SM eight CTAs; one where a
  // row is shorter than a chunk
  int segs = chunks > 0 ? cdiv(chunks, 4096) : 1;
  while ((long long)segs * N < 2LL * kTargetCtas && chunks / (segs * 2) >= kLgThreads) segs *= 2;
  p.segs = segs;
  return launch_pdl(token_logprobs_grad_kernel<T>, dim3((unsigned)((long long)segs * N)),
                    dim3(kLgThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_token_logprobs(const void* z, int dtype, long long ld, const int32_t* tokens,
                                  int N, int V, int K, float* logprob, float* entropy, int32_t* rank,
                                  float* row_max, float* row_sumexp, int32_t* top_ids,
                                  float* top_logprobs, int* err, cudaStream_t stream) {
  LpParams p = {};
  p.z = z; p.ld = ld; p.tokens = tokens; p.N = N; p.V = V; p.K = K;
  p.logprob = logprob; p.entropy = entropy; p.rank = rank; p.row_max = row_max;
  p.row_sumexp = row_sumexp; p.top_ids = top_ids; p.top_logprobs = top_logprobs; p.err = err;
  switch (dtype) {
    case DSPARK_F32: return launch_lp<float>(p, stream);
    case DSPARK_BF16: return launch_lp<__nv_bfloat16>(p, stream);
    default: return launch_lp<__half>(p, stream);
  }
}

cudaError_t launch_token_logprobs_grad(const void* z, int dtype, long long ld, const int32_t* tokens,
                                       int N, int V, const float* row_max, const float* row_sumexp,
                                       const float* entropy, const float* d_logprob,
                                       const float* d_entropy, void* dz, long long ld_dz, int* err,
                                       cudaStream_t stream) {
  LgParams p = {};
  p.z = z; p.ld = ld; p.tokens = tokens; p.V = V; p.row_max = row_max; p.row_sumexp = row_sumexp;
  p.entropy = entropy; p.d_logprob = d_logprob; p.d_entropy = d_entropy; p.dz = dz; p.ld_dz = ld_dz;
  p.err = err;
  switch (dtype) {
    case DSPARK_F32: return launch_lg<float>(p, N, stream);
    case DSPARK_BF16: return launch_lg<__nv_bfloat16>(p, N, stream);
    default: return launch_lg<__half>(p, N, stream);
  }
}

}  // namespace dspark
