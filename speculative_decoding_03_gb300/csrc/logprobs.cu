// Log probabilities of given tokens, entropy, rank and top alternatives of rows of logits,
// and the gradient of the first two.
//
// billytse.dev DSpark page, section 1: the target's distribution of a position is the
// softmax of its logits row.  With m = max_v z_v and s = sum_v exp(z_v - m):
//   logprob = z_y - m - log s,   entropy = log s - sum_v exp(z_v - m) (z_v - m) / s,
//   rank    = 1 + #{v : z_v > z_y, or z_v = z_y and v < y},
// and the K largest logits (ties to the smallest v) with their log probabilities.
//
// Bound by the one read of the row from HBM.  A row is cut into the CTAs of a cluster
// (1, 2, 4 or 8): a thread keeps its softmax sums and the maximum of everything it read in
// registers, and the maximum of each batch it read in shared memory; nothing is selected
// while streaming.  The K-th largest of the group maxima of 2 K or more groups of threads
// is a lower bound of the K-th largest logit that only slightly more than K elements reach
// (-G log(1 - K / G) of them for G groups of random data: 89 at K = 64, G = 128); the few
// batches whose maximum reaches it (or the token's logit, for the rank) are read again
// from L2.  Those candidates are ranked by counting, and the CTAs merge their K best
// through distributed shared memory.
#include "internal.h"
#include "rows.cuh"

namespace dspark {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpBatch = 4;                 // 16-byte chunks a thread loads at once
constexpr int kLpCap = 1024;                // candidate keys of a CTA
constexpr int kLpList = 512;                // slots listed to be read again
constexpr int kLpTop = kMaxTop;             // most alternatives
constexpr int kLpMaxSlots = 64;             // batch maxima kept per thread

struct LpParams {
  const void* z;
  long long ld;
  const int32_t* tokens;     // may be null: every row is used, no logprob and no rank
  int V, K, slots, per_slot; // per_slot batches share a slot of batch maxima
  float* logprob;
  float* entropy;
  int32_t* rank;
  float* row_max;
  float* row_sumexp;
  int32_t* top_ids;
  float* top_logprobs;
  int* err;
};

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

struct LpShared {
  unsigned long long cand[kLpCap];
  unsigned long long best[kLpTop];                    // this CTA's K best, descending
  unsigned long long all[8 * kLpTop];                 // every CTA's, for the merge
  float gmax[kLpThreads];
  float4 part[kLpThreads / 32];
  float4 stat;                                        // m, s, t, (int) elements before y
  int n_best, n_cand, n_list, before, merged[kLpTop];
  int list[kLpList];
  float thr;
};

// best[0 .. K) = the K largest of cand[0 .. n), descending; returns min(n, K).  All threads.
__device__ __forceinline__ int select_top(LpShared& sh, int n, int K) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const unsigned long long key = sh.cand[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += sh.cand[j] > key;
    if (r < K) sh.best[r] = key;
  }
  __syncthreads();
  return n < K ? n : K;
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 4) token_logprobs_kernel(LpParams a, int C) {
  constexpr int N = Chunk<T>::N;
  __shared__ LpShared sh;
  extern __shared__ float slot_max[];       // [slots][kLpThreads]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)(blockIdx.x / C);
  const int c = (int)(blockIdx.x - (unsigned)n * C);
  const int V = a.V, K = a.K;
  pdl_wait();
  pdl_launch_dependents();
  const int y = a.tokens ? a.tokens[n] : -1;
  if (a.tokens && (y < 0 || y >= V)) {      // the same in every CTA of the cluster
    if (c == 0) {
      if (tid == 0) {
        if (y != -1) set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
        a.logprob[n] = 0.f;
        a.rank[n] = 0;
        if (a.entropy) a.entropy[n] = 0.f;
        if (a.row_max) a.row_max[n] = -INFINITY;
        if (a.row_sumexp) a.row_sumexp[n] = 0.f;
      }
      for (int j = tid; j < K; j += kLpThreads) {
        a.top_ids[(size_t)n * K + j] = -1;
        a.top_logprobs[(size_t)n * K + j] = -INFINITY;
      }
    }
    return;
  }
  const T* row = static_cast<const T*>(a.z) + (long long)n * a.ld;
  const RowChunks rc = row_chunks(row, V);
  const uint4* body = reinterpret_cast<const uint4*>(row + rc.head);
  const int c0 = (int)((long long)rc.chunks * c / C), c1 = (int)((long long)rc.chunks * (c + 1) / C);
  const float zy = a.tokens ? elem_to_float(row[y]) : INFINITY;

  // ---- one pass: sums, this thread's maximum and its batch maxima
  RunningSoftmax rs;
  rs.init();
  float tmax = -INFINITY;
  // CTA 0 takes the elements outside the 16-byte chunks, one to a thread
  const int loose_n = c == 0 ? rc.head + rc.tail : 0;
  const int loose = tid < rc.head ? tid : V - rc.tail + (tid - rc.head);
  if (tid < loose_n) {
    const float z = elem_to_float(row[loose]);
    rs.add_one(z);
    tmax = fmaxf(tmax, z);
  }
  const int span = kLpThreads * kLpBatch;
  int at = c0 + tid, in_slot = 0;
  float* slot = slot_max + tid;
  float smax = -INFINITY;
  for (; at + (kLpBatch - 1) * kLpThreads < c1; at += span) {
    uint4 q[kLpBatch];
#pragma unroll
    for (int g = 0; g < kLpBatch; ++g) q[g] = __ldg(body + at + g * kLpThreads);
#pragma unroll
    for (int g = 0; g < kLpBatch; ++g) {
      float z[N];
      unpack_chunk<T>(q[g], z);
      const float bm = max_of(z);
      smax = fmaxf(smax, bm);
      rs.template add<N>(z, bm);
    }
    if (++in_slot == a.per_slot) {
      *slot = smax;
      slot += kLpThreads;
      tmax = fmaxf(tmax, smax);
      smax = -INFINITY;
      in_slot = 0;
    }
  }
  for (; at < c1; at += kLpThreads) {
    float z[N];
    unpack_chunk<T>(__ldg(body + at), z);
    const float bm = max_of(z);
    smax = fmaxf(smax, bm);
    rs.template add<N>(z, bm);
    in_slot = 1;
  }
  if (in_slot) {
    *slot = smax;
    slot += kLpThreads;
    tmax = fmaxf(tmax, smax);
  }
  const int used = (int)((slot - slot_max) / kLpThreads);

  // ---- the CTA's statistics
  float m = warp_max(tmax);
  if (lane == 0) sh.part[warp].x = m;
  if (tid == 0) {
    sh.n_cand = 0;
    sh.n_list = 0;
    sh.before = 0;
    sh.n_best = 0;
    sh.thr = -INFINITY;
  }
  __syncthreads();
  m = sh.part[0].x;
#pragma unroll
  for (int w = 1; w < kLpThreads / 32; ++w) m = fmaxf(m, sh.part[w].x);
  __syncthreads();
  float s, t;
  rs.finish(m, s, t);
  s = warp_sum(s);
  t = warp_sum(t);
  if (lane == 0) sh.part[warp] = make_float4(0.f, s, t, 0.f);
  // ---- a lower bound of the CTA's K-th largest element
  int G = 32;
  while (G < 2 * K && G < kLpThreads) G <<= 1;
  if (K > 0) {
    sh.gmax[tid] = tmax;
    __syncthreads();
    float g = -INFINITY;
    if (tid < G)
      for (int j = tid; j < kLpThreads; j += G) g = fmaxf(g, sh.gmax[j]);
    __syncthreads();
    if (tid < G) sh.gmax[tid] = g;
    __syncthreads();
    if (tid < G) {
      int r = 0;
      for (int j = 0; j < G; j += 4) {
        const float4 o = *reinterpret_cast<const float4*>(&sh.gmax[j]);
        r += (o.x > g || (o.x == g && j < tid)) + (o.y > g || (o.y == g && j + 1 < tid)) +
             (o.z > g || (o.z == g && j + 2 < tid)) + (o.w > g || (o.w == g && j + 3 < tid));
      }
      if (r == K - 1) sh.thr = g;
    }
  }
  __syncthreads();
  const float thr = K > 0 ? sh.thr : INFINITY;

  // ---- candidates for the K best and the elements before y: the batches that reach either
  const float reach = fminf(thr, zy);
  int before = 0;
  auto consider = [&](float z, int v) {
    if (z > zy || (z == zy && v < y)) ++before;
    if (K > 0 && z >= thr) {
      const int at = atomicAdd(&sh.n_cand, 1);
      if (at < kLpCap) sh.cand[at] = top_key(z, v);
    }
  };
  if (K > 0 || a.tokens) {
    if (tid < loose_n) consider(elem_to_float(row[loose]), loose);
    auto look = [&](int i) {
      float z[N];
      unpack_chunk<T>(__ldg(body + i), z);
      const float bm = max_of(z);
      if (bm >= reach) {
        const int v = rc.head + i * N;
#pragma unroll
        for (int e = 0; e < N; ++e) consider(z[e], v + e);
      }
    };
    // the slots that reach it, listed, then their chunks dealt over all threads
    for (int u = 0; u < used; ++u)
      if (slot_max[u * kLpThreads + tid] >= reach) {
        const int at = atomicAdd(&sh.n_list, 1);
        if (at < kLpList) sh.list[at] = u * kLpThreads + tid;
      }
    __syncthreads();
    const int per = a.per_slot * kLpBatch;
    if (sh.n_list <= kLpList) {
      const int tasks = sh.n_list * per;
      for (int k = tid; k < tasks; k += kLpThreads) {
        const int e = sh.list[k / per], g = k % per;
        const int i = c0 + (e & (kLpThreads - 1)) + ((e / kLpThreads) * per + g) * kLpThreads;
        if (i < c1) look(i);
      }
    } else {
      for (int u = 0; u < used; ++u) {
        if (slot_max[u * kLpThreads + tid] < reach) continue;
        const int from = c0 + tid + u * per * kLpThreads, to = min(c1, from + per * kLpThreads);
        for (int i = from; i < to; i += kLpThreads) look(i);
      }
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0 && before) atomicAdd(&sh.before, before);
  __syncthreads();
  if (K > 0) {
    int n_cand = sh.n_cand;
    if (n_cand > kLpCap) {
      // more elements at or above the bound than keys fit (equal logits, or all the large
      // ones in few threads' hands): the same selection tile by tile, keeping the K best
      int kept = 0;
      auto sweep = [&](int from, int to) {
        for (int base = from; base < to; base += kLpCap / 2) {
          __syncthreads();
          if (tid == 0) sh.n_cand = kept;
          for (int j = tid; j < kept; j += kLpThreads) sh.cand[j] = sh.best[j];
          const unsigned long long floor_key = kept == K ? sh.best[K - 1] : 0ull;
          __syncthreads();
          for (int v = base + tid; v < min(to, base + kLpCap / 2); v += kLpThreads) {
            const float z = elem_to_float(row[v]);
            const unsigned long long key = top_key(z, v);
            if (z == z && key > floor_key) sh.cand[atomicAdd(&sh.n_cand, 1)] = key;
          }
          __syncthreads();
          if (sh.n_cand > kept) kept = select_top(sh, sh.n_cand, K);
        }
      };
      if (c == 0) sweep(0, rc.head);
      sweep(rc.head + c0 * N, rc.head + c1 * N);
      if (c == 0) sweep(V - rc.tail, V);
      n_cand = -1;
      if (tid == 0) sh.n_best = kept;
    }
    if (n_cand >= 0) {
      const int got = select_top(sh, n_cand, K);
      if (tid == 0) sh.n_best = got;
    }
  }
  if (C > 1 && K > 0) {
    __syncthreads();
    for (int j = sh.n_best + tid; j < K; j += kLpThreads) sh.best[j] = 0ull;
  }
  if (tid == 0) {
    float S = 0.f, Tm = 0.f;
    for (int w = 0; w < kLpThreads / 32; ++w) {
      S += sh.part[w].y;
      Tm += sh.part[w].z;
    }
    sh.stat = make_float4(m, S, Tm, __int_as_float(sh.before));
  }
  __syncthreads();

  // ---- the cluster's statistics and its K best
  float M = m, S, Tm;
  int total_before = 0;
  if (C > 1) {
    cluster_sync();
    // lane o reads CTA o's statistics
    const float4 p = lane < C ? cluster_ld_f4(cluster_map(&sh.stat, lane))
                              : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    M = warp_max(p.x);
    const float d = p.x - M, f = p.y != 0.f ? ex2_approx(d * kLog2e) : 0.f;
    S = warp_sum(p.y != 0.f ? p.y * f : 0.f);
    Tm = warp_sum(f > 0.f ? f * (p.z + d * p.y) : 0.f);
    total_before = __reduce_add_sync(0xffffffffu, lane < C ? __float_as_int(p.w) : 0);
  } else {
    S = sh.stat.y;
    Tm = sh.stat.z;
    total_before = __float_as_int(sh.stat.w);
  }
  const bool bad = !(S <= FLT_MAX);         // NaN or +inf among the logits
  const float logs = logf(S);
  if (c == 0 && tid == 0) {
    const float nan = __int_as_float(0x7FC00000);
    if (a.tokens) {
      a.logprob[n] = bad ? nan : S > 0.f ? zy - M - logs : -INFINITY;
      a.rank[n] = bad ? 0 : total_before + 1;
    }
    if (a.entropy) a.entropy[n] = bad ? nan : S > 0.f ? logs - Tm / S : 0.f;
    if (a.row_max) a.row_max[n] = M;
    if (a.row_sumexp) a.row_sumexp[n] = bad ? nan : S;
  }
  if (K > 0) {
    auto put = [&](int r, unsigned long long key) {
      const size_t o = (size_t)n * K + r;
      const float nan = __int_as_float(0x7FC00000);
      a.top_ids[o] = bad ? -1 : key_index(key);
      a.top_logprobs[o] = bad ? nan : S > 0.f ? key_value(key) - M - logs : -INFINITY;
    };
    int total = sh.n_best;
    if (C > 1) {
      // every list to this CTA's shared memory (0 beyond a list's end)
      int got = 0;
      if (lane < C)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(got) : "r"(cluster_map(&sh.n_best, lane)) : "memory");
      total = __reduce_add_sync(0xffffffffu, got);
      for (int p = tid; p < C * K; p += kLpThreads) {
        const int o = p / K, j = p - o * K;
        // (best is 0 from a list's end on)
        sh.all[o * kLpTop + j] = cluster_ld_u64(cluster_map(&sh.best[0], o) + 8u * j);
      }
      for (int j = tid; j < K; j += kLpThreads) sh.merged[j] = 0;
      __syncthreads();
      const int mine = sh.n_best;
      for (int p = tid; p < mine * C; p += kLpThreads) {
        const int j = p / C, o = p - j * C;
        const unsigned long long key = sh.best[j];
        int lo = 0, hi = K;                 // keys of list o above this one
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (sh.all[o * kLpTop + mid] > key) lo = mid + 1;
          else hi = mid;
        }
        if (lo) atomicAdd(&sh.merged[j], lo);
      }
      __syncthreads();
      for (int j = tid; j < mine; j += kLpThreads)
        if (sh.merged[j] < K) put(sh.merged[j], sh.best[j]);
    } else {
      for (int j = tid; j < total; j += kLpThreads) put(j, sh.best[j]);
    }
    if (c == 0)
      for (int j = total + tid; j < K; j += kLpThreads) {
        a.top_ids[(size_t)n * K + j] = -1;
        a.top_logprobs[(size_t)n * K + j] = bad ? __int_as_float(0x7FC00000) : -INFINITY;
      }
  }
  if (C > 1) cluster_sync();                // no CTA leaves while another reads its lists
}

// ------------------------------------------------------------------------------ gradient
// dz_v = g_lp ([v = y] - p_v) - g_H p_v (log p_v + H), p_v = exp(z_v - m) / s: one read and
// one write of the row, nothing kept between them, so a grid of independent segments.
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

// CTAs a row is cut into: enough work items to fill the GPU several times over (4 CTAs an
// SM), but no segment below 2048 chunks (32 KB), under which a CTA's fixed work shows
int row_ctas(long long rows, long long chunks) {
  int C = 1;
  while (C < 8 && (rows * C < 4LL * kTargetCtas) && chunks / (2 * C) >= 2048) C *= 2;
  // few rows: the latency of a segment counts, down to one batch per thread
  while (C < 8 && rows * C < 152 && chunks / (2 * C) >= kLpThreads) C *= 2;
  return C;
}

template <typename T>
cudaError_t launch_lp(LpParams p, int N, cudaStream_t stream) {
  const int chunks = p.V / Chunk<T>::N;
  const int C = row_ctas(N, chunks);
  const int batches = cdiv(cdiv(chunks + 1, C), kLpThreads * kLpBatch) + 1;
  p.per_slot = cdiv(batches, kLpMaxSlots);
  p.slots = cdiv(batches, p.per_slot) + 1;
  const size_t smem = (size_t)p.slots * kLpThreads * sizeof(float);
  static std::atomic<int> cache[kMaxCachedDevices];
  const int ok = per_device_grid(cache, [] {
    return cudaFuncSetAttribute(token_logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (kLpMaxSlots + 2) * kLpThreads * (int)sizeof(float)) == cudaSuccess ? 1 : -1;
  });
  if (ok <= 0) return cudaErrorInvalidConfiguration;
  return launch_rows_cluster(token_logprobs_kernel<T>, (long long)N * C, C, kLpThreads, smem, stream, p, C);
}

template <typename T>
cudaError_t launch_lg(LgParams p, int N, cudaStream_t stream) {
  const int chunks = p.V / Chunk<T>::N;
  // segments of about 4096 chunks (64 KB), or as many as give every SM eight CTAs
  int segs = cdiv(chunks, 4096);
  while ((long long)segs * N < 2LL * kTargetCtas && chunks / (segs * 2) >= kLgThreads) segs *= 2;
  if (segs < 1) segs = 1;
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
  p.z = z; p.ld = ld; p.tokens = tokens; p.V = V; p.K = K;
  p.logprob = logprob; p.entropy = entropy; p.rank = rank; p.row_max = row_max;
  p.row_sumexp = row_sumexp; p.top_ids = top_ids; p.top_logprobs = top_logprobs; p.err = err;
  switch (dtype) {
    case DSPARK_F32: return launch_lp<float>(p, N, stream);
    case DSPARK_BF16: return launch_lp<__nv_bfloat16>(p, N, stream);
    default: return launch_lp<__half>(p, N, stream);
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
