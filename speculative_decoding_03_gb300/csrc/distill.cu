// Distillation of the student's logits from a teacher's top logits: loss, expected
// acceptance, and the gradient with respect to the student's logits.
//
// xhh.club DSpark page (acceptance rule: min(p, q) summed over the vocabulary is the
// probability that a drafted token is accepted) and weigao.cc DSpark-vs-MTP page, "loss"
// (cross entropy, total variation, position weights): with p the softmax of the teacher's
// K logits t / tau, q the softmax of the student's row z / tau, and label y,
//   loss = w (c_kl sum_k p_k (log p_k - log q_k) + c_tv sum_k max(0, p_k - q_k)
//             + c_ce (-log q_y)),        accept = sum_k min(p_k, q_k).
// (p sums to 1 over the K entries, so sum max(0, p - q) is the total variation distance, and
// accept is the acceptance by a target cut to them.)
// Every term's gradient is A q_v - a_v with a_k = c_kl p_k + c_tv q_k [q_k < p_k] (and c_ce
// at the label), A = sum of all a:
//   dz_v = g w / tau (A q_v - sum_{k : id_k = v} a_k).
//
// Bound by one read and one write of the row.  A cluster of CTAs holds a whole row in
// shared memory, so the gradient needs no second read of it: sums, one exchange of the
// warps' sums between the cluster's CTAs, gradient from the same shared memory.  Clusters
// are persistent, and nothing in a row waits for a whole CTA: a producer warp refills each
// 16 KB piece of the row's part with the next row's bytes as soon as the eight consumer
// warps have left it, a teacher warp prepares the next row's entries (ids, softmax, the
// student's logits at them), and a warp sends its sums to every CTA of the cluster with
// stores that complete on that CTA's barrier.  An element that the teacher names is written
// a second time by the warp that wrote it first.  Rows beyond a cluster's shared memory read
// their rest again.
//
// Measured on a GB300 (copy rate 6782 GB/s): 1280 rows of 129280 in fp32, 1216 of them with a
// weight, 206 us = 6.26 TB/s (0.92 of the copy rate); 1920 rows of 151936 in bf16, 1824 with a
// weight, 199 us = 5.73 TB/s (0.85).  What is left is the consumers' own work: a build without
// stores, without loads or without the exchange took as long.  8 consumer warps and 16 KB
// pieces: 16 warps 345 against 266 us, 8 KB 213 against 206, 32 KB 232; one CTA an SM with twice
// the ring 447 against 266.
#include "internal.h"
#include "rows.cuh"
#include "sm100_ptx.cuh"

namespace dspark {
namespace {

using namespace sm100;

constexpr int kDsWarps = 8;                         // consumer warps
constexpr int kDsThreads = kDsWarps * 32;           // consumer threads
constexpr int kDsBlock = kDsThreads + 64;           // and the producer's and the teacher's warp
constexpr int kDsPiece = 16 * 1024;                 // bytes of a bulk copy
constexpr int kPieceChunks = kDsPiece / 16;
constexpr int kRing = 6;                            // pieces of a CTA: 96 KB, two CTAs an SM
constexpr int kDsTarget = 80 * 1024;                // most of them one row's, the rest the next's
constexpr int kShare = kPieceChunks / kDsThreads;   // chunks of a piece for a consumer thread
constexpr int kSumsLane = 8 * kDsWarps / 32;        // warps' sums a lane reads
constexpr int kPer = kMaxTop / 32;                  // entries of a lane

struct DsParams {
  const void* z;
  long long ld;
  const int32_t* ids;        // [N][K]
  const float* t;            // [N][K]
  const int32_t* labels;     // [N] or null
  const float* weights;      // [N] or null
  const float* d_loss;       // [N] or null
  int N, V, K;
  int resident;              // 16-byte chunks of a row's part kept in shared memory
  float inv_tau, c_kl, c_tv, c_ce;
  float* loss;
  float* accept;
  void* dz;
  long long ld_dz;
  int* err;
};

struct Teacher {
  int id[kMaxTop];           // -1: no entry, or none with weight
  float p[kMaxTop], log_p[kMaxTop], z[kMaxTop];
  int own[kMaxTop];          // entries of this CTA's part of the row
  float sum_p, zy;
  int y, any, n_own, twice, y_own;   // twice: an id of theirs occurs more than once;
                                     // y_own: y is in this part and not among the ids
};

struct DsShared {
  float2 sums[2][8 * kDsWarps];          // (reference, sum) of every consumer warp of the cluster
  Teacher teacher[2];
  uint64_t full[kRing], empty[kRing], sums_full[2], teacher_full[2], teacher_free[2];
};

// The teacher's entries of row n and its label into `te`, by one warp.
template <typename T>
__device__ __forceinline__ void read_teacher(const DsParams& a, int n, const RowPart<T>& r, bool first_part,
                                             Teacher& te) {
  const int lane = threadIdx.x & 31, K = a.K, V = a.V;
  const T* row = r.row;
  int id[kPer];
  float t[kPer], p[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = lane + 32 * i;
    id[i] = k < K ? a.ids[(size_t)n * K + k] : -1;
    t[i] = k < K ? a.t[(size_t)n * K + k] : -INFINITY;
  }
  int y = a.labels ? a.labels[n] : -1;
  if (y < -1 || y >= V) {
    if (lane == 0) set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
    y = -1;
  }
  float tm = -INFINITY;
  bool nan = false;                          // (the maximum passes over NaN)
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (id[i] < -1 || id[i] >= V) {
      set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
      id[i] = -1;
    }
    if (id[i] < 0) t[i] = -INFINITY;
    nan |= t[i] != t[i];
    tm = fmaxf(tm, t[i]);
  }
  const float zy = y >= 0 ? elem_to_float(row[y]) : 0.f;
  float z[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) z[i] = id[i] >= 0 ? elem_to_float(row[id[i]]) : 0.f;
  tm = warp_max(tm);
  // NaN or +inf among the entries: every p is NaN, and the row shows it
  const bool any = tm > -INFINITY || __any_sync(0xffffffffu, nan);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (!any) id[i] = -1;                    // entries without weight are like any element
    // over the temperature only now: t / tau itself may be beyond fp32, or lose the difference
    t[i] = (t[i] - tm) * a.inv_tau;
    p[i] = id[i] >= 0 ? expf(t[i]) : 0.f;
    sum += p[i];
  }
  sum = warp_sum(sum);
  const float log_sum = logf(sum);
  auto owned = [&](int v) {
    if (v < r.rc.head || v >= V - r.rc.tail) return v >= 0 && first_part;
    const int at = (v - r.rc.head) / Chunk<T>::N;
    return at >= r.c0 && at < r.c1;
  };
  float sum_p = 0.f;
  bool y_named = false;
  int n_own = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = lane + 32 * i;
    if (32 * i >= K) break;
    if (id[i] >= 0) p[i] /= sum;
    sum_p += p[i];
    y_named |= id[i] >= 0 && id[i] == y;
    if (k < K) {
      te.id[k] = id[i];
      te.p[k] = p[i];
      te.log_p[k] = t[i] - log_sum;
      te.z[k] = z[i];
    }
    const bool mine = owned(id[i]);
    const unsigned all = __ballot_sync(0xffffffffu, mine);
    if (mine) te.own[n_own + __popc(all & ((1u << lane) - 1u))] = k;
    n_own += __popc(all);
  }
  sum_p = warp_sum(sum_p);
  y_named = __any_sync(0xffffffffu, y_named);
  __syncwarp();
  bool twice = false;
  if (n_own <= 32) {
    const int v = lane < n_own ? te.id[te.own[lane]] : -1 - lane;
    twice = __popc(__match_any_sync(0xffffffffu, v)) > 1;
  } else {
    for (int j = 0; j < n_own; ++j) {
      const int o = te.id[te.own[j]];
      for (int i = lane; i < j; i += 32) twice |= te.id[te.own[i]] == o;
    }
  }
  twice = __any_sync(0xffffffffu, twice);
  if (lane == 0) {
    te.sum_p = sum_p;
    te.zy = zy;
    te.y = y;
    te.any = any;
    te.n_own = n_own;
    te.twice = twice;
    te.y_own = !y_named && owned(y);
  }
  __syncwarp();
}

// What follows a row's sums: q = exp((z - M) / tau) / S.
struct RowEnd {
  const DsParams& a;
  const Teacher& te;
  int n;
  float w, M, S, logs, kl2;
  float sum_a, gw, scale;    // A; g w / tau; A g w / (tau S), 0 for a row of zeroes
  __device__ __forceinline__ RowEnd(const DsParams& a_, const Teacher& te_, int n_, float w_, float M_, float S_)
      : a(a_), te(te_), n(n_), w(w_), M(M_), S(S_), logs(logf(S_)), kl2(a_.inv_tau * kLog2e) {}
  __device__ __forceinline__ float log_q(float z) const { return (z - M) * a.inv_tau - logs; }
  // a_k of an entry; products with a zero coefficient are left out (0 * inf)
  __device__ __forceinline__ float coef(float p, float q) const {
    float x = a.c_kl != 0.f ? a.c_kl * p : 0.f;
    if (q < p) x += a.c_tv * q;
    return x;
  }
  __device__ __forceinline__ float ay() const { return te.y >= 0 ? a.c_ce : 0.f; }
  __device__ __forceinline__ bool on() const { return te.any || te.y >= 0; }
  // the gradient's factors, by a whole warp
  __device__ __forceinline__ void factors(float g) {
    const int lane = threadIdx.x & 31;
    sum_a = (te.any && a.c_kl != 0.f ? a.c_kl * te.sum_p : 0.f) + ay();
    if (a.c_tv != 0.f && te.any) {
      float tv = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        if (k < a.K && te.id[k] >= 0) {
          const float q = expf(log_q(te.z[k]));
          tv += q < te.p[k] ? q : 0.f * te.p[k];   // (a NaN stays one)
        }
      }
      sum_a += a.c_tv * warp_sum(tv);
    }
    gw = g * w * a.inv_tau;
    // (a row with NaN or +inf shows it, whatever its coefficients)
    scale = on() && (sum_a * gw != 0.f || !(S <= FLT_MAX)) ? sum_a * gw / S : 0.f;
  }
  // the gradient of a chunk, without the entries' own terms
  template <typename T>
  __device__ __forceinline__ uint4 grad(const uint4& q) const {
    constexpr int N = Chunk<T>::N;
    const F2 nM = f2(-M, -M), kk = f2(kl2, kl2), sc = f2(scale, scale);
    float z[N];
    unpack_chunk<T>(q, z);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float x, y;
      f2_get(f2_mul(f2_add(f2(z[i], z[i + 1]), nM), kk), x, y);
      f2_get(f2_mul(f2(ex2_approx(x), ex2_approx(y)), sc), z[i], z[i + 1]);
    }
    return pack_chunk<T>(z);
  }
  __device__ __forceinline__ float grad_one(float z) const { return ex2_approx((z - M) * kl2) * scale; }
  // The entries' own elements and the label's, A q - sum of a over the entries with this id,
  // for those that `mine` gives to this warp; after the row's chunks.
  template <typename T, typename Mine>
  __device__ __forceinline__ void write_entries(T* out, Mine&& mine) const {
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < te.n_own; i += 32) {
      const int k = te.own[i], v = te.id[k];
      if (!mine(v)) continue;
      const float q = expf(log_q(te.z[k]));
      float av = v == te.y ? ay() : 0.f;
      if (te.twice) {                        // in entry order, so that equal ids write the same
        for (int j = 0; j < a.K; ++j)
          if (te.id[j] == v) av += coef(te.p[j], q);
      } else {
        av += coef(te.p[k], q);
      }
      out[v] = elem_from_float<T>(gw * (sum_a * q - av));
    }
    if (lane == 0 && te.y_own && mine(te.y))
      out[te.y] = elem_from_float<T>(gw * (sum_a * expf(log_q(te.zy)) - ay()));
  }
  // loss and acceptance, by a whole warp
  __device__ __forceinline__ void write_loss() const {
    const int lane = threadIdx.x & 31;
    float kl = 0.f, tv = 0.f, acc = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int k = lane + 32 * i;
      if (k < a.K && te.id[k] >= 0) {
        const float lq = log_q(te.z[k]), q = expf(lq), p = te.p[k];
        if (p != 0.f) kl += p * (te.log_p[k] - lq);
        const float d = p - q;
        tv += d > 0.f ? d : 0.f * d;         // (a NaN stays one)
        acc += (d > 0.f ? q : p) + 0.f * d;
      }
    }
    kl = warp_sum(kl);
    tv = warp_sum(tv);
    acc = warp_sum(acc);
    if (lane == 0) {
      float l = 0.f;
      if (te.any && a.c_kl != 0.f) l += a.c_kl * kl;
      if (te.any && a.c_tv != 0.f) l += a.c_tv * tv;
      if (te.y >= 0 && a.c_ce != 0.f) l -= a.c_ce * log_q(te.zy);
      a.loss[n] = on() ? l * w : 0.f;
      a.accept[n] = te.any ? acc : 0.f;
    }
  }
};

// zeroes of part c of 2^log_C of an output row, by `threads` threads
template <typename T>
__device__ __forceinline__ void zero_row(T* out, int V, int c, int log_C, int t, int threads) {
  const RowChunks oc = row_chunks(out, V);
  uint4* o4 = reinterpret_cast<uint4*>(out + oc.head);
  const int e0 = (int)((long long)oc.chunks * c >> log_C), e1 = (int)((long long)oc.chunks * (c + 1) >> log_C);
  for (int i = e0 + t; i < e1; i += threads) __stcs(o4 + i, make_uint4(0u, 0u, 0u, 0u));
  if (c == 0 && t < oc.head + oc.tail)
    out[t < oc.head ? t : V - oc.tail + (t - oc.head)] = elem_from_float<T>(0.f);
}

// Short rows: a CTA of four warps a row, the sums and the gradient from two reads (the second
// finds the row in L1 or L2).  Many small CTAs an SM hide a row's steps behind other rows:
// 2000 rows of 4000 in fp32 18 us, 26 by the ring; of 8000 31 and 32.
constexpr int kShortThreads = 128;
constexpr int kShortChunks = 2048;          // 32 KB
template <typename T, bool Grad>
__global__ void __launch_bounds__(kShortThreads, 8) distill_short_kernel(DsParams a) {
  constexpr int N = Chunk<T>::N;
  __shared__ Teacher te;
  __shared__ float2 sums_s[kShortThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = blockIdx.x, V = a.V;
  pdl_wait();
  pdl_launch_dependents();
  T* out = Grad ? static_cast<T*>(a.dz) + (long long)n * a.ld_dz : nullptr;
  const float w = a.weights ? a.weights[n] : 1.f;
  if (w == 0.f) {                            // a masked row: nothing of it is read
    if constexpr (Grad) zero_row(out, V, 0, 0, tid, kShortThreads);
    if (tid == 0) {
      a.loss[n] = 0.f;
      a.accept[n] = 0.f;
    }
    return;
  }
  const RowPart<T> r = row_part<T>(a.z, a.ld, n, V, 0, 0, 0x7FFFFFFF);
  if (warp == 0) read_teacher<T>(a, n, r, true, te);
  RunningSum rs;
  rs.init(a.inv_tau);
  const int loose_n = r.rc.head + r.rc.tail;
  const int loose = tid < r.rc.head ? tid : V - r.rc.tail + (tid - r.rc.head);
  const float zl = tid < loose_n ? elem_to_float(r.row[loose]) : -INFINITY;
  constexpr int G = 16 / N;                  // chunks of 16 elements
  int j = tid;
  for (; j + (G - 1) * kShortThreads < r.held; j += G * kShortThreads) {
    uint4 q[G];
#pragma unroll
    for (int u = 0; u < G; ++u) q[u] = r.body[j + u * kShortThreads];
    float z[16];
#pragma unroll
    for (int u = 0; u < G; ++u) {
      float x[N];
      unpack_chunk<T>(q[u], x);
#pragma unroll
      for (int e = 0; e < N; ++e) z[u * N + e] = x[e];
    }
    rs.add(z);
  }
  for (; j < r.held; j += kShortThreads) {
    float z[N];
    unpack_chunk<T>(r.body[j], z);
    rs.add(z);
  }
  if (tid < loose_n) rs.add_one(zl);
  const float wm = warp_max(rs.reference());
  const float ws = warp_sum(rs.at(wm));
  if (lane == 0) sums_s[warp] = make_float2(wm, ws);
  __syncthreads();                           // also: the teacher's entries are read
  float M = -INFINITY, S = 0.f;
#pragma unroll
  for (int i = 0; i < kShortThreads / 32; ++i) M = fmaxf(M, sums_s[i].x);
#pragma unroll
  for (int i = 0; i < kShortThreads / 32; ++i)
    if (sums_s[i].y != 0.f) S += sums_s[i].y * ex2_approx((sums_s[i].x - M) * (a.inv_tau * kLog2e));
  RowEnd end(a, te, n, w, M, S);
  if constexpr (Grad) {
    end.factors(a.d_loss ? a.d_loss[n] : 1.f);
    if (end.scale == 0.f) {
      zero_row(out, V, 0, 0, tid, kShortThreads);
    } else {
      const bool same = ((reinterpret_cast<uintptr_t>(r.row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
      T* o = out + r.rc.head;
#pragma unroll 4
      for (int i = tid; i < r.held; i += kShortThreads) {
        const uint4 v = end.grad<T>(r.body[i]);
        if (same) {
          __stcs(reinterpret_cast<uint4*>(o) + i, v);
        } else {                             // output rows off the input rows' 16-byte grid
          const T* ve = reinterpret_cast<const T*>(&v);
#pragma unroll
          for (int e = 0; e < N; ++e) o[(long long)i * N + e] = ve[e];
        }
      }
      if (tid < loose_n) out[loose] = elem_from_float<T>(end.grad_one(zl));
      __syncthreads();                       // the entries' elements after the row's
      if (warp == 0) end.write_entries(out, [](int) { return true; });
    }
  }
  if (warp == kShortThreads / 32 - 1) end.write_loss();
}

template <typename T, bool Grad>
__global__ void __launch_bounds__(kDsBlock, 2) distill_kernel(DsParams a, int log_C) {
  constexpr int N = Chunk<T>::N;
  extern __shared__ __align__(128) uint4 rows_s[];
  __shared__ DsShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = 1 << log_C;                  // CTAs of a row
  const int c = (int)(blockIdx.x & (C - 1)), first = (int)(blockIdx.x >> log_C), step = (int)(gridDim.x >> log_C);
  const int V = a.V;
  const int pieces = (a.resident + kPieceChunks - 1) / kPieceChunks;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kDsWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sums_full[i], 1);
      mbar_init(&sh.teacher_full[i], 1);
      mbar_init(&sh.teacher_free[i], kDsWarps);
    }
    fence_mbar_init();
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  bool late = false;                         // a bounded wait ran out: give up

  if (warp == kDsWarps) {
    // ---- producer: a row's part piece by piece, each as soon as its last reader is gone
    if (lane == 0) {
      int sent = 0;                          // pieces so far; slot sent % kRing
      for (int n = first; n < a.N && !late; n += step) {
        if (a.weights && a.weights[n] == 0.f) continue;
        const RowPart<T> r = row_part<T>(a.z, a.ld, n, a.V, c, log_C, a.resident);
        for (int i = 0; i < pieces; ++i, ++sent) {
          const int slot = sent % kRing, use = sent / kRing;
          if (use > 0 && !mbar_wait(&sh.empty[slot], (use - 1) & 1)) { late = true; break; }
          const int k = max(0, min(kPieceChunks, r.held - i * kPieceChunks));
          mbar_arrive_expect_tx(&sh.full[slot], (uint32_t)k * 16u);
          if (k > 0)
            bulk_load(rows_s + slot * kPieceChunks, r.body + r.c0 + i * kPieceChunks, (uint32_t)k * 16u,
                      &sh.full[slot]);
        }
      }
      // copies in flight end before the CTA does (at once, unless the consumers gave up)
      for (int j = max(0, sent - kRing); j < sent; ++j) mbar_wait(&sh.full[j % kRing], (j / kRing) & 1);
    }
  } else if (warp == kDsWarps + 1) {
    // ---- teacher: the entries of the next rows
    int it = 0;
    for (int n = first; n < a.N && !late; n += step) {
      if (a.weights && a.weights[n] == 0.f) continue;
      const int b = it & 1;
      late = it >= 2 && !mbar_wait(&sh.teacher_free[b], ((it >> 1) - 1) & 1);
      late = __any_sync(0xffffffffu, late);
      if (late) break;
      read_teacher<T>(a, n, row_part<T>(a.z, a.ld, n, a.V, c, log_C, a.resident), c == 0, sh.teacher[b]);
      if (lane == 0) mbar_arrive(&sh.teacher_full[b]);
      ++it;
    }
  } else {
    int it = 0;
    int slot0 = 0;                           // the row's first piece
    uint32_t phase0 = 0;
    float w_next = first < a.N && a.weights ? a.weights[first] : 1.f;
    for (int n = first; n < a.N; n += step) {
      const float w = w_next;
      if (n + step < a.N && a.weights) w_next = a.weights[n + step];
      T* out = Grad ? static_cast<T*>(a.dz) + (long long)n * a.ld_dz : nullptr;
      auto zero_out = [&] {
        if constexpr (Grad) zero_row(out, V, c, log_C, tid, kDsThreads);
      };
      if (w == 0.f) {                        // a masked row: nothing of it is read
        zero_out();
        if (c == 0 && tid == 0) {
          a.loss[n] = 0.f;
          a.accept[n] = 0.f;
        }
        continue;
      }
      const int b = it & 1;
      const uint32_t buf_phase = (it >> 1) & 1;
      if (tid == 0) mbar_arrive_expect_tx(&sh.sums_full[b], (uint32_t)(C * kDsWarps * 8));
      const RowPart<T> r = row_part<T>(a.z, a.ld, n, a.V, c, log_C, a.resident);
      const float g = a.d_loss ? a.d_loss[n] : 1.f;

      // ---- sums
      RunningSum rs;
      rs.init(a.inv_tau);
      const int loose_n = c == 0 ? r.rc.head + r.rc.tail : 0;
      const int loose = tid < r.rc.head ? tid : V - r.rc.tail + (tid - r.rc.head);
      float zl = 0.f;
      if (tid < loose_n) {
        zl = elem_to_float(r.row[loose]);
        rs.add_one(zl);
      }
      // G chunks at once
      auto take = [&](const auto& q) {
        constexpr int G = sizeof(q) / sizeof(q[0]);
        float z[G * N];
#pragma unroll
        for (int u = 0; u < G; ++u) {
          float x[N];
          unpack_chunk<T>(q[u], x);
#pragma unroll
          for (int e = 0; e < N; ++e) z[u * N + e] = x[e];
        }
        rs.add(z);
      };
      auto take_one = [&](const uint4& q) {
        const uint4 one[1] = {q};
        take(one);
      };
      int slot = slot0;
      uint32_t phase = phase0;
      auto next_piece = [&] {
        if (++slot == kRing) {
          slot = 0;
          phase ^= 1;
        }
      };
      for (int i = 0; i < pieces; ++i, next_piece()) {
        if (!late && !mbar_wait(&sh.full[slot], phase)) late = true;
        const uint4* piece = rows_s + slot * kPieceChunks + tid;
        const int left = r.held - i * kPieceChunks;
        if (left >= kPieceChunks) {
          uint4 q[kShare];
#pragma unroll
          for (int u = 0; u < kShare; ++u) q[u] = piece[u * kDsThreads];
          take(q);
        } else {
          for (int j = 0; j + tid < left; j += kDsThreads) take_one(piece[j]);
        }
        if constexpr (!Grad) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.empty[slot]);
        }
      }
      for (int j = r.c0 + r.held + tid; j < r.c1; j += kDsThreads) take_one(r.body[j]);
      const float wm = warp_max(rs.reference());
      const float s = warp_sum(rs.at(wm));
      // the teacher's entries are read (from the row, too) before any CTA can write it
      Teacher& te = sh.teacher[b];
      if (!late && !mbar_wait(&sh.teacher_full[b], buf_phase)) late = true;
      if (lane < C) send_f2(&sh.sums[b][c * kDsWarps + warp], &sh.sums_full[b], lane, wm, s);
      if (!late && !wait_cluster(&sh.sums_full[b], buf_phase)) late = true;
      late = __any_sync(0xffffffffu, late);
      if (late) break;
      float2 part[kSumsLane];
      float M = -INFINITY, S = 0.f;
#pragma unroll
      for (int i = 0; i < kSumsLane; ++i) {
        part[i] = lane + 32 * i < C * kDsWarps ? sh.sums[b][lane + 32 * i] : make_float2(-INFINITY, 0.f);
        M = fmaxf(M, part[i].x);
      }
      M = warp_max(M);
      const float kl2 = a.inv_tau * kLog2e;
#pragma unroll
      for (int i = 0; i < kSumsLane; ++i)
        if (part[i].y != 0.f) S += part[i].y * ex2_approx((part[i].x - M) * kl2);
      S = warp_sum(S);
      RowEnd end(a, te, n, w, M, S);

      if constexpr (Grad) {
        end.factors(g);
        if (end.scale == 0.f) {
          zero_out();
          __syncwarp();
          slot = slot0;
          for (int i = 0; i < pieces; ++i, next_piece())
            if (lane == 0) mbar_arrive(&sh.empty[slot]);
        } else {
          const bool same = ((reinterpret_cast<uintptr_t>(r.row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
          T* o = out + r.rc.head;
          auto put = [&](int j, const uint4& q) {
            const uint4 v = end.grad<T>(q);
            if (same) {
              __stcs(reinterpret_cast<uint4*>(o) + j, v);
            } else {                         // output rows off the input rows' 16-byte grid
              const T* ve = reinterpret_cast<const T*>(&v);
#pragma unroll
              for (int e = 0; e < N; ++e) o[(long long)j * N + e] = ve[e];
            }
          };
          slot = slot0;
          for (int i = 0; i < pieces; ++i, next_piece()) {
            const uint4* piece = rows_s + slot * kPieceChunks + tid;
            const int left = r.held - i * kPieceChunks, at = r.c0 + i * kPieceChunks + tid;
            if (left >= kPieceChunks) {
              uint4 q[kShare];
#pragma unroll
              for (int u = 0; u < kShare; ++u) q[u] = piece[u * kDsThreads];
#pragma unroll
              for (int u = 0; u < kShare; ++u) put(at + u * kDsThreads, q[u]);
            } else {
              for (int j = 0; j + tid < left; j += kDsThreads) put(at + j, piece[j]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[slot]);
          }
          for (int j = r.c0 + r.held + tid; j < r.c1; j += kDsThreads) put(j, r.body[j]);
          if (tid < loose_n) out[loose] = elem_from_float<T>(end.grad_one(zl));
          // the entries' elements after the row's, by the warp that wrote them first (those
          // outside the chunks: warp 0)
          __syncwarp();
          end.write_entries(out, [&](int v) {
            const int at = (v - r.rc.head) / N - r.c0;
            return (v < r.rc.head || v >= V - r.rc.tail ? 0 : (at & (kDsThreads - 1)) >> 5) == warp;
          });
        }
      }
      if (warp == kDsWarps - 1 && (it & (C - 1)) == c) end.write_loss();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.teacher_free[b]);
      slot0 += pieces;
      if (slot0 >= kRing) {
        slot0 -= kRing;
        phase0 ^= 1;
      }
      ++it;
    }
  }
  if (late) set_device_error(a.err, DSPARK_ERR_TIMEOUT);
  __syncwarp();
  if (C > 1) cluster_sync();                 // no CTA leaves while another may still send to it
}

template <typename T, bool Grad>
cudaError_t launch(DsParams p, cudaStream_t stream) {
  const int chunks = p.V / Chunk<T>::N;
  if (chunks <= kShortChunks)
    return launch_pdl(distill_short_kernel<T, Grad>, dim3((unsigned)p.N), dim3(kShortThreads), 0, stream, p);
  int C = 1, log_C = 0;
  // the row's part of a CTA small enough that some of the ring is left for the next row's;
  // more CTAs a row while there are fewer than two an SM, as long as each has 8 KB
  while (C < 8 && (long long)cdiv(chunks, C) * 16 > kDsTarget) C *= 2, ++log_C;
  while (C < 8 && (long long)p.N * C < 304 && chunks / (2 * C) >= 512) C *= 2, ++log_C;
  const int part = cdiv(chunks, C) + 1;
  p.resident = part < kRing * kPieceChunks ? part : kRing * kPieceChunks;
  const size_t smem = (size_t)kRing * kDsPiece;
  // clusters that the device holds at once: more would wait for these to end
  static std::atomic<int> cache[4][kMaxCachedDevices];
  const int most = device_clusters(cache[log_C], distill_kernel<T, Grad>, C,
                                   kDsBlock, smem);
  if (most <= 0) return cudaErrorInvalidConfiguration;
  const long long clusters = p.N < most ? p.N : most;
  return launch_rows_cluster(distill_kernel<T, Grad>, clusters * C, C, kDsBlock, smem, stream, p, log_C);
}

}  // namespace

cudaError_t launch_distill(const void* z, int dtype, long long ld, const int32_t* ids, const float* t,
                           const int32_t* labels, const float* weights, const float* d_loss, int N,
                           int V, int K, float inv_tau, float c_kl, float c_tv, float c_ce, float* loss,
                           float* accept, void* dz, long long ld_dz, int* err, cudaStream_t stream) {
  DsParams p = {};
  p.z = z; p.ld = ld; p.ids = ids; p.t = t; p.labels = labels; p.weights = weights; p.d_loss = d_loss;
  p.N = N; p.V = V; p.K = K; p.inv_tau = inv_tau; p.c_kl = c_kl; p.c_tv = c_tv; p.c_ce = c_ce;
  p.loss = loss; p.accept = accept; p.dz = dz; p.ld_dz = ld_dz; p.err = err;
  switch (dtype) {
    case DSPARK_F32: return dz ? launch<float, true>(p, stream) : launch<float, false>(p, stream);
    case DSPARK_BF16:
      return dz ? launch<__nv_bfloat16, true>(p, stream) : launch<__nv_bfloat16, false>(p, stream);
    default: return dz ? launch<__half, true>(p, stream) : launch<__half, false>(p, stream);
  }
}

}  // namespace dspark
