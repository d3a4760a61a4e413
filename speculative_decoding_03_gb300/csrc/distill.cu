// Distillation of the student's logits from a teacher's top logits: loss, expected
// acceptance, and the gradient with respect to the student's logits.
//
// xhh.club DSpark page (acceptance rule: min(p, q) summed over the vocabulary is the
// probability that a drafted token is accepted) and weigao.cc DSpark-vs-MTP page, "loss"
// (cross entropy, total variation, position weights): with p the softmax of the teacher's
// K logits t / tau, q the softmax of the student's row z / tau, and label y,
//   loss = w (c_kl sum_k p_k (log p_k - log q_k) + c_tv sum_k max(0, p_k - q_k)
//             + c_ce (-log q_y)),        accept = sum_k min(p_k, q_k).
// (p sums to 1 over the K entries, so sum max(0, p - q) is the total variation distance.)
// Every term's gradient is A q_v - a_v with a_k = c_kl p_k + c_tv q_k [q_k < p_k] (and c_ce
// at the label), A = sum of all a:
//   dz_v = g w / tau (A q_v - sum_{k : id_k = v} a_k).
//
// Bound by one read and one write of the row.  A cluster of CTAs holds a whole row in
// shared memory (bulk copies, a few pieces deep so that the sums start on the first), so
// the gradient needs no second read: sums, one exchange through distributed shared memory,
// gradient from the same shared memory.  Several CTAs an SM overlap one row's reads with
// another's writes.  Rows beyond a cluster's shared memory read their rest again.
#include "internal.h"
#include "rows.cuh"
#include "sm100_ptx.cuh"

namespace dspark {
namespace {

using namespace sm100;

constexpr int kDsThreads = 256;
constexpr int kDsPiece = 16 * 1024;                 // bytes of a bulk copy
constexpr int kDsMaxPieces = 13;
constexpr int kDsMost = kDsMaxPieces * kDsPiece;    // resident bytes of a CTA (208 KB)
constexpr int kDsTarget = 72 * 1024;                // three CTAs an SM

struct DsParams {
  const void* z;
  long long ld;
  const int32_t* ids;        // [N][K]
  const float* t;            // [N][K]
  const int32_t* labels;     // [N] or null
  const float* weights;      // [N] or null
  const float* d_loss;       // [N] or null
  int V, K;
  int resident;              // 16-byte chunks of a CTA kept in shared memory
  float inv_tau, c_kl, c_tv, c_ce;
  float* loss;
  float* accept;
  void* dz;
  long long ld_dz;
  int* err;
};

struct DsShared {
  float4 part[kDsThreads / 32];
  float4 stat;
  int id[kMaxTop + 4];
  float a[kMaxTop + 4];
  float q[kMaxTop + 4];
  float scale;               // A g w / (tau s)
  float sum_a, gw;
  uint64_t bar[kDsMaxPieces];
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

template <typename T, bool Grad>
__global__ void __launch_bounds__(kDsThreads, 4) distill_kernel(DsParams a, int C) {
  constexpr int N = Chunk<T>::N;
  extern __shared__ __align__(128) uint4 rows_s[];
  __shared__ DsShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)(blockIdx.x / C);
  const int c = (int)(blockIdx.x - (unsigned)n * C);
  const int V = a.V, K = a.K;
  const T* row = static_cast<const T*>(a.z) + (long long)n * a.ld;
  T* out = Grad ? static_cast<T*>(a.dz) + (long long)n * a.ld_dz : nullptr;
  pdl_wait();
  pdl_launch_dependents();

  auto zero_out = [&] {
    if constexpr (Grad) {
      const RowChunks oc = row_chunks(out, V);
      uint4* o4 = reinterpret_cast<uint4*>(out + oc.head);
      const int e0 = (int)((long long)oc.chunks * c / C), e1 = (int)((long long)oc.chunks * (c + 1) / C);
      for (int i = e0 + tid; i < e1; i += kDsThreads) __stcs(o4 + i, make_uint4(0u, 0u, 0u, 0u));
      if (c == 0 && tid < oc.head + oc.tail)
        out[tid < oc.head ? tid : V - oc.tail + (tid - oc.head)] = elem_from_float<T>(0.f);
    }
  };
  const float w = a.weights ? a.weights[n] : 1.f;
  if (w == 0.f) {                            // a masked row: nothing of it is read
    zero_out();
    if (c == 0 && tid == 0) {
      a.loss[n] = 0.f;
      a.accept[n] = 0.f;
    }
    return;
  }

  const RowChunks rc = row_chunks(row, V);
  const uint4* body = reinterpret_cast<const uint4*>(row + rc.head);
  const int c0 = (int)((long long)rc.chunks * c / C), c1 = (int)((long long)rc.chunks * (c + 1) / C);
  const int held = min(c1 - c0, a.resident);
  constexpr int kPieceChunks = kDsPiece / 16;
  const int pieces = (held + kPieceChunks - 1) / kPieceChunks;
  if (tid == 0) {
    for (int i = 0; i < pieces; ++i) mbar_init(&sh.bar[i], 1);
    fence_mbar_init();
    for (int i = 0; i < pieces; ++i) {
      const int k = min(kPieceChunks, held - i * kPieceChunks);
      mbar_arrive_expect_tx(&sh.bar[i], (uint32_t)k * 16u);
      bulk_load(rows_s + i * kPieceChunks, body + c0 + i * kPieceChunks, (uint32_t)k * 16u, &sh.bar[i]);
    }
  }
  __syncthreads();

  // ---- the teacher's entries (warp 0, up to 4 a lane) and the label, read before any CTA
  // can write the gradient over the row
  constexpr int kPer = kMaxTop / 32;
  int id[kPer], y = -1;
  float tt[kPer], pk[kPer], zk[kPer], zy = 0.f;
  bool any = false;
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int k = lane + 32 * i;
      id[i] = k < K ? a.ids[(size_t)n * K + k] : -1;
      if (id[i] < -1 || id[i] >= V) {
        set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
        id[i] = -1;
      }
      tt[i] = id[i] >= 0 ? a.t[(size_t)n * K + k] * a.inv_tau : -INFINITY;
      zk[i] = id[i] >= 0 ? elem_to_float(row[id[i]]) : 0.f;
    }
    if (a.labels) {
      y = a.labels[n];
      if (y < -1 || y >= V) {
        if (lane == 0) set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
        y = -1;
      }
      if (y >= 0) zy = elem_to_float(row[y]);
    }
    // the teacher's softmax, while the row arrives: tt becomes log p
    float tm = -INFINITY, ps = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) tm = fmaxf(tm, tt[i]);
    tm = warp_max(tm);
    any = tm > -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      pk[i] = id[i] >= 0 && any ? expf(tt[i] - tm) : 0.f;
      ps += pk[i];
    }
    ps = warp_sum(ps);
    const float log_ps = logf(ps);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      pk[i] = any ? pk[i] / ps : 0.f;
      tt[i] = tt[i] - tm - log_ps;
    }
  }

  // ---- sums
  RunningSoftmax<false> rs;
  rs.init(a.inv_tau);
  float tmax = -INFINITY;
  const int loose_n = c == 0 ? rc.head + rc.tail : 0;
  const int loose = tid < rc.head ? tid : V - rc.tail + (tid - rc.head);
  float zl = 0.f;
  if (tid < loose_n) {
    zl = elem_to_float(row[loose]);
    rs.add_one(zl);
    tmax = fmaxf(tmax, zl);
  }
  auto take = [&](const uint4& q) {
    float z[N];
    unpack_chunk<T>(q, z);
    float bm = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) bm = fmaxf(bm, z[i]);
    tmax = fmaxf(tmax, bm);
    rs.template add<N>(z, bm);
  };
  bool late = false;
  for (int i = 0; i < pieces; ++i) {
    if (!late && !mbar_wait(&sh.bar[i], 0)) late = true;
    const int end = min(held, (i + 1) * kPieceChunks);
    for (int j = i * kPieceChunks + tid; j < end; j += kDsThreads) take(rows_s[j]);
  }
  for (int j = c0 + held + tid; j < c1; j += kDsThreads) take(body[j]);
  float m = warp_max(tmax);
  if (lane == 0) sh.part[warp].x = m;
  __syncthreads();
  m = sh.part[0].x;
#pragma unroll
  for (int i = 1; i < kDsThreads / 32; ++i) m = fmaxf(m, sh.part[i].x);
  float s, unused;
  rs.finish(m, s, unused);
  if (late) {                                // a copy that never arrived: the row becomes NaN
    set_device_error(a.err, DSPARK_ERR_TIMEOUT);
    s = __int_as_float(0x7FC00000);
  }
  s = warp_sum(s);
  if (lane == 0) sh.part[warp].y = s;
  __syncthreads();
  if (tid == 0) {
    float S = 0.f;
    for (int i = 0; i < kDsThreads / 32; ++i) S += sh.part[i].y;
    sh.stat = make_float4(m, S, 0.f, 0.f);
  }
  __syncthreads();
  float M = m, S;
  if (C > 1) {
    cluster_sync();                          // also: every CTA has read its teacher entries
    // lane o reads CTA o's sums
    const float4 p = lane < C ? cluster_ld_f4(cluster_map(&sh.stat, lane))
                              : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    M = warp_max(p.x);
    S = warp_sum(p.y != 0.f ? p.y * ex2_approx((p.x - M) * (a.inv_tau * kLog2e)) : 0.f);
  } else {
    S = sh.stat.y;
  }

  // ---- loss, acceptance and the entries' coefficients
  if (warp == 0) {
    const float logs = logf(S);
    float kl = 0.f, tv = 0.f, acc = 0.f, sum_a = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float ak = 0.f, q = 0.f;
      if (id[i] >= 0) {
        const float lq = (zk[i] - M) * a.inv_tau - logs;
        q = expf(lq);
        if (any) {
          const float p = pk[i];
          if (p != 0.f) kl += p * (tt[i] - lq);
          tv += fmaxf(p - q, 0.f);
          acc += fminf(p, q);
          // products with a zero coefficient are left out: 0 * inf
          if (a.c_kl != 0.f) ak = a.c_kl * p;
          if (q < p) ak += a.c_tv * q;
        }
      }
      sum_a += ak;
      const int k = lane + 32 * i;
      if (k < K) {
        sh.id[k] = any ? id[i] : -1;         // entries without weight are like any element
        sh.a[k] = ak;
        sh.q[k] = q;
      }
    }
    kl = warp_sum(kl);
    tv = warp_sum(tv);
    acc = warp_sum(acc);
    sum_a = warp_sum(sum_a);
    if (lane == 0) {
      const float lqy = (zy - M) * a.inv_tau - logs;
      const float ay = y >= 0 ? a.c_ce : 0.f;
      sh.id[K] = y;
      sh.a[K] = ay;
      sh.q[K] = y >= 0 ? expf(lqy) : 0.f;
      const bool on = any || y >= 0;
      const float g = a.d_loss ? a.d_loss[n] : 1.f;
      sum_a += ay;
      sh.sum_a = sum_a;
      sh.gw = g * w * a.inv_tau;
      sh.scale = on && sum_a * sh.gw != 0.f ? sum_a * sh.gw / S : 0.f;
      if (c == 0) {
        float l = 0.f;
        if (any && a.c_kl != 0.f) l += a.c_kl * kl;
        if (any && a.c_tv != 0.f) l += a.c_tv * tv;
        if (y >= 0 && a.c_ce != 0.f) l -= a.c_ce * lqy;
        a.loss[n] = on ? l * w : 0.f;
        a.accept[n] = any ? acc : 0.f;
      }
    }
  }
  if constexpr (Grad) {
    __syncthreads();
    const float scale = sh.scale;
    // the entries' own elements: sum over equal ids in entry order (the same in every
    // thread that holds one of them, so that two writes of an element agree)
    int fix_at = -1;
    float fix = 0.f;
    if (tid <= K) {
      const int v = sh.id[tid];
      if (v >= 0) {
        float av = 0.f;
        for (int j = 0; j <= K; ++j)
          if (sh.id[j] == v) av += sh.a[j];
        fix_at = v;
        fix = sh.gw * (sh.sum_a * sh.q[tid] - av);
      }
    }
    if (scale == 0.f) {
      zero_out();
    } else {
      const F2 nM = f2(-M, -M), kk = f2(a.inv_tau * kLog2e, a.inv_tau * kLog2e), sc = f2(scale, scale);
      auto grad = [&](const uint4& q) {
        float z[N];
        unpack_chunk<T>(q, z);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          float x, yv;
          f2_get(f2_mul(f2_add(f2(z[i], z[i + 1]), nM), kk), x, yv);
          f2_get(f2_mul(f2(ex2_approx(x), ex2_approx(yv)), sc), z[i], z[i + 1]);
        }
        return pack_chunk<T>(z);
      };
      const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
      if (same) {
        uint4* o4 = reinterpret_cast<uint4*>(out + rc.head);
        for (int j = tid; j < held; j += kDsThreads) __stcs(o4 + c0 + j, grad(rows_s[j]));
        for (int j = c0 + held + tid; j < c1; j += kDsThreads) __stcs(o4 + j, grad(body[j]));
      } else {                               // output rows off the input rows' 16-byte grid
        T* o = out + rc.head;
        for (int j = c0 + tid; j < c1; j += kDsThreads) {
          const uint4 g = grad(j < c0 + held ? rows_s[j - c0] : body[j]);
          const T* ge = reinterpret_cast<const T*>(&g);
#pragma unroll
          for (int e = 0; e < N; ++e) o[(long long)j * N + e] = ge[e];
        }
      }
      if (tid < loose_n)
        out[loose] = elem_from_float<T>(ex2_approx((zl - M) * (a.inv_tau * kLog2e)) * scale);
    }
    if (scale != 0.f) {
      __syncthreads();                       // the entries' elements after the row's
      const bool loose_at = fix_at >= 0 && (fix_at < rc.head || fix_at >= V - rc.tail);
      const int at = fix_at >= 0 && !loose_at ? (fix_at - rc.head) / N : -1;
      // an element of another CTA's part is that CTA's to write
      if (fix_at >= 0 && (loose_at ? c == 0 : at >= c0 && at < c1)) out[fix_at] = elem_from_float<T>(fix);
    }
  }
  if (C > 1) cluster_sync();                 // no CTA leaves while another reads its sums
}

template <typename T, bool Grad>
cudaError_t launch(DsParams p, int N, cudaStream_t stream) {
  const int chunks = p.V / Chunk<T>::N;
  int C = 1;
  // the row's part of a CTA small enough for three CTAs an SM; more CTAs a row while there
  // are fewer than two an SM, as long as each has 8 KB
  while (C < 8 && (long long)cdiv(chunks, C) * 16 > kDsTarget) C *= 2;
  while (C < 8 && (long long)N * C < 304 && chunks / (2 * C) >= 512) C *= 2;
  const int part = cdiv(chunks, C) + 1;
  p.resident = part * 16LL <= kDsMost ? part : kDsMost / 16;
  const size_t smem = (size_t)p.resident * 16;
  static std::atomic<int> cache[kMaxCachedDevices];
  const int ok = per_device_grid(cache, [] {
    return cudaFuncSetAttribute(distill_kernel<T, Grad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kDsMost) == cudaSuccess ? 1 : -1;
  });
  if (ok <= 0) return cudaErrorInvalidConfiguration;
  return launch_rows_cluster(distill_kernel<T, Grad>, (long long)N * C, C, kDsThreads, smem, stream, p, C);
}

}  // namespace

cudaError_t launch_distill(const void* z, int dtype, long long ld, const int32_t* ids, const float* t,
                           const int32_t* labels, const float* weights, const float* d_loss, int N,
                           int V, int K, float inv_tau, float c_kl, float c_tv, float c_ce, float* loss,
                           float* accept, void* dz, long long ld_dz, int* err, cudaStream_t stream) {
  DsParams p = {};
  p.z = z; p.ld = ld; p.ids = ids; p.t = t; p.labels = labels; p.weights = weights; p.d_loss = d_loss;
  p.V = V; p.K = K; p.inv_tau = inv_tau; p.c_kl = c_kl; p.c_tv = c_tv; p.c_ce = c_ce;
  p.loss = loss; p.accept = accept; p.dz = dz; p.ld_dz = ld_dz; p.err = err;
  switch (dtype) {
    case DSPARK_F32: return dz ? launch<float, true>(p, N, stream) : launch<float, false>(p, N, stream);
    case DSPARK_BF16:
      return dz ? launch<__nv_bfloat16, true>(p, N, stream) : launch<__nv_bfloat16, false>(p, N, stream);
    default: return dz ? launch<__half, true>(p, N, stream) : launch<__half, false>(p, N, stream);
  }
}

}  // namespace dspark
