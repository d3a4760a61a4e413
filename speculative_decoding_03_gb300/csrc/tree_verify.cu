// Verification of a tree (or chain) of drafted tokens against the target's probabilities, from
// given uniform numbers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "target.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct VerifyParams {
  const void *p, *q;
  long long ld_p, ld_q;
  int V, log_C;
  const int32_t* tokens;
  const float* uniforms;
  TargetRows rows;
  int32_t *accept_len, *path, *out_tokens, *n_out;
  int* err;
};

// A sum of non-negative fp32 numbers kept as hi + lo: Knuth's two-sum gives each addition's
// rounding exactly, so that sums over a row are good to 2^-45 of themselves.  (Sums in 64 bits
// would run at a sixty-fourth of the rate.)
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

// What is left of the row p after `rejected` children: r = p, then r = max(r - s q, 0) for
// each child drawn from q (s the sum before it, 1 at first), or r = 0 at their tokens.
struct Left {
  int rounds;                // of q
  const float* s;
  int points;                // rejected point masses
  const int* token;
  __device__ __forceinline__ float of(float p, float q) const {
    float r = p;
    for (int j = 0; j < rounds; ++j) r = fmaxf(__fmaf_rn(-s[j], q, r), 0.f);
    return r;
  }
  __device__ __forceinline__ bool struck(int v) const {
    bool hit = false;
    for (int j = 0; j < points; ++j) hit = hit || token[j] == v;
    return hit;
  }
};

// The part of a row that one warp of the request's cluster sums: 16-byte chunks c0 .. c1 - 1 of
// the row p, and the elements before the first chunk (the first warp) or behind the last.
template <typename T>
struct Part {
  const T *p, *q;            // q null: none
  RowChunks rc;
  bool q_fits;               // q's chunks start where p's do
  int c0, c1;
  int V;
  // the elements of chunk c (rc.head + c N ..): p into x, q into y
  __device__ __forceinline__ void load(int c, uint4& x, uint4& y, float (&yf)[Chunk<T>::N]) const {
    constexpr int N = Chunk<T>::N;
    x = *(reinterpret_cast<const uint4*>(p + rc.head) + c);
    if (!q) return;
    if (q_fits) {
      y = *(reinterpret_cast<const uint4*>(q + rc.head) + c);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) yf[e] = elem_to_float(q[rc.head + (long long)c * N + e]);
    }
  }
};

template <typename T>
__device__ __forceinline__ void left_of_chunk(const Part<T>& part, const Left& left, bool struck, int c,
                                              const uint4& x, const uint4& y, const float (&yf)[Chunk<T>::N],
                                              float (&r)[Chunk<T>::N]) {
  constexpr int N = Chunk<T>::N;
  unpack_chunk<T>(x, r);
  if (left.rounds) {
    float g[N];
    if (part.q_fits) unpack_chunk<T>(y, g);
#pragma unroll
    for (int e = 0; e < N; ++e) r[e] = left.of(r[e], part.q_fits ? g[e] : yf[e]);
  }
  if (struck) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (left.struck(part.rc.head + c * N + e)) r[e] = 0.f;
  }
}

template <typename T>
__device__ __forceinline__ float left_of_element(const Part<T>& part, const Left& left, int v) {
  if (left.struck(v)) return 0.f;
  const float p = elem_to_float(part.p[v]);
  return left.rounds ? left.of(p, elem_to_float(part.q[v])) : p;
}

__device__ __forceinline__ double warp_sum_f64(double x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}
// inclusive sums over the lanes
__device__ __forceinline__ double warp_scan_f64(double x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const double y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// One cluster of C CTAs a request.  Every CTA walks the tree by itself on the few elements that
// decide (the rows of p and q are read only at the tokens); sums over a whole row, which a
// second child drawn from q and the last draw need, are shared out over the cluster's warps in
// order of the vocabulary.  So a request reads its last node's rows of p and q once, which
// bounds a large batch; one request's time is its chain of dependent loads.
template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int N = Chunk<T>::N;
  __shared__ int par_s[kMaxTree], tok_s[kMaxTree];
  __shared__ float u_s[kMaxTree], p_s[kMaxTree], q_s[kMaxTree];
  __shared__ float round_s[kMaxTree];        // s before round j of q
  __shared__ int point_s[kMaxTree];          // rejected point masses of the current node
  __shared__ int path_s[kMaxTree];
  __shared__ double warp_sum_s[2][kWarps];   // by pass, read by the cluster
  __shared__ double all_s[kMaxCluster * kWarps + 1];
  __shared__ double scan_s[kWarps];
  __shared__ int state_s[6];
  __shared__ double left_s;
  __shared__ int pick_s;
  pdl_wait();
  pdl_launch_dependents();
  const int C = 1 << p.log_C, rank = blockIdx.x & (C - 1), b = blockIdx.x >> p.log_C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RequestRows rr = request_rows(p.rows, b, p.err);
  const int n = rr.n;
  const T* P = static_cast<const T*>(p.p);
  const T* Q = static_cast<const T*>(p.q);
  for (int i = tid; i < n; i += kThreads) {
    const int row = rr.row0 + i;
    const int up = i ? parent_of(p.rows.parents, row, i, p.err) : -1;
    int x = i ? p.tokens[row] : 0;
    if (x < 0 || x >= p.V) {
      set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
      x = -1;
    }
    par_s[i] = up;
    tok_s[i] = x;
    u_s[i] = p.uniforms[row];
    if (up >= 0 && x >= 0) {
      p_s[i] = elem_to_float(P[(rr.row0 + up) * p.ld_p + x]);
      q_s[i] = Q ? elem_to_float(Q[(rr.row0 + up) * p.ld_q + x]) : 1.f;
    }
  }
  if (tid == 0) {
    state_s[0] = 0;        // the current node
    state_s[1] = 1;        // the next node to look at
    state_s[2] = 0;        // accepted
    state_s[3] = 0;        // rounds of q (with the sum of the last still unknown)
    state_s[4] = 0;        // rejected point masses
    left_s = 1.0;          // s
  }
  __syncthreads();

  int pass = 0;
  for (;;) {
    // ---- the walk, until a sum over the row is needed (state_s[5]: 1) or it ends (2)
    if (tid == 0) {
      int at = state_s[0], i = state_s[1], accepted = state_s[2], rounds = state_s[3], points = state_s[4];
      double s = left_s;
      int why = n > 0 ? 2 : 3;
      for (; i < n; ++i) {
        if (par_s[i] != at) continue;
        const int x = tok_s[i];
        if (x < 0) continue;                       // (reported above; never accepted)
        if (rounds > 0 && s < 0.0) {               // not known yet
          why = 1;
          break;
        }
        float r = p_s[i];
        bool yes;
        if (Q) {
          for (int j = 0; j < rounds; ++j) r = fmaxf(__fmaf_rn(-round_s[j], q_s[i], r), 0.f);
          yes = (double)u_s[i] * (double)q_s[i] * s < (double)r;
        } else {
          for (int j = 0; j < points; ++j)
            if (point_s[j] == x) r = 0.f;
          yes = (double)u_s[i] * s < (double)r;
        }
        if (yes) {
          path_s[accepted++] = i;
          at = i;
          rounds = points = 0;
          s = 1.0;
        } else if (Q) {
          round_s[rounds++] = (float)s;
          s = -1.0;
        } else {
          s -= (double)r;
          point_s[points++] = x;
        }
      }
      state_s[0] = at;
      state_s[1] = i;
      state_s[2] = accepted;
      state_s[3] = rounds;
      state_s[4] = points;
      state_s[5] = why;
      left_s = s;
    }
    __syncthreads();
    const int why = state_s[5];
    if (why == 3) break;
    Left left = {state_s[3], round_s, state_s[4], point_s};
    const int row = rr.row0 + state_s[0];

    double total = 0.0;
    Part<T> part;
    bool struck = false;
    for (int attempt = 0; attempt < 2; ++attempt) {
      // ---- the warp's part of the row
      const int W = C * kWarps, w = rank * kWarps + warp;
      part.p = P + row * p.ld_p;
      part.q = left.rounds ? Q + row * p.ld_q : nullptr;
      part.V = p.V;
      part.rc = row_chunks(part.p, p.V);
      part.q_fits = part.q && ((reinterpret_cast<uintptr_t>(part.p) ^ reinterpret_cast<uintptr_t>(part.q)) & 15u) == 0;
      part.c0 = (int)((long long)part.rc.chunks * w / W);
      part.c1 = (int)((long long)part.rc.chunks * (w + 1) / W);
      struck = false;
      for (int j = 0; j < left.points; ++j) {
        const int c = (left.token[j] - part.rc.head) / N;
        struck = struck || (left.token[j] >= part.rc.head && c >= part.c0 && c < part.c1);
      }
      Sum2 sum = {0.f, 0.f};
      constexpr int kBatch = 4;
      for (int c = part.c0 + lane; c < part.c1; c += 32 * kBatch) {
        uint4 x[kBatch], y[kBatch];
        float yf[kBatch][N];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (c + 32 * u < part.c1) part.load(c + 32 * u, x[u], y[u], yf[u]);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (c + 32 * u >= part.c1) break;
          float r[N];
          left_of_chunk(part, left, struck, c + 32 * u, x[u], y[u], yf[u], r);
#pragma unroll
          for (int e = 0; e < N; ++e) sum.add(r[e]);
        }
      }
      if (w == 0 && lane < part.rc.head) sum.add(left_of_element(part, left, lane));
      if (w == W - 1 && lane < part.rc.tail) sum.add(left_of_element(part, left, p.V - part.rc.tail + lane));
      const double mine = warp_sum_f64(sum.value());
      // ---- the cluster's sums.  Two buffers: a CTA writes one again only after the others
      // have read it, since the barrier of the pass between lies behind those reads.
      if (lane == 0) warp_sum_s[pass & 1][warp] = mine;
      if (C > 1) cluster_sync();
      else __syncthreads();
      if (tid < W)
        all_s[tid] = C > 1 ? __longlong_as_double((long long)cluster_ld_u64(
                                 cluster_map(&warp_sum_s[pass & 1][tid & (kWarps - 1)], (uint32_t)(tid / kWarps))))
                           : warp_sum_s[pass & 1][tid];
      ++pass;
      __syncthreads();
      if (warp == 0) {
        // exclusive sums, in the vocabulary's order
        double carry = 0.0;
        for (int t0 = 0; t0 < W; t0 += 32) {
          const double x = t0 + lane < W ? all_s[t0 + lane] : 0.0;
          const double in = warp_scan_f64(x), before = __shfl_up_sync(0xffffffffu, in, 1);
          if (t0 + lane < W) all_s[t0 + lane] = carry + (lane ? before : 0.0);
          carry += __shfl_sync(0xffffffffu, in, 31);
        }
        if (lane == 0) all_s[W] = carry;
      }
      __syncthreads();
      total = all_s[W];
      if (why == 1 || total > 0.0 || (!left.rounds && !left.points)) break;
      left.rounds = left.points = 0;         // nothing is left: from the target's own row
    }
    if (why == 1) {
      if (tid == 0) left_s = (double)(float)total;     // s is held in 32 bits
      __syncthreads();
      continue;
    }

    // ---- the last draw: the first v whose sum up to it exceeds u total
    const int W = C * kWarps;
    const bool valid = total > 0.0 && total < INFINITY;
    const double t = (double)u_s[0] * total;
    int target = W - 1;                      // the warp part that holds it
    if (tid == 0) pick_s = -1;
    if (valid) {
      // (the last part that is not empty and starts at or before t)
      int best = 0;
      for (int w0 = lane; w0 < W; w0 += 32)
        if (all_s[w0] <= t && all_s[w0 + 1] > all_s[w0]) best = max(best, w0);
      target = __reduce_max_sync(0xffffffffu, best);
    }
    __syncthreads();
    if (valid && target / kWarps == rank) {
      // this CTA's threads share the part's chunks out again, in order
      const int w = target;
      const int c0 = (int)((long long)part.rc.chunks * w / W), c1 = (int)((long long)part.rc.chunks * (w + 1) / W);
      const int head = w == 0 ? part.rc.head : 0, tail = w == W - 1 ? part.rc.tail : 0;
      const int each = (c1 - c0 + kThreads - 1) / kThreads;
      // thread's elements v0 .. v1 - 1
      const int a0 = min(c0 + tid * each, c1), a1 = min(c0 + (tid + 1) * each, c1);
      const int v0 = tid == 0 ? part.rc.head + c0 * N - head : part.rc.head + a0 * N;
      const int v1 = part.rc.head + a1 * N + (tid == kThreads - 1 ? tail : 0);
      Sum2 sum = {0.f, 0.f};
      for (int v = v0; v < v1; ++v) sum.add(left_of_element(part, left, v));
      const double mine = sum.value(), in = warp_scan_f64(mine);
      if (lane == 31) scan_s[warp] = in;
      __syncthreads();
      double before = all_s[w];
      for (int k = 0; k < warp; ++k) before += scan_s[k];
      const double up_to = before + in;
      // the first thread that goes beyond t; by rounding there may be none, then the last
      // thread that has anything
      const unsigned beyond = __ballot_sync(0xffffffffu, mine > 0.0 && up_to > t);
      const unsigned any = __ballot_sync(0xffffffffu, mine > 0.0);
      int key = INT_MAX;
      if (beyond) key = warp * 32 + __ffs(beyond) - 1;
      else if (any) key = (1 << 20) - (warp * 32 + 31 - __clz(any));   // (the last is the least of these)
      __shared__ int key_s;
      if (tid == 0) key_s = INT_MAX;
      __syncthreads();
      if (lane == 0) atomicMin(&key_s, key);
      __syncthreads();
      const int k = key_s, who = k > (1 << 19) && k != INT_MAX ? (1 << 20) - k : k;
      if (tid == who) {
        double acc = before + (in - mine);
        int pick = -1;
        for (int v = v0; v < v1; ++v) {
          const float r = left_of_element(part, left, v);
          if (!(r > 0.f)) continue;
          pick = v;
          acc += (double)r;
          if (acc > t) break;
        }
        pick_s = pick;
      }
      __syncthreads();
    }
    // ---- results: the CTA that drew, or the first where nothing can be drawn
    const bool writer = valid ? target / kWarps == rank : rank == 0;
    if (writer) {
      const int accepted = state_s[2];
      if (tid == 0 && pick_s < 0) set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
      for (int j = tid; j < p.rows.N; j += kThreads) {
        const long long at = (long long)b * p.rows.N + j;
        p.path[at] = j < accepted ? path_s[j] : -1;
        p.out_tokens[at] = j < accepted ? tok_s[path_s[j]] : j == accepted ? pick_s : -1;
      }
      if (tid == 0) {
        p.accept_len[b] = accepted;
        p.n_out[b] = accepted + 1;
      }
    }
    break;
  }
  if (n == 0 && rank == 0) {                 // no tokens: no answer
    for (int j = tid; j < p.rows.N; j += kThreads) {
      p.path[(long long)b * p.rows.N + j] = -1;
      p.out_tokens[(long long)b * p.rows.N + j] = -1;
    }
    if (tid == 0) {
      p.accept_len[b] = 0;
      p.n_out[b] = 0;
    }
  }
  if (C > 1) cluster_sync();                 // nobody leaves while its sums may still be read
}

template <typename T>
cudaError_t verify_for(VerifyParams p, cudaStream_t stream) {
  // CTAs a request: as many as keep the device busy, while every warp has a few chunks
  const int chunks = cdiv(p.V, Chunk<T>::N);
  p.log_C = 0;
  while (p.log_C < 3 && (p.rows.B << p.log_C) < 608 && chunks >= (kThreads << (p.log_C + 1))) ++p.log_C;
  return launch_rows_cluster(verify_kernel<T>, (long long)p.rows.B << p.log_C, 1 << p.log_C, kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_tree_verify(const void* p, const void* q, int dtype, long long ld_p, long long ld_q, int V,
                               const int32_t* tokens, const float* uniforms, const TargetRows& rows,
                               int32_t* accept_len, int32_t* path, int32_t* out_tokens, int32_t* n_out, int* err,
                               cudaStream_t stream) {
  const VerifyParams a = {p, q, ld_p, ld_q, V, 0, tokens, uniforms, rows, accept_len, path, out_tokens, n_out, err};
  switch (dtype) {
    case DSPARK_F32: return verify_for<float>(a, stream);
    case DSPARK_BF16: return verify_for<__nv_bfloat16>(a, stream);
    default: return verify_for<__half>(a, stream);
  }
}

}  // namespace dspark
