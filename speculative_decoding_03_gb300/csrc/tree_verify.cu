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

constexpr int kThreads = 512, kWarps = kThreads / 32;
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

// Numbers kept as hi + lo, hi the nearest fp32 to both: Knuth's two-sum gives an addition's
// rounding exactly and a fused multiply-add a product's, so that sums over a row are good to
// 2^-45 of themselves.  (64-bit arithmetic runs at a sixty-fourth of the rate here, and an
// addition takes some hundred cycles: walk, scans and draw in it took 12 of 20 us.)
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {       // hi + lo not renormalised
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
  }
  __device__ __forceinline__ Sum2 normal() const {     // |hi| >= |lo|
    const float s = hi + lo;
    return {s, lo - (s - hi)};
  }
  // (both renormalised)
  __device__ __forceinline__ bool beyond(const Sum2& o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
};
__device__ __forceinline__ Sum2 operator+(const Sum2& a, const Sum2& b) {      // not renormalised
  Sum2 r = a;
  r.add(b.hi);
  r.lo += b.lo;
  return r;
}
__device__ __forceinline__ Sum2 operator*(const Sum2& a, const Sum2& b) {
  const float p = a.hi * b.hi;
  const Sum2 r = {p, fmaf(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi)};
  return r.normal();
}
__device__ __forceinline__ Sum2 shfl_up(const Sum2& a, int m) {
  return {__shfl_up_sync(0xffffffffu, a.hi, m), __shfl_up_sync(0xffffffffu, a.lo, m)};
}
__device__ __forceinline__ Sum2 warp_sum(Sum2 x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
    x = x + Sum2{__shfl_xor_sync(0xffffffffu, x.hi, m), __shfl_xor_sync(0xffffffffu, x.lo, m)};
  return x;
}
// inclusive sums over the lanes
__device__ __forceinline__ Sum2 warp_scan(Sum2 x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const Sum2 y = shfl_up(x, m);
    if (lane >= m) x = y + x;
  }
  return x;
}

// max(x, 0), NaN where x is (fmaxf would make it 0, and the row's sum would not show it)
__device__ __forceinline__ float above_zero(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// What is left of the row p after `rejected` children: r = p, then r = max(r - s q, 0) for
// each child drawn from q (s the sum before it, 1 at first), or r = 0 at their tokens.
struct Left {
  int rounds;                // of q
  const float* s;            // before round j > 0
  int points;                // rejected point masses
  const int* token;
  template <int N>
  __device__ __forceinline__ void of(float (&r)[N], const float (&q)[N]) const {
#pragma unroll
    for (int e = 0; e < N; ++e) r[e] = above_zero(r[e] - q[e]);       // s is 1 before the first
    for (int j = 1; j < rounds; ++j) {
      const float minus = -s[j];
#pragma unroll
      for (int e = 0; e < N; ++e) r[e] = above_zero(__fmaf_rn(minus, q[e], r[e]));
    }
  }
  __device__ __forceinline__ bool struck(int v) const {
    bool hit = false;
    for (int j = 0; j < points; ++j) hit = hit || token[j] == v;
    return hit;
  }
};

// A node's rows: whole 16-byte chunks of p, and the elements before the first and behind the
// last.  q's chunks are loaded whole where they start where p's do.
template <typename T>
struct NodeRow {
  static constexpr int N = Chunk<T>::N;
  const T *p, *q;            // q null: not needed
  RowChunks rc;
  bool q_fits;
  int V;
  __device__ __forceinline__ NodeRow(const T* p_, const T* q_, int V_) : p(p_), q(q_), V(V_) {
    rc = row_chunks(p, V);
    q_fits = q && ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) == 0;
  }
  // chunk c as loaded; mode 0: p alone, 1: and q's chunk, 2: and q's elements
  struct Raw {
    uint4 x, y;
  };
  template <int M>
  __device__ __forceinline__ Raw load(int c) const {
    Raw w;
    w.x = __ldcs(reinterpret_cast<const uint4*>(p + rc.head) + c);
    if constexpr (M == 1) w.y = __ldcs(reinterpret_cast<const uint4*>(q + rc.head) + c);
    if constexpr (M == 2) {
      T one[N];
#pragma unroll
      for (int e = 0; e < N; ++e) one[e] = q[rc.head + (long long)c * N + e];
      w.y = *reinterpret_cast<const uint4*>(one);
    }
    return w;
  }
  // what is left of a loaded chunk; `near`: a struck token may lie in it
  template <int M>
  __device__ __forceinline__ void left_of(const Raw& w, const Left& left, bool near, int c, float (&r)[N]) const {
    unpack_chunk<T>(w.x, r);
    if constexpr (M > 0) {
      float g[N];
      unpack_chunk<T>(w.y, g);
      left.of(r, g);
    }
    if (M == 0 && near) {
      const int v0 = rc.head + c * N;
      for (int j = 0; j < left.points; ++j) {
        const int at = left.token[j] - v0;
#pragma unroll
        for (int e = 0; e < N; ++e) r[e] = at == e ? 0.f : r[e];
      }
    }
  }
  __device__ __forceinline__ Raw load_any(int c) const { return !q ? load<0>(c) : q_fits ? load<1>(c) : load<2>(c); }
  __device__ __forceinline__ void left_of_any(const Raw& w, const Left& left, int c, float (&r)[N]) const {
    if (q) left_of<1>(w, left, false, c, r);
    else left_of<0>(w, left, true, c, r);
  }
  __device__ __forceinline__ float element(const Left& left, int v) const {
    if (left.struck(v)) return 0.f;
    float r[1] = {elem_to_float(p[v])};
    if (left.rounds) {
      const float g[1] = {elem_to_float(q[v])};
      left.of(r, g);
    }
    return r[0];
  }
};

template <int M>
struct Int {
  static constexpr int value = M;
};

struct Node {                // a token of the walk, and the target's probability of it
  int up, tok;
  float u, p;
};

// u q s < r in effect exactly: q and r times 2^64, so that products of tiny numbers keep their
// low parts
__device__ __forceinline__ bool accepts(float u, float q, const Sum2& s, float r) {
  constexpr float kUp = 0x1p64f;
  const float a = q * kUp, b = u * a;
  const Sum2 x = Sum2{b, fmaf(u, a, -b)} * s;
  return (x.hi - r * kUp) + x.lo < 0.f;
}
struct Walk {                // where the walk stands: its node, the next one to look at
  int at, next, accepted, rounds, points, row0;
};

// One cluster of C CTAs a request.  The first warp of every CTA walks the tree on the few
// elements that decide (the rows of p and q are read only at the tokens), a lane two nodes; sums
// over a whole row, which a second child drawn from q and the last draw need, are shared out
// over the cluster's warps in order of the vocabulary.  So a request reads its last node's rows
// of p and q once, which bounds a large batch; one request's time is its chain of dependent
// loads: the tokens, the elements at them, the row, and the part of it that holds the draw.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int N = Chunk<T>::N;
  constexpr int kParts = kMaxCluster * kWarps, kLaneParts = kParts / 32;
  using Row = NodeRow<T>;
  __shared__ float round_s[kMaxTree];        // s before round j of q
  __shared__ int point_s[kMaxTree];          // rejected point masses of the current node
  __shared__ int path_s[kMaxTree], taken_s[kMaxTree];
  __shared__ float2 sums_s[2][kParts];       // the cluster's warps' sums, by pass
  __shared__ __align__(8) uint64_t sums_bar[2];
  __shared__ Sum2 before_s[kParts + 1];      // the sums before each part, and of all
  __shared__ Sum2 scan_s[kWarps];
  __shared__ int state_s[5];                 // row, accepted, rounds, points, why the walk stopped
  __shared__ Node node_s[kMaxTree];
  __shared__ float q_s[kMaxTree];
  __shared__ Walk walk_s;
  __shared__ float draw_s, ends_s[32];
  __shared__ int pick_s, key_s, part_s[2];
  const int C = 1 << p.log_C, W = C * kWarps, rank = blockIdx.x & (C - 1), b = blockIdx.x >> p.log_C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    sm100::mbar_init(&sums_bar[0], 1);
    sm100::mbar_init(&sums_bar[1], 1);
    sm100::fence_mbar_init();
    sm100::mbar_arrive_expect_tx(&sums_bar[0], (uint32_t)(W * sizeof(float2)));
    sm100::mbar_arrive_expect_tx(&sums_bar[1], (uint32_t)(W * sizeof(float2)));
  }
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();
  const T* P = static_cast<const T*>(p.p);
  const T* Q = static_cast<const T*>(p.q);

  // ---- the walk's nodes: two a lane of the first warp, which alone reads them again
  if (warp == 0) {
    const RequestRows rr = request_rows(p.rows, b, p.err);
    float u[2] = {0.f, 0.f}, pv[2] = {0.f, 0.f}, qv[2] = {1.f, 1.f};
    int up[2] = {-1, -1}, tok[2] = {-1, -1};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      if (i >= rr.n) continue;
      u[h] = p.uniforms[rr.row0 + i];
      if (i == 0) continue;
      up[h] = parent_of(p.rows.parents, rr.row0 + i, i, p.err);
      tok[h] = p.tokens[rr.row0 + i];
      if (tok[h] < 0 || tok[h] >= p.V) {
        set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
        up[h] = -1;                          // never accepted
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (up[h] >= 0) {
        pv[h] = elem_to_float(P[(rr.row0 + up[h]) * p.ld_p + tok[h]]);
        if (Q) qv[h] = elem_to_float(Q[(rr.row0 + up[h]) * p.ld_q + tok[h]]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      node_s[lane + 32 * h] = {up[h], tok[h], u[h], pv[h]};
      q_s[lane + 32 * h] = qv[h];
    }
    if (lane == 0) {
      draw_s = u[0];
      walk_s = {0, 1, 0, 0, 0, rr.row0};
      state_s[4] = rr.n > 0 ? 0 : 3;
    }
    __syncwarp();
  }

  for (int pass = 0;; ) {
    // ---- the walk, until a sum over the row is needed (why 1) or it ends (why 2)
    if (warp == 0 && state_s[4] != 3) {
      int why = 2;
      const Node na = node_s[lane], nb = node_s[lane + 32];
      const float qa = q_s[lane], qb = q_s[lane + 32];
      auto [at, next, accepted, rounds, points, row0] = walk_s;
      Sum2 s = {pass > 0 ? before_s[W].hi : 1.f, 0.f};     // a row's sum is held in 32 bits
      bool have = true;                      // s is known
      // a node's first child is tried against s = 1 and p itself: all nodes' at once
      const Sum2 one = {1.f, 0.f};
      const unsigned yes_lo = __ballot_sync(0xffffffffu, accepts(na.u, qa, one, na.p));
      const unsigned yes_hi = __ballot_sync(0xffffffffu, accepts(nb.u, qb, one, nb.p));
      for (;;) {
        const unsigned lo = __ballot_sync(0xffffffffu, na.up == at && lane >= next);
        const unsigned hi = __ballot_sync(0xffffffffu, nb.up == at && lane + 32 >= next);
        if (!(lo | hi)) break;
        if (!have) {
          why = 1;
          break;
        }
        const int i = lo ? __ffs(lo) - 1 : __ffs(hi) + 31, from = i & 31;
        const bool high = i >= 32;
        const int x = __shfl_sync(0xffffffffu, high ? nb.tok : na.tok, from);
        float r[1] = {__shfl_sync(0xffffffffu, high ? nb.p : na.p, from)};
        next = i + 1;
        bool yes = ((high ? yes_hi : yes_lo) >> from) & 1;
        if (rounds | points) {
          const float ui = __shfl_sync(0xffffffffu, high ? nb.u : na.u, from);
          const float qi = __shfl_sync(0xffffffffu, high ? qb : qa, from);
          if (Q) {
            const float g[1] = {qi};
            const Left left = {rounds, round_s, 0, nullptr};
            left.of(r, g);
          } else {
            const bool gone = (lane < points && point_s[lane] == x) || (lane + 32 < points && point_s[lane + 32] == x);
            if (__any_sync(0xffffffffu, gone)) r[0] = 0.f;
          }
          yes = accepts(ui, qi, s, r[0]);
        }
        if (yes) {
          if (lane == 0) {
            path_s[accepted] = i;
            taken_s[accepted] = x;
          }
          ++accepted;
          at = i;
          rounds = points = 0;
          s = {1.f, 0.f};
        } else if (Q) {
          if (lane == 0) round_s[rounds] = s.hi;
          ++rounds;
          have = false;
        } else {
          s.add(-r[0]);
          s = s.normal();
          if (r[0] == r[0]) {                // (NaN stays, for the row's sum to show)
            if (lane == 0) point_s[points] = x;
            ++points;
          }
        }
        __syncwarp();
      }
      if (lane == 0) {
        walk_s = {at, next, accepted, rounds, points, row0};
        state_s[0] = row0 + at;
        state_s[1] = accepted;
        state_s[2] = rounds;
        state_s[3] = points;
        state_s[4] = why;
      }
    }
    __syncthreads();
    const int why = state_s[4];
    if (why == 3) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      break;
    }
    const long long row = state_s[0];
    Left left = {state_s[2], round_s, state_s[3], point_s};

    Sum2 total = {0.f, 0.f};
    bool late = false;
    for (int attempt = 0; attempt < 2; ++attempt) {
      // ---- the warp's part of the row: chunks c0 .. c1 - 1
      const Row nr(P + row * p.ld_p, left.rounds ? Q + row * p.ld_q : nullptr, p.V);
      const int w = rank * kWarps + warp;
      const int c0 = (int)((long long)nr.rc.chunks * w / W), c1 = (int)((long long)nr.rc.chunks * (w + 1) / W);
      Sum2 sum = {0.f, 0.f};
      auto part = [&](auto mode) {           // 0: p alone, 1: q's chunks too, 2: q's elements
        constexpr int M = decltype(mode)::value;
        constexpr int kBatch = M == 0 ? 8 : M == 1 ? 5 : 2;     // chunks that a lane waits for at once
        for (int c = c0 + lane; c < c1; c += 32 * kBatch) {
          typename Row::Raw raw[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) raw[k] = nr.template load<M>(min(c + 32 * k, c1 - 1));
          // whether a struck token lies in these chunks (a batch spans 32 kBatch of them)
          bool near = false;
          if (M == 0)
            for (int j = 0; j < left.points; ++j) {
              const int d = left.token[j] - nr.rc.head - (c - lane) * N;
              near = near || (d >= 0 && d < 32 * kBatch * N);
            }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if (c + 32 * k >= c1) break;
            float r[N];
            nr.template left_of<M>(raw[k], left, near, c + 32 * k, r);
#pragma unroll
            for (int e = 0; e < N; ++e) sum.add(r[e]);
          }
        }
      };
      if (!nr.q) part(Int<0>{});
      else if (nr.q_fits) part(Int<1>{});
      else part(Int<2>{});
      if (w == 0 && lane < nr.rc.head) sum.add(nr.element(left, lane));
      if (w == W - 1 && lane < nr.rc.tail) sum.add(nr.element(left, p.V - nr.rc.tail + lane));
      const Sum2 mine = warp_sum(sum);
      if (pass == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // its barriers can be sent to
      // ---- to the whole cluster.  Two buffers, whose barriers count the sums' bytes: one is
      // sent to again only in the next pass but one, after its reader has sent in the next.
      const int buf = pass & 1;
      if (lane < C) send_f2(&sums_s[buf][w], &sums_bar[buf], lane, mine.hi, mine.lo);
      if (warp == 0) {
        late = !wait_cluster(&sums_bar[buf], (pass >> 1) & 1);
        if (lane == 0) sm100::mbar_arrive_expect_tx(&sums_bar[buf], (uint32_t)(W * sizeof(float2)));
        // the sums before each part, in the vocabulary's order: some parts in a row a lane
        Sum2 x[kLaneParts], in = {0.f, 0.f};
        const int each = (W + 31) / 32;
#pragma unroll
        for (int k = 0; k < kLaneParts; ++k) {
          const int i = lane * each + k;
          x[k] = in;
          if (k < each && i < W) in = in + Sum2{sums_s[buf][i].x, sums_s[buf][i].y};
        }
        const Sum2 up_to = warp_scan(in);
        Sum2 before = shfl_up(up_to, 1);
        if (lane == 0) before = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kLaneParts; ++k)
          if (k < each && lane * each + k < W) before_s[lane * each + k] = (before + x[k]).normal();
        if (lane == 31) before_s[W] = up_to.normal();
        if (__any_sync(0xffffffffu, late) && lane == 0) {
          set_device_error(p.err, DSPARK_ERR_TIMEOUT);
          state_s[4] = 4;
        }
      }
      ++pass;
      __syncthreads();
      if (state_s[4] == 4) break;
      total = before_s[W];
      if (why == 1 || total.hi != 0.f || (!left.rounds && !left.points)) break;
      left.rounds = left.points = 0;         // nothing is left: from the target's own row
    }
    if (state_s[4] == 4) break;
    if (why == 1) continue;

    // ---- the last draw: the first v whose sum up to it exceeds u total
    const bool valid = total.hi > 0.f && total.hi < INFINITY;
    const Sum2 t = Sum2{draw_s, 0.f} * total;
    // the last part that is not empty and starts at or before t
    int target = 0;
    for (int w0 = lane; w0 < W; w0 += 32)
      if (!before_s[w0].beyond(t) && before_s[w0 + 1].beyond(before_s[w0])) target = w0;
    target = __reduce_max_sync(0xffffffffu, target);
    const bool writer = valid ? target / kWarps == rank : rank == 0;
    if (writer) {
      if (tid == 0) pick_s = -1;
      if (valid) {
        const Row nr(P + row * p.ld_p, left.rounds ? Q + row * p.ld_q : nullptr, p.V);
        int c0 = (int)((long long)nr.rc.chunks * target / W), c1 = (int)((long long)nr.rc.chunks * (target + 1) / W);
        bool with_head = target == 0, with_tail = target == W - 1;
        Sum2 base = before_s[target];
        constexpr int kHold = 2;             // chunks that a thread holds
        for (;;) {
          // the threads share the chunks out again, in order; more than they hold are narrowed
          // down to one thread's first
          const int each = (c1 - c0 + kThreads - 1) / kThreads;
          const bool last = each <= kHold;
          const int a0 = min(c0 + tid * each, c1), a1 = min(a0 + each, c1);
          const bool mine_head = with_head && tid == 0, mine_tail = with_tail && tid == kThreads - 1;
          float held[kHold][N];
          Sum2 sum = {0.f, 0.f};
          if (mine_head)
            for (int v = 0; v < nr.rc.head; ++v) sum.add(nr.element(left, v));
          if (last) {
            typename Row::Raw raw[kHold];
#pragma unroll
            for (int k = 0; k < kHold; ++k)
              if (a0 + k < a1) raw[k] = nr.load_any(a0 + k);
#pragma unroll
            for (int k = 0; k < kHold; ++k)
              if (a0 + k < a1) {
                nr.left_of_any(raw[k], left, a0 + k, held[k]);
#pragma unroll
                for (int e = 0; e < N; ++e) sum.add(held[k][e]);
              }
          } else {
            for (int c = a0; c < a1; ++c) {
              float r[N];
              nr.left_of_any(nr.load_any(c), left, c, r);
#pragma unroll
              for (int e = 0; e < N; ++e) sum.add(r[e]);
            }
          }
          if (mine_tail)
            for (int v = p.V - nr.rc.tail; v < p.V; ++v) sum.add(nr.element(left, v));
          const Sum2 mine = sum, in = warp_scan(mine);
          if (lane == 31) scan_s[warp] = in;
          if (tid == 0) key_s = INT_MAX;
          __syncthreads();
          // the warps' sums again by every warp: the sums before its own
          const Sum2 warps = warp_scan(lane < kWarps ? scan_s[lane] : Sum2{0.f, 0.f});
          const int wb = max(warp - 1, 0);
          Sum2 before = {__shfl_sync(0xffffffffu, warps.hi, wb), __shfl_sync(0xffffffffu, warps.lo, wb)};
          before = warp ? base + before : base;
          Sum2 mine_before = shfl_up(in, 1);
          mine_before = lane ? before + mine_before : before;
          // the first thread that goes beyond t; by rounding there may be none, then the last
          // thread that has anything
          const unsigned beyond = __ballot_sync(0xffffffffu, mine.hi > 0.f && (before + in).normal().beyond(t));
          const unsigned any = __ballot_sync(0xffffffffu, mine.hi > 0.f);
          if (lane == 0 && any)
            atomicMin(&key_s, beyond ? warp * 32 + __ffs(beyond) - 1
                                     : (1 << 20) - (warp * 32 + 31 - __clz(any)));   // (the last is the least of these)
          __syncthreads();
          const int k = key_s, who = k > (1 << 19) && k != INT_MAX ? (1 << 20) - k : k;
          if (who >= kThreads) break;        // (nothing: pick_s stays -1)
          if (last) {
            // the elements of that thread, at most 32 of them with a row's ends, a lane each
            const int first = nr.rc.head + min(c0 + who * each, c1) * N - (with_head && who == 0 ? nr.rc.head : 0);
            if (tid == who) {
              int m = 0;
              if (mine_head)
                for (int v = 0; v < nr.rc.head; ++v) ends_s[m++] = nr.element(left, v);
#pragma unroll
              for (int h = 0; h < kHold; ++h)
                if (a0 + h < a1) {
#pragma unroll
                  for (int e = 0; e < N; ++e) ends_s[m + e] = held[h][e];
                  m += N;
                }
              if (mine_tail)
                for (int v = p.V - nr.rc.tail; v < p.V; ++v) ends_s[m++] = nr.element(left, v);
              for (; m < 32; ++m) ends_s[m] = 0.f;
              scan_s[0] = mine_before;
            }
            __syncthreads();
            if (warp == 0) {
              const float r = ends_s[lane];
              const Sum2 up_to = (scan_s[0] + warp_scan({r, 0.f})).normal();
              const unsigned past = __ballot_sync(0xffffffffu, r > 0.f && up_to.beyond(t));
              const unsigned some = __ballot_sync(0xffffffffu, r > 0.f);
              if (lane == 0) pick_s = first + (past ? __ffs(past) - 1 : 31 - __clz(some));
            }
            break;
          }
          if (tid == who) {
            scan_s[0] = mine_before;
            part_s[0] = a0;
            part_s[1] = a1;
          }
          __syncthreads();
          base = scan_s[0];
          c0 = part_s[0];
          c1 = part_s[1];
          with_head = with_head && who == 0;
          with_tail = with_tail && who == kThreads - 1;
          __syncthreads();
        }
      }
      __syncthreads();
      // ---- results
      const int k = state_s[1];
      if (tid == 0 && pick_s < 0) set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
      for (int j = tid; j < p.rows.N; j += kThreads) {
        const long long o = (long long)b * p.rows.N + j;
        p.path[o] = j < k ? path_s[j] : -1;
        p.out_tokens[o] = j < k ? taken_s[j] : j == k ? pick_s : -1;
      }
      if (tid == 0) {
        p.accept_len[b] = k;
        p.n_out[b] = k + 1;
      }
    }
    break;
  }
  if (state_s[4] >= 3 && rank == 0) {        // no tokens, or a wait ran out: no answer
    for (int j = tid; j < p.rows.N; j += kThreads) {
      p.path[(long long)b * p.rows.N + j] = -1;
      p.out_tokens[(long long)b * p.rows.N + j] = -1;
    }
    if (tid == 0) {
      p.accept_len[b] = 0;
      p.n_out[b] = 0;
    }
  }
  if (state_s[4] >= 3) cluster_sync();       // (else it has all that is sent to it)
}

template <typename T>
cudaError_t verify_for(VerifyParams p, cudaStream_t stream) {
  // CTAs a request: as many as the device holds at once, two an SM, while every warp has a few
  // chunks.  (256 chains of 129280 in fp32: 39 us with two CTAs each, 46 and 66 with four and
  // eight, whose walks and draws come in more waves; 64 trees of 151936 in bf16: 15 us with
  // four, 21 with eight.)
  const int chunks = cdiv(p.V, Chunk<T>::N);
  p.log_C = 0;
  while (p.log_C < 3 && (p.rows.B << (p.log_C + 1)) <= 304 && chunks >= (kThreads << (p.log_C + 1))) ++p.log_C;
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
