// Embedding lookup with scaling, and its gradient summed over every token's occurrences.
//
// billytse.dev DSpark page, section 3.3: W1 is the previous token's small embedding; the
// Markov bias reads its rows by token id.  out[n] = scale W[id_n] (0 where id_n is -1), and
// the table's gradient is dW[v] = scale sum_{n : id_n = v} d_out[n].
//
// The lookup is a copy bound by memory: a warp a row, 16 bytes a lane.
//
// The gradient sums in a fixed order, so equal inputs give equal bits: the positions are
// sorted by (id, position), and tiles of consecutive sorted positions are summed in fp32,
// whatever the token frequencies.  A run of one id inside a tile is written at once; a run
// that crosses tiles leaves partial sums that are joined in tile order, first within a CTA
// (8 tiles, shared memory), then by a last kernel (workspace).  Up to 8192 positions are
// sorted by counting (every item against every key, 1 launch), more by a radix sort of 9
// bits a pass.  The table's zeroes are the bulk of the bytes: CTAs of every launch
// write a share of them, beside the sort and the sums.
#include "internal.h"
#include "rows.cuh"

namespace dspark {
namespace {

constexpr int kEmThreads = 256;
constexpr int kEmWarps = kEmThreads / 32;
constexpr int kRankMost = 8192;             // positions sorted by counting
constexpr int kRankItems = 32;              // items of a counting CTA, 8 threads each
constexpr int kRadixBits = 9, kRadix = 1 << kRadixBits;
constexpr int kRadixTile = 2048;            // keys of a radix CTA
constexpr int kRadixRounds = kRadixTile / kEmThreads;

// ---------------------------------------------------------------------------- lookup
struct EmParams {
  const void* W;
  long long ld;
  const int32_t* ids;
  int N, V, D;
  float scale;
  void* out;
  long long ld_out;
  int* err;
};

template <typename O, int N>
__device__ __forceinline__ void store_vec(O* p, const float (&v)[N]) {
  constexpr int M = Chunk<O>::N;
#pragma unroll
  for (int j = 0; j < N / M; ++j) {
    float w[M];
#pragma unroll
    for (int e = 0; e < M; ++e) w[e] = v[j * M + e];
    reinterpret_cast<uint4*>(p)[j] = pack_chunk<O>(w);
  }
}

template <typename T, typename O, bool Vec>
__global__ void __launch_bounds__(kEmThreads) embed_kernel(EmParams a) {
  constexpr int N = Chunk<T>::N;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  // rows, or the parts of `cols` columns of rows, one to a warp
  constexpr int kCols = 32 * N * 4;
  const int parts = (a.D + kCols - 1) / kCols;
  const long long units = (long long)a.N * parts;
  const long long u = (long long)blockIdx.x * kEmWarps + (threadIdx.x >> 5);
  if (u >= units) return;
  const int n = (int)(u / parts), d0 = (int)(u - (long long)n * parts) * kCols;
  const int d1 = min(a.D, d0 + kCols);
  const int id = a.ids[n];
  O* out = static_cast<O*>(a.out) + (long long)n * a.ld_out;
  const bool in = id >= 0 && id < a.V;
  if (!in && id != -1 && lane == 0) set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
  const T* row = static_cast<const T*>(a.W) + (long long)(in ? id : 0) * a.ld;
  if constexpr (Vec) {
    uint4 q[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = d0 + (g * 32 + lane) * N;
      q[g] = in && d < d1 ? __ldg(reinterpret_cast<const uint4*>(row + d)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = d0 + (g * 32 + lane) * N;
      if (d >= d1) break;
      float v[N];
      unpack_chunk<T>(q[g], v);
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] *= a.scale;
      if (!in) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = 0.f;
      }
      store_vec<O, N>(out + d, v);
    }
  } else {
#pragma unroll 4
    for (int d = d0 + lane; d < d1; d += 32)
      out[d] = elem_from_float<O>(in ? elem_to_float(row[d]) * a.scale : 0.f);
  }
}

// ---------------------------------------------------------------------------- gradient
struct EgParams {
  const void* d_out;
  long long ld;
  const int32_t* ids;
  int N, V, D;
  float scale;
  int accumulate;
  void* dW;
  long long ld_w;
  int elem_w;                // bytes of an element of dW
  int* err;
  int* key[2];               // sorted ids (V where there is no token), two buffers
  int* pos[2];               // their positions
  int* counts;               // [radix tiles][kRadix]
  float* part;               // [CTA tiles][2][D]: a run that came in, a run that goes on
  int P, tiles, cols;        // positions of a warp's tile, CTA tiles, column blocks
};

__device__ __forceinline__ int key_of(const EgParams& a, int n) {
  const int id = a.ids[n];
  if (id >= 0 && id < a.V) return id;
  if (id != -1) set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
  return a.V;
}

// The table's zeroes are dealt over every launch of the call (`fill` CTAs of each), so that
// they hide the sort and the sums: before the sums all rows of a CTA's share, with the sums
// and after them only the rows that no position has.
struct Fill {
  int first;                 // the launch's first filling CTA in its grid
  int from, all;             // its share is part (blockIdx - first) + from of `all`
};
__device__ __forceinline__ void share_of(const EgParams& a, const Fill& f, int& v0, int& v1) {
  const long long part = f.from + ((int)blockIdx.x - f.first);
  v0 = (int)((long long)a.V * part / f.all);
  v1 = (int)((long long)a.V * (part + 1) / f.all);
}
// `bytes` zeroes from p on, by `threads` threads
__device__ __forceinline__ void zero_bytes(char* p, long long bytes, int t, int threads) {
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  const int head = (int)min(bytes, (long long)((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u));
  uint4* q = reinterpret_cast<uint4*>(p + head);
  const long long n4 = (bytes - head) / 16;
  long long i = t;
  for (; i + 3 * threads < n4; i += 4 * threads) {
    __stcs(q + i, z);
    __stcs(q + i + threads, z);
    __stcs(q + i + 2 * threads, z);
    __stcs(q + i + 3 * threads, z);
  }
  for (; i < n4; i += threads) __stcs(q + i, z);
  const int tail = (int)(bytes - head - n4 * 16);
  if (t < head) p[t] = 0;
  if (t < tail) p[bytes - tail + t] = 0;
}
__device__ __forceinline__ void fill_rows(const EgParams& a, const Fill& f) {
  int v0, v1;
  share_of(a, f, v0, v1);
  const long long row = (long long)a.D * a.elem_w, step = a.ld_w * a.elem_w;
  char* base = static_cast<char*>(a.dW) + v0 * step;
  if (step == row) {
    zero_bytes(base, row * (v1 - v0), threadIdx.x, kEmThreads);
  } else {
    for (int v = threadIdx.x >> 5; v < v1 - v0; v += kEmWarps)
      zero_bytes(base + v * step, row, threadIdx.x & 31, 32);
  }
}
// The same without the rows of the sorted keys: `block` threads mark them in shared memory,
// kFillRows rows at a time.
constexpr int kFillRows = 2048;
__device__ __forceinline__ void fill_other_rows(const EgParams& a, const Fill& f, const int* skey,
                                                uint32_t* marks, int block) {
  __shared__ int found_s;
  int v0, v1;
  share_of(a, f, v0, v1);
  const long long row = (long long)a.D * a.elem_w, step = a.ld_w * a.elem_w;
  char* base = static_cast<char*>(a.dW);
  // the first sorted position of a key >= v0: `block` probes at a time
  int lo = 0, hi = a.N;
  while (hi > lo) {
    const int width = (hi - lo + block - 1) / block;
    const int at = lo + (int)threadIdx.x * width;
    __syncthreads();
    if (threadIdx.x == 0) found_s = 0;
    __syncthreads();
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && skey[at] < v0);
    if ((threadIdx.x & 31) == 0 && below) atomicAdd(&found_s, __popc(below));
    __syncthreads();
    const int n = found_s;                  // probes 0 .. n - 1 are below v0
    const int end = hi;
    hi = min(end, lo + n * width);
    lo = n == 0 ? lo : lo + (n - 1) * width + 1;
    if (n == 0) hi = lo;
  }
  for (int r0 = v0; r0 < v1; r0 += kFillRows) {
    const int r1 = min(v1, r0 + kFillRows);
    __syncthreads();
    for (int i = threadIdx.x; i < kFillRows / 32; i += block) marks[i] = 0u;
    __syncthreads();
    // this part's keys, `block` at a time
    for (;;) {
      const int i = lo + threadIdx.x;
      const int k = i < a.N ? skey[i] : a.V;
      if (k < r1) atomicOr(&marks[(k - r0) >> 5], 1u << ((k - r0) & 31));
      const int n = __syncthreads_count(k < r1);
      lo += n;
      if (n < block) break;
    }
    for (int v = r0 + (threadIdx.x >> 5); v < r1; v += block / 32)
      if (!(marks[(v - r0) >> 5] >> ((v - r0) & 31) & 1u)) zero_bytes(base + v * step, row, threadIdx.x & 31, 32);
  }
}

// every item's place among all keys: the keys below it, and the equal ones before it
__global__ void __launch_bounds__(kEmThreads) eg_rank_kernel(EgParams a, Fill f) {
  extern __shared__ int4 keys4[];
  int* keys = reinterpret_cast<int*>(keys4);
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x >= f.first) {
    fill_rows(a, f);
    return;
  }
  const int n4 = (a.N + 3) / 4;
  for (int i = threadIdx.x; i < 4 * n4; i += kEmThreads) keys[i] = i < a.N ? key_of(a, i) : 0x7FFFFFFF;
  __syncthreads();
  const int item = blockIdx.x * kRankItems + (threadIdx.x >> 3), sub = threadIdx.x & 7;
  const int k = item < a.N ? keys[item] : 0;
  int r = 0;
  const int own = item >> 2;
  for (int j = sub; j < n4; j += 8) {
    const int4 o = keys4[j];
    if (j == own) {
      const int m = 4 * j;
      r += (o.x < k || (o.x == k && m < item)) + (o.y < k || (o.y == k && m + 1 < item)) +
           (o.z < k || (o.z == k && m + 2 < item)) + (o.w < k || (o.w == k && m + 3 < item));
    } else {
      const int below = j < own ? k : k - 1;
      r += (o.x <= below) + (o.y <= below) + (o.z <= below) + (o.w <= below);
    }
  }
#pragma unroll
  for (int m = 4; m >= 1; m >>= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
  if (sub == 0 && item < a.N) {
    a.key[0][r] = k;
    a.pos[0][r] = item;
  }
}

// radix pass: digit counts of every tile
__global__ void __launch_bounds__(kEmThreads) eg_count_kernel(EgParams a, int pass, Fill f) {
  __shared__ int hist[kRadix];
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x >= f.first) {
    fill_rows(a, f);
    return;
  }
  for (int i = threadIdx.x; i < kRadix; i += kEmThreads) hist[i] = 0;
  __syncthreads();
  const int* in = a.key[(pass & 1) ^ 1];
  const int base = blockIdx.x * kRadixTile, shift = pass * kRadixBits;
#pragma unroll
  for (int i = 0; i < kRadixRounds; ++i) {
    const int n = base + i * kEmThreads + threadIdx.x;
    if (n < a.N) {
      const int k = pass == 0 ? key_of(a, n) : in[n];
      atomicAdd(&hist[(k >> shift) & (kRadix - 1)], 1);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRadix; i += kEmThreads) a.counts[(size_t)blockIdx.x * kRadix + i] = hist[i];
}

// radix pass: every key to its place, equal digits in their order
__global__ void __launch_bounds__(kEmThreads) eg_scatter_kernel(EgParams a, int pass, Fill f) {
  __shared__ int wh[kEmWarps][kRadix];
  __shared__ int base_s[kRadix];
  __shared__ int warp_s[kEmWarps];
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x >= f.first) {
    fill_rows(a, f);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shift = pass * kRadixBits;
  const int* in_k = a.key[(pass & 1) ^ 1];
  const int* in_p = a.pos[(pass & 1) ^ 1];
  for (int i = tid; i < kEmWarps * kRadix; i += kEmThreads) (&wh[0][0])[i] = 0;
  // bins 2 tid and 2 tid + 1: keys of this digit in the tiles before, and in all
  int before[2] = {0, 0}, all[2] = {0, 0};
  const int tile = blockIdx.x;
#pragma unroll 8
  for (int t = 0; t < f.first; ++t) {
    const int2 n = *reinterpret_cast<const int2*>(a.counts + (size_t)t * kRadix + 2 * tid);
    all[0] += n.x;
    all[1] += n.y;
    if (t < tile) {
      before[0] += n.x;
      before[1] += n.y;
    }
  }
  const int pair = all[0] + all[1];
  int scan = pair;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, scan, m);
    if (lane >= m) scan += o;
  }
  if (lane == 31) warp_s[warp] = scan;
  __syncthreads();                          // also: wh is zero
  int first = scan - pair;
  for (int w = 0; w < warp; ++w) first += warp_s[w];
  base_s[2 * tid] = first + before[0];
  base_s[2 * tid + 1] = first + all[0] + before[1];
  // this warp's keys, in order, 32 at a time
  int k[kRadixRounds], p[kRadixRounds], r[kRadixRounds];
  const int from = tile * kRadixTile + warp * (kRadixTile / kEmWarps);
#pragma unroll
  for (int i = 0; i < kRadixRounds; ++i) {
    const int n = from + 32 * i + lane;
    const bool on = n < a.N;
    k[i] = !on ? 0 : pass == 0 ? key_of(a, n) : in_k[n];
    p[i] = !on ? -1 : pass == 0 ? n : in_p[n];
  }
#pragma unroll
  for (int i = 0; i < kRadixRounds; ++i) {
    const int d = p[i] >= 0 ? (k[i] >> shift) & (kRadix - 1) : kRadix;    // kRadix: no key
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const int had = p[i] >= 0 ? wh[warp][d] : 0;
    __syncwarp();
    if (p[i] >= 0 && lane == __ffs(same) - 1) wh[warp][d] = had + __popc(same);
    __syncwarp();
    r[i] = had + __popc(same & ((1u << lane) - 1u));
  }
  __syncthreads();
  for (int b = tid; b < kRadix; b += kEmThreads) {
    int sum = base_s[b];
#pragma unroll
    for (int w = 0; w < kEmWarps; ++w) {
      const int x = wh[w][b];
      wh[w][b] = sum;
      sum += x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRadixRounds; ++i)
    if (p[i] >= 0) {
      const int to = wh[warp][(k[i] >> shift) & (kRadix - 1)] + r[i];
      a.key[pass & 1][to] = k[i];
      a.pos[pass & 1][to] = p[i];
    }
}

// A lane's N columns of column block cb: vector columns lie together, scalar ones 32 apart.
template <int N, bool Vec>
__device__ __forceinline__ int column(int cb, int lane, int e) {
  return Vec ? (cb * 32 + lane) * N + e : cb * 32 * N + e * 32 + lane;
}

template <typename O, int N, bool Vec>
__device__ __forceinline__ void add_to_row(const EgParams& a, int v, int cb, int lane, const float (&acc)[N]) {
  O* row = static_cast<O*>(a.dW) + (long long)v * a.ld_w;
  float x[N];
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = acc[e] * a.scale;
  const int d = column<N, Vec>(cb, lane, 0);
  if (Vec) {
    if (d >= a.D) return;
    if (a.accumulate) {
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] += elem_to_float(row[d + e]);
    }
    store_vec<O, N>(row + d, x);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int de = column<N, Vec>(cb, lane, e);
      if (de < a.D) row[de] = elem_from_float<O>(a.accumulate ? x[e] + elem_to_float(row[de]) : x[e]);
    }
  }
}

template <int N, bool Vec>
__device__ __forceinline__ void put_part(const EgParams& a, int tile, int slot, int cb, int lane,
                                         const float (&acc)[N]) {
  float* p = a.part + ((size_t)tile * 2 + slot) * a.D;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int d = column<N, Vec>(cb, lane, e);
    if (d < a.D) p[d] = acc[e];
  }
}

// Sums of the sorted positions: CTA = 8 consecutive tiles of P positions (a warp each) x one
// column block.
template <typename T, typename O, bool Vec>
__global__ void __launch_bounds__(kEmThreads) eg_sum_kernel(EgParams a, int buf, Fill f) {
  constexpr int N = Chunk<T>::N;
  constexpr int kAhead = 8;                 // rows in flight
  __shared__ float part_s[kEmWarps][2][N][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = blockIdx.x / a.cols, cb = blockIdx.x - cta * a.cols;
  pdl_wait();
  pdl_launch_dependents();
  const int* skey = a.key[buf];
  const int* spos = a.pos[buf];
  if ((int)blockIdx.x >= f.first) {
    fill_other_rows(a, f, skey, reinterpret_cast<uint32_t*>(part_s), kEmThreads);
    return;
  }
  const int P = a.P, V = a.V;
  const int cta0 = cta * kEmWarps * P;
  const int i0 = min(a.N, cta0 + warp * P), i1 = min(a.N, i0 + P), cnt = i1 - i0;
  const int key = lane < cnt ? skey[i0 + lane] : V;
  const int pos = lane < cnt ? spos[i0 + lane] : 0;
  const int prev = cnt > 0 && i0 > 0 ? skey[i0 - 1] : -1;
  const int next = i1 < a.N ? skey[i1] : V;
  const T* base = static_cast<const T*>(a.d_out);
  float acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.f;
  int run = __shfl_sync(0xffffffffu, key, 0);
  bool came_in = prev == run;
  auto flush = [&](bool goes_on) {
    if (run >= V) return;
    if (!came_in && !goes_on) {
      add_to_row<O, N, Vec>(a, run, cb, lane, acc);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) part_s[warp][came_in ? 0 : 1][e][lane] = acc[e];
    }
  };
  for (int j0 = 0; j0 < cnt; j0 += kAhead) {
    uint4 q[kAhead];
    float sc[Vec ? 1 : kAhead][N];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      const int k = __shfl_sync(0xffffffffu, key, j & 31), p = __shfl_sync(0xffffffffu, pos, j & 31);
      const bool on = j < cnt && k < V;
      const T* row = base + (long long)p * a.ld;
      if constexpr (Vec) {
        const int d = column<N, Vec>(cb, lane, 0);
        q[u] = on && d < a.D ? __ldcs(reinterpret_cast<const uint4*>(row + d)) : make_uint4(0u, 0u, 0u, 0u);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int d = column<N, Vec>(cb, lane, e);
          sc[u][e] = on && d < a.D ? elem_to_float(row[d]) : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= cnt) break;
      const int k = __shfl_sync(0xffffffffu, key, j & 31);
      if (k != run) {
        flush(false);
        run = k;
        came_in = false;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.f;
      }
      if constexpr (Vec) {
        float x[N];
        unpack_chunk<T>(q[u], x);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] += x[e];
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] += sc[u][e];
      }
    }
  }
  const bool goes_on = cnt > 0 && next == run;
  flush(goes_on);
  __syncthreads();
  // ---- runs across this CTA's tiles: summed by the warp in whose tile they begin, and by
  // warp 0 for the run that came in from the CTA before
  const int cta1 = min(a.N, cta0 + kEmWarps * P);
  auto join = [&](int k, int first_slot) {
    // tiles of this CTA that hold k from `warp` on; k goes on after the last of them?
    const bool beyond = cta1 < a.N && skey[cta1] == k;
    float sum[N];
#pragma unroll
    for (int e = 0; e < N; ++e) sum[e] = part_s[warp][first_slot][e][lane];
    for (int w = warp + 1; w < kEmWarps; ++w) {
      const int s0 = cta0 + w * P;
      if (s0 >= a.N || skey[s0] != k) break;
#pragma unroll
      for (int e = 0; e < N; ++e) sum[e] += part_s[w][0][e][lane];
    }
    if (first_slot == 0) {
      put_part<N, Vec>(a, cta, 0, cb, lane, sum);
    } else if (beyond) {
      put_part<N, Vec>(a, cta, 1, cb, lane, sum);
    } else {
      add_to_row<O, N, Vec>(a, k, cb, lane, sum);
    }
  };
  const int first_key = __shfl_sync(0xffffffffu, key, 0);
  if (warp == 0 && prev == first_key && first_key < V) join(first_key, 0);
  if (goes_on && !came_in && run < V) join(run, 1);
}

// Runs across CTA tiles: CTA (t, cb) sums the run that begins in t and goes on.  Four warps
// take consecutive parts of its tiles, joined in order.
template <typename O, int N, bool Vec>
__global__ void __launch_bounds__(128) eg_join_kernel(EgParams a, int buf, Fill f) {
  __shared__ float part_s[4][N][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x / a.cols, cb = blockIdx.x - t * a.cols;
  pdl_wait();
  pdl_launch_dependents();
  const int* skey = a.key[buf];
  if ((int)blockIdx.x >= f.first) {
    fill_other_rows(a, f, skey, reinterpret_cast<uint32_t*>(part_s), 128);
    return;
  }
  const int span = kEmWarps * a.P;
  const int i0 = t * span, i1 = i0 + span;
  if (i1 >= a.N) return;
  const int k = skey[i1];
  if (k >= a.V || skey[i1 - 1] != k) return;
  if (skey[i0] == k && i0 > 0 && skey[i0 - 1] == k) return;   // began before this tile
  int lo = i1 + 1, hi = a.N;                // the run's end
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (skey[mid] == k) lo = mid + 1;
    else hi = mid;
  }
  const int n = (lo - 1) / span - t;        // tiles after t that hold it
  const int u0 = (int)((long long)n * warp / 4), u1 = (int)((long long)n * (warp + 1) / 4);
  float sum[N];
#pragma unroll
  for (int e = 0; e < N; ++e) sum[e] = 0.f;
#pragma unroll 4
  for (int u = u0; u < u1; ++u) {
    const float* p = a.part + (size_t)(t + 1 + u) * 2 * a.D;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int d = column<N, Vec>(cb, lane, e);
      if (d < a.D) sum[e] += p[d];
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) part_s[warp][e][lane] = sum[e];
  __syncthreads();
  if (warp == 0) {
    const float* p = a.part + ((size_t)t * 2 + 1) * a.D;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int d = column<N, Vec>(cb, lane, e);
      sum[e] = d < a.D ? p[d] : 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) sum[e] += part_s[w][e][lane];
    }
    add_to_row<O, N, Vec>(a, k, cb, lane, sum);
  }
}

struct EgPlan {
  int P, tiles, radix_tiles, passes;
  size_t off_key[2], off_pos[2], off_counts, off_part, total;
};
EgPlan eg_plan(int N, int V, int D) {
  EgPlan p = {};
  // a lane's columns are 4 fp32 or 8 16-bit elements: the tile size goes by 4, the finer
  // block.  Tiles of 32 positions when that gives every SM two CTAs, else of 8.
  const long long cols = cdiv(D, 128);
  p.P = (long long)cdiv(N, 32 * kEmWarps) * cols >= 304 ? 32 : 8;
  p.tiles = cdiv(N, kEmWarps * p.P);
  p.radix_tiles = N > kRankMost ? cdiv(N, kRadixTile) : 0;
  int bits = 1;
  while (bits < 31 && (V >> bits) != 0) ++bits;         // keys 0 .. V
  p.passes = cdiv(bits, kRadixBits);
  size_t o = 256;
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && p.radix_tiles == 0) { p.off_key[1] = p.off_key[0]; p.off_pos[1] = p.off_pos[0]; break; }
    p.off_key[i] = o; o = align_up(o + (size_t)N * 4, 256);
    p.off_pos[i] = o; o = align_up(o + (size_t)N * 4, 256);
  }
  p.off_counts = o; o = align_up(o + (size_t)p.radix_tiles * kRadix * 4, 256);
  p.off_part = o; o = align_up(o + (size_t)p.tiles * 2 * D * 4, 256);
  p.total = o;
  return p;
}

bool rows_aligned(const void* p, long long ld, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * elem) % 16 == 0;
}

template <typename T, typename O>
cudaError_t launch_em(const EmParams& p, cudaStream_t stream) {
  const bool vec = rows_aligned(p.W, p.ld, sizeof(T)) && rows_aligned(p.out, p.ld_out, sizeof(O)) &&
                   p.D % Chunk<T>::N == 0;
  const long long units = (long long)p.N * cdiv(p.D, 32 * Chunk<T>::N * 4);
  const dim3 grid((unsigned)((units + kEmWarps - 1) / kEmWarps));
  return vec ? launch_pdl(embed_kernel<T, O, true>, grid, dim3(kEmThreads), 0, stream, p)
             : launch_pdl(embed_kernel<T, O, false>, grid, dim3(kEmThreads), 0, stream, p);
}

template <typename T, typename O, bool Vec>
cudaError_t launch_eg_sums(EgParams p, int buf, int fill, int from, int all, cudaStream_t stream) {
  p.cols = cdiv(p.D, 32 * Chunk<T>::N);
  const int ctas = p.tiles * p.cols;
  Fill f = {ctas, from, all};
  cudaError_t e = launch_pdl(eg_sum_kernel<T, O, Vec>, dim3((unsigned)(ctas + fill)), dim3(kEmThreads), 0,
                             stream, p, buf, f);
  if (e == cudaSuccess && p.tiles > 1) {
    f.from += fill;
    e = launch_pdl(eg_join_kernel<O, Chunk<T>::N, Vec>, dim3((unsigned)(ctas + fill)), dim3(128), 0, stream,
                   p, buf, f);
  }
  return e;
}

template <typename T, typename O>
cudaError_t launch_eg(EgParams p, void* ws, cudaStream_t stream) {
  const EgPlan plan = eg_plan(p.N, p.V, p.D);
  for (int i = 0; i < 2; ++i) {
    p.key[i] = ws_at<int>(ws, plan.off_key[i]);
    p.pos[i] = ws_at<int>(ws, plan.off_pos[i]);
  }
  p.counts = ws_at<int>(ws, plan.off_counts);
  p.part = ws_at<float>(ws, plan.off_part);
  p.P = plan.P;
  p.tiles = plan.tiles;
  p.elem_w = sizeof(O);
  int buf = 0, done = 0;
  cudaError_t e = cudaSuccess;
  // filling CTAs of each launch: four an SM, but no more than there are 16 KB to write
  const int launches = (plan.radix_tiles ? 2 * plan.passes : 1) + (p.N > 0) + (plan.tiles > 1);
  const long long most = (long long)p.V * p.D * p.elem_w / (16384LL * launches) + 1;
  const int fill = p.accumulate ? 0 : (int)(most < 4 * 152 ? most : 4 * 152);
  const int all = launches * fill;
  if (plan.radix_tiles == 0) {
    const int ctas = cdiv(p.N, kRankItems);
    if (ctas + fill > 0)
      e = launch_pdl(eg_rank_kernel, dim3(ctas + fill), dim3(kEmThreads), align_up((size_t)p.N * 4, 16), stream,
                     p, Fill{ctas, 0, all});
    if (p.N == 0) return e;
    done = 1;
  } else {
    for (int i = 0; i < plan.passes && e == cudaSuccess; ++i) {
      const dim3 grid(plan.radix_tiles + fill);
      e = launch_pdl(eg_count_kernel, grid, dim3(kEmThreads), 0, stream, p, i,
                     Fill{plan.radix_tiles, done++ * fill, all});
      if (e == cudaSuccess)
        e = launch_pdl(eg_scatter_kernel, grid, dim3(kEmThreads), 0, stream, p, i,
                       Fill{plan.radix_tiles, done++ * fill, all});
    }
    buf = (plan.passes - 1) & 1;
  }
  if (e != cudaSuccess) return e;
  const bool vec = rows_aligned(p.d_out, p.ld, sizeof(T)) && rows_aligned(p.dW, p.ld_w, sizeof(O)) &&
                   p.D % Chunk<T>::N == 0;
  return vec ? launch_eg_sums<T, O, true>(p, buf, fill, done * fill, all, stream)
             : launch_eg_sums<T, O, false>(p, buf, fill, done * fill, all, stream);
}

}  // namespace

size_t embed_grad_bytes(int N, int V, int D) { return eg_plan(N, V, D).total; }

cudaError_t launch_embed(const void* W, int dtype, long long ld, const int32_t* ids, int N, int V, int D,
                         float scale, void* out, int out_dtype, long long ld_out, int* err,
                         cudaStream_t stream) {
  const EmParams p = {W, ld, ids, N, V, D, scale, out, ld_out, err};
  if (dtype == DSPARK_F32) return launch_em<float, float>(p, stream);
  if (dtype == DSPARK_BF16)
    return out_dtype == DSPARK_F32 ? launch_em<__nv_bfloat16, float>(p, stream)
                                   : launch_em<__nv_bfloat16, __nv_bfloat16>(p, stream);
  return out_dtype == DSPARK_F32 ? launch_em<__half, float>(p, stream) : launch_em<__half, __half>(p, stream);
}

cudaError_t launch_embed_grad(const void* d_out, int dtype, long long ld, const int32_t* ids, int N, int V,
                              int D, float scale, int accumulate, void* dW, int w_dtype, long long ld_w,
                              int* err, void* ws, cudaStream_t stream) {
  EgParams p = {};
  p.d_out = d_out; p.ld = ld; p.ids = ids; p.N = N; p.V = V; p.D = D; p.scale = scale;
  p.accumulate = accumulate; p.dW = dW; p.ld_w = ld_w; p.err = err;
  if (dtype == DSPARK_F32) return launch_eg<float, float>(p, ws, stream);
  if (dtype == DSPARK_BF16)
    return w_dtype == DSPARK_F32 ? launch_eg<__nv_bfloat16, float>(p, ws, stream)
                                 : launch_eg<__nv_bfloat16, __nv_bfloat16>(p, ws, stream);
  return w_dtype == DSPARK_F32 ? launch_eg<__half, float>(p, ws, stream) : launch_eg<__half, __half>(p, ws, stream);
}

}  // namespace dspark
