// Embedding lookup with scaling, and its gradient summed over every token's occurrences.
//
// billytse.dev DSpark page, section 3.3: W1 is the previous token's small embedding; the
// Markov bias reads its rows by token id.  out[n] = scale W[id_n] (0 where id_n is -1), and
// the table's gradient is dW[v] = scale sum_{n : id_n = v} d_out[n].
//
// The lookup is a copy bound by memory: a warp a row (or 2 KB of it), 16 bytes a lane.  16384
// rows of 2560 in bf16: 19.9 us for 168 MB, some of them from L2.
//
// The gradient sums in a fixed order, so equal inputs give equal bits: the positions are
// sorted by (id, position), and tiles of consecutive sorted positions are summed in fp32,
// whatever the token frequencies.  A run of one id inside a tile is written at once; a run
// that crosses tiles leaves partial sums that are joined in tile order, first within a CTA
// (8 tiles, shared memory), then by a last kernel (workspace).  The sort is a stable
// radix sort of 9 bits a pass, by one cluster of CTAs where the zeroes hide it or positions are
// few (1 launch), else by the grid (2 launches a pass); up to 2048 positions need none (eg_range_kernel).  The
// table's zeroes, the bulk of the bytes, are written in the sort's launch by the CTAs that do
// not sort, so that the sort hides behind them.
//
// Measured on a GB300 (copy rate 6782 GB/s; a plain memset writes 7.5 TB/s): 32768 positions of
// 151936 x 2560 in bf16, tokens by 1 / rank, 167 us for 946 MB = 5.68 TB/s (sort and zeroes 115,
// sums 41, join under 10); 1280 positions of 129280 x 256 in fp32, 26 us for 134 MB = 5.2 TB/s (a
// memset of the table alone takes 21).
#include "internal.h"
#include "rows.cuh"

namespace dspark {
namespace {

constexpr int kEmThreads = 256;
constexpr int kEmWarps = kEmThreads / 32;
constexpr int kSortMost = 8192;             // positions always sorted by one cluster
// bytes of zeroes for each position that make the cluster's sort the shorter way
constexpr long long kSortHidden = 4000;
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
// Filling CTA `part` of `parts` zeroes its share of the table's rows.
__device__ __forceinline__ void fill_rows(const EgParams& a, int part, int parts) {
  const int v0 = (int)((long long)a.V * part / parts), v1 = (int)((long long)a.V * (part + 1) / parts);
  const long long row = (long long)a.D * a.elem_w, step = a.ld_w * a.elem_w;
  char* base = static_cast<char*>(a.dW) + v0 * step;
  if (step == row) {
    zero_bytes(base, row * (v1 - v0), threadIdx.x, kEmThreads);
  } else {
    for (int v = threadIdx.x >> 5; v < v1 - v0; v += kEmWarps)
      zero_bytes(base + v * step, row, threadIdx.x & 31, 32);
  }
}

struct RadixShared {
  int warp[kEmWarps][kRadix];   // a warp's keys of each digit, then its places
  int base[kRadix];             // places of the next tile's keys of each digit
  int hist[kRadix];
  int sum[kEmWarps];
};

// The keys [from, from + kRadixTile) below `end` to their places, equal digits in their order;
// rs.base moves on.  All threads; rs.base is ready.
__device__ __forceinline__ void scatter_tile(const EgParams& a, int pass, int from, int end, RadixShared& rs) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shift = pass * kRadixBits;
  const int* in_k = a.key[(pass & 1) ^ 1];
  const int* in_p = a.pos[(pass & 1) ^ 1];
  __syncthreads();                          // rs.warp is free
  for (int i = tid; i < kEmWarps * kRadix; i += kEmThreads) (&rs.warp[0][0])[i] = 0;
  int k[kRadixRounds], p[kRadixRounds], r[kRadixRounds];
#pragma unroll
  for (int i = 0; i < kRadixRounds; ++i) {
    const int n = from + warp * (kRadixTile / kEmWarps) + 32 * i + lane;
    const bool on = n < end;
    k[i] = !on ? 0 : pass == 0 ? key_of(a, n) : in_k[n];
    p[i] = !on ? -1 : pass == 0 ? n : in_p[n];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRadixRounds; ++i) {
    const int d = p[i] >= 0 ? (k[i] >> shift) & (kRadix - 1) : kRadix;    // kRadix: no key
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const int had = p[i] >= 0 ? rs.warp[warp][d] : 0;
    __syncwarp();
    if (p[i] >= 0 && lane == __ffs(same) - 1) rs.warp[warp][d] = had + __popc(same);
    __syncwarp();
    r[i] = had + __popc(same & ((1u << lane) - 1u));
  }
  __syncthreads();
  for (int b = tid; b < kRadix; b += kEmThreads) {
    int sum = rs.base[b];
#pragma unroll
    for (int w = 0; w < kEmWarps; ++w) {
      const int x = rs.warp[w][b];
      rs.warp[w][b] = sum;
      sum += x;
    }
    rs.base[b] = sum;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRadixRounds; ++i)
    if (p[i] >= 0) {
      const int to = rs.warp[warp][(k[i] >> shift) & (kRadix - 1)] + r[i];
      a.key[pass & 1][to] = k[i];
      a.pos[pass & 1][to] = p[i];
    }
}

// rs.base of a part whose digits 2 tid and 2 tid + 1 have `before` keys in earlier parts and
// `all` in all parts.  All threads.
__device__ __forceinline__ void radix_base(const int (&before)[2], const int (&all)[2], RadixShared& rs) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = all[0] + all[1];
  int scan = pair;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, scan, m);
    if (lane >= m) scan += o;
  }
  if (lane == 31) rs.sum[warp] = scan;
  __syncthreads();
  int first = scan - pair;
  for (int w = 0; w < warp; ++w) first += rs.sum[w];
  rs.base[2 * tid] = first + before[0];
  rs.base[2 * tid + 1] = first + all[0] + before[1];
}

// digit counts of the keys [from, end), by all threads
__device__ __forceinline__ void radix_hist(const EgParams& a, int pass, int from, int end, RadixShared& rs) {
  const int tid = threadIdx.x;
  const int* in = a.key[(pass & 1) ^ 1];
  __syncthreads();
  for (int i = tid; i < kRadix; i += kEmThreads) rs.hist[i] = 0;
  __syncthreads();
  for (int n = from + tid; n < from + (end - from + 31) / 32 * 32; n += kEmThreads) {
    // (whole warps: lanes of one digit add once)
    const int k = n >= end ? -1 : pass == 0 ? key_of(a, n) : in[n];
    const int d = k < 0 ? kRadix : (k >> (pass * kRadixBits)) & (kRadix - 1);
    const unsigned same = __match_any_sync(0xffffffffu, d);
    if (k >= 0 && (tid & 31) == __ffs(same) - 1) atomicAdd(&rs.hist[d], __popc(same));
  }
  __syncthreads();
}

// The whole sort by one cluster of 8 CTAs, each with an eighth of the keys; the grid's other
// clusters write the table's zeroes meanwhile.
__global__ void __launch_bounds__(kEmThreads) eg_sort_kernel(EgParams a, int passes) {
  __shared__ RadixShared rs;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x >= 8) {
    fill_rows(a, blockIdx.x - 8, gridDim.x - 8);
    return;
  }
  const int c = blockIdx.x, tid = threadIdx.x;
  const int from = (int)((long long)a.N * c / 8), end = (int)((long long)a.N * (c + 1) / 8);
  for (int pass = 0; pass < passes; ++pass) {
    radix_hist(a, pass, from, end, rs);
    cluster_sync();
    int before[2] = {0, 0}, all[2] = {0, 0};
#pragma unroll
    for (int o = 0; o < 8; ++o) {
      const unsigned long long two = cluster_ld_u64(cluster_map(&rs.hist[2 * tid], o));
      const int n0 = (int)(uint32_t)two, n1 = (int)(two >> 32);
      all[0] += n0;
      all[1] += n1;
      if (o < c) {
        before[0] += n0;
        before[1] += n1;
      }
    }
    radix_base(before, all, rs);
    for (int t = from; t < end; t += kRadixTile) scatter_tile(a, pass, t, end, rs);
    cluster_sync();                         // the keys are in place, and the counts are read
  }
}

// radix pass over many keys: digit counts of every tile; in the first pass the grid's CTAs
// beyond the tiles write the table's zeroes
__global__ void __launch_bounds__(kEmThreads) eg_count_kernel(EgParams a, int pass, int tiles) {
  __shared__ RadixShared rs;
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x >= tiles) {
    fill_rows(a, blockIdx.x - tiles, gridDim.x - tiles);
    return;
  }
  const int from = blockIdx.x * kRadixTile;
  radix_hist(a, pass, from, min(a.N, from + kRadixTile), rs);
  for (int i = threadIdx.x; i < kRadix; i += kEmThreads) a.counts[(size_t)blockIdx.x * kRadix + i] = rs.hist[i];
}

// radix pass: every key to its place
__global__ void __launch_bounds__(kEmThreads) eg_scatter_kernel(EgParams a, int pass) {
  __shared__ RadixShared rs;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, tile = blockIdx.x, tiles = gridDim.x;
  int before[2] = {0, 0}, all[2] = {0, 0};
#pragma unroll 8
  for (int t = 0; t < tiles; ++t) {
    const int2 n = *reinterpret_cast<const int2*>(a.counts + (size_t)t * kRadix + 2 * tid);
    all[0] += n.x;
    all[1] += n.y;
    if (t < tile) {
      before[0] += n.x;
      before[1] += n.y;
    }
  }
  radix_base(before, all, rs);
  scatter_tile(a, pass, tile * kRadixTile, a.N, rs);
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
__global__ void __launch_bounds__(kEmThreads) eg_sum_kernel(EgParams a, int buf) {
  constexpr int N = Chunk<T>::N;
  constexpr int kAhead = 8;                 // rows in flight
  __shared__ float part_s[kEmWarps][2][N][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = blockIdx.x / a.cols, cb = blockIdx.x - cta * a.cols;
  pdl_wait();
  pdl_launch_dependents();
  const int* skey = a.key[buf];
  const int* spos = a.pos[buf];
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
__global__ void __launch_bounds__(128) eg_join_kernel(EgParams a, int buf) {
  __shared__ float part_s[4][N][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x / a.cols, cb = blockIdx.x - t * a.cols;
  pdl_wait();
  pdl_launch_dependents();
  const int* skey = a.key[buf];
  const int span = kEmWarps * a.P;
  const int i0 = t * span, i1 = i0 + span;
  if (i1 >= a.N) return;
  const int k = skey[i1];
  if (k >= a.V || skey[i1 - 1] != k) return;
  if (skey[i0] == k && i0 > 0 && skey[i0 - 1] == k) return;   // began before this tile
  // tiles after t that hold it: those that begin with it, 128 looked at together
  int n = 0;
  for (;;) {
    const long long at = (long long)(t + 1 + n + (int)threadIdx.x) * span;
    const int more = __syncthreads_count(at < a.N && skey[at] == k);
    n += more;
    if (more < 128) break;
  }
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

// Few positions of narrow rows: a CTA owns the table rows [range kRangeRows ..) of one column block (of all of
// them where rows are not 16-byte aligned).  It finds the positions of its rows among all ids,
// orders them by (id, position) with a counting sort in shared memory, zeroes the rows that
// have none and sums the others: one launch, and nothing waits for anything.  A run of
// kLongRun positions or more is summed by the CTA's eight warps, joined in order.
constexpr int kRangeMost = 2048;            // positions
constexpr int kRangeRows = 2048;            // rows of a CTA, at most
constexpr int kRangeCols = 4;               // column blocks (512 bytes of d_out), at most
constexpr int kLongRun = 64;
template <typename T, typename O, bool Vec>
__global__ void __launch_bounds__(kEmThreads) eg_range_kernel(EgParams a, int rows, int col_ctas) {
  constexpr int N = Chunk<T>::N;
  constexpr int kAhead = 8;
  __shared__ int count_s[kRangeRows];       // positions of a row
  __shared__ int start_s[kRangeRows];       // its first place in pos_s, then the place after its last
  __shared__ int row_s[kRangeMost];         // of every position: its row here, or -1
  __shared__ int pos_s[kRangeMost];
  __shared__ int hit_s[kRangeMost];         // rows with positions: short runs first, long ones last
  __shared__ int n_short_s, n_long_s, next_s;
  __shared__ float part_s[kEmWarps][N][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int range = blockIdx.x / col_ctas, cb0 = blockIdx.x - range * col_ctas;
  const int cb1 = Vec ? cb0 + 1 : a.cols;
  const int v0 = range * rows, n_rows = min(a.V - v0, rows);
  pdl_wait();
  pdl_launch_dependents();
  for (int i = tid; i < n_rows; i += kEmThreads) count_s[i] = 0;
  if (tid == 0) n_short_s = n_long_s = next_s = 0;
  __syncthreads();
  for (int n = tid; n < a.N; n += kEmThreads) {
    const int id = a.ids[n], v = id - v0;
    const bool in = v >= 0 && v < n_rows;
    if (in) atomicAdd(&count_s[v], 1);
    row_s[n] = in ? v : -1;
    if (blockIdx.x == 0 && (id < -1 || id >= a.V)) set_device_error(a.err, DSPARK_ERR_DEVICE_CHECK);
  }
  __syncthreads();
  if (warp == 0) {
    // ---- where each row's positions begin (consecutive rows to a lane), and the rows that
    // have any
    const int each = (n_rows + 31) / 32, r0 = min(n_rows, lane * each), r1 = min(n_rows, r0 + each);
    int sum = 0;
    for (int v = r0; v < r1; ++v) sum += count_s[v];
    int scan = sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, scan, m);
      if (lane >= m) scan += o;
    }
    int at = scan - sum;
    for (int v = r0; v < r1; ++v) {
      const int c = count_s[v];
      start_s[v] = at;
      at += c;
      if (c >= kLongRun) hit_s[kRangeMost - 1 - atomicAdd(&n_long_s, 1)] = v;
      else if (c > 0) hit_s[atomicAdd(&n_short_s, 1)] = v;
    }
    __syncwarp();
    // ---- places in position order: 32 positions at a time, equal ids by lane
    for (int n0 = 0; n0 < a.N; n0 += 32) {
      const int n = n0 + lane, v = n < a.N ? row_s[n] : -1;
      const bool in = v >= 0;
      if (!__any_sync(0xffffffffu, in)) continue;
      const unsigned same = __match_any_sync(0xffffffffu, in ? v : -1);
      if (in) pos_s[start_s[v] + __popc(same & ((1u << lane) - 1u))] = n;
      __syncwarp();
      if (in && lane == __ffs(same) - 1) start_s[v] += __popc(same);
      __syncwarp();
    }
    // the places are ready: this warp begins the sums while the others fill
    asm volatile("bar.arrive 1, %0;" ::"n"(kEmThreads) : "memory");
  } else {
    if (!a.accumulate) {
      // ---- the rows without a position
      constexpr int kFillers = kEmWarps - 1;
      const long long step = a.ld_w * a.elem_w;
      char* base = static_cast<char*>(a.dW) + v0 * step;
      if (Vec) {
        constexpr int kUnits = N * (int)sizeof(O) / 16;     // 16-byte stores of a lane
        const int d = column<N, Vec>(cb0, lane, 0);
        // rows of fewer than 32 lanes' columns: several at once
        const int lanes = min(32, (a.D - cb0 * 32 * N) / N);
        int log_each = 0;
        while (lanes <= 16 >> log_each) ++log_each;
        const int each = 1 << log_each, width = 32 >> log_each;
        const int mine = lane & (width - 1);
        char* at = base + (long long)(d - (lane - mine) * N) * sizeof(O);
#pragma unroll 4
        for (int v = (warp - 1) * each + (lane >> (5 - log_each)); v < n_rows; v += kFillers * each)
          if (mine < lanes && count_s[v] == 0) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
              __stcs(reinterpret_cast<uint4*>(at + v * step) + u, make_uint4(0u, 0u, 0u, 0u));
          }
      } else {
        for (int v = warp - 1; v < n_rows; v += kFillers)
          if (count_s[v] == 0) zero_bytes(base + v * step, (long long)a.D * a.elem_w, lane, 32);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kEmThreads) : "memory");
  }
  // ---- sums; start_s is now the place after a row's last
  const T* in = static_cast<const T*>(a.d_out);
  auto sum_run = [&](int from, int to, int cb, float (&acc)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    for (int j0 = from; j0 < to; j0 += kAhead) {
      uint4 q[kAhead];
      float sc[Vec ? 1 : kAhead][N];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool on = j0 + u < to;
        const T* row = in + (long long)pos_s[on ? j0 + u : from] * a.ld;
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
        if (j0 + u >= to) break;
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
  };
  float acc[N];
  // short runs, a warp each, as warps come free
  for (;;) {
    int h = 0;
    if (lane == 0) h = atomicAdd(&next_s, 1);
    h = __shfl_sync(0xffffffffu, h, 0);
    if (h >= n_short_s) break;
    const int v = hit_s[h];
    for (int cb = cb0; cb < cb1; ++cb) {
      sum_run(start_s[v] - count_s[v], start_s[v], cb, acc);
      add_to_row<O, N, Vec>(a, v0 + v, cb, lane, acc);
    }
  }
  __syncthreads();
  for (int h = 0; h < n_long_s; ++h) {
    const int v = hit_s[kRangeMost - 1 - h], n = count_s[v], from = start_s[v] - n;
    for (int cb = cb0; cb < cb1; ++cb) {
      sum_run(from + n * warp / kEmWarps, from + n * (warp + 1) / kEmWarps, cb, acc);
#pragma unroll
      for (int e = 0; e < N; ++e) part_s[warp][e][lane] = acc[e];
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < kEmWarps; ++w)
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] += part_s[w][e][lane];
        add_to_row<O, N, Vec>(a, v0 + v, cb, lane, acc);
      }
      __syncthreads();
    }
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
  p.radix_tiles = N > kSortMost ? cdiv(N, kRadixTile) : 0;
  int bits = 1;
  while (bits < 31 && (V >> bits) != 0) ++bits;         // keys 0 .. V
  p.passes = cdiv(bits, kRadixBits);
  size_t o = 256;
  for (int i = 0; i < 2; ++i) {
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
cudaError_t launch_eg_sums(EgParams p, int buf, cudaStream_t stream) {
  p.cols = cdiv(p.D, 32 * Chunk<T>::N);
  const int ctas = p.tiles * p.cols;
  cudaError_t e = launch_pdl(eg_sum_kernel<T, O, Vec>, dim3((unsigned)ctas), dim3(kEmThreads), 0, stream, p, buf);
  if (e == cudaSuccess && p.tiles > 1)
    e = launch_pdl(eg_join_kernel<O, Chunk<T>::N, Vec>, dim3((unsigned)ctas), dim3(128), 0, stream, p, buf);
  return e;
}

template <typename T, typename O, bool Vec>
cudaError_t launch_eg_range(EgParams p, cudaStream_t stream) {
  p.cols = cdiv(p.D, 32 * Chunk<T>::N);
  const int col_ctas = Vec ? p.cols : 1;
  // two CTAs an SM (1280 positions of 129280 x 256 in fp32: 26.8 us; four 29.3), or as many as
  // keep a CTA's rows within shared memory
  int ranges = cdiv(2 * 152, col_ctas);
  if (ranges < cdiv(p.V, kRangeRows)) ranges = cdiv(p.V, kRangeRows);
  if (ranges > p.V) ranges = p.V;
  const int rows = cdiv(p.V, ranges);
  return launch_pdl(eg_range_kernel<T, O, Vec>, dim3((unsigned)(cdiv(p.V, rows) * col_ctas)),
                    dim3(kEmThreads), 0, stream, p, rows, col_ctas);
}

template <typename T, typename O>
cudaError_t launch_eg(EgParams p, void* ws, cudaStream_t stream) {
  p.elem_w = sizeof(O);
  const bool vec = rows_aligned(p.d_out, p.ld, sizeof(T)) && rows_aligned(p.dW, p.ld_w, sizeof(O)) &&
                   p.D % Chunk<T>::N == 0;
  if (p.N == 0 && p.accumulate) return cudaSuccess;
  // (1280 positions of 129280 x 256 in fp32, 2 column blocks: 26 us and 32 by the sort; of
  // 30000 x 2560, 20 blocks: 78 and 57)
  if (p.N <= kRangeMost && cdiv(p.D, 32 * Chunk<T>::N) <= kRangeCols)
    return vec ? launch_eg_range<T, O, true>(p, stream) : launch_eg_range<T, O, false>(p, stream);
  const EgPlan plan = eg_plan(p.N, p.V, p.D);
  for (int i = 0; i < 2; ++i) {
    p.key[i] = ws_at<int>(ws, plan.off_key[i]);
    p.pos[i] = ws_at<int>(ws, plan.off_pos[i]);
  }
  p.counts = ws_at<int>(ws, plan.off_counts);
  p.part = ws_at<float>(ws, plan.off_part);
  p.P = plan.P;
  p.tiles = plan.tiles;
  const int buf = (plan.passes - 1) & 1;
  cudaError_t e = cudaSuccess;
  // zeroing CTAs: four an SM, but no more than there are 16 KB to write
  const long long most = (long long)p.V * p.D * p.elem_w / 16384 + 1;
  const int fill = p.accumulate ? 0 : (int)(most < 4 * 152 ? align_up((size_t)most, 8) : 4 * 152);
  // by the grid where the zeroes would not hide the cluster's sort: of 151936 x 256 in bf16 (78
  // MB) 16384, 32768, 131072 positions take 40, 60, 170 us by the cluster, 45, 54, 73 by the grid
  if (p.N <= kSortMost || (!p.accumulate && (long long)p.V * p.D * p.elem_w >= kSortHidden * p.N)) {
    e = launch_rows_cluster(eg_sort_kernel, 8 + fill, 8, kEmThreads, 0, stream, p, plan.passes);
  } else {
    for (int i = 0; i < plan.passes && e == cudaSuccess; ++i) {
      e = launch_pdl(eg_count_kernel, dim3(plan.radix_tiles + (i == 0 ? fill : 0)), dim3(kEmThreads), 0, stream, p,
                     i, plan.radix_tiles);
      if (e == cudaSuccess)
        e = launch_pdl(eg_scatter_kernel, dim3(plan.radix_tiles), dim3(kEmThreads), 0, stream, p, i);
    }
  }
  if (e != cudaSuccess || p.N == 0) return e;   // (no position: the zeroes are the gradient)
  return vec ? launch_eg_sums<T, O, true>(p, buf, stream) : launch_eg_sums<T, O, false>(p, buf, stream);
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
