// Keys and values of drafted tokens in a paged cache: appending them, normalised and rotated
// on the way, and keeping the accepted ones.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "target.cuh"

namespace dspark {
namespace {

struct AppendParams {
  HeadRows q, k, v;
  char *q_out, *k_cache, *v_cache;
  long long q_out_row, q_out_head;
  CacheStrides cs;
  TargetRows rows;
  TargetSlots slots;
  Rotation rot;
  HeadNorm norm;
  int q_heads, parts;
  int* err;
};

constexpr int kMaxHalf = 128;            // pairs of a head (head_dim <= 256)

// Cosine and sine of position x frequency, which is reduced to a turn in whole numbers: the
// frequency's 24 bits times 2^64 / (2 pi), rounded to a whole number (half a unit for each unit of
// frequency), are cut off to whole 2^-64 turns (a unit), and the position's multiple wraps at
// whole turns by itself.  So a position is off by (frequency / 2 + 1) 2^-64 of a turn at most, and
// position 2^30 at frequencies up to 1 by 1.5 x 2^-34 before it is rounded to fp32 (an fp32 product
// would be off by some turns), without an instruction in 64-bit floating point: those take
// 100 cycles and more here, and five of them stood between a row's length and its stores.
__device__ __forceinline__ float2 turn_of(int position, float freq) {
  constexpr unsigned long long kTurns = 2935890503282001226ull;      // 2^64 / (2 pi)
  const uint32_t bits = __float_as_uint(freq);
  const int exponent = (int)(bits >> 23 & 255);
  const unsigned long long m = (unsigned long long)(exponent ? (bits & 0x7fffffu) | 0x800000u : (bits & 0x7fffffu) << 1) << 40;
  const unsigned long long hi = __umul64hi(m, kTurns), lo = m * kTurns;   // |freq| = m 2^(exponent - 190)
  const int up = exponent - 126;                                     // turns x 2^64 = (hi:lo >> 64) 2^up
  unsigned long long turns = up <= -64 || up >= 128 ? 0 : up < 0 ? hi >> -up : up == 0 ? hi
                           : up < 64 ? hi << up | lo >> (64 - up) : lo << (up - 64);
  turns *= (unsigned long long)(long long)position;
  if (bits >> 31) turns = 0 - turns;
  float2 cs;
  sincospif((float)(long long)turns * 0x1p-63f, &cs.y, &cs.x);
  if (exponent == 255) cs.x = cs.y = __int_as_float(0x7fc00000);     // of no angle
  return cs;
}

// The last of the B requests whose rows start at or before `row`, 32 looked at at once by the
// warp; -1: none does.
__device__ __forceinline__ int request_of_row(const int32_t* starts, int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, end = B;
  while (end - lo > 32) {
    const int step = (end - lo + 31) / 32, at = lo + lane * step;
    const int before = __popc(__ballot_sync(0xffffffffu, at < end && starts[at < end ? at : lo] <= row));
    if (before == 0) return -1;
    lo += (before - 1) * step;
    end = min(lo + step, end);
  }
  const int at = lo + lane;
  return lo - 1 + __popc(__ballot_sync(0xffffffffu, at < end && starts[at < end ? at : lo] <= row));
}

// A row's LG lanes a head vector (16 bytes a lane): x' = rot(x rsqrt(mean x^2 + eps) w), sums and
// products in fp32 and one rounding where it is stored.  Each element is read and written once, so
// memory bounds it.  A warp takes a row, or one of `parts` parts of its heads, and waits for no
// other: a lane has the same elements of each of its heads, so it holds their cosines and sines
// in registers, 1 to 4 of which each lane computes for the warp.
constexpr int kAppendWarps = 8, kAppendBatch = 4, kAppendCtas = 4, kAppendMost = 16;

template <typename T, int LG>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendCtas) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int G = 32 / LG;               // heads side by side
  __shared__ float2 turn_s[kAppendWarps][kMaxHalf];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane & (LG - 1), group = lane / LG;
  const long long task = (long long)blockIdx.x * kAppendWarps + warp;
  const long long place = task / p.parts;
  const int part = (int)(task - place * p.parts);
  int b;
  long long first_row;                     // of the request's token 0, as the starts have it
  if (p.rows.starts) {
    // a place is a row: it finds its request, and one for each request checks what is said of that
    if (place < p.rows.B && part == 0 && lane == 0) {
      const RequestRows r = request_rows(p.rows, (int)place, p.err);
      if (r.n > 0) request_length(p.slots, (int)place, r.n, p.err);
    }
    if (place >= p.rows.rows) return;
    b = request_of_row(p.rows.starts, p.rows.B, (int)place);
    if (b < 0) return;
    first_row = p.rows.starts[b];
  } else {
    b = (int)(place / p.rows.N);
    first_row = (long long)b * p.rows.N;
  }
  if (b >= p.rows.B) return;
  const int length = p.slots.lengths[b];
  const RequestRows r = request_rows(p.rows, b, p.err);
  // (starts that descend may find a request that begins behind the row)
  if (place < first_row || place - first_row >= r.n) return;
  const int i = (int)(place - first_row);
  const int len = checked_length(p.slots, length, r.n, p.err);
  if (len < 0) return;
  const int row = r.row0 + i, slot = len + i;
  const int D = p.cs.head_dim, half = p.rot.inv_freq ? p.rot.rotated / 2 : 0;
  const bool on = at * 8 < D;
  const int n_q = p.q_heads, n_qk = n_q + p.cs.heads, step = p.parts * G;
  const T* q = static_cast<const T*>(p.q.p) + row * p.q.row + at * 8;
  const T* k = static_cast<const T*>(p.k.p) + row * p.k.row + at * 8;
  auto load = [&](int first, uint4 (&x)[kAppendBatch]) {
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u) {
      const int vec = first + u * step + group;
      x[u] = make_uint4(0, 0, 0, 0);
      if (vec < n_qk && on)
        x[u] = *reinterpret_cast<const uint4*>(vec < n_q ? q + vec * p.q.head : k + (vec - n_q) * p.k.head);
    }
  };
  uint4 x[kAppendBatch];
  load(part * G, x);
  const int page = slot_page(p.slots, b, slot, p.err);

  // ---- the angles of this lane's elements
  float c[8], s[8];
  const int h8 = half / 8;                 // (half a multiple of 8: pairs are whole chunks apart)
  const bool low = at < h8, rotated = at < 2 * h8;
  if (half) {
    int depth = i;
    if (p.rows.parents) {
      // a tree has at most 64 tokens: the warp holds their parents, two a lane
      const int a = lane < r.n ? parent_of(p.rows.parents, r.row0 + lane, lane, p.err) : -1;
      const int d = lane + 32 < r.n ? parent_of(p.rows.parents, r.row0 + lane + 32, lane + 32, p.err) : -1;
      depth = -1;
      for (int up = i; up >= 0; ++depth) {
        const int lo = __shfl_sync(0xffffffffu, a, up & 31), hi = __shfl_sync(0xffffffffu, d, up & 31);
        up = up < 32 ? lo : hi;
      }
    }
    for (int j = lane; j < half; j += 32) turn_s[warp][j] = turn_of(len + depth, p.rot.inv_freq[j]);
    __syncwarp();
    if (rotated) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 t = turn_s[warp][p.rot.interleaved ? at * 4 + e / 2 : (low ? at : at - h8) * 8 + e];
        c[e] = t.x;
        s[e] = (p.rot.interleaved ? !(e & 1) : low) ? -t.y : t.y;
      }
    }
  }
  const int other = !rotated ? at : low ? at + h8 : at - h8;

  T* q_out = reinterpret_cast<T*>(p.q_out) + row * p.q_out_row + at * 8;
  const long long line = page < 0 ? 0 : page * p.cs.page + (slot & ((1 << p.slots.page_shift) - 1)) * p.cs.slot;
  T* k_cache = reinterpret_cast<T*>(p.k_cache) + line + at * 8;
  const bool norm = p.norm.q_weight || p.norm.k_weight;
  for (int first = part * G; first < n_qk; first += kAppendBatch * step) {
    if (first != part * G) load(first, x);
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u) {
      const int vec = first + u * step + group;
      if (vec - group >= n_qk) break;      // (the same for every lane)
      const bool is_q = vec < n_q;
      const float* weight = is_q ? p.norm.q_weight : p.norm.k_weight;
      uint4 y = x[u];
      if (norm || half) {                  // (what is neither normalised nor rotated passes as its bits)
        float f[8];
        unpack_chunk<T>(x[u], f);
        if (norm) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(f[e], f[e], sum);
#pragma unroll
          for (int m = LG / 2; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
          if (weight && on) {
            const float scale = 1.f / sqrtf(sum / (float)D + p.norm.eps);
            const float4 w0 = reinterpret_cast<const float4*>(weight)[2 * at], w1 = reinterpret_cast<const float4*>(weight)[2 * at + 1];
            const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * scale * wv[e];
          }
        }
        if (half) {
          float g[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            g[e] = p.rot.interleaved ? f[e ^ 1] : __shfl_sync(0xffffffffu, f[e], other, LG);
          if (rotated) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(f[e], c[e], g[e] * s[e]);
          }
        }
        if (weight || half) y = pack_chunk<T>(f);
      }
      if (!on || vec >= n_qk) continue;
      if (is_q) *reinterpret_cast<uint4*>(q_out + vec * p.q_out_head) = y;
      else if (page >= 0) *reinterpret_cast<uint4*>(k_cache + (vec - n_q) * p.cs.head) = y;
    }
  }
  // ---- values
  const T* v = static_cast<const T*>(p.v.p) + row * p.v.row + at * 8;
  T* v_cache = reinterpret_cast<T*>(p.v_cache) + line + at * 8;
  if (page < 0 || !on) return;
  for (int first = (p.parts - 1 - part) * G + group; first < p.cs.heads; first += kAppendBatch * step) {
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u)
      if (first + u * step < p.cs.heads) x[u] = *reinterpret_cast<const uint4*>(v + (first + u * step) * p.v.head);
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u)
      if (first + u * step < p.cs.heads) *reinterpret_cast<uint4*>(v_cache + (first + u * step) * p.cs.head) = x[u];
  }
}

template <typename T>
cudaError_t append_for(AppendParams p, cudaStream_t stream) {
  const int chunks = p.cs.head_dim / 8;
  int lg = 2;
  while (lg < chunks) lg *= 2;
  static std::atomic<int> cache[kMaxCachedDevices];
  const int sms = per_device_grid(cache, []() { return 1; });
  if (sms <= 0) return cudaErrorInvalidConfiguration;
  // as many warps as the device holds, none without a head and none with more than 16 head
  // vectors: a row alone takes 3.4 us in 20 parts and 5.3 in 3; 12,004 rows of 9 KB take 47.5 us in one
  // part each (69% of the copy bandwidth), 50 and 55 in two and four, 62 with a fifth CTA an SM, whose
  // registers do not suffice; 2500 places of 40 heads of 256 45 us in one part each and 24 in three
  const long long places = !p.rows.starts ? (long long)p.rows.N * p.rows.B
                         : p.rows.rows > p.rows.B ? p.rows.rows : p.rows.B;
  const int most = cdiv(p.q_heads + p.cs.heads, 32 / lg);
  const long long wanted = (long long)sms * kAppendCtas * kAppendWarps / places;
  const int least = cdiv(most, kAppendMost);
  p.parts = wanted < least ? least : wanted < most ? (int)wanted : most;
  const long long ctas = (places * p.parts + kAppendWarps - 1) / kAppendWarps;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)ctas), dim3(32 * kAppendWarps), 0, stream, p);
  };
  switch (lg) {
    case 2: return go(append_kernel<T, 2>);
    case 4: return go(append_kernel<T, 4>);
    case 8: return go(append_kernel<T, 8>);
    case 16: return go(append_kernel<T, 16>);
    default: return go(append_kernel<T, 32>);
  }
}

// ------------------------------------------------------------------------ keeping
struct KeepParams {
  uint4 *k, *v;                          // 8 elements each
  CacheStrides cs;                       // strides in 16-byte chunks here
  TargetSlots slots;
  const int32_t *path, *accept_len;
  int N;
  int* err;
};

// Accepted token j of a request moves from slot len + path[j] to len + 1 + j.  path[j] > j (a
// node comes after its ancestors), so a target lies before every source that is still to be
// read, and a batch's loads may all go before its stores.  One CTA a request, layer and side;
// the bytes moved bound it, and for a few requests the chain of dependent loads (length, path,
// page, line).
__global__ void __launch_bounds__(256) keep_kernel(const __grid_constant__ KeepParams p) {
  constexpr int kBatch = 8;
  __shared__ long long source_s[kMaxTree], target_s[kMaxTree];
  __shared__ int moves_s;
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, layer = blockIdx.x >> 1, tid = threadIdx.x;
  if (tid < 32) {
    const int a = p.accept_len[b], length = p.slots.lengths[b];
    int moves = 0;
    if (a < 0 || a > p.N - 1) {
      set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
    } else if (a > 0 && checked_length(p.slots, length, 1 + a, p.err) >= 0) {
      // (a request of which nothing is kept may have its pages full)
      const int len = length;
      for (int j0 = 0; j0 < a; j0 += 32) {
        const int j = j0 + tid;
        long long from = -1, to = -1;
        if (j < a) {
          const int node = p.path[(long long)b * p.N + j];
          const long long last = ((long long)p.slots.max_pages << p.slots.page_shift) - 1;
          if (node <= j || node >= p.N || (long long)len + node > last) {
            set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
          } else if (node != j + 1) {
            const int mask = (1 << p.slots.page_shift) - 1;
            const int s0 = len + node, s1 = len + 1 + j;
            const int g0 = slot_page(p.slots, b, s0, p.err), g1 = slot_page(p.slots, b, s1, p.err);
            if (g0 >= 0 && g1 >= 0) {
              from = g0 * p.cs.page + (s0 & mask) * p.cs.slot;
              to = g1 * p.cs.page + (s1 & mask) * p.cs.slot;
            }
          }
        }
        const unsigned on = __ballot_sync(0xffffffffu, from >= 0);
        const int at = moves + __popc(on & ((1u << tid) - 1));
        if (from >= 0) {
          source_s[at] = from;
          target_s[at] = to;
        }
        moves += __popc(on);
      }
    }
    if (tid == 0) moves_s = moves;
  }
  __syncthreads();
  const int moves = moves_s, chunks = p.cs.head_dim / 8, width = p.cs.heads * chunks;
  uint4* base = (blockIdx.x & 1 ? p.v : p.k) + layer * p.cs.layer;
  for (int c = tid; c < width; c += blockDim.x) {
    uint4* at = base + (c / chunks) * p.cs.head + c % chunks;
    for (int j0 = 0; j0 < moves; j0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (j0 + u < moves) x[u] = at[source_s[j0 + u]];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (j0 + u < moves) at[target_s[j0 + u]] = x[u];
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const HeadRows& q, const HeadRows& k, const HeadRows& v, int q_heads, void* q_out,
                                long long q_out_row, long long q_out_head, void* k_cache, void* v_cache,
                                const CacheStrides& cs, int dtype, const TargetRows& rows, const TargetSlots& slots,
                                const Rotation& rot, const HeadNorm& norm, int* err, cudaStream_t stream) {
  AppendParams p = {q, k, v, static_cast<char*>(q_out), static_cast<char*>(k_cache), static_cast<char*>(v_cache),
                    q_out_row, q_out_head, cs, rows, slots, rot, norm, q_heads, 1, err};
  return dtype == DSPARK_BF16 ? append_for<__nv_bfloat16>(p, stream) : append_for<__half>(p, stream);
}

cudaError_t launch_cache_keep(void* k_cache, void* v_cache, const CacheStrides& cs, const TargetSlots& slots, int B,
                              int N, const int32_t* path, const int32_t* accept_len, int* err,
                              cudaStream_t stream) {
  KeepParams p = {static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), cs, slots, path, accept_len, N, err};
  p.cs.page /= 8;
  p.cs.slot /= 8;
  p.cs.head /= 8;
  p.cs.layer /= 8;
  int threads = cdiv((long long)cs.heads * cs.head_dim / 8, 32) * 32;
  if (threads > 256) threads = 256;
  return launch_pdl(keep_kernel, dim3(2u * (unsigned)cs.layers, (unsigned)B), dim3(threads), 0, stream, p);
}

}  // namespace dspark
