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
  int q_heads;
  int* err;
};

constexpr int kMaxHalf = 128;            // pairs of a head (head_dim <= 256)

// Cosine and sine of position x frequency.  The product is formed and reduced by multiples of
// 2 pi (its double and the next 53 bits: Cody and Waite's two-term reduction) in 64 bits: at
// position 2^20 an fp32 product is off by up to 0.03, at 2^31 this one by 3e-7.
__device__ __forceinline__ float2 turn_of(int position, float freq) {
  const double angle = (double)position * (double)freq;
  const double turns = rint(angle * 0.15915494309189535);
  double r = fma(turns, -6.283185307179586, angle);
  r = fma(turns, -2.4492935982947064e-16, r);
  float2 cs;
  sincosf((float)r, &cs.y, &cs.x);
  return cs;
}

// One CTA a row, LG lanes a head vector (16 bytes a lane): x' = rot(x rsqrt(mean x^2 + eps) w),
// sums and products in fp32 and one rounding where it is stored.  Each element is read and
// written once, so memory bounds it; a row's loads are all issued before its angles are
// computed, once for all its heads.
template <typename T, int LG>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kBatch = 4;
  __shared__ float cos_s[kMaxHalf], sin_s[kMaxHalf];
  __shared__ int depth_s;
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, i = blockIdx.x, tid = threadIdx.x;
  const RequestRows r = request_rows(p.rows, b, p.err);
  if (i >= r.n) return;
  const int len = request_length(p.slots, b, r.n, p.err);
  if (len < 0) return;
  const int row = r.row0 + i, slot = len + i;
  const int D = p.cs.head_dim, lane = tid & (LG - 1), group = tid / LG, groups = blockDim.x / LG;
  const bool on = lane * 8 < D;
  const int n_vec = p.q_heads + 2 * p.cs.heads;
  auto source = [&](int vec) {
    const HeadRows& h = vec < p.q_heads ? p.q : vec < p.q_heads + p.cs.heads ? p.k : p.v;
    const int head = vec < p.q_heads ? vec : vec < p.q_heads + p.cs.heads ? vec - p.q_heads : vec - p.q_heads - p.cs.heads;
    return reinterpret_cast<const uint4*>(static_cast<const T*>(h.p) + row * h.row + head * h.head) + lane;
  };
  uint4 x[kBatch];
  auto load = [&](int first) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int vec = first + u * groups;
      if (vec < n_vec && on) x[u] = *source(vec);
    }
  };
  load(group);
  const int page = slot_page(p.slots, b, slot, p.err);
  const int half = p.rot.inv_freq ? p.rot.rotated / 2 : 0;
  if (half) {
    int depth = i;
    if (p.rows.parents) {
      // a tree has at most 64 tokens: the first warp holds its parents, two a lane
      if (tid < 32) {
        const int a = tid < r.n ? parent_of(p.rows.parents, r.row0 + tid, tid, p.err) : -1;
        const int c = tid + 32 < r.n ? parent_of(p.rows.parents, r.row0 + tid + 32, tid + 32, p.err) : -1;
        depth = -1;
        for (int at = i; at >= 0; ++depth) {
          const int lo = __shfl_sync(0xffffffffu, a, at & 31), hi = __shfl_sync(0xffffffffu, c, at & 31);
          at = at < 32 ? lo : hi;
        }
        if (tid == 0) depth_s = depth;
      }
      __syncthreads();
      depth = depth_s;
    }
    for (int j = tid; j < half; j += blockDim.x) {
      const float2 cs = turn_of(len + depth, p.rot.inv_freq[j]);
      cos_s[j] = cs.x;
      sin_s[j] = cs.y;
    }
    __syncthreads();
  }
  const long long line = page < 0 ? 0
      : page * p.cs.page + (slot & ((1 << p.slots.page_shift) - 1)) * p.cs.slot;
  for (int first = group; first - group < n_vec; first += kBatch * groups) {
    if (first != group) load(first);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int vec = first + u * groups;
      if (first - group + u * groups >= n_vec) break;      // (the same for every lane)
      const bool is_q = vec < p.q_heads, is_k = !is_q && vec < p.q_heads + p.cs.heads;
      const bool live = vec < n_vec && on;
      const float* w = is_q ? p.norm.q_weight : is_k ? p.norm.k_weight : nullptr;
      uint4 y = x[u];
      // (all lanes of a warp take part in the exchanges, whatever their vectors are)
      if (p.norm.q_weight || p.norm.k_weight || half) {
        float f[8];
        unpack_chunk<T>(live ? x[u] : make_uint4(0, 0, 0, 0), f);
        if (p.norm.q_weight || p.norm.k_weight) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(f[e], f[e], s);
#pragma unroll
          for (int m = LG / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
          if (w && live) {
            const float scale = 1.f / sqrtf(s / (float)D + p.norm.eps);
            const float4 w0 = reinterpret_cast<const float4*>(w)[2 * lane], w1 = reinterpret_cast<const float4*>(w)[2 * lane + 1];
            const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * scale * wv[e];
          }
        }
        if (half && p.rot.interleaved) {
          if ((is_q || is_k) && lane * 8 < 2 * half) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float c = cos_s[lane * 4 + e / 2], s = sin_s[lane * 4 + e / 2];
              const float a = f[e], d = f[e + 1];
              f[e] = a * c - d * s;
              f[e + 1] = d * c + a * s;
            }
          }
        } else if (half) {
          // pair j of element j and j + half, half a multiple of 8: whole chunks apart
          const int h8 = half / 8;
          const bool low = lane < h8, rotated = lane < 2 * h8;
          const int other = rotated ? (low ? lane + h8 : lane - h8) : lane;
          float g[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = __shfl_sync(0xffffffffu, f[e], other, LG);
          if ((is_q || is_k) && rotated) {
            const int j0 = (low ? lane : lane - h8) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float c = cos_s[j0 + e], s = sin_s[j0 + e];
              f[e] = low ? f[e] * c - g[e] * s : f[e] * c + g[e] * s;
            }
          }
        }
        // values, and what is neither normalised nor rotated, pass as their bits
        if ((is_q || is_k) && (w || half)) y = pack_chunk<T>(f);
      }
      if (!live) continue;
      if (is_q) {
        *(reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.q_out) + row * p.q_out_row + vec * p.q_out_head) + lane) = y;
      } else if (page >= 0) {
        const int head = vec - p.q_heads - (is_k ? 0 : p.cs.heads);
        T* cache = reinterpret_cast<T*>(is_k ? p.k_cache : p.v_cache);
        *(reinterpret_cast<uint4*>(cache + line + head * p.cs.head) + lane) = y;
      }
    }
  }
}

template <typename T>
cudaError_t append_for(const AppendParams& p, cudaStream_t stream) {
  const int chunks = p.cs.head_dim / 8;
  int lg = 2;
  while (lg < chunks) lg *= 2;
  const int n_vec = p.q_heads + 2 * p.cs.heads;
  int threads = cdiv((long long)n_vec * lg, 32) * 32;
  if (threads > 256) threads = 256;
  const dim3 grid((unsigned)p.rows.N, (unsigned)p.rows.B);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(threads), 0, stream, p); };
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
    const int a = p.accept_len[b], len = request_length(p.slots, b, 1, p.err);
    int moves = 0;
    if (a < 0 || a > p.N - 1) {
      set_device_error(p.err, DSPARK_ERR_DEVICE_CHECK);
    } else if (len >= 0) {
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
                    q_out_row, q_out_head, cs, rows, slots, rot, norm, q_heads, err};
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
