// Device helpers of the kernels that stream rows of logits or of a table in 32, bf16 or
// fp16 bits: 16-byte chunks unpacked to fp32, packed two-wide fp32 arithmetic, the chunk
// layout of a row that may start off a 16-byte border, thread-block-cluster barriers
// with reads and messages between CTAs' shared memory, and running softmax sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <stdint.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace dspark {

// ---------------------------------------------------------------------- element types
template <typename T>
struct Chunk {
  static constexpr int N = 16 / (int)sizeof(T);      // elements of a 16-byte chunk
};

__device__ __forceinline__ float elem_to_float(float x) { return x; }
__device__ __forceinline__ float elem_to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float elem_to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T elem_from_float(float x);
template <>
__device__ __forceinline__ float elem_from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 elem_from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half elem_from_float<__half>(float x) { return __float2half_rn(x); }

__device__ __forceinline__ void unpack(const uint4& q, float (&v)[4], float*) {
  v[0] = __uint_as_float(q.x);
  v[1] = __uint_as_float(q.y);
  v[2] = __uint_as_float(q.z);
  v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8], __nv_bfloat16*) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8], __half*) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ void unpack_chunk(const uint4& q, float (&v)[Chunk<T>::N]) {
  unpack(q, v, static_cast<T*>(nullptr));
}

// one rounding to nearest even per element (none for fp32)
__device__ __forceinline__ uint4 pack(const float (&v)[4], float*) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[8], __nv_bfloat16*) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&v)[8], __half*) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ uint4 pack_chunk(const float (&v)[Chunk<T>::N]) {
  return pack(v, static_cast<T*>(nullptr));
}

// --------------------------------------------------------- two fp32 lanes per instruction
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(F2 a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// A row of V elements as `head` single elements up to the first 16-byte border, `chunks`
// whole 16-byte chunks, and `tail` single elements.
struct RowChunks {
  int head, chunks, tail;
};
template <typename T>
__device__ __forceinline__ RowChunks row_chunks(const T* row, int V) {
  constexpr int N = Chunk<T>::N;
  RowChunks c;
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
  c.head = off ? (int)((16u - off) / sizeof(T)) : 0;
  if (c.head > V) c.head = V;
  c.chunks = (V - c.head) / N;
  c.tail = V - c.head - c.chunks * N;
  return c;
}

// ------------------------------------------------------------------------- clusters
// every CTA of the cluster arrives, then waits; orders shared-memory accesses between CTAs
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(const void* smem, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "r"(rank));
  return a;
}
__device__ __forceinline__ unsigned long long cluster_ld_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// the largest of the warp's values that are not NaN
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// the largest of n elements that are not NaN
template <int n>
__device__ __forceinline__ float max_of(const float (&z)[n]) {
  float m[n];
#pragma unroll
  for (int i = 0; i < n; ++i) m[i] = z[i];
#pragma unroll
  for (int w = 1; w < n; w *= 2)
#pragma unroll
    for (int i = 0; i + w < n; i += 2 * w) m[i] = fmaxf(m[i], m[i + w]);
  return m[0];
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// ---------------------------------------------------------------- copies and messages
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          sm100::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
      : "memory");
}
// stores into CTA `rank`'s copy of *dst, counted in bytes by its copy of *bar
__device__ __forceinline__ void send_f2(float2* dst, uint64_t* bar, uint32_t rank, float x, float y) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                   cluster_map(dst, rank)),
               "f"(x), "f"(y), "r"(cluster_map(bar, rank))
               : "memory");
}
__device__ __forceinline__ void send_f(float* dst, uint64_t* bar, uint32_t rank, float x) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                   cluster_map(dst, rank)),
               "r"(__float_as_uint(x)), "r"(cluster_map(bar, rank))
               : "memory");
}
__device__ __forceinline__ void send_u64(unsigned long long* dst, uint64_t* bar, uint32_t rank,
                                         unsigned long long x) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                   cluster_map(dst, rank)),
               "l"(x), "r"(cluster_map(bar, rank))
               : "memory");
}
// a wait on data that other CTAs of the cluster send
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity) {
  const long long t0 = sm100::sm_cycles();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(sm100::smem_u32(bar)), "r"(parity), "r"(10000000u)
        : "memory");
    if (ok) return true;
    if (sm100::sm_cycles() - t0 > sm100::kWaitCycles) return false;
  }
}

template <typename T>
struct RowPart {             // a CTA's part [c0, c1) of a row's chunks, `held` of them kept
  const T* row;
  const uint4* body;
  RowChunks rc;
  int c0, c1, held;
};
template <typename T>
__device__ __forceinline__ RowPart<T> row_part(const void* z, long long ld, int n, int V, int c, int log_C,
                                               int most) {
  RowPart<T> r;
  r.row = static_cast<const T*>(z) + (long long)n * ld;
  r.rc = row_chunks(r.row, V);
  r.body = reinterpret_cast<const uint4*>(r.row + r.rc.head);
  r.c0 = (int)((long long)r.rc.chunks * c >> log_C);
  r.c1 = (int)((long long)r.rc.chunks * (c + 1) >> log_C);
  r.held = min(r.c1 - r.c0, most);
  return r;
}

// ------------------------------------------------------------- running softmax statistics
// s = sum exp(z - R) and t = sum exp(z - R) (z - R) over the elements seen, against a
// reference R that a batch raises to its own maximum only when it exceeds R by more than
// kMargin: sums stay below V e^8, and the rescale is rare.  Elements of -inf contribute
// nothing; NaN and +inf make s NaN.
constexpr float kMargin = 8.f;

struct RunningSoftmax {
  float R;
  F2 s, t;
  __device__ __forceinline__ void init() {
    R = -FLT_MAX;
    s = f2(0.f, 0.f);
    t = f2(0.f, 0.f);
  }
  // n (even) elements; bm: their maximum (NaN ignored)
  template <int n>
  __device__ __forceinline__ void add(const float (&z)[n], float bm) {
    if (bm - R > kMargin) {                  // also the first batch: R = -FLT_MAX
      const float d = R - bm;                // < 0, may be -inf (then s = t = 0)
      const float f = ex2_approx(d * kLog2e);
      float a, b, u, v;
      f2_get(s, a, b);
      f2_get(t, u, v);
      t = f > 0.f ? f2(f * (u + d * a), f * (v + d * b)) : f2(0.f, 0.f);
      s = f2(f * a, f * b);
      R = bm;
    }
    const F2 nR = f2(-R, -R), kk = f2(kLog2e, kLog2e);
    F2 tb = f2(0.f, 0.f);
    F2 sb[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      const F2 d = f2_add(f2(z[i], z[i + 1]), nR);
      float x, y;
      f2_get(f2_mul(d, kk), x, y);
      const F2 e = f2(ex2_approx(x), ex2_approx(y));
      sb[i / 2 & 1] = f2_add(sb[i / 2 & 1], e);
      tb = f2_fma(e, d, tb);
    }
    s = f2_add(s, f2_add(sb[0], sb[1]));
    float u, v;
    f2_get(tb, u, v);
    if (!(fabsf(u + v) <= FLT_MAX)) {        // an element of -inf: 0 * -inf
      u = 0.f;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float d = z[i] - R;
        if (d > -FLT_MAX) u = fmaf(ex2_approx(d * kLog2e), d, u);
      }
      tb = f2(u, 0.f);
    }
    t = f2_add(t, tb);
  }
  __device__ __forceinline__ void add_one(float z) {
    const float two[2] = {z, -INFINITY};
    add<2>(two, z == z ? z : R);
  }
  // the sums moved to the reference m >= R (m finite unless nothing was seen)
  __device__ __forceinline__ void finish(float m, float& so, float& to) const {
    float a, b, u, v;
    f2_get(s, a, b);
    f2_get(t, u, v);
    so = a + b;
    to = 0.f;
    if (so == 0.f) return;
    const float d = R - m;
    const float f = ex2_approx(d * kLog2e);
    to = f > 0.f ? f * ((u + v) + d * so) : 0.f;
    so *= f;
  }
};

// s = sum exp(k (z - R)) alone, without a maximum per element: R is raised (to a batch's
// maximum, which only then is looked for) when the sum leaves [2^-20, 2^14], which the first
// batch with an element above -inf does and after it only elements about 10 / k above R.  (A
// wider range would cost logarithms of the sum digits: they are taken relative to R.)
struct RunningSum {
  float R, k;
  F2 s;
  __device__ __forceinline__ void init(float inv_temperature) {
    R = -FLT_MAX;
    k = inv_temperature;
    s = f2(0.f, 0.f);
  }
  template <int n>
  __device__ __forceinline__ F2 batch(const float (&z)[n]) const {
    const F2 nR = f2(-R, -R), kk = f2(k * kLog2e, k * kLog2e);
    F2 sb[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      float x, y;
      f2_get(f2_mul(f2_add(f2(z[i], z[i + 1]), nR), kk), x, y);
      sb[i / 2 & 1] = f2_add(sb[i / 2 & 1], f2(ex2_approx(x), ex2_approx(y)));
    }
    return f2_add(sb[0], sb[1]);
  }
  template <int n>
  __device__ __forceinline__ void add(const float (&z)[n]) {
    F2 t = f2_add(s, batch<n>(z));
    float a, b;
    f2_get(t, a, b);
    if (!(a + b >= 0x1p-20f && a + b <= 0x1p14f)) {
      const float bm = max_of(z);
      float u, v;
      f2_get(s, u, v);
      if (bm > R || (u + v == 0.f && bm > -INFINITY)) {
        const float f = u + v == 0.f ? 0.f : ex2_approx((R - bm) * k * kLog2e);
        s = f2(f * u, f * v);
        R = bm;
      }
      t = f2_add(s, batch<n>(z));
    }
    s = t;
  }
  __device__ __forceinline__ void add_one(float z) {
    const float two[2] = {z, -INFINITY};
    add<2>(two);
  }
  // the reference of what was seen (-inf: nothing above -inf), and the sum moved to m >= it
  __device__ __forceinline__ float reference() const { return sum() == 0.f ? -INFINITY : R; }
  __device__ __forceinline__ float sum() const {
    float a, b;
    f2_get(s, a, b);
    return a + b;
  }
  __device__ __forceinline__ float at(float m) const {
    return sum() == 0.f ? 0.f : sum() * ex2_approx((R - m) * k * kLog2e);
  }
};

}  // namespace dspark
