// Shared device helpers of the operators that read a [T, V] logits matrix: element
// types, a row seen as 16-byte vectors whatever its address, block reductions in a
// fixed order, and 2^x to about 2^-33 in 32-bit operations.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "tim_common.cuh"

namespace tim {

// ---------------------------------------------------------------------------
// Element types
template <int kDtype>
struct Elem;

template <>
struct Elem<TIM_F32> {
  using raw = float;
  static constexpr int kVec = 4;  // elements of a 16-byte vector
  static __device__ __forceinline__ float widen(raw x) { return x; }
  static __device__ __forceinline__ raw narrow(float x) { return x; }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};

template <>
struct Elem<TIM_BF16> {
  using raw = __nv_bfloat16;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float widen(raw x) { return __bfloat162float(x); }
  static __device__ __forceinline__ raw narrow(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Elem<TIM_F16> {
  using raw = __half;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float widen(raw x) { return __half2float(x); }
  static __device__ __forceinline__ raw narrow(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// ---------------------------------------------------------------------------
// A row of V elements as 16-byte vectors.  Rows may start at any multiple of the
// element size (odd V, a padded stride), so the vectors are those of the aligned
// addresses: element i of the row is slot i + shift, vector j holds the slots
// j kVec .. j kVec + kVec - 1, and only the first and the last vector can hold slots
// that are not the row's.  Those two are read and written element by element, so no
// byte outside the row is touched.
template <int kDtype>
struct Row {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  const raw* p;  // first element
  int shift;     // slots before it in its 16-byte vector
  int V;

  __device__ __forceinline__ Row(const void* base, int64_t row, int64_t ld, int V_)
      : p(static_cast<const raw*>(base) + row * ld), V(V_) {
    shift = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(raw));
  }
  __device__ __forceinline__ int nvec() const { return (shift + V + E::kVec - 1) / E::kVec; }
  __device__ __forceinline__ bool whole(int j) const {
    return j * E::kVec >= shift && (j + 1) * E::kVec <= shift + V;
  }
  // the raw vector j; slots outside the row read as -inf
  __device__ __forceinline__ uint4 load(int j) const {
    const raw* q = p - shift + static_cast<int64_t>(j) * E::kVec;
    if (whole(j)) return __ldg(reinterpret_cast<const uint4*>(q));
    return load_edge(j);
  }
  __device__ __noinline__ uint4 load_edge(int j) const {
    const raw* q = p - shift + static_cast<int64_t>(j) * E::kVec;
    float v[E::kVec];
#pragma unroll
    for (int i = 0; i < E::kVec; ++i) {
      const int s = j * E::kVec + i - shift;
      v[i] = (s >= 0 && s < V) ? E::widen(q[i]) : -INFINITY;
    }
    return E::pack(v);
  }
  __device__ __forceinline__ float at(int i) const { return E::widen(p[i]); }
  // vector j itself, and the vectors w0 <= j < w1 that are whole
  __device__ __forceinline__ const uint4* vec() const {
    return reinterpret_cast<const uint4*>(p - shift);
  }
  __device__ __forceinline__ int w0() const { return shift != 0 ? 1 : 0; }
  __device__ __forceinline__ int w1() const { return (shift + V) / E::kVec; }
};

// Lets a kernel use `bytes` of dynamic shared memory, once a device: `done` has a bit for each.
template <class Kernel>
inline cudaError_t allow_smem(Kernel* kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---------------------------------------------------------------------------
// Two fp32 operations in one instruction.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 ex2x2(F2 a) {
  const float2 t = unpack2(a);
  return f2(ex2_approx(t.x), ex2_approx(t.y));
}

// ---------------------------------------------------------------------------
// A row over a cluster of CTAs.  Each CTA holds one contiguous slice of the row's vectors in
// shared memory, brought there by one asynchronous bulk copy, so a row is read from memory
// once whatever is done with it.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* smem, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(smem)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

__device__ __forceinline__ void cluster_store32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The slice of CTA `rank` of `size`: vectors j0 .. j0 + n - 1 of the row.
struct Slice {
  int j0, n;
};
__device__ __forceinline__ Slice slice_of(int nvec, int rank, int size) {
  const int per = (nvec + size - 1) / size;
  const int j0 = min(nvec, rank * per);
  return Slice{j0, min(nvec, j0 + per) - j0};
}

// Starts the slice's copy into `dst` (called by one thread; `bar` counts one arrival).  The
// row's first and last vectors may hold bytes that are not the row's: those are left to
// load_slice_edges.
template <int kDtype>
__device__ __forceinline__ void load_slice(const Row<kDtype>& r, const Slice& s, uint4* dst,
                                           uint64_t* bar) {
  int a = s.j0, b = s.j0 + s.n;
  if (a < b && !r.whole(a)) ++a;
  if (a < b && !r.whole(b - 1)) --b;
  const uint32_t bytes = static_cast<uint32_t>(b - a) * 16u;
  mbar_arrive_expect_tx(bar, bytes);
  if (bytes != 0)
    bulk_load(dst + (a - s.j0), r.p - r.shift + static_cast<int64_t>(a) * Elem<kDtype>::kVec,
              bytes, bar);
}
template <int kDtype>
__device__ __forceinline__ void load_slice_edges(const Row<kDtype>& r, const Slice& s, uint4* dst) {
  if (threadIdx.x < 2 && s.n > 0) {
    const int j = threadIdx.x == 0 ? s.j0 : s.j0 + s.n - 1;
    if (!r.whole(j)) dst[j - s.j0] = r.load_edge(j);
  }
}

// How a row of V elements is spread: CTAs a row and threads a CTA, from the size of a row alone,
// so that a row is split the same way in every batch.
struct RowPlan {
  int cluster, threads;
  uint32_t slice_bytes;
};
inline RowPlan plan_row(int V, int elem_bytes) {
  const int64_t vecs = (static_cast<int64_t>(V) * elem_bytes + 15) / 16 + 1;
  RowPlan p;
  p.cluster = 1;
  while (p.cluster < 8 && (vecs + p.cluster - 1) / p.cluster * 16 > 40960) p.cluster *= 2;
  const int64_t per = (vecs + p.cluster - 1) / p.cluster;
  p.slice_bytes = static_cast<uint32_t>(per * 16);
  p.threads = p.slice_bytes > 40960 ? 512 : 256;
  return p;
}

// T rows, a cluster of `cluster` CTAs each.
template <class Args>
inline cudaError_t launch_clusters(void (*kernel)(const Args), int64_t T, int cluster, int threads,
                                   size_t smem, cudaStream_t stream, const Args& a) {
  if (T * cluster > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T * cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ---------------------------------------------------------------------------
// Pairs of floats (value h + l, |l| at most half a step of h): about 2^-45.  A row's few
// scalars are computed in these: the fp64 units of this part are so few that a hundred fp64
// operations a row cost more than streaming the row.
struct Df {
  float h, l;
};
__device__ __forceinline__ Df two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Df quick_two_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Df two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
// An infinite or NaN h stays what it is.
__device__ __forceinline__ Df renorm(float h, float l) {
  const Df r = quick_two_sum(h, l);
  return fabsf(r.h) < INFINITY ? r : Df{r.h, 0.f};
}
__device__ __forceinline__ Df df(float a) { return {a, 0.f}; }
__device__ __forceinline__ Df operator-(Df a) { return {-a.h, -a.l}; }
__device__ __forceinline__ Df operator+(Df a, Df b) {
  const Df s = two_sum(a.h, b.h);
  return fabsf(s.h) < INFINITY ? renorm(s.h, s.l + (a.l + b.l)) : Df{s.h, 0.f};
}
__device__ __forceinline__ Df operator-(Df a, Df b) { return a + (-b); }
__device__ __forceinline__ Df operator*(Df a, Df b) {
  const Df p = two_prod(a.h, b.h);
  return fabsf(p.h) < INFINITY ? renorm(p.h, fmaf(a.h, b.l, fmaf(a.l, b.h, p.l))) : Df{p.h, 0.f};
}
__device__ __forceinline__ Df reciprocal(Df a) {
  const float r = 1.f / a.h;
  return renorm(r, r * fmaf(-r, a.l, fmaf(-r, a.h, 1.f)));
}

// ---------------------------------------------------------------------------
// 2^x in fixed point.
//
// x = z * K with K = Kh + Kl (a float and its remainder) is split at the multiple of 1/256
// next to z Kh (the sum with a number whose last place is 1/256) into n + j/256 + g, where
// one multiply-add gives z Kh less that multiple with one rounding, |g| <= 2^-9, and
//   2^x = 2^n * T[j] * (1 + p),  p = 2^g - 1 = g ln2 + g^2 ln2^2/2 + g^3 ln2^3/6
// (the next term is below 2^-41).  T is a table at scale 2^62 and p is taken at scale
// 2^32, so T[j] (1 + p) is one 32 x 32 -> 64-bit multiply-add.  The largest error is the
// rounding of p in 32 bits, about 2^-33.  Sums of such numbers are sums of integers: they
// do not depend on any order.
struct Pow2Table {
  unsigned long long t[256];
};

// floor(sqrt(x)) of a 128-bit number, bit by bit
constexpr unsigned long long isqrt128(unsigned __int128 x) {
  unsigned long long r = 0;
  for (int b = 63; b >= 0; --b) {
    const unsigned long long c = r | (1ull << b);
    if (static_cast<unsigned __int128>(c) * c <= x) r = c;
  }
  return r;
}

// 2^(j/256) at scale 2^62: products of the square roots 2^(1/2), 2^(1/4), ..., 2^(1/256)
constexpr Pow2Table make_pow2_table() {
  unsigned long long root[8] = {};
  unsigned long long r = 1ull << 63;  // 2 at scale 2^62
  for (int i = 0; i < 8; ++i) {
    r = isqrt128(static_cast<unsigned __int128>(r) << 62);
    root[i] = r;
  }
  Pow2Table T = {};
  for (int j = 0; j < 256; ++j) {
    unsigned __int128 v = static_cast<unsigned __int128>(1) << 62;
    for (int i = 0; i < 8; ++i)
      if (j & (128 >> i)) v = (v * root[i] + (static_cast<unsigned __int128>(1) << 61)) >> 62;
    T.t[j] = static_cast<unsigned long long>(v);
  }
  return T;
}

// What a row's logits are raised with: 2^((z - c) K), where c is subtracted only if `recentre`.
struct Pow2Row {
  float kh, kl;  // K = log2(e) / temperature
  float c;
  bool recentre;
};

constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596299e-8f;  // log2(e) as a pair
constexpr float kLn2Hi = 0.693147182f, kLn2Lo = -1.90465421e-9f;    // ln 2 as a pair

// w and n with 2^((z - c) K) = w 2^(n - 62).  |(z - c) K| must be below 2^14.
constexpr float kPow2Magic = 49152.f;  // 1.5 * 2^15: a sum's last place is 1/256
__device__ __forceinline__ unsigned long long pow2_fixed(float z, const Pow2Row& k,
                                                         const unsigned long long* table, int& n) {
  float t, g;
  if (k.recentre) {
    // z - c = d + e exactly
    const float d = z - k.c, b = d - z;
    const float e = (z - (d - b)) + (-k.c - b);
    t = fmaf(d, k.kh, kPow2Magic);
    g = fmaf(e, k.kh, fmaf(d, k.kl, fmaf(d, k.kh, kPow2Magic - t)));
  } else {
    t = fmaf(z, k.kh, kPow2Magic);
    g = fmaf(z, k.kl, fmaf(z, k.kh, kPow2Magic - t));
  }
  const int ti = __float_as_int(t) - __float_as_int(kPow2Magic);
  // p at scale 2^32
  const float p = g * fmaf(g, fmaf(g, 238388336.0f, 1031764992.0f), 2977044472.0f);
  const unsigned long long T = table[ti & 255];
  n = ti >> 8;
  return T + static_cast<unsigned long long>(static_cast<long long>(static_cast<int>(T >> 32)) *
                                             __float2int_rn(p));
}
// The table, one copy a translation unit.
static __device__ const Pow2Table g_pow2_table = make_pow2_table();

// 2^((z - c) K) as a pair of floats; 0 below 2^-126, so that the caller need not care about
// pow2_fixed's range.  (z - c) K must be at most 100.
__device__ __forceinline__ Df pow2_df(float z, const Pow2Row& k,
                                      const unsigned long long* table = g_pow2_table.t) {
  const float x = (k.recentre ? z - k.c : z) * k.kh;
  if (!(x > -126.f)) return {x <= -126.f ? 0.f : __int_as_float(0x7FC00000), 0.f};  // NaN stays
  int n;
  const unsigned long long w = pow2_fixed(z, k, table, n);
  // the top 48 of w's 62 or 63 bits, 24 in each part
  const float scale = __int_as_float((n + 127) << 23);
  const float h = static_cast<float>(static_cast<uint32_t>(w >> 39)) * (scale * 0x1p-23f);
  const float l = static_cast<float>(static_cast<uint32_t>(w >> 15) & 0xFFFFFFu) * (scale * 0x1p-47f);
  return renorm(h, l);
}

// e^x
__device__ __forceinline__ Df exp_df(float x, const unsigned long long* table = g_pow2_table.t) {
  return pow2_df(x, Pow2Row{kLog2eHi, kLog2eLo, 0.f, false}, table);
}

// ln a for 2^-126 <= a < 2^127: l = ln of the leading bits in fp32, then
// ln a = l + ln(a e^-l) with the small second term from its series.
__device__ __forceinline__ Df log_df(Df a, const unsigned long long* table = g_pow2_table.t) {
  const int e = static_cast<int>(__float_as_uint(a.h) >> 23) - 127;
  const float s = __int_as_float((127 - e) << 23);
  const Df f = {a.h * s, a.l * s};
  const float l = __logf(f.h);
  const Df r = f * exp_df(-l, table) - df(1.f);
  const Df ln = df(l) + renorm(r.h, r.l - 0.5f * r.h * r.h);
  return Df{kLn2Hi, kLn2Lo} * df(static_cast<float>(e)) + ln;
}

}  // namespace tim
