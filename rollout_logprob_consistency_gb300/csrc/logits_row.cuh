// Shared device helpers of the operators that read a [T, V] logits matrix: element
// types, a row seen as 16-byte vectors whatever its address, block reductions in a
// fixed order, and 2^x to about 2^-33 in 32-bit operations.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
};

// ---------------------------------------------------------------------------
// 2^x in fixed point.
//
// x = z * K with K = Kh + Kl (a float and its remainder).  z * Kh is taken exactly as
// ph + pl; ph is split at multiples of 1/256 into n + j/256 + g, |g| <= 2^-9 plus the
// small pl, and
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

constexpr int kPow2Bits = 8;

// What a row's logits are raised with: 2^((z - c) K), c = 0 or the row's largest logit.
struct Pow2Row {
  float kh, kl;   // K = log2(e) / temperature
  float c;        // subtracted first when `recentre`
  int recentre;   // |max K| is too large for the split of z K itself
};

__device__ __forceinline__ Pow2Row pow2_row(float temperature, float zmax) {
  const double K = 1.4426950408889634 / static_cast<double>(temperature);
  Pow2Row r;
  r.kh = static_cast<float>(K);
  r.kl = static_cast<float>(K - static_cast<double>(r.kh));
  r.recentre = !(fabs(static_cast<double>(zmax) * K) < 8192.0);
  r.c = r.recentre ? zmax : 0.f;
  return r;
}

// w and n with 2^((z - c) K) = w 2^(n - 62).  |(z - c) K| must be below 2^14.
__device__ __forceinline__ unsigned long long pow2_fixed(float z, const Pow2Row& k,
                                                         const unsigned long long* table, int& n) {
  constexpr float kMagic = 49152.f;  // 1.5 * 2^15: the sum's last place is 1/256
  float ph, pl;
  if (k.recentre) {
    // z - c = d + e exactly
    const float d = z - k.c, b = d - z;
    const float e = (z - (d - b)) + (-k.c - b);
    ph = d * k.kh;
    pl = fmaf(e, k.kh, fmaf(d, k.kl, fmaf(d, k.kh, -ph)));
  } else {
    ph = z * k.kh;
    pl = fmaf(z, k.kl, fmaf(z, k.kh, -ph));
  }
  const float t = ph + kMagic;
  const float g = (ph - (t - kMagic)) + pl;
  const int ti = __float_as_int(t) - __float_as_int(kMagic);
  // p at scale 2^32
  const float p = g * fmaf(g, fmaf(g, 238388336.0f, 1031764992.0f), 2977044472.0f);
  const unsigned long long T = table[ti & 255];
  n = ti >> kPow2Bits;
  return T + static_cast<unsigned long long>(static_cast<long long>(static_cast<int>(T >> 32)) *
                                             __float2int_rn(p));
}

// The same as a double, for x above -900.
__device__ __forceinline__ double pow2_double(float z, const Pow2Row& k,
                                              const unsigned long long* table) {
  int n;
  const unsigned long long w = pow2_fixed(z, k, table, n);
  return static_cast<double>(w) * __longlong_as_double(static_cast<long long>(n - 62 + 1023) << 52);
}

// The table, one copy a translation unit.
static __device__ const Pow2Table g_pow2_table = make_pow2_table();

}  // namespace tim
