// What the two kernels of the sampler share: keys, the integer weights of a row and its scale,
// the settings of a row, and the results.
#pragma once

#include <cmath>

#include "logits_row.cuh"

namespace tim {
namespace sampling {

using u64 = unsigned long long;

struct SampleArgs {
  static constexpr bool kBorder = false;  // whether write_row uses a row's border
  const void* logits;
  int64_t ld;
  int V;
  const float* uniform;
  float temperature;
  int top_k;
  float top_p;
  float min_p;
  const float* row_temperature;
  const int32_t* row_top_k;
  const float* row_top_p;
  const float* row_min_p;
  int32_t* ids;
  float* logprob;
  float* lse;
  int32_t* kept;
  int* status;
};

// Monotone map of float bits to unsigned (larger float -> larger key; -0 and +0 are one).
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t f = __float_as_uint(z + 0.f);
  return (f & 0x80000000u) ? ~f : (f | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
constexpr uint32_t kNegInfKey = 0x007FFFFFu;  // key_of(-inf)

// Levels of 8 bits after which a key of the type is known: the bits below are its sign's.
template <int kDtype>
constexpr int kLevels = kDtype == TIM_F32 ? 4 : kDtype == TIM_F16 ? 3 : 2;

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Elementwise maximum of two vectors' elements, NaN if either is.
template <int kDtype>
__device__ __forceinline__ uint4 max_vec(uint4 a, const uint4& b) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  const uint32_t* y = reinterpret_cast<const uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == TIM_F32)
      asm("max.NaN.f32 %0, %0, %1;" : "+r"(x[i]) : "r"(y[i]));
    else if constexpr (kDtype == TIM_BF16)
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(y[i]));
    else
      asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(y[i]));
  }
  return a;
}
template <int kDtype>
__device__ __forceinline__ uint4 min_vec(uint4 a, const uint4& b) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  const uint32_t* y = reinterpret_cast<const uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == TIM_F32)
      asm("min.f32 %0, %0, %1;" : "+r"(x[i]) : "r"(y[i]));
    else if constexpr (kDtype == TIM_BF16)
      asm("min.bf16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(y[i]));
    else
      asm("min.f16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(y[i]));
  }
  return a;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int kDtype>
__device__ __forceinline__ uint4 neg_inf_vec() {
  const uint32_t w = kDtype == TIM_F32 ? 0xFF800000u : kDtype == TIM_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  return make_uint4(w, w, w, w);
}

// The largest element of a vector, NaN if any is.
template <int kDtype>
__device__ __forceinline__ float max_of(const uint4& u) {
  float v[Elem<kDtype>::kVec];
  Elem<kDtype>::unpack(u, v);
  float m = v[0];
#pragma unroll
  for (int i = 1; i < Elem<kDtype>::kVec; ++i) m = max_nan(m, v[i]);
  return m;
}

// The smallest, of none that is NaN.
template <int kDtype>
__device__ __forceinline__ float min_of(const uint4& u) {
  float v[Elem<kDtype>::kVec];
  Elem<kDtype>::unpack(u, v);
  float m = v[0];
#pragma unroll
  for (int i = 1; i < Elem<kDtype>::kVec; ++i) m = fminf(m, v[i]);
  return m;
}

// A row's settings; k = 0, top_p >= 1 and min_p = 0 where a filter is off.
struct Settings {
  float u, tau, top_p, min_p;
  int k, bad;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t row) {
  Settings t;
  t.u = __ldg(a.uniform + row);
  t.tau = a.row_temperature ? __ldg(a.row_temperature + row) : a.temperature;
  t.k = a.row_top_k ? __ldg(a.row_top_k + row) : a.top_k;
  t.top_p = a.row_top_p ? __ldg(a.row_top_p + row) : a.top_p;
  t.min_p = a.row_min_p ? __ldg(a.row_min_p + row) : a.min_p;
  t.bad = t.u >= 0.f && t.u < 1.f && (t.tau == 0.f || (t.tau >= 1e-6f && t.tau <= 1e6f)) &&
                  t.top_p > 0.f && t.min_p >= 0.f && t.min_p <= 1.f
              ? 0
              : TIM_ERR_INVALID_ARG;
  if (t.tau == 0.f) {  // greedy
    t.tau = 1.f;
    t.k = 1;
  }
  if (t.k <= 0 || t.k >= a.V) t.k = 0;
  return t;
}

template <int kDtype>
__device__ __forceinline__ Row<kDtype> row_of(const SampleArgs& a, int64_t row) {
  return Row<kDtype>(a.logits, row, a.ld, a.V);
}
__device__ __forceinline__ bool wanted(const SampleArgs&, int64_t) { return true; }

// What a row's weights are taken with.
struct RowState {
  Pow2Row pw;
  Df inv_tau;
  float M;      // largest logit
  int top;      // a weight w 2^(n - 62) is taken as w >> (top - n)
  uint32_t kc;  // kept: key > kc, or key == kc and id <= idc
  int idc;
};

// The weights.  2^x = 2^n T[j] (1 + p) as in pow2_fixed, laid out for sums over a row, which the integer
// pipe bounds:
//  - n is the whole number next to x, not below it, from one fp32 multiply-add whose last place is 1
//    (its factor 1 - 2^-24 makes every half go down); T[j] = 2^(j/256) for j <= 128 and 2^(j/256 - 1)
//    above.  32 bits of it, a quarter of the bank conflicts of 64;
//  - p from a multiply-add whose last place is 1 as well, so that its bits are 2^31 p and a constant.
// T and 1 + p at scale 2^31 are each off by 2^-31.5 and 2^-32 and a little: the product, at scale
// 2^62, by less than 2^-30.5.
constexpr float kUnitMagic = 12582912.f;  // 1.5 * 2^23: a sum's last place is 1
struct Tables {
  u64 fine[256];  // pow2_fixed's
  uint32_t t[256];
};
__device__ __forceinline__ void load_tables(Tables& tables, int tid, int threads) {
  for (int i = tid; i < 256; i += threads) {
    const u64 x = __ldg(&g_pow2_table.t[i]);
    const int down = i <= 128 ? 31 : 32;
    tables.fine[i] = x;
    tables.t[i] = static_cast<uint32_t>((x + (1ull << (down - 1))) >> down);
  }
}
// A row's scale as weight_of takes it: a weight w 2^(n - 62) becomes w >> (top - n).
__device__ __forceinline__ uint32_t shift_of(int top) {
  return static_cast<uint32_t>(top) + __float_as_uint(kUnitMagic) + static_cast<uint32_t>(kPow2Magic);
}
// t = x + kPow2Magic rounded to 1/256, g = x less that multiple of 1/256.  Any x below 2^14 will do:
// what is far below the scale gives a shift above 63, or a number without meaning that is as large,
// and the shift instruction makes that 0.
__device__ __forceinline__ u64 weight_of(float t, float g, uint32_t shift, const uint32_t* table) {
  const float p = fmaf(g, fmaf(g, fmaf(g, 119194168.0f, 515882496.0f), 1488522236.0f), kUnitMagic);
  const float n = fmaf(t, 1.f - 0x1p-24f, kUnitMagic);
  const uint32_t q = __float_as_uint(p) + (0x80000000u - __float_as_uint(kUnitMagic));
  u64 w = static_cast<u64>(table[__float_as_uint(t) & 255u]) * q;
  asm("shr.u64 %0, %0, %1;" : "+l"(w) : "r"(shift - __float_as_uint(n)));
  return w;
}
// Two of them, the fp32 part in packed operations: the same bits.  magic: kPow2Magic and whatever is to be
// added to z K, a multiple of 1/256.
struct PairScale {
  F2 kh, kl, magic;
};
__device__ __forceinline__ PairScale pair_scale(float kh, float kl, float magic) {
  return PairScale{f2(kh, kh), f2(kl, kl), f2(magic, magic)};
}
__device__ __forceinline__ void weights_of_two(float z0, float z1, const PairScale& s, uint32_t shift,
                                               const uint32_t* table, u64& w0, u64& w1) {
  const F2 z = f2(z0, z1), unit = f2(kUnitMagic, kUnitMagic);
  const F2 t = fma2(z, s.kh, s.magic);
  const F2 g = fma2(z, s.kl, fma2(z, s.kh, fma2(t, f2(-1.f, -1.f), s.magic)));
  const F2 c2 = f2(515882496.0f, 515882496.0f), c1 = f2(1488522236.0f, 1488522236.0f);
  const F2 p = fma2(g, fma2(g, fma2(g, f2(119194168.0f, 119194168.0f), c2), c1), unit);
  const float2 n = unpack2(fma2(t, f2(1.f - 0x1p-24f, 1.f - 0x1p-24f), unit));
  const float2 ts = unpack2(t), ps = unpack2(p);
  const uint32_t one = 0x80000000u - __float_as_uint(kUnitMagic);
  w0 = static_cast<u64>(table[__float_as_uint(ts.x) & 255u]) * (__float_as_uint(ps.x) + one);
  w1 = static_cast<u64>(table[__float_as_uint(ts.y) & 255u]) * (__float_as_uint(ps.y) + one);
  asm("shr.u64 %0, %0, %1;" : "+l"(w0) : "r"(shift - __float_as_uint(n.x)));
  asm("shr.u64 %0, %0, %1;" : "+l"(w1) : "r"(shift - __float_as_uint(n.y)));
}
// Without recentring.
__device__ __forceinline__ u64 weight_at(float z, float kh, float kl, uint32_t shift,
                                         const uint32_t* table) {
  const float t = fmaf(z, kh, kPow2Magic);
  return weight_of(t, fmaf(z, kl, fmaf(z, kh, kPow2Magic - t)), shift, table);
}
__device__ __forceinline__ u64 weight(float z, const RowState& s, const Tables& tables) {
  if (!s.pw.recentre) return weight_at(z, s.pw.kh, s.pw.kl, shift_of(s.top), tables.t);
  // logits so far apart that a float's step can be many octaves; z - c = d + e exactly
  if (!((z - s.pw.c) * s.pw.kh > static_cast<float>(s.top) - 64.f)) return 0;
  const float d = z - s.pw.c, b = d - z, e = (z - (d - b)) + (-s.pw.c - b);
  const float t = fmaf(d, s.pw.kh, kPow2Magic);
  const float g = fmaf(e, s.pw.kh, fmaf(d, s.pw.kl, fmaf(d, s.pw.kh, kPow2Magic - t)));
  return weight_of(t, g, shift_of(s.top), tables.t);
}
__device__ __forceinline__ bool keeps(uint32_t key, int id, const RowState& s) {
  return key > s.kc || (key == s.kc && id <= s.idc);
}


__device__ __forceinline__ void set_temperature(RowState& st, float tau) {
  st.inv_tau = reciprocal(df(tau));
  const Df K = Df{kLog2eHi, kLog2eLo} * st.inv_tau;
  st.pw.kh = K.h;
  st.pw.kl = K.l;
}

// The scale: N bounds the largest weight and `most` the sum of all relative to it, so the row's
// total is below 2^60.
__device__ __forceinline__ void set_scale(RowState& st, float most) {
  const Df mk = df(st.M) * Df{st.pw.kh, st.pw.kl};
  st.pw.recentre = !(fabsf(mk.h) < 8192.f);  // too large to split z K itself
  st.pw.c = st.pw.recentre ? st.M : 0.f;
  const int N = st.pw.recentre ? 0 : static_cast<int>(ceilf(mk.h));
  st.top = N + 3 + ilogbf(most);
}

// Sum over the threads before this one of the CTA, and over all; `warps` of them have any.
template <int kThreads>
__device__ __forceinline__ u64 block_scan(u64 v, u64* scratch, int warps, u64& total) {
  const u64 incl = warp_scan(v);
  if ((threadIdx.x & 31) == 31) scratch[threadIdx.x >> 5] = incl;
  __syncthreads();
  u64 before = incl - v;
  total = 0;
  for (int i = 0; i < warps; ++i) {
    const u64 x = scratch[i];
    if (i < static_cast<int>(threadIdx.x >> 5)) before += x;
    total += x;
  }
  return before;
}

// Descending bitonic sort of n2 (a power of two) keys by the CTA.  A warp's 32 pairs of a step of
// stride up to 32 are its own 64 keys, so only the wider steps need the whole CTA.
template <int kThreads>
__device__ __forceinline__ void sort_desc(u64* b, int n2) {
  for (int k = 2; k <= n2; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int p = threadIdx.x; p < (n2 >> 1); p += kThreads) {
        const int i = ((p & ~(j - 1)) << 1) | (p & (j - 1));
        const u64 x = b[i], y = b[i + j];
        if ((x < y) == ((i & k) == 0)) {
          b[i] = y;
          b[i + j] = x;
        }
      }
      if (j > 32 || (j == 1 && k > 32))
        __syncthreads();
      else
        __syncwarp();
    }
  }
  __syncthreads();
}

// total f rounded down, and whether something was rounded off: exact, in integers (this part has few
// fp64 units: a conversion and a product by every warp would take microseconds).  0 <= f < 1.
__device__ __forceinline__ u64 share_of(u64 total, float f, bool& more) {
  const uint32_t bits = __float_as_uint(f);
  const int e = static_cast<int>(bits >> 23);
  const u64 m = e == 0 ? bits : (bits & 0x7FFFFFu) | 0x800000u;  // f = m 2^-s
  const int s = 150 - max(e, 1);
  const u64 hi = __umul64hi(total, m), lo = total * m;
  if (s < 64) {
    more = (lo & ((1ull << s) - 1)) != 0;
    return (hi << (64 - s)) | (lo >> s);
  }
  const int r = s - 64;  // hi < 2^24
  more = lo != 0 || (hi & ((1ull << min(r, 32)) - 1)) != 0;
  return r >= 32 ? 0 : hi >> r;
}
// Before how much weight top-p keeps a token: the smallest whole number not below p total.
__device__ __forceinline__ u64 top_p_target(u64 total, float p) {
  bool more;
  const u64 t = share_of(total, p, more);
  return max(t + (more ? 1 : 0), static_cast<u64>(1));
}
// The draw: the token at which the running sum first exceeds this.
__device__ __forceinline__ u64 draw_target(u64 total, float u) {
  bool more;
  return share_of(total, u, more);
}

// The first key that min-p keeps.
__device__ __forceinline__ uint32_t min_p_key(float M, float tau, float min_p) {
  if (!(min_p > 0.f)) return kNegInfKey + 1;
  const bool tiny = min_p < 0x1p-126f;
  const Df ln = log_df(df(tiny ? min_p * 0x1p64f : min_p)) -
                (tiny ? Df{kLn2Hi, kLn2Lo} * df(64.f) : df(0.f));
  const Df cut = df(M) + df(tau) * ln;
  return max(key_of(cut.h) + (cut.l > 0.f ? 1u : 0u),  // the first float that is not below
             kNegInfKey + 1);
}

__device__ __forceinline__ void write_bad(const SampleArgs& a, int64_t row, int code) {
  set_status(a.status, code);
  a.ids[row] = -1;
  a.logprob[row] = a.lse[row] = __int_as_float(0x7FC00000);
  a.kept[row] = 0;
}

// ln of a sum of weights as a pair: the leading 48 bits, and the scale
__device__ __forceinline__ Df log_total(u64 total, int top, const Tables& tables) {
  const int lz = __clzll(static_cast<long long>(total));
  const u64 t = total << lz;
  const Df f = renorm(static_cast<float>(static_cast<uint32_t>(t >> 40)) * 0x1p-24f,
                      static_cast<float>(static_cast<uint32_t>(t >> 16) & 0xFFFFFFu) * 0x1p-48f);
  const float e = static_cast<float>(64 - lz + top - 62);
  return log_df(f, tables.fine) + Df{kLn2Hi, kLn2Lo} * df(e);
}

// The border of a row without filters: key << 32 | ~id of the last token above -inf.
constexpr u64 kAllKept = static_cast<u64>(kNegInfKey + 1) << 32;

// total: kept weights' sum; x: logit of the token; n: tokens kept; by one thread
__device__ __forceinline__ void write_row(const SampleArgs& a, const RowState& st,
                                          const Tables& tables, int64_t row, int id, float x,
                                          u64 total, int n, u64) {
  const Df ln = log_total(total, st.top, tables);
  const float base = st.pw.recentre ? st.pw.c : 0.f;
  const Df lse = ln + df(base) * st.inv_tau;
  a.ids[row] = id;
  a.logprob[row] = n == 1 ? 0.f : ((df(x) - df(base)) * st.inv_tau - ln).h;
  a.lse[row] = n == 1 ? (df(st.M) * st.inv_tau).h : lse.h;
  a.kept[row] = n;
}

}  // namespace sampling
}  // namespace tim
