// Sampling from a [T, V] logits matrix with temperature, top-k, top-p and min-p, from
// given uniform numbers.
//
// Order the tokens of a row by (logit descending, id ascending); s = z / tau.
//   top-k   the first k of them: the set K
//   top-p   q = softmax of s over K; a token is kept while the q-mass before it is < p
//   min-p   exp(s - s_max) >= min_p
//   token   the smallest id v with  sum_{kept w <= v} exp(s_w) > u * sum_kept exp(s)
// What is kept is "key above a border key, or equal to it with an id up to a border id",
// so a row is described by two numbers and is never sorted.
//
// A token drawn, or the last one that top-p keeps, is decided by sums of up to hundreds of
// thousands of exponentials against a border: rounding them to 32 bits would move the
// border past tokens.  Every weight is therefore taken to 2^-33 (pow2_fixed) and summed as a
// 64-bit integer at a scale fixed by an approximate first sum, so that the row's total is
// near 2^60: the sums are exact in that scale and do not depend on the order or the split.
#include <cmath>

#include "logits_row.cuh"

namespace tim {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
using u64 = unsigned long long;

struct SampleArgs {
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

__device__ __forceinline__ Pow2Row pow2_row(float temperature, float zmax) {
  const double K = 1.4426950408889634 / static_cast<double>(temperature);
  Pow2Row r;
  r.kh = static_cast<float>(K);
  r.kl = static_cast<float>(K - static_cast<double>(r.kh));
  r.recentre = !(fabs(static_cast<double>(zmax) * K) < 8192.0);  // too large for the split of z K
  r.c = r.recentre ? zmax : 0.f;
  return r;
}

// Monotone map of float bits to unsigned (larger float -> larger key; -0 and +0 are one).
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t f = __float_as_uint(z + 0.f);
  return (f & 0x80000000u) ? ~f : (f | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
constexpr uint32_t kNegInfKey = 0x007FFFFFu;  // key_of(-inf)

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

struct Shared {
  u64 table[256];
  u64 mass[kBins];
  uint32_t count[kBins];
  u64 warp[kWarps];
  float warpf[kWarps];
  u64 pick_acc;
  u64 pick_in;
  uint32_t pick_digit;
  int pick_all;
  int found;
  int bad;
};

struct RowState {
  Pow2Row pw;
  int top;      // weights are w 2^(n - top) at the row's scale: shift = top - n
  uint32_t kc;  // kept: key > kc, or key == kc and id <= idc
  int idc;
};

// The integer weight of a logit at the row's scale.
__device__ __forceinline__ u64 weight(float z, const RowState& s, const u64* table) {
  int n;
  const u64 w = pow2_fixed(z, s.pw, table, n);
  return w >> min(s.top - n, 63);
}

__device__ __forceinline__ bool keeps(uint32_t key, int id, const RowState& s) {
  return key > s.kc || (key == s.kc && id <= s.idc);
}

// Calls f(id, z) for the row's elements in this warp's contiguous slice, lane order being id
// order within each step of 32 vectors.
template <int kDtype, class F>
__device__ __forceinline__ void for_slice(const Row<kDtype>& r, int warp, F&& f) {
  using E = Elem<kDtype>;
  const int nvec = r.nvec();
  const int per = (nvec + kWarps * 32 - 1) / (kWarps * 32) * 32;
  const int j0 = warp * per, j1 = min(nvec, j0 + per);
  for (int jj = j0; jj < j1; jj += 32) {
    const int j = jj + (threadIdx.x & 31);
    float v[E::kVec];
    if (j < j1) {
      E::unpack(r.load(j), v);
    } else {
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) v[i] = -INFINITY;
    }
    f(j * E::kVec - r.shift, v);
  }
}

// Border of the tokens whose measure before them, in (key descending, id ascending) order,
// is below `target`; measure 1 (kMass false) or the weight.  Only tokens that `s` keeps
// count.  On return s.kc / s.idc hold the border; digits of 8 bits from the top.
template <int kDtype, bool kMass>
__device__ void select_border(const Row<kDtype>& r, RowState& s, float zlow, u64 target,
                              Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t prefix = 0;
  u64 acc = 0, in = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      sh.mass[i] = 0;
      sh.count[i] = 0;
    }
    __syncthreads();
    for_slice(r, warp, [&](int id0, const auto& v) {
#pragma unroll
      for (int i = 0; i < Elem<kDtype>::kVec; ++i) {
        const uint32_t key = key_of(v[i]);
        if (shift < 24 && (key >> (shift + 8)) != prefix) continue;
        if (!keeps(key, id0 + i, s)) continue;
        const int d = (key >> shift) & 255;
        atomicAdd(&sh.count[d], 1u);
        if (kMass && v[i] >= zlow) atomicAdd(&sh.mass[d], weight(v[i], s, sh.table));
      }
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 a = acc;
      int d = 255;
      for (; d > 0; --d) {
        const u64 h = kMass ? sh.mass[d] : static_cast<u64>(sh.count[d]);
        if (a + h >= target) break;
        a += h;
      }
      sh.pick_digit = d;
      sh.pick_all = d == 0 && a + (kMass ? sh.mass[0] : static_cast<u64>(sh.count[0])) < target;
      sh.pick_acc = a;
      sh.pick_in = sh.count[d];
    }
    __syncthreads();
    if (sh.pick_all) return;  // fewer than the target: every one of them stays
    prefix = (prefix << 8) | sh.pick_digit;
    acc = sh.pick_acc;
    in = sh.pick_in;
    __syncthreads();
  }
  // the border key's tokens have equal measures: how many of them, in id order
  u64 w = 1;
  if (kMass) {
    const float z = key_value(prefix);
    w = z >= zlow ? weight(z, s, sh.table) : 0;
    if (w == 0) w = 1;
  }
  const u64 want = (target - acc + w - 1) / w;
  if (want >= in) {
    if (prefix != s.kc) {
      s.kc = prefix;
      s.idc = INT32_MAX;
    }
    return;
  }
  // the id of the want-th of them
  u64 mine = 0;
  for_slice(r, warp, [&](int id0, const auto& v) {
#pragma unroll
    for (int i = 0; i < Elem<kDtype>::kVec; ++i)
      mine += key_of(v[i]) == prefix && keeps(prefix, id0 + i, s) ? 1 : 0;
  });
  mine = warp_sum(mine);
  if (lane == 0) sh.warp[warp] = mine;
  __syncthreads();
  u64 before = 0;
  for (int i = 0; i < warp; ++i) before += sh.warp[i];
  if (before < want && want <= before + mine) {
    u64 run = before;
    for_slice(r, warp, [&](int id0, const auto& v) {
      int c = 0;
#pragma unroll
      for (int i = 0; i < Elem<kDtype>::kVec; ++i)
        c += key_of(v[i]) == prefix && keeps(prefix, id0 + i, s) ? 1 : 0;
      int incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += u;
      }
      u64 at = run + incl - c;
      if (at < want && want <= at + c) {
#pragma unroll
        for (int i = 0; i < Elem<kDtype>::kVec; ++i)
          if (key_of(v[i]) == prefix && keeps(prefix, id0 + i, s) && ++at == want)
            sh.found = id0 + i;
      }
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    });
  }
  __syncthreads();
  s.kc = prefix;
  s.idc = sh.found;
  __syncthreads();
}

template <int kDtype>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  using E = Elem<kDtype>;
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  const float u = a.uniform[row];
  float tau = a.row_temperature ? a.row_temperature[row] : a.temperature;
  int k = a.row_top_k ? a.row_top_k[row] : a.top_k;
  const float top_p = a.row_top_p ? a.row_top_p[row] : a.top_p;
  const float min_p = a.row_min_p ? a.row_min_p[row] : a.min_p;
  const bool args_ok = u >= 0.f && u < 1.f && (tau == 0.f || (tau >= 1e-6f && tau <= 1e6f)) &&
                       top_p > 0.f && min_p >= 0.f && min_p <= 1.f;
  if (tau == 0.f) {
    tau = 1.f;
    k = 1;
  }
  for (int i = threadIdx.x; i < 256; i += kThreads) sh.table[i] = g_pow2_table.t[i];
  if (threadIdx.x == 0) {
    sh.bad = args_ok ? 0 : TIM_ERR_INVALID_ARG;
    sh.found = -1;
  }
  __syncthreads();

  float m = -INFINITY;
  bool nan = false;
  for_slice(r, warp, [&](int, const auto& v) {
#pragma unroll
    for (int i = 0; i < E::kVec; ++i) {
      m = fmaxf(m, v[i]);
      nan |= !(v[i] < INFINITY);
    }
  });
  if (nan) sh.bad = TIM_ERR_NONFINITE;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (lane == 0) sh.warpf[warp] = m;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) m = fmaxf(m, sh.warpf[i]);
  int bad = sh.bad;
  if (bad == 0 && m == -INFINITY) bad = TIM_ERR_NONFINITE;
  if (bad != 0) {
    if (threadIdx.x == 0) {
      set_status(a.status, bad);
      a.ids[row] = -1;
      a.logprob[row] = a.lse[row] = __int_as_float(0x7FC00000);
      a.kept[row] = 0;
    }
    return;
  }
  __syncthreads();

  // approximate total, relative to the largest
  const float k2 = static_cast<float>(1.4426950408889634 / static_cast<double>(tau));
  float sum = 0.f;
  for_slice(r, warp, [&](int, const auto& v) {
#pragma unroll
    for (int i = 0; i < E::kVec; ++i) sum += ex2_approx((v[i] - m) * k2);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) sh.warpf[warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int i = 0; i < kWarps; ++i) sum += sh.warpf[i];
  __syncthreads();

  RowState s;
  s.pw = pow2_row(tau, m);
  // weights relative to 2^N >= the largest; the total near 2^60
  const double K = 1.4426950408889634 / static_cast<double>(tau);
  const double mk = s.pw.recentre ? 0.0 : static_cast<double>(m) * K;
  const int N = static_cast<int>(ceil(mk));
  const int scale = 60 - ilogbf(sum);
  s.top = N + 62 - scale;
  s.kc = kNegInfKey;
  s.idc = INT32_MIN;
  // below this a weight is 0: the first bound keeps 2^x within pow2_fixed's range
  const float zlow = static_cast<float>(
      fmax(static_cast<double>(m) - 80.0 / K, -3.4028234663852886e38));

  if (k > 0 && k < a.V) select_border<kDtype, false>(r, s, zlow, static_cast<u64>(k), sh);
  auto kept_mass = [&]() {
    u64 mine = 0;
    for_slice(r, warp, [&](int id0, const auto& v) {
#pragma unroll
      for (int i = 0; i < E::kVec; ++i)
        if (v[i] >= zlow && keeps(key_of(v[i]), id0 + i, s)) mine += weight(v[i], s, sh.table);
    });
    mine = warp_sum(mine);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = mine;
    __syncthreads();
    u64 t = 0;
    for (int i = 0; i < kWarps; ++i) t += sh.warp[i];
    return t;
  };
  if (top_p < 1.f) {
    const u64 total = kept_mass();
    u64 target = static_cast<u64>(ceil(static_cast<double>(total) * static_cast<double>(top_p)));
    target = max(target, 1ull);
    __syncthreads();
    select_border<kDtype, true>(r, s, zlow, target, sh);
  }
  if (min_p > 0.f) {
    const double cut = static_cast<double>(m) + static_cast<double>(tau) * log(static_cast<double>(min_p));
    const uint32_t kmin = key_of(__double2float_ru(cut));
    if (kmin > s.kc) {
      s.kc = kmin;
      s.idc = INT32_MAX;
    }
  }
  const u64 total = kept_mass();
  const u64 target = static_cast<u64>(static_cast<double>(total) * static_cast<double>(u));
  // the first token whose running sum exceeds the target, and the number kept
  u64 mine = sh.warp[warp];
  u64 before = 0;
  for (int i = 0; i < warp; ++i) before += sh.warp[i];
  __syncthreads();
  u64 n_kept = 0;
  for_slice(r, warp, [&](int id0, const auto& v) {
#pragma unroll
    for (int i = 0; i < E::kVec; ++i) n_kept += keeps(key_of(v[i]), id0 + i, s) ? 1 : 0;
  });
  n_kept = warp_sum(n_kept);
  if (lane == 0) sh.mass[warp] = n_kept;
  if (before <= target && target < before + mine) {
    u64 run = before;
    for_slice(r, warp, [&](int id0, const auto& v) {
      u64 w[E::kVec], c = 0;
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) {
        w[i] = v[i] >= zlow && keeps(key_of(v[i]), id0 + i, s) ? weight(v[i], s, sh.table) : 0;
        c += w[i];
      }
      u64 incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
      }
      u64 at = run + incl - c;
      if (at <= target && target < at + c) {
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) {
          if (at <= target && target < at + w[i]) sh.found = id0 + i;
          at += w[i];
        }
      }
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    });
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int id = sh.found;
    u64 n = 0;
    for (int i = 0; i < kWarps; ++i) n += sh.mass[i];
    const double base = s.pw.recentre ? static_cast<double>(m) : 0.0;
    const double inv_tau = 1.0 / static_cast<double>(tau);
    // ln sum = ln(total) in the weights' unit
    const double ls = log(static_cast<double>(total)) +
                      static_cast<double>(s.top - 62) * 0.6931471805599453;
    const double x = (static_cast<double>(r.at(id)) - base) * inv_tau;
    a.ids[row] = id;
    a.logprob[row] = n == 1 ? 0.f : static_cast<float>(x - ls);
    a.lse[row] = n == 1 ? static_cast<float>(static_cast<double>(m) * inv_tau)
                        : static_cast<float>(base * inv_tau + ls);
    a.kept[row] = static_cast<int32_t>(n);
  }
}

}  // namespace

cudaError_t launch_sample(const void* logits, int dtype, int64_t ld, int64_t T, int V,
                          const float* uniform, const tim_sample_params& p, int32_t* ids,
                          float* logprob, float* lse, int32_t* kept, int* status,
                          cudaStream_t stream) {
  const SampleArgs a = {logits, ld, V, uniform, p.temperature, p.top_k, p.top_p, p.min_p,
                        p.row_temperature, p.row_top_k, p.row_top_p, p.row_min_p, ids, logprob,
                        lse, kept, status};
  const unsigned g = static_cast<unsigned>(T);
  if (dtype == TIM_F32)
    sample_kernel<TIM_F32><<<g, kThreads, 0, stream>>>(a);
  else if (dtype == TIM_BF16)
    sample_kernel<TIM_BF16><<<g, kThreads, 0, stream>>>(a);
  else
    sample_kernel<TIM_F16><<<g, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tim
