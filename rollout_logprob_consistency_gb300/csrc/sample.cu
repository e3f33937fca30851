// Sampling from a [T, V] logits matrix with temperature, top-k, top-p and min-p, from
// given uniform numbers.
//
// Order the tokens of a row by (logit descending, id ascending); s = z / tau.
//   top-k   the first k of them: the set K
//   top-p   q = softmax of s over K; a token is kept while the q-mass before it is < p
//   min-p   exp(s - s_max) >= min_p
//   token   the smallest id v with  sum_{kept w <= v} exp(s_w) > u * sum_kept exp(s)
//
// A token drawn, or the last one that top-p keeps, is decided by sums of up to hundreds of
// thousands of exponentials against a border: rounding them to 32 bits would move the
// border past tokens.  Every weight that decides is therefore taken to 2^-33 (pow2_fixed) and
// summed as a 64-bit integer, at a scale that puts the row's total between 2^53 and 2^60: the
// sums are exact in that scale and do not depend on the order or the split.
//
// A row is held in shared memory by a cluster of CTAs (one read of memory), a slice each.  A
// thread's largest logits of its part of the slice bound everything else:
//  - sum over the threads of (largest weight x elements) bounds the row's total: the scale;
//  - the k-th largest of the threads' maxima is a bound that every top-k logit meets (they
//    are k different logits), found to 1/256 of their range by a histogram of them;
//  - only threads whose maximum meets the bound look at their elements again.
// Two ways follow:
//  few   the tokens above the bound (top-k's; for top-p the logit below which all tokens
//        together hold less than 1 - p; min-p's own) fit a list of kCap: rank 0 sorts it and
//        decides alone.  Top-p without top-k needs the row's total: a sum in fp32 with a proven
//        error decides unless the border lies within that error.
//  wide  everything else, the unfiltered row first of all: what is kept is "key above a border
//        key, or equal to it with an id up to a border id", found digit by digit with
//        histograms of counts or integer weights, and the token by running sums over chunks.
// Both give the same token: the weights and sums are the same integers.
#include <cmath>

#include "logits_row.cuh"

namespace tim {

namespace {

constexpr int kBins = 256;
constexpr int kMaxCluster = 8;
constexpr int kCap = 512;      // tokens of the list
constexpr int kListK = 256;    // largest top-k that the list serves
constexpr int kMaxSteps = 64;  // 32-vector steps of a warp's part: at most 24580 vectors over 16 warps
constexpr float kSumError = 0x1p-17f;  // of the fp32 sum, see approximate_sum
using u64 = unsigned long long;

struct SampleArgs {
  const void* logits;
  int64_t ld;
  int V;
  int cluster;
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

__device__ __forceinline__ uint32_t remote_load(const void* smem, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(smem, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote_add(void* smem, uint32_t rank, uint32_t v) {
  uint32_t r;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(r)
               : "r"(cluster_addr(smem, rank)), "r"(v)
               : "memory");
  return r;
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

// Everything of a row that all its CTAs agree on.
struct RowState {
  Pow2Row pw;
  Df inv_tau;
  float M;      // largest logit
  int top;      // a weight w 2^(n - 62) of pow2_fixed is w >> (top - n)
  float zlow;   // logits below have weight 0 and are raised to this one
  uint32_t kc;  // kept: key > kc, or key == kc and id <= idc
  int idc;
};

__device__ __forceinline__ u64 weight(float z, const RowState& s, const u64* table) {
  int n;
  if (s.pw.recentre) {
    // logits so far apart that a float's step can be many octaves
    if (!((z - s.pw.c) * s.pw.kh > static_cast<float>(s.top) - 62.5f)) return 0;
  } else {
    z = fmaxf(z, s.zlow);
  }
  const u64 w = pow2_fixed(z, s.pw, table, n);
  return w >> min(s.top - n, 63);
}
__device__ __forceinline__ bool keeps(uint32_t key, int id, const RowState& s) {
  return key > s.kc || (key == s.kc && id <= s.idc);
}

struct Select {  // the wide way's histograms
  uint32_t count[2][kBins], lo[2][kBins], hi[2][kBins];
};
struct List {
  u64 key[kCap];  // key << 32 | ~id: larger comes first
  u64 w[kCap];
};

template <int kThreads>
struct Shared {
  u64 table[256];
  union {
    Select sel;
    List list;
  };
  u64 xch[2][kMaxCluster][2];
  // of every warp of every CTA: largest key, and a sum relative to it
  uint32_t gkey[kMaxCluster * kThreads / 32];
  float gsum[kMaxCluster * kThreads / 32];
  uint32_t hist[kBins];  // of the threads' maxima
  u64 warp[kThreads / 32];
  uint32_t warpu[kThreads / 32];
  u64 step[kMaxSteps];  // sums over 32 vectors each, of one warp's part
  u64 acc;
  uint32_t digit, in, bound;
  uint32_t list_n;
  int all, found, count_lo, count_hi;
  uint64_t bar;
};

template <int kDtype, int kThreads>
struct Sampler {
  using E = Elem<kDtype>;
  static constexpr int kVec = E::kVec;
  static constexpr int kWarps = kThreads / 32;

  const SampleArgs& a;
  Shared<kThreads>& sh;
  const uint4* slice;
  Row<kDtype> r;
  Slice s;
  int rank, tid, warp, lane, phase;
  RowState st;

  // ---- among the CTAs of the row: every CTA's two numbers to every CTA
  __device__ __forceinline__ void exchange(u64 x, u64 y) {  // called by all; warp 0's values
    if (warp == 0 && lane < a.cluster) {
      cluster_store(cluster_addr(&sh.xch[phase & 1][rank][0], lane), x);
      cluster_store(cluster_addr(&sh.xch[phase & 1][rank][1], lane), y);
    }
    cluster_arrive();
    cluster_wait();
    ++phase;
  }
  __device__ __forceinline__ u64 got(int rank_, int i) const { return sh.xch[(phase - 1) & 1][rank_][i]; }

  // id of slot i of the slice's vector j
  __device__ __forceinline__ int id_of(int j, int i) const { return (s.j0 + j) * kVec + i - r.shift; }
  __device__ __forceinline__ bool in_row(int id) const { return id >= 0 && id < a.V; }

  // ---- sums over the slice.  A warp has a contiguous part of it, in steps of 32 vectors.
  __device__ __forceinline__ int part_steps() const { return (s.n + kThreads - 1) / kThreads; }
  __device__ __forceinline__ int part_start(int w) const { return w * part_steps() * 32; }

  // The sum of f(z, id) over the slice; sh.warp[] gets the parts' sums.  f(v, id0, ends) is the sum
  // of a vector.
  template <class F>
  __device__ __forceinline__ u64 slice_sum(F&& f) {
    const int j0 = part_start(warp), j1 = min(s.n, j0 + part_steps() * 32);
    u64 sum = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
      float v[kVec];
      E::unpack(slice[j], v);
      sum += f(v, id_of(j, 0));
    }
    sum = warp_sum(sum);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = sum;
    __syncthreads();
    u64 t = 0;
    for (int i = 0; i < kWarps; ++i) t += sh.warp[i];
    return t;
  }
  // The token at which the running sum first exceeds `target` (below the CTA's sum), in every
  // thread; after slice_sum(f), by the whole CTA.  one(z, id) is a token's number.
  template <class F, class G>
  __device__ __forceinline__ int locate(u64 target, F&& f, G&& one) {
    int w = 0;
    for (; w < kWarps - 1 && target >= sh.warp[w]; ++w) target -= sh.warp[w];
    const int j0 = part_start(w), j1 = min(s.n, j0 + part_steps() * 32);
    for (int i = warp; j0 + i * 32 < j1; i += kWarps) {
      const int j = j0 + i * 32 + lane;
      u64 sum = 0;
      if (j < j1) {
        float v[kVec];
        E::unpack(slice[j], v);
        sum = f(v, id_of(j, 0));
      }
      sum = warp_sum(sum);
      if (lane == 0) sh.step[i] = sum;
    }
    __syncthreads();
    int i = 0;
    for (; j0 + (i + 1) * 32 < j1 && target >= sh.step[i]; ++i) target -= sh.step[i];
    if (warp == 0) {
      const int j = j0 + i * 32 + lane;
      u64 x[kVec], sum = 0;
      float v[kVec];
      const int id0 = id_of(j, 0);
      if (j < j1) E::unpack(slice[j], v);
#pragma unroll
      for (int q = 0; q < kVec; ++q) {
        x[q] = j < j1 ? one(v[q], id0 + q) : 0;
        sum += x[q];
      }
      u64 at = warp_scan(sum) - sum;
#pragma unroll
      for (int q = 0; q < kVec; ++q) {
        if (at <= target && target < at + x[q]) sh.found = id0 + q;
        at += x[q];
      }
    }
    __syncthreads();
    return sh.found;
  }

  // ---- the wide way's border.  Among the tokens that the state keeps: the last one before which
  // the measure (1, or with kMass the weight) is below `target`; the state then keeps up to it.
  template <bool kMass>
  __device__ void select_border(u64 target) {
    uint32_t prefix = 0, in = 0;
    u64 acc = 0;
    const uint32_t kc = st.kc;
    const int idc = st.idc;
    for (int level = 0; level < kLevels<kDtype>; ++level) {
      const int shift = 24 - 8 * level, b = level & 1;
      for (int i = tid; i < kBins; i += kThreads)
        sh.sel.count[b][i] = sh.sel.lo[b][i] = sh.sel.hi[b][i] = 0;
      __syncthreads();
      for (int j = tid; j < s.n; j += kThreads) {
        float v[kVec];
        E::unpack(slice[j], v);
        const int id0 = id_of(j, 0);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const uint32_t key = key_of(v[i]);
          if (level > 0 && (key >> (shift + 8)) != prefix) continue;
          if (!(key > kc || (key == kc && id0 + i <= idc))) continue;
          const int d = (key >> shift) & 255;
          atomicAdd(&sh.sel.count[b][d], 1u);
          if (kMass) {  // a 64-bit sum from two 32-bit ones
            const u64 w = weight(v[i], st, sh.table);
            const uint32_t wl = static_cast<uint32_t>(w);
            const uint32_t old = atomicAdd(&sh.sel.lo[b][d], wl);
            const uint32_t wh = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
            if (wh != 0) atomicAdd(&sh.sel.hi[b][d], wh);
          }
        }
      }
      cluster_arrive();
      cluster_wait();
      // digit 255 - tid, all CTAs'; their running sums from the top
      uint32_t cnt = 0;
      u64 h = 0;
      if (tid < kBins) {
        const int d = 255 - tid;
        for (int c = 0; c < a.cluster; ++c) {
          const uint32_t n = remote_load(&sh.sel.count[b][d], c);
          cnt += n;
          if (!kMass)
            h += n;
          else if (n != 0)
            h += (static_cast<u64>(remote_load(&sh.sel.hi[b][d], c)) << 32) +
                 remote_load(&sh.sel.lo[b][d], c);
        }
      }
      const u64 incl = warp_scan(h);
      if (lane == 31) sh.warp[warp] = incl;
      if (tid == 0) sh.all = 1;
      __syncthreads();
      u64 before = acc + incl - h;
      for (int i = 0; i < min(warp, kBins / 32); ++i) before += sh.warp[i];
      if (tid < kBins && before < target && target <= before + h) {
        sh.digit = 255 - tid;
        sh.acc = before;
        sh.in = cnt;
        sh.all = 0;
      }
      __syncthreads();
      const bool all = sh.all != 0;  // fewer than the target: every one of them stays
      prefix = (prefix << 8) | sh.digit;
      acc = sh.acc;
      in = sh.in;
      __syncthreads();
      if (all) return;
    }
    const int rest = 32 - 8 * kLevels<kDtype>;
    uint32_t key = rest == 0 ? prefix : prefix << rest;
    if (rest != 0 && !(key & 0x80000000u)) key |= (1u << rest) - 1u;  // a negative number's
    // the border key's tokens have equal measures: how many of them, in id order
    const u64 w = kMass ? max(weight(key_value(key), st, sh.table), 1ull) : 1ull;
    const u64 want = (target - acc + w - 1) / w;
    if (want >= in) {
      if (key != kc) {
        st.kc = key;
        st.idc = INT32_MAX;
      }
      return;
    }
    auto tie = [&](float z, int id) -> u64 {
      return key_of(z) == key && (key > kc || id <= idc) && in_row(id) ? 1 : 0;
    };
    auto ties = [&](const float(&v)[kVec], int id0) {
      u64 n = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) n += tie(v[i], id0 + i);
      return n;
    };
    const u64 mine = slice_sum(ties);
    exchange(mine, 0);
    u64 before = 0;
    int owner = 0;
    for (; owner < a.cluster - 1 && before + got(owner, 0) < want; ++owner) before += got(owner, 0);
    int id = 0;
    if (rank == owner) id = locate(want - 1 - before, ties, tie);
    exchange(static_cast<u64>(id), 0);
    st.kc = key;
    st.idc = static_cast<int>(got(owner, 0));
  }

  __device__ __forceinline__ u64 kept_weight(float z, int id) const {
    return keeps(key_of(z), id, st) && in_row(id) ? weight(z, st, sh.table) : 0;
  }

  // total: kept weights' sum; x: logit of the token; one thread
  __device__ void write_row(int64_t row, int id, float x, u64 total, int n) {
    // ln total as a pair: the leading 48 bits, and the scale
    const int lz = __clzll(static_cast<long long>(total));
    const u64 t = total << lz;
    const Df f = renorm(static_cast<float>(static_cast<uint32_t>(t >> 40)) * 0x1p-24f,
                        static_cast<float>(static_cast<uint32_t>(t >> 16) & 0xFFFFFFu) * 0x1p-48f);
    const float e = static_cast<float>(64 - lz + st.top - 62);
    const Df ln = log_df(f) + Df{kLn2Hi, kLn2Lo} * df(e);
    const float base = st.pw.recentre ? st.pw.c : 0.f;
    const Df lse = ln + df(base) * st.inv_tau;
    a.ids[row] = id;
    a.logprob[row] = n == 1 ? 0.f : ((df(x) - df(base)) * st.inv_tau - ln).h;
    a.lse[row] = n == 1 ? (df(st.M) * st.inv_tau).h : lse.h;
    a.kept[row] = n;
  }

  // The scale: N bounds the largest weight and 2^e the sum of all relative to it, so the row's
  // total is below 2^60.
  __device__ __forceinline__ void set_scale(float most) {
    const Df mk = df(st.M) * Df{st.pw.kh, st.pw.kl};
    st.pw.recentre = !(fabsf(mk.h) < 8192.f);  // too large to split z K itself
    st.pw.c = st.pw.recentre ? st.M : 0.f;
    const int N = st.pw.recentre ? 0 : static_cast<int>(ceilf(mk.h));
    st.top = N + 3 + ilogbf(most);
    // top - n <= 63 for all logits from here up
    st.zlow = ((static_cast<float>(st.top) - 62.5f) / st.pw.kh);
  }

  // Sum and count of the whole row from every CTA's.
  __device__ __forceinline__ u64 total_of(u64 mine, u64 n, u64& all) {
    exchange(mine, n);
    u64 t = 0;
    all = 0;
    for (int c = 0; c < a.cluster; ++c) {
      t += got(c, 0);
      all += got(c, 1);
    }
    return t;
  }

  // The draw, f and one being the kept tokens' weights and n their number in the slice.
  template <class F, class G>
  __device__ __forceinline__ void draw(int64_t row, float u, uint32_t n, F&& f, G&& one) {
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    __syncthreads();
    if (lane == 0) sh.warpu[warp] = n;
    const u64 mine = slice_sum(f);
    n = 0;
    for (int i = 0; i < kWarps; ++i) n += sh.warpu[i];
    u64 all;
    const u64 total = total_of(mine, n, all);
    const u64 target = static_cast<u64>(static_cast<double>(total) * static_cast<double>(u));
    u64 before = 0;
    for (int c = 0; c < rank; ++c) before += got(c, 0);
    if (before <= target && target < before + mine) {  // one CTA of the row
      const int id = locate(target - before, f, one);
      if (tid == 0) write_row(row, id, r.at(id), total, static_cast<int>(all));
    }
  }

  // ---- the wide way, by all CTAs
  __device__ void wide(int64_t row, float u, int k, float top_p, uint32_t kmin) {
    st.kc = kNegInfKey;
    st.idc = INT32_MIN;
    for (int i = tid; i < 256; i += kThreads) sh.table[i] = __ldg(&g_pow2_table.t[i]);
    __syncthreads();
    auto one = [&](float z, int id) { return kept_weight(z, id); };
    auto kept = [&](const float(&v)[kVec], int id0) {
      u64 t = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) t += one(v[i], id0 + i);
      return t;
    };
    u64 all;
    if (k > 0) select_border<false>(static_cast<u64>(k));
    if (top_p < 1.f) {
      const u64 total = total_of(slice_sum(kept), 0, all);
      const u64 target =
          static_cast<u64>(ceil(static_cast<double>(total) * static_cast<double>(top_p)));
      select_border<true>(max(target, 1ull));
    }
    if (kmin > st.kc) {
      st.kc = kmin;
      st.idc = INT32_MAX;
    }
    uint32_t n = 0;
    for (int j = tid; j < s.n; j += kThreads) {
      float v[kVec];
      E::unpack(slice[j], v);
      const int id0 = id_of(j, 0);
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        n += keeps(key_of(v[i]), id0 + i, st) && in_row(id0 + i) ? 1 : 0;
    }
    draw(row, u, n, kept, one);
  }

  // ---- the unfiltered row, by all CTAs
  __device__ void plain(int64_t row, float u) {
    for (int i = tid; i < 256; i += kThreads) sh.table[i] = __ldg(&g_pow2_table.t[i]);
    // all tokens but those of -inf are kept: only a thread that meets one counts
    uint4 low = make_uint4(0, 0, 0, 0);
    uint32_t n = 0;
    if (tid < s.n) {
      low = slice[tid];
      for (int j = tid + kThreads; j < s.n; j += kThreads) low = min_vec<kDtype>(low, slice[j]);
      float v[kVec];
      E::unpack(low, v);
      bool some = false;
#pragma unroll
      for (int i = 0; i < kVec; ++i) some |= v[i] == -INFINITY;
      if (!some) {
        n = static_cast<uint32_t>((s.n - tid + kThreads - 1) / kThreads) * kVec;
      } else {
        for (int j = tid; j < s.n; j += kThreads) {
          E::unpack(slice[j], v);
#pragma unroll
          for (int i = 0; i < kVec; ++i) n += v[i] > -INFINITY ? 1 : 0;
        }
      }
    }
    __syncthreads();
    auto one = [&](float z, int) { return weight(z, st, sh.table); };
    if (st.pw.recentre) {
      draw(row, u, n, [&](const float(&v)[kVec], int) {
        u64 t = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) t += one(v[i], 0);
        return t;
      }, one);
    } else {
      const Pow2Pair k = {f2(st.pw.kh, st.pw.kh), f2(st.pw.kl, st.pw.kl),
                          static_cast<uint32_t>(st.top) + (__float_as_uint(kPow2Magic) >> 8)};
      const float zlow = st.zlow;
      draw(row, u, n, [&](const float(&v)[kVec], int) {
        u64 t = 0;
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
          u64 w0, w1;
          pow2_shifted(f2(fmaxf(v[i], zlow), fmaxf(v[i + 1], zlow)), k, sh.table, w0, w1);
          t += w0 + w1;
        }
        return t;
      }, one);
    }
  }

  // ---- the few way: rank 0 with the list of n tokens; `complete`: it holds all that min-p keeps.
  // False: the row's total is not known well enough (only with a positive `sum`, the fp32 total in
  // units of 2^(max K)).
  __device__ bool few(int64_t row, float u, int n, int k, float top_p, uint32_t kmin,
                      bool complete, float sum) {
    List& L = sh.list;
    constexpr int kPer = (kCap + kThreads - 1) / kThreads;
    // sorted by counting how many come before
    u64 mine[kPer];
    int at[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = tid + q * kThreads;
      at[q] = 0;
      mine[q] = i < n ? L.key[i] : 0;
      if (i < n)
        for (int j = 0; j < n; ++j) at[q] += L.key[j] > mine[q] ? 1 : 0;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (tid + q * kThreads < n) L.key[at[q]] = mine[q];
    if (tid == 0) sh.count_lo = sh.count_hi = 0;
    __syncthreads();
    if (k > 0) n = min(n, k);
    // weights in order, kPer a thread, and their running sum
    u64 w[kPer], sum_w = 0;
    uint32_t key[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = tid * kPer + q;
      key[q] = i < n ? static_cast<uint32_t>(L.key[i] >> 32) : 0u;
      w[q] = i < n ? weight(key_value(key[q]), st, g_pow2_table.t) : 0;
      sum_w += w[q];
      if (i < n) L.w[i] = w[q];
    }
    const u64 incl = warp_scan(sum_w);
    if (lane == 31) sh.warp[warp] = incl;
    __syncthreads();
    u64 before = incl - sum_w, total = 0;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += sh.warp[i];
      total += sh.warp[i];
    }
    u64 lo = ~0ull, hi = ~0ull;  // top-p keeps a token while the sum before it is below
    if (top_p < 1.f) {
      const double p = static_cast<double>(top_p);
      if (sum > 0.f) {
        // the total in the weights' unit: 2^(max K - top + 62)
        const Df mk = st.pw.recentre ? df(0.f) : df(st.M) * Df{st.pw.kh, st.pw.kl};
        const float whole = rintf(mk.h), frac = (mk.h - whole) + mk.l;
        const double unit =
            static_cast<double>(pow2_df(frac, Pow2Row{1.f, 0.f, 0.f, false}).h) *
            __longlong_as_double(static_cast<long long>(static_cast<int>(whole) - st.top + 62 + 1023) << 52);
        const double P = p * static_cast<double>(sum) * unit;
        lo = static_cast<u64>(P * (1.0 - static_cast<double>(kSumError)));
        hi = static_cast<u64>(P * (1.0 + static_cast<double>(kSumError))) + 1;
        if (hi > total && !complete) lo = 0;  // the list may not reach the border
      } else {
        lo = hi = max(static_cast<u64>(ceil(static_cast<double>(total) * p)), 1ull);
      }
    }
    int c_lo = 0, c_hi = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (tid * kPer + q < n) {
        const bool min_ok = key[q] >= kmin;
        c_lo += before < lo && min_ok ? 1 : 0;
        c_hi += before < hi && min_ok ? 1 : 0;
      }
      before += w[q];
    }
    if (c_lo != 0) atomicAdd(&sh.count_lo, c_lo);
    if (c_hi != 0) atomicAdd(&sh.count_hi, c_hi);
    __syncthreads();
    const int m = sh.count_lo;
    if (m != sh.count_hi) return false;
    // the draw, by id: what the kept tokens of lower ids weigh
    u64 kept = 0, below[kPer];
    int id[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = tid + q * kThreads;
      below[q] = 0;
      id[q] = i < m ? static_cast<int>(~static_cast<uint32_t>(L.key[i])) : -1;
    }
    if (tid - lane < m) {  // this warp has tokens
      for (int j = 0; j < m; ++j) {
        const u64 wj = L.w[j];
        const int idj = static_cast<int>(~static_cast<uint32_t>(L.key[j]));
        kept += wj;
#pragma unroll
        for (int q = 0; q < kPer; ++q) below[q] += idj < id[q] ? wj : 0;
      }
      const u64 target = static_cast<u64>(static_cast<double>(kept) * static_cast<double>(u));
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int i = tid + q * kThreads;
        if (i < m && below[q] <= target && target < below[q] + L.w[i])
          write_row(row, id[q], key_value(static_cast<uint32_t>(L.key[i] >> 32)), kept, m);
      }
    }
    return true;
  }
};

// fp32 sum of 2^((z - c) K) over a thread's vectors.  A term's argument carries two roundings of
// 2^-24 (below 40 octaves: 3.3e-6 of the term; terms further down are below 2^-40 of the
// largest), the exponential 2^-22, and the sum of up to 100 terms in four partial sums 2^-24 a
// term: together below kSumError = 7.6e-6 of the row's sum.
template <int kDtype>
__device__ __forceinline__ float approximate_sum(const uint4* slice, int n, int first, int step,
                                                 float c, float k) {
  using E = Elem<kDtype>;
  const F2 ref = f2(-c, -c), kk = f2(k, k);
  F2 acc = f2(0.f, 0.f), acc2 = acc;
#pragma unroll 4
  for (int j = first; j < n; j += step) {
    float v[E::kVec];
    E::unpack(slice[j], v);
#pragma unroll
    for (int i = 0; i < E::kVec; i += 4) {
      acc = add2(acc, ex2x2(mul2(add2(f2(v[i], v[i + 1]), ref), kk)));
      acc2 = add2(acc2, ex2x2(mul2(add2(f2(v[i + 2], v[i + 3]), ref), kk)));
    }
  }
  const float2 t = unpack2(add2(acc, acc2));
  return t.x + t.y;
}

template <int kDtype, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 2)
    sample_kernel(const SampleArgs a) {
  using E = Elem<kDtype>;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint4 slice_mem[];
  __shared__ Shared<kThreads> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x / a.cluster;
  const int rank = static_cast<int>(cluster_rank());
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  const Slice s = slice_of(r.nvec(), rank, a.cluster);

  cluster_arrive();
  if (tid == 0) {
    mbar_init(&sh.bar, 1);
    fence_mbarrier_init();
    load_slice(r, s, slice_mem, &sh.bar);
    sh.list_n = 0;
    sh.bound = 0;
  }
  load_slice_edges(r, s, slice_mem);
  for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
  const float u = __ldg(a.uniform + row);
  float tau = a.row_temperature ? __ldg(a.row_temperature + row) : a.temperature;
  int k = a.row_top_k ? __ldg(a.row_top_k + row) : a.top_k;
  const float top_p = a.row_top_p ? __ldg(a.row_top_p + row) : a.top_p;
  const float min_p = a.row_min_p ? __ldg(a.row_min_p + row) : a.min_p;
  int bad = u >= 0.f && u < 1.f && (tau == 0.f || (tau >= 1e-6f && tau <= 1e6f)) && top_p > 0.f &&
                    min_p >= 0.f && min_p <= 1.f
                ? 0
                : TIM_ERR_INVALID_ARG;
  if (tau == 0.f) {
    tau = 1.f;
    k = 1;
  }
  k = k <= 0 || k >= a.V ? 0 : k;
  Sampler<kDtype, kThreads> S{a, sh, slice_mem, r, s, rank, tid, warp, lane, 0, {}};
  RowState& st = S.st;
  st.inv_tau = reciprocal(df(tau));
  const Df K = Df{kLog2eHi, kLog2eLo} * st.inv_tau;
  st.pw.kh = K.h;
  st.pw.kl = K.l;
  const bool list_k = k > 0 && k <= kListK;
  const bool need_sum = k == 0 && top_p < 1.f;
  const bool all_kept = k == 0 && top_p >= 1.f && min_p == 0.f;
  const int never = 0;
  __syncthreads();  // the barrier and the edges
  if (!mbar_wait(&sh.bar, 0, &never)) set_status(a.status, TIM_ERR_TIMEOUT);

  // ---- the largest logit of each thread; of each warp, to every CTA of the row
  float tmax = -INFINITY;
  if (tid < s.n) {
    uint4 m = slice_mem[tid];
#pragma unroll 4
    for (int j = tid + kThreads; j < s.n; j += kThreads) m = max_vec<kDtype>(m, slice_mem[j]);
    float v[E::kVec];
    E::unpack(m, v);
    tmax = v[0];
#pragma unroll
    for (int i = 1; i < E::kVec; ++i) tmax = max_nan(tmax, v[i]);
  }
  const uint32_t mykey = !(tmax < INFINITY) ? 0xFFFFFFFFu : key_of(tmax);
  const uint32_t wkey = __reduce_max_sync(0xFFFFFFFFu, mykey);
  float sum = 0.f;
  if (wkey > kNegInfKey && wkey != 0xFFFFFFFFu) {
    // relative to the warp's largest: all its weights, or the threads' largest
    const float wmax = key_value(wkey);
    if (need_sum)
      sum = approximate_sum<kDtype>(slice_mem, s.n, tid, kThreads, wmax, K.h);
    else if (!list_k)
      sum = ex2_approx((tmax - wmax) * K.h);
    if (!list_k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
  }
  cluster_wait();  // every CTA of the row runs
  if (lane < a.cluster) {
    const int g = rank * kWarps + warp;
    cluster_store32(cluster_addr(&sh.gkey[g], lane), wkey);
    if (!list_k) cluster_store32(cluster_addr(&sh.gsum[g], lane), __float_as_uint(sum));
  }
  cluster_arrive();
  cluster_wait();
  const int groups = a.cluster * kWarps;
  uint32_t hi = 0;
  for (int g = lane; g < groups; g += 32) hi = max(hi, sh.gkey[g]);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  if (bad == 0 && (hi == 0xFFFFFFFFu || hi <= kNegInfKey)) bad = TIM_ERR_NONFINITE;
  if (bad != 0) {  // the same in every CTA of the row
    if (rank == 0 && tid == 0) {
      set_status(a.status, bad);
      a.ids[row] = -1;
      a.logprob[row] = a.lse[row] = __int_as_float(0x7FC00000);
      a.kept[row] = 0;
    }
    return;
  }
  const float M = key_value(hi);
  st.M = M;
  // the groups' sums relative to the row's largest
  auto row_sum = [&]() {
    float t = 0.f;
    for (int g = lane; g < groups; g += 32) {
      const uint32_t key = sh.gkey[g];
      if (key > kNegInfKey) t += sh.gsum[g] * ex2_approx((key_value(key) - M) * K.h);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    return t;
  };
  // the elements of a thread, at most
  const float of_thread = static_cast<float>(
      ((r.nvec() + a.cluster - 1) / a.cluster + kThreads - 1) / kThreads * E::kVec);
  if (all_kept) {
    S.set_scale(row_sum() * of_thread);
    S.plain(row, u);
    return;
  }

  // ---- a bound for the list
  uint32_t kmin = kNegInfKey + 1;  // min-p keeps from here up
  if (min_p > 0.f) {
    const bool tiny = min_p < 0x1p-126f;
    const Df ln = log_df(df(tiny ? min_p * 0x1p64f : min_p)) -
                  (tiny ? Df{kLn2Hi, kLn2Lo} * df(64.f) : df(0.f));
    const Df cut = df(M) + df(tau) * ln;
    kmin = max(key_of(cut.h) + (cut.l > 0.f ? 1u : 0u),  // the first float that is not below
               kNegInfKey + 1);
  }
  // the list holds all tokens from the key `bound` up
  uint32_t bound = kNegInfKey + 1;
  bool listed = min_p > 0.f && top_p >= 1.f;
  if (listed) bound = kmin;
  if (list_k) {
    uint32_t b = hi;
    if (k > 1 && k <= groups) {
      // the k-th largest of the warps' largest: four threads a key, counting those before it
      const int g = tid >> 2;
      int before = 0;
      if (g < groups) {
        const uint32_t mine = sh.gkey[g];
        for (int i = tid & 3; i < groups; i += 4) {
          const uint32_t other = sh.gkey[i];
          before += other > mine || (other == mine && i < g) ? 1 : 0;
        }
      }
      before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
      before += __shfl_xor_sync(0xFFFFFFFFu, before, 2);
      if (g < groups && before == k - 1) sh.bound = sh.gkey[g];
      __syncthreads();
      b = max(sh.bound, kNegInfKey + 1);
    } else if (k > 1) {
      // more than there are warps: the threads' maxima in 256 bins from the largest down, over 64
      // octaves or units; the last bin bounds nothing
      const float range = fmaxf(64.f, 64.f / K.h);
      const float per_bin = range * (1.f / 255.f), inv = 1.f / per_bin;
      if (mykey > kNegInfKey)
        atomicAdd(&sh.hist[static_cast<int>(fminf((M - tmax) * inv, 255.f))], 1u);
      cluster_arrive();
      cluster_wait();
      uint32_t incl = 0;
      if (tid < kBins)
        for (int c = 0; c < a.cluster; ++c) incl += remote_load(&sh.hist[tid], c);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) sh.warpu[warp] = incl;
      if (tid == 0) sh.digit = kBins;
      __syncthreads();
      for (int i = 0; i < warp; ++i) incl += sh.warpu[i];
      if (tid < kBins && incl >= static_cast<uint32_t>(k)) atomicMin(&sh.digit, tid);
      __syncthreads();
      const uint32_t bin = sh.digit;
      // every maximum of the bins up to this one is above the bin's lower end
      b = bin < 255u ? max(key_of(M - (static_cast<float>(bin) + 1.01f) * per_bin), kNegInfKey + 1)
                     : kNegInfKey + 1;
    }
    listed = listed || b > kNegInfKey + 1;
    bound = max(bound, b);
  } else if (need_sum) {
    sum = row_sum();
    // the tokens below this hold less than 1 - p of the mass, were there V of them
    const float share = (1.f - top_p) * sum * (1.f - 0x1p-10f) / static_cast<float>(a.V);
    if (share > 0.f) {
      const float low = M + (__log2f(share) - 0x1p-10f) / K.h;
      bound = max(max(key_of(low), kmin), kNegInfKey + 1);
      listed = true;
    }
  }
  if (listed) {
    const float least = key_value(bound);
    if (tmax >= least) {
      for (int j = tid; j < s.n; j += kThreads) {
        float v[E::kVec];
        E::unpack(slice_mem[j], v);
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) {
          if (v[i] >= least) {
            const uint32_t at = remote_add(&sh.list_n, 0, 1u);
            if (at < kCap)
              cluster_store(cluster_addr(&sh.list.key[at], 0),
                            (static_cast<u64>(key_of(v[i])) << 32) |
                                static_cast<uint32_t>(~static_cast<uint32_t>(S.id_of(j, i))));
          }
        }
      }
    }
    cluster_arrive();
    cluster_wait();
    const uint32_t n = remote_load(&sh.list_n, 0);
    if (n <= kCap) {
      if (!need_sum) {
        // the others have nothing left to do; rank 0's memory was read before this
        cluster_arrive();
        if (rank != 0) return;
        S.set_scale(static_cast<float>(kCap));
        S.few(row, u, static_cast<int>(n), k, top_p, kmin, bound == kmin, 0.f);
        cluster_wait();
        return;
      }
      bool done = true;
      if (rank == 0) {
        S.set_scale(sum);
        done = S.few(row, u, static_cast<int>(n), k, top_p, kmin, bound == kmin, sum);
      }
      S.exchange(done ? 1 : 0, 0);
      if (S.got(0, 0) != 0) return;
    } else {
      cluster_arrive();  // rank 0's list is read no more: its memory serves the histograms
      cluster_wait();
    }
  }
  if (list_k) {  // the groups' sums were not taken
    sum = ex2_approx((tmax - M) * K.h);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    __syncthreads();
    if (lane == 0) sh.warpu[warp] = __float_as_uint(sum);
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < kWarps; ++i) sum += __uint_as_float(sh.warpu[i]);
    S.exchange(__float_as_uint(sum), 0);
    sum = 0.f;
    for (int c = 0; c < a.cluster; ++c) sum += __uint_as_float(static_cast<uint32_t>(S.got(c, 0)));
  } else if (!need_sum) {
    sum = row_sum();
  }
  S.set_scale(need_sum ? sum : sum * of_thread);
  S.wide(row, u, k, top_p, kmin);
  cluster_arrive();  // the others may still read this CTA's memory
  cluster_wait();
}

template <int kDtype, int kThreads>
cudaError_t launch_rows(const SampleArgs& a, int64_t T, const RowPlan& p, cudaStream_t stream) {
  const size_t smem = p.slice_bytes;
  auto* kernel = sample_kernel<kDtype, kThreads>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_clusters(kernel, T, p.cluster, kThreads, smem, stream, a);
}
template <int kDtype>
cudaError_t launch_type(SampleArgs a, int64_t T, cudaStream_t stream) {
  const RowPlan p = plan_row(a.V, sizeof(typename Elem<kDtype>::raw));
  a.cluster = p.cluster;
  return p.threads == 256 ? launch_rows<kDtype, 256>(a, T, p, stream)
                          : launch_rows<kDtype, 512>(a, T, p, stream);
}

}  // namespace

cudaError_t launch_sample(const void* logits, int dtype, int64_t ld, int64_t T, int V,
                          const float* uniform, const tim_sample_params& p, int32_t* ids,
                          float* logprob, float* lse, int32_t* kept, int* status,
                          cudaStream_t stream) {
  const SampleArgs a = {logits, ld, V, 1, uniform, p.temperature, p.top_k, p.top_p, p.min_p,
                        p.row_temperature, p.row_top_k, p.row_top_p, p.row_min_p, ids, logprob,
                        lse, kept, status};
  return dtype == TIM_F32    ? launch_type<TIM_F32>(a, T, stream)
         : dtype == TIM_BF16 ? launch_type<TIM_BF16>(a, T, stream)
                             : launch_type<TIM_F16>(a, T, stream);
}

}  // namespace tim
