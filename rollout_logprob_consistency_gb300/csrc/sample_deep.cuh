// The sampler's rows that no short list decides, by one CTA: a nucleus of thousands of tokens, a
// large top-k, ties at a border, a top-p border within the fp32 sum's error, the unfiltered row.
//
// The row was read once from memory and comes from L2 from here on.  What is kept is "key above a
// border key, or equal to it with an id up to a border id"; the token is found by running sums over
// 32 parts of the row.  A border takes two passes.  The first sums the tokens' masses (fp32, as
// 32-bit integers), or counts them, in bins of 1/64 octave: the border is then in one bin, or two.
// The second sums the integer weights of all, and of those above these bins part by part, and lists
// the tokens within; sorted and walked, they give the border exactly, and what each part keeps.
// Where the list would be too long (thousands of tokens of one value) or the bins do not hold the
// border, it is found digit by digit of the keys with histograms of counts or integer weights, which
// serves every row.
//
// Bound by the issue of the weights' integer arithmetic, some 27 instructions a token.  A row of 151936
// fp32 logits in a CTA of 1024 threads takes 65 us with its stream: bins 12, weights 27, list and border
// 8, draw 4; 128 rows of top-p 0.95 in temperature 0.7 take 84 us.  A second launch with a cluster of
// eight CTAs a row took 50 us a row on four SMs and 187 us for these.  512 unfiltered rows of bf16 logits
// take 91 us, at 0.8 instructions a cycle and scheduler on the SMs that have four of them.
#pragma once

#include "sample.cuh"

namespace tim {
namespace sampling {

constexpr int kDeepBins = 256;
constexpr int kBins = 2048;     // of 1/64 octave
constexpr int kDeepCap = 2048;  // tokens of the border's bins
constexpr int kSteps = 128;     // 32-vector steps of a 32nd of the row, of 98305 vectors at most: 97

struct DeepShared {
  union {
    uint32_t bin[kBins + 32];
    u64 list[kDeepCap];  // key << 32 | ~id
    struct {
      uint32_t count[2][kDeepBins], lo[2][kDeepBins], hi[2][kDeepBins];
    } sel;
    u64 step[kSteps];  // sums over 32 vectors each, of one part
  };
};
struct DeepScratch {
  uint32_t part_lo[32], part_hi[32];
  int part_e[32];
  int bin_lo, bin_hi, found;
  uint32_t list_n, digit, in;
  u64 acc, border;
  int all;
};

template <int kDtype, int kThreads>
struct Deep {
  using E = Elem<kDtype>;
  static constexpr int kVec = E::kVec;
  static constexpr int kWarps = kThreads / 32;
  // Vectors of a thread: with four of 16-bit logits the border's passes spill (98 us a row against 88),
  // the unfiltered row's does not and is faster for it (512 rows 91 us against 100).
  static constexpr int kInFlight = kVec == 8 ? 2 : 4;
  static constexpr int kStream = 4;
  static constexpr int kParts = 32;    // of the row, for its running sums

  const SampleArgs& a;
  DeepShared& sh;
  DeepScratch& sc;
  const Tables& table;
  u64* warp64;       // 32: of the row's parts
  u64* total64;      // kWarps
  uint32_t* warp32;  // kWarps
  const Row<kDtype>& r;
  RowState st;
  int tid, warp, lane;

  __device__ __forceinline__ int id_of(int j, int i) const { return j * kVec + i - r.shift; }
  __device__ __forceinline__ bool in_row(int id) const { return id >= 0 && id < a.V; }

  // f(x, j) of the row's vectors j0, j0 + stride, ... below end; slots that are not the row's hold -inf.
  template <class F>
  __device__ __forceinline__ void each(int j0, int end, int stride, F&& f) const {
    const int w0 = r.w0(), w1 = r.w1();
    const uint4* const vec = r.vec();
    for (; j0 < end; j0 += kInFlight * stride) {
      uint4 x[kInFlight];
#pragma unroll
      for (int n = 0; n < kInFlight; ++n) {
        const int j = j0 + n * stride;
        if (j >= w0 && j < min(w1, end))
          x[n] = __ldg(vec + j);
        else if (j < end)
          x[n] = r.load_edge(j);
      }
#pragma unroll
      for (int n = 0; n < kInFlight; ++n)
        if (j0 + n * stride < end) f(x[n], j0 + n * stride);
    }
  }

  // ---- sums over the row in 32 contiguous parts, of steps of 32 vectors; a warp has one or more.
  __device__ __forceinline__ int part() const {
    return (r.nvec() + kParts * 32 - 1) / (kParts * 32) * 32;
  }

  // The sum of f(v, id0) over the row's vectors; warp64[] gets the parts' sums.
  template <class F>
  __device__ __forceinline__ u64 row_sum(F&& f) {
    __syncthreads();
    for (int p = warp; p < kParts; p += kWarps) {
      const int j0 = p * part(), j1 = min(r.nvec(), j0 + part());
      u64 sum = 0;
      each(j0 + lane, j1, 32, [&](const uint4& x, int j) {
        float v[kVec];
        E::unpack(x, v);
        sum += f(v, id_of(j, 0));
      });
      sum = warp_sum(sum);
      if (lane == 0) warp64[p] = sum;
    }
    __syncthreads();
    return warp_sum(warp64[lane]);
  }
  // The token at which the running sum first exceeds `target` (below the row's sum), in every
  // thread; after row_sum(f), by the whole CTA.  one(z, id) is a token's number.  The parts' sums may
  // be more than their tokens' by a rounding; a part with a sum has a token with one.
  template <class F, class G>
  __device__ __forceinline__ int locate(u64 target, F&& f, G&& one) {
    const u64 of = warp64[lane], to_here = warp_scan(of);
    const int w = min(__popc(__ballot_sync(0xFFFFFFFFu, target >= to_here)), kParts - 1);
    target -= __shfl_sync(0xFFFFFFFFu, to_here - of, w);
    const int j0 = w * part(), j1 = min(r.nvec(), j0 + part()), steps = (j1 - j0 + 31) / 32;
    // lanes beyond the part's end take part in the sums
    const int last = j0 + steps * 32;
    each(j0 + tid, last, kThreads, [&](const uint4& x, int j) {
      u64 sum = 0;
      if (j < j1) {
        float v[kVec];
        E::unpack(x, v);
        sum = f(v, id_of(j, 0));
      }
      sum = warp_sum(sum);
      if (lane == 0) sh.step[(j - j0) >> 5] = sum;
    });
    __syncthreads();
    u64 there = 0;
    for (int i = lane; i < steps; i += 32) there += sh.step[i];
    target = min(target, warp_sum(there) - 1);
    int i = 0;
    for (;; i += 32) {
      const u64 x = i + lane < steps ? sh.step[i + lane] : 0, at = warp_scan(x);
      const unsigned past = __ballot_sync(0xFFFFFFFFu, target < at);
      const int to = past != 0 ? __ffs(past) - 1 : 31;
      if (past != 0 || i + 32 >= steps) {
        target -= __shfl_sync(0xFFFFFFFFu, at - x, to);
        i += to;
        break;
      }
      target -= __shfl_sync(0xFFFFFFFFu, at, 31);
    }
    if (warp == 0) {
      const int j = j0 + i * 32 + lane;
      u64 x[kVec], sum = 0;
      float v[kVec];
      const int id0 = id_of(j, 0);
      if (j < j1) E::unpack(r.load(j), v);
#pragma unroll
      for (int q = 0; q < kVec; ++q) {
        x[q] = j < j1 ? one(v[q], id0 + q) : 0;
        sum += x[q];
      }
      u64 at = warp_scan(sum) - sum;
#pragma unroll
      for (int q = 0; q < kVec; ++q) {
        if (at <= target && target < at + x[q]) sc.found = id0 + q;
        at += x[q];
      }
    }
    __syncthreads();
    return sc.found;
  }

  // A 64-bit shared-memory sum from two 32-bit ones.
  static __device__ __forceinline__ void add_weight(uint32_t* lo, uint32_t* hi, u64 w) {
    const uint32_t wl = static_cast<uint32_t>(w);
    const uint32_t old = atomicAdd(lo, wl);
    const uint32_t wh = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
    if (wh != 0) atomicAdd(hi, wh);
  }

  // An upper bound, near enough, of the sum of all weights relative to the largest, in every thread.
  __device__ __forceinline__ float bound() const {
    float most = 0.f;
    each(tid, r.nvec(), kThreads, [&](const uint4& x, int) {
      float v[kVec];
      E::unpack(x, v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) most += ex2_approx((v[i] - st.M) * st.pw.kh);
    });
    return total_of(most);
  }
  __device__ __forceinline__ float total_of(float most) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most += __shfl_xor_sync(0xFFFFFFFFu, most, o);
    __syncthreads();
    if (lane == 0) warp32[warp] = __float_as_uint(most);
    __syncthreads();
    most = lane < kWarps ? __uint_as_float(warp32[lane]) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most += __shfl_xor_sync(0xFFFFFFFFu, most, o);
    __syncthreads();
    return fmaxf(most, 1.f) * 1.001f;
  }

  // ---- the border by digits.  Among the tokens that the state keeps: the last one before which
  // the measure (1, or with kMass the weight) is below `target`; the state then keeps up to it.
  template <bool kMass>
  __device__ __forceinline__ void select_border(u64 target) {
    uint32_t prefix = 0, in = 0;
    u64 acc = 0;
    const uint32_t kc = st.kc;
    const int idc = st.idc;
    for (int level = 0; level < kLevels<kDtype>; ++level) {
      const int shift = 24 - 8 * level, b = level & 1;
      __syncthreads();
      for (int i = tid; i < kDeepBins; i += kThreads)
        sh.sel.count[b][i] = sh.sel.lo[b][i] = sh.sel.hi[b][i] = 0;
      if (tid == 0) sc.all = 1;
      __syncthreads();
      each(tid, r.nvec(), kThreads, [&](const uint4& x, int j) {
        float v[kVec];
        E::unpack(x, v);
        const int id0 = id_of(j, 0);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const uint32_t key = key_of(v[i]);
          if (level > 0 && (key >> (shift + 8)) != prefix) continue;
          if (!(key > kc || (key == kc && id0 + i <= idc))) continue;
          const int d = (key >> shift) & 255;
          atomicAdd(&sh.sel.count[b][d], 1u);
          if (kMass) add_weight(&sh.sel.lo[b][d], &sh.sel.hi[b][d], weight(v[i], st, table));
        }
      });
      __syncthreads();
      // digits from the top, kOf of a thread
      constexpr int kOf = kThreads >= kDeepBins ? 1 : kDeepBins / kThreads;
      u64 h[kOf], sum = 0;
#pragma unroll
      for (int q = 0; q < kOf; ++q) {
        const int d = kDeepBins - 1 - (tid * kOf + q);
        h[q] = d < 0 ? 0
               : kMass ? (static_cast<u64>(sh.sel.hi[b][d]) << 32) + sh.sel.lo[b][d]
                       : sh.sel.count[b][d];
        sum += h[q];
      }
      u64 before = warp_scan(sum);
      if (lane == 31) total64[warp] = before;
      __syncthreads();
      before += acc - sum;
      for (int i = 0; i < warp; ++i) before += total64[i];
#pragma unroll
      for (int q = 0; q < kOf; ++q) {
        if (before < target && target <= before + h[q]) {
          const int d = kDeepBins - 1 - (tid * kOf + q);
          sc.digit = d;
          sc.acc = before;
          sc.in = sh.sel.count[b][d];
          sc.all = 0;
        }
        before += h[q];
      }
      __syncthreads();
      if (sc.all != 0) return;  // fewer than the target: every one of them stays
      prefix = (prefix << 8) | sc.digit;
      acc = sc.acc;
      in = sc.in;
    }
    const int rest = 32 - 8 * kLevels<kDtype>;
    uint32_t key = rest == 0 ? prefix : prefix << rest;
    if (rest != 0 && !(key & 0x80000000u)) key |= (1u << rest) - 1u;  // a negative number's
    // the border key's tokens have equal measures: how many of them, in id order
    const u64 w = kMass ? max(weight(key_value(key), st, table), 1ull) : 1ull;
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
    row_sum(ties);
    const int id = locate(want - 1, ties, tie);
    st.kc = key;
    st.idc = id;
  }

  __device__ __forceinline__ u64 kept_weight(float z, int id) const {
    return keeps(key_of(z), id, st) && in_row(id) ? weight(z, st, table) : 0;
  }
  // The logits that the state does not keep become -inf.
  __device__ __forceinline__ void drop(float (&v)[kVec], int id0, float zc) const {
    if (st.idc == INT32_MAX) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = v[i] >= zc ? v[i] : -INFINITY;
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        v[i] = v[i] > zc || (v[i] == zc && id0 + i <= st.idc) ? v[i] : -INFINITY;
    }
  }
  // Sum of weights, without recentring.
  __device__ __forceinline__ u64 weights_of(const float (&v)[kVec], uint32_t shift) const {
    u64 t = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) t += weight_at(v[i], st.pw.kh, st.pw.kl, shift, table.t);
    return t;
  }
  // The border by bins: the last kept token before which there are less than k tokens, or (kMass)
  // less than p of the kept weights.  `most` bounds the sum of the weights relative to the largest.
  // With kMass warp64[] then holds what the parts of the row keep, and `kept` how many tokens.
  // False: not found this way (the state is as before).
  template <bool kMass>
  __device__ __forceinline__ bool narrow(int k, float p, float most, uint32_t& kept) {
    const uint32_t shift = shift_of(st.top);
    const float zc = key_value(st.kc), M = st.M;
    const bool whole = st.kc == kNegInfKey;  // nothing is dropped yet
    const int nvec = r.nvec();
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) sh.bin[i] = 0;
    if (tid < 32) sc.part_lo[tid] = sc.part_hi[tid] = 0;
    if (tid == 0) {
      sc.list_n = 0;
      sc.bin_lo = sc.bin_hi = kBins;
      sc.all = 1;
    }
    __syncthreads();
    // ---- the bins.  Masses at a scale at which they sum to 2^30 up to 2^32, each rounded to a whole unit:
    // V / 2 of them, 7e-5 of the sum at V = 151936 and within the 2^-13 below up to V = 262144.  Where the
    // error is larger the list may not hold the border, which shows, and digits find it.
    const float per = 64.f * st.pw.kh, scale = static_cast<float>(30 - ilogbf(most));
    each(tid, nvec, kThreads, [&](const uint4& x, int j) {
      float v[kVec];
      E::unpack(x, v);
      if (!whole) drop(v, id_of(j, 0), zc);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float d = M - v[i];
        const int b = __float_as_int(fmaf(d, per, kUnitMagic)) - __float_as_int(kUnitMagic);
        const uint32_t m = kMass ? __float2uint_rn(ex2_approx(fmaf(-d, st.pw.kh, scale))) : 1u;
        // all that is far below: not to one word
        atomicAdd(&sh.bin[b < kBins ? b : kBins + lane], m);
      }
    });
    __syncthreads();
    constexpr int kPer = kBins / kThreads;
    uint32_t n[kPer], at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) at += n[i] = sh.bin[tid * kPer + i];
    uint32_t sum = at;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, at, o);
      if (lane >= o) at += up;
    }
    if (lane == 31) warp32[warp] = at;
    __syncthreads();
    at -= sum;
    uint32_t all = 0;
    for (int i = 0; i < kWarps; ++i) {
      all += warp32[i];
      if (i < warp) at += warp32[i];
    }
    // the first bins at which the target may and must be reached
    const float want = kMass ? p * static_cast<float>(all) : 0.f;
    const uint32_t least = kMass ? static_cast<uint32_t>(want * (1.f - 0x1p-13f)) : static_cast<uint32_t>(k);
    const uint32_t sure = kMass ? min(static_cast<uint32_t>(want * (1.f + 0x1p-13f)) + 1u, all)
                                : static_cast<uint32_t>(k);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t past = at + n[i];
      if (n[i] != 0 && at < sure && sure <= past) sc.bin_hi = tid * kPer + i;
      if (n[i] != 0 && (at < least || at == 0) && least <= past) sc.bin_lo = tid * kPer + i;
      at = past;
    }
    __syncthreads();
    const int lo = sc.bin_lo, hi = sc.bin_hi;
    if (lo > hi || hi >= kBins) return false;
    // a bin holds (M - z) per from half below it to half above
    const float z_hi = M - (static_cast<float>(lo) - 0.51f) / per;
    const float z_lo = M - (static_cast<float>(hi) + 0.51f) / per;

    // ---- the weights of all, of those above in each part, and the tokens within
    u64 mine = 0;
    float count = 0.f;  // of those above
    for (int q = warp; q < kParts; q += kWarps) {
      const int j0 = q * part(), j1 = min(nvec, j0 + part());
      u64 above = 0;
      each(j0 + lane, j1, 32, [&](const uint4& x, int j) {
        float v[kVec];
        E::unpack(x, v);
        if (!whole) drop(v, id_of(j, 0), zc);
        bool some = false;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const bool over = v[i] >= z_hi;
          if (kMass) {
            const u64 w = weight_at(v[i], st.pw.kh, st.pw.kl, shift, table.t);
            mine += w;
            if (over) above += w;
          }
          if (over) count += 1.f;
          some |= !over && v[i] >= z_lo;
        }
        if (some) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            if (v[i] < z_lo || v[i] >= z_hi) continue;
            const uint32_t to = atomicAdd(&sc.list_n, 1u);
            if (to < kDeepCap)
              sh.list[to] = (static_cast<u64>(key_of(v[i])) << 32) |
                            static_cast<uint32_t>(~static_cast<uint32_t>(id_of(j, i)));
          }
        }
      });
      if (kMass) {
        above = warp_sum(above);
        if (lane == 0) warp64[q] = above;
      }
    }
    mine = warp_sum(mine);
    const uint32_t warp_n = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(count));
    __syncthreads();
    if (lane == 0) {
      warp32[warp] = warp_n;
      if (kMass) total64[warp] = mine;
    }
    __syncthreads();
    const int len = static_cast<int>(sc.list_n);
    if (len > kDeepCap) return false;
    uint32_t over = 0;
    u64 total = 0;
    for (int i = 0; i < kWarps; ++i) {
      over += warp32[i];
      if (kMass) total += total64[i];
    }
    const u64 acc = kMass ? warp_sum(warp64[lane]) : over;
    const u64 target = kMass ? top_p_target(total, p) : static_cast<u64>(k);

    // ---- the list in order, and the last token before which there is less than the target
    int n2 = 64;
    while (n2 < len) n2 <<= 1;
    for (int i = len + tid; i < n2; i += kThreads) sh.list[i] = 0;
    __syncthreads();
    sort_desc<kThreads>(sh.list, n2);
    constexpr int kOf = kDeepCap / kThreads;
    const int of = (n2 + kThreads - 1) / kThreads;  // of a thread
    u64 w[kOf], here = 0;
#pragma unroll
    for (int q = 0; q < kOf; ++q) {
      const int i = tid * of + q;
      w[q] = q >= of || i >= len ? 0
             : kMass             ? weight(key_value(static_cast<uint32_t>(sh.list[i] >> 32)), st, table)
                                 : 1;
      here += w[q];
    }
    u64 before = warp_scan(here);
    if (lane == 31) total64[warp] = before;
    __syncthreads();
    before += acc - here;
    for (int i = 0; i < warp; ++i) before += total64[i];
#pragma unroll
    for (int q = 0; q < kOf; ++q) {
      const int i = tid * of + q;
      if (before < target && w[q] != 0) {
        if (before + w[q] >= target) {
          sc.border = sh.list[i];
          sc.in = static_cast<uint32_t>(i) + 1;
          sc.all = 0;
        }
        if (kMass) {
          const int id = static_cast<int>(~static_cast<uint32_t>(sh.list[i]));
          const int to = (id + r.shift) / kVec / part();
          add_weight(&sc.part_lo[to], &sc.part_hi[to], w[q]);
        }
      }
      before += w[q];
    }
    __syncthreads();
    if (sc.all != 0 || acc >= target) return false;
    st.kc = static_cast<uint32_t>(sc.border >> 32);
    st.idc = static_cast<int>(~static_cast<uint32_t>(sc.border));
    kept = over + sc.in;
    if (kMass && warp == 0)
      warp64[lane] += (static_cast<u64>(sc.part_hi[lane]) << 32) + sc.part_lo[lane];
    __syncthreads();
    return true;
  }

  // The draw, f and one being the kept tokens' weights, of `n` tokens; after row_sum(f).
  template <class F, class G>
  __device__ __forceinline__ void draw(int64_t row, float u, u64 total, uint32_t n, F&& f, G&& one) {
    const int id = locate(draw_target(total, u), f, one);
    if (tid == 0) write_row(a, st, table, row, id, r.at(id), total, static_cast<int>(n));
  }
  // Sum of a count over the CTA's threads.
  __device__ __forceinline__ uint32_t count_all(uint32_t n) {
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    __syncthreads();
    if (lane == 0) warp32[warp] = n;
    __syncthreads();
    return __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? warp32[lane] : 0u);
  }

  // ---- the filtered row
  __device__ __forceinline__ void filtered(int64_t row, float u, int k, float top_p, uint32_t kmin,
                                           float most) {
    st.kc = kNegInfKey;
    st.idc = INT32_MAX;
    auto one = [&](float z, int id) { return kept_weight(z, id); };
    uint32_t n = 0;
    if (k > 0 && (st.pw.recentre || !narrow<false>(k, 0.f, most, n)))
      select_border<false>(static_cast<u64>(k));
    bool summed = false;  // the parts of what is kept
    if (top_p < 1.f) {
      summed = !st.pw.recentre && narrow<true>(0, top_p, most, n);
      if (!summed) {
        const u64 total = row_sum([&](const float(&v)[kVec], int id0) {
          u64 t = 0;
#pragma unroll 1
          for (int i = 0; i < kVec; ++i) t += one(v[i], id0 + i);
          return t;
        });
        select_border<true>(top_p_target(total, top_p));
      }
    }
    if (kmin > st.kc) {
      st.kc = kmin;
      st.idc = INT32_MAX;
      summed = false;
    }
    const float zc = key_value(st.kc);
    auto finish = [&](auto&& kept) {
      u64 total;
      uint32_t all = n;
      if (summed) {
        total = warp_sum(warp64[lane]);
      } else {
        n = 0;
        total = row_sum(kept);
        all = count_all(n);
      }
      draw(row, u, total, all, kept, one);
    };
    if (st.pw.recentre) {
      finish([&](const float(&v)[kVec], int id0) {
        u64 t = 0;
#pragma unroll 1
        for (int i = 0; i < kVec; ++i) {
          n += keeps(key_of(v[i]), id0 + i, st) && in_row(id0 + i) ? 1 : 0;
          t += one(v[i], id0 + i);
        }
        return t;
      });
    } else {
      const uint32_t shift = shift_of(st.top);
      // what a vector keeps; slots that are not the row's hold -inf
      finish([&](const float(&x)[kVec], int id0) {
        float v[kVec];
        uint32_t here = 0;
        if (st.idc == INT32_MAX) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) here += x[i] >= zc ? 1 : 0;
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i) here += x[i] > zc || (x[i] == zc && id0 + i <= st.idc) ? 1 : 0;
        }
        if (here == 0) return static_cast<u64>(0);
        n += here;
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = x[i];
        drop(v, id0, zc);
        return weights_of(v, shift);
      });
    }
  }

  // ---- the unfiltered row: all tokens but those of -inf are kept.  One pass from memory: a lane sums
  // at a scale of its own, 2^(51 - e) with e at or above its largest x = z K, shifted right where e
  // grows; at most 2^11.6 tokens of a lane, so below 2^63.  A part's sum is that of its lanes' at
  // 2^(46 - e) for the largest e, below 2^63 again, and off by 2^-40 of the row's at most.
  __device__ __forceinline__ void plain(int64_t row, float u, int bad) {
    const int w0 = r.w0(), w1 = r.w1(), nvec = r.nvec();
    const uint4* const vec = r.vec();
    uint4 high = neg_inf_vec<kDtype>(), low = high;  // of all the lane's vectors so far
    bool first = true;
    uint32_t n = 0;
    int e = INT32_MIN / 4;
    for (int q = warp; q < kParts; q += kWarps) {
      const int end = min(nvec, (q + 1) * part());
      u64 sum = 0;
      for (int j0 = q * part() + lane; j0 < end; j0 += kStream * 32) {
        uint4 x[kStream];
#pragma unroll
        for (int i = 0; i < kStream; ++i) {
          const int j = j0 + i * 32;
          if (j >= w0 && j < min(w1, end))
            x[i] = __ldg(vec + j);
          else
            x[i] = j < end ? r.load_edge(j) : j0 >= w0 && j0 < w1 ? x[0] : neg_inf_vec<kDtype>();
        }
        if (first) low = x[0];
        first = false;
        const uint4 was = high;
#pragma unroll
        for (int i = 0; i < kStream; ++i) {
          high = max_vec<kDtype>(high, x[i]);
          low = min_vec<kDtype>(low, x[i]);
        }
        if (((high.x ^ was.x) | (high.y ^ was.y) | (high.z ^ was.z) | (high.w ^ was.w)) != 0) {
          const int ceil_x = min(__float2int_ru(fmaf(max_of<kDtype>(high), st.pw.kh, 0.01f)), 1 << 20);
          if (ceil_x > e) {
            sum = ceil_x - e < 64 ? sum >> (ceil_x - e) : 0;
            e = ceil_x;
          }
        }
        const uint32_t shift = shift_of(e + 11);
#pragma unroll
        for (int i = 0; i < kStream; ++i) {
          float v[kVec];
          E::unpack(x[i], v);
          const u64 w = weights_of(v, shift);
          if (j0 + i * 32 < end) sum += w;
        }
      }
      const int most_e = __reduce_max_sync(0xFFFFFFFFu, e);
      sum = warp_sum((sum >> 5) >> min(most_e - e, 63));
      if (lane == 0) {
        warp64[q] = sum;
        sc.part_e[q] = most_e;
      }
    }
    // the tokens above -inf: a lane that has met none of it has its vectors' slots
    for (int q = warp; q < kParts; q += kWarps) {
      const int j0 = q * part() + lane, end = min(nvec, (q + 1) * part());
      if (j0 >= end) continue;
      if (min_of<kDtype>(low) > -INFINITY) {
        n += static_cast<uint32_t>((end - j0 + 31) / 32) * kVec;
      } else {
        each(j0, end, 32, [&](const uint4& x, int) {
          float v[kVec];
          E::unpack(x, v);
#pragma unroll
          for (int c = 0; c < kVec; ++c) n += v[c] > -INFINITY ? 1 : 0;
        });
      }
    }
    const float tmax = max_of<kDtype>(high);
    uint32_t key = !(tmax < INFINITY) ? 0xFFFFFFFFu : key_of(tmax);
    key = __reduce_max_sync(0xFFFFFFFFu, key);
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) {
      warp32[warp] = key;
      total64[warp] = n;
    }
    __syncthreads();
    key = __reduce_max_sync(0xFFFFFFFFu, lane < kWarps ? warp32[lane] : 0u);
    n = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? static_cast<uint32_t>(total64[lane]) : 0u);
    if (bad == 0 && (key == 0xFFFFFFFFu || key <= kNegInfKey)) bad = TIM_ERR_NONFINITE;
    if (bad != 0) {
      if (tid == 0) write_bad(a, row, bad);
      return;
    }
    st.M = key_value(key);
    auto one = [&](float z, int) { return weight(z, st, table); };
    if (!(fabsf(st.M * st.pw.kh) < 8000.f)) {
      // beyond what weight_at splits: again, relative to the largest
      set_scale(st, bound());
      auto all = [&](const float(&v)[kVec], int) {
        u64 t = 0;
#pragma unroll 1
        for (int i = 0; i < kVec; ++i) t += one(v[i], 0);
        return t;
      };
      const u64 total = row_sum(all);
      draw(row, u, total, n, all, one);
      return;
    }
    // the row's scale: its total at 2^58 or 2^59
    const int part_e = sc.part_e[lane], most_e = __reduce_max_sync(0xFFFFFFFFu, part_e);
    const u64 mine = warp64[lane];
    const u64 about = warp_sum((mine >> 5) >> min(most_e - part_e, 63));  // at 2^(41 - most_e)
    st.pw.recentre = false;
    st.pw.c = 0.f;
    st.top = most_e - 41 + 63 - __clzll(static_cast<long long>(about)) + 4;
    // The parts at that scale, 2^(62 - top).  One that has less than 2^14 units, 2^-44 of the row, might
    // have no token of a whole one (2^13.6 tokens a part at most) and is left out.
    const int d = 16 + part_e - st.top;
    u64 scaled = d >= 0 ? mine << min(d, 63) : mine >> min(-d, 63);
    if (scaled < 16384) scaled = 0;
    __syncthreads();
    if (warp == 0) warp64[lane] = scaled;
    const uint32_t shift = shift_of(st.top);
    const u64 total = warp_sum(scaled);
    __syncthreads();
    draw(row, u, total, n, [&](const float(&v)[kVec], int) { return weights_of(v, shift); }, one);
  }
};

}  // namespace sampling
}  // namespace tim
