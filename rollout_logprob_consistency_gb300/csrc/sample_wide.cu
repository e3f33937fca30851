// The sampler's rows that no short list decides: the unfiltered row, a nucleus of thousands of
// tokens, a large top-k, ties at a border.
//
// A row is held in shared memory by a cluster of CTAs, a slice each.  What is kept is "key above
// a border key, or equal to it with an id up to a border id", the token is found by running sums.
// The border is found in three passes over the slices.  The first counts the tokens in bins of
// 1/32 octave of their weight: the counts place the border in one bin (top-k) or, a bin's weights
// being within 2.2% of one another, in a few (top-p).  The second sums the integer weights of all
// and of those above these bins, and counts and sums in bins of 1/256 octave (or more) within them: the border's is then known exactly.  The third lists the tokens of that one; rank 0 sorts
// the list and walks it.  Where the list would be too long (thousands of tokens of one value) or
// the border lies among tokens without weight, the border is found digit by digit of the
// keys with histograms of counts or integer weights, which serves every row.
// A thread's largest logit gives the scale: the sum over the threads of (largest weight x
// elements) bounds the row's total, and is at most that many times too large.
#include <type_traits>

#include "sample.cuh"

namespace tim {

using namespace sampling;

namespace {

constexpr int kBins = 256;
constexpr int kMaxCluster = 8;
constexpr int kCoarse = 2048;  // bins of 1/32 octave
constexpr int kFine = 1024;    // bins of 1/256 octave and more
constexpr int kCap = 1024;     // tokens of one fine bin
constexpr int kMaxSteps = 64;  // 32-vector steps of a warp's part: at most 24580 vectors over 16 warps

struct WideArgs : SampleArgs {
  int64_t T;
  int cluster;
};

__device__ __forceinline__ uint32_t remote_load(const void* smem, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(smem, rank)) : "memory");
  return v;
}
struct Select {  // the wide way's histograms
  uint32_t count[2][kBins], lo[2][kBins], hi[2][kBins];
};
struct Fine {  // counts and integer weights, in two words, of the fine bins
  alignas(16) uint32_t count[kFine];
  alignas(16) uint32_t lo[kFine];
  alignas(16) uint32_t hi[kFine];
};

// What finding a border takes; the kernel for unfiltered rows goes without.
struct Border {
  union {
    Select sel;
    Fine fine;
  };
  union {
    alignas(16) uint32_t coarse[kCoarse];
    u64 list[kCap];  // key << 32 | ~id; rank 0's takes all CTAs'
  };
  float warpf[2][16];
  int bin_lo, bin_hi;
  uint32_t list_n, above, digit, in;
  u64 acc;
  int all;
};
struct NoBorder {};
template <int kThreads, bool kPlain>
struct Shared : std::conditional_t<kPlain, NoBorder, Border> {
  u64 table[256];
  u64 xch[2][kMaxCluster][2];
  // of every warp of every CTA: largest key, and the threads' largest weights relative to it
  uint32_t gkey[kMaxCluster * kThreads / 32];
  float gsum[kMaxCluster * kThreads / 32];
  u64 warp[kThreads / 32];
  uint32_t warpu[kThreads / 32], warpv[kThreads / 32];
  u64 step[kMaxSteps];  // sums over 32 vectors each, of one warp's part
  int found;
  uint64_t bar;
};

__device__ __forceinline__ uint2 remote_load2(const void* smem, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(cluster_addr(smem, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 remote_load4(const void* smem, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_addr(smem, rank))
               : "memory");
  return v;
}
template <int kDtype, int kThreads, bool kPlain>
struct Sampler {
  using E = Elem<kDtype>;
  static constexpr int kVec = E::kVec;
  static constexpr int kWarps = kThreads / 32;

  const WideArgs& a;
  Shared<kThreads, kPlain>& sh;
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
          if (kMass)
            add_weight(&sh.sel.lo[b][d], &sh.sel.hi[b][d], weight(v[i], st, sh.table));
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

  // ---- without recentring: vectors at once
  __device__ __forceinline__ Pow2Pair pair() const {
    return {f2(st.pw.kh, st.pw.kh), f2(st.pw.kl, st.pw.kl),
            static_cast<uint32_t>(st.top) + (__float_as_uint(kPow2Magic) >> 8)};
  }
  // The logits that the state does not keep become one without weight.
  __device__ __forceinline__ void drop(float (&v)[kVec], int id0, float zc) const {
    const float zlow = st.zlow;
    if (st.idc == INT32_MAX) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = v[i] >= zc ? fmaxf(v[i], zlow) : zlow;
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        v[i] = v[i] > zc || (v[i] == zc && id0 + i <= st.idc) ? fmaxf(v[i], zlow) : zlow;
    }
  }
  // Sum of the weights of logits from zlow up.
  __device__ __forceinline__ u64 weights_of(const float (&v)[kVec], const Pow2Pair& k) const {
    u64 t = 0;
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
      u64 w0, w1;
      pow2_shifted(f2(v[i], v[i + 1]), k, sh.table, w0, w1);
      t += w0 + w1;
    }
    return t;
  }
  // Where a logit from zlow up lies, in 1/256 octaves below 2^N, N the whole number above max K.
  // Never lower for a lower logit: the product and its rounding are monotone.
  __device__ __forceinline__ int place_base() const {
    return __float_as_int(kPow2Magic) + (static_cast<int>(ceilf((df(st.M) * Df{st.pw.kh, st.pw.kl}).h)) << 8);
  }
  __device__ __forceinline__ int place_of(float z, int base) const {
    return max(base - __float_as_int(fmaf(z, st.pw.kh, kPow2Magic)), 0);
  }
  // A 64-bit shared-memory sum from two 32-bit ones.
  static __device__ __forceinline__ void add_weight(uint32_t* lo, uint32_t* hi, u64 w) {
    const uint32_t wl = static_cast<uint32_t>(w);
    const uint32_t old = atomicAdd(lo, wl);
    const uint32_t wh = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
    if (wh != 0) atomicAdd(hi, wh);
  }
  // Sum of a value over the CTA's threads, in all of them.
  __device__ __forceinline__ u64 cta_sum(u64 v) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = v;
    __syncthreads();
    u64 t = 0;
    for (int i = 0; i < kWarps; ++i) t += sh.warp[i];
    return t;
  }
  // The kept logits of vector j, the others without weight.
  __device__ __forceinline__ void kept_vector(int j, float zc, bool whole, float (&v)[kVec]) const {
    E::unpack(slice[j], v);
    if (whole) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = fmaxf(v[i], st.zlow);
    } else {
      drop(v, id_of(j, 0), zc);
    }
  }

  // f(i, word i) of a thread's fine bins in another CTA, one load.
  template <class F>
  static __device__ __forceinline__ void remote_fine(const uint32_t* at, int c, F&& f) {
    static_assert(kFine / kThreads == 4 || kFine / kThreads == 2, "one load a thread");
    if constexpr (kFine / kThreads == 4) {
      const uint4 x = remote_load4(at, c);
      f(0, x.x);
      f(1, x.y);
      f(2, x.z);
      f(3, x.w);
    } else {
      const uint2 x = remote_load2(at, c);
      f(0, x.x);
      f(1, x.y);
    }
  }

  // The border by bins: the last kept token before which there are less than k tokens, or (kMass)
  // less than p of the kept weights.  False: not found this way (the state is as before).
  template <bool kMass>
  __device__ bool narrow(int k, float p) {
    const Pow2Pair pw = pair();
    const int base = place_base();
    const float zc = key_value(st.kc);
    const bool whole = st.kc == kNegInfKey;  // nothing is dropped yet
    for (int i = tid; i < kCoarse; i += kThreads) sh.coarse[i] = 0;
    for (int i = tid; i < kFine; i += kThreads) sh.fine.count[i] = sh.fine.lo[i] = sh.fine.hi[i] = 0;
    if (tid == 0) {
      sh.list_n = 0;
      sh.bin_lo = sh.bin_hi = kCoarse;
    }
    __syncthreads();
    // ---- the coarse counts
    for (int j = tid; j < s.n; j += kThreads) {
      float v[kVec];
      kept_vector(j, zc, whole, v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) atomicAdd(&sh.coarse[min(place_of(v[i], base) >> 3, kCoarse - 1)], 1u);
    }
    // from this bin on there are tokens without weight, or dropped
    const int low = min(place_of(st.zlow, base) >> 3, kCoarse - 1);
    cluster_arrive();
    cluster_wait();
    // this thread's bins, of all CTAs; their running counts and bounds of their mass
    constexpr int kPer = kCoarse / kThreads;
    uint32_t n[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) n[i] = 0;
    for (int c = 0; c < a.cluster; ++c) {
#pragma unroll
      for (int i = 0; i < kPer; i += 4) {
        const uint4 x = remote_load4(&sh.coarse[tid * kPer + i], c);
        n[i] += x.x;
        n[i + 1] += x.y;
        n[i + 2] += x.z;
        n[i + 3] += x.w;
      }
    }
    uint32_t count = 0;
    float f_lo = 0.f, f_hi = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      count += n[i];
      if (kMass) {
        const float x = -static_cast<float>(8 * (tid * kPer + i)) * (1.f / 256.f);
        f_lo += static_cast<float>(n[i]) * ex2_approx(x - 7.6f / 256.f);
        f_hi += static_cast<float>(n[i]) * ex2_approx(x + 0.6f / 256.f);
      }
    }
    uint32_t c_at = count;
    float lo_at = f_lo, hi_at = f_hi;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, c_at, o);
      const float l = __shfl_up_sync(0xFFFFFFFFu, lo_at, o);
      const float h = __shfl_up_sync(0xFFFFFFFFu, hi_at, o);
      if (lane >= o) {
        c_at += up;
        lo_at += l;
        hi_at += h;
      }
    }
    if (lane == 31) {
      sh.warpu[warp] = c_at;
      sh.warpf[0][warp] = lo_at;
      sh.warpf[1][warp] = hi_at;
    }
    __syncthreads();
    c_at -= count;
    lo_at -= f_lo;
    hi_at -= f_hi;
    // bounds of the target relative to 2^N, with room for the roundings of the fp32 sums
    float want_lo = 0.f, want_hi = 0.f;
    for (int i = 0; i < kWarps; ++i) {
      want_lo += sh.warpf[0][i];
      want_hi += sh.warpf[1][i];
      if (i < warp) {
        c_at += sh.warpu[i];
        lo_at += sh.warpf[0][i];
        hi_at += sh.warpf[1][i];
      }
    }
    want_lo *= 0.9995f * p;
    want_hi *= 1.0005f * p;
    const uint32_t c_first = c_at;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * kPer + i;
      // the first bin that reaches the target (between threads rounding may name two)
      if (kMass) {
        const float x = -static_cast<float>(8 * b) * (1.f / 256.f);
        const bool lo_was = lo_at >= want_hi, hi_was = hi_at >= want_lo;
        lo_at += static_cast<float>(n[i]) * ex2_approx(x - 7.6f / 256.f);
        hi_at += static_cast<float>(n[i]) * ex2_approx(x + 0.6f / 256.f);
        if (!hi_was && hi_at >= want_lo) atomicMin(&sh.bin_lo, b);
        if (!lo_was && lo_at >= want_hi) atomicMin(&sh.bin_hi, b);
      } else if (c_at < static_cast<uint32_t>(k) && c_at + n[i] >= static_cast<uint32_t>(k)) {
        sh.bin_lo = b;
      }
      c_at += n[i];
    }
    __syncthreads();
    const int lo = sh.bin_lo, hi = kMass ? sh.bin_hi : lo;
    if (hi >= low) return false;  // the same in every CTA
    c_at = c_first;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (tid * kPer + i == lo) sh.above = c_at;
      c_at += n[i];
    }

    // ---- the weights of all and of those above, and the fine bins within
    const int first = 8 * lo, last = 8 * hi + 7;
    int shift = 0;  // 1/256 octave a fine bin, or as much as lets them cover those bins
    while (((last - first) >> shift) >= kFine) ++shift;
    u64 mine = 0, above = 0;
    for (int j = tid; j < s.n; j += kThreads) {
      float v[kVec];
      kept_vector(j, zc, whole, v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int at = place_of(v[i], base);
        if (at >= first && at <= last) {
          const int b = (at - first) >> shift;
          atomicAdd(&sh.fine.count[b], 1u);
          if (kMass) add_weight(&sh.fine.lo[b], &sh.fine.hi[b], weight(v[i], st, sh.table));
        }
      }
      if (kMass) {
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
          u64 w0, w1;
          pow2_shifted(f2(v[i], v[i + 1]), pw, sh.table, w0, w1);
          mine += w0 + w1;
          above += place_of(v[i], base) < first ? w0 : 0;
          above += place_of(v[i + 1], base) < first ? w1 : 0;
        }
      }
    }
    if (kMass) {
      mine = cta_sum(mine);
      above = cta_sum(above);
    }
    u64 acc;
    const u64 total = total_of(mine, above, acc);
    if (!kMass) acc = sh.above;
    const u64 target = kMass ? top_p_target(total, p) : static_cast<u64>(k);
    // the fine bin that the border is in, from all CTAs' sums
    constexpr int kEach = kFine / kThreads;
    u64 m[kEach], part = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      n[i] = 0;
      m[i] = 0;
    }
    for (int c = 0; c < a.cluster; ++c) {
      remote_fine(&sh.fine.count[tid * kEach], c, [&](int i, uint32_t x) { n[i] += x; });
      if (kMass) {
        remote_fine(&sh.fine.lo[tid * kEach], c, [&](int i, uint32_t x) { m[i] += x; });
        remote_fine(&sh.fine.hi[tid * kEach], c,
                    [&](int i, uint32_t x) { m[i] += static_cast<u64>(x) << 32; });
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (!kMass) m[i] = n[i];
      part += m[i];
    }
    u64 before = warp_scan(part);
    __syncthreads();
    if (lane == 31) sh.warp[warp] = before;
    if (tid == 0) sh.all = 1;
    __syncthreads();
    before += acc - part;
    for (int i = 0; i < warp; ++i) before += sh.warp[i];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (before < target && target <= before + m[i]) {
        sh.digit = tid * kEach + i;
        sh.acc = before;
        sh.in = n[i];
        sh.all = 0;
      }
      before += m[i];
    }
    __syncthreads();
    // none: the bounds of the bins' mass did not hold; or too many of one value
    if (sh.all != 0 || sh.in > kCap) return false;
    const int place = first + (static_cast<int>(sh.digit) << shift), len = static_cast<int>(sh.in);
    acc = sh.acc;

    // ---- its tokens, and whether they are all of one value
    uint32_t key_lo = 0xFFFFFFFFu, key_hi = 0;
    for (int j = tid; j < s.n; j += kThreads) {
      float v[kVec];
      kept_vector(j, zc, whole, v);
      uint32_t in = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) in |= (place_of(v[i], base) - place) >> shift == 0 ? 1u << i : 0u;
      for (; in != 0; in &= in - 1) {
        const int i = __ffs(in) - 1;
        const uint32_t key = key_of(E::widen(reinterpret_cast<const typename E::raw*>(slice + j)[i]));
        key_lo = min(key_lo, key);
        key_hi = max(key_hi, key);
        sh.list[atomicAdd(&sh.list_n, 1u)] =
            (static_cast<u64>(key) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(id_of(j, i)));
      }
    }
    key_lo = __reduce_min_sync(0xFFFFFFFFu, key_lo);
    key_hi = __reduce_max_sync(0xFFFFFFFFu, key_hi);
    __syncthreads();
    if (lane == 0) {
      sh.warpu[warp] = key_lo;
      sh.warpv[warp] = key_hi;
    }
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) {
      key_lo = min(key_lo, sh.warpu[i]);
      key_hi = max(key_hi, sh.warpv[i]);
    }
    const int listed = static_cast<int>(sh.list_n);
    exchange(static_cast<u64>(listed), (static_cast<u64>(key_hi) << 32) | key_lo);
    int at = 0;  // in the lists of the ranks before
    for (int c = 0; c < a.cluster; ++c) {
      if (c < rank) at += static_cast<int>(got(c, 0));
      key_lo = min(key_lo, static_cast<uint32_t>(got(c, 1)));
      key_hi = max(key_hi, static_cast<uint32_t>(got(c, 1) >> 32));
    }
    if (key_lo == key_hi) {
      // equal weights: so many of them by id; the one that is last is in one CTA's list
      const u64 w = kMass ? weight(key_value(key_lo), st, sh.table) : 1;
      const int want = static_cast<int>((target - acc + w - 1) / w) - 1 - at;
      if (tid == 0) sh.found = -1;
      __syncthreads();
      if (want >= 0 && want < listed) {
        for (int i = tid; i < listed; i += kThreads) {
          const u64 mine = sh.list[i];
          int before = 0;
          for (int q = 0; q < listed; ++q) before += sh.list[q] > mine ? 1 : 0;
          if (before == want) sh.found = static_cast<int>(~static_cast<uint32_t>(mine));
        }
      }
      __syncthreads();
      exchange(static_cast<u64>(static_cast<int64_t>(sh.found)), 0);
      st.kc = key_lo;
      for (int c = 0; c < a.cluster; ++c)
        if (static_cast<int>(got(c, 0)) >= 0) st.idc = static_cast<int>(got(c, 0));
      return true;
    }
    // to rank 0: behind the lists of the ranks before, its own being in place
    if (rank != 0)
      for (int i = tid; i < listed; i += kThreads)
        cluster_store(cluster_addr(&sh.list[at + i], 0), sh.list[i]);
    cluster_arrive();
    cluster_wait();
    u64 border = 0;
    if (rank == 0) {
      int n2 = 1;
      while (n2 < len) n2 <<= 1;
      for (int i = len + tid; i < n2; i += kThreads) sh.list[i] = 0;
      __syncthreads();
      sort_desc<kThreads>(sh.list, n2);
      constexpr int kOf = kCap / kThreads;
      u64 w[kOf];
      part = 0;
#pragma unroll
      for (int q = 0; q < kOf; ++q) {
        const int i = tid * kOf + q;
        w[q] = i >= len ? 0 : kMass ? weight(key_value(static_cast<uint32_t>(sh.list[i] >> 32)), st, sh.table) : 1;
        part += w[q];
      }
      before = warp_scan(part);
      if (lane == 31) sh.warp[warp] = before;
      __syncthreads();
      before += acc - part;
      for (int i = 0; i < warp; ++i) before += sh.warp[i];
#pragma unroll
      for (int q = 0; q < kOf; ++q) {
        // the last token before which there is less than the target
        if (before < target && before + w[q] >= target) sh.acc = sh.list[tid * kOf + q];
        before += w[q];
      }
      __syncthreads();
      border = sh.acc;
    }
    exchange(border, 0);
    border = got(0, 0);
    st.kc = static_cast<uint32_t>(border >> 32);
    st.idc = static_cast<int>(~static_cast<uint32_t>(border));
    return true;
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

  // The draw, f and one being the kept tokens' weights; f counts them in n.
  template <class F, class G>
  __device__ __forceinline__ void draw(int64_t row, float u, uint32_t& n, F&& f, G&& one) {
    const u64 mine = slice_sum(f);
    const uint32_t warp_n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) sh.warpu[warp] = warp_n;
    __syncthreads();
    uint32_t cta_n = 0;
    for (int i = 0; i < kWarps; ++i) cta_n += sh.warpu[i];
    u64 all;
    const u64 total = total_of(mine, cta_n, all);
    const u64 target = draw_target(total, u);
    u64 before = 0;
    for (int c = 0; c < rank; ++c) before += got(c, 0);
    if (before <= target && target < before + mine) {  // one CTA of the row
      const int id = locate(target - before, f, one);
      if (tid == 0) write_row(a, st, sh.table, row, id, r.at(id), total, static_cast<int>(all));
    }
  }

  // ---- the filtered row, by all CTAs
  __device__ void wide(int64_t row, float u, int k, float top_p, uint32_t kmin) {
    st.kc = kNegInfKey;
    st.idc = INT32_MIN;
    auto one = [&](float z, int id) { return kept_weight(z, id); };
    auto kept = [&](const float(&v)[kVec], int id0) {
      u64 t = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) t += one(v[i], id0 + i);
      return t;
    };
    if (k > 0 && (st.pw.recentre || !narrow<false>(k, 0.f))) {
      cluster_arrive();  // the histograms share their memory with the fine bins, before and after
      cluster_wait();
      select_border<false>(static_cast<u64>(k));
      cluster_arrive();
      cluster_wait();
    }
    if (top_p < 1.f && (st.pw.recentre || !narrow<true>(0, top_p))) {
      u64 all;
      const u64 total = total_of(slice_sum(kept), 0, all);
      select_border<true>(top_p_target(total, top_p));
    }
    if (kmin > st.kc) {
      st.kc = kmin;
      st.idc = INT32_MAX;
    }
    const float zc = key_value(st.kc);
    uint32_t n = 0;
    if (st.pw.recentre) {
      draw(row, u, n, [&](const float(&v)[kVec], int id0) {
        u64 t = 0;
#pragma unroll 1
        for (int i = 0; i < kVec; ++i) {
          n += keeps(key_of(v[i]), id0 + i, st) && in_row(id0 + i) ? 1 : 0;
          t += one(v[i], id0 + i);
        }
        return t;
      }, one);
    } else {
      const Pow2Pair pw = pair();
      draw(row, u, n, [&](const float(&x)[kVec], int id0) {
        float v[kVec];
        bool some = false;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          v[i] = x[i];
          some |= x[i] >= zc;
          // slots that are not the row's hold -inf
          n += x[i] > zc || (x[i] == zc && id0 + i <= st.idc && in_row(id0 + i)) ? 1 : 0;
        }
        if (!some) return static_cast<u64>(0);
        drop(v, id0, zc);
        return weights_of(v, pw);
      }, one);
    }
  }

  // ---- the unfiltered row, by all CTAs
  __device__ void plain(int64_t row, float u) {
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
      const Pow2Pair k = pair();
      const float zlow = st.zlow;
      draw(row, u, n, [&](const float(&x)[kVec], int) {
        float v[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = fmaxf(x[i], zlow);
        return weights_of(v, k);
      }, one);
    }
  }
};

// Whether the mark of a row is that of an undecided one of this cluster.
__device__ __forceinline__ bool is_mine(int kept, int64_t cluster, int64_t clusters) {
  return kept <= kUndecided && (kUndecided - kept) % static_cast<int>(clusters) == static_cast<int>(cluster);
}

template <int kDtype, int kThreads, bool kPlain>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 2)
    sample_wide_kernel(const WideArgs a) {
  using E = Elem<kDtype>;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint4 slice_mem[];
  __shared__ Shared<kThreads, kPlain> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int64_t clusters = gridDim.x / a.cluster, first = blockIdx.x / a.cluster;

  pdl_wait();  // what the list kernel decided
  if constexpr (!kPlain) {
    if (blockIdx.x == 0 && tid == 0) a.status[kCountWord] = 0;
    // Nothing to be done is the usual case.  All CTAs of a cluster see the same: only they write
    // their rows, and none does before the others have come to the first barrier.
    bool any = false;
    for (int64_t row = tid; row < a.T; row += kThreads) any |= is_mine(__ldcg(a.kept + row), first, clusters);
    if (!__syncthreads_or(any)) return;
  }
  cluster_arrive();
  if (tid == 0) {
    mbar_init(&sh.bar, 1);
    fence_mbarrier_init();
  }
  for (int i = tid; i < 256; i += kThreads) sh.table[i] = __ldg(&g_pow2_table.t[i]);
  __syncthreads();
  cluster_wait();  // every CTA of the cluster runs
  uint32_t parity = 0;
  int phase = 0;
  for (int64_t base = 0; base < a.T; base += kPlain ? a.T : 32) {
    // which of the next rows are this cluster's; unfiltered rows are one a cluster
    unsigned todo = 1;
    if constexpr (!kPlain) {
      const int64_t row = base + lane;
      todo = __ballot_sync(0xFFFFFFFFu, row < a.T && is_mine(__ldcg(a.kept + row), first, clusters));
      if (todo == 0) continue;
      // a CTA that is behind must not see what this one writes of a row that it has still to test
      cluster_arrive();
      cluster_wait();
    }
    for (; todo != 0; todo &= todo - 1) {
      const int64_t row = kPlain ? first : base + (__ffs(todo) - 1);
      const Row<kDtype> r(a.logits, row, a.ld, a.V);
      const Slice s = slice_of(r.nvec(), rank, a.cluster);
      if (tid == 0) load_slice(r, s, slice_mem, &sh.bar);
      load_slice_edges(r, s, slice_mem);
      const Settings set = settings_of(a, row);
      int bad = set.bad;
      Sampler<kDtype, kThreads, kPlain> S{a, sh, slice_mem, r, s, rank, tid, warp, lane, phase, {}};
      RowState& st = S.st;
      set_temperature(st, set.tau);
      const int never = 0;
      __syncthreads();  // the edges
      if (!mbar_wait(&sh.bar, parity, &never)) set_status(a.status, TIM_ERR_TIMEOUT);
      parity ^= 1u;

      // ---- the largest logit of each thread; of each warp, to every CTA of the row
      float tmax = -INFINITY;
      if (tid < s.n) {
        uint4 m = slice_mem[tid];
#pragma unroll 4
        for (int j = tid + kThreads; j < s.n; j += kThreads) m = max_vec<kDtype>(m, slice_mem[j]);
        tmax = max_of<kDtype>(m);
      }
      const uint32_t mykey = !(tmax < INFINITY) ? 0xFFFFFFFFu : key_of(tmax);
      const uint32_t wkey = __reduce_max_sync(0xFFFFFFFFu, mykey);
      float sum = 0.f;
      if (wkey > kNegInfKey && wkey != 0xFFFFFFFFu) {
        sum = ex2_approx((tmax - key_value(wkey)) * st.pw.kh);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      }
      if (lane < a.cluster) {
        const int g = rank * kWarps + warp;
        cluster_store32(cluster_addr(&sh.gkey[g], lane), wkey);
        cluster_store32(cluster_addr(&sh.gsum[g], lane), __float_as_uint(sum));
      }
      cluster_arrive();
      cluster_wait();
      const int groups = a.cluster * kWarps;
      uint32_t hi = 0;
      for (int g = lane; g < groups; g += 32) hi = max(hi, sh.gkey[g]);
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      if (bad == 0 && (hi == 0xFFFFFFFFu || hi <= kNegInfKey)) bad = TIM_ERR_NONFINITE;
      if (bad != 0) {  // the same in every CTA of the row
        if (rank == 0 && tid == 0) write_bad(a, row, bad);
      } else {
        const float M = key_value(hi);
        st.M = M;
        sum = 0.f;
        for (int g = lane; g < groups; g += 32) {
          const uint32_t key = sh.gkey[g];
          if (key > kNegInfKey) sum += sh.gsum[g] * ex2_approx((key_value(key) - M) * st.pw.kh);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        // the elements of a thread, at most
        const int per_cta = (r.nvec() + a.cluster - 1) / a.cluster;
        set_scale(st, sum * static_cast<float>((per_cta + kThreads - 1) / kThreads * E::kVec));
        if constexpr (kPlain) {
          S.plain(row, set.u);
        } else {
          if (set.k == 0 && set.top_p >= 1.f && set.min_p == 0.f)
            S.plain(row, set.u);
          else
            S.wide(row, set.u, set.k, set.top_p, min_p_key(M, set.tau, set.min_p));
        }
      }
      phase = S.phase;
      // the next row's copy overwrites the slice, and its sums this row's in the other CTAs
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      cluster_arrive();
      cluster_wait();
    }
  }
}

template <int kDtype, int kThreads, bool kPlain>
cudaError_t launch_rows(WideArgs a, const RowPlan& p, cudaStream_t stream, int num_sms) {
  const size_t smem = p.slice_bytes;
  auto* kernel = sample_wide_kernel<kDtype, kThreads, kPlain>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kernel, plan_row(TIM_LOGITS_MAX_V, sizeof(typename Elem<kDtype>::raw)).slice_bytes, allowed);
  if (e != cudaSuccess) return e;
  a.cluster = p.cluster;
  // a cluster a row, or where rows are to be looked for among the decided ones as many clusters
  // as fit at once
  int64_t clusters = a.T;
  if (!kPlain) {
    const int64_t fit = static_cast<int64_t>(num_sms) * 2 / p.cluster;
    if (clusters > fit) clusters = fit;
  }
  return launch_clusters(kernel, clusters, p.cluster, kThreads, smem, stream, a, !kPlain);
}
template <int kDtype>
cudaError_t launch_type(const WideArgs& a, bool plain, cudaStream_t stream, int num_sms) {
  const RowPlan p = plan_row(a.V, sizeof(typename Elem<kDtype>::raw));
  // Filtered rows that come here are few and wait on one another's exchanges: 512 threads, two CTAs
  // an SM (96 mixed rows 106 us, with 256 and three 157).  Unfiltered ones may be many: 256 where
  // the slice is small, for four CTAs an SM.
  if (!plain) return launch_rows<kDtype, 512, false>(a, p, stream, num_sms);
  return p.threads == 256 ? launch_rows<kDtype, 256, true>(a, p, stream, num_sms)
                          : launch_rows<kDtype, 512, true>(a, p, stream, num_sms);
}

}  // namespace

// plain: no row is filtered, and all are done; else those that the list kernel left.
cudaError_t launch_sample_wide(const SampleArgs& args, int dtype, int64_t T, bool plain,
                               cudaStream_t stream, int num_sms) {
  WideArgs a;
  static_cast<SampleArgs&>(a) = args;
  a.T = T;
  a.cluster = 1;
  return dtype == TIM_F32    ? launch_type<TIM_F32>(a, plain, stream, num_sms)
         : dtype == TIM_BF16 ? launch_type<TIM_BF16>(a, plain, stream, num_sms)
                             : launch_type<TIM_F16>(a, plain, stream, num_sms);
}

}  // namespace tim
