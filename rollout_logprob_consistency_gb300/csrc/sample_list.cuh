// The sampler's main kernel, for whatever says which rows there are, with which settings, and where
// their results go (Args: SampleArgs for tim_sample, VerifyArgs for the rows of a verification).
//
// Order the tokens of a row by (logit descending, id ascending); s = z / tau.
//   top-k   the first k of them: the set K
//   top-p   q = softmax of s over K; a token is kept while the q-mass before it is < p
//   min-p   exp(s - s_max) >= min_p
//   token   the smallest id v with  sum_{kept w <= v} exp(s_w) > u * sum_kept exp(s)
//
// A token drawn, or the last one that top-p keeps, is decided by sums of up to hundreds of
// thousands of exponentials against a border: rounding them to 32 bits would move the
// border past tokens.  Every weight that decides is therefore taken to 2^-30.5 (weight_of) and
// summed as a 64-bit integer, at a scale that puts the total between 2^50 and 2^60 (a list's, of 2048
// tokens at most, between 2^47 and 2^60): the sums are exact in that scale and do not depend on the
// order or the split, and what a token loses below one unit is 2^-31 of the total for all together.
//
// A row has one CTA, which reads it from memory once: while it streams, every thread notes the
// largest logits of blocks of its vectors (and, for top-p alone, a running sum in fp32).  They bound
// the tokens that can be kept:
//  - the k-th largest of the threads' (or groups of threads') maxima is met by every top-k
//    logit, they being k different logits;
//  - for top-p the logit below which V tokens together would hold less than 1 - p;
//  - min-p's own bound.
// Only the blocks whose maximum meets the bound are read again (from L2); their tokens above it
// are sorted and decided with integer weights.  Top-p alone needs the row's total: the fp32 sum
// with its error bound decides unless the border lies within that error.  A row that this does not
// decide is read again as often as it takes (sample_deep.cuh).  Few unfiltered rows are a cluster's
// each (sample_plain.cu).
//
// Many rows are bound by memory: 1024 rows of 151936 bf16 logits with top-k 50 and top-p 0.95 take 82 us,
// 3.8 TB/s; in a CTA's 90 us of life 62 are the stream, 4 the bound, 15 the second look in a loaded
// memory system, 5 the decision.  One row takes 13 us: 3.5 the stream, the rest that chain.
#pragma once

#include "sample_deep.cuh"

namespace tim {
namespace sampling {

constexpr int kCap = 2048;     // tokens of the list
constexpr int kListK = 1024;   // largest top-k that the list serves
constexpr int kMaximaBins = 256;
constexpr uint32_t kWant = 384;  // maxima that a top-p list is to hold
constexpr int kUnroll = 4;     // vectors of a thread in flight
constexpr int kMaxima = 5120;  // of blocks of the row, kept while it streams
constexpr float kSumError = 0x1p-16f;  // of the fp32 sum, see its place

// Orders are found by counting up to here, a token a thread at most (rows of a list of 200 take 33 us so
// against 39 with a sort, 1024 rows of 65 in CTAs of 128 threads 82 against 86 with four a thread).
template <int kThreads>
constexpr int kCount = kThreads > 256 ? kThreads / 2 : 128;

// Blocks to be read again; eight CTAs of 128 threads have to fit an SM.
template <int kThreads>
constexpr int kItems = kThreads > 128 ? 2048 : 1024;

template <int kThreads>
struct Shared {
  Tables table;
  union {
    float top[kMaxima];  // of block b of thread t: top[b kThreads + t]
    struct {
      u64 key[kCap];  // key << 32 | ~id: larger comes first
      u64 w[kCount<kThreads>];  // of the first tokens
    };
    DeepShared deep;
  };
  DeepScratch scratch;
  uint32_t group[kThreads > kMaximaBins ? kThreads : kMaximaBins];
  uint16_t item[kItems<kThreads>];  // blocks to be read again: the places of their maxima
  u64 warp[32], total[kThreads / 32];
  uint32_t warpu[kThreads / 32];
  float warpf[kThreads / 32];
  uint32_t bound;
  int items, n, count_lo, count_hi, hopeless;
};

// f 2^e as a whole number, e at least 24 - (exponent of f)
__device__ __forceinline__ u64 scaled_up(float f, int e) {
  const int x = static_cast<int>(__float_as_uint(f) >> 23) - 150 + e;  // f = m 2^(x - e)
  const u64 m = (__float_as_uint(f) & 0x7FFFFFu) | 0x800000u;
  return x >= 0 ? m << min(x, 39) : m >> min(-x, 63);
}

// Threads that share the work of one of n things: a power of two up to 32.
template <int kThreads>
__device__ __forceinline__ int sharers(int n) {
  int s = 32;
  while (s > 1 && s * n > kThreads) s >>= 1;
  return s;
}

// The row's token from the list of n tokens in sh.key, by the whole CTA; `complete`: the list
// holds all that min-p keeps.  For top-p of the whole row, `sum` > 0 is the row's fp32 total in units
// of 2^(max K).  False: the list ends before the border, or the border lies within the total's error.
//
// Few tokens' orders are found by counting: a token's comparisons are shared by as many threads as
// there are, with no barrier between them; for more of them the squares cost more than a sort.
template <int kThreads, class Args>
__device__ __forceinline__ bool decide(const Args& a, const RowState& st, Shared<kThreads>& sh,
                                       int64_t row, float u, int n, int k, float top_p,
                                       uint32_t kmin, bool complete, float sum) {
  constexpr int kCounted = kCount<kThreads>;
  const int tid = threadIdx.x, lane = tid & 31;
  u64 lo = ~0ull, hi = ~0ull;  // top-p keeps a token while the sum before it is below
  if (sum > 0.f) {
    // the total in the weights' unit: 2^(max K - top + 62)
    const Df mk = st.pw.recentre ? df(0.f) : df(st.M) * Df{st.pw.kh, st.pw.kl};
    const float whole = rintf(mk.h), frac = (mk.h - whole) + mk.l;
    const float P = top_p * sum * pow2_df(frac, Pow2Row{1.f, 0.f, 0.f, false}, sh.table.fine).h;
    const int e = static_cast<int>(whole) - st.top + 62;
    lo = scaled_up(P * (1.f - kSumError), e);
    hi = scaled_up(P * (1.f + kSumError), e) + 1;
    if (!complete) {  // whether the list reaches the border, before any order is looked for
      u64 listed = 0;
      for (int i = tid; i < n; i += kThreads)
        listed += weight(key_value(static_cast<uint32_t>(sh.key[i] >> 32)), st, sh.table);
      u64 all;
      block_scan<kThreads>(listed, sh.warp, kThreads / 32, all);
      __syncthreads();
      if (hi > all) return false;
    }
  }
  if (k == 0 && top_p >= 1.f) {
    // min-p alone: all of the list is kept, in any order
  } else if (n <= kCounted) {
    const int each = sharers<kThreads>(n), i = tid / each;
    const u64 mine = i < n ? sh.key[i] : 0;
    int at = 0;
    if ((tid - lane) / each < n) {
#pragma unroll 4
      for (int j = tid & (each - 1); j < n; j += each) at += sh.key[j] > mine ? 1 : 0;
    }
    for (int o = 1; o < each; o <<= 1) at += __shfl_xor_sync(0xFFFFFFFFu, at, o);
    __syncthreads();
    if (i < n && (tid & (each - 1)) == 0) sh.key[at] = mine;
  } else {
    int n2 = 64;
    while (n2 < n) n2 <<= 1;
    for (int i = n + tid; i < n2; i += kThreads) sh.key[i] = 0;
    __syncthreads();
    sort_desc<kThreads>(sh.key, n2);
  }
  if (tid == 0) sh.count_lo = sh.count_hi = 0;
  __syncthreads();
  if (k > 0) n = min(n, k);
  // weights in order, and their running sum: a thread has `per` of them in a row
  const int per = (n + kThreads - 1) / kThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
  u64 part = 0;
  for (int i = i0; i < i1; ++i) {
    const u64 w = weight(key_value(static_cast<uint32_t>(sh.key[i] >> 32)), st, sh.table);
    if (i < kCounted) sh.w[i] = w;
    part += w;
  }
  u64 total;
  u64 before = block_scan<kThreads>(part, sh.warp, (n + 32 * per - 1) / (32 * per), total);
  if (top_p < 1.f && k > 0) lo = hi = top_p_target(total, top_p);
  int c_lo = 0, c_hi = 0;
  for (int i = i0; i < i1; ++i) {
    const bool min_ok = static_cast<uint32_t>(sh.key[i] >> 32) >= kmin;
    c_lo += before < lo && min_ok ? 1 : 0;
    c_hi += before < hi && min_ok ? 1 : 0;
    before += i < kCounted ? sh.w[i]
                           : weight(key_value(static_cast<uint32_t>(sh.key[i] >> 32)), st, sh.table);
  }
  if ((tid - lane) * per < n) {  // this warp has tokens
    c_lo = __reduce_add_sync(0xFFFFFFFFu, c_lo);
    c_hi = __reduce_add_sync(0xFFFFFFFFu, c_hi);
    if (lane == 0 && (c_lo | c_hi) != 0) {
      atomicAdd(&sh.count_lo, c_lo);
      atomicAdd(&sh.count_hi, c_hi);
    }
  }
  __syncthreads();
  const int m = sh.count_lo;
  if (m != sh.count_hi) return false;
  // the last token kept; of min-p alone, whose list has no order, its first key
  const u64 border = k == 0 && top_p >= 1.f ? static_cast<u64>(kmin) << 32 : sh.key[m - 1];
  // the draw, by id
  if (m <= kCounted) {
    // what the kept tokens of lower ids weigh
    const int each = sharers<kThreads>(m), i = tid / each;
    if ((tid - lane) / each >= m) return true;  // a warp without tokens
    const int id = i < m ? static_cast<int>(~static_cast<uint32_t>(sh.key[i])) : -1;
    u64 kept = 0, below = 0;
#pragma unroll 4
    for (int j = tid & (each - 1); j < m; j += each) {
      const u64 w = sh.w[j];
      kept += w;
      below += static_cast<int>(~static_cast<uint32_t>(sh.key[j])) < id ? w : 0;
    }
    for (int o = 1; o < each; o <<= 1) {
      kept += __shfl_xor_sync(0xFFFFFFFFu, kept, o);
      below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
    }
    const u64 target = draw_target(kept, u);
    if (i < m && (tid & (each - 1)) == 0 && below <= target && target < below + sh.w[i])
      write_row(a, st, sh.table, row, id, key_value(static_cast<uint32_t>(sh.key[i] >> 32)), kept, m,
                border);
    return true;
  }
  // sorted once more, by id: the low word on top descends as the id ascends
  int n2 = 64;
  while (n2 < m) n2 <<= 1;
  if constexpr (Args::kBorder) __syncthreads();  // every thread has read it
  for (int i = tid; i < n2; i += kThreads) {
    const u64 x = sh.key[i];
    sh.key[i] = i < m ? (x << 32) | (x >> 32) : 0;
  }
  __syncthreads();
  sort_desc<kThreads>(sh.key, n2);
  const int each = (m + kThreads - 1) / kThreads, j0 = min(m, tid * each), j1 = min(m, j0 + each);
  part = 0;
  for (int i = j0; i < j1; ++i)
    part += weight(key_value(static_cast<uint32_t>(sh.key[i])), st, sh.table);
  before = block_scan<kThreads>(part, sh.warp, (m + 32 * each - 1) / (32 * each), total);
  const u64 target = draw_target(total, u);
  for (int i = j0; i < j1; ++i) {
    const u64 x = sh.key[i], w = weight(key_value(static_cast<uint32_t>(x)), st, sh.table);
    if (before <= target && target < before + w)
      write_row(a, st, sh.table, row, static_cast<int>(~static_cast<uint32_t>(x >> 32)),
                key_value(static_cast<uint32_t>(x)), total, m, border);
    before += w;
  }
  return true;
}

template <int kDtype, int kThreads, class Args>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_list_kernel(const Args a) {
  using E = Elem<kDtype>;
  constexpr int kWarps = kThreads / 32;
  __shared__ Shared<kThreads> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x;
  if (!wanted(a, row)) return;
  const Row<kDtype> r = row_of<kDtype>(a, row);
  const Settings set = settings_of(a, row);
  const bool list_k = set.k > 0 && set.k <= kListK;
  const bool need_sum = set.k == 0 && set.top_p < 1.f;
  const bool list_min = set.min_p > 0.f && set.top_p >= 1.f;
  if (tid == 0) sh.items = sh.n = sh.hopeless = 0;
  load_tables(sh.table, tid, kThreads);
  RowState st;
  set_temperature(st, set.tau);
  if (set.k == 0 && !need_sum && !list_min) {
    __syncthreads();
    Deep<kDtype, kThreads, Args> deep{a,        sh.deep, sh.scratch, sh.table, sh.warp, sh.total,
                                sh.warpu, r,       st,         tid,      warp,    lane};
    deep.plain(row, set.u, set.bad);
    return;
  }

  // ---- one pass: the largest logit of each of the thread's blocks, and the fp32 sum
  const int nvec = r.nvec();
  const int steps = (nvec + kThreads - 1) / kThreads;  // vectors of a thread
  // steps of a block: whole groups of kUnroll, as few as there is room for their maxima
  constexpr int kGroups = kMaxima / kThreads * kUnroll;
  const int block = (steps + kGroups - 1) / kGroups * kUnroll;
  const int blocks = (steps + block - 1) / block;
  float tmax = -INFINITY, run = -INFINITY;
  // The sum is relative to a reference of the thread that follows its largest logit, 8 octaves late,
  // and is taken in three levels (a group of kUnroll vectors, a block, the row).  Its error, 2^-24 a
  // rounding:
  //  - a term's argument has two roundings and the remainder of K: 2.5 x 2^-24 |x| ln2.  The mass of
  //    V <= 2^19 tokens lies within 19 octaves of the largest: below 2.0e-6;
  //  - its exponential 2^-22; at most 5 changes of the reference in 40 octaves 2^-22 each: 1.5e-6;
  //  - at most 8 + 1 + 8 + 40 additions in a thread and 10 among them: 4.0e-6;
  //  - the joining of the threads' sums and what decide() multiplies it with: 1.0e-6.
  // Together below kSumError = 1.5e-5.
  F2 acc = f2(0.f, 0.f), whole = acc;
  const F2 kk = f2(st.pw.kh, st.pw.kh);
  const float late = 8.f / st.pw.kh;
  const uint4* const vec = r.vec() + tid;
  const int w0 = r.w0(), w1 = r.w1(), full = w1 / kThreads;  // steps that all threads have whole
  uint4 x[kUnroll];
  for (int b = 0; b < blocks; ++b) {
    float bmax = -INFINITY;
    const int end = min(steps, (b + 1) * block);
    for (int i = b * block; i < end; i += kUnroll) {
      const uint4* p = vec + i * kThreads;
      if (i >= w0 && i + kUnroll <= full) {
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) x[n] = __ldg(p + n * kThreads);
      } else {  // the row's ends, which may be partly others'
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
          const int j = tid + (i + n) * kThreads;
          x[n] = j >= w0 && j < w1 ? __ldg(p + n * kThreads)
                 : j < nvec        ? r.load_edge(j)
                                   : neg_inf_vec<kDtype>();
        }
      }
      uint4 m = x[0];
#pragma unroll
      for (int n = 1; n < kUnroll; ++n) m = max_vec<kDtype>(m, x[n]);
      const float most = max_of<kDtype>(m);
      bmax = max_nan(bmax, most);
      if (need_sum) {
        if (most > run + late || run == -INFINITY) {
          const float f = run == -INFINITY ? 0.f : ex2_approx((run - most) * st.pw.kh);
          acc = mul2(acc, f2(f, f));
          whole = mul2(whole, f2(f, f));
          run = most;
        }
        const float from = run == -INFINITY ? 0.f : -run;
        const F2 ref = f2(from, from);
        F2 part = f2(0.f, 0.f), part2 = part;
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
          float v[E::kVec];
          E::unpack(x[n], v);
#pragma unroll
          for (int q = 0; q < E::kVec; q += 4) {
            part = add2(part, ex2x2(mul2(add2(f2(v[q], v[q + 1]), ref), kk)));
            part2 = add2(part2, ex2x2(mul2(add2(f2(v[q + 2], v[q + 3]), ref), kk)));
          }
        }
        acc = add2(acc, add2(part, part2));
      }
    }
    whole = add2(whole, acc);
    acc = f2(0.f, 0.f);
    sh.top[b * kThreads + tid] = bmax;
    tmax = max_nan(tmax, bmax);
  }
  // ---- the row's largest
  const uint32_t mykey = !(tmax < INFINITY) ? 0xFFFFFFFFu : key_of(tmax);
  uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, mykey);
  if (lane == 0) sh.warpu[warp] = hi;
  // The k-th largest is looked for among groups of 2^shift threads, at least twice as many as k:
  // about 1.4 k tokens then meet it, and a group's threads share its count.  Where there are not
  // that many threads, among all blocks, by a histogram.
  int shift = 5;
  while (shift > 0 && (kThreads >> shift) < 2 * set.k) --shift;
  const int each = 1 << shift;
  const bool by_group = list_k && (kThreads >> shift) >= 2 * set.k;
  if (by_group) {
    uint32_t g = mykey;
    for (int o = 1; o < each; o <<= 1) g = max(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
    if ((tid & (each - 1)) == 0) sh.group[tid >> shift] = g;
  }
  __syncthreads();
  hi = __reduce_max_sync(0xFFFFFFFFu, lane < kWarps ? sh.warpu[lane] : 0u);
  int bad = set.bad;
  if (bad == 0 && (hi == 0xFFFFFFFFu || hi <= kNegInfKey)) bad = TIM_ERR_NONFINITE;
  if (bad != 0) {
    if (tid == 0) write_bad(a, row, bad);
    return;
  }
  const float M = key_value(hi);
  st.M = M;
  float sum = 0.f;
  if (need_sum) {
    const float2 t = unpack2(whole);
    sum = run == -INFINITY ? 0.f : (t.x + t.y) * ex2_approx((run - M) * st.pw.kh);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) sh.warpf[warp] = sum;
    __syncthreads();
    sum = lane < kWarps ? sh.warpf[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  }
  // ---- the list holds all tokens from the key `bound` up
  const uint32_t kmin = min_p_key(M, set.tau, set.min_p);
  uint32_t bound = list_min ? kmin : kNegInfKey + 1;
  if (by_group) {
    const int groups = kThreads >> shift, g = tid >> shift;
    const uint32_t mine = sh.group[g];
    int before = 0;
    for (int i = tid & (each - 1); i < groups; i += each) {
      const uint32_t other = sh.group[i];
      before += other > mine || (other == mine && i < g) ? 1 : 0;
    }
    for (int o = 1; o < each; o <<= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    if (before == set.k - 1) sh.bound = mine;
    __syncthreads();
    bound = max(bound, sh.bound);
  } else if (list_k || need_sum) {
    // For top-p: the tokens below this hold less than 1 - p of the mass, were there V of them.  That
    // can be thousands; as much of the list as is sure to fit serves most rows, and where it ends
    // before the border does decide() says so.
    if (need_sum) {
      const float share = (1.f - set.top_p) * sum * (1.f - 0x1p-10f) / static_cast<float>(a.V);
      if (share > 0.f)
        bound = max(key_of(M + (__log2f(share) - 0x1p-10f) / st.pw.kh), kmin);
    }
    const uint32_t want = need_sum ? kWant : static_cast<uint32_t>(set.k);
    // in 256 bins from the largest logit down, over as much as the threads' maxima span, 64 octaves
    // or units at most; a logit further down is in the last bin, which bounds nothing
    for (int i = tid; i < kMaximaBins; i += kThreads) sh.group[i] = 0;
    uint32_t lo = __reduce_min_sync(0xFFFFFFFFu, mykey > kNegInfKey ? mykey : 0xFFFFFFFFu);
    if (lane == 0) sh.warp[warp] = lo;  // warpu may still be read
    __syncthreads();
    lo = __reduce_min_sync(0xFFFFFFFFu,
                           lane < kWarps ? static_cast<uint32_t>(sh.warp[lane]) : 0xFFFFFFFFu);
    const float range = fminf(M - key_value(lo), fmaxf(64.f, 64.f / st.pw.kh));
    const float per_bin = range * (1.f / 254.f), inv = per_bin > 0.f ? 1.f / per_bin : 0.f;
    for (int b = 0; b < blocks; ++b) {
      const float t = sh.top[b * kThreads + tid];
      if (t > -INFINITY) atomicAdd(&sh.group[static_cast<int>(fminf((M - t) * inv, 255.f))], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // a lane has eight bins; the first at which k maxima are reached
      uint32_t count[8], part = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) part += count[i] = sh.group[lane * 8 + i];
      uint32_t at = part;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, at, o);
        if (lane >= o) at += up;
      }
      at -= part;
      if (lane == 0) sh.bound = kNegInfKey + 1;
      __syncwarp();
      int last = -1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int bin = lane * 8 + i;
        // every maximum of the bins up to this one is above its lower end
        if (at < want && want <= at + count[i] && bin < 255) {
          sh.bound = max(key_of(M - (static_cast<float>(bin) + 1.01f) * per_bin), kNegInfKey + 1);
          last = bin;
        }
        at += count[i];
      }
      if (need_sum) {
        // a nucleus far beyond the list needs none: what the maxima hold, at most, and half as much more
        last = __reduce_max_sync(0xFFFFFFFFu, last);
        float held = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (lane * 8 + i <= last)
            held += static_cast<float>(count[i]) *
                    ex2_approx(static_cast<float>(-(lane * 8 + i)) * per_bin * st.pw.kh);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) held += __shfl_xor_sync(0xFFFFFFFFu, held, o);
        if (lane == 0) sh.hopeless = sh.bound > bound && held * 1.5f < set.top_p * sum ? 1 : 0;
      }
    }
    __syncthreads();
    bound = max(bound, sh.bound);
  }
  const bool whole_row = bound <= kNegInfKey + 1;  // all that is not -inf
  bool done = (list_k || need_sum || list_min) && (!whole_row || list_min || a.V <= kCap) &&
              sh.hopeless == 0;
  bound = max(bound, kNegInfKey + 1);
  // each block is at most so many times its maximum: a bound of the sum of all, for the scale
  float held = 0.f;
  if (!need_sum && !list_k) {
    for (int b = 0; b < blocks; ++b) held += ex2_approx((sh.top[b * kThreads + tid] - M) * st.pw.kh);
    held *= static_cast<float>(block * E::kVec);
  }
  if (done) {
    // the blocks to be read again
    const float least = key_value(bound);
    for (int b = 0; b < blocks; ++b) {
      const bool again = tmax >= least && sh.top[b * kThreads + tid] >= least;
      const unsigned who = __ballot_sync(0xFFFFFFFFu, again);
      if (who == 0) continue;
      int at = 0;
      if (lane == 0) at = atomicAdd(&sh.items, __popc(who));
      at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(who & ((1u << lane) - 1u));
      if (again && at < kItems<kThreads>) sh.item[at] = static_cast<uint16_t>(b * kThreads + tid);
    }
    __syncthreads();
    const int items = sh.items <= kItems<kThreads> ? sh.items : 0;
    if (tid == 0 && sh.items > kItems<kThreads>) sh.n = kCap + 1;
    // all their vectors at once, kUnroll of a thread in flight; the scale meanwhile
    const int vecs = items * block;
    for (int i0 = tid; i0 < vecs; i0 += kUnroll * kThreads) {
      int at[kUnroll];
#pragma unroll
      for (int n = 0; n < kUnroll; ++n) {
        const int i = i0 + n * kThreads;
        at[n] = -1;
        if (i < vecs) {
          const int q = i / block, it = sh.item[q];
          const int step = it / kThreads * block + (i - q * block);
          const int j = it % kThreads + step * kThreads;
          if (step < steps && j < nvec) at[n] = j;
        }
        if (at[n] >= 0) x[n] = r.load(at[n]);
      }
      if (*static_cast<volatile int*>(&sh.n) > kCap) break;  // full: nothing more is looked for
#pragma unroll
      for (int n = 0; n < kUnroll; ++n) {
        if (at[n] < 0 || !(max_of<kDtype>(x[n]) >= least)) continue;
        float v[E::kVec];
        E::unpack(x[n], v);
#pragma unroll
        for (int e = 0; e < E::kVec; ++e) {
          if (v[e] >= least) {
            const int to = atomicAdd(&sh.n, 1);
            if (to < kCap)
              sh.key[to] = (static_cast<u64>(key_of(v[e])) << 32) |
                           static_cast<uint32_t>(~static_cast<uint32_t>(at[n] * E::kVec + e - r.shift));
          }
        }
      }
    }
    set_scale(st, need_sum ? sum : static_cast<float>(kCap));
    __syncthreads();
    const int n = sh.n;
    done = n <= kCap;
    if (done) {
      // with all tokens in the list, top-p's total is the list's
      const bool by_sum = need_sum && !whole_row;
      done = decide(a, st, sh, row, set.u, n, need_sum && whole_row ? n : set.k,
                              set.top_p, kmin, bound == kmin, by_sum ? sum : 0.f);
    }
  }
  if (done) return;

  // ---- all of the row again
  Deep<kDtype, kThreads, Args> deep{a,        sh.deep, sh.scratch, sh.table, sh.warp, sh.total,
                              sh.warpu, r,       st,         tid,      warp,    lane};
  // the scale: a bound of the sum of all, near enough; top-k's maxima are overwritten
  const float most = need_sum ? sum * 1.001f : list_k ? deep.bound() : deep.total_of(held);
  set_scale(deep.st, most);
  deep.filtered(row, set.u, set.k, set.top_p, kmin, most);
}

}  // namespace sampling
}  // namespace tim
