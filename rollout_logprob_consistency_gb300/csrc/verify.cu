// Verification of drafted tokens against a target's logits, from given uniform numbers.
//
// Per sequence, with p_j and q_j the distributions that the sampler's filters leave of the target's
// and the drafter's logits at position j (sample_list.cuh; without a drafter's logits q_j is certain
// of x_j):
//   x_j is accepted while  u_j q_j(x_j) < p_j(x_j)
//   at the first that is not, the token is drawn from r = max(p_j - q_j, 0): the smallest v with
//   sum_{w <= v} r_w > u' sum r  (from p where r is next to nothing);  after the last draft, from p
// so that what comes out is distributed as p, whatever q is.
//
// Two launches.  The first is the sampler's main kernel over the rows of both matrices, position by
// position: it leaves each row's border (the last token kept), its normaliser and, for the target's,
// the token that u' draws from p.  With more rows than SMs the CTA that is the second to finish a
// position's two rows decides on its draft, and rows behind a refused draft that have not been begun
// by then are not read: nothing of the result comes from them.  The second launch has a cluster of
// CTAs for each sequence.  Where a draft is refused its two rows are read again, mostly from L2: p and q
// as 64-bit integers at scale 2^60, good to 2^-30.3 each, so that the sums of max(p - q, 0) are exact
// in that scale and do not depend on the split; the part of the row into which the border falls is
// shared out among its CTA, and a warp walks its piece.
//
// 128 sequences of four drafts over 151936 bf16 tokens without filters take 143 us and 56: the first
// launch weighs every token of the rows that are needed (as tim_sample, bound by the integer pipe; 170 us
// with all rows), the second two weights a token of 90 row pairs.  48
// sequences with settings of their own take 103 us and 25: the longest rows are nuclei of tens of
// thousands of tokens.  One sequence takes 30 us from a cold L2 where all its drafts are accepted and
// 44 where one is refused: chains of dependent steps.
#include "verify.cuh"

#include <algorithm>
#include <type_traits>

#include "sample_list.cuh"

namespace tim {

using namespace sampling;

namespace {

// What the first launch leaves of a row.
struct alignas(16) VerifyRow {
  u64 border;          // key << 32 | ~id of the last token kept
  float M;             // largest logit
  float lse_h, lse_l;  // ln sum_kept exp(s) - M / tau as a pair
  float logprob;       // of the token drawn
  int id;              // the token drawn
  int bad;
};

// What is decided of a draft: ln p of the token, and the code of a position that cannot be decided.
struct Decision {
  float logprob;
  int code;
};

struct VerifyArgs {
  static constexpr bool kBorder = true;
  VerifyMatrix target, draft;
  int64_t B;
  int N, V, dtype;
  int cluster;   // CTAs of a sequence in the second launch
  bool in_rows;  // drafts are decided on as their rows are finished; else by the second launch
  const int32_t* ids;
  const float* uniform;
  const float* uniform_draw;
  tim_sample_params target_set, draft_set;
  VerifyRow* rows;    // B (N + 1) of the target, B N of the draft
  Decision* decided;     // B N
  uint32_t* refused;  // B: the first position that ends a sequence, all ones at first
  uint32_t* done;     // B N: finished rows of a position, less one at first
  int32_t* out_ids;
  float* out_logprob;
  int32_t* out_accepted;
  int* status;
};
__host__ __device__ __forceinline__ bool draft_given(const VerifyArgs& a) {
  return a.draft.logits != nullptr;
}

// A row of the first launch: position by position, in each the sequences' target and draft.
struct Where {
  int64_t b;
  int j;
  bool target;
};
__device__ __forceinline__ Where where(const VerifyArgs& a, int64_t at) {
  const uint32_t row = static_cast<uint32_t>(at);  // B (2 N + 1) < 2^28
  const uint32_t of = static_cast<uint32_t>(draft_given(a) ? 2 * a.B : a.B), j = row / of;
  const uint32_t i = row - j * of;
  const bool pair = draft_given(a) && static_cast<int>(j) < a.N;
  return Where{static_cast<int64_t>(pair ? i >> 1 : i), static_cast<int>(j), !pair || (i & 1) == 0};
}
__device__ __forceinline__ VerifyRow& state_of(const VerifyArgs& a, const Where& w) {
  return a.rows[w.target ? w.b * (a.N + 1) + w.j : a.B * (a.N + 1) + w.b * a.N + w.j];
}
template <int kDtype>
__device__ __forceinline__ Row<kDtype> row_of(const VerifyArgs& a, int64_t row) {
  using raw = typename Elem<kDtype>::raw;
  const Where w = where(a, row);
  const VerifyMatrix& m = w.target ? a.target : a.draft;
  return Row<kDtype>(static_cast<const raw*>(m.logits) + w.b * m.ld_seq + w.j * m.ld_pos, 0, 0, a.V);
}
__device__ __forceinline__ bool refused_before(const VerifyArgs& a, const Where& w) {
  return __ldcg(a.refused + w.b) < static_cast<uint32_t>(w.j);
}
// Rows behind the end of a sequence's drafts are not read (the target's at the end still is), nor those
// behind a refused draft.
__device__ __forceinline__ bool wanted(const VerifyArgs& a, int64_t row) {
  const Where w = where(a, row);
  const int32_t* const ids = a.ids + w.b * a.N;
  const int n = w.target ? w.j : w.j + 1;
  bool all = true;
  for (int i = threadIdx.x & 31; i < n; i += 32) all = all && __ldg(ids + i) >= 0;
  all = __all_sync(0xFFFFFFFFu, all);
  if (!a.in_rows) {
    pdl_launch_dependents();  // the second launch may load its tables
    return all;
  }
  return __syncthreads_and(all && !refused_before(a, w)) != 0;
}
__device__ __forceinline__ bool in_range(float u) { return u >= 0.f && u < 1.f; }
__device__ __forceinline__ Settings settings_of(const VerifyArgs& a, int64_t b, bool target) {
  const tim_sample_params &p = a.target_set, &q = a.draft_set;
  SampleArgs s;
  s.V = a.V;
  s.uniform = a.uniform_draw;
  s.temperature = target ? p.temperature : q.temperature;
  s.top_k = target ? p.top_k : q.top_k;
  s.top_p = target ? p.top_p : q.top_p;
  s.min_p = target ? p.min_p : q.min_p;
  s.row_temperature = target ? p.row_temperature : q.row_temperature;
  s.row_top_k = target ? p.row_top_k : q.row_top_k;
  s.row_top_p = target ? p.row_top_p : q.row_top_p;
  s.row_min_p = target ? p.row_min_p : q.row_min_p;
  return settings_of(s, b);
}
__device__ __forceinline__ Settings settings_of(const VerifyArgs& a, int64_t row) {
  const Where w = where(a, row);
  return settings_of(a, w.b, w.target);
}

__device__ __forceinline__ bool keeps(const VerifyRow& r, float z, int id) {
  return ((static_cast<u64>(key_of(z)) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(id))) >=
         r.border;
}
// ln of the probability of a kept token of logit z
__device__ __forceinline__ Df log_prob(const VerifyRow& r, float z, float tau) {
  return (df(z) - df(r.M)) * reciprocal(df(tau)) - Df{r.lse_h, r.lse_l};
}
// ln u for 0 < u < 1
__device__ __forceinline__ Df log_uniform(float u) {
  return u < 0x1p-100f ? log_df(df(u * 0x1p100f)) - Df{kLn2Hi, kLn2Lo} * df(100.f) : log_df(df(u));
}
__device__ __forceinline__ VerifyRow read_row(const VerifyRow* p) {
  static_assert(sizeof(VerifyRow) == 32, "two vectors");
  uint4 v[2] = {__ldcg(reinterpret_cast<const uint4*>(p)), __ldcg(reinterpret_cast<const uint4*>(p) + 1)};
  return *reinterpret_cast<const VerifyRow*>(v);
}

// Whether the draft of a position whose rows are finished is accepted.
template <int kDtype>
__device__ __forceinline__ Decision decide_draft(const VerifyArgs& a, int64_t b, int j, bool& accepted) {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  const int64_t at = b * a.N + j;
  const int id = __ldg(a.ids + at);
  const VerifyRow p = read_row(a.rows + b * (a.N + 1) + j);
  const float u = __ldg(a.uniform + at);
  Decision r = {0.f, p.bad};
  accepted = false;
  if (id >= a.V) r.code = TIM_ERR_TOKEN_RANGE;
  if (r.code == 0 && !in_range(u)) r.code = TIM_ERR_INVALID_ARG;
  if (r.code != 0) return r;
  const float z = E::widen(
      __ldg(static_cast<const raw*>(a.target.logits) + b * a.target.ld_seq + j * a.target.ld_pos + id));
  const Df ln_p = log_prob(p, z, settings_of(a, b, true).tau);
  Df ln_q = df(0.f);
  bool certain = u == 0.f;  // whatever q is
  if (draft_given(a)) {
    const VerifyRow q = read_row(a.rows + a.B * (a.N + 1) + at);
    const float zq = E::widen(
        __ldg(static_cast<const raw*>(a.draft.logits) + b * a.draft.ld_seq + j * a.draft.ld_pos + id));
    r.code = q.bad;
    certain = certain || !keeps(q, zq, id);
    ln_q = log_prob(q, zq, settings_of(a, b, false).tau);
  }
  // in logarithms: p and q may both lie below the range of a float
  accepted = r.code == 0 && keeps(p, z, id) && (certain || (log_uniform(u) + ln_q - ln_p).h < 0.f);
  r.logprob = ln_p.h;
  return r;
}

// A row of a position is finished: the last of them decides on its draft.
template <int kDtype>
__device__ __noinline__ void finished(const VerifyArgs& a, int64_t b, int j) {
  const int64_t at = b * a.N + j;
  if (j >= a.N || __ldg(a.ids + at) < 0) return;
  __threadfence();
  if (draft_given(a)) {
    if (atomicAdd(a.done + at, 1u) == 0xFFFFFFFFu) return;
    __threadfence();
  }
  bool accepted;
  a.decided[at] = decide_draft<kDtype>(a, b, j, accepted);
  if (!accepted) atomicMin(a.refused + b, static_cast<uint32_t>(j));
}

__device__ __forceinline__ void leave(const VerifyArgs& a, int64_t row, const VerifyRow& r) {
  const Where w = where(a, row);
  state_of(a, w) = r;
  if (!a.in_rows) return;
  a.dtype == TIM_F32    ? finished<TIM_F32>(a, w.b, w.j)
  : a.dtype == TIM_BF16 ? finished<TIM_BF16>(a, w.b, w.j)
                        : finished<TIM_F16>(a, w.b, w.j);
}
// What cannot be read ends its sequence, if that gets there: only then is it reported.
__device__ __forceinline__ void write_bad(const VerifyArgs& a, int64_t row, int code) {
  VerifyRow r = {};
  r.bad = code;
  leave(a, row, r);
}
__device__ __forceinline__ void write_row(const VerifyArgs& a, const RowState& st,
                                          const Tables& tables, int64_t row, int id, float x,
                                          u64 total, int n, u64 border) {
  VerifyRow r;
  const float base = st.pw.recentre ? st.pw.c : 0.f;
  const Df ln = n == 1 ? df(0.f)
                       : log_total(total, st.top, tables) + (df(base) - df(st.M)) * st.inv_tau;
  r.border = border;
  r.M = st.M;
  r.lse_h = ln.h;
  r.lse_l = ln.l;
  r.logprob = n == 1 ? 0.f : ((df(x) - df(st.M)) * st.inv_tau - ln).h;
  r.id = id;
  r.bad = 0;
  leave(a, row, r);
}

// ---- the second launch

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct FinishShared {
  Tables fine;
  uint32_t table[2][256];
  u64 part[kMaxCluster * kWarps];  // of every warp of every CTA
  u64 step[kWarps];
  u64 left;
  int n, refused, bad, owner, found;
};

// A row of one matrix at the refused position: its kept tokens' probabilities at scale 2^60,
// 2^((z - M) K - lse log2e).  What is added to z K, as a multiple of 1/256, goes to the exponent
// (weights_of_two takes any), the rest of it into a table of the row's own, so that what is expanded
// stays within 2^-9.  Where z K itself is too large to split, z - M is taken first.
template <int kDtype>
struct Dist {
  const typename Elem<kDtype>::raw* p;
  float zc, M, kh, kl, magic;  // kept: above zc, or zc with an id up to idc
  int idc;
  bool all, recentre;  // all: whatever is above -inf is kept
  const uint32_t* table;

  __device__ __forceinline__ void set(const VerifyRow& r, const void* logits, float tau, uint32_t* to,
                                      const Tables& fine) {
    const Df K = Df{kLog2eHi, kLog2eLo} * reciprocal(df(tau));
    p = static_cast<const typename Elem<kDtype>::raw*>(logits);
    zc = key_value(static_cast<uint32_t>(r.border >> 32));
    idc = static_cast<int>(min(~static_cast<uint32_t>(r.border), 0x7FFFFFFFu));
    all = r.border <= kAllKept;
    M = r.M;
    kh = K.h;
    kl = K.l;
    const Df mk = df(M) * K;
    recentre = !(fabsf(mk.h) < 8192.f);
    Df c = Df{kLog2eHi, kLog2eLo} * Df{-r.lse_h, -r.lse_l};
    if (!recentre) c = c - mk;
    const float whole = rintf(c.h * 256.f) * (1.f / 256.f);
    magic = kPow2Magic + whole;
    table = to;
    const Df rest = renorm(c.h - whole, c.l);
    const Df f = pow2_df(rest.h, Pow2Row{1.f, 0.f, 0.f, false}, fine.fine) *
                 (df(1.f) + Df{kLn2Hi, kLn2Lo} * df(rest.l));
    // f at scale 2^48 (its leading part is a multiple of 2^-24), 2^(j/256) at scale 2^62
    const u64 scaled = (static_cast<u64>(f.h * 0x1p24f) << 24) +
                       static_cast<u64>(static_cast<int64_t>(f.l * 0x1p48f));
    for (int j = threadIdx.x; j < 256; j += kThreads) {
      const u64 t = __umul64hi(fine.fine[j], scaled << 14);  // scale 2^60
      const int down = j <= 128 ? 29 : 30;
      to[j] = static_cast<uint32_t>((t + (1ull << (down - 1))) >> down);
    }
  }
  __device__ __forceinline__ float keep(float z, int id) const {
    return z > zc || (z == zc && id <= idc) ? z : -INFINITY;
  }
  // of a logit far from 0; rare, and not worth its place between the others
  __device__ __noinline__ u64 far(float z) const {
    // z - M = d + e exactly
    const float d = z - M, b = d - z, e = (z - (d - b)) + (-M - b);
    if (!(d * kh > -128.f)) return 0;
    const float t = fmaf(d, kh, magic);
    const float g = fmaf(e, kh, fmaf(d, kl, fmaf(d, kh, magic - t)));
    return weight_of(t, g, shift_of(2), table);
  }
  // of the tokens id and id + 1
  __device__ __forceinline__ void two(float z0, float z1, int id, u64& w0, u64& w1) const {
    if (!all) {
      z0 = keep(z0, id);
      z1 = keep(z1, id + 1);
    }
    if (recentre) {
      w0 = far(z0);
      w1 = far(z1);
    } else {
      weights_of_two(z0, z1, pair_scale(kh, kl, magic), shift_of(2), table, w0, w1);
    }
  }
};

// kWide: both rows in 16-byte vectors, which begin `shift` tokens before them; else token by token.
template <int kDtype, bool kWide>
struct Residual {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  static constexpr int kOf = kWide ? E::kVec : 1;  // tokens a lane looks at together
  using Loaded = std::conditional_t<kWide, uint4, raw>;
  const Dist<kDtype>&p, &q;
  int V, shift, x;  // x: what the drafter is certain of, -1 with its logits

  __device__ __forceinline__ int groups() const { return (shift + V + kOf - 1) / kOf; }
  __device__ __forceinline__ Loaded load(const raw* row, int j) const {
    const int id0 = j * kOf - shift;
    if constexpr (kWide) {
      if (id0 >= 0 && id0 + kOf <= V) return __ldg(reinterpret_cast<const uint4*>(row + id0));
      float z[kOf];
#pragma unroll
      for (int i = 0; i < kOf; ++i)
        z[i] = id0 + i >= 0 && id0 + i < V ? E::widen(row[id0 + i]) : -INFINITY;
      return E::pack(z);
    } else {
      return __ldg(row + id0);
    }
  }
  // f(token, r of it) in order, of group j's tokens that have any; two at a time, so that few are held.
  template <class F>
  __device__ __forceinline__ void each(const Loaded& lp, const Loaded& lq, int j, F&& f) const {
    constexpr int kHeld = kOf + kOf % 2;
    const int id0 = j * kOf - shift;
    float zp[kHeld], zq[kHeld];
    if constexpr (kWide) {
      E::unpack(lp, zp);
      E::unpack(lq, zq);
    } else {
      zp[0] = E::widen(lp);
      zq[0] = E::widen(lq);
      zp[1] = zq[1] = -INFINITY;
    }
    bool any = false;
#pragma unroll
    for (int i = 0; i < kOf; ++i) any |= zp[i] >= p.zc;
    if (!any) return;
#pragma unroll
    for (int i = 0; i < kHeld; i += 2) {
      u64 a0, a1, b0, b1;
      p.two(zp[i], zp[i + 1], id0 + i, a0, a1);
      if (x < 0) {
        q.two(zq[i], zq[i + 1], id0 + i, b0, b1);
      } else {
        b0 = id0 + i == x ? a0 : 0;
        b1 = id0 + i + 1 == x ? a1 : 0;
      }
      f(id0 + i, a0 > b0 ? a0 - b0 : 0);
      f(id0 + i + 1, a1 > b1 ? a1 - b1 : 0);
    }
  }

  // The token, in every thread of the CTA that has it; -1 in the others, -2 where r sums to less than
  // 2^-28: p and q are good to 2^-30.3 each, so two that agree leave up to 2^-29.3.
  //
  // Sums over parts of the row, one a warp of the cluster, then over pieces of the part that the border falls
  // into, one a warp of its CTA; a warp then walks its piece.
  __device__ __forceinline__ int draw(FinishShared& sh, float u, int cluster) const {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_rank()), parts = cluster * kWarps;
    const int part = (groups() + parts * 32 - 1) / (parts * 32) * 32;
    const raw* const other = x < 0 ? q.p : p.p;
    int j0 = min(groups(), (rank * kWarps + warp) * part), j1 = min(groups(), j0 + part);
    if (tid == 0) sh.owner = sh.found = -1;
#pragma unroll 1
    for (int level = 0;; ++level) {
      u64 sum = 0;
      Loaded lp, lq;
      int j = j0 + lane;
      if (j < j1) {
        lp = load(p.p, j);
        lq = load(other, j);
      }
      while (j < j1) {  // the next vectors are on their way meanwhile
        const int at = j;
        const Loaded zp = lp, zq = lq;
        j += 32;
        if (j < j1) {
          lp = load(p.p, j);
          lq = load(other, j);
        }
        each(zp, zq, at, [&](int, u64 r) { sum += r; });
      }
      sum = warp_sum(sum);
      if (level == 0) {
        const int mine = rank * kWarps + warp;
        if (lane < cluster) cluster_store(cluster_addr(&sh.part[mine], lane), sum);
        cluster_arrive();
        cluster_wait();
        u64 before = 0, total = 0;
        for (int i = lane; i < parts; i += 32) {
          total += sh.part[i];
          before += i < mine ? sh.part[i] : 0;
        }
        total = warp_sum(total);
        before = warp_sum(before);
        if (total < 1ull << 32) return -2;
        const u64 target = draw_target(total, u);
        if (before <= target && target < before + sum && lane == 0) {
          sh.owner = warp;
          sh.left = target - before;
        }
        __syncthreads();
        if (sh.owner < 0) return -1;
        const int o0 = min(groups(), (rank * kWarps + sh.owner) * part), o1 = min(groups(), o0 + part);
        const int piece = (part / 32 + kWarps - 1) / kWarps * 32;
        j0 = min(o1, o0 + warp * piece);
        j1 = min(o1, j0 + piece);
        continue;
      }
      if (lane == 0) sh.step[warp] = sum;
      __syncthreads();
      const u64 target = sh.left;
      u64 before = 0;
      for (int i = 0; i < warp; ++i) before += sh.step[i];
      if (before <= target && target < before + sum) {
        for (int i = j0; i < j1; i += 32) {
          u64 r[kOf + kOf % 2] = {}, here = 0;
          j = i + lane;
          if (j < j1) {
            int n = 0;
            each(load(p.p, j), load(other, j), j, [&](int, u64 x) {
              r[n++] = x;
              here += x;
            });
          }
          const u64 to = warp_scan(here), all = __shfl_sync(0xFFFFFFFFu, to, 31);
          if (target < before + all) {
            u64 at = before + to - here;
#pragma unroll
            for (int n = 0; n < kOf; ++n) {
              if (at <= target && target < at + r[n]) sh.found = j * kOf - shift + n;
              at += r[n];
            }
            break;
          }
          before += all;
        }
      }
      __syncthreads();
      return sh.found;
    }
  }
};

// What comes of a sequence's drafts, by one warp: writes those that are accepted; sh.n of them, the token
// that is refused there or -1, and the code of a position that cannot be decided.
template <int kDtype>
__device__ __forceinline__ void gather_drafts(const VerifyArgs& a, int64_t b, bool writes,
                                              FinishShared& sh) {
  const int lane = threadIdx.x & 31;
  const int32_t* const ids = a.ids + b * a.N;
  const uint32_t known = a.in_rows ? a.refused[b] : 0xFFFFFFFFu;
  for (int j0 = 0; j0 <= a.N; j0 += 32) {
    const int j = j0 + lane;
    const int id = j < a.N ? __ldg(ids + j) : -1;
    // up to the end of the drafts or the first that was refused
    const unsigned ends = __ballot_sync(0xFFFFFFFFu, id < 0 || static_cast<uint32_t>(j) >= known);
    const int end = ends != 0 ? __ffs(ends) - 1 : 32;
    Decision r = {0.f, 0};
    bool accepted = false;
    if (lane < end && a.in_rows) {
      r = a.decided[b * a.N + j];
      accepted = true;
    } else if (lane < end) {
      r = decide_draft<kDtype>(a, b, j, accepted);
    } else if (lane == end) {
      if (id >= 0)
        r = a.decided[b * a.N + j];
      else
        r.code = id < -1 ? TIM_ERR_TOKEN_RANGE : a.rows[b * (a.N + 1) + j].bad;
    }
    const unsigned stops = __ballot_sync(0xFFFFFFFFu, !accepted);
    const int n = stops != 0 ? __ffs(stops) - 1 : 32;  // accepted of these
    if (writes && lane < n) {
      a.out_ids[b * (a.N + 1) + j] = id;
      a.out_logprob[b * (a.N + 1) + j] = r.logprob;
    }
    if (stops != 0) {
      if (lane == n) {
        sh.n = j;
        sh.refused = id;
        sh.bad = r.code;
      }
      return;
    }
  }
}

template <int kDtype>
__global__ void __launch_bounds__(kThreads, 2) verify_finish_kernel(const VerifyArgs a) {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  __shared__ FinishShared sh;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / a.cluster, out = b * (a.N + 1);
  const bool writes = cluster_rank() == 0;
  const VerifyRow* const ps = a.rows + b * (a.N + 1);
  const VerifyRow* const qs = a.rows + a.B * (a.N + 1) + b * a.N;
  const raw* const target = static_cast<const raw*>(a.target.logits) + b * a.target.ld_seq;
  const raw* const draft = static_cast<const raw*>(a.draft.logits) + b * a.draft.ld_seq;
  const float tau = settings_of(a, b, true).tau, draft_tau = settings_of(a, b, false).tau;
  cluster_arrive();
  load_tables(sh.fine, tid, kThreads);
  pdl_wait();
  if (tid < 32) gather_drafts<kDtype>(a, b, writes, sh);
  __syncthreads();
  cluster_wait();  // every CTA of the cluster runs
  const int n = sh.n, refused = sh.refused;
  if (sh.bad != 0) {  // the same in every CTA of the cluster, here and below
    if (!writes) return;
    if (tid == 0) {
      set_status(a.status, sh.bad);
      a.out_accepted[b] = 0;
    }
    for (int j = tid; j <= a.N; j += kThreads) {
      a.out_ids[out + j] = -1;
      a.out_logprob[out + j] = __int_as_float(0x7FC00000);
    }
    return;
  }
  if (writes) {
    if (tid == 0) a.out_accepted[b] = n;
    for (int j = n + 1 + tid; j <= a.N; j += kThreads) {
      a.out_ids[out + j] = -1;
      a.out_logprob[out + j] = 0.f;
    }
  }
  const VerifyRow p = ps[n];
  int id = -2;
  if (refused >= 0) {
    Dist<kDtype> P, Q;
    const raw* const z = target + static_cast<int64_t>(n) * a.target.ld_pos;
    const raw* const zq = draft + static_cast<int64_t>(n) * a.draft.ld_pos;
    P.set(p, z, tau, sh.table[0], sh.fine);
    if (draft_given(a)) Q.set(qs[n], zq, draft_tau, sh.table[1], sh.fine);
    __syncthreads();
    const float u = __ldg(a.uniform_draw + b);
    const int x = draft_given(a) ? -1 : refused;
    const uintptr_t at = reinterpret_cast<uintptr_t>(z);
    if (x >= 0 || ((at ^ reinterpret_cast<uintptr_t>(zq)) & 15u) == 0)
      id = Residual<kDtype, true>{P, Q, a.V, static_cast<int>((at & 15u) / sizeof(raw)), x}.draw(sh, u, a.cluster);
    else
      id = Residual<kDtype, false>{P, Q, a.V, 0, x}.draw(sh, u, a.cluster);
  }
  if (tid != 0) return;
  if (id >= 0) {
    a.out_ids[out + n] = id;
    a.out_logprob[out + n] =
        log_prob(p, E::widen(target[static_cast<int64_t>(n) * a.target.ld_pos + id]), tau).h;
  } else if (id == -2 && writes) {  // the target's own draw
    a.out_ids[out + n] = p.id;
    a.out_logprob[out + n] = p.logprob;
  }
}

template <int kDtype>
cudaError_t launch_type(const VerifyArgs& a, cudaStream_t stream, int num_sms) {
  const int64_t rows = a.B * (a.N + 1) + (draft_given(a) ? a.B * a.N : 0);
  const unsigned g = static_cast<unsigned>(rows);
  // As few threads a row as let the rows of a position run at once (sample.cu has the same for all its
  // rows): the next position's then come when something is known of this one's drafts.
  const int64_t wave = a.in_rows ? (draft_given(a) ? 2 * a.B : a.B) : rows;
  if (wave <= num_sms)
    sample_list_kernel<kDtype, 1024, VerifyArgs><<<g, 1024, 0, stream>>>(a);
  else if (wave <= 2 * num_sms)
    sample_list_kernel<kDtype, 512, VerifyArgs><<<g, 512, 0, stream>>>(a);
  else if (wave <= 4 * num_sms)
    sample_list_kernel<kDtype, 256, VerifyArgs><<<g, 256, 0, stream>>>(a);
  else
    sample_list_kernel<kDtype, 128, VerifyArgs><<<g, 128, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Where all rows run at once the second launch comes up beside them and waits for their end: one
  // sequence 29 us so, 34 without.
  if (a.B * a.cluster > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.in_rows ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, verify_finish_kernel<kDtype>, a);
}

struct VerifyWs {
  size_t rows_off, decided_off, counts_off, counts, total;
};
VerifyWs verify_ws(int64_t B, int32_t N) {
  const size_t b = static_cast<size_t>(B), n = static_cast<size_t>(N);
  VerifyWs w;
  w.rows_off = 1024;
  w.decided_off = w.rows_off + b * (2 * n + 1) * sizeof(VerifyRow);
  w.counts_off = w.decided_off + b * n * sizeof(Decision);
  w.counts = b * (n + 1) * 4;
  w.total = align_up(w.counts_off + w.counts, 1024);
  return w;
}

}  // namespace

size_t verify_bytes(int64_t B, int32_t N) { return verify_ws(B, N).total; }

cudaError_t launch_verify(const VerifyMatrix& target, const VerifyMatrix& draft, int dtype, int64_t B,
                          int N, int V, const int32_t* ids, const float* uniform,
                          const float* uniform_draw, const tim_sample_params& target_set,
                          const tim_sample_params& draft_set, int32_t* out_ids, float* out_logprob,
                          int32_t* out_accepted, void* ws, cudaStream_t stream, int num_sms) {
  VerifyArgs a = {};
  a.target = target;
  a.draft = draft;
  a.B = B;
  a.N = N;
  a.V = V;
  a.ids = ids;
  a.uniform = uniform;
  a.uniform_draw = uniform_draw;
  a.target_set = target_set;
  a.draft_set = draft_set;
  const VerifyWs w = verify_ws(B, N);
  uint8_t* const mem = static_cast<uint8_t*>(ws);
  a.dtype = dtype;
  a.rows = reinterpret_cast<VerifyRow*>(mem + w.rows_off);
  a.decided = reinterpret_cast<Decision*>(mem + w.decided_off);
  a.refused = reinterpret_cast<uint32_t*>(mem + w.counts_off);
  a.done = a.refused + B;
  a.out_ids = out_ids;
  a.out_logprob = out_logprob;
  a.out_accepted = out_accepted;
  a.status = static_cast<int*>(ws);
  // Eight CTAs a sequence up to a third of the SMs, four beyond: what is done once a CTA (the drafts, the
  // tables) then weighs less.  Both launches with eight and with four, 4 drafts, 151936 bf16 tokens, unfiltered:
  // 24 sequences 95 us and 96, 48 123 and 133, 56 137 and 137, 64 145 and 139, 128 221 and 210 (in the
  // second launch alone 65 and 55, two: 62); with top-k 50 and top-p 0.95 56 sequences 109 and 101.
  a.cluster = 3 * B <= num_sms ? kMaxCluster : kMaxCluster / 2;
  // Rows that run all at once have nothing to gain from what the others say, and a chain less each.
  a.in_rows = B * (N + 1) + (draft_given(a) ? B * N : 0) > num_sms;
  if (a.in_rows) {
    const cudaError_t e = cudaMemsetAsync(a.refused, 0xFF, w.counts, stream);
    if (e != cudaSuccess) return e;
  }
  return dtype == TIM_F32    ? launch_type<TIM_F32>(a, stream, num_sms)
         : dtype == TIM_BF16 ? launch_type<TIM_BF16>(a, stream, num_sms)
                             : launch_type<TIM_F16>(a, stream, num_sms);
}

}  // namespace tim
