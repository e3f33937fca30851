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
// Two launches.  The first is the sampler's main kernel over all rows of both matrices at once: it
// leaves each row's border (the last token kept), its normaliser and, for the target's, the token
// that u' draws from p.  The second has a cluster of CTAs for each sequence: every CTA decides on the
// drafts (a lane a position, few loads), and where one is refused its two rows are read again, mostly
// from L2: p and q as 64-bit integers at scale 2^60, good to 2^-30.3 each, so that the sums of
// max(p - q, 0) are exact in that scale and do not depend on the split; the warp in whose part of the
// row the border falls walks it once more.
#include "verify.cuh"

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

struct VerifyArgs {
  static constexpr bool kBorder = true;
  VerifyMatrix target, draft;
  int64_t B;
  int N, V;
  const int32_t* ids;
  const float* uniform;
  const float* uniform_draw;
  tim_sample_params target_set, draft_set;
  VerifyRow* rows;  // B (N + 1) of the target, B N of the draft
  int32_t* out_ids;
  float* out_logprob;
  int32_t* out_accepted;
  int* status;
};
__host__ __device__ __forceinline__ bool draft_given(const VerifyArgs& a) {
  return a.draft.logits != nullptr;
}

// A row of the first launch: the target's first, then the drafter's.
struct Where {
  int64_t b;
  int j;
  bool target;
};
__device__ __forceinline__ Where where(const VerifyArgs& a, int64_t row) {
  const int64_t targets = a.B * (a.N + 1);
  Where w;
  w.target = row < targets;
  const int of = w.target ? a.N + 1 : a.N;
  if (!w.target) row -= targets;
  w.b = row / of;
  w.j = static_cast<int>(row - w.b * of);
  return w;
}
template <int kDtype>
__device__ __forceinline__ Row<kDtype> row_of(const VerifyArgs& a, int64_t row) {
  using raw = typename Elem<kDtype>::raw;
  const Where w = where(a, row);
  const VerifyMatrix& m = w.target ? a.target : a.draft;
  return Row<kDtype>(static_cast<const raw*>(m.logits) + w.b * m.ld_seq + w.j * m.ld_pos, 0, 0, a.V);
}
// Rows behind the end of a sequence's drafts are not read: the target's at the end still is.
__device__ __forceinline__ bool wanted(const VerifyArgs& a, int64_t row) {
  const Where w = where(a, row);
  const int32_t* const ids = a.ids + w.b * a.N;
  const int n = w.target ? w.j : w.j + 1;
  bool all = true;
  for (int i = threadIdx.x & 31; i < n; i += 32) all = all && __ldg(ids + i) >= 0;
  return __all_sync(0xFFFFFFFFu, all);
}
__device__ __forceinline__ bool in_range(float u) { return u >= 0.f && u < 1.f; }
__device__ __forceinline__ Settings settings_of(const VerifyArgs& a, int64_t b, bool target) {
  const tim_sample_params& p = target ? a.target_set : a.draft_set;
  SampleArgs s = {};
  s.V = a.V;
  s.uniform = a.uniform_draw;
  s.temperature = p.temperature;
  s.top_k = p.top_k;
  s.top_p = p.top_p;
  s.min_p = p.min_p;
  s.row_temperature = p.row_temperature;
  s.row_top_k = p.row_top_k;
  s.row_top_p = p.row_top_p;
  s.row_min_p = p.row_min_p;
  return settings_of(s, b);
}
__device__ __forceinline__ Settings settings_of(const VerifyArgs& a, int64_t row) {
  const Where w = where(a, row);
  return settings_of(a, w.b, w.target);
}
__device__ __forceinline__ void write_bad(const VerifyArgs& a, int64_t row, int code) {
  set_status(a.status, code);
  VerifyRow r = {};
  r.bad = code;
  a.rows[row] = r;
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
  a.rows[row] = r;
}

// ---- the second launch

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kParts = kCluster * kWarps;  // of a row, one a warp
constexpr int kAhead = 2;                  // vectors of a lane and matrix in flight

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

struct FinishShared {
  Tables fine;
  uint32_t table[2][256];
  u64 part[kParts];
  int n, refused, bad, found;
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
  // of a logit far from 0
  __device__ __forceinline__ u64 far(float z) const {
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
  __device__ __forceinline__ int draw(FinishShared& sh, float u) const {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = (groups() + kParts * 32 - 1) / (kParts * 32) * 32;
    const int mine = static_cast<int>(cluster_rank()) * kWarps + warp;
    const int j0 = min(groups(), mine * part), j1 = min(groups(), j0 + part);
    const raw* const other = x < 0 ? q.p : p.p;
    u64 sum = 0;
    for (int j = j0 + lane; j < j1; j += kAhead * 32) {
      Loaded lp[kAhead], lq[kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n)
        if (j + n * 32 < j1) {
          lp[n] = load(p.p, j + n * 32);
          lq[n] = load(other, j + n * 32);
        }
#pragma unroll
      for (int n = 0; n < kAhead; ++n)
        if (j + n * 32 < j1) each(lp[n], lq[n], j + n * 32, [&](int, u64 r) { sum += r; });
    }
    sum = warp_sum(sum);
    if (lane < kCluster) cluster_store(cluster_addr(&sh.part[mine], lane), sum);
    if (tid == 0) sh.found = -1;
    cluster_arrive();
    cluster_wait();
    u64 before = 0, total = 0;
#pragma unroll
    for (int i = lane; i < kParts; i += 32) {
      total += sh.part[i];
      before += i < mine ? sh.part[i] : 0;
    }
    total = warp_sum(total);
    before = warp_sum(before);
    if (total < 1ull << 32) return -2;
    const u64 target = draw_target(total, u);
    if (before <= target && target < before + sum) {  // this warp's part: once more, a step at a time
      for (int i = j0; i < j1; i += 32) {
        const int j = i + lane;
        u64 here = 0;
        Loaded lp, lq;
        if (j < j1) {
          lp = load(p.p, j);
          lq = load(other, j);
          each(lp, lq, j, [&](int, u64 r) { here += r; });
        }
        const u64 to = warp_scan(here), all = __shfl_sync(0xFFFFFFFFu, to, 31);
        if (target < before + all) {
          u64 at = before + to - here;
          if (at <= target && target < at + here)  // one lane
            each(lp, lq, j, [&](int id, u64 r) {
              if (at <= target && target < at + r) sh.found = id;
              at += r;
            });
          break;
        }
        before += all;
      }
    }
    __syncthreads();
    return sh.found;
  }
};

// The drafts of a sequence, by one warp: a lane a position.  Writes what is accepted; sh.n of them, the
// token that is refused there or -1, and the code of a position that cannot be decided.
template <int kDtype>
__device__ __forceinline__ void decide_drafts(const VerifyArgs& a, int64_t b, const VerifyRow* ps,
                                              const VerifyRow* qs,
                                              const typename Elem<kDtype>::raw* target,
                                              const typename Elem<kDtype>::raw* draft, float tau,
                                              float draft_tau, bool writes, FinishShared& sh) {
  using E = Elem<kDtype>;
  const int lane = threadIdx.x & 31;
  const int32_t* const ids = a.ids + b * a.N;
  int n = 0;
  for (int j0 = 0; j0 <= a.N; j0 += 32) {
    const int j = j0 + lane;
    const int id = j < a.N ? __ldg(ids + j) : -1;
    // a row is there for every position up to the end of the drafts
    const unsigned ends = __ballot_sync(0xFFFFFFFFu, id < 0);
    const bool reached = j <= a.N && (ends & ((1u << lane) - 1u)) == 0;
    int code = 0;
    bool stop = true;
    float lp = 0.f;
    if (reached) {
      const VerifyRow p = ps[j];
      code = id < -1 || id >= a.V ? TIM_ERR_TOKEN_RANGE : p.bad;
      if (id >= 0 && code == 0) {
        const float u = __ldg(a.uniform + b * a.N + j);
        const float z = E::widen(target[static_cast<int64_t>(j) * a.target.ld_pos + id]);
        const Df ln_p = log_prob(p, z, tau);
        Df ln_q = df(0.f);
        bool certain = u == 0.f;  // whatever q is
        if (!in_range(u)) code = TIM_ERR_INVALID_ARG;
        if (draft_given(a)) {
          const VerifyRow q = qs[j];
          const float zq = E::widen(draft[static_cast<int64_t>(j) * a.draft.ld_pos + id]);
          if (q.bad != 0) code = q.bad;
          certain = certain || !keeps(q, zq, id);
          ln_q = log_prob(q, zq, draft_tau);
        }
        // in logarithms: p and q may both lie below the range of a float
        stop = !(keeps(p, z, id) && (certain || (log_uniform(u) + ln_q - ln_p).h < 0.f));
        lp = ln_p.h;
      }
    }
    const unsigned stops = __ballot_sync(0xFFFFFFFFu, stop || code != 0);
    const int k = stops != 0 ? __ffs(stops) - 1 : 32;  // accepted of these
    if (writes && lane < k) {
      a.out_ids[b * (a.N + 1) + j] = id;
      a.out_logprob[b * (a.N + 1) + j] = lp;
    }
    n += k;
    if (stops != 0) {
      if (lane == k) {
        sh.n = n;
        sh.refused = id;
        sh.bad = code;
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
  const int64_t b = blockIdx.x / kCluster, out = b * (a.N + 1);
  const bool writes = cluster_rank() == 0;
  const VerifyRow* const ps = a.rows + b * (a.N + 1);
  const VerifyRow* const qs = a.rows + a.B * (a.N + 1) + b * a.N;
  const raw* const target = static_cast<const raw*>(a.target.logits) + b * a.target.ld_seq;
  const raw* const draft = static_cast<const raw*>(a.draft.logits) + b * a.draft.ld_seq;
  const float tau = settings_of(a, b, true).tau, draft_tau = settings_of(a, b, false).tau;
  cluster_arrive();
  if (tid < 32) decide_drafts<kDtype>(a, b, ps, qs, target, draft, tau, draft_tau, writes, sh);
  load_tables(sh.fine, tid, kThreads);
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
      id = Residual<kDtype, true>{P, Q, a.V, static_cast<int>((at & 15u) / sizeof(raw)), x}.draw(sh, u);
    else
      id = Residual<kDtype, false>{P, Q, a.V, 0, x}.draw(sh, u);
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
  // threads a row as in sample.cu
  if (rows <= num_sms)
    sample_list_kernel<kDtype, 1024, VerifyArgs><<<g, 1024, 0, stream>>>(a);
  else if (rows <= 2 * num_sms)
    sample_list_kernel<kDtype, 512, VerifyArgs><<<g, 512, 0, stream>>>(a);
  else if (rows <= 4 * num_sms)
    sample_list_kernel<kDtype, 256, VerifyArgs><<<g, 256, 0, stream>>>(a);
  else
    sample_list_kernel<kDtype, 128, VerifyArgs><<<g, 128, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_clusters(verify_finish_kernel<kDtype>, a.B, kCluster, kThreads, 0, stream, a);
}

}  // namespace

size_t verify_bytes(int64_t B, int32_t N) {
  return align_up(1024 + static_cast<size_t>(B) * (2 * static_cast<size_t>(N) + 1) * sizeof(VerifyRow),
                  1024);
}

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
  a.rows = reinterpret_cast<VerifyRow*>(static_cast<uint8_t*>(ws) + 1024);
  a.out_ids = out_ids;
  a.out_logprob = out_logprob;
  a.out_accepted = out_accepted;
  a.status = static_cast<int*>(ws);
  return dtype == TIM_F32    ? launch_type<TIM_F32>(a, stream, num_sms)
         : dtype == TIM_BF16 ? launch_type<TIM_BF16>(a, stream, num_sms)
                             : launch_type<TIM_F16>(a, stream, num_sms);
}

}  // namespace tim
