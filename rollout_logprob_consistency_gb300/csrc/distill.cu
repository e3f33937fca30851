// Distillation from a teacher's top logits: per-row loss over a [T, V] logits matrix, and
// its gradient with respect to the logits.
//
// With s = z / tau, p = softmax(s), the teacher's head H (the entries of the row with an
// id and a finite logprob ln q_k), Q = sum q_k, P = sum_{H} p_k, and the tokens outside H
// as one more bucket with p_r = 1 - P and q_r = 1 - Q (the tail, where asked for):
//   forward KL  L = sum_H q_k (ln q_k - ln p_k) + q_r (ln q_r - ln p_r)
//     dL/ds_v = p_v (Q + q_r) - q_v          for v in H
//             = p_v (Q - q_r P / p_r)        outside
//   reverse KL  L = sum_H p_k (ln p_k - ln q_k) + p_r (ln p_r - ln q_r)
//     with a = ln p - ln q and B = sum_H (a_k + 1) p_k + (a_r + 1) p_r:
//     dL/ds_v = p_v (a_v + 1 - B)            for v in H
//             = p_v (a_r + 1 - B)            outside (without the tail: -p_v B)
// so outside the head every gradient is one row constant times p_v.
//
// p_r is the sum over the tokens outside H, not 1 - P: a teacher's head usually holds
// nearly all the mass and the difference would keep few digits.  The streaming pass
// therefore leaves the head's tokens out (a bitmap in shared memory marks them) and the
// head's exponentials are taken on their own, to 2^-33, and every sum over the head is held in
// pairs of floats: the loss is a difference of near numbers.
#include <cmath>

#include "logits_row.cuh"

namespace tim {

namespace {

constexpr int kBackThreads = 256;
constexpr int kMaxWarps = 16;
constexpr int kMaxCluster = 8;
constexpr float kTailFloor = 0x1p-20f;  // a teacher's tail up to this is rounding
constexpr float kTailLeast = 0x1p-100f;  // below this share of the mass the student has no tail

struct DistillArgs {
  const void* logits;
  int64_t ld;
  int V;
  int K;
  const int32_t* ids;
  const float* lp;
  float kh, kl;      // log2(e) / temperature as a pair
  float inv_h, inv_l;  // 1 / temperature as a pair
  int kind;
  int tail;
  int cluster;
  float* loss;
  float* lse;    // forward only
  float* saved;  // forward only: [T][TIM_DISTILL_SAVED]
  const float* grad;
  void* dlogits;
  int64_t ldd;
  int* status;
};

// What the backward needs of a row, as saved by the forward.
enum Saved { kMax = 0, kInvSum, kLogSum, kRest, kHead, kLive };

__device__ __forceinline__ bool in_head(int id, float lp) { return id >= 0 && lp != -INFINITY; }

// Vector j of the row, to the same elements of `out`; one store where the two addresses agree
// modulo 16 bytes and the vector is whole.
template <int kDtype>
__device__ __forceinline__ void store_vector(typename Elem<kDtype>::raw* out, const Row<kDtype>& r,
                                             int j, bool same,
                                             const float (&v)[Elem<kDtype>::kVec]) {
  using E = Elem<kDtype>;
  if (same && r.whole(j)) {
    *reinterpret_cast<uint4*>(out - r.shift + static_cast<int64_t>(j) * E::kVec) = E::pack(v);
    return;
  }
#pragma unroll
  for (int i = 0; i < E::kVec; ++i) {
    const int e = j * E::kVec + i - r.shift;
    if (e >= 0 && e < r.V) out[e] = E::narrow(v[i]);
  }
}

struct HeadSums {
  Df e, q, qx, ex;  // sums of e_k, q_k, q_k (ln q_k - x_k), e_k (x_k - ln q_k)
};

__device__ __forceinline__ Df scaled(float z, float c, const DistillArgs& a) {  // (z - c) / tau
  return (df(z) - df(c)) * Df{a.inv_h, a.inv_l};
}

// The gradient of a vector's tokens as if all were outside the head.
template <int kVec>
__device__ __forceinline__ void gradient_vector(float (&v)[kVec], F2 ref, F2 k, F2 c) {
#pragma unroll
  for (int i = 0; i < kVec; i += 2) {
    const float2 t = unpack2(mul2(c, ex2x2(mul2(add2(f2(v[i], v[i + 1]), ref), k))));
    v[i] = t.x;
    v[i + 1] = t.y;
  }
}

// One entry's gradient with respect to s, M the row's maximum.
__device__ __forceinline__ float head_gradient(const DistillArgs& a, float z, float lq, float M,
                                               float logS, float inv, float c_head) {
  const float p = pow2_df(z, Pow2Row{a.kh, a.kl, M, true}).h * inv;
  if (a.kind == TIM_DISTILL_FORWARD_KL) return fmaf(p, c_head, -exp_df(lq).h);
  return p == 0.f ? 0.f : p * (scaled(z, M, a) - df(lq) + df(c_head - logS)).h;
}

__device__ __forceinline__ Df bcast(Df v, int lane = 0) {
  return {__shfl_sync(0xFFFFFFFFu, v.h, lane), __shfl_sync(0xFFFFFFFFu, v.l, lane)};
}

// The row's constants in fp32, from which its gradients follow (good to about 2^-22), from the
// sum `rest` of the weights outside the head relative to M and the head's sums relative to hmax.
struct RowConstants {
  float inv, logS;  // of the sum relative to M: reciprocal and logarithm
  float c_rest, c_head;
};
__device__ __forceinline__ RowConstants row_constants(const DistillArgs& a, float M, float hmax,
                                                      float rest, const HeadSums& h) {
  const bool near = hmax == M || hmax == -INFINITY;
  const float x = near ? 0.f : (hmax - M) * a.kh, shift = x * kLn2Hi;
  const float f = ex2_approx(x);
  const float P0 = h.e.h * f, S = rest + P0, Q = h.q.h;
  RowConstants t;
  t.inv = 1.f / S;
  t.logS = logf(S);
  const float P = P0 * t.inv, pr = rest * t.inv;
  const float qr = (df(1.f) - h.q).h;
  const bool tail = a.tail != 0 && qr > kTailFloor && pr > kTailLeast;
  if (a.kind == TIM_DISTILL_FORWARD_KL) {
    t.c_rest = tail ? Q - qr * (P0 / rest) : Q;
    t.c_head = tail ? Q + qr : Q;
  } else {
    float B = (P0 != 0.f ? h.ex.h * f * t.inv - P * (t.logS - shift) : P0) + P;
    t.c_rest = 0.f;
    if (tail) {
      t.c_rest = logf(pr / qr) + 1.f;
      B += pr * t.c_rest;
    }
    t.c_rest -= B;
    t.c_head = 1.f - B;
  }
  return t;
}

// The row's loss and lse, from the same sums, in pairs of floats.  Called by a whole warp with the
// same arguments: its lanes take the logarithms and reciprocals of different numbers at once, and
// every lane returns the result.
struct RowLoss {
  float loss, lse;
};
__device__ __forceinline__ RowLoss row_loss(const DistillArgs& a, float M, float hmax, float rest,
                                            const HeadSums& h) {
  const int lane = threadIdx.x & 31;
  const bool none = hmax == -INFINITY;  // no token of the head has any mass: all its terms are 0
  const Df shift = none ? df(0.f) : scaled(hmax, M, a);  // <= 0
  const Df f = none || hmax == M ? df(1.f) : pow2_df(hmax, Pow2Row{a.kh, a.kl, M, true});
  const Df P0 = h.e * f, Q = h.q, S = df(rest) + P0;
  const Df qr = df(1.f) - Q;
  // lane 0: S, lane 1: rest, lane 2: q_r
  const Df x = lane == 0 ? S : lane == 1 ? df(rest) : qr;
  const bool fine = x.h >= 0x1p-126f && x.h < INFINITY;
  const Df log_x = fine ? log_df(x) : df(__int_as_float(0x7FC00000));
  const Df logS = bcast(log_x), inv = reciprocal(S);
  const Df pr = df(rest) * inv;
  const Df up = logS - shift;                                 // ln p_k = x_k - up
  const Df ar = bcast(log_x, 1) - logS - bcast(log_x, 2);     // ln p_r - ln q_r
  Df L;
  if (a.kind == TIM_DISTILL_FORWARD_KL)
    L = h.qx + Q * up;
  else
    L = P0.h != 0.f ? ((h.ex * f) - P0 * up) * inv : P0;
  if (a.tail != 0 && qr.h > kTailFloor && pr.h > kTailLeast)
    L = a.kind == TIM_DISTILL_FORWARD_KL ? L - qr * ar : L + pr * ar;
  return {L.h, (df(M) * Df{a.inv_h, a.inv_l} + logS).h};
}

__device__ __forceinline__ Df shfl_xor(Df v, int o) {
  return {__shfl_xor_sync(0xFFFFFFFFu, v.h, o), __shfl_xor_sync(0xFFFFFFFFu, v.l, o)};
}
__device__ __forceinline__ HeadSums warp_sum(HeadSums h, int from) {
  for (int o = from; o > 0; o >>= 1) {
    h.e = h.e + shfl_xor(h.e, o);
    h.q = h.q + shfl_xor(h.q, o);
    h.qx = h.qx + shfl_xor(h.qx, o);
    h.ex = h.ex + shfl_xor(h.ex, o);
  }
  return h;
}

// (max, sum) of two parts.
__device__ __forceinline__ void merge(float& m, float& sum, float m2, float s2, float k2) {
  const float mm = fmaxf(m, m2), base = mm == -INFINITY ? 0.f : mm;
  sum = sum * ex2_approx((m - base) * k2) + s2 * ex2_approx((m2 - base) * k2);
  m = mm;
}

// Loss of a row by a cluster of CTAs, and with kGrad its gradient for a known grad[row].
//
// Each CTA holds its slice of the row in shared memory, so the gradient costs one write and no
// second read.  While the slice is on its way every CTA does the head's terms (the same in all
// of them: no second exchange is needed), then sums its slice's other tokens relative to the
// head's maximum, sends the sum to the others and all combine them in rank order.  Nothing
// else has to be known before the sum: a weight relative to the head's maximum only overflows
// if a token lies 2^127 above the whole head, and then that slice is summed again with a running
// maximum.
// 256 threads a CTA: five CTAs an SM, as many as 40 KB slices fit.
template <int kDtype, bool kGrad, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 5 : 2) distill_kernel(const DistillArgs a) {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  extern __shared__ uint4 slice_mem[];
  __shared__ HeadSums red[kMaxWarps];
  __shared__ float redm[kMaxWarps], reds[kMaxWarps];
  __shared__ float s_hmax[kMaxWarps];
  __shared__ uint64_t part[kMaxCluster][2];  // (reference, sum) and the error code of every CTA
  __shared__ uint64_t head_part[kMaxCluster][4];
  __shared__ RowConstants s_terms;
  __shared__ float s_M;
  __shared__ int s_bad;
  __shared__ uint64_t bar;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int warps = kThreads / 32;
  const int64_t row = blockIdx.x / a.cluster;
  const int rank = static_cast<int>(cluster_rank());
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  const Slice s = slice_of(r.nvec(), rank, a.cluster);
  uint8_t* marks = reinterpret_cast<uint8_t*>(slice_mem + s.n);  // a byte a vector: ids met
  const int32_t* ids = a.ids + row * a.K;
  const float* lp = a.lp + row * a.K;
  raw* out = nullptr;
  if constexpr (kGrad) out = static_cast<raw*>(a.dlogits) + row * a.ldd;

  cluster_arrive();  // this CTA runs: the others may write to its memory after their wait
  if (tid == 0) {
    s_bad = 0;
    mbar_init(&bar, 1);
    fence_mbarrier_init();
  }
  for (int i = tid; i < (s.n + 3) / 4; i += kThreads)
    reinterpret_cast<uint32_t*>(marks)[i] = 0u;
  // Calls f(id, ln q, z) for this thread's entries that are in the head; the first one's values
  // are loaded once.
  const int id0 = tid < a.K ? __ldg(ids + tid) : -1;
  const float lq0 = tid < a.K ? __ldg(lp + tid) : 0.f;
  auto usable = [&](int id, float lq) { return in_head(id, lq) && id < a.V && lq <= 1.f; };
  const float z0 = usable(id0, lq0) ? r.at(id0) : 0.f;
  auto for_head = [&](auto&& f) {
    if (usable(id0, lq0)) f(id0, lq0, z0);
    for (int k = tid + kThreads; k < a.K; k += kThreads) {
      const int id = __ldg(ids + k);
      const float lq = __ldg(lp + k);
      if (usable(id, lq)) f(id, lq, r.at(id));
    }
  };
  int bad = 0, any = 0;
  for (int k = tid; k < a.K; k += kThreads) {
    const int id = k == tid ? id0 : __ldg(ids + k);
    const float lq = k == tid ? lq0 : __ldg(lp + k);
    if (id < -1 || id >= a.V)
      bad = TIM_ERR_TOKEN_RANGE;
    else if (id >= 0 && !(lq <= 1.f) && bad == 0)  // not the logarithm of a probability, or NaN
      bad = TIM_ERR_INVALID_ARG;
    else if (in_head(id, lq))
      any = 1;
  }
  if (!__syncthreads_or(any | bad)) {  // the same in every CTA of the row: no entries
    if (rank == 0 && tid == 0) {
      a.loss[row] = 0.f;
      if constexpr (!kGrad) {
        a.lse[row] = 0.f;
        float* saved = a.saved + row * TIM_DISTILL_SAVED;
        for (int i = 0; i < TIM_DISTILL_SAVED; ++i) saved[i] = 0.f;
      }
    }
    if constexpr (kGrad) {
      const Row<kDtype> o(out, 0, 0, a.V);  // the output's own vectors
      const Slice so = slice_of(o.nvec(), rank, a.cluster);
      const float zeros[E::kVec] = {};
      for (int j = so.j0 + tid; j < so.j0 + so.n; j += kThreads)
        store_vector<kDtype>(out, o, j, true, zeros);
    }
    cluster_wait();
    return;
  }
  if (tid == 0) load_slice(r, s, slice_mem, &bar);
  load_slice_edges(r, s, slice_mem);

  // ---- the head, while the slice is on its way
  float hmax = -INFINITY;
  for_head([&](int id, float, float z) {
    hmax = fmaxf(hmax, z);
    const int slot = id + r.shift - s.j0 * E::kVec;
    if (slot >= 0 && slot < s.n * E::kVec) {
      uint32_t* w = reinterpret_cast<uint32_t*>(marks) + slot / E::kVec / 4;
      const uint32_t bit = 1u << (slot / E::kVec % 4 * 8 + slot % E::kVec);
      if ((atomicOr(w, bit) & bit) && bad == 0) bad = TIM_ERR_INVALID_ARG;  // an id twice
    }
  });
  if (bad != 0) atomicMax(&s_bad, bad);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) hmax = fmaxf(hmax, __shfl_xor_sync(0xFFFFFFFFu, hmax, o));
  if (lane == 0) s_hmax[warp] = hmax;
  __syncthreads();
  for (int i = 0; i < min(warps, (a.K + 31) / 32); ++i) hmax = fmaxf(hmax, s_hmax[i]);
  const float href = hmax == -INFINITY ? 0.f : hmax;
  // entry rank + cluster i is thread i's
  const int head_n = (a.K - rank + a.cluster - 1) / a.cluster, head_warps = (head_n + 31) / 32;
  if (tid < head_warps * 32) {
    HeadSums h = {};
    const int k = rank + a.cluster * tid;
    if (k < a.K) {
      const int id = __ldg(ids + k);
      const float lq = __ldg(lp + k);
      if (usable(id, lq)) {
        const float z = r.at(id);
        const Df t = df(lq) - scaled(z, href, a);
        h.e = pow2_df(z, Pow2Row{a.kh, a.kl, href, true});
        h.q = exp_df(lq);
        if (h.q.h != 0.f) h.qx = h.q * t;
        if (h.e.h != 0.f) h.ex = -(h.e * t);
      }
    }
    h = warp_sum(h, 16);
    if (lane == 0) red[warp] = h;
  }

  // ---- the slice: sum of 2^((z - reference) log2e / tau) outside the head
  const float k2 = a.kh;
  const int never = 0;
  if (!mbar_wait(&bar, 0, &never)) set_status(a.status, TIM_ERR_TIMEOUT);
  // the head's tokens leave the slice: 2^-inf = 0 in the sum, and their gradients come later
  for_head([&](int id, float, float) {
    const int slot = id + r.shift - s.j0 * E::kVec;
    if (slot >= 0 && slot < s.n * E::kVec)
      reinterpret_cast<raw*>(slice_mem)[slot] = E::narrow(-INFINITY);
  });
  __syncthreads();
  float m = href, sum;
  {
    const F2 ref = f2(-href, -href), kk = f2(k2, k2);
    F2 acc = f2(0.f, 0.f), acc2 = acc;
    const uint4* end = slice_mem + s.n;
#pragma unroll 4
    for (const uint4* p = slice_mem + tid; p < end; p += kThreads) {
      float v[E::kVec];
      E::unpack(*p, v);
#pragma unroll
      for (int i = 0; i < E::kVec; i += 4) {
        acc = add2(acc, ex2x2(mul2(add2(f2(v[i], v[i + 1]), ref), kk)));
        acc2 = add2(acc2, ex2x2(mul2(add2(f2(v[i + 2], v[i + 3]), ref), kk)));
      }
    }
    const float2 t = unpack2(add2(acc, acc2));
    sum = t.x + t.y;
  }
  auto publish = [&]() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      merge(m, sum, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, sum, o), k2);
    if (lane == 0) {
      redm[warp] = m;
      reds[warp] = sum;
    }
  };
  publish();
  // an infinite sum, or a head without mass to refer to: again, with a running maximum
  if (__syncthreads_or(!(sum < INFINITY) || hmax == -INFINITY)) {
    m = -INFINITY;
    sum = 0.f;
    for (int j = tid; j < s.n; j += kThreads) {
      float v[E::kVec];
      E::unpack(slice_mem[j], v);
      float vm = m;
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) vm = fmaxf(vm, v[i]);
      if (vm > m) {
        sum *= ex2_approx((m - vm) * k2);
        m = vm;
      }
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) sum += ex2_approx((v[i] - base) * k2);
    }
    publish();
    __syncthreads();
  }
  cluster_wait();
  // the loss alone is rank 0's work
  const int readers = kGrad ? a.cluster : 1;
  if (warp == 0) {
    m = lane < warps ? redm[lane] : -INFINITY;
    sum = lane < warps ? reds[lane] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
      merge(m, sum, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, sum, o), k2);
    if (lane < readers) {
      cluster_store(cluster_addr(&part[rank][0], lane),
                    (static_cast<uint64_t>(__float_as_uint(sum)) << 32) | __float_as_uint(m));
      cluster_store(cluster_addr(&part[rank][1], lane), static_cast<uint64_t>(s_bad));
    }
  } else if (warp == 1) {
    HeadSums h = {};
    if (lane < head_warps) h = red[lane];
    if (head_warps > 1) h = warp_sum(h, 8);
    const Df out[4] = {h.e, h.q, h.qx, h.ex};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Df v = bcast(out[i]);
      if (lane < readers)
        cluster_store(cluster_addr(&head_part[rank][i], lane),
                      (static_cast<uint64_t>(__float_as_uint(v.l)) << 32) | __float_as_uint(v.h));
    }
  }
  cluster_arrive();
  if (!kGrad && rank != 0) return;  // having arrived
  cluster_wait();
  // all parts, combined in rank order by a whole warp; every lane has the result
  struct Combined {
    float M, rest;
    int code;
    HeadSums h;
  };
  auto combine = [&]() {
    const bool mine = lane < a.cluster;
    const float mi = mine ? __uint_as_float(static_cast<uint32_t>(part[lane][0])) : -INFINITY;
    float rest = mine ? __uint_as_float(static_cast<uint32_t>(part[lane][0] >> 32)) : 0.f;
    Combined t = {};
    t.code = __reduce_max_sync(0xFFFFFFFFu, mine ? static_cast<int>(part[lane][1]) : 0);
    HeadSums h = {};
    if (mine) {
      Df* d[4] = {&h.e, &h.q, &h.qx, &h.ex};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t u = head_part[lane][i];
        *d[i] = Df{__uint_as_float(static_cast<uint32_t>(u)),
                   __uint_as_float(static_cast<uint32_t>(u >> 32))};
      }
    }
    if (a.cluster > 1) h = warp_sum(h, 4);
    float M = fmaxf(hmax, mi);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    // a part of -inf alone has sum 0, one with a NaN has NaN
    if (mi != -INFINITY) rest *= ex2_approx((mi - M) * k2);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) rest += __shfl_xor_sync(0xFFFFFFFFu, rest, o);
    t.M = __shfl_sync(0xFFFFFFFFu, M, 0);
    t.rest = __shfl_sync(0xFFFFFFFFu, rest, 0);
    t.h = HeadSums{bcast(h.e), bcast(h.q), bcast(h.qx), bcast(h.ex)};
    return t;
  };
  const float nan = __int_as_float(0x7FC00000);
  auto write_loss = [&](const Combined& t) {
    const RowLoss v = row_loss(a, t.M, hmax, t.rest, t.h);
    if (lane == 0) {
      if (t.code != 0)
        set_status(a.status, t.code);
      else if (!(isfinite(v.lse) && isfinite(v.loss)))
        set_status(a.status, TIM_ERR_NONFINITE);
      a.loss[row] = t.code != 0 ? nan : v.loss;
      if constexpr (!kGrad) a.lse[row] = t.code != 0 ? nan : v.lse;
    }
  };
  if (warp == 0) {
    const Combined t = combine();
    if (lane == 0) {
      RowConstants c = row_constants(a, t.M, hmax, t.rest, t.h);
      if (t.code != 0) c.c_rest = c.c_head = nan;
      s_terms = c;
      s_M = t.M;
      if constexpr (!kGrad) {
        float* saved = a.saved + row * TIM_DISTILL_SAVED;
        saved[kMax] = t.M;
        saved[kInvSum] = c.inv;
        saved[kLogSum] = c.logS;
        saved[kRest] = c.c_rest;
        saved[kHead] = c.c_head;
        saved[kLive] = t.code != 0 ? nan : 1.f;
        saved[kLive + 1] = saved[kLive + 2] = 0.f;
      }
    }
    __syncwarp();
    if (!kGrad) write_loss(t);
  }
  if constexpr (!kGrad) return;

  // ---- the gradient, from the slice in shared memory
  __syncthreads();
  const float w = __ldg(a.grad + row);
  const float g = w * a.inv_h;
  const RowConstants t = s_terms;
  const float M = s_M;
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(r.p)) & 15u) == 0;
  if (w == 0.f) {
    const float zeros[E::kVec] = {};
    for (int j = tid; j < s.n; j += kThreads) store_vector<kDtype>(out, r, s.j0 + j, same, zeros);
    if (rank == 0 && warp == 0) write_loss(combine());
    return;
  }
  const float c = t.c_rest * t.inv * g;
  const F2 ref = f2(-M, -M), kk = f2(k2, k2), cc = f2(c, c);
  int j0 = 0, j1 = 0;  // the vectors that are one store each
  if (same && s.n > 0) {
    j0 = r.whole(s.j0) ? 0 : 1;
    j1 = max(j0, r.whole(s.j0 + s.n - 1) ? s.n : s.n - 1);
  }
  uint4* const to = reinterpret_cast<uint4*>(out - r.shift + static_cast<int64_t>(s.j0) * E::kVec);
#pragma unroll 4
  for (int j = j0 + tid; j < j1; j += kThreads) {
    float v[E::kVec];
    E::unpack(slice_mem[j], v);
    gradient_vector(v, ref, kk, cc);
    to[j] = E::pack(v);
  }
  // the others: the row's ends, or all where the output lies otherwise
  auto store_edge = [&](int j) {
    float v[E::kVec];
    E::unpack(slice_mem[j], v);
    gradient_vector(v, ref, kk, cc);
    store_vector<kDtype>(out, r, s.j0 + j, same, v);
  };
  if (tid < j0) store_edge(tid);
  for (int j = j1 + tid; j < s.n; j += kThreads) store_edge(j);
  if (rank == 0 && warp == warps - 1) write_loss(combine());  // nothing waits for the loss
  __syncthreads();  // the head's tokens are written again, after the whole slice
  for_head([&](int id, float lq, float z) {
    const int slot = id + r.shift - s.j0 * E::kVec;
    if (slot >= 0 && slot < s.n * E::kVec)
      out[id] = E::narrow(head_gradient(a, z, lq, M, t.logS, t.inv, t.c_head) * g);
  });
}

// The gradient alone, from what the forward saved: a CTA a slice of a row, reading and writing
// it once; the head's tokens are written again after the slice.
constexpr int kBackUnroll = 4;  // vectors of a thread in flight
template <int kDtype>
__global__ void __launch_bounds__(kBackThreads) distill_backward_kernel(const DistillArgs a) {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  const int64_t row = blockIdx.x / a.cluster;
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  const Slice s = slice_of(r.nvec(), blockIdx.x % a.cluster, a.cluster);
  raw* out = static_cast<raw*>(a.dlogits) + row * a.ldd;
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(r.p)) & 15u) == 0;
  const float* saved = a.saved + row * TIM_DISTILL_SAVED;
  const float w = __ldg(a.grad + row), live = saved[kLive], g = w * a.inv_h;
  const bool zero = live == 0.f || w == 0.f;
  const float k2 = a.kh;
  const float M = saved[kMax], inv = saved[kInvSum];
  const float c = live * saved[kRest] * inv * g;  // NaN for a row the forward refused
  for (int j0 = threadIdx.x; j0 < s.n; j0 += kBackUnroll * kBackThreads) {
    uint4 u[kBackUnroll];
#pragma unroll
    for (int n = 0; n < kBackUnroll; ++n) {
      const int j = j0 + n * kBackThreads;
      if (!zero && j < s.n) u[n] = r.load(s.j0 + j);
    }
#pragma unroll
    for (int n = 0; n < kBackUnroll; ++n) {
      const int j = j0 + n * kBackThreads;
      if (j >= s.n) break;
      float v[E::kVec];
      if (zero) {
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) v[i] = 0.f;
      } else {
        E::unpack(u[n], v);
        gradient_vector(v, f2(-M, -M), f2(k2, k2), f2(c, c));
      }
      store_vector<kDtype>(out, r, s.j0 + j, same, v);
    }
  }
  if (zero || live != live) return;
  __syncthreads();
  const float logS = saved[kLogSum];
  for (int k = threadIdx.x; k < a.K; k += kBackThreads) {
    const int id = __ldg(a.ids + row * a.K + k);
    const float lq = __ldg(a.lp + row * a.K + k);
    const int slot = id + r.shift - s.j0 * E::kVec;
    if (!in_head(id, lq) || id >= a.V || slot < 0 || slot >= s.n * E::kVec) continue;
    out[id] = E::narrow(head_gradient(a, r.at(id), lq, M, logS, inv, saved[kHead]) * g);
  }
}

// The temperature's pairs.
void set_temperature(DistillArgs& a, float temperature) {
  const double k = 1.4426950408889634 / static_cast<double>(temperature);
  const double inv = 1.0 / static_cast<double>(temperature);
  a.kh = static_cast<float>(k);
  a.kl = static_cast<float>(k - static_cast<double>(a.kh));
  a.inv_h = static_cast<float>(inv);
  a.inv_l = static_cast<float>(inv - static_cast<double>(a.inv_h));
}

template <int kDtype, bool kGrad, int kThreads>
cudaError_t launch_rows(const DistillArgs& a, int64_t T, const RowPlan& p, cudaStream_t stream) {
  const size_t smem = p.slice_bytes + p.slice_bytes / 16 + 16;  // the slice and its marks
  auto* kernel = distill_kernel<kDtype, kGrad, kThreads>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_clusters(kernel, T, p.cluster, kThreads, smem, stream, a);
}
template <int kDtype, bool kGrad>
cudaError_t launch_rows(DistillArgs a, int64_t T, cudaStream_t stream) {
  const RowPlan p = plan_row(a.V, sizeof(typename Elem<kDtype>::raw));
  a.cluster = p.cluster;
  return p.threads == 256 ? launch_rows<kDtype, kGrad, 256>(a, T, p, stream)
                          : launch_rows<kDtype, kGrad, 512>(a, T, p, stream);
}

template <int kDtype>
cudaError_t launch_back(DistillArgs a, int64_t T, cudaStream_t stream) {
  a.cluster = plan_row(a.V, sizeof(typename Elem<kDtype>::raw)).cluster;
  if (T * a.cluster > INT32_MAX) return cudaErrorInvalidValue;
  distill_backward_kernel<kDtype>
      <<<static_cast<unsigned>(T * a.cluster), kBackThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_distill(const void* logits, int dtype, int64_t ld, int64_t T, int V,
                           const int32_t* ids, const float* lp, int K, float temperature, int kind,
                           int tail, float* loss, float* lse, float* saved, int* status,
                           cudaStream_t stream) {
  DistillArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.V = V;
  a.K = K;
  a.ids = ids;
  a.lp = lp;
  set_temperature(a, temperature);
  a.kind = kind;
  a.tail = tail;
  a.loss = loss;
  a.lse = lse;
  a.saved = saved;
  a.status = status;
  return dtype == TIM_F32    ? launch_rows<TIM_F32, false>(a, T, stream)
         : dtype == TIM_BF16 ? launch_rows<TIM_BF16, false>(a, T, stream)
                             : launch_rows<TIM_F16, false>(a, T, stream);
}

cudaError_t launch_distill_grad(const void* logits, int dtype, int64_t ld, int64_t T, int V,
                                const int32_t* ids, const float* lp, int K, float temperature,
                                int kind, int tail, const float* grad, float* loss, void* dlogits,
                                int64_t ldd, int* status, cudaStream_t stream) {
  DistillArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.V = V;
  a.K = K;
  a.ids = ids;
  a.lp = lp;
  set_temperature(a, temperature);
  a.kind = kind;
  a.tail = tail;
  a.loss = loss;
  a.grad = grad;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.status = status;
  return dtype == TIM_F32    ? launch_rows<TIM_F32, true>(a, T, stream)
         : dtype == TIM_BF16 ? launch_rows<TIM_BF16, true>(a, T, stream)
                             : launch_rows<TIM_F16, true>(a, T, stream);
}

cudaError_t launch_distill_backward(const void* logits, int dtype, int64_t ld, int64_t T, int V,
                                    const int32_t* ids, const float* lp, int K, float temperature,
                                    int kind, const float* saved, const float* grad, void* dlogits,
                                    int64_t ldd, cudaStream_t stream) {
  DistillArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.V = V;
  a.K = K;
  a.ids = ids;
  a.lp = lp;
  set_temperature(a, temperature);
  a.kind = kind;
  a.saved = const_cast<float*>(saved);
  a.grad = grad;
  a.dlogits = dlogits;
  a.ldd = ldd;
  return dtype == TIM_F32    ? launch_back<TIM_F32>(a, T, stream)
         : dtype == TIM_BF16 ? launch_back<TIM_BF16>(a, T, stream)
                             : launch_back<TIM_F16>(a, T, stream);
}

}  // namespace tim
