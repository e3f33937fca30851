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
constexpr float kTailFloor = 0x1p-20f;  // a teacher's tail up to this is rounding
// A warp's sum outside the head, relative to the head's largest, is taken again from here on: relative to
// its own largest, so that a row's sum, its reciprocal and their products stay far from fp32's ends, and
// arguments of 2^x where they are precise.
constexpr float kRestFar = 0x1p40f;
// The same where the tail counts and no warp's sum reaches this: p_r may be anything down to
// kTailOctaves below the row's largest weight, the least that 64 bits hold.
constexpr float kRestNear = 0x1p-40f;
constexpr float kTailOctaves = 1074.f;

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
  int parts;  // backward: CTAs a row
  float* loss;
  float* lse;    // forward only
  float* saved;  // forward only: [T][TIM_DISTILL_SAVED]
  const float* grad;
  void* dlogits;
  int64_t ldd;
  int* status;
};

// What the backward needs of a row, as saved by the forward.
enum Saved { kMax = 0, kInvSum, kLogSum, kRest, kHead, kLive, kRef };

__device__ __forceinline__ bool in_head(int id, float lp) { return id >= 0 && lp != -INFINITY; }

// The 16 bytes from byte `at` (below 16) on of the 32 in lo, hi.
__device__ __forceinline__ uint4 bytes_from(const uint4& lo, const uint4& hi, int at) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = (at & 8) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = (at & 4) ? w[i + 1] : w[i];
  const int bits = (at & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
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

// The gradient of a slice's tokens, c 2^((z - zref) log2e / tau), or zeros without a read.  The slice is of
// the output's vectors, o; where the input's lie at other addresses modulo 16 bytes, one is put together
// from two (1122 fp16 rows of 151936 at a stride of 43 more: 458 us with a store an element,
// 199 so).
constexpr int kGradUnroll = 4;  // vectors of a thread in flight
template <int kDtype, int kThreads>
__device__ __forceinline__ void gradient_slice(const DistillArgs& a, const Row<kDtype>& r,
                                               const Row<kDtype>& o, const Slice& s,
                                               typename Elem<kDtype>::raw* out, float zref,
                                               float c, bool zero) {
  using E = Elem<kDtype>;
  if (s.n <= 0) return;
  // the vectors that are one store each
  const int j0 = s.j0 + (o.whole(s.j0) ? 0 : 1);
  const int j1 = max(j0, s.j0 + s.n - (o.whole(s.j0 + s.n - 1) ? 0 : 1));
  const F2 ref = f2(-zref, -zref), kk = f2(a.kh, a.kh), cc = f2(c, c);
  const int delta = r.shift - o.shift;  // an element's slot in the input less that in the output
  const uint4* const from = r.vec();
  uint4* const to = reinterpret_cast<uint4*>(out - o.shift);
  auto put = [&](int j, const uint4& u) {
    float v[E::kVec];
    E::unpack(u, v);
    gradient_vector(v, ref, kk, cc);
    __stcs(to + j, E::pack(v));
  };
  if (zero) {
    for (int j = j0 + threadIdx.x; j < j1; j += kThreads) to[j] = make_uint4(0, 0, 0, 0);
  } else if (delta == 0) {
    for (int j = j0 + threadIdx.x; j < j1; j += kGradUnroll * kThreads) {
      uint4 u[kGradUnroll];
#pragma unroll
      for (int n = 0; n < kGradUnroll; ++n)
        if (j + n * kThreads < j1) u[n] = __ldcs(from + j + n * kThreads);
#pragma unroll
      for (int n = 0; n < kGradUnroll; ++n)
        if (j + n * kThreads < j1) put(j + n * kThreads, u[n]);
    }
  } else {
    const int back = delta < 0 ? 1 : 0;
    const int at = (delta + back * E::kVec) * static_cast<int>(sizeof(typename E::raw));
    const int w0 = r.w0(), w1 = r.w1();
    constexpr int kPairs = kGradUnroll / 2;
    for (int j = j0 + threadIdx.x; j < j1; j += kPairs * kThreads) {
      uint4 u[kPairs][2];
#pragma unroll
      for (int n = 0; n < kPairs; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = j + n * kThreads - back + h;
          if (j + n * kThreads < j1) u[n][h] = i >= w0 && i < w1 ? __ldg(from + i) : r.load_edge(i);
        }
      }
#pragma unroll
      for (int n = 0; n < kPairs; ++n)
        if (j + n * kThreads < j1) put(j + n * kThreads, bytes_from(u[n][0], u[n][1], at));
    }
  }
  // the row's ends, which may be partly others': a thread an element
  if (static_cast<int>(threadIdx.x) < 2 * E::kVec) {
    const bool first = static_cast<int>(threadIdx.x) < E::kVec;
    if (first ? j0 > s.j0 : j1 < s.j0 + s.n) {
      const int j = first ? s.j0 : s.j0 + s.n - 1;
      const int e = j * E::kVec + static_cast<int>(threadIdx.x) % E::kVec - o.shift;
      if (e >= 0 && e < a.V) {
        float v[2] = {zero ? 0.f : r.at(e), 0.f};
        if (!zero) gradient_vector(v, ref, kk, cc);
        out[e] = E::narrow(v[0]);
      }
    }
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
// sum `rest` of the weights outside the head relative to ref, the head's sums relative to hmax, and the
// row's largest M.  Outside the head the gradient is c_rest inv 2^((z - ref) log2e / tau): where the
// rest is far below, its tokens' shares of it, which carry q_r, need no number as small as p_r.
struct RowConstants {
  float inv, logS;  // of the sum relative to M: reciprocal and logarithm
  float c_rest, c_head;
  bool tail;
};
__device__ __forceinline__ RowConstants row_constants(const DistillArgs& a, float M, float hmax,
                                                      float ref, float rest, const HeadSums& h) {
  const bool near = hmax == M || hmax == -INFINITY;
  const float x = near ? 0.f : (hmax - M) * a.kh, shift = x * kLn2Hi;
  const float f = ex2_approx(x);
  const float down = ref == M ? 0.f : (ref - M) * a.kh;  // octaves, <= 0
  const float r = ex2_approx(down), rest_M = rest * r;
  const float P0 = h.e.h * f, S = rest_M + P0, Q = h.q.h;
  RowConstants t;
  t.inv = 1.f / S;
  t.logS = logf(S);
  const float P = P0 * t.inv, pr = rest * t.inv;  // p_r is pr r
  const float qr = (df(1.f) - h.q).h;
  t.tail = a.tail != 0 && qr > kTailFloor && rest > 0.f && down > -kTailOctaves;
  if (a.kind == TIM_DISTILL_FORWARD_KL) {
    t.c_rest = t.tail ? Q * r - qr * (P0 / rest) : Q * r;
    t.c_head = t.tail ? Q + qr : Q;
  } else {
    float B = (P0 != 0.f ? h.ex.h * f * t.inv - P * (t.logS - shift) : P0) + P;
    t.c_rest = 0.f;
    if (t.tail) {
      t.c_rest = logf(pr / qr) + down * kLn2Hi + 1.f;
      B += pr * r * t.c_rest;
    }
    t.c_rest = (t.c_rest - B) * r;
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
__device__ __forceinline__ RowLoss row_loss(const DistillArgs& a, float M, float hmax, float ref,
                                            float rest, const HeadSums& h, bool tail) {
  const int lane = threadIdx.x & 31;
  const bool none = hmax == -INFINITY;  // no token of the head has any mass: all its terms are 0
  const Df shift = none ? df(0.f) : scaled(hmax, M, a);  // <= 0
  const Df f = none || hmax == M ? df(1.f) : pow2_df(hmax, Pow2Row{a.kh, a.kl, M, true});
  // what is far below the largest counts in S with fp32's relative precision, and no more is seen of it
  const Df down = ref == M ? df(0.f) : scaled(ref, M, a);  // <= 0
  const float rest_M = ref == M ? rest : rest * ex2_approx((ref - M) * a.kh);
  const Df P0 = h.e * f, Q = h.q, S = df(rest_M) + P0;
  const Df qr = df(1.f) - Q;
  // lane 0: S, lane 1: rest, lane 2: q_r
  const Df x = lane == 0 ? S : lane == 1 ? df(rest) : qr;
  const bool fine = x.h >= 0x1p-126f && x.h < 0x1p127f;  // what log_df takes
  const Df log_x = fine ? log_df(x) : df(__int_as_float(0x7FC00000));
  const Df logS = bcast(log_x), inv = reciprocal(S);
  const Df pr = df(rest_M) * inv;
  const Df up = logS - shift;                                 // ln p_k = x_k - up
  const Df ar = bcast(log_x, 1) + down - logS - bcast(log_x, 2);  // ln p_r - ln q_r
  Df L;
  if (a.kind == TIM_DISTILL_FORWARD_KL)
    L = h.qx + Q * up;
  else
    L = P0.h != 0.f ? ((h.ex * f) - P0 * up) * inv : P0;
  if (tail)
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

// Loss of a row by one CTA that streams it, and with kGrad the gradient in a second pass, which
// finds the row in L2 as far as those in flight, two an SM, fit it: a CTA's fixed work is spread over a
// whole row, and a row's bits cannot depend on the batch.  A row whose sum outside the head is taken
// again (kRestFar, kRestNear) is read once more: 512 such rows of 151936 bf16 logits 95 us against 44.
//
// Bound by memory.  2048 rows of 151936 bf16 logits, K = 64: the loss 115 us, 5.4 TB/s (512 threads and
// two CTAs an SM 136, 128 and eight 121; a cluster of eight CTAs a row with its slice in shared memory
// 205); with the gradient, a quarter of the rows masked, 234 us for 1.09 GB, 4.7 TB/s (256 and four 249,
// one of 1024 238, the cluster 260; plain stores and cached second reads 255).
// In flight are 92 MB of such rows, and 28% of the second reading comes from memory; of fp32 rows 185 MB,
// and 81%: 512 of them, 564 MB read for 311, take 149 us.
template <bool kGrad>
constexpr int kRowThreads = kGrad ? 512 : 256;
constexpr int kRowUnroll = 4;  // vectors of a thread in flight, and as many being summed
template <int kDtype, bool kGrad>
__global__ void __launch_bounds__(kRowThreads<kGrad>, kGrad ? 2 : 4)
    distill_kernel(const DistillArgs a) {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  constexpr int kThreads = kRowThreads<kGrad>, warps = kThreads / 32, U = kRowUnroll;
  extern __shared__ uint4 marks_mem[];  // a byte a vector: which of its tokens are the head's
  __shared__ HeadSums red[kMaxWarps];
  __shared__ float redm[kMaxWarps], reds[kMaxWarps], s_hmax[kMaxWarps];
  __shared__ RowConstants s_terms;
  __shared__ float s_M, s_ref;
  __shared__ int s_bad, s_far, s_near;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x;
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  const int nvec = r.nvec();
  uint8_t* marks = reinterpret_cast<uint8_t*>(marks_mem);
  const int32_t* ids = a.ids + row * a.K;
  const float* lp = a.lp + row * a.K;
  raw* out = nullptr;
  if constexpr (kGrad) out = static_cast<raw*>(a.dlogits) + row * a.ldd;

  const int id0 = tid < a.K ? __ldg(ids + tid) : -1;
  const float lq0 = tid < a.K ? __ldg(lp + tid) : 0.f;
  if (tid == 0) s_bad = s_far = s_near = 0;
  for (int i = tid; i < (nvec + 15) / 16; i += kThreads) marks_mem[i] = make_uint4(0, 0, 0, 0);
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
  if (!__syncthreads_or(any | bad)) {  // no entries
    if (tid == 0) {
      a.loss[row] = 0.f;
      if constexpr (!kGrad) {
        a.lse[row] = 0.f;
        float* saved = a.saved + row * TIM_DISTILL_SAVED;
        for (int i = 0; i < TIM_DISTILL_SAVED; ++i) saved[i] = 0.f;
      }
    }
    if constexpr (kGrad) {
      const Row<kDtype> o(out, 0, 0, a.V);
      gradient_slice<kDtype, kThreads>(a, r, o, Slice{0, o.nvec()}, out, 0.f, 0.f, true);
    }
    return;
  }
  // the first vectors are on their way while the head is done
  const uint4* const vec = r.vec();
  const int w1 = r.w1();
  uint4 u[U];
#pragma unroll
  for (int n = 0; n < U; ++n) {
    const int j = tid + n * kThreads;
    if (j < nvec) u[n] = r.load(j);
  }
  float hmax = -INFINITY;
  for_head([&](int id, float, float z) {
    hmax = fmaxf(hmax, z);
    const int slot = id + r.shift;
    uint32_t* w = reinterpret_cast<uint32_t*>(marks) + slot / E::kVec / 4;
    const uint32_t bit = 1u << (slot / E::kVec % 4 * 8 + slot % E::kVec);
    if ((atomicOr(w, bit) & bit) && bad == 0) bad = TIM_ERR_INVALID_ARG;  // an id twice
  });
  if (bad != 0) atomicMax(&s_bad, bad);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) hmax = fmaxf(hmax, __shfl_xor_sync(0xFFFFFFFFu, hmax, o));
  if (lane == 0) s_hmax[warp] = hmax;
  __syncthreads();
  const int head_warps = min(warps, (a.K + 31) / 32);
  for (int i = 0; i < head_warps; ++i) hmax = fmaxf(hmax, s_hmax[i]);
  const float href = hmax == -INFINITY ? 0.f : hmax;
  if (warp < head_warps) {
    HeadSums h = {};
    for_head([&](int, float lq, float z) {
      const Df t = df(lq) - scaled(z, href, a);
      const Df e = pow2_df(z, Pow2Row{a.kh, a.kl, href, true}), q = exp_df(lq);
      h.e = h.e + e;
      h.q = h.q + q;
      if (q.h != 0.f) h.qx = h.qx + q * t;
      if (e.h != 0.f) h.ex = h.ex - e * t;
    });
    h = warp_sum(h, 16);
    if (lane == 0) red[warp] = h;
  }

  // ---- sum of 2^((z - reference) log2e / tau) outside the head
  const float k2 = a.kh;
  auto unmarked = [&](const uint4& x, int j, float(&v)[E::kVec]) {
    E::unpack(x, v);
    const uint32_t mk = marks[j];
    if (mk != 0) {
#pragma unroll
      for (int i = 0; i < E::kVec; ++i)
        if ((mk >> i) & 1u) v[i] = -INFINITY;
    }
  };
  float m = href, sum;
  {
    const F2 ref = f2(-href, -href), kk = f2(k2, k2);
    F2 acc = f2(0.f, 0.f), acc2 = acc;
    for (int j0 = tid; j0 < nvec; j0 += U * kThreads) {
      uint4 w[U];
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int j = j0 + (U + n) * kThreads;
        if (j < w1)
          w[n] = __ldg(vec + j);
        else if (j < nvec)
          w[n] = r.load_edge(j);
      }
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int j = j0 + n * kThreads;
        if (j < nvec) {
          float v[E::kVec];
          unmarked(u[n], j, v);
#pragma unroll
          for (int i = 0; i < E::kVec; i += 4) {
            acc = add2(acc, ex2x2(mul2(add2(f2(v[i], v[i + 1]), ref), kk)));
            acc2 = add2(acc2, ex2x2(mul2(add2(f2(v[i + 2], v[i + 3]), ref), kk)));
          }
        }
        u[n] = w[n];
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
  if (lane == 0 && !(sum < kRestFar)) s_far = 1;
  if (lane == 0 && sum >= kRestNear) s_near = 1;
  __syncthreads();
  bool again = s_far != 0 || hmax == -INFINITY;
  if (a.tail != 0 && s_near == 0) {
    Df Q = df(0.f);
    for (int i = 0; i < head_warps; ++i) Q = Q + red[i].q;
    again |= (df(1.f) - Q).h > kTailFloor * 0.5f;
  }
  // far above the head, far below it, or a head without mass to refer to: again, with a running maximum
  if (again) {
    m = -INFINITY;
    sum = 0.f;
    for (int j = tid; j < nvec; j += kThreads) {
      float v[E::kVec];
      unmarked(r.load(j), j, v);
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
  const float nan = __int_as_float(0x7FC00000);
  HeadSums hs = {};
  float M = 0.f;
  bool tail = false;
  if (warp == 0) {
    m = lane < warps ? redm[lane] : -INFINITY;
    sum = lane < warps ? reds[lane] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
      merge(m, sum, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, sum, o), k2);
    m = __shfl_sync(0xFFFFFFFFu, m, 0);
    sum = __shfl_sync(0xFFFFFFFFu, sum, 0);
    if (lane < head_warps) hs = red[lane];
    if (head_warps > 1) hs = warp_sum(hs, 8);
    hs = HeadSums{bcast(hs.e), bcast(hs.q), bcast(hs.qx), bcast(hs.ex)};
    M = fmaxf(hmax, m);
    if (m == -INFINITY) m = M;  // nothing outside
    RowConstants c = row_constants(a, M, hmax, m, sum, hs);
    tail = c.tail;
    if (lane == 0) {
      if (s_bad != 0) c.c_rest = c.c_head = nan;
      s_terms = c;
      s_M = M;
      s_ref = m;
      if constexpr (!kGrad) {
        float* saved = a.saved + row * TIM_DISTILL_SAVED;
        saved[kMax] = M;
        saved[kInvSum] = c.inv;
        saved[kLogSum] = c.logS;
        saved[kRest] = c.c_rest;
        saved[kHead] = c.c_head;
        saved[kLive] = s_bad != 0 ? nan : 1.f;
        saved[kRef] = m;
        saved[kRef + 1] = 0.f;
      }
    }
    __syncwarp();
  }
  if (kGrad) __syncthreads();
  if (warp == 0) {  // nothing waits for the loss
    const RowLoss v = row_loss(a, M, hmax, m, sum, hs, tail);
    if (lane == 0) {
      if (s_bad != 0)
        set_status(a.status, s_bad);
      else if (!(isfinite(v.lse) && isfinite(v.loss)))
        set_status(a.status, TIM_ERR_NONFINITE);
      a.loss[row] = s_bad != 0 ? nan : v.loss;
      if constexpr (!kGrad) a.lse[row] = s_bad != 0 ? nan : v.lse;
    }
  }
  if constexpr (kGrad) {
    const float w = __ldg(a.grad + row), g = w * a.inv_h;
    const RowConstants t = s_terms;
    const Row<kDtype> o(out, 0, 0, a.V);
    gradient_slice<kDtype, kThreads>(a, r, o, Slice{0, o.nvec()}, out, s_ref,
                                     t.c_rest * t.inv * g, w == 0.f);
    if (w == 0.f) return;
    __syncthreads();  // the head's tokens are written again, after the whole row
    M = s_M;
    for_head([&](int id, float lq, float z) {
      out[id] = E::narrow(head_gradient(a, z, lq, M, t.logS, t.inv, t.c_head) * g);
    });
  }
}

// The gradient alone, from what the forward saved: a CTA a slice of a row, reading and writing
// it once; the head's tokens are written again after the slice.  Bound by memory: 512 rows of
// 151936 bf16 logits 52 us, 6.0 TB/s read and written.
template <int kDtype>
__global__ void __launch_bounds__(kBackThreads) distill_backward_kernel(const DistillArgs a) {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  const int64_t row = blockIdx.x / a.parts;
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  raw* out = static_cast<raw*>(a.dlogits) + row * a.ldd;
  const Row<kDtype> o(out, 0, 0, a.V);
  const Slice s = slice_of(o.nvec(), blockIdx.x % a.parts, a.parts);
  const float* saved = a.saved + row * TIM_DISTILL_SAVED;
  const float w = __ldg(a.grad + row), live = saved[kLive], g = w * a.inv_h;
  const bool zero = live == 0.f || w == 0.f;
  const float M = saved[kMax], inv = saved[kInvSum];
  // NaN for a row the forward refused
  gradient_slice<kDtype, kBackThreads>(a, r, o, s, out, saved[kRef], live * saved[kRest] * inv * g,
                                       zero);
  if (zero || live != live) return;
  __syncthreads();
  const float logS = saved[kLogSum];
  for (int k = threadIdx.x; k < a.K; k += kBackThreads) {
    const int id = __ldg(a.ids + row * a.K + k);
    const float lq = __ldg(a.lp + row * a.K + k);
    const int slot = id + o.shift - s.j0 * E::kVec;
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

template <int kDtype, bool kGrad>
cudaError_t launch_rows(const DistillArgs& a, int64_t T, cudaStream_t stream) {
  auto marks = [](int64_t V) {
    return static_cast<size_t>(V * sizeof(typename Elem<kDtype>::raw) / 16 + 2 + 31) / 16 * 16;
  };
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(distill_kernel<kDtype, kGrad>, marks(TIM_LOGITS_MAX_V), allowed);
  if (e != cudaSuccess) return e;
  const size_t smem = marks(a.V);
  distill_kernel<kDtype, kGrad><<<static_cast<unsigned>(T), kRowThreads<kGrad>, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int kDtype>
cudaError_t launch_back(DistillArgs a, int64_t T, cudaStream_t stream) {
  a.parts = plan_row(a.V, sizeof(typename Elem<kDtype>::raw)).cluster;
  if (T * a.parts > INT32_MAX) return cudaErrorInvalidValue;
  distill_backward_kernel<kDtype>
      <<<static_cast<unsigned>(T * a.parts), kBackThreads, 0, stream>>>(a);
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
