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
// head's exponentials are taken on their own, to 2^-33, with every sum over the head in
// fp64: the loss is a difference of near numbers.
#include <cmath>

#include "logits_row.cuh"

namespace tim {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr float kTailFloor = 9.5367431640625e-7f;  // 2^-20

struct DistillArgs {
  const void* logits;
  int64_t ld;
  int V;
  int K;
  const int32_t* ids;
  const float* lp;
  float temperature;
  int kind;
  int tail;
  float* loss;
  float* lse;
  float* saved;  // [T][TIM_DISTILL_SAVED]
  const float* grad;
  void* dlogits;
  int64_t ldd;
  int* status;
};

// What the backward needs of a row, as saved by the forward.
enum Saved { kMax = 0, kInvSum, kLogSum, kLogSumLo, kRest, kHead, kLive };

// Sum of a double over the block, the same in every thread; a fixed order.
__device__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += red[i];
  return s;
}

__device__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float m = -INFINITY;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) m = fmaxf(m, red[i]);
  return m;
}

__device__ __forceinline__ bool in_head(int id, float lp) { return id >= 0 && lp != -INFINITY; }

template <int kDtype>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a) {
  using E = Elem<kDtype>;
  extern __shared__ uint32_t bitmap[];  // one bit a slot of the row
  __shared__ double red[kWarps];
  __shared__ float redf[kWarps];
  __shared__ int s_count, s_bad;
  const int64_t row = blockIdx.x;
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  const int32_t* ids = a.ids + row * a.K;
  const float* lp = a.lp + row * a.K;
  const int nvec = r.nvec();
  const int words = (nvec * E::kVec + 31) / 32;
  for (int i = threadIdx.x; i < words; i += kThreads) bitmap[i] = 0u;
  if (threadIdx.x == 0) s_count = s_bad = 0;
  __syncthreads();
  float hmax = -INFINITY;
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const int id = ids[k];
    const float q = lp[k];
    if (id < -1 || id >= a.V) {
      s_bad = TIM_ERR_TOKEN_RANGE;
    } else if (id >= 0 && !(q <= 1.f)) {  // not the logarithm of a probability, or NaN
      s_bad = TIM_ERR_INVALID_ARG;
    } else if (in_head(id, q)) {
      const int s = id + r.shift;
      const uint32_t bit = 1u << (s & 31);
      if (atomicOr(&bitmap[s >> 5], bit) & bit) s_bad = TIM_ERR_INVALID_ARG;
      hmax = fmaxf(hmax, r.at(id));
      s_count = 1;
    }
  }
  __syncthreads();
  float* saved = a.saved + row * TIM_DISTILL_SAVED;
  if (s_bad != 0 || s_count == 0) {
    if (threadIdx.x == 0) {
      const float v = s_bad != 0 ? __int_as_float(0x7FC00000) : 0.f;
      if (s_bad != 0) set_status(a.status, s_bad);
      a.loss[row] = v;
      a.lse[row] = v;
      for (int i = 0; i < TIM_DISTILL_SAVED; ++i) saved[i] = 0.f;
      saved[kLive] = s_bad != 0 ? __int_as_float(0x7FC00000) : 0.f;
    }
    return;
  }

  // the tokens outside the head: running maximum and sum of 2^((z - max) log2e / tau)
  const float k2 = static_cast<float>(1.4426950408889634 / static_cast<double>(a.temperature));
  float m = -INFINITY, sum = 0.f;
  for (int j = threadIdx.x; j < nvec; j += kThreads) {
    float v[E::kVec];
    E::unpack(r.load(j), v);
    const int s0 = j * E::kVec;
    uint32_t marks = (bitmap[s0 >> 5] >> (s0 & 31)) & ((1u << E::kVec) - 1u);
    if (marks != 0) {
#pragma unroll
      for (int i = 0; i < E::kVec; ++i)
        if ((marks >> i) & 1u) v[i] = -INFINITY;
    }
    float vm = v[0];
#pragma unroll
    for (int i = 1; i < E::kVec; ++i) vm = fmaxf(vm, v[i]);
    if (vm > m) {
      sum *= ex2_approx((m - vm) * k2);
      m = vm;
    }
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < E::kVec; ++i) sum += ex2_approx((v[i] - base) * k2);
  }
  const float M = fmaxf(block_max(m, redf), block_max(hmax, redf));
  const double rest =
      block_sum(m == -INFINITY ? static_cast<double>(sum)  // 0, or NaN
                               : static_cast<double>(sum * ex2_approx((m - M) * k2)), red);

  // the head
  Pow2Row pw = pow2_row(a.temperature, M);
  pw.recentre = 1;
  pw.c = M;
  const double inv_tau = 1.0 / static_cast<double>(a.temperature);
  double sE = 0, sQ = 0, sQX = 0, sEX = 0;
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const int id = ids[k];
    const float lq = lp[k];
    if (!in_head(id, lq)) continue;
    const float z = r.at(id);
    const double x = (static_cast<double>(z) - M) * inv_tau;  // ln p_k + ln S
    const double e = x < -600.0 ? 0.0 : pow2_double(z, pw, g_pow2_table.t);
    Pow2Row qw = pow2_row(1.f, 0.f);
    const double q = lq < -600.f ? 0.0 : pow2_double(lq, qw, g_pow2_table.t);
    sE += e;
    sQ += q;
    if (q != 0.0) sQX += q * (static_cast<double>(lq) - x);
    if (e != 0.0) sEX += e * (x - static_cast<double>(lq));
  }
  const double P0 = block_sum(sE, red), Q = block_sum(sQ, red);
  const double QX = block_sum(sQX, red), EX = block_sum(sEX, red);
  if (threadIdx.x == 0) {
    const double S = rest + P0, logS = log(S);
    const double P = P0 / S, pr = rest / S;
    double qr = 1.0 - Q;
    const bool tail = a.tail != 0 && qr > static_cast<double>(kTailFloor) && rest > 0.0;
    if (!tail) qr = 0.0;
    double L, c_rest, c_head;
    if (a.kind == TIM_DISTILL_FORWARD_KL) {
      L = QX + Q * logS;
      c_rest = Q;
      c_head = Q + qr;
      if (tail) {
        L += qr * (log(qr) - log(pr));
        c_rest -= qr * P / pr;
      }
    } else {
      L = EX / S - P * logS;
      double B = L + P;
      c_rest = 0.0;
      if (tail) {
        const double ar = log(pr) - log(qr);
        L += pr * ar;
        B += pr * (ar + 1.0);
        c_rest = ar + 1.0;
      }
      c_rest -= B;
      c_head = 1.0 - B;
    }
    const double lse = static_cast<double>(M) * inv_tau + logS;
    if (!(isfinite(lse) && isfinite(L))) set_status(a.status, TIM_ERR_NONFINITE);
    a.loss[row] = static_cast<float>(L);
    a.lse[row] = static_cast<float>(lse);
    const float ls = static_cast<float>(logS);
    saved[kMax] = M;
    saved[kInvSum] = static_cast<float>(1.0 / S);
    saved[kLogSum] = ls;
    saved[kLogSumLo] = static_cast<float>(logS - static_cast<double>(ls));
    saved[kRest] = static_cast<float>(c_rest);
    saved[kHead] = static_cast<float>(c_head);
    saved[kLive] = 1.f;
    saved[kLive + 1] = 0.f;
  }
}

template <int kDtype>
__global__ void __launch_bounds__(kThreads) distill_backward_kernel(const DistillArgs a) {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  const int64_t row = blockIdx.x;
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  raw* out = static_cast<raw*>(a.dlogits) + row * a.ldd;
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(r.p)) & 15u) == 0;
  const float* saved = a.saved + row * TIM_DISTILL_SAVED;
  const float live = saved[kLive], g = a.grad[row] / a.temperature;
  const int nvec = r.nvec();
  const bool zero = live == 0.f || g == 0.f;
  const float k2 = static_cast<float>(1.4426950408889634 / static_cast<double>(a.temperature));
  const float M = saved[kMax], inv = saved[kInvSum];
  const float c = live * saved[kRest] * inv * g;  // NaN for a row the forward refused
  for (int j = threadIdx.x; j < nvec; j += kThreads) {
    float v[E::kVec];
    if (zero) {
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) v[i] = 0.f;
    } else {
      E::unpack(r.load(j), v);
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) v[i] = c * ex2_approx((v[i] - M) * k2);
    }
    if (same && r.whole(j)) {
      *reinterpret_cast<uint4*>(out - r.shift + static_cast<int64_t>(j) * E::kVec) = E::pack(v);
    } else {
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) {
        const int s = j * E::kVec + i - r.shift;
        if (s >= 0 && s < a.V) out[s] = E::narrow(v[i]);
      }
    }
  }
  if (zero || live != live) return;
  __syncthreads();  // the head's tokens are written again, after the whole row
  Pow2Row pw = pow2_row(a.temperature, M);
  pw.recentre = 1;
  pw.c = M;
  const double inv_tau = 1.0 / static_cast<double>(a.temperature);
  const double logS = static_cast<double>(saved[kLogSum]) + static_cast<double>(saved[kLogSumLo]);
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const int id = a.ids[row * a.K + k];
    const float lq = a.lp[row * a.K + k];
    if (!in_head(id, lq) || id >= a.V) continue;
    const float z = r.at(id);
    const double x = (static_cast<double>(z) - M) * inv_tau;
    const double p =
        x < -600.0 ? 0.0 : pow2_double(z, pw, g_pow2_table.t) * static_cast<double>(inv);
    double d;
    if (a.kind == TIM_DISTILL_FORWARD_KL) {
      Pow2Row qw = pow2_row(1.f, 0.f);
      const double q = lq < -600.f ? 0.0 : pow2_double(lq, qw, g_pow2_table.t);
      d = p * saved[kHead] - q;
    } else {
      d = p == 0.0 ? 0.0 : p * (x - logS - lq + saved[kHead]);
    }
    out[id] = E::narrow(static_cast<float>(d * g));
  }
}

template <int kDtype>
cudaError_t launch_forward(const DistillArgs& a, int64_t T, cudaStream_t stream) {
  const size_t smem = (static_cast<size_t>(a.V) + 16 + 31) / 32 * 4 + 16;
  cudaError_t e = cudaFuncSetAttribute(distill_kernel<kDtype>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  distill_kernel<kDtype><<<static_cast<unsigned>(T), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int kDtype>
cudaError_t launch_backward(const DistillArgs& a, int64_t T, cudaStream_t stream) {
  distill_backward_kernel<kDtype><<<static_cast<unsigned>(T), kThreads, 0, stream>>>(a);
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
  a.temperature = temperature;
  a.kind = kind;
  a.tail = tail;
  a.loss = loss;
  a.lse = lse;
  a.saved = saved;
  a.status = status;
  return dtype == TIM_F32    ? launch_forward<TIM_F32>(a, T, stream)
         : dtype == TIM_BF16 ? launch_forward<TIM_BF16>(a, T, stream)
                             : launch_forward<TIM_F16>(a, T, stream);
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
  a.temperature = temperature;
  a.kind = kind;
  a.saved = const_cast<float*>(saved);
  a.grad = grad;
  a.dlogits = dlogits;
  a.ldd = ldd;
  return dtype == TIM_F32    ? launch_backward<TIM_F32>(a, T, stream)
         : dtype == TIM_BF16 ? launch_backward<TIM_BF16>(a, T, stream)
                             : launch_backward<TIM_F16>(a, T, stream);
}

}  // namespace tim
