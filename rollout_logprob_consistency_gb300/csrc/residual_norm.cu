// The residual update after a block, with the norms before and after it, and its gradient.
//
//   n  = x / sqrt(mean x^2 + eps) gamma_post   (or x)          x: the block's output
//   h' = h + scale g n                                          g: a gate a channel, a token, an element
//   y  = h' / sqrt(mean h'^2 + eps) gamma                       the next block's input
//
// h' is rounded to its type before y is taken from it: y is the norm of the h' that is stored, which is
// what a later reader of it has (tim_logprob's final norm sums in another order, so an element of its
// own y in some thousand is a step of the type away from this one's).
//
// Memory's: a row is read once into registers and its one or two sums are taken by the CTA that
// holds it.  How a row is split over threads depends on d and on whether all of the call's rows are whole
// 16-byte vectors (addresses, strides and d alike; see Cols): a row's bits do not depend on the other
// rows or on their number, but a copy of it at another alignment may differ in the last one.
#include "residual_norm.cuh"

#include <algorithm>
#include <type_traits>

#include "logits_row.cuh"

namespace tim {
namespace {

// A row's elements: thread t holds kVecs vectors of 16 bytes.  kWide: they are whole vectors of
// memory, t, t + threads, ...; else (rows that do not start at 16-byte boundaries, or end between
// them) the same registers are filled with single elements, neighbouring threads' next to one another.
// What lies beyond the row reads as 0.
template <int kDtype, bool kWide>
struct Cols {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  static constexpr int kVec = E::kVec;
  static __device__ __forceinline__ int col(int k, int i) {
    const int v = k * blockDim.x;
    return kWide ? (v + threadIdx.x) * kVec + i : v * kVec + i * blockDim.x + threadIdx.x;
  }
  static __device__ __forceinline__ uint4 load(const void* p, int k, int d) {
    const raw* const row = static_cast<const raw*>(p);
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (kWide) {
      if (col(k, 0) < d) u = *reinterpret_cast<const uint4*>(row + col(k, 0));
    } else {
      raw* const to = reinterpret_cast<raw*>(&u);
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (col(k, i) < d) to[i] = row[col(k, i)];
    }
    return u;
  }
  static __device__ __forceinline__ void store(void* p, int k, int d, const uint4& u) {
    raw* const row = static_cast<raw*>(p);
    if constexpr (kWide) {
      if (col(k, 0) < d) *reinterpret_cast<uint4*>(row + col(k, 0)) = u;
    } else {
      const raw* const from = reinterpret_cast<const raw*>(&u);
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (col(k, i) < d) row[col(k, i)] = from[i];
    }
  }
  static __device__ __forceinline__ const void* at(const void* p, int64_t offset) {
    return static_cast<const raw*>(p) + offset;
  }
  static __device__ __forceinline__ void* at(void* p, int64_t offset) {
    return static_cast<raw*>(p) + offset;
  }
};

// The sums of up to three numbers over a warp, in a fixed order, with fewer exchanges than three times
// five: the first halves what the lanes hold by handing one number over for another.  Sum n is
// lane lane_of(n)'s.
__device__ __forceinline__ int lane_of(int n) { return n == 0 ? 0 : n == 1 ? 16 : 8; }
template <int kN>
__device__ __forceinline__ float warp_sums(const float (&v)[kN]) {
  const int lane = threadIdx.x & 31;
  float r = v[0];
  if constexpr (kN > 1) {
    const bool up = (lane & 16) != 0;
    r = (up ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[0] : v[1], 16);
  } else {
    r += __shfl_xor_sync(0xFFFFFFFFu, r, 16);
  }
  if constexpr (kN > 2) {
    const float c = v[2] + __shfl_xor_sync(0xFFFFFFFFu, v[2], 16);
    const bool up = (lane & 8) != 0;
    r = (up ? c : r) + __shfl_xor_sync(0xFFFFFFFFu, up ? r : c, 8);
  } else {
    r += __shfl_xor_sync(0xFFFFFFFFu, r, 8);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
  return r;
}
// Over the CTA, in every thread.  Two calls in a row need different scratch.
template <int kN>
__device__ __forceinline__ void block_sum(float (&v)[kN], float (*scratch)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const float mine = warp_sums(v);
#pragma unroll
  for (int n = 0; n < kN; ++n)
    if (lane == lane_of(n)) scratch[n][warp] = mine;
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kN; ++n) v[n] = lane < warps ? scratch[n][lane] : 0.f;
  const float all = warp_sums(v);
#pragma unroll
  for (int n = 0; n < kN; ++n) v[n] = __shfl_sync(0xFFFFFFFFu, all, lane_of(n));
}

// Where row's gate begins: of a channel gate all rows'.
template <class C>
__device__ __forceinline__ const void* gate_of(const tim_block& b, int64_t row) {
  return C::at(b.gate, b.gate_kind == TIM_GATE_CHANNEL ? 0 : row * b.ld_gate);
}

template <int kDtype, bool kWide, int kVecs, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) residual_norm_kernel(const NormArgs a) {
  using E = Elem<kDtype>;
  using C = Cols<kDtype, kWide>;
  constexpr int kVec = E::kVec;
  __shared__ float scratch[2][1][32];
  const tim_block& b = a.b;
  const int64_t row = blockIdx.x;
  const int d = b.d;
  const float inv_d = 1.f / static_cast<float>(d);
  uint4 xs[kVecs], hs[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    xs[k] = C::load(C::at(b.block, row * b.ld_block), k, d);
    hs[k] = C::load(C::at(a.residual, row * a.ld_residual), k, d);
  }
  float r1 = 1.f;
  if (b.gamma_post != nullptr) {
    float ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      float v[kVec];
      E::unpack(xs[k], v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) ss[0] = fmaf(v[i], v[i], ss[0]);
    }
    block_sum(ss, scratch[0]);
    r1 = rsqrtf(ss[0] * inv_d + b.eps);
  }
  const void* const gate = gate_of<C>(b, row);
  const float by_row = b.gate_kind == TIM_GATE_TOKEN
                           ? E::widen(*static_cast<const typename E::raw*>(gate))
                           : 1.f;
  float ss[1] = {0.f};
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    float n[kVec], v[kVec], w[kVec];
    E::unpack(xs[k], n);
    E::unpack(hs[k], v);
    if (b.gamma_post != nullptr) {
      E::unpack(C::load(b.gamma_post, k, d), w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) n[i] = n[i] * r1 * w[i];
    }
    if (b.gate_kind >= TIM_GATE_CHANNEL) {
      E::unpack(C::load(gate, k, d), w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) n[i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = fmaf(b.scale, n[i] * by_row, v[i]);
    hs[k] = E::pack(v);
    C::store(C::at(a.out_h, row * a.ld_h), k, d, hs[k]);
    E::unpack(hs[k], v);
#pragma unroll
    for (int i = 0; i < kVec; ++i) ss[0] = fmaf(v[i], v[i], ss[0]);
  }
  if (b.gamma == nullptr) return;
  block_sum(ss, scratch[1]);
  const float r2 = rsqrtf(ss[0] * inv_d + b.eps);
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    float v[kVec], w[kVec];
    E::unpack(hs[k], v);
    E::unpack(C::load(b.gamma, k, d), w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = (v[i] * r2) * w[i];
    C::store(C::at(a.out_y, row * a.ld_y), k, d, E::pack(v));
  }
}

// ---- the gradient.  With H the whole gradient of h':
//   H      = dh' + r2 gamma dy - h' r2^3/d sum(gamma dy h')      dh = H
//   dn     = scale g H,  dg = scale n H (summed over what a gate is shared by)
//   dx     = r1 gamma_post dn - x r1^3/d sum(gamma_post dn x)   (or dn)
//   dgamma = sum_t dy h' r2,  dgamma_post = sum_t dn x r1
// Two sums a row, the second from the first: with t = H gamma_post x all that is left are
//   q = sum t (of a gate a channel or an element: sum g t),
//   dx = scale g r1 (gamma_post H - x r1^2/d q),   dg = scale r1 t   (a token's: scale r1 q).
// A CTA takes every gridDim-th row; the sums over its rows stay in registers, a thread's columns, and are
// left in the workspace for residual_fold_kernel.
//
// 16384 rows of 4096 bf16 with both norms and a gate a token take 158 us, 5.1 TB/s, and the fold 4.5.  Waiting
// bounds it: with what a row keeps in registers 16 warps share an SM, and between a row's two sums over the
// CTA they wait beside too few others (issue slots 47% used, DRAM 62%; stalled for shared memory and exchanges
// 1.8 warps a cycle issued, for memory 1.7, for fixed latencies 1.6, at barriers 0.5).
//
// kStages: the rows that are on their way to shared memory while one is worked on, copied by the
// threads that will read them, so that they wait for their own copies alone.  0: rows are read where
// they lie, each time they are needed: rows of more than 1024 vectors, for which an SM's shared memory would
// not do (4096 rows of 16384 bf16 306 us where their bytes would take 119), and rows that are not whole
// vectors (16384 rows of 4096 bf16 with a stride of 4099 1162 us).  Those kernels spill: more than 1024 vectors
// 208 to 392 bytes a thread where they are whole (fp32 up to 2048 none) and 148 to 1480 where they are not, fewer
// that are not whole 24 to 472 in 16 bits.

// Where a row's four operands come from.
template <int kDtype, bool kWide, int kVecs, int kThreads, int kStages>
struct RowSource {
  using C = Cols<kDtype, kWide>;
  const NormGradArgs& a;
  uint4* mem;
  const void* at[4];  // block, h, dy, dh; null: zeros

  __device__ __forceinline__ void point(int64_t row) {
    at[0] = C::at(a.b.block, row * a.b.ld_block);
    at[1] = a.h != nullptr ? C::at(a.h, row * a.ld_h) : nullptr;
    at[2] = a.dy != nullptr ? C::at(a.dy, row * a.ld_dy) : nullptr;
    at[3] = a.dh != nullptr ? C::at(a.dh, row * a.ld_dh) : nullptr;
  }
  __device__ __forceinline__ uint4* slot(int stage, int t, int k) const {
    return mem + ((stage * 4 + t) * kVecs + k) * kThreads + threadIdx.x;
  }
  // Zeros where no copy will write.
  __device__ __forceinline__ void clear() {
    point(0);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        if (at[t] == nullptr || C::col(k, 0) >= a.b.d)
          for (int s = 0; s < kStages; ++s) *slot(s, t, k) = make_uint4(0u, 0u, 0u, 0u);
  }
  // Starts the copies of a row, if there is one; a group for the wait either way.
  __device__ __forceinline__ void start(int64_t row, int stage) {
    if (row < a.b.T) {
      point(row);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
          if (at[t] != nullptr && C::col(k, 0) < a.b.d)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot(stage, t, k))),
                         "l"(C::at(at[t], C::col(k, 0)))
                         : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // The gammas and a channel gate, which every row needs.
  __device__ __forceinline__ uint4* shared_slot(int n, int k) const {
    return mem + ((kStages * 4 + n) * kVecs + k) * kThreads + threadIdx.x;
  }
  __device__ __forceinline__ void keep(int n, const void* p) const {
    if (p == nullptr) return;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) *shared_slot(n, k) = C::load(p, k, a.b.d);
  }
  __device__ __forceinline__ uint4 kept(int n, const void* p, int k) const {
    if constexpr (kStages == 0)
      return C::load(p, k, a.b.d);
    else
      return *shared_slot(n, k);
  }
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  }
  __device__ __forceinline__ uint4 get(int stage, int t, int k) const {
    if constexpr (kStages == 0) {
      return at[t] != nullptr ? C::load(at[t], k, a.b.d) : make_uint4(0u, 0u, 0u, 0u);
    } else {
      return *slot(stage, t, k);
    }
  }
};

// CTAs of an SM, at most six: those of 64 threads would leave many parts to the fold.
template <int kVecs, int kThreads>
constexpr int kResident = kVecs * kThreads > 512 ? 1 : std::min(1024 / (kThreads * kVecs), 6);

template <int kDtype, bool kWide, int kVecs, int kThreads, int kStages, bool kChannel>
__global__ void __launch_bounds__(kThreads, kResident<kVecs, kThreads>)
    residual_norm_backward_kernel(const NormGradArgs a) {
  using E = Elem<kDtype>;
  using C = Cols<kDtype, kWide>;
  constexpr int kVec = E::kVec, kHalf = kVec / 2;
  extern __shared__ uint4 ring[];
  __shared__ float scratch1[3][32], scratch2[1][32];
  const tim_block& b = a.b;
  const int d = b.d;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool pre = a.dy != nullptr, post = b.gamma_post != nullptr;
  constexpr bool by_channel = kChannel;
  const bool by_element = !kChannel && b.gate_kind == TIM_GATE_ELEMENT;
  const bool by_token = !kChannel && b.gate_kind == TIM_GATE_TOKEN;
  RowSource<kDtype, kWide, kVecs, kThreads, kStages> src{a, ring, {}};
  if constexpr (kStages > 0) {
    src.clear();
    src.keep(0, b.gamma);
    src.keep(1, b.gamma_post);
    if (by_channel) src.keep(2, b.gate);
#pragma unroll
    for (int s = 0; s < kStages; ++s)
      src.start(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
  }
  auto load2 = [](const uint4& u, F2 (&v)[kHalf]) {
    float f[kVec];
    E::unpack(u, f);
#pragma unroll
    for (int i = 0; i < kHalf; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
  };
  auto pack2 = [](const F2 (&v)[kHalf]) {
    float f[kVec];
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      const float2 t = unpack2(v[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
    return E::pack(f);
  };
  F2 acc_pre[kVecs][kHalf], acc_post[kVecs][kHalf], acc_gate[kVecs][kHalf];
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int i = 0; i < kHalf; ++i) acc_pre[k][i] = acc_post[k][i] = acc_gate[k][i] = f2(0.f, 0.f);
  // a token's gate is asked for a row ahead
  auto gate_at = [&](int64_t row) {
    return row < b.T ? E::widen(*static_cast<const typename E::raw*>(gate_of<C>(b, row))) : 0.f;
  };
  float row_gate = by_token ? gate_at(blockIdx.x) : 1.f;
  int stage = 0;
  for (int64_t row = blockIdx.x; row < b.T; row += gridDim.x) {
    if constexpr (kStages > 0)
      src.wait();
    else
      src.point(row);
    // H holds gamma dy until its sums are known
    F2 t1[3] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
    F2 H[kVecs][kHalf];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      F2 v[kHalf], w[kHalf];
      if (pre) {
        load2(src.get(stage, 1, k), v);
        load2(src.get(stage, 2, k), H[k]);
        load2(src.kept(0, b.gamma, k), w);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          H[k][i] = mul2(H[k][i], w[i]);
          t1[0] = fma2(v[i], v[i], t1[0]);
          t1[1] = fma2(H[k][i], v[i], t1[1]);
        }
      }
      if (post) {
        load2(src.get(stage, 0, k), v);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) t1[2] = fma2(v[i], v[i], t1[2]);
      }
    }
    float s1[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const float2 t = unpack2(t1[i]);
      s1[i] = t.x + t.y;
    }
    if (pre || post) block_sum(s1, scratch1);
    const float r2 = pre ? rsqrtf(s1[0] * inv_d + b.eps) : 0.f;
    // r^2 and r^3 alone may leave fp32's range where the gradient is well within it
    const float c2 = pre ? r2 * (inv_d * s1[1]) * r2 : 0.f;
    const float r1 = post ? rsqrtf(s1[2] * inv_d + b.eps) : 1.f;
    const float by_row = b.scale * row_gate;  // all of the gate that is not an element's own
    if (by_token) row_gate = gate_at(row + gridDim.x);
    const F2 r2s = f2(r2, r2), c2s = f2(-c2, -c2), by_r1 = f2(by_row * r1, by_row * r1);
    F2 tq = f2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      F2 v[kHalf], w[kHalf], u[kHalf];
      load2(src.get(stage, 3, k), w);
      if (pre) {
        load2(src.get(stage, 1, k), v);
        load2(src.get(stage, 2, k), u);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          H[k][i] = fma2(r2s, fma2(c2s, v[i], H[k][i]), w[i]);
          acc_pre[k][i] = fma2(mul2(u[i], v[i]), r2s, acc_pre[k][i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) H[k][i] = w[i];
      }
      C::store(C::at(a.out_dresidual, row * a.ld_dresidual), k, d, pack2(H[k]));
      load2(src.get(stage, 0, k), u);
      if (post) load2(src.kept(1, b.gamma_post, k), w);
      if (by_channel || by_element) {
        F2 t[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) t[i] = mul2(post ? mul2(H[k][i], w[i]) : H[k][i], u[i]);
        if (by_channel) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) acc_gate[k][i] = fma2(t[i], by_r1, acc_gate[k][i]);
        } else {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) t[i] = mul2(t[i], by_r1);
          C::store(C::at(a.out_dgate, row * a.ld_dgate), k, d, pack2(t));
        }
        load2(by_channel ? src.kept(2, b.gate, k) : C::load(gate_of<C>(b, row), k, d), v);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) H[k][i] = mul2(H[k][i], v[i]);
      }
      if (post) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          const F2 t = mul2(H[k][i], u[i]);
          acc_post[k][i] = fma2(t, by_r1, acc_post[k][i]);
          tq = fma2(t, w[i], tq);
          H[k][i] = mul2(H[k][i], w[i]);
        }
      } else if (by_token) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) tq = fma2(H[k][i], u[i], tq);
      }
    }
    const float2 tqs = unpack2(tq);
    float q[1] = {tqs.x + tqs.y};
    if (post || by_token) block_sum(q, scratch2);
    if (by_token && threadIdx.x == 0) static_cast<float*>(a.out_dgate)[row] = b.scale * r1 * q[0];
    const float c1 = post ? r1 * (inv_d * q[0]) * r1 : 0.f;
    const F2 c1s = f2(-c1, -c1);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (post) {
        F2 u[kHalf];
        load2(src.get(stage, 0, k), u);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) H[k][i] = mul2(by_r1, fma2(c1s, u[i], H[k][i]));
      } else {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) H[k][i] = mul2(by_r1, H[k][i]);
      }
      C::store(C::at(a.out_dblock, row * a.ld_dblock), k, d, pack2(H[k]));
    }
    if constexpr (kStages > 0) {
      src.start(row + static_cast<int64_t>(kStages) * gridDim.x, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    // with two sums a row each one's barrier parts the other's scratch from the next row's; with one:
    if ((pre || post) != (post || by_token)) __syncthreads();
  }
  float* const part = a.partial + static_cast<int64_t>(blockIdx.x) * 3 * d;
  auto leave = [&](int which, int k, const F2 (&v)[kHalf]) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = C::col(k, i);
      const float2 t = unpack2(v[i / 2]);
      if (c < d) part[which * d + c] = i % 2 == 0 ? t.x : t.y;
    }
  };
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    if (b.gamma != nullptr) leave(0, k, acc_pre[k]);
    if (post) leave(1, k, acc_post[k]);
    if (by_channel) leave(2, k, acc_gate[k]);
  }
}

// out[c] (+)= sum over the CTAs of part[.][which][c], in order: a CTA has 32 columns of one kind, and
// its warps share the parts of a column.
constexpr int kFoldWarps = 32;
struct FoldArgs {
  const float* partial;
  int parts, d, accumulate;
  float* out[3];
};
__global__ void __launch_bounds__(32 * kFoldWarps) residual_fold_kernel(const FoldArgs a) {
  __shared__ float sum[kFoldWarps][32];
  float* const out = a.out[blockIdx.y];
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const int per = (a.parts + kFoldWarps - 1) / kFoldWarps;
  float acc = 0.f;
  if (c < a.d) {
    const float* const p = a.partial + static_cast<int64_t>(blockIdx.y) * a.d + c;
    const int i1 = min(a.parts, (warp + 1) * per);
#pragma unroll 8
    for (int i = warp * per; i < i1; ++i) acc += __ldg(p + static_cast<int64_t>(i) * 3 * a.d);
  }
  sum[warp][lane] = acc;
  __syncthreads();
  if (warp != 0 || c >= a.d) return;
#pragma unroll
  for (int w = 1; w < kFoldWarps; ++w) acc += sum[w][lane];
  out[c] = a.accumulate ? out[c] + acc : acc;
}

bool wide(const void* p, int64_t ld, int es) {
  return p == nullptr ||
         ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * es)) & 15u) == 0;
}
int elem_bytes(int dtype) { return dtype == TIM_F32 ? 4 : 2; }
// Whether the operands that both directions take have rows of whole vectors.
bool wide(const tim_block& b) {
  const int es = elem_bytes(b.dtype);
  return b.d * es % 16 == 0 && wide(b.block, b.ld_block, es) && wide(b.gamma, 0, es) &&
         wide(b.gamma_post, 0, es) && (b.gate_kind != TIM_GATE_CHANNEL || wide(b.gate, 0, es)) &&
         (b.gate_kind != TIM_GATE_ELEMENT || wide(b.gate, b.ld_gate, es));
}

template <int kN>
using Int = std::integral_constant<int, kN>;

// f(vectors of a thread, threads a row), by the row's vectors alone.  Two vectors beyond 256: the gradient
// of rows of 4096 bf16 took 158 us so, 168 with one vector and twice the threads, 239 with four.  The
// update itself takes 170 us so for 32768 rows of 4096 bf16, 215 with one and 164 with four; for 16384 of 8192
// 217, 342 and 175; for 32768 of 2048, with one vector here, 102 and 86 with two.
template <int kDtype, class F>
cudaError_t with_split(int nvec, F&& f) {
  if (nvec <= 64) return f(Int<1>(), Int<64>());
  if (nvec <= 128) return f(Int<1>(), Int<128>());
  if (nvec <= 256) return f(Int<1>(), Int<256>());
  if (nvec <= 512) return f(Int<2>(), Int<256>());
  if (nvec <= 1024) return f(Int<2>(), Int<512>());
  if constexpr (kDtype == TIM_F32) {
    if (nvec > 2048) return f(Int<4>(), Int<1024>());
  }
  return f(Int<2>(), Int<1024>());
}
constexpr int kMaxParts = 1024;

template <int kDtype, bool kWide>
cudaError_t launch_forward(const NormArgs& a, cudaStream_t stream) {
  const int nvec = (a.b.d + Elem<kDtype>::kVec - 1) / Elem<kDtype>::kVec;
  return with_split<kDtype>(nvec, [&](auto vecs, auto threads) {
    residual_norm_kernel<kDtype, kWide, vecs.value, threads.value>
        <<<static_cast<unsigned>(a.b.T), threads.value, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

// Rows of a CTA in shared memory, beside what every row needs: two, so that two CTAs of 256 threads share
// an SM (three rows leave room for one: 277 us instead of 171); none where an SM's memory would not do.
template <int kVecs, int kThreads>
constexpr int kRowsAhead = kVecs * kThreads <= 1024 ? 2 : 0;

template <int kDtype, bool kWide>
cudaError_t launch_backward(const NormGradArgs& a, cudaStream_t stream, int num_sms) {
  const int nvec = (a.b.d + Elem<kDtype>::kVec - 1) / Elem<kDtype>::kVec;
  FoldArgs f = {};
  f.partial = a.partial;
  f.d = a.b.d;
  f.accumulate = a.accumulate;
  if (a.b.gamma != nullptr) f.out[0] = a.out_dgamma;
  if (a.b.gamma_post != nullptr) f.out[1] = a.out_dgamma_post;
  if (a.b.gate_kind == TIM_GATE_CHANNEL) f.out[2] = static_cast<float*>(a.out_dgate);
  const cudaError_t e = with_split<kDtype>(nvec, [&](auto vecs, auto threads) {
    constexpr int kVecs = vecs.value, kThreads = threads.value;
    constexpr int kStages = kWide ? kRowsAhead<kVecs, kThreads> : 0;
    constexpr size_t smem =
        kStages == 0 ? 0 : static_cast<size_t>(kStages * 4 + 3) * kVecs * kThreads * 16;
    auto launch = [&](auto channel) {
      auto* const kernel =
          residual_norm_backward_kernel<kDtype, kWide, kVecs, kThreads, kStages, channel.value>;
      static std::atomic<uint64_t> allowed{0};
      if (smem > 0) {
        const cudaError_t err = allow_smem(kernel, smem, allowed);
        if (err != cudaSuccess) return err;
      }
      const int64_t resident = static_cast<int64_t>(num_sms) * kResident<kVecs, kThreads>;
      f.parts = static_cast<int>(std::min<int64_t>(std::min<int64_t>(a.b.T, resident), kMaxParts));
      kernel<<<f.parts, kThreads, smem, stream>>>(a);
      return cudaGetLastError();
    };
    return a.b.gate_kind == TIM_GATE_CHANNEL ? launch(std::bool_constant<true>())
                                             : launch(std::bool_constant<false>());
  });
  if (e != cudaSuccess) return e;
  if (f.out[0] == nullptr && f.out[1] == nullptr && f.out[2] == nullptr) return e;
  residual_fold_kernel<<<dim3((a.b.d + 31) / 32, 3), 32 * kFoldWarps, 0, stream>>>(f);
  return cudaGetLastError();
}

// f(type, whether rows are whole vectors)
template <class F>
cudaError_t by_type(int dtype, bool w, F&& f) {
  using Yes = std::bool_constant<true>;
  using No = std::bool_constant<false>;
  if (dtype == TIM_F32) return w ? f(Int<TIM_F32>(), Yes()) : f(Int<TIM_F32>(), No());
  if (dtype == TIM_BF16) return w ? f(Int<TIM_BF16>(), Yes()) : f(Int<TIM_BF16>(), No());
  return w ? f(Int<TIM_F16>(), Yes()) : f(Int<TIM_F16>(), No());
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs& a, cudaStream_t stream) {
  const int es = elem_bytes(a.b.dtype);
  const bool w = wide(a.b) && wide(a.residual, a.ld_residual, es) && wide(a.out_h, a.ld_h, es) &&
                 wide(a.out_y, a.ld_y, es);
  return by_type(a.b.dtype, w, [&](auto type, auto is_wide) {
    return launch_forward<type.value, is_wide.value>(a, stream);
  });
}

size_t residual_norm_backward_bytes(int64_t T, int d) {
  return align_up(1024 + static_cast<size_t>(std::min<int64_t>(T, kMaxParts)) * 3 *
                             static_cast<size_t>(d) * 4,
                  1024);
}

cudaError_t launch_residual_norm_backward(const NormGradArgs& a, cudaStream_t stream, int num_sms) {
  const int es = elem_bytes(a.b.dtype);
  const bool w = wide(a.b) && wide(a.h, a.ld_h, es) && wide(a.dh, a.ld_dh, es) &&
                 wide(a.dy, a.ld_dy, es) && wide(a.out_dresidual, a.ld_dresidual, es) &&
                 wide(a.out_dblock, a.ld_dblock, es) &&
                 (a.b.gate_kind != TIM_GATE_ELEMENT || wide(a.out_dgate, a.ld_dgate, es));
  return by_type(a.b.dtype, w, [&](auto type, auto is_wide) {
    return launch_backward<type.value, is_wide.value>(a, stream, num_sms);
  });
}

}  // namespace tim
