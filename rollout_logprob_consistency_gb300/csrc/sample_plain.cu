// Few unfiltered rows: a cluster of CTAs holds a row in shared memory, a slice each, and finds the
// token by running sums of integer weights.  One row of 151936 logits takes 14 us, most of it the
// launch and the two exchanges; a CTA alone takes 29 for 8 such rows (sample.cu, which says from
// where on that is the better way).
//
// A thread's largest logit gives the scale: the sum over the threads of (largest weight x
// elements) bounds the row's total, and is at most that many times too large.
#include "sample.cuh"

namespace tim {

using namespace sampling;

namespace {

constexpr int kMaxCluster = 8;
constexpr int kMaxSteps = 64;  // 32-vector steps of a warp's part: at most 24580 vectors over 16 warps

struct PlainArgs : SampleArgs {
  int cluster;
};

template <int kThreads>
struct Shared {
  Tables table;
  u64 xch[kMaxCluster][2];  // every CTA's sum and count
  // of every warp of every CTA: largest key, and the threads' largest weights relative to it
  uint32_t gkey[kMaxCluster * kThreads / 32];
  float gsum[kMaxCluster * kThreads / 32];
  u64 warp[kThreads / 32];
  uint32_t warpu[kThreads / 32];
  u64 step[kMaxSteps];  // sums over 32 vectors each, of one warp's part
  int found;
  uint64_t bar;
};

template <int kDtype, int kThreads>
struct Sampler {
  using E = Elem<kDtype>;
  static constexpr int kVec = E::kVec;
  static constexpr int kWarps = kThreads / 32;

  const PlainArgs& a;
  Shared<kThreads>& sh;
  const uint4* slice;
  Row<kDtype> r;
  Slice s;
  int rank, tid, warp, lane;
  RowState st;

  // id of slot i of the slice's vector j
  __device__ __forceinline__ int id_of(int j, int i) const { return (s.j0 + j) * kVec + i - r.shift; }

  // ---- sums over the slice.  A warp has a contiguous part of it, in steps of 32 vectors.
  __device__ __forceinline__ int part_steps() const { return (s.n + kThreads - 1) / kThreads; }
  __device__ __forceinline__ int part_start(int w) const { return w * part_steps() * 32; }

  // The sum of f(v, id0) over the slice's vectors; sh.warp[] gets the parts' sums.
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

  // Sum of weights, without recentring.
  __device__ __forceinline__ u64 weights_of(const float (&v)[kVec], uint32_t shift) const {
    u64 t = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) t += weight_at(v[i], st.pw.kh, st.pw.kl, shift, sh.table.t);
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
    if (warp == 0 && lane < a.cluster) {  // to every CTA of the row
      cluster_store(cluster_addr(&sh.xch[rank][0], lane), mine);
      cluster_store(cluster_addr(&sh.xch[rank][1], lane), cta_n);
    }
    cluster_arrive();
    cluster_wait();
    u64 total = 0, all = 0, before = 0;
    for (int c = 0; c < a.cluster; ++c) {
      if (c < rank) before += sh.xch[c][0];
      total += sh.xch[c][0];
      all += sh.xch[c][1];
    }
    const u64 target = draw_target(total, u);
    if (before <= target && target < before + mine) {  // one CTA of the row
      const int id = locate(target - before, f, one);
      if (tid == 0) write_row(a, st, sh.table, row, id, r.at(id), total, static_cast<int>(all));
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
      const uint32_t shift = shift_of(st.top);
      draw(row, u, n, [&](const float(&v)[kVec], int) { return weights_of(v, shift); }, one);
    }
  }
};

template <int kDtype, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 2)
    sample_plain_kernel(const PlainArgs a) {
  using E = Elem<kDtype>;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint4 slice_mem[];
  __shared__ Shared<kThreads> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int64_t row = blockIdx.x / a.cluster;

  cluster_arrive();
  const Row<kDtype> r(a.logits, row, a.ld, a.V);
  const Slice s = slice_of(r.nvec(), rank, a.cluster);
  if (tid == 0) {
    mbar_init(&sh.bar, 1);
    fence_mbarrier_init();
    load_slice(r, s, slice_mem, &sh.bar);
  }
  load_slice_edges(r, s, slice_mem);
  load_tables(sh.table, tid, kThreads);
  const Settings set = settings_of(a, row);
  int bad = set.bad;
  Sampler<kDtype, kThreads> S{a, sh, slice_mem, r, s, rank, tid, warp, lane, {}};
  RowState& st = S.st;
  set_temperature(st, set.tau);
  const int never = 0;
  __syncthreads();
  cluster_wait();  // every CTA of the cluster runs
  const bool late = !mbar_wait(&sh.bar, 0, &never);  // then the row is refused, by all its CTAs
  if (late) set_status(a.status, TIM_ERR_TIMEOUT);

  // ---- the largest logit of each thread; of each warp, to every CTA of the row
  float tmax = -INFINITY;
  if (tid < s.n) {
    uint4 m = slice_mem[tid];
#pragma unroll 4
    for (int j = tid + kThreads; j < s.n; j += kThreads) m = max_vec<kDtype>(m, slice_mem[j]);
    tmax = max_of<kDtype>(m);
  }
  const uint32_t mykey = late || !(tmax < INFINITY) ? 0xFFFFFFFFu : key_of(tmax);
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
    S.plain(row, set.u);
  }
  cluster_arrive();  // no CTA leaves while another may still write to it
  cluster_wait();
  if (late) mbar_wait(&sh.bar, 0, &never);  // nor with its copy on the way
}

template <int kDtype, int kThreads>
cudaError_t launch_rows(PlainArgs a, int64_t T, const RowPlan& p, cudaStream_t stream) {
  auto* kernel = sample_plain_kernel<kDtype, kThreads>;
  static std::atomic<uint64_t> allowed{0};
  const RowPlan largest = plan_row(TIM_LOGITS_MAX_V, sizeof(typename Elem<kDtype>::raw));
  const cudaError_t e = allow_smem(kernel, largest.slice_bytes, allowed);
  if (e != cudaSuccess) return e;
  a.cluster = p.cluster;
  return launch_clusters(kernel, T, p.cluster, kThreads, p.slice_bytes, stream, a);
}
template <int kDtype>
cudaError_t launch_type(const PlainArgs& a, int64_t T, cudaStream_t stream) {
  const RowPlan p = plan_row(a.V, sizeof(typename Elem<kDtype>::raw));
  return p.threads == 256 ? launch_rows<kDtype, 256>(a, T, p, stream)
                          : launch_rows<kDtype, 512>(a, T, p, stream);
}

}  // namespace

cudaError_t launch_sample_plain(const SampleArgs& args, int dtype, int64_t T, cudaStream_t stream) {
  PlainArgs a;
  static_cast<SampleArgs&>(a) = args;
  a.cluster = 1;
  return dtype == TIM_F32    ? launch_type<TIM_F32>(a, T, stream)
         : dtype == TIM_BF16 ? launch_type<TIM_BF16>(a, T, stream)
                             : launch_type<TIM_F16>(a, T, stream);
}

}  // namespace tim
