// The tokens of a batch in the order of their ids, equal ids in the order of their rows: a radix sort in one
// launch, by a cluster of CTAs that keep all of it in their shared memory.  The other clusters of
// the launch, if there are any, zero the table's gradient meanwhile.  More tokens than a cluster holds are
// sorted in runs, a cluster each, and the runs merged two by two, a launch a round: a token's place
// is its own in its run and, by a binary search, how many of the other run go before it.
//
// A pass orders by 9 bits of the id, lowest first.  Every warp has 32 kItems tokens that follow one
// another in the list and counts its digits, equal ones of a step ranked by lane; the counts of a
// digit's earlier warps, then of its earlier CTAs (whose totals are exchanged), then of all lower
// digits give each token its place, and it is stored there, in whichever CTA that is.  V = 151936
// takes two passes, three cluster barriers.
#pragma once

#include <algorithm>

#include "logits_row.cuh"

namespace tim {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;
constexpr int kSortItems = 16;  // of a thread, at most
constexpr int kSortRows = kSortCluster * kSortThreads * kSortItems;
constexpr int kDigitBits = 9;
constexpr int64_t kZeroChunk = 65536;  // bytes zeroed by a CTA at least
constexpr int kDigits = 1 << kDigitBits;

struct SortArgs {
  const int32_t* ids;
  int T, V, passes;
  uint32_t size;  // CTAs of a cluster
  uint32_t runs;  // of kSortRows tokens but for the last, a cluster each
  uint32_t* out_id;  // V: no token
  uint32_t* out_row;
  int* status;
  uint8_t* zero;  // zero_bytes of it become 0, by the clusters behind the runs'
  int64_t zero_bytes;
};

// Bytes [a, b) of the zeroed memory, by a CTA.
__device__ __forceinline__ void zero_range(uint8_t* p, int64_t a, int64_t b) {
  const int64_t whole = (b - a) / 16;
  uint4* const v = reinterpret_cast<uint4*>(p + a);
  for (int64_t i = threadIdx.x; i < whole; i += blockDim.x) v[i] = make_uint4(0u, 0u, 0u, 0u);
  const int64_t rest = a + whole * 16 + threadIdx.x;
  if (rest < b) p[rest] = 0;
}
// Element-aligned memory: its first bytes up to a 16-byte boundary, and what follows in chunks that go
// round among the CTAs: of 1 MB where every CTA has one, 1.24 GB take 187 us so, 201 in chunks of 64 KB
// and 210 in one share each; of 64 KB for less memory, 64 MB take 13 us so and 20 in chunks of 1 MB.
__device__ __forceinline__ void zero_share(uint8_t* p, int64_t bytes, int part, int parts) {
  const int64_t head = min(bytes, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u));
  if (part == 0 && static_cast<int64_t>(threadIdx.x) < head) p[threadIdx.x] = 0;
  p += head;
  bytes -= head;
  const int64_t chunk = bytes >= parts * 16 * kZeroChunk ? 16 * kZeroChunk : kZeroChunk;
  for (int64_t a = part * chunk; a < bytes; a += parts * chunk)
    zero_range(p, a, min(bytes, a + chunk));
}

template <int kItems>
struct SortShared {
  uint64_t item[kSortThreads * kItems];  // id << 32 | row
  uint32_t total[kSortCluster][kDigits];
  uint32_t base[kDigits];
  uint32_t warp[kDigits / 32];
  uint16_t count[kSortWarps][kDigits];
};

template <int kItems>
__global__ void __launch_bounds__(kSortThreads, kItems <= 4 ? 2 : 1) embed_sort_kernel(const SortArgs a) {
  extern __shared__ uint4 sort_mem[];
  SortShared<kItems>& sh = *reinterpret_cast<SortShared<kItems>*>(sort_mem);
  constexpr int kOfCta = kSortThreads * kItems;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), size = a.size;
  const uint32_t run = blockIdx.x / size;
  if (run >= a.runs) {
    zero_share(a.zero, a.zero_bytes, blockIdx.x - a.runs * size, gridDim.x - a.runs * size);
    return;
  }
  const uint32_t t0 = run * kSortRows;
  const uint32_t T = min(static_cast<uint32_t>(a.T) - t0, static_cast<uint32_t>(kSortRows));
  const uint32_t first = warp * 32 * kItems + lane;        // of the CTA's tokens
  uint32_t id[kItems], row[kItems], place[kItems];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    row[k] = rank * kOfCta + first + k * 32;
    id[k] = static_cast<uint32_t>(a.V);  // none, and beyond the end: last, in order
    if (row[k] < T) {
      const int t = __ldg(a.ids + t0 + row[k]);
      bad |= t < -1 || t >= a.V;
      if (t >= 0 && t < a.V) id[k] = static_cast<uint32_t>(t);
    }
  }
  if (bad) set_status(a.status, TIM_ERR_TOKEN_RANGE);
  cluster_arrive();
  cluster_wait();  // every CTA of the cluster runs
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * kDigitBits;
    if (pass > 0) {
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const uint64_t x = sh.item[first + k * 32];
        id[k] = static_cast<uint32_t>(x >> 32);
        row[k] = static_cast<uint32_t>(x);
      }
    }
    uint16_t* const mine = sh.count[warp];
    for (int i = lane; i < kDigits / 2; i += 32) reinterpret_cast<uint32_t*>(mine)[i] = 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const uint32_t digit = (id[k] >> shift) & (kDigits - 1);
      const unsigned same = __match_any_sync(0xFFFFFFFFu, digit);
      const uint32_t before = mine[digit];
      place[k] = before + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if ((same >> lane) == 1u) mine[digit] = static_cast<uint16_t>(before + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    if (tid < kDigits) {  // over the warps
      uint32_t n = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t x = sh.count[w][tid];
        sh.count[w][tid] = static_cast<uint16_t>(n);
        n += x;
      }
      for (uint32_t c = 0; c < size; ++c) cluster_store32(cluster_addr(&sh.total[rank][tid], c), n);
    }
    cluster_arrive();
    cluster_wait();
    uint32_t before = 0, all = 0, at = 0;
    if (tid < kDigits) {
      for (uint32_t c = 0; c < size; ++c) {
        const uint32_t n = sh.total[c][tid];
        if (c < rank) before += n;
        all += n;
      }
      at = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, at, o);
        if (lane >= o) at += up;
      }
      if (lane == 31) sh.warp[warp] = at;
    }
    __syncthreads();
    if (tid < kDigits) {
      for (int w = 0; w < warp; ++w) before += sh.warp[w];
      sh.base[tid] = before + at - all;
    }
    __syncthreads();
    const bool last = pass + 1 == a.passes;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const uint32_t digit = (id[k] >> shift) & (kDigits - 1);
      const uint32_t to = sh.base[digit] + mine[digit] + place[k];
      if (last) {
        if (to < T) {
          a.out_id[t0 + to] = id[k];
          a.out_row[t0 + to] = t0 + row[k];
        }
      } else {
        cluster_store(cluster_addr(&sh.item[to % kOfCta], to / kOfCta),
                      static_cast<uint64_t>(id[k]) << 32 | row[k]);
      }
    }
    if (!last) {
      cluster_arrive();
      cluster_wait();
    }
  }
}

// Of two neighbouring runs of `len` one that is twice as long (a last run may be shorter, or alone).  Equal
// ids of the first go before those of the second, so that rows stay in order.
constexpr int kMergeThreads = 256;
__global__ void __launch_bounds__(kMergeThreads)
    embed_merge_kernel(const uint32_t* id, const uint32_t* row, uint32_t T, uint32_t len,
                       uint32_t* out_id, uint32_t* out_row) {
  const uint32_t i = blockIdx.x * kMergeThreads + threadIdx.x;  // T < 2^31
  if (i >= T) return;
  const uint32_t first = i / len * len, a = (i / len & 1u) != 0 ? first - len : first;  // a + 2 len < 2^32
  const uint32_t b = min(a + len, T), end = min(b + len, T);
  const uint32_t v = __ldg(id + i);
  const bool second = i >= b;
  uint32_t lo = second ? a : b, hi = second ? b : end;
  const uint32_t from = lo;
  while (lo < hi) {  // the first of the other run that does not go before
    const uint32_t mid = lo + (hi - lo) / 2, x = __ldg(id + mid);
    if (second ? x <= v : x < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  const uint32_t to = (second ? i - len : i) + (lo - from);
  out_id[to] = v;
  out_row[to] = __ldg(row + i);
}

template <int kItems>
cudaError_t launch_sort(const SortArgs& a, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(embed_sort_kernel<kItems>, sizeof(SortShared<kItems>), allowed);
  if (e != cudaSuccess) return e;
  // as many CTAs as an SM's threads take twice over, or as there are chunks
  const int64_t chunks = (a.zero_bytes + kZeroChunk - 1) / kZeroChunk;
  const int64_t others = std::min<int64_t>((chunks + a.size - 1) / a.size, 2 * num_sms / a.size);
  return launch_clusters(embed_sort_kernel<kItems>, a.runs + others, static_cast<int>(a.size),
                         kSortThreads, sizeof(SortShared<kItems>), stream, a);
}

// The ids of T tokens in order, and their rows, in sorted[0] (sorted[1]: as much memory again, for more
// than kSortRows); ids that are none, or out of range (noted in the status word), as V at the end.
struct Sorted {
  uint32_t *id, *row;
};
cudaError_t launch_embed_sort(const int32_t* ids, int T, int V, const Sorted (&sorted)[2], int* status,
                              void* zero, int64_t zero_bytes, int num_sms, cudaStream_t stream) {
  int bits = 1;
  while (bits < 32 && (static_cast<uint32_t>(V) >> bits) != 0) ++bits;
  SortArgs a = {};
  a.ids = ids;
  a.T = T;
  a.V = V;
  a.passes = (bits + kDigitBits - 1) / kDigitBits;
  a.size = 1;
  while (a.size < kSortCluster && a.size * kSortThreads * 4 < static_cast<uint32_t>(T)) a.size *= 2;
  a.runs = (static_cast<uint32_t>(T) + kSortRows - 1) / kSortRows;
  int rounds = 0;
  while ((1u << rounds) < a.runs) ++rounds;
  int at = rounds & 1;  // so that the last round ends in sorted[0]
  a.out_id = sorted[at].id;
  a.out_row = sorted[at].row;
  a.status = status;
  a.zero = static_cast<uint8_t*>(zero);
  a.zero_bytes = zero_bytes;
  cudaError_t e = a.size * kSortThreads * 4 >= static_cast<uint32_t>(T)
                      ? launch_sort<4>(a, num_sms, stream)
                      : launch_sort<kSortItems>(a, num_sms, stream);
  for (int r = 0; r < rounds && e == cudaSuccess; ++r, at ^= 1) {
    embed_merge_kernel<<<(static_cast<unsigned>(T) + kMergeThreads - 1) / kMergeThreads, kMergeThreads, 0,
                         stream>>>(sorted[at].id, sorted[at].row, static_cast<uint32_t>(T),
                                   static_cast<uint32_t>(kSortRows) << r, sorted[at ^ 1].id,
                                   sorted[at ^ 1].row);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace
}  // namespace tim
