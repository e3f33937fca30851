// Embedding lookup with a scale, and its gradient by sorted tokens.
//
//   out[t] = scale table[ids[t]]                      (fp32 product, one rounding)
//   dtable[v] (+)= scale sum_{t: ids[t] = v} dy[t]    (fp32 sums in a fixed order, one rounding)
//
// The lookup is memory's: distinct rows read, T rows written.
//
// The gradient is a sum over equal tokens, so the tokens are sorted first (embed_sort.cuh's one
// launch for up to 131072 of them: the order of equal ids is their order in the batch), and the sorted
// list is cut into pieces of a fixed number of rows.  A piece's CTA walks its rows with a column vector a
// thread and an fp32 running sum, writes the tokens that lie wholly within, and leaves the sums of the
// first and the last where they go on beyond it; a second launch joins those in order.  No atomics: the
// same call gives the same bits.  The table's gradient is zeroed by the rest of the sort's launch, which
// has eight SMs' work otherwise; with `accumulate` it is added to.
//
// 32768 tokens of 4096 bf16 into 151936 rows take 187 to 196 us for sort and zeros (1.24 GB, 6.4 to
// 6.6 TB/s; the sort alone 18), 61 for the pieces and 9 for the joins.  Zeroing only the rows without a token, in
// the launch of the pieces, took 302 + 18 + 11.
#include "embed_sort.cuh"
#include <type_traits>

#include "logits_row.cuh"

namespace tim {
namespace {

// ---- the lookup

// 32768 tokens of 4096 bf16 from 151936 rows, 14400 of them distinct, take 63 us, 6.1 TB/s with every distinct
// row counted once; 8 vectors a thread, 64 or 256 threads and streaming stores take 62 to 66.
constexpr int kLookupThreads = 128;
constexpr int kLookupVecs = 4;  // of a thread, in flight together

struct LookupArgs {
  const void* table;
  int64_t ld;
  const int32_t* ids;
  int V, d;
  float scale;
  void* out;
  int64_t ldo;
  int* status;
};

// kWide: rows of whole 16-byte vectors at both sides; else an element a load (32768 tokens of 4096 bf16, any of
// 151936, take 84 us and, in rows of 4099, 146).
template <int kDtype, bool kWide>
__global__ void __launch_bounds__(kLookupThreads) embed_kernel(const LookupArgs a) {
  using E = Elem<kDtype>;
  using raw = typename E::raw;
  constexpr int kOf = kWide ? E::kVec : 1;
  const int64_t row = blockIdx.x;
  const int id = __ldg(a.ids + row);
  const bool bad = id < -1 || id >= a.V;
  if (bad && threadIdx.x == 0 && blockIdx.y == 0) set_status(a.status, TIM_ERR_TOKEN_RANGE);
  raw* const out = static_cast<raw*>(a.out) + row * a.ldo;
  const raw* const from = static_cast<const raw*>(a.table) + (id >= 0 && !bad ? id : 0) * a.ld;
  const int n = a.d / kOf;  // whole where kWide
  for (int c0 = blockIdx.y * kLookupThreads * kLookupVecs + threadIdx.x; c0 < n;
       c0 += gridDim.y * kLookupThreads * kLookupVecs) {
    if (bad || id < 0) {
      const raw fill = E::narrow(bad ? __int_as_float(0x7FC00000) : 0.f);
#pragma unroll
      for (int k = 0; k < kLookupVecs; ++k) {
        const int c = c0 + k * kLookupThreads;
        if (c < n)
          for (int i = 0; i < kOf; ++i) out[c * kOf + i] = fill;
      }
      continue;
    }
    if constexpr (kWide) {
      uint4 x[kLookupVecs];
#pragma unroll
      for (int k = 0; k < kLookupVecs; ++k) {
        const int c = c0 + k * kLookupThreads;
        if (c < n) x[k] = __ldg(reinterpret_cast<const uint4*>(from) + c);
      }
#pragma unroll
      for (int k = 0; k < kLookupVecs; ++k) {
        const int c = c0 + k * kLookupThreads;
        if (c >= n) continue;
        float v[E::kVec];
        E::unpack(x[k], v);
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) v[i] *= a.scale;
        reinterpret_cast<uint4*>(out)[c] = E::pack(v);
      }
    } else {
      raw x[kLookupVecs];
#pragma unroll
      for (int k = 0; k < kLookupVecs; ++k) {
        const int c = c0 + k * kLookupThreads;
        if (c < n) x[k] = from[c];
      }
#pragma unroll
      for (int k = 0; k < kLookupVecs; ++k) {
        const int c = c0 + k * kLookupThreads;
        if (c < n) out[c] = E::narrow(E::widen(x[k]) * a.scale);
      }
    }
  }
}

bool wide(const void* p, int64_t ld, int d, int es) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * es) |
           static_cast<uintptr_t>(static_cast<int64_t>(d) * es)) & 15u) == 0;
}

template <int kDtype>
cudaError_t launch_lookup(const LookupArgs& a, int64_t T, cudaStream_t stream) {
  constexpr int es = sizeof(typename Elem<kDtype>::raw);
  const bool w = wide(a.table, a.ld, a.d, es) && wide(a.out, a.ldo, a.d, es);
  const int n = w ? a.d / Elem<kDtype>::kVec : a.d;
  const int per = kLookupThreads * kLookupVecs;
  const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>(std::min((n + per - 1) / per, 64)));
  if (w)
    embed_kernel<kDtype, true><<<grid, kLookupThreads, 0, stream>>>(a);
  else
    embed_kernel<kDtype, false><<<grid, kLookupThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// ---- the gradient

constexpr int kGradThreads = 256;
constexpr int kRows = 8;       // rows in flight
constexpr int kMaxPiece = 64;  // rows of a piece, or of a step of a long one
// Of a batch, whose first and last tokens' sums are kept.  131073 tokens of 2048 bf16, any of 151936, take
// 273 us so and 285 with half as many; a frequent token's pieces are joined by one CTA, so that 262144 tokens of
// which a seventh are alike take 571 us so and 464 with half as many.
constexpr int kMaxPieces = 2 * kSortRows / kMaxPiece;

constexpr uint32_t kNoId = 0xFFFFFFFFu;  // no token's, nor V

struct GradArgs {
  const void* dy;
  int64_t ld;
  const uint32_t* id;   // sorted; V: none
  const uint32_t* row;  // the rows in that order
  int T, V, d, piece, pieces, slices;
  float scale;
  void* out;
  int accumulate;
  float* partial;  // [pieces][2][d]: of a piece's first and last token
};

// kVec columns of a row as they lie in memory: a 16-byte vector where rows are whole vectors, else one (32768
// tokens of 4096 bf16 into 151936 bf16 rows 295 us and, from rows of 4099, 379).
template <int kDtype, int kVec>
struct Loaded {
  using E = Elem<kDtype>;
  std::conditional_t<kVec == 1, typename E::raw, uint4> x;
  __device__ __forceinline__ void load(const typename E::raw* p) {
    x = __ldg(reinterpret_cast<const decltype(x)*>(p));
  }
  __device__ __forceinline__ void add_to(float (&acc)[kVec]) const {
    if constexpr (kVec == 1) {
      acc[0] += E::widen(x);
    } else {
      float v[kVec];
      E::unpack(x, v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] += v[i];
    }
  }
};
// kVec columns of the table's gradient, of type kOut.
template <int kOut, int kVec>
__device__ __forceinline__ void store_cols(typename Elem<kOut>::raw* p, const float (&acc)[kVec],
                                           float scale, int accumulate) {
  using E = Elem<kOut>;
  if constexpr (kVec == 1) {
    p[0] = E::narrow(accumulate ? fmaf(acc[0], scale, E::widen(p[0])) : acc[0] * scale);
  } else {
#pragma unroll
    for (int q = 0; q < kVec; q += E::kVec) {
      uint4* const at = reinterpret_cast<uint4*>(p + q);
      float v[E::kVec];
      if (accumulate) {
        E::unpack(*at, v);
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) v[i] = fmaf(acc[q + i], scale, v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) v[i] = acc[q + i] * scale;
      }
      *at = E::pack(v);
    }
  }
}

// kLong: pieces of more than kMaxPiece rows, taken in steps of as many.
template <int kDtype, int kOut, int kVec, bool kLong>
__global__ void __launch_bounds__(kGradThreads, kLong ? 3 : 4) embed_grad_kernel(const GradArgs a) {
  using raw = typename Elem<kDtype>::raw;
  using raw_out = typename Elem<kOut>::raw;
  __shared__ uint32_t ids[kMaxPiece + 2], rows[kMaxPiece];
  const int tid = threadIdx.x, n = a.d / kVec;
  const uint32_t none = static_cast<uint32_t>(a.V);
  // a piece of the sorted list, a slice of the columns
  const int p = blockIdx.x / a.slices, c = (blockIdx.x % a.slices) * kGradThreads + tid;
  const int end = min(a.piece, a.T - p * a.piece) + p * a.piece;
  const raw* const dy = static_cast<const raw*>(a.dy) + c * kVec;
  float acc[kVec] = {};
  uint32_t cur = 0, before = 0;
  bool first = true;
  auto flush = [&](uint32_t next) {  // next: the id behind the piece, or none's
    if (cur >= none) return;
    const bool from_before = first && before == cur, goes_on = next == cur;
    if (from_before || goes_on) {
      float* const to =
          a.partial + (static_cast<int64_t>(p) * 2 + (from_before ? 0 : 1)) * a.d + c * kVec;
#pragma unroll
      for (int i = 0; i < kVec; ++i) to[i] = acc[i];
    } else {
      store_cols<kOut, kVec>(static_cast<raw_out*>(a.out) + static_cast<int64_t>(cur) * a.d + c * kVec,
                             acc, a.scale, a.accumulate);
    }
  };
  auto walk = [&](int len) {
    for (int r0 = 0; r0 < len; r0 += kRows) {
      if (ids[1 + r0] >= none) {  // only such follow
        flush(kNoId);
        cur = none;
        return;
      }
      Loaded<kDtype, kVec> v[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (r0 + k < len && ids[1 + r0 + k] < none)
          v[k].load(dy + static_cast<int64_t>(rows[r0 + k]) * a.ld);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (r0 + k >= len) break;
        const uint32_t id = ids[1 + r0 + k];
        if (id != cur) {
          flush(kNoId);
          cur = id;
          first = false;
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
        }
        if (id >= none) return;
        v[k].add_to(acc);
      }
    }
  };
  for (int i0 = p * a.piece;;) {
    const int len = kLong ? min(kMaxPiece, end - i0) : end - i0;
    for (int i = tid; i < len + 2; i += kGradThreads) {
      const int at = i0 - 1 + i;
      ids[i] = at >= 0 && at < a.T ? __ldg(a.id + at) : kNoId;
      if (i < len) rows[i] = __ldg(a.row + i0 + i);
    }
    __syncthreads();
    if (!kLong && c >= n) return;
    if (!kLong || i0 == p * a.piece) {
      before = ids[0];
      cur = ids[1];
    }
    if (!kLong || c < n) walk(len);
    i0 += len;
    if (!kLong || i0 == end || ids[len] >= none) {  // cur is none's in the last of these
      if (!kLong || c < n) flush(ids[len + 1]);
      return;
    }
    __syncthreads();  // every thread has read this step's
  }
}

// The tokens whose rows lie in several pieces: the CTA of the piece where one begins adds its parts.
template <int kOut, int kVec>
__global__ void __launch_bounds__(kGradThreads) embed_join_kernel(const GradArgs a) {
  using raw_out = typename Elem<kOut>::raw;
  const int p = blockIdx.x / a.slices, c = (blockIdx.x % a.slices) * kGradThreads + threadIdx.x;
  const int i0 = p * a.piece;
  if (a.T - i0 <= a.piece) return;  // all but the last piece are whole
  const int i1 = i0 + a.piece;
  const uint32_t id = __ldg(a.id + i1 - 1), next = __ldg(a.id + i1);
  const uint32_t before = i0 > 0 ? __ldg(a.id + i0 - 1) : kNoId;
  if (id >= static_cast<uint32_t>(a.V) || next != id || before == id) return;  // or begins earlier
  if (c >= a.d / kVec) return;
  float acc[kVec];
  const float* const part = a.partial + c * kVec;
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = part[(static_cast<int64_t>(p) * 2 + 1) * a.d + i];
  for (int q = p + 1; q < a.pieces; q += kRows) {
    float v[kRows][kVec];
    bool in[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      in[k] = q + k < a.pieces && __ldg(a.id + static_cast<int64_t>(q + k) * a.piece) == id;
      if (in[k]) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[k][i] = part[static_cast<int64_t>(q + k) * 2 * a.d + i];
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (!in[k]) break;
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] += v[k][i];
    }
    if (!in[kRows - 1]) break;
  }
  store_cols<kOut, kVec>(static_cast<raw_out*>(a.out) + static_cast<int64_t>(id) * a.d + c * kVec, acc,
                         a.scale, a.accumulate);
}

template <int kDtype, int kOut, int kVec>
cudaError_t launch_grad(const GradArgs& args, cudaStream_t stream) {
  GradArgs a = args;
  a.slices = (a.d / kVec + kGradThreads - 1) / kGradThreads;
  const int64_t work = static_cast<int64_t>(a.pieces) * a.slices;
  auto* const kernel = a.piece > kMaxPiece ? embed_grad_kernel<kDtype, kOut, kVec, true>
                                           : embed_grad_kernel<kDtype, kOut, kVec, false>;
  kernel<<<static_cast<unsigned>(work), kGradThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.pieces == 1) return e;
  embed_join_kernel<kOut, kVec><<<static_cast<unsigned>(work), kGradThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <int kDtype>
cudaError_t launch_grad_type(const GradArgs& a, int out_dtype, cudaStream_t stream) {
  constexpr int es = sizeof(typename Elem<kDtype>::raw), kVec = Elem<kDtype>::kVec;
  const int eo = out_dtype == TIM_F32 ? 4 : 2;
  const bool w = wide(a.dy, a.ld, a.d, es) && wide(a.out, a.d, a.d, eo);
  if (out_dtype == TIM_F32)
    return w ? launch_grad<kDtype, TIM_F32, kVec>(a, stream)
             : launch_grad<kDtype, TIM_F32, 1>(a, stream);
  if constexpr (kDtype != TIM_F32) {
    if (out_dtype == kDtype)
      return w ? launch_grad<kDtype, kDtype, kVec>(a, stream)
               : launch_grad<kDtype, kDtype, 1>(a, stream);
  }
  return cudaErrorInvalidValue;
}

// Rows of a piece: few where there are few, for the SMs' sake, and so many that kMaxPieces pieces do.  With 16
// and with 64 rows, tokens of 4096 bf16, any of 32003, added to fp32: 1000 tokens take 36 us and 62, 4096 60
// and 82, 8192 86 and 94 (99 and 92 where a sixth are alike, by its joins), 16384 131 and 127 (162 and 119).
int piece_rows(int64_t T) {
  if (T <= 8192) return 16;
  const int64_t steps = (T + kMaxPiece - 1) / kMaxPiece;
  return static_cast<int>((steps + kMaxPieces - 1) / kMaxPieces) * kMaxPiece;
}

struct EmbedWs {
  size_t sorted_off[2], list, partial_off, total;  // a list: ids, then rows
};
EmbedWs embed_ws(int64_t T, int d) {
  const size_t n = static_cast<size_t>(T);
  EmbedWs w;
  w.list = align_up(n * 4, 1024);
  w.sorted_off[0] = 1024;
  w.sorted_off[1] = w.sorted_off[0] + 2 * w.list;
  w.partial_off = w.sorted_off[1] + (T > kSortRows ? 2 * w.list : 0);
  // fewer tokens than n can have more pieces (a smaller call with this workspace)
  const size_t small = (std::min<size_t>(n, 8192) + 15) / 16;
  const size_t large = std::min<size_t>((n + kMaxPiece - 1) / kMaxPiece, kMaxPieces);
  w.total = align_up(w.partial_off + std::max(small, large) * 2 * static_cast<size_t>(d) * 4, 1024);
  return w;
}

}  // namespace

cudaError_t launch_embed(const void* table, int dtype, int64_t ld, const int32_t* ids, int64_t T,
                         int V, int d, float scale, void* out, int64_t ldo, int* status,
                         cudaStream_t stream) {
  const LookupArgs a = {table, ld, ids, V, d, scale, out, ldo, status};
  return dtype == TIM_F32    ? launch_lookup<TIM_F32>(a, T, stream)
         : dtype == TIM_BF16 ? launch_lookup<TIM_BF16>(a, T, stream)
                             : launch_lookup<TIM_F16>(a, T, stream);
}

size_t embed_backward_bytes(int64_t T, int d) { return embed_ws(T, d).total; }

cudaError_t launch_embed_backward(const void* dy, int dtype, int64_t ld, const int32_t* ids, int64_t T,
                                  int V, int d, float scale, void* out, int out_dtype, int accumulate,
                                  void* ws, cudaStream_t stream, int num_sms) {
  const EmbedWs w = embed_ws(T, d);
  uint8_t* const b = static_cast<uint8_t*>(ws);
  Sorted sorted[2];
  for (int i = 0; i < 2; ++i) {
    sorted[i].id = reinterpret_cast<uint32_t*>(b + w.sorted_off[i]);
    sorted[i].row = reinterpret_cast<uint32_t*>(b + w.sorted_off[i] + w.list);
  }
  GradArgs a = {};
  a.dy = dy;
  a.ld = ld;
  a.id = sorted[0].id;
  a.row = sorted[0].row;
  a.T = static_cast<int>(T);
  a.V = V;
  a.d = d;
  a.piece = piece_rows(T);
  a.pieces = static_cast<int>((T + a.piece - 1) / a.piece);
  a.scale = scale;
  a.out = out;
  a.accumulate = accumulate;
  a.partial = reinterpret_cast<float*>(b + w.partial_off);
  const int64_t table = static_cast<int64_t>(V) * d * (out_dtype == TIM_F32 ? 4 : 2);
  const cudaError_t e = launch_embed_sort(ids, a.T, V, sorted, static_cast<int*>(ws), out,
                                          accumulate ? 0 : table, num_sms, stream);
  if (e != cudaSuccess) return e;
  return dtype == TIM_F32    ? launch_grad_type<TIM_F32>(a, out_dtype, stream)
         : dtype == TIM_BF16 ? launch_grad_type<TIM_BF16>(a, out_dtype, stream)
                             : launch_grad_type<TIM_F16>(a, out_dtype, stream);
}

}  // namespace tim
