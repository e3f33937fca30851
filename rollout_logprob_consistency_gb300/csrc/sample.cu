// Sampling from a [T, V] logits matrix with temperature, top-k, top-p and min-p, from given uniform
// numbers: sample_list.cuh has the definition and the kernel, here it is launched for tim_sample's rows.
#include "sample_list.cuh"

namespace tim {

using namespace sampling;

cudaError_t launch_sample_plain(const SampleArgs& args, int dtype, int64_t T, cudaStream_t stream);

namespace {

template <int kDtype>
cudaError_t launch_list(const SampleArgs& a, int64_t T, cudaStream_t stream, int num_sms) {
  // As few threads a row as let all rows run at once: a row's stream then lasts as long as all of
  // them need the memory, and what follows it comes once, not once a wave.
  const unsigned g = static_cast<unsigned>(T);
  if (T <= num_sms)
    sample_list_kernel<kDtype, 1024, SampleArgs><<<g, 1024, 0, stream>>>(a);
  else if (T <= 2 * num_sms)
    sample_list_kernel<kDtype, 512, SampleArgs><<<g, 512, 0, stream>>>(a);
  else if (T <= 4 * num_sms)
    sample_list_kernel<kDtype, 256, SampleArgs><<<g, 256, 0, stream>>>(a);
  else
    sample_list_kernel<kDtype, 128, SampleArgs><<<g, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(const void* logits, int dtype, int64_t ld, int64_t T, int V,
                          const float* uniform, const tim_sample_params& p, int32_t* ids,
                          float* logprob, float* lse, int32_t* kept, int* status,
                          cudaStream_t stream, int num_sms) {
  const SampleArgs a = {logits, ld, V, uniform, p.temperature, p.top_k, p.top_p, p.min_p,
                        p.row_temperature, p.row_top_k, p.row_top_p, p.row_min_p, ids, logprob,
                        lse, kept, status};
  // Every row unfiltered, and few of them: a cluster a row.  151936 logits in bf16: 16 rows 16 us (a CTA
  // each 29), 38 rows 21 (31), 76 rows 31 (31), 152 rows 45 (33); in fp32 38 rows 27 (31), 76 rows 41 (33).
  const bool plain = p.row_temperature == nullptr && p.temperature != 0.f &&
                     p.row_top_k == nullptr && (p.top_k <= 0 || p.top_k >= V) &&
                     p.row_top_p == nullptr && p.top_p >= 1.f && p.row_min_p == nullptr &&
                     p.min_p == 0.f;
  if (plain && 3 * T <= num_sms) return launch_sample_plain(a, dtype, T, stream);
  return dtype == TIM_F32    ? launch_list<TIM_F32>(a, T, stream, num_sms)
         : dtype == TIM_BF16 ? launch_list<TIM_BF16>(a, T, stream, num_sms)
                             : launch_list<TIM_F16>(a, T, stream, num_sms);
}

}  // namespace tim
