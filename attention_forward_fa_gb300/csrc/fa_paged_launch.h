// Launches of the paged operators that the host side (fa_paged.cu) shares with
// the second translation unit of their kernels (fa_paged8.cu).
#pragma once
#include <algorithm>

#include "fa_decode8.cuh"
#include "fa_host.h"
#include "fa_kv_append.cuh"
#include "fa_kv_move.cuh"
#include "fa_wide.cuh"

namespace fa_host {

template <int FORM, bool BF16, int D, bool INTERLEAVED>
cudaError_t launch_append(const fa::AppendParams& p, long long pieces, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long long items = 2LL * p.k_items + p.q_items;
  const long long loop = std::max(1LL, (long long)fa::kAppendLoopBlocks * sms / items) * items;   // (an item per block)
  return pieces > (long long)fa::kAppendBlocks * sms
             ? launch_dependent(fa::fa_kv_append_kernel<BF16, D, INTERLEAVED, true, FORM>, (unsigned)loop,
                                fa::kAppendThreads, 0, st, p, (int)pieces)
             : launch_dependent(fa::fa_kv_append_kernel<BF16, D, INTERLEAVED, false, FORM>, (unsigned)pieces,
                                fa::kAppendThreads, 0, st, p, (int)pieces);
}
template <int FORM>
cudaError_t launch_append(const fa::AppendParams& p, bool fp16, int D, bool interleaved, long long pieces, cudaStream_t st) {
  if (D == 128)
    return fp16 ? (interleaved ? launch_append<FORM, false, 128, true>(p, pieces, st) : launch_append<FORM, false, 128, false>(p, pieces, st))
                : (interleaved ? launch_append<FORM, true, 128, true>(p, pieces, st) : launch_append<FORM, true, 128, false>(p, pieces, st));
  return fp16 ? (interleaved ? launch_append<FORM, false, 64, true>(p, pieces, st) : launch_append<FORM, false, 64, false>(p, pieces, st))
              : (interleaved ? launch_append<FORM, true, 64, true>(p, pieces, st) : launch_append<FORM, true, 64, false>(p, pieces, st));
}

cudaError_t launch_append_placed(const fa::AppendParams& p, bool fp16, int D, bool interleaved, long long pieces, cudaStream_t st);
cudaError_t launch_append8(const fa::AppendParams& p, bool fp16, int D, bool interleaved, long long pieces, cudaStream_t st);
int launch_decode8(fa::Decode8Params& p, bool fp16, int D, long long keys, cudaStream_t st);   // an FA_* code
int launch_wide(fa::WideParams& p, bool fp16, int D, bool eight, long long keys, cudaStream_t st);   // an FA_* code
cudaError_t launch_read(const fa::ReadParams& p, bool fp16, int D, bool eight, unsigned blocks, cudaStream_t st);
cudaError_t launch_keep(const fa::KeepParams& p, bool fp16, int D, bool eight, unsigned blocks, cudaStream_t st);

}  // namespace fa_host
