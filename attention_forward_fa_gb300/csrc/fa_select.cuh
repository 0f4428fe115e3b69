// fa_select_pages: the pages of a sequence whose keys can score highest.
#pragma once
#include "fa_paged.cuh"

namespace fa {

struct SelectParams {
  PagedKv kv;
  const uint16_t* q;
  int32_t* out;
  const int32_t* kv_lens;
  double* score;          // [B * Hkv, max_pages]
  int Hq, Hkv, G, Sq, max_sel, first, last;
  int* status;
};

constexpr int kSelectThreads = 512;

// One block per (sequence, KV head): a warp per page computes its score in 64
// bits; a page is listed when fewer than max_sel pages rank before it.
template <bool BF16, int D>
__global__ void __launch_bounds__(kSelectThreads) fa_select_kernel(const SelectParams p) {
  constexpr int E = D / 32;
  __shared__ int s_warp[kSelectThreads / 32];
  __shared__ int s_base;
  const int hk = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = max(0, paged_len(p.kv, p.kv_lens[b], p.status));
  const int ps = 1 << p.kv.page_shift;
  const int n = (len + ps - 1) >> p.kv.page_shift;
  double* score = p.score + (long long)blockIdx.x * p.kv.max_pages;
  const int rows = p.G * p.Sq;
  const uint16_t* q = p.q + ((long long)b * p.Hq + hk * p.G) * p.Sq * D;
  for (int s = warp; s < n; s += kSelectThreads / 32) {
    double best = -INFINITY;
    const int id = paged_id(p.kv, b, s, p.status);
    if (id >= 0) {
      const long long at = ((long long)id * p.Hkv + hk) * D + lane * E;
      for (int r = 0; r < rows; ++r) {
        double x = 0.;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const double w = lo16_f32<BF16>(q[(long long)r * D + lane * E + e]);
          x += fmax(w * (double)lo16_f32<BF16>(p.kv.k_min[at + e]), w * (double)lo16_f32<BF16>(p.kv.k_max[at + e]));
        }
#pragma unroll
        for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        best = fmax(best, x);
      }
      if (s < p.first || s >= n - p.last) best = INFINITY;
    }
    if (lane == 0) score[s] = best;
  }
  if (threadIdx.x == 0) s_base = 0;
  __syncthreads();
  int32_t* out = p.out + (long long)blockIdx.x * p.max_sel;
  for (int s0 = 0; s0 < n; s0 += kSelectThreads) {
    const int s = s0 + threadIdx.x;
    bool take = false;
    if (s < n) {
      const double x = score[s];
      int before = 0;
      for (int j = 0; j < n; ++j) before += score[j] > x || (score[j] == x && j < s);
      take = before < p.max_sel;
    }
    const unsigned mask = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_warp[warp] = __popc(mask);
    __syncthreads();
    int at = s_base + __popc(mask & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    if (take) out[at] = s;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 0; w < kSelectThreads / 32; ++w) s_base += s_warp[w];
    __syncthreads();
  }
  for (int s = s_base + threadIdx.x; s < p.max_sel; s += kSelectThreads) out[s] = -1;
}

}  // namespace fa
