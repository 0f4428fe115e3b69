// fa_decode: attention of a sequence's newest tokens over its pages.
#pragma once
#include "fa_paged.cuh"

namespace fa {

struct DecodeParams {
  PagedKv kv;
  const uint16_t* q;
  void* o;
  float* lse;
  const int32_t* kv_lens;
  const int32_t* sel;   // [B, Hkv, max_sel] or null
  int max_sel;
  int B, Hq, Hkv, G, Sq;
  int pre_tokens;
  float scale_log2;
  int* status;
};

// One block per row: its four warps take the keys in turn, each with a running
// maximum m, sum l and unnormalised O of its own, joined at the end.
template <bool BF16, int D>
__global__ void __launch_bounds__(128) fa_decode_row_kernel(const DecodeParams p) {
  constexpr int E = D / 32;
  __shared__ float s_o[4][D];
  __shared__ float s_m[4], s_l[4];
  const int i = blockIdx.x % p.Sq;
  const int h = (blockIdx.x / p.Sq) % p.Hq;
  const int b = blockIdx.x / p.Sq / p.Hq;
  const int hk = h / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = max(0, paged_len(p.kv, p.kv_lens[b], p.status));
  const int tok = len - p.Sq + i;
  const int low = p.pre_tokens >= 0 ? max(0, tok - p.pre_tokens) : 0;
  const int ps = 1 << p.kv.page_shift;
  const int pages = (len + ps - 1) >> p.kv.page_shift;
  const long long row = ((long long)b * p.Hq + h) * p.Sq + i;
  float qv[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint16_t x = p.q[row * D + lane * E + e];
    qv[e] = lo16_f32<BF16>(x);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int32_t* sel = p.sel ? p.sel + ((long long)b * p.Hkv + hk) * p.max_sel : nullptr;
  const int n = sel ? p.max_sel : pages;
  for (int s = 0; s < n; ++s) {
    const int page = sel ? sel[s] : s;
    if (page < 0 || page >= pages) continue;
    const int k0 = page << p.kv.page_shift;
    if (k0 > tok || k0 + ps <= low) continue;
    const int id = paged_id(p.kv, b, page, p.status);
    if (id < 0) continue;
    for (int j = warp; j < ps; j += 4) {
      if (k0 + j > tok || k0 + j < low) continue;
      const uint16_t* kr = p.kv.k + (long long)id * p.kv.k_sp + hk * p.kv.k_sh + j * p.kv.k_ss + lane * E;
      const uint16_t* vr = p.kv.v + (long long)id * p.kv.v_sp + hk * p.kv.v_sh + j * p.kv.v_ss + lane * E;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x += qv[e] * lo16_f32<BF16>(kr[e]);
#pragma unroll
      for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      x *= p.scale_log2;
      const float mn = fmaxf(m, x);
      const float base = mn > -INFINITY ? mn : 0.f;
      const float r = exp2f(m - base), e0 = exp2f(x - base);
      l = l * r + e0;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * r + e0 * lo16_f32<BF16>(vr[e]);
      m = mn;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float base = m > -INFINITY ? m : 0.f;
  l = 0.f;
  for (int w = 0; w < 4; ++w) l += s_l[w] * exp2f(s_m[w] - base);
  if (threadIdx.x < D / 2) {
    float a = 0.f, c = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float f = exp2f(s_m[w] - base);
      a += f * s_o[w][2 * threadIdx.x];
      c += f * s_o[w][2 * threadIdx.x + 1];
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    reinterpret_cast<uint32_t*>(p.o)[(row * D) / 2 + threadIdx.x] = pack16x2<BF16>(a * inv, c * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : INFINITY;
}

}  // namespace fa
