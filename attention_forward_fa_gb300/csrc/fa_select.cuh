// fa_select_pages: the pages of a sequence whose keys can score highest.
//
// With q+ and q- the positive and negative parts of q, a page's score is a plain
// product, sum_d max(q_d min_d, q_d max_d) = q+ . max + q- . min, so that the
// bounds stream through the tensor cores once for all rows of a group: pages
// are the 16-row side of mma.m16n8k16, rows the 8-column side, and both operands
// go from memory to registers in the order in which they lie (a permutation of
// the channels that is the same on both sides changes no sum).  HBM bound: 4 D
// bytes per page and KV head.
//
// The answer is a list of whole numbers, the one that 64-bit arithmetic gives,
// while these scores carry fp32 error.  So each page also gets
// a = |q| . (|max| + |min|), which bounds that error by e = 2^-14 a (at most 32
// steps of 17 addends, each truncated to 2^-23 of the largest, for 256
// products), and the second kernel takes what lies more than 2 e above the
// threshold, drops what lies more than 2 e below, and scores the few in between
// (two of 2048 on normal data) again in 64 bits.  Why that is right: let T be
// the k-th largest approximate score and E the k-th largest exact one.  Moving
// each value by at most e moves the k-th largest by at most e, so |E - T| <= e;
// a score above T + 2 e is exactly above T + e >= E, one below T - 2 e below E.
#pragma once
#include "fa_decode.cuh"   // mma_16x8

namespace fa {

struct SelectParams {
  PagedKv kv;
  const uint16_t* q;
  int32_t* out;
  const int32_t* kv_lens;
  float2* score;          // [B * Hkv, max_pages]: score, error scale; later 64-bit scores of the near ones
  int32_t* near;          // [B * Hkv, max_pages]: pages near the threshold
  int32_t* mark;          // [B * Hkv, max_pages]: of those, which are taken
  int Hq, Hkv, rows, max_sel, first, last;   // rows = G * Sq
  int chunks;             // blocks of pages per (sequence, KV head)
  int* status;
};

constexpr int kScoreWarps = 4;
constexpr int kScorePages = 16 * kScoreWarps;   // pages per block
constexpr int kSelectThreads = 512;
constexpr int kSelectCached = 8192;             // scores kept in shared memory
constexpr float kScoreEps = 1.f / 16384.f;

__device__ __forceinline__ int select_pages_of(const PagedKv& c, int len) {
  if (len < 0 || len > (c.max_pages << c.page_shift)) return 0;
  return (len + (1 << c.page_shift) - 1) >> c.page_shift;
}

template <bool BF16, int D>
__global__ void __launch_bounds__(32 * kScoreWarps) fa_page_score_kernel(const SelectParams p) {
  constexpr int C = D / 32;
  pdl_launch_dependents();
  pdl_wait_prior();
  const int unit = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int b = unit / p.Hkv, hk = unit % p.Hkv;
  const int n = select_pages_of(p.kv, p.kv_lens[b]);
  if (chunk == 0 && hk == 0 && threadIdx.x == 0) (void)paged_len(p.kv, p.kv_lens[b], p.status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int s0 = chunk * kScorePages + warp * 16;
  if (s0 >= n) return;
  // pages s0 + g and s0 + g + 8: 8 channels at 32 c + 8 t4 of either bound
  uint4 mn[2][C], mx[2][C];
  bool good[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int s = s0 + g + 8 * j;
    const int id = s < n ? paged_id(p.kv, b, s, p.status) : -1;
    good[j] = id >= 0;
    const long long at = ((long long)max(id, 0) * p.Hkv + hk) * D + 8 * t4;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      mn[j][c] = good[j] ? __ldg(reinterpret_cast<const uint4*>(p.kv.k_min + at + 32 * c)) : make_uint4(0, 0, 0, 0);
      mx[j][c] = good[j] ? __ldg(reinterpret_cast<const uint4*>(p.kv.k_max + at + 32 * c)) : make_uint4(0, 0, 0, 0);
    }
  }
  const uint16_t* q = p.q + ((long long)b * p.Hq * (p.rows / (p.Hq / p.Hkv)) + (long long)hk * p.rows) * D + 8 * t4;
  float best[2] = {-INFINITY, -INFINITY}, scale[2] = {0.f, 0.f};
  bool odd[2] = {false, false};       // a score that is not finite: only 64 bits can tell
  auto magnitude = [](uint32_t x) { return x & 0x7FFF7FFFu; };
  for (int r0 = 0; r0 < p.rows; r0 += 8) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, err[4] = {0.f, 0.f, 0.f, 0.f};
    const bool on = r0 + g < p.rows;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint4 w = on ? __ldg(reinterpret_cast<const uint4*>(q + (long long)(r0 + g) * D + 32 * c)) : make_uint4(0, 0, 0, 0);
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
      const uint32_t lo[2][4] = {{mn[0][c].x, mn[0][c].y, mn[0][c].z, mn[0][c].w}, {mn[1][c].x, mn[1][c].y, mn[1][c].z, mn[1][c].w}};
      const uint32_t hi[2][4] = {{mx[0][c].x, mx[0][c].y, mx[0][c].z, mx[0][c].w}, {mx[1][c].x, mx[1][c].y, mx[1][c].z, mx[1][c].w}};
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        const uint32_t ah[4] = {hi[0][h], hi[1][h], hi[0][h + 1], hi[1][h + 1]};
        const uint32_t al[4] = {lo[0][h], lo[1][h], lo[0][h + 1], lo[1][h + 1]};
        mma_16x8<BF16>(acc, ah, max16x2<BF16>(x[h], 0u), max16x2<BF16>(x[h + 1], 0u));
        mma_16x8<BF16>(acc, al, min16x2<BF16>(x[h], 0u), min16x2<BF16>(x[h + 1], 0u));
        const uint32_t bh[4] = {magnitude(ah[0]), magnitude(ah[1]), magnitude(ah[2]), magnitude(ah[3])};
        const uint32_t bl[4] = {magnitude(al[0]), magnitude(al[1]), magnitude(al[2]), magnitude(al[3])};
        mma_16x8<BF16>(err, bh, magnitude(x[h]), magnitude(x[h + 1]));
        mma_16x8<BF16>(err, bl, magnitude(x[h]), magnitude(x[h + 1]));
      }
    }
    // lane (g, t4): pages g (0, 1) and g + 8 (2, 3), rows 2 t4 and 2 t4 + 1
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (r0 + 2 * t4 + (e & 1) >= p.rows) continue;
      best[e >> 1] = fmaxf(best[e >> 1], acc[e]);
      scale[e >> 1] = fmaxf(scale[e >> 1], err[e]);
      odd[e >> 1] |= !(fabsf(acc[e]) < INFINITY) || !(err[e] < INFINITY);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      best[j] = fmaxf(best[j], __shfl_xor_sync(0xffffffffu, best[j], w));
      scale[j] = fmaxf(scale[j], __shfl_xor_sync(0xffffffffu, scale[j], w));
      odd[j] |= __shfl_xor_sync(0xffffffffu, (int)odd[j], w) != 0;
    }
    const int s = s0 + g + 8 * j;
    if (t4 == 0 && s < n)      // a page that is none scores below all others
      p.score[(long long)unit * p.kv.max_pages + s] =
          good[j] ? make_float2(odd[j] ? 0.f : best[j], odd[j] ? INFINITY : scale[j]) : make_float2(-INFINITY, 0.f);
  }
}

// fp32 as an unsigned number of the same order
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// One block per (sequence, KV head): the threshold by a radix selection over
// the scores, the pages near it in 64 bits, the list in ascending order.
template <bool BF16, int D>
__global__ void __launch_bounds__(kSelectThreads) fa_select_kernel(const SelectParams p) {
  constexpr int kWarps = kSelectThreads / 32;
  constexpr int E = D / 32;
  __shared__ uint32_t s_key[kSelectCached];
  __shared__ int s_hist[256];
  __shared__ int s_warp[kWarps];
  __shared__ float s_top[kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left, s_near;
  pdl_launch_dependents();
  pdl_wait_prior();
  const int unit = blockIdx.x;
  const int b = unit / p.Hkv, hk = unit % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = select_pages_of(p.kv, p.kv_lens[b]);
  int32_t* out = p.out + (long long)unit * p.max_sel;
  if (n <= p.max_sel) {
    for (int s = tid; s < p.max_sel; s += kSelectThreads) out[s] = s < n ? s : -1;
    return;
  }
  const long long base = (long long)unit * p.kv.max_pages;
  const float2* score = p.score + base;
  const int lo_s = p.first, hi_s = n - p.last;     // the pages that compete: more than `want`
  const int want = p.max_sel - p.first - p.last;
  float eps = 0.f;
  for (int s = lo_s + tid; s < hi_s; s += kSelectThreads) {
    const float2 x = score[s];
    eps = fmaxf(eps, x.y);
    if (s - lo_s < kSelectCached) s_key[s - lo_s] = ordered(x.x);
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) eps = fmaxf(eps, __shfl_xor_sync(0xffffffffu, eps, w));
  if (lane == 0) s_top[warp] = eps;
  if (tid == 0) s_prefix = 0, s_left = want, s_near = 0;
  auto key = [&](int s) { return s - lo_s < kSelectCached ? s_key[s - lo_s] : ordered(score[s].x); };

  // the want-th largest key, eight bits at a time
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) s_hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      for (int s = lo_s + tid; s < hi_s; s += kSelectThreads) {
        const uint32_t k = key(s);
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&s_hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {   // lane i has digits 255 - 8 i down to 248 - 8 i
        int c[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += c[e] = s_hist[255 - 8 * lane - e];
        int inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, inc, d);
          if (lane >= d) inc += x;
        }
        const int left = s_left;
        __syncwarp();
        int above = inc - sum;
        if (above < left && left <= inc) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (above < left && left <= above + c[e]) {
              s_prefix = (prefix << 8) | (uint32_t)(255 - 8 * lane - e);
              s_left = left - above;
              break;
            }
            above += c[e];
          }
        }
      }
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  eps = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) eps = fmaxf(eps, s_top[w]);
  // in 64 bits, so that the rounding of the limits adds nothing
  const double mid = want > 0 ? (double)unordered(s_prefix) : INFINITY;
  const double two = 2.0 * (kScoreEps * (double)eps + 0x1p-100);   // (products may underflow)
  const bool blind = !(two < INFINITY);           // a bound that is not finite: all of them in 64 bits
  const double above = mid + two, below = mid - two;
  // 0: out, 1: taken, 2: near.  A page that is none (-inf) is never near a finite threshold.
  auto kind = [&](int s) {
    if (s < lo_s || s >= hi_s) return 1;
    if (want == 0) return 0;
    if (blind) return 2;
    const double x = (double)unordered(key(s));
    return x > above ? 1 : x >= below ? 2 : 0;
  };
  // each thread has a run of pages, so that counts in thread order are counts in page order
  const int run = (n + kSelectThreads - 1) / kSelectThreads;
  const int a0 = min(n, tid * run), a1 = min(n, a0 + run);
  int sure = 0, near = 0;
  for (int s = a0; s < a1; ++s) {
    const int k = kind(s);
    sure += k == 1;
    near += k == 2;
  }
  int packed = __reduce_add_sync(0xffffffffu, sure);
  if (lane == 0) s_warp[warp] = packed;
  if (near) atomicAdd(&s_near, near);
  __syncthreads();
  int n_sure = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) n_sure += s_warp[w];
  const int n_near = s_near;
  const int take = p.max_sel - n_sure;            // of the near ones
  __syncthreads();
  if (n_near > take) {                            // (block-uniform) some of them have to go
    if (tid == 0) s_near = 0;
    __syncthreads();
    for (int s = a0; s < a1; ++s)
      if (kind(s) == 2) p.near[base + atomicAdd(&s_near, 1)] = s;
    __syncthreads();
    double* exact = reinterpret_cast<double*>(p.score + base);   // by place in the list, over scores that ...
    const uint16_t* q = p.q + ((long long)b * p.Hq * (p.rows / (p.Hq / p.Hkv)) + (long long)hk * p.rows) * D + E * lane;
    // ... pages past the cached ones still need: their kinds are kept in `mark` first
    for (int s = a0; s < a1; ++s) p.mark[base + s] = kind(s) == 1;
    __syncthreads();
    for (int i = warp; i < n_near; i += kWarps) {
      const int s = p.near[base + i];
      const int id = p.kv.table[(long long)b * p.kv.table_stride + s];
      double best = -INFINITY;
      if (id >= 0 && id < p.kv.num_pages) {
        const long long at = ((long long)id * p.Hkv + hk) * D + E * lane;
        double mn[E], mx[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          mn[e] = lo16_f32<BF16>(p.kv.k_min[at + e]);
          mx[e] = lo16_f32<BF16>(p.kv.k_max[at + e]);
        }
        for (int r = 0; r < p.rows; ++r) {
          double x = 0.;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const double w = lo16_f32<BF16>(q[(long long)r * D + e]);
            x += w > 0. ? w * mx[e] : w * mn[e];
          }
#pragma unroll
          for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
          best = fmax(best, x);
        }
      }
      if (lane == 0) exact[i] = best;
    }
    __syncthreads();
    for (int i = tid; i < n_near; i += kSelectThreads) {
      const double x = exact[i];
      const int s = p.near[base + i];
      int before = 0;
      for (int j = 0; j < n_near; ++j) before += exact[j] > x || (exact[j] == x && p.near[base + j] < s);
      if (before < take) p.mark[base + s] = 1;
    }
    __syncthreads();
  }
  const bool marked = n_near > take;
  auto taken = [&](int s) { return marked ? p.mark[base + s] != 0 : kind(s) != 0; };
  int mine = 0;
  for (int s = a0; s < a1; ++s) mine += taken(s);
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int place = inc - mine;
  for (int w = 0; w < warp; ++w) place += s_warp[w];
  for (int s = a0; s < a1; ++s)
    if (taken(s) && place < p.max_sel) out[place++] = s;
}

}  // namespace fa
