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
// a = |q| . (|max| + |min|), which bounds that error by e = 2^-17 a: two matrix
// instructions at a time start from zero and truncate their addends, exact
// products and the sum so far, to 2^-23 of the largest (33 2^-23 of the sum of
// magnitudes at most), and up to 8 such pairs are added with 2^-24 each;
// (66 + 8) 2^-24 < 2^-17.  (One accumulator through all of them would need 2^-14,
// and leave four pages of 2048 in doubt instead of one half.)  The
// second kernel takes what lies more than 2 e above the threshold, drops what
// lies more than 2 e below, and scores what is in between again in 64 bits.  Why that is right: let T be
// the k-th largest approximate score and E the k-th largest exact one.  Moving
// each value by at most e moves the k-th largest by at most e, so |E - T| <= e;
// a score above T + 2 e is exactly above T + e >= E, one below T - 2 e below E.
// (T itself is only followed down to an interval shorter than 2 e.)
#pragma once
#include "fa_decode.cuh"   // mma_16x8

namespace fa {

struct SelectParams {
  PagedKv kv;
  const uint16_t* q;
  int32_t* out;
  const int32_t* kv_lens;
  float2* score;          // [B * Hkv, max_pages]: score, error scale
  unsigned long long* exact;   // [B * Hkv, max_pages] each: what does not fit shared memory of the pages
  int32_t* near;          //   near the threshold: their 64-bit scores, their numbers and (a bit each)
  uint32_t* mark;         //   which of them are taken
  int B, Hkv, rows, max_sel, first, last;   // rows = G * Sq
  int chunks;             // runs of kScorePages per (sequence, KV head)
  int* status;
};

constexpr int kScorePages = 16;                 // pages that a block of one warp scores at a time
constexpr int kScoreBlocks = 56;                // blocks per SM at most
constexpr int kSelectThreads = 512;
constexpr int kKeys = 8;                        // scores per thread held in registers (4096 pages)
constexpr int kNearCached = 256;                // pages near the threshold kept in shared memory
constexpr float kScoreEps = 1.f / 131072.f;

__device__ __forceinline__ int select_pages_of(const PagedKv& c, int len) {
  if (len < 0 || len > (c.max_pages << c.page_shift)) return 0;
  return (len + (1 << c.page_shift) - 1) >> c.page_shift;
}

// Pages of a sequence that have to be scored: none where the list has room for all.
__device__ __forceinline__ int scored_pages_of(const SelectParams& p, int len) {
  const int n = select_pages_of(p.kv, len);
  return n > p.max_sel ? n : 0;
}

// A warp scores 16 pages.  Each lane copies to shared memory, all at once, the very 16-byte pieces that
// it will feed to the matrix instructions, so that nothing has to be exchanged and no register waits
// for memory: 8 KB in flight per warp (D 128), 24 warps per SM.  (Measured with the second kernel,
// 2048 pages of 64 (sequence, KV head) pairs, D 128, 67 MB of bounds: this 22.7 us, of which 15.6 are
// this kernel's; 32 pages per warp 24.4 us, 48 25.9 us, 64 25.5 us: fewer, longer blocks end
// unevenly; bounds loaded to registers, 12 warps per SM, 38.6 us; one long run of pages per warp
// through a ring of three groups 35 us: it leaves the latency of the matrix instructions bare.)
template <bool BF16, int D>
__device__ __forceinline__ void score_pages(const SelectParams& p, uint4 (&s_in)[2][2][D / 32][32], int unit, int b,
                                            int first, int n) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x, g = lane >> 2, t4 = lane & 3;
  const int hk = unit - b * p.Hkv;
  const int ids = lane < 16 && first + lane < n ? paged_id(p.kv, b, first + lane, p.status) : -1;
  // of pages first + g and first + g + 8: 8 channels at 32 c + 8 t4 of either bound
  bool good[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int id = __shfl_sync(0xffffffffu, ids, g + 8 * j);
    good[j] = id >= 0;
    if (id < 0) continue;          // (its stale bounds reach no other page's products)
    const long long at = ((long long)id * p.Hkv + hk) * D + 8 * t4;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      cp_async16(smem_u32(&s_in[0][j][c][lane]), p.kv.k_min + at + 32 * c);
      cp_async16(smem_u32(&s_in[1][j][c][lane]), p.kv.k_max + at + 32 * c);
    }
  }
  cp_async_commit();
  const uint16_t* q = p.q + (long long)unit * p.rows * D + 8 * t4;   // [B, Hkv, rows, D]
  auto magnitude = [](uint32_t x) { return x & 0x7FFF7FFFu; };
  float best[2] = {-INFINITY, -INFINITY}, scale[2] = {0.f, 0.f};
  bool odd[2] = {false, false};    // a score that is not finite: only 64 bits can tell
  for (int r0 = 0; r0 < p.rows; r0 += 8) {
    uint4 w[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      w[c] = r0 + g < p.rows ? *reinterpret_cast<const uint4*>(q + (long long)(r0 + g) * D + 32 * c) : make_uint4(0, 0, 0, 0);
    if (r0 == 0) cp_async_wait_all();          // (every lane its own copies)
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, err[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint4 l0 = s_in[0][0][c][lane], l1 = s_in[0][1][c][lane];
      const uint4 h0 = s_in[1][0][c][lane], h1 = s_in[1][1][c][lane];
      const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
      const uint32_t lo[2][4] = {{l0.x, l0.y, l0.z, l0.w}, {l1.x, l1.y, l1.z, l1.w}};
      const uint32_t hi[2][4] = {{h0.x, h0.y, h0.z, h0.w}, {h1.x, h1.y, h1.z, h1.w}};
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        const uint32_t ah[4] = {hi[0][h], hi[1][h], hi[0][h + 1], hi[1][h + 1]};
        const uint32_t al[4] = {lo[0][h], lo[1][h], lo[0][h + 1], lo[1][h + 1]};
        float u[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};   // from zero: see the bound above
        mma_16x8<BF16>(u, ah, max16x2<BF16>(x[h], 0u), max16x2<BF16>(x[h + 1], 0u));
        mma_16x8<BF16>(u, al, min16x2<BF16>(x[h], 0u), min16x2<BF16>(x[h + 1], 0u));
        const uint32_t bh[4] = {magnitude(ah[0]), magnitude(ah[1]), magnitude(ah[2]), magnitude(ah[3])};
        const uint32_t bl[4] = {magnitude(al[0]), magnitude(al[1]), magnitude(al[2]), magnitude(al[3])};
        mma_16x8<BF16>(v, bh, magnitude(x[h]), magnitude(x[h + 1]));
        mma_16x8<BF16>(v, bl, magnitude(x[h]), magnitude(x[h + 1]));
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += u[e], err[e] += v[e];
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
    for (int x = 1; x < 4; x <<= 1) {
      best[j] = fmaxf(best[j], __shfl_xor_sync(0xffffffffu, best[j], x));
      scale[j] = fmaxf(scale[j], __shfl_xor_sync(0xffffffffu, scale[j], x));
      odd[j] |= __shfl_xor_sync(0xffffffffu, (int)odd[j], x) != 0;
    }
    const int s = first + g + 8 * j;
    if (t4 == 0 && s < n)            // a page that is none scores below all others
      p.score[(long long)unit * p.kv.max_pages + s] =
          good[j] ? make_float2(odd[j] ? 0.f : best[j], odd[j] ? INFINITY : scale[j]) : make_float2(-INFINITY, 0.f);
  }
}

// A block per run of 16 pages that the table has room for, or, where that were more than kScoreBlocks per
// SM, so many blocks that each look at 32 of their runs at once for those that hold pages: tables
// have room for more than most sequences use.  (64 sequences of 188 pages, 8 KV heads of 64, room for
// 8192: 24 us, a block per run 277 us; where all room is used the loop costs, 23.4 us against 22.7 us
// in the case above.)
template <bool BF16, int D, bool MANY>
__global__ void __launch_bounds__(32) fa_page_score_kernel(const SelectParams p) {
  __shared__ __align__(16) uint4 s_in[2][2][D / 32][32];   // [bound][page half][step][lane]
  pdl_wait_prior();
  pdl_launch_dependents();   // (after the wait: the next kernel may read the lengths as it starts)
  const int lane = threadIdx.x;
  if constexpr (!MANY) {
    const int unit = blockIdx.x / p.chunks, first = blockIdx.x % p.chunks * kScorePages, b = unit / p.Hkv;
    const int len = p.kv_lens[b], n = scored_pages_of(p, len);
    if (first == 0 && unit == b * p.Hkv && lane == 0) (void)paged_len(p.kv, len, p.status);
    if (first >= n) return;
    score_pages<BF16, D>(p, s_in, unit, b, first, n);
  } else {
    const unsigned runs = (unsigned)p.B * p.Hkv * p.chunks;   // (below 2^31)
    for (unsigned run0 = blockIdx.x; run0 < runs; run0 += 32 * gridDim.x) {
      const unsigned run = run0 + gridDim.x * lane;
      const int unit = (int)(run / (unsigned)p.chunks), first = (int)(run % (unsigned)p.chunks) * kScorePages;
      const int b = unit / p.Hkv, len = run < runs ? p.kv_lens[b] : 0, n = scored_pages_of(p, len);
      if (run < runs && first == 0 && unit == b * p.Hkv) (void)paged_len(p.kv, len, p.status);
      for (unsigned live = __ballot_sync(0xffffffffu, first < n); live; live &= live - 1) {
        const int at = __ffs(live) - 1;
        score_pages<BF16, D>(p, s_in, __shfl_sync(0xffffffffu, unit, at), __shfl_sync(0xffffffffu, b, at),
                             __shfl_sync(0xffffffffu, first, at), __shfl_sync(0xffffffffu, n, at));
      }
    }
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
  __shared__ int s_hist[256];
  __shared__ int2 s_warp[kWarps];
  __shared__ unsigned long long s_exact[kNearCached];
  __shared__ int32_t s_list[kNearCached];
  __shared__ uint32_t s_mark[kNearCached / 32 + 1];
  __shared__ float s_top[kWarps];
  __shared__ uint32_t s_lo[kWarps], s_hi[kWarps];
  __shared__ int s_digit;
  __shared__ int s_left;
  const int unit = blockIdx.x;
  const int b = unit / p.Hkv, hk = unit % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = select_pages_of(p.kv, __ldcg(p.kv_lens + b));
  pdl_launch_dependents();
  pdl_wait_prior();
  int32_t* out = p.out + (long long)unit * p.max_sel;
  if (n <= p.max_sel) {
    for (int s = tid; s < p.max_sel; s += kSelectThreads) out[s] = s < n ? s : -1;
    return;
  }
  const long long base = (long long)unit * p.kv.max_pages;
  const float2* score = p.score + base;
  const int lo_s = p.first, hi_s = n - p.last;     // the pages that compete: more than `want`
  const int want = p.max_sel - p.first - p.last;
  // Each thread has a run of pages, so that counts in thread order are counts in page order.  Their
  // keys stay in registers where a run is at most kKeys, and are read again (from L2) in every pass
  // over longer runs, kKeys at a time.
  const int run = (n + kSelectThreads - 1) / kSelectThreads;
  const int a0 = min(n, tid * run), a1 = min(n, a0 + run);
  uint32_t keys[kKeys];
  auto competes = [&](int s) { return s >= lo_s && s < min(hi_s, a1); };
  float eps = 0.f;
  uint32_t kmin = 0xffffffffu, kmax = 0;
  for (int s0 = a0; s0 < a1; s0 += kKeys) {
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      if (!competes(s0 + j)) continue;
      const float2 x = score[s0 + j];
      keys[j] = ordered(x.x);
      eps = fmaxf(eps, x.y);
      kmin = min(kmin, keys[j]);
      kmax = max(kmax, keys[j]);
    }
  }
  auto fetch = [&](int s0) {
    if (run <= kKeys) return;
#pragma unroll
    for (int j = 0; j < kKeys; ++j)
      if (competes(s0 + j)) keys[j] = ordered(score[s0 + j].x);
  };
#pragma unroll
  for (int w = 16; w; w >>= 1) eps = fmaxf(eps, __shfl_xor_sync(0xffffffffu, eps, w));
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) s_top[warp] = eps, s_lo[warp] = kmin, s_hi[warp] = kmax;
  if (tid < 256) s_hist[tid] = 0;
  if (tid <= kNearCached / 32) s_mark[tid] = 0;
  if (tid == 0) s_left = want;
  __syncthreads();
  // (every warp by itself over the 16 partial results)
  eps = s_top[lane % kWarps];
#pragma unroll
  for (int w = kWarps / 2; w; w >>= 1) eps = fmaxf(eps, __shfl_xor_sync(0xffffffffu, eps, w));
  kmin = __reduce_min_sync(0xffffffffu, s_lo[lane % kWarps]);
  kmax = __reduce_max_sync(0xffffffffu, s_hi[lane % kWarps]);
  const float two = __fmul_ru(2.f * kScoreEps, eps) + 0x1p-100f;   // 2 e (products may underflow)

  // The digit that the s_left-th largest of the counted has, and how many of that digit are still to be
  // taken; clears the counts.
  auto pick = [&]() {
    __syncthreads();
    if (warp == 0) {   // lane i has digits 255 - 8 i down to 248 - 8 i
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += c[e] = s_hist[255 - 8 * lane - e];
#pragma unroll
      for (int e = 0; e < 8; ++e) s_hist[255 - 8 * lane - e] = 0;
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
        int e = 0;
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (e == i && above + c[i] < left) above += c[i], e = i + 1;
        s_digit = 255 - 8 * lane - e;
        s_left = left - above;
      }
    }
    __syncthreads();
  };

  // the want-th largest key, up to eight bits at a time below the bits that all keys share
  // (scores have few exponents: without that the first passes would count into one place), until
  // what is left undecided is less than the scores' errors: T is then that interval
  uint32_t prefix = kmin;
  int bits = 0;                                      // undecided
  if (want > 0 && kmin != kmax) {
    bits = 32 - __clz(kmin ^ kmax);
    prefix = bits < 32 ? kmin >> bits : 0;
    while (bits > 0) {
      const int w = min(bits, 8), shift = bits - w;
#pragma unroll 1
      for (int s0 = a0; s0 < a1; s0 += kKeys) {
        fetch(s0);
#pragma unroll
        for (int j = 0; j < kKeys; ++j)
          if (competes(s0 + j) && (bits == 32 || (keys[j] >> bits) == prefix))
            atomicAdd(&s_hist[(keys[j] >> shift) & ((1u << w) - 1)], 1);
      }
      pick();
      prefix = prefix << w | (uint32_t)s_digit;
      bits = shift;
      if (unordered(prefix << bits | ((1u << bits) - 1)) - unordered(prefix << bits) <= two) break;
    }
  }
  // the limits, rounded outwards, as keys (a zero limit takes the sign that keeps zeros near)
  const bool blind = !(two < INFINITY);           // a bound that is not finite: all of them in 64 bits
  const float up = __fadd_ru(unordered(prefix << bits | ((1u << bits) - 1)), two);
  const float down = __fadd_rd(unordered(prefix << bits), -two);
  const uint32_t above = ordered(up == 0.f ? 0.f : up), below = ordered(down == 0.f ? -0.f : down);
  // Which pages of [s0, s0 + kKeys) are taken and which near, as bits.  (A page that is none, -inf,
  // is never near a finite threshold.)
  auto sort_out = [&](int s0, unsigned& sure, unsigned& near) {
    fetch(s0);
    sure = near = 0;
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      const int s = s0 + j;
      if (s >= a1) continue;
      if (!competes(s)) sure |= 1u << j;                  // first or last: always
      else if (want > 0 && !blind && keys[j] > above) sure |= 1u << j;
      else if (want > 0 && (blind || keys[j] >= below)) near |= 1u << j;
    }
  };
  unsigned sure_bits = 0, near_bits = 0;                  // of the run's last kKeys (its only ones, mostly)
  int sure = 0, near = 0;
#pragma unroll 1
  for (int s0 = a0; s0 < a1; s0 += kKeys) {
    sort_out(s0, sure_bits, near_bits);
    sure += __popc(sure_bits);
    near += __popc(near_bits);
  }
  int2 inc = make_int2(sure, near);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc.x, d), y = __shfl_up_sync(0xffffffffu, inc.y, d);
    if (lane >= d) inc.x += x, inc.y += y;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  // of all, and before this run: every warp adds up the 16 by itself
  const int2 part = lane < kWarps ? s_warp[lane] : make_int2(0, 0);
  const int n_sure = __reduce_add_sync(0xffffffffu, part.x), n_near = __reduce_add_sync(0xffffffffu, part.y);
  int place = __reduce_add_sync(0xffffffffu, lane < warp ? part.x : 0) + inc.x - sure;
  const int near0 = __reduce_add_sync(0xffffffffu, lane < warp ? part.y : 0) + inc.y - near;
  const int take = p.max_sel - n_sure;                 // of the near ones
  const bool choose = n_near > take;                   // (block-uniform) some of them have to go
  const bool small = n_near <= kNearCached;
  unsigned long long* exact = small ? s_exact : p.exact + base;
  int32_t* list = small ? s_list : p.near + base;
  uint32_t* mark = small ? s_mark : p.mark + base;
  if (choose) {
#pragma unroll 1
    for (int s0 = a0, i = near0; s0 < a1; s0 += kKeys) {
      if (run > kKeys) sort_out(s0, sure_bits, near_bits);
      for (unsigned x = near_bits; x; x &= x - 1, ++i) {
        exact[i] = 0;
        list[i] = s0 + __ffs(x) - 1;
      }
    }
    if (tid == 0) s_left = take;
    __syncthreads();
    // Eight lanes per page and row, D / 8 channels each; the rows' maximum as an ordered number.  (64-bit
    // sums are slow here, two a cycle and SM: a whole warp per page and row spends more of them on
    // adding up its lanes than on the products.  2048 pages all alike, 4 rows of 64 channels: that
    // took 995 us, this 540.)
    constexpr int kItems = kSelectThreads / 8;
    const int sub = lane & 7;
    const uint16_t* q = p.q + (long long)unit * p.rows * D + D / 8 * sub;
    const int step_page = kItems / p.rows, step_row = kItems % p.rows;
    int mine = (tid >> 3) / p.rows, row = (tid >> 3) % p.rows;
#pragma unroll 1
    while (__any_sync(0xffffffffu, mine < n_near)) {
      const int id = mine < n_near ? p.kv.table[(long long)b * p.kv.table_stride + list[mine]] : -1;
      const bool good = id >= 0 && id < p.kv.num_pages;  // else below all others
      double x = 0.;
      if (good) {
        const long long at = ((long long)id * p.Hkv + hk) * D + D / 8 * sub;
#pragma unroll
        for (int e = 0; e < D / 8; e += 8) {
          const uint4 wq = *reinterpret_cast<const uint4*>(q + (long long)row * D + e);
          const uint4 lo = *reinterpret_cast<const uint4*>(p.kv.k_min + at + e);
          const uint4 hi = *reinterpret_cast<const uint4*>(p.kv.k_max + at + e);
          auto add = [&](uint32_t y, uint32_t l, uint32_t h) {
            const float q0 = lo16_f32<BF16>(y), q1 = hi16_f32<BF16>(y);
            x = fma((double)q0, (double)(q0 > 0.f ? lo16_f32<BF16>(h) : lo16_f32<BF16>(l)), x);
            x = fma((double)q1, (double)(q1 > 0.f ? hi16_f32<BF16>(h) : hi16_f32<BF16>(l)), x);
          };
          add(wq.x, lo.x, hi.x);
          add(wq.y, lo.y, hi.y);
          add(wq.z, lo.z, hi.z);
          add(wq.w, lo.w, hi.w);
        }
      }
#pragma unroll
      for (int w = 4; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      if (good && sub == 0) {
        const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.);   // (-0 as 0)
        atomicMax(exact + mine, u >> 63 ? ~u : u | 0x8000000000000000ull);
      }
      mine += step_page;
      row += step_row;
      if (row >= p.rows) row -= p.rows, ++mine;
    }
    __syncthreads();
    // (the list is in page order: of equal scores the first are taken)
    if (small) {
      if (tid < n_near) {
        const unsigned long long x = exact[tid];
        int ahead = 0;
#pragma unroll 1
        for (int j = 0; j < n_near; ++j) ahead += exact[j] > x || (exact[j] == x && j < tid);
        if (ahead < take) atomicOr(&mark[tid >> 5], 1u << (tid & 31));
      }
    } else {   // many alike: their take-th largest (take >= 1: fewer than `want` lie above the threshold)
      unsigned long long top = 0;
#pragma unroll 1
      for (int shift = 56; shift >= 0; shift -= 8) {
#pragma unroll 1
        for (int i = tid; i < n_near; i += kSelectThreads) {
          const unsigned long long x = exact[i];
          if (shift == 56 || x >> (shift + 8) == top) atomicAdd(&s_hist[(x >> shift) & 255], 1);
        }
        pick();
        top = top << 8 | (unsigned)s_digit;
      }
      int before = 0;                    // of those that equal it
#pragma unroll 1
      for (int i0 = 0; i0 < n_near; i0 += kSelectThreads) {
        const int i = i0 + tid;
        const unsigned long long x = i < n_near ? exact[i] : 0;
        const bool same = i < n_near && x == top;
        const unsigned sames = __ballot_sync(0xffffffffu, same);
        if (lane == 0) s_warp[warp].x = __popc(sames);
        __syncthreads();
        const int c = lane < kWarps ? s_warp[lane].x : 0;
        const int at = before + __reduce_add_sync(0xffffffffu, lane < warp ? c : 0) + __popc(sames & ((1u << lane) - 1));
        before += __reduce_add_sync(0xffffffffu, c);
        const unsigned word = __ballot_sync(0xffffffffu, i < n_near && (x > top || (same && at < s_left)));
        if (lane == 0 && i < n_near) mark[i >> 5] = word;
        __syncthreads();
      }
    }
    __syncthreads();
  }
  if (choose) {
    for (int w = 0; w < near0 >> 5; ++w) place += __popc(mark[w]);
    place += __popc(mark[near0 >> 5] & ((1u << (near0 & 31)) - 1));
  } else {
    place += near0;
  }
#pragma unroll 1
  for (int s0 = a0, i = near0; s0 < a1; s0 += kKeys) {
    if (run > kKeys) sort_out(s0, sure_bits, near_bits);
#pragma unroll 1
    for (unsigned x = sure_bits | near_bits; x; x &= x - 1) {
      const int j = __ffs(x) - 1;
      bool in = true;
      if (near_bits >> j & 1) {
        in = !choose || (mark[i >> 5] >> (i & 31) & 1);
        ++i;
      }
      if (in && place < p.max_sel) out[place++] = s0 + j;
    }
  }
}

}  // namespace fa
