// fa_decode over an 8-bit cache: the schedule, the ring and the join are those of
// fa_decode.cuh; what differs is what a tile is and how it enters the products.
//
//   * A tile is 128 keys, so that it has the bytes of a 16-bit tile of 64, and a
//     row of a tile is one swizzled span of D bytes.  The scale bytes of a page's
//     and head's slots lie side by side; two short bulk copies bring those of a
//     sub-block along with its K and V.
//   * The codes become fp16 in registers, exactly (e4m3 and e5m2 lie inside
//     fp16).  ldmatrix moves 16-bit pairs, that is pairs of codes: of K a lane
//     gets four neighbouring channels of a key, which are taken as channels
//     (2 t, 2 t + 1) and (2 t + 8, 2 t + 9) of a step (a product may take the
//     channels in any order, and Q is laid out alike); of V transposed it gets
//     two channels of two keys, whose even channels become rows 0-7 of the
//     product and whose odd ones rows 8-15.
//   * Q is fp16 too: a bf16 row is multiplied by the power of two that brings its
//     largest channel below 2^15.  That is exact for channels down to 2^-29 of the
//     largest; below, the error is under 2^-39 of it.
//   * A key's scale multiplies its scores (and the scale of Q, in fp32, exactly).
//     A value's scale 2^e joins the exponent of the probability: with s' = s + e
//     (log2 units) and the running reference m over s', the probability that goes
//     into the value product is 2^(s' - m), the weight of the value's codes, and
//     the sum of the softmax takes 2^(s' - m) 2^-e.  So the product's operands are
//     as large as what they add, whatever the scales.  Where 2^(s' - m) could be below
//     2^-126 of a key whose part of the sum counts (its e more than kFarScales below
//     that of a key that the reference followed) the sum takes 2^(s' - e - m) instead.
//   * A value row that is not finite (scale byte 255, codes 0) weighs in the sum as
//     any other and has a NaN for its P in the rows that see it, so that their
//     answers are NaN and no other row's.
//   * P is one fp16 where the answer is bf16: its rounding, 2^-11 of each key's
//     contribution at most, is a quarter of the answer's own.  An fp16 answer gets a
//     hi + lo pair (one fp16 would add as much as its own rounding: 2.9e-4 against 2.1e-4
//     of the answer over 64 sequences of up to 8192 tokens).
//
// Measured (32 query heads on 8 KV heads of 128, both kernels): 8 sequences of 131072
// tokens, e4m3, bf16 314 us, 6.90 TB/s of codes and scales (the 16-bit cache: 600 us);
// 64 of mixed lengths up to 8192, e5m2, fp16, pages of 16 96 us, 5.9 TB/s; one of 517
// tokens 6.5 us; 16 of 4096, 4 and 16 rows, 30 and 35.  Up to 16 rows bound by HBM; from
// there by the warp-level products (16 trees over up to 8192 tokens: 46 us at 24 rows, 59 at
// 32, and, in two passes, 82 at 48, of which the bytes are 21).  ptxas reports 28 to 32 bytes
// of spills with heads of 128 at 16 rows (bf16) and at 32, none elsewhere.
#pragma once
#include <type_traits>

#include "fa_decode.cuh"
#include "fa_paged8.cuh"

namespace fa {

constexpr int kDec8Tile = 128;      // keys per tile
constexpr int kDec8Groups = 8;      // of 16 keys; a consumer scores two
// Teams of four consumers and a producer, each with a ring and a range of its own, that share one CTA
// per SM.  (As CTAs of their own, three per SM at 128 registers, they left an SM with two where the
// kernel started beside the last CTAs of the one before it: five warps each fill the four register
// files only from the right first one on.  The third then ran alone at the end, and 8 sequences of
// 131072 tokens took 435 us back to back against 310 us one by one.)
// (Two where a third's shared memory or registers do not fit.)
template <bool BF16, int NT>
constexpr int kDec8Teams = NT == 1 || (NT == 2 && BF16) ? 3 : 2;

// (P' is lost below 2^-126, m is at most the largest s' less 7: a key of the tiles that take it all the same, up to 95
// below the largest e by tcgen05, then has less than 2^-38 of the share of the sum that the key of the largest s' has.)
constexpr int kFarScales = 80;
// Scale bytes of values are at least kLeastExp + 127: from one below this no other is far, and nobody has to know it.
constexpr uint32_t kLargeScale = kLeastExp + 127 + kFarScales + 1;

struct Decode8Params {
  DecodeCore c;
  const uint8_t* k_scale;      // [num_pages, Hkv, page size]
  const uint8_t* v_scale;
  int e5m2;
  CUtensorMap tm_k;            // (D bytes, slots, heads, pages)
  CUtensorMap tm_v;
};

template <bool BF16, int D, int NT>
struct Decode8Smem {
  using P = std::conditional_t<BF16, uint2, uint4>;              // 16 keys' P of a lane: hi, or hi and lo
  static constexpr int kHalf = kDec8Tile * D;                    // K or V of a tile
  static constexpr int kStages = 2 * (128 / D);                  // 64 KB
  static constexpr bool kQShared = NT > 2;
  static constexpr int kScaleOff = kStages * 2 * kHalf;          // bytes [stages][K, V][128]
  static constexpr int kPOff = kScaleOff + kStages * 2 * kDec8Tile;              // P [8 x 16 keys][NT][lane]
  static constexpr int kQOff = kPOff + kDec8Groups * NT * 32 * (int)sizeof(P);   // uint2 [NT][D / 16][lane]
  static constexpr int kFacOff = kQOff + (kQShared ? NT * (D / 16) * 256 : 0);   // float [8 NT]: Q's scales
  static constexpr int kMaxOff = kFacOff + 8 * NT * 4;                           // float [warps][8 NT]
  static constexpr int kSumOff = kMaxOff + kDecWarps * 8 * NT * 4;
  static constexpr int kMetaOff = kSumOff + kDecWarps * 8 * NT * 4;              // int [stages][8]
  static constexpr int kBarOff = kMetaOff + kStages * kDec8Groups * 4;
  static constexpr int kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr int kTeam = (kMiscOff + 64 + 1023) / 1024 * 1024;   // (swizzled tiles start on 1024 bytes)
  static constexpr int kBytes = kTeam * kDec8Teams<BF16, NT>;
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int slot, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(0), "r"(slot), "r"(head), "r"(page)
      : "memory");
}
// `bytes` (a multiple of 16) from a 16-byte aligned address
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
// fp16 pairs of the codes in bytes 0, 1 and 2, 3
template <bool E5M2>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E5M2)
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e5m2x2 %0, a;\n cvt.rn.f16x2.e5m2x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  else
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

template <bool BF16, int D, int NT, bool E5M2>
__global__ void __launch_bounds__(kDecThreads * kDec8Teams<BF16, NT>, 1) fa_decode8_kernel(const __grid_constant__ Decode8Params params) {
  const DecodeCore& p = params.c;
  using SM = Decode8Smem<BF16, D, NT>;
  using P = typename SM::P;
  constexpr int NS = SM::kStages;
  constexpr int KC = D / 16;                   // 16-byte chunks of a row
  extern __shared__ __align__(1024) uint8_t smem_all[];
  const int team = threadIdx.x / kDecThreads;
  uint8_t* smem = smem_all + team * SM::kTeam;
  const uint32_t sbase = smem_u32(smem);
  const int warp = (threadIdx.x % kDecThreads) >> 5, lane = threadIdx.x & 31;
  const int cta = team * gridDim.x + blockIdx.x;     // as the schedule counts: few ranges get an SM each
  auto FULL = [&](int s) { return sbase + SM::kBarOff + 8 * s; };
  auto EMPTY = [&](int s) { return sbase + SM::kBarOff + 8 * (NS + s); };
  int* s_meta = reinterpret_cast<int*>(smem + SM::kMetaOff);   // per stage: first key of each 16, or -1
  DecodeWalk* s_walk = reinterpret_cast<DecodeWalk*>(smem + SM::kMiscOff);
  int* s_len = reinterpret_cast<int*>(smem + SM::kMiscOff + 24);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + SM::kMiscOff + 28);
  int* s_top = reinterpret_cast<int*>(smem + SM::kMiscOff + 32);             // per warp: its largest scale byte of a value

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&params.tm_k);
    tma_prefetch_desc(&params.tm_v);
    for (int s = 0; s < NS; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), kDecWarps);
    }
    fence_mbar_init();
    *s_abort = 0;
  }
  // In this order: the join kernel may then read the lengths as soon as it runs.
  pdl_wait_prior();
  pdl_launch_dependents();
  if (warp == kDecWarps) decode_start<kDec8Tile>(p, cta, lane, s_walk, s_len);
  else if (cta == 0) decode_report(p);
  __syncthreads();
  DecodeWalk walk = *s_walk;
  const WaitCtx wc{s_abort, p.status, p.timeout_ns};
  const int box_shift = min(p.page_shift, 7);     // slots per copy
  const int box = 1 << box_shift;

  if (warp == kDecWarps) {
    // ============================================================ producer
    int len = *s_len;
    int it = 0;
    bool dead = false;
    const int nsub = kDec8Tile >> box_shift;          // copies of K (and V) per tile
    const uint32_t sub_bytes = (uint32_t)box * D;
    while (walk.left > 0 && !dead) {
      const DecodeSpan s = decode_span<kDec8Tile>(p, len);
      const int b = walk.b, hk = walk.unit / p.groups;
      const DecodePiece d = decode_step(walk, s.n, p.units);
      if (walk.b != b && walk.left > 0) len = decode_len(p, walk.b);
      const int t0 = d.t0, nt = d.nt;
      const int n_pages = (s.hi + (1 << p.page_shift) - 1) >> p.page_shift;
      auto look_up = [&](int c, int& id, int& slot, int& key) {
        decode_look_up<kDec8Tile>(p, s, b, hk, n_pages, c, (t0 + nt) * nsub, box_shift, id, slot, key);
      };
      int id, slot, key, id2 = -1, slot2 = 0, key2 = -1;
      const int per = 32 / nsub;                          // tiles per look-up
      look_up(t0 * nsub + lane, id, slot, key);
      for (int j = 0; j < nt; ++j, ++it) {
        const int in = j & (per - 1);
        if (in == 0 && j) id = id2, slot = slot2, key = key2;
        const int st = it % NS;
        bool ok = true;
        if (lane == 0 && it >= NS) ok = wait_bar(EMPTY(st), (it / NS - 1) & 1, wc);
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          dead = true;
          break;
        }
        const int sub = lane - in * nsub;
        const bool mine = sub >= 0 && sub < nsub && id >= 0;
        const unsigned live = __ballot_sync(0xffffffffu, mine);
        // lanes 0 to 7: the first key of each 16
        const int off = 16 * lane;
        const int first = __shfl_sync(0xffffffffu, key, in * nsub + ((off & (kDec8Tile - 1)) >> box_shift));
        if (lane < kDec8Groups) s_meta[st * kDec8Groups + lane] = first < 0 ? -1 : first + (off & (box - 1));
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(FULL(st), 2u * (sub_bytes + (uint32_t)box) * __popc(live));
        __syncwarp();
        if (mine) {
          const uint32_t dst = sbase + (uint32_t)st * 2 * SM::kHalf + (uint32_t)sub * sub_bytes;
          tma_load_4d(dst, &params.tm_k, FULL(st), slot, hk, id);
          tma_load_4d(dst + SM::kHalf, &params.tm_v, FULL(st), slot, hk, id);
          const long long at = (((long long)id * p.Hkv + hk) << p.page_shift) + slot;
          const uint32_t to = sbase + SM::kScaleOff + (uint32_t)st * 2 * kDec8Tile + (uint32_t)sub * box;
          bulk_load(to, params.k_scale + at, box, FULL(st));
          bulk_load(to + kDec8Tile, params.v_scale + at, box, FULL(st));
        }
        // the next look-up, a look-up's tiles ahead of its use
        if (in == 0) look_up((t0 + j + per) * nsub + lane, id2, slot2, key2);
      }
    }
    // Every copy lands before the CTA ends, whether or not some wait expired.
    if (lane == 0)
      for (int i = max(0, it - NS); i < it; ++i) drain_bar(FULL(i % NS), (i / NS) & 1, wc.timeout);
    return;
  }

  // ============================================================ consumers
  constexpr int DC = D / 64;                         // 16-channel chunks of this warp's quarter of O
  const int g = lane >> 2, t4 = lane & 3;
  P* s_p = reinterpret_cast<P*>(smem + SM::kPOff);
  uint2* s_q = reinterpret_cast<uint2*>(smem + SM::kQOff);
  float* s_fac = reinterpret_cast<float*>(smem + SM::kFacOff);
  float* s_max = reinterpret_cast<float*>(smem + SM::kMaxOff);
  float* s_sum = reinterpret_cast<float*>(smem + SM::kSumOff);
  auto sync = [&]() { named_sync(1 + 2 * team, 32 * kDecWarps); };
  // Key r of a stage is row r, D bytes; its 16-byte chunk c lies at place c ^ turn(r) (128-byte swizzle
  // for rows of 128 bytes, 64-byte swizzle for rows of 64).
  auto turn = [](int r) { return (uint32_t)(D == 128 ? r & 7 : (r >> 1) & 3); };
  // this lane's row of each ldmatrix: of K keys 0-7, 8-15 at chunk c, the same at chunk c + 1; of V keys
  // 0-7 .. 24-31 at one chunk
  const uint32_t krow = (uint32_t)(32 * warp + (lane & 15)) * D;
  const uint32_t kturn = turn(lane & 15), kodd = lane >> 4;
  const uint32_t vrow = SM::kHalf + (uint32_t)lane * D, vturn = turn(lane);

  int next_len = *s_len;
  int it = 0;
  bool dead = false;
  auto first_row = [&](const DecodeWalk& w) {
    return ((long long)w.b * p.Hkv + w.unit / p.groups) * p.rows + (w.unit % p.groups) * 8 * NT;
  };
  while (walk.left > 0) {
    const int len = next_len, rg = walk.unit % p.groups, b = walk.b;
    const long long row0 = first_row(walk);
    const DecodeSpan s = decode_span<kDec8Tile>(p, len);
    const DecodePiece d = decode_step(walk, s.n, p.units);
    if (walk.left > 0) {           // what the next unit will want: its length, and Q on its way to L1
      if (walk.b != b) next_len = decode_len(p, walk.b);
      if (warp == 0) {
        const uint8_t* x = reinterpret_cast<const uint8_t*>(p.q + first_row(walk) * D);
        const int bytes = min(8 * NT, p.rows - (walk.unit % p.groups) * 8 * NT) * D * 2;
        for (int i = 128 * lane; i < bytes; i += 128 * 32)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(x + i));
      }
    }
    if (d.nt == 0) continue;       // nothing but the charge
    const int rows = min(8 * NT, p.rows - rg * 8 * NT);

    // Q as the B operand: lane (g, t4) holds row g, channels 4 t4 .. 4 t4 + 3 of every chunk, as fp16;
    // fac: what its scores are multiplied by
    uint2 qf[SM::kQShared ? 1 : NT][SM::kQShared ? 1 : KC];
    float fac[NT][2];
    auto load_q = [&](int n, uint2 (&x)[KC]) {
      const int row = n * 8 + g;
      const uint2* src = reinterpret_cast<const uint2*>(p.q + (row0 + row) * D) + t4;
#pragma unroll
      for (int c = 0; c < KC; ++c) x[c] = row < rows ? src[4 * c] : make_uint2(0, 0);
      if (!BF16) return p.scale_log2;
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < KC; ++c) top = max_u16x2(max_u16x2(top, x[c].x & 0x7FFF7FFFu), x[c].y & 0x7FFF7FFFu);
      top = max(top & 0xFFFFu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max((int)(top >> 7), 127 - 100) - 127 - 14;         // the row's largest is below 2^(e + 15)
      const float f = __uint_as_float((uint32_t)(127 - e) << 23);       // (-114 <= e <= 114)
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        x[c].x = pack_f16x2(lo16_f32<true>(x[c].x) * f, hi16_f32<true>(x[c].x) * f);
        x[c].y = pack_f16x2(lo16_f32<true>(x[c].y) * f, hi16_f32<true>(x[c].y) * f);
      }
      return p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
    };
    if constexpr (SM::kQShared) {   // (the last unit's reads of it lie before its last barrier)
      for (int n = warp; n < NT; n += kDecWarps) {
        uint2 x[KC];
        const float f = load_q(n, x);
#pragma unroll
        for (int c = 0; c < KC; ++c) s_q[(n * KC + c) * 32 + lane] = x[c];
        if (t4 == 0) s_fac[n * 8 + g] = f;
      }
      sync();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(s_fac + n * 8 + 2 * t4);
        fac[n][0] = f.x, fac[n][1] = f.y;
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float f = load_q(n, qf[n]);
        fac[n][0] = __shfl_sync(0xffffffffu, f, 8 * t4);
        fac[n][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
      }
    }
    const int drafts = p.ancestors ? decode_drafts(p, b, len) : 0;
    const int tok_min = p.ancestors ? len - drafts - 1 : len - p.Sq;      // as in fa_decode_kernel
    const int low_max = p.pre_tokens >= 0 ? len - 1 - p.pre_tokens : 0;   // lowest key that all rows see

    uint32_t far = 0;                // value scales below this byte are far from one that the references followed
    float o[NT][DC][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = kNoScore;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < DC; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

    for (int j = 0; j < d.nt; ++j, ++it) {
      const int st = it % NS;
      // (after an expired wait: the barriers below still see every warp, the answer is void)
      if (!dead) dead = !__all_sync(0xffffffffu, wait_bar(FULL(st), (it / NS) & 1, wc));
      const uint32_t base = sbase + (uint32_t)st * 2 * SM::kHalf;
      const int* meta = s_meta + st * kDec8Groups;
      const uint8_t* scales = smem + SM::kScaleOff + st * 2 * kDec8Tile;
      float c[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[u][n][e] = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < KC / 2; ++k2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t r[4], a0[4], a1[4];
          ldmatrix4(base + krow + u * 16 * D + (((2 * k2 + kodd) ^ kturn) << 4), r);
          codes4<E5M2>(r[0], a0[0], a0[2]);
          codes4<E5M2>(r[1], a0[1], a0[3]);
          codes4<E5M2>(r[2], a1[0], a1[2]);
          codes4<E5M2>(r[3], a1[1], a1[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 x = SM::kQShared ? s_q[(n * KC + 2 * k2) * 32 + lane] : qf[SM::kQShared ? 0 : n][SM::kQShared ? 0 : 2 * k2];
            const uint2 y = SM::kQShared ? s_q[(n * KC + 2 * k2 + 1) * 32 + lane] : qf[SM::kQShared ? 0 : n][SM::kQShared ? 0 : 2 * k2 + 1];
            mma_16x8<false>(c[u][n], a0, x.x, x.y);
            mma_16x8<false>(c[u][n], a1, y.x, y.y);
          }
        }
      }
      // scores in log2 units with the value's exponent added; lane (g, t4): keys g (c0, c1) and g + 8
      // (c2, c3) of each 16, rows 2 t4, 2 t4 + 1
      float over = -INFINITY;        // the most that one exceeds its row's reference by
      float back[2][2];              // 2^-e of the lane's keys' values
      bool odd = false;              // whether one of them is large, not finite, or far
      const uint32_t near = min(far, kLargeScale);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int kq = meta[2 * warp + u];
        // 16 keys that were not copied (their codes are stale) lie past every row's token
        const int key0 = kq < 0 ? 0x7FFFFF00 : kq;
        const bool all = key0 + 15 <= tok_min && key0 >= low_max;
        float kf[2], ve[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int at = 32 * warp + 16 * u + 8 * x + g;
          uint32_t ks = scales[at], vs = scales[kDec8Tile + at];
          if (!all) {                // scales of keys that no row sees may be anything
            const int key = key0 + g + 8 * x;
            if (key >= s.hi || key < s.lo) ks = vs = 127;
          }
          odd = odd || vs - near >= kLargeScale - near;    // (unsigned: below `near`, or from kLargeScale on)
          if (vs == kScaleNone) vs = 127;
          kf[x] = scale_of(ks);
          ve[x] = (float)((int)vs - 127);
          back[u][x] = __uint_as_float((254u - vs) << 23);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[u][n][e] = fmaf(c[u][n][e] * fac[n][e & 1], kf[e >> 1], ve[e >> 1]);
        if (!all) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + g + 8 * (e >> 1);
              const int i = p.Sq == 1 ? 0 : (rg * 8 * NT + n * 8 + 2 * t4 + (e & 1)) % p.Sq;
              const int t = tok_min + (p.ancestors ? 0 : i);
              bool see = key <= t && (p.pre_tokens < 0 || key >= t - p.pre_tokens);
              if (p.ancestors && !see) see = decode_ancestor(p, b, drafts, i, key - t - 1);
              if (!see) c[u][n][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) over = fmaxf(over, c[u][n][e] - m[n][e & 1]);   // (NaN is dropped)
      }
      if (named_or(2 + 2 * team, 32 * kDecWarps, over > kMaxOver + kLift<false>)) {   // the references move up
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float mx[2] = {fmaxf(fmaxf(c[0][n][0], c[0][n][2]), fmaxf(c[1][n][0], c[1][n][2])),
                         fmaxf(fmaxf(c[0][n][1], c[0][n][3]), fmaxf(c[1][n][1], c[1][n][3]))};
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], w));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], w));
          }
          if (g == 0) *reinterpret_cast<float2*>(s_max + (warp * NT + n) * 8 + 2 * t4) = make_float2(mx[0], mx[1]);
        }
        uint32_t most = 0;             // (of scales that are not large it does not matter)
        if (__any_sync(0xffffffffu, odd)) {
          const int r = 32 * warp + lane, first = meta[r >> 4], key = first + (r & 15);
          const uint32_t vs = first >= 0 && key >= s.lo && key < s.hi ? scales[kDec8Tile + r] : 0;
          most = __reduce_max_sync(0xffffffffu, vs == kScaleNone ? 0 : vs);
        }
        if (lane == 0) s_top[warp] = (int)most;
        sync();
        const int4 tops = *reinterpret_cast<const int4*>(s_top);
        if (const int top = max(max(tops.x, tops.y), max(tops.z, tops.w)) - kFarScales; top > (int)far) {
          far = (uint32_t)top;
          odd = true;                  // (this tile's own keys may be far from those that the references now follow)
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float top[2] = {m[n][0], m[n][1]}, f[2];
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            const float2 x = *reinterpret_cast<const float2*>(s_max + (w * NT + n) * 8 + 2 * t4);
            top[0] = fmaxf(top[0], x.x - kLift<false>);
            top[1] = fmaxf(top[1], x.y - kLift<false>);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float by = m[n][e] - top[e], a = ex2_floor(by);
            f[e] = ex2_approx(by);
            m[n][e] = top[e];
            l[n][e] *= ex2_approx(by - a);                 // (1 but where 2^by is no fp32 number)
            l[n][e] *= ex2_approx(a);
          }
#pragma unroll
          for (int i = 0; i < DC; ++i) {
            o[n][i][0] *= f[0];
            o[n][i][1] *= f[1];
            o[n][i][2] *= f[0];
            o[n][i][3] *= f[1];
          }
        }
      }
      if (__any_sync(0xffffffffu, odd)) {
        // The weights of these keys join the sum here, without their values' exponents.  Values that are not
        // finite: P becomes 2^100, an fp16 infinity, which times the row's codes of 0 is NaN.  (What a row does
        // not see stays -infinity, a NaN key's score NaN; |m| 2^-22: more than a rounding of m.)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t vs = scales[kDec8Tile + 32 * warp + 16 * u + 8 * x + g];
            if (vs >= far && vs != kScaleNone) continue;
            const float e_v = vs == kScaleNone ? 0.f : (float)((int)vs - 127);
            back[u][x] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& y = c[u][n][2 * x + e];
                l[n][e] += ex2_approx(y - e_v - m[n][e]);
                if (vs == kScaleNone && y > -INFINITY) y = m[n][e] + fmaxf(100.f, fabsf(m[n][e]) * 0x1p-22f);
              }
          }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float p0 = ex2_approx(c[u][n][0] - m[n][0]), p1 = ex2_approx(c[u][n][1] - m[n][1]);
          const float p2 = ex2_approx(c[u][n][2] - m[n][0]), p3 = ex2_approx(c[u][n][3] - m[n][1]);
          l[n][0] = fmaf(p0, back[u][0], fmaf(p2, back[u][1], l[n][0]));
          l[n][1] = fmaf(p1, back[u][0], fmaf(p3, back[u][1], l[n][1]));
          const uint32_t h0 = pack_f16x2(p0, p1), h1 = pack_f16x2(p2, p3);
          P& at = s_p[((2 * warp + u) * NT + n) * 32 + lane];
          if constexpr (BF16)
            at = make_uint2(transpose8(h0), transpose8(h1));
          else
            at = make_uint4(transpose8(h0), transpose8(h1), transpose8(pack_residual_x2(p0, p1, h0, false)),
                            transpose8(pack_residual_x2(p2, p3, h1, false)));
        }
      sync();
      // Keys that no row sees have P = 0, and their V may hold anything (or be stale): it becomes 0.
      bool whole = true;
#pragma unroll
      for (int q = 0; q < kDec8Groups; ++q) whole = whole && meta[q] >= s.lo && meta[q] + 16 <= s.hi;
      // The tile's sum starts from zero and is added to O by itself, as in fa_decode_kernel.
      float sum[NT][DC][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < DC; ++i) sum[n][i][0] = sum[n][i][1] = sum[n][i][2] = sum[n][i][3] = 0.f;
#pragma unroll
      for (int q2 = 0; q2 < kDec8Groups / 2; ++q2) {
        uint32_t v[2][DC][4];
#pragma unroll
        for (int i = 0; i < DC; ++i) {
          uint32_t r[4];
          ldmatrix4_trans(base + vrow + q2 * 32 * D + (((uint32_t)(warp * DC + i) ^ vturn) << 4), r);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            // bytes: even channel of two keys, odd channel of the two
            codes4<E5M2>(__byte_perm(r[2 * u], 0, 0x3120), v[u][i][0], v[u][i][1]);
            codes4<E5M2>(__byte_perm(r[2 * u + 1], 0, 0x3120), v[u][i][2], v[u][i][3]);
          }
        }
        if (!whole) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int k0 = meta[2 * q2 + u];
            auto seen = [&](int k) { return k0 >= 0 && k0 + k >= s.lo && k0 + k < s.hi; };
            const uint32_t keep0 = (seen(2 * t4) ? 0xffffu : 0u) | (seen(2 * t4 + 1) ? 0xffff0000u : 0u);
            const uint32_t keep1 = (seen(2 * t4 + 8) ? 0xffffu : 0u) | (seen(2 * t4 + 9) ? 0xffff0000u : 0u);
#pragma unroll
            for (int i = 0; i < DC; ++i) {
              v[u][i][0] &= keep0;
              v[u][i][1] &= keep0;
              v[u][i][2] &= keep1;
              v[u][i][3] &= keep1;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const P pp = s_p[((2 * q2 + u) * NT + n) * 32 + lane];
#pragma unroll
            for (int i = 0; i < DC; ++i) mma_16x8<false>(sum[n][i], v[u][i], pp.x, pp.y);
            if constexpr (!BF16) {
#pragma unroll
              for (int i = 0; i < DC; ++i) mma_16x8<false>(sum[n][i], v[u][i], pp.z, pp.w);
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < DC; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][i][e] += sum[n][i][e];
      // A warp that gave up hands back no stage, as in fa_decode_kernel.
      __syncwarp();
      if (lane == 0 && !dead) mbar_arrive(EMPTY(st));
    }

    // ---- the unit's sums; each warp writes its channels
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
      if (g == 0) *reinterpret_cast<float2*>(s_sum + (warp * NT + n) * 8 + 2 * t4) = make_float2(l[n][0], l[n][1]);
    }
    sync();
    const bool direct = d.t0 == 0 && d.nt == s.n;
    const long long part0 = (2LL * cta + (d.t0 == 0 ? 1 : 0)) * (8 * NT);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float2 x = *reinterpret_cast<const float2*>(s_sum + (w * NT + n) * 8 + 2 * t4);
        sum[0] += x.x;
        sum[1] += x.y;
      }
      // lane (g, t4): rows 2 t4 and 2 t4 + 1, channels 2 g and 2 g + 1 of each chunk
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = n * 8 + 2 * t4 + e;
        if (direct) {
          const float inv = sum[e] > 0.f ? 1.f / sum[e] : 0.f;
          if (row < rows) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (row0 + row) * D + 16 * warp * DC) + g;
#pragma unroll
            for (int i = 0; i < DC; ++i) dst[8 * i] = pack16x2<BF16>(o[n][i][e] * inv, o[n][i][e + 2] * inv);
          }
        } else {
          float2* dst = reinterpret_cast<float2*>(p.part_o + (part0 + row) * D + 16 * warp * DC) + g;
#pragma unroll
          for (int i = 0; i < DC; ++i) dst[8 * i] = make_float2(o[n][i][e], o[n][i][e + 2]);
        }
        if (warp == 0 && g == 0) {
          if (!direct) p.part_ml[part0 + row] = make_float2(m[n][e], sum[e]);
          else if (row < rows)
            p.lse[row0 + row] = sum[e] == 0.f ? INFINITY : (m[n][e] + log2f(sum[e])) * 0.6931471805599453f;   // (NaN stays)
        }
      }
    }
  }
}

}  // namespace fa
