// fa_decode_ext with many rows per KV head (a tree of drafts, a chunk of a prompt,
// large groups): the schedule, the pieces and the join of fa_decode.cuh with the
// tcgen05 tensor cores.
//
// Past about 32 rows the warp-level products of fa_decode_kernel take longer than
// the keys' bytes (1.4 us a row for 16 sequences of 4096 tokens on 8 KV heads).
// Here up to 128 rows are the lanes of one accumulator, a row per softmax thread,
// and a tile of 128 keys costs about 1000 cycles of the tensor cores whatever the
// rows, below the 2900 that its 64 KB take from memory (an 8-bit tile: 1450); a
// unit of up to 256 rows has two such slots, which share every key tile.
//
//   * One CTA per SM; per slot four softmax warps, a producer warp, a warp whose
//     first lane issues the MMAs, and over an 8-bit cache four converter warps.
//     All hand-offs are mbarriers with bounded waits; no role waits for another in
//     any other way, so that an expired wait ends every role by the abort flag.
//   * Loads K(0), V(0), K(1), ... go through one ring of operand tiles (128 keys,
//     D / 64 chunks of 64 channels, 128-byte swizzle).  A 16-bit tile comes by TMA, a box
//     per page part and chunk; an 8-bit one comes as codes into a second ring, and
//     the converters write it as fp16 into the operand ring.
//   * The K codes of a tile are multiplied by 2^(e_k - E_k), E_k the largest exponent
//     of its seen keys, which leaves one factor per tile for the scores.  (Exact while
//     a row's scale is within 2^15, of e5m2 2^8, of the tile's largest; of smaller rows what
//     is below 2^-33 of the largest key is lost.)  Values alike with E_v, which joins the
//     exponent of the probabilities as in fa_decode8.cuh, but only in tiles whose values'
//     scales are within those limits, so that every product's operand is exact; in others
//     the codes stay and the softmax threads take each key's exponent, which is slow.
//   * S(t, j + 1) is issued behind P V (t, j), so that its commit says that O is at rest:
//     the softmax threads may then move their references and rescale O.
//   * P is written over S: as a hi + lo pair of the cache's type (16-bit: 64 + 64 columns,
//     which takes the upper half of S first), or as one fp16 (8-bit).
//   * Up to kWideFlush tiles of a piece add up in TMEM, where the adder cuts off what it adds
//     (about 2^-24 of the sum each 16 keys, always towards zero: 2^-15 over 8192 keys);
//     then the softmax threads add O to the piece's place in scratch in fp32.
#pragma once
#include <type_traits>

#include "fa_decode8.cuh"

namespace fa {

constexpr int kWideTile = 128;
constexpr int kWideInfo = 8;       // tiles whose keys and scales are kept: a producer is at most six ahead

constexpr int kWideFlush = 64;     // tiles that add up in TMEM

struct WideParams {
  DecodeCore c;
  const uint8_t* k_scale;          // 8-bit caches
  const uint8_t* v_scale;
  int e5m2;
  CUtensorMap tm_k;                // 16-bit: (64 channels, slots, D / 64, heads, pages); 8-bit: (D, slots, heads, pages)
  CUtensorMap tm_v;
};

struct WideTileInfo {              // of an 8-bit tile
  float k_scale;                   // 2^E_k
  float v_exp;                     // E_v
  float v_back;                    // 2^-E_v
  int each;                        // the values' exponents are taken key by key
};

template <int D, bool EIGHT, int SLOTS>
struct WideSmem {
  static constexpr int kOp = 128 * D * 2;                        // an operand tile: Q of a slot, K or V
  static constexpr int kStages = EIGHT ? (D == 128 ? 3 : 4) : (D == 128 ? (SLOTS == 2 ? 5 : 6) : 10);
  static constexpr int kRawStages = !EIGHT ? 0 : D == 128 ? (SLOTS == 2 ? 3 : 5) : 8;
  static constexpr int kRaw = 128 * D;                           // codes of K or V of a tile
  static constexpr int kRingOff = SLOTS * kOp;
  static constexpr int kRawOff = kRingOff + kStages * kOp;
  static constexpr int kScaleOff = kRawOff + kRawStages * kRaw;  // bytes [kWideInfo][K, V][128]
  static constexpr int kMetaOff = kScaleOff + (EIGHT ? kWideInfo * 256 : 0);     // int [kWideInfo][8]
  static constexpr int kInfoOff = kMetaOff + kWideInfo * 32;     // WideTileInfo [kWideInfo]
  static constexpr int kBarOff = kInfoOff + kWideInfo * 16;
  static constexpr int kBars = 2 * kStages + 2 * kRawStages + 3 * SLOTS + 2;
  static constexpr int kMiscOff = kBarOff + kBars * 8;
  static constexpr int kBytes = kMiscOff + 64;
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};
template <bool EIGHT, int SLOTS>
constexpr int kWideThreads = 32 * (4 * SLOTS + 2 + (EIGHT ? 4 : 0));

__device__ __forceinline__ void tma_load_5d_chunk(uint32_t dst, const void* tmap, uint32_t bar, int slot, int chunk,
                                                  int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(0), "r"(slot), "r"(chunk), "r"(head), "r"(page)
      : "memory");
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <bool BF16, int D, bool EIGHT, int SLOTS>
__global__ void __launch_bounds__(kWideThreads<EIGHT, SLOTS>, 1) fa_wide_kernel(const __grid_constant__ WideParams params) {
  const DecodeCore& p = params.c;
  using SM = WideSmem<D, EIGHT, SLOTS>;
  constexpr int NS = SM::kStages, RS = EIGHT ? SM::kRawStages : 1;
  constexpr int kRows = 128 * SLOTS;
  constexpr bool kP16 = EIGHT || !BF16;               // the type of P (and of Q, K and V as operands): fp16 or bf16
  constexpr float kLiftP = kLift<!kP16>;
  constexpr int kProducer = 4 * SLOTS, kIssuer = kProducer + 1, kConvert = kIssuer + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto BAR = [&](int i) { return sbase + SM::kBarOff + 8 * i; };
  auto FULL = [&](int s) { return BAR(s); };                       // an operand tile is there
  auto EMPTY = [&](int s) { return BAR(NS + s); };                 // its MMAs are done
  auto RFULL = [&](int s) { return BAR(2 * NS + s); };             // codes are there
  auto REMPTY = [&](int s) { return BAR(2 * NS + RS + s); };       // they are converted
  constexpr int kB = 2 * NS + 2 * SM::kRawStages;
  auto SFULL = [&](int t) { return BAR(kB + t); };                 // S of slot t
  auto PREADY = [&](int t) { return BAR(kB + SLOTS + t); };        // P of slot t, O rescaled
  auto OFULL = [&](int t) { return BAR(kB + 2 * SLOTS + t); };     // O of slot t, at a piece's end
  const uint32_t QREADY = BAR(kB + 3 * SLOTS), DRAIN = BAR(kB + 3 * SLOTS + 1);
  int* s_meta = reinterpret_cast<int*>(smem + SM::kMetaOff);       // per tile: first key of each 16, or -1
  WideTileInfo* s_info = reinterpret_cast<WideTileInfo*>(smem + SM::kInfoOff);
  DecodeWalk* s_walk = reinterpret_cast<DecodeWalk*>(smem + SM::kMiscOff);
  int* s_len = reinterpret_cast<int*>(smem + SM::kMiscOff + 24);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + SM::kMiscOff + 28);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + SM::kMiscOff + 32);

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&params.tm_k);
    tma_prefetch_desc(&params.tm_v);
    for (int s = 0; s < NS; ++s) {
      mbar_init(FULL(s), EIGHT ? 4 : 1);
      mbar_init(EMPTY(s), 1);
    }
    if constexpr (EIGHT)
      for (int s = 0; s < RS; ++s) {
        mbar_init(RFULL(s), 1);
        mbar_init(REMPTY(s), 4);
      }
    for (int t = 0; t < SLOTS; ++t) {
      mbar_init(SFULL(t), 1);
      mbar_init(PREADY(t), 4);
      mbar_init(OFULL(t), 1);
    }
    mbar_init(QREADY, 4 * SLOTS);
    mbar_init(DRAIN, 1);
    fence_mbar_init();
    *s_abort = 0;
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(s_tmem), 256 * SLOTS);
    tmem_relinquish();
    tc_fence_before();
  }
  // In this order: the join kernel may then read the lengths as soon as it runs.
  pdl_wait_prior();
  pdl_launch_dependents();
  if (warp == kProducer) decode_start<kWideTile>(p, blockIdx.x, lane, s_walk, s_len);
  else if (blockIdx.x == 0 && warp < kDecWarps) decode_report(p);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  DecodeWalk walk = *s_walk;
  int next_len = *s_len;
  const WaitCtx wc{s_abort, p.status, p.timeout_ns};
  const int box_shift = min(p.page_shift, 7);     // slots per copy
  const int box = 1 << box_shift;
  // The next piece: its sequence, unit, span and tiles, and its number among this role's tiles.
  struct Piece {
    int b, unit, len;
    DecodeSpan s;
    DecodePiece d;
  };
  auto next_piece = [&](Piece& x) {
    while (walk.left > 0) {
      x.len = next_len;
      x.b = walk.b;
      x.unit = walk.unit;
      x.s = decode_span<kWideTile>(p, x.len);
      x.d = decode_step(walk, x.s.n, p.units);
      if (walk.b != x.b && walk.left > 0) next_len = decode_len(p, walk.b);
      if (x.d.nt) return true;
    }
    return false;
  };
  Piece x;

  if (warp == kProducer) {
    // ============================================================ producer
    int tile = 0;                                     // of this CTA; its loads are 2 tile (K) and 2 tile + 1 (V)
    bool dead = false;
    const int nsub = kWideTile >> box_shift;
    while (!dead && next_piece(x)) {
      const int hk = x.unit / p.groups;
      const int n_pages = (x.s.hi + (1 << p.page_shift) - 1) >> p.page_shift;
      auto look_up = [&](int c, int& id, int& slot, int& key) {
        decode_look_up<kWideTile>(p, x.s, x.b, hk, n_pages, c, (x.d.t0 + x.d.nt) * nsub, box_shift, id, slot, key);
      };
      int id, slot, key, id2 = -1, slot2 = 0, key2 = -1;
      const int per = 32 / nsub;                          // tiles per look-up
      look_up(x.d.t0 * nsub + lane, id, slot, key);
      for (int j = 0; j < x.d.nt && !dead; ++j, ++tile) {
        const int in = j & (per - 1);
        if (in == 0 && j) id = id2, slot = slot2, key = key2;
        const int sub = lane - in * nsub;
        const bool mine = sub >= 0 && sub < nsub && id >= 0;
        const unsigned live = __ballot_sync(0xffffffffu, mine);
        const int off = 16 * lane;
        const int first = __shfl_sync(0xffffffffu, key, in * nsub + ((off & (kWideTile - 1)) >> box_shift));
        const int at = tile % kWideInfo;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const int ld = 2 * tile + kind;
          const int st = ld % (EIGHT ? RS : NS), n = ld / (EIGHT ? RS : NS);
          bool ok = true;
          if (lane == 0 && n > 0) ok = wait_bar(EIGHT ? REMPTY(st) : EMPTY(st), (n - 1) & 1, wc);
          if (!__shfl_sync(0xffffffffu, ok, 0)) {
            dead = true;
            // (the loads up to here land below; `tile` counts whole tiles, a K without its V is waited for here)
            if (kind == 1 && lane == 0) {
              const int k = ld - 1, ks = k % (EIGHT ? RS : NS);
              drain_bar(EIGHT ? RFULL(ks) : FULL(ks), (k / (EIGHT ? RS : NS)) & 1, wc.timeout);
            }
            break;
          }
          // (the place of tile - kWideInfo: all its readers are done, see kWideInfo)
          if (kind == 0 && lane < 8) s_meta[at * 8 + lane] = first < 0 ? -1 : first + (off & (box - 1));
          __syncwarp();
          const uint32_t bar = EIGHT ? RFULL(st) : FULL(st);
          const uint32_t each = EIGHT ? (uint32_t)box * D + (kind == 0 ? 2u * box : 0u) : (uint32_t)box * D * 2;
          if (lane == 0) mbar_arrive_expect_tx(bar, each * __popc(live));
          __syncwarp();
          if (mine) {
            const void* tm = kind ? &params.tm_v : &params.tm_k;
            if constexpr (EIGHT) {
              tma_load_4d(sbase + SM::kRawOff + st * SM::kRaw + sub * box * D, tm, bar, slot, hk, id);
              if (kind == 0) {       // both scales with K: the softmax needs the values' before V
                const long long from = (((long long)id * p.Hkv + hk) << p.page_shift) + slot;
                const uint32_t to = sbase + SM::kScaleOff + at * 256 + sub * box;
                bulk_load(to, params.k_scale + from, box, bar);
                bulk_load(to + 128, params.v_scale + from, box, bar);
              }
            } else {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_5d_chunk(sbase + SM::kRingOff + st * SM::kOp + c * (128 * 128) + sub * box * 128, tm, bar, slot, c, hk, id);
            }
          }
        }
        // the next look-up, a look-up's tiles ahead of its use
        if (in == 0 && !dead) look_up((x.d.t0 + j + per) * nsub + lane, id2, slot2, key2);
        if (dead) break;
      }
    }
    // every copy lands before the CTA ends, whether or not some wait expired
    if (lane == 0) {
      constexpr int N = EIGHT ? RS : NS;
      const int end = 2 * tile;
      for (int i = max(0, end - N); i < end; ++i) drain_bar(EIGHT ? RFULL(i % N) : FULL(i % N), (i / N) & 1, wc.timeout);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // ============================================================ MMA issue
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_f16(128, 128, !kP16, false);
      constexpr uint32_t kIdescO = idesc_f16(128, D, !kP16, true);
      const uint64_t q0 = sw128_desc(sbase, 16, 1024);
      const uint64_t k0 = sw128_desc(sbase + SM::kRingOff, 16, 1024);
      const uint64_t v0 = sw128_desc(sbase + SM::kRingOff, 128 * 128, 1024);
      int tile = 0, piece = 0;
      bool ok = true;
      int p_phase = 0;                                 // of PREADY: tiles so far
      auto scores = [&](int t, int ld) {
        const uint64_t a = q0 + ((t * SM::kOp) >> 4), b = k0 + (((ld % NS) * SM::kOp) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
          mma_ss(tmem + 128 * t, a + off, b + off, kIdescS, kk > 0);
        }
        mma_commit(SFULL(t));
      };
      while (ok && next_piece(x)) {
        ok = wait_bar(QREADY, piece & 1, wc);
        if (ok) ok = wait_bar(FULL((2 * tile) % NS), ((2 * tile) / NS) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < SLOTS; ++t) scores(t, 2 * tile);
        mma_commit(EMPTY((2 * tile) % NS));
        for (int j = 0; j < x.d.nt && ok; ++j, ++tile, ++p_phase) {
          const int vl = 2 * tile + 1, kl = 2 * tile + 2;
          ok = wait_bar(FULL(vl % NS), (vl / NS) & 1, wc);
          const bool more = j + 1 < x.d.nt;
          for (int t = 0; t < SLOTS && ok; ++t) {
            ok = wait_bar(PREADY(t), p_phase & 1, wc);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = v0 + (((vl % NS) * SM::kOp) >> 4);
            const uint32_t o = tmem + 128 * SLOTS + 128 * t, s = tmem + 128 * t;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) mma_ts(o, s + 8 * kk, b + (kk * 2048 >> 4), kIdescO, j % kWideFlush || kk);
            if constexpr (!EIGHT) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) mma_ts(o, s + 64 + 8 * kk, b + (kk * 2048 >> 4), kIdescO, 1);
            }
            if (t == SLOTS - 1) mma_commit(EMPTY(vl % NS));
            if (!more) {
              mma_commit(OFULL(t));
              continue;
            }
            if (t == 0) ok = wait_bar(FULL(kl % NS), (kl / NS) & 1, wc);
            if (!ok) break;
            if (t == 0) tc_fence_after();
            scores(t, kl);
            if (t == SLOTS - 1) mma_commit(EMPTY(kl % NS));
          }
        }
        ++piece;
      }
      // whatever is in flight ends before the tensor memory and the tiles are given up
      mma_commit(DRAIN);
      drain_bar(DRAIN, 0, wc.timeout);
    }
    __syncwarp();
  } else if (EIGHT && warp >= kConvert) {
    // ============================================================ converters
    const int tid = threadIdx.x - 32 * kConvert;
    int tile = 0;
    bool dead = false;
    while (!dead && next_piece(x)) {
      for (int j = 0; j < x.d.nt && !dead; ++j, ++tile) {
        const int at = tile % kWideInfo;
        uint8_t* scales = smem + SM::kScaleOff + at * 256;
        const int* meta = s_meta + at * 8;
        int top_k = 0, top_v = 0;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const int ld = 2 * tile + kind, rs = ld % RS, st = ld % NS;
          if (!__all_sync(0xffffffffu, wait_bar(RFULL(rs), (ld / RS) & 1, wc))) dead = true;
          if (!dead && ld >= NS && !__all_sync(0xffffffffu, wait_bar(EMPTY(st), (ld / NS - 1) & 1, wc))) dead = true;
          if (dead) break;
          auto seen = [&](int r) {
            const int k = meta[r >> 4] < 0 ? -1 : meta[r >> 4] + (r & 15);
            return k >= x.s.lo && k < x.s.hi;
          };
          if (kind == 0) {           // every warp for itself: the largest exponents of the seen keys, the values' least
            int low_v = 255;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 32 * i + lane;
              if (!seen(r)) continue;
              const int ks = scales[r], vs = scales[128 + r];
              top_k = max(top_k, ks), top_v = max(top_v, vs), low_v = min(low_v, vs);
            }
            top_k = __reduce_max_sync(0xffffffffu, top_k);
            top_v = __reduce_max_sync(0xffffffffu, top_v);
            low_v = __reduce_min_sync(0xffffffffu, low_v);
            const bool each = top_v - low_v > (params.e5m2 ? 8 : 15);
            if (top_v == 0 || each) top_v = 0;                     // (0: the codes of V stay as they are)
            if (tid == 0)
              s_info[at] = WideTileInfo{scale_of(top_k), top_v ? (float)(top_v - 127) : 0.f,
                                        top_v ? __uint_as_float((uint32_t)(254 - top_v) << 23) : 1.f, each};
          }
          const uint8_t* raw = smem + SM::kRawOff + rs * SM::kRaw;
          const uint32_t op = sbase + SM::kRingOff + st * SM::kOp;
          const int top = kind ? top_v : top_k;
          auto convert = [&](auto format) {
            constexpr bool E5M2 = decltype(format)::value;
#pragma unroll 4
            for (int i = tid; i < 128 * (D / 16); i += 128) {
              const int r = i / (D / 16), c = i % (D / 16);
              const bool on = seen(r);
              uint4 w = *reinterpret_cast<const uint4*>(raw + i * 16);
              if (!on) w = make_uint4(0, 0, 0, 0);
              uint32_t h[8];
              codes4<E5M2>(w.x, h[0], h[1]);
              codes4<E5M2>(w.y, h[2], h[3]);
              codes4<E5M2>(w.z, h[4], h[5]);
              codes4<E5M2>(w.w, h[6], h[7]);
              if (top && on) {       // 2^(e - E) as an fp16, exactly, down to 2^-24
                const int e = (int)scales[128 * kind + r] - top;
                const uint32_t f = pack_f16x2(0.f, e < -126 ? 0.f : __uint_as_float((uint32_t)(127 + e) << 23)) >> 16;
                const uint32_t f2 = f | f << 16;
#pragma unroll
                for (int q = 0; q < 8; ++q) h[q] = mul_f16x2(h[q], f2);
              }
              const uint32_t to = op + (c >> 2) * (128 * 128) + r * 128;
              const uint32_t a = ((2 * (c & 3)) ^ (r & 7)) << 4, b = a ^ 16u;
              const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
              const bool swap = (c >> 2) & 1;      // (the two chunks of a row in the two orders: no bank twice)
              st_shared_v4(to + (swap ? b : a), swap ? hi : lo);
              st_shared_v4(to + (swap ? a : b), swap ? lo : hi);
            }
          };
          if (params.e5m2) convert(std::true_type{});
          else convert(std::false_type{});
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(FULL(st));
            mbar_arrive(REMPTY(rs));
          }
        }
      }
    }
  } else {
    // ============================================================ softmax: a row per thread
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;                 // of the slot
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 * t + lanes, tO = tmem + 128 * SLOTS + 128 * t + lanes;
    int tile = 0, piece = 0;
    bool dead = false;
    while (!dead && next_piece(x)) {
      const int hk = x.unit / p.groups, rg = x.unit % p.groups;
      const int r0 = rg * kRows + 128 * t;             // this slot's first row of the KV head
      const long long at0 = ((long long)x.b * p.Hkv + hk) * p.rows + r0;
      const bool mine = r0 + row < p.rows;
      // Q into its slot (the last piece's S products of it are done), as fp16 of a power of two times it
      // over an 8-bit cache
      float fac = p.scale_log2;
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (at0 + row) * D);
        uint4 w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w[c] = mine ? src[c] : make_uint4(0, 0, 0, 0);
        if constexpr (EIGHT && BF16) {
          uint32_t top = 0;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            top = max_u16x2(top, max_u16x2(w[c].x & 0x7FFF7FFFu, w[c].y & 0x7FFF7FFFu));
            top = max_u16x2(top, max_u16x2(w[c].z & 0x7FFF7FFFu, w[c].w & 0x7FFF7FFFu));
          }
          top = max(top & 0xFFFFu, top >> 16);
          const int e = max((int)(top >> 7), 127 - 100) - 127 - 14;       // as in fa_decode8_kernel
          const float f = __uint_as_float((uint32_t)(127 - e) << 23);
          auto half = [&](uint32_t u) { return pack_f16x2(lo16_f32<true>(u) * f, hi16_f32<true>(u) * f); };
#pragma unroll
          for (int c = 0; c < D / 8; ++c) w[c] = make_uint4(half(w[c].x), half(w[c].y), half(w[c].z), half(w[c].w));
          fac *= __uint_as_float((uint32_t)(127 + e) << 23);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          st_shared_v4(sbase + t * SM::kOp + (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4), w[c]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(QREADY);
      }
      const int drafts = p.ancestors ? decode_drafts(p, x.b, x.len) : 0;
      const int base = x.len - drafts;                                        // a tree's first draft
      const int i_row = p.Sq == 1 ? 0 : (r0 + row) % p.Sq;
      const int tok = p.ancestors ? base - 1 : x.len - p.Sq + i_row;          // keys up to it are seen
      const int all_hi = p.ancestors ? base - 1 : x.len - p.Sq;               // by every row
      const int all_lo = p.pre_tokens >= 0 ? x.len - 1 - p.pre_tokens : 0;    // and from here on
      const int low = p.pre_tokens >= 0 ? tok - p.pre_tokens : 0;
      float m = kNoScore, l = 0.f, m_acc = kNoScore;   // m_acc: the reference of what has left TMEM
      const bool direct = x.d.t0 == 0 && x.d.nt == x.s.n;
      // this row's place in scratch: a piece's answer, before that the sum that has left TMEM (of a unit that is
      // finished here the place of the one that begins after it)
      const long long part = (2LL * blockIdx.x + (x.d.t0 == 0 ? 1 : 0)) * kRows + 128 * t + row;
      uint4* acc = reinterpret_cast<uint4*>(p.part_o + part * D);
      auto plus = [&](uint4 a, float g, const uint32_t* u) {      // a g + u
        return make_uint4(__float_as_uint(fmaf(__uint_as_float(a.x), g, __uint_as_float(u[0]))),
                          __float_as_uint(fmaf(__uint_as_float(a.y), g, __uint_as_float(u[1]))),
                          __float_as_uint(fmaf(__uint_as_float(a.z), g, __uint_as_float(u[2]))),
                          __float_as_uint(fmaf(__uint_as_float(a.w), g, __uint_as_float(u[3]))));
      };

      for (int j = 0; j < x.d.nt; ++j, ++tile) {
        if (!__all_sync(0xffffffffu, wait_bar(SFULL(t), tile & 1, wc))) {
          dead = true;
          break;
        }
        tc_fence_after();
        const int* meta = s_meta + (tile % kWideInfo) * 8;
        const int4 ka = *reinterpret_cast<const int4*>(meta), kb = *reinterpret_cast<const int4*>(meta + 4);
        const int first = min(min(min(ka.x, ka.y), min(ka.z, ka.w)), min(min(kb.x, kb.y), min(kb.z, kb.w)));
        const int last = max(max(max(ka.x, ka.y), max(ka.z, ka.w)), max(max(kb.x, kb.y), max(kb.z, kb.w))) + 15;
        const bool all = first >= max(all_lo, 0) && last <= all_hi;
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
        if (!all) {
          auto group = [&](int k0) -> uint32_t {       // the keys of 16 that this row sees before a tree
            if (k0 < 0) return 0;
            const int n = min(max(tok + 1 - k0, 0), 16), z = min(max(low - k0, 0), 16);
            return ((1u << n) - 1u) & ~((1u << z) - 1u);
          };
          const int keys[8] = {ka.x, ka.y, ka.z, ka.w, kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) vis[c] = group(keys[2 * c]) | group(keys[2 * c + 1]) << 16;
          if (p.ancestors) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (max(keys[2 * c], keys[2 * c + 1]) + 15 < base) continue;
              // lane: one of the 32 keys; the warp's rows one by one
              const int k0 = lane < 16 ? keys[2 * c] : keys[2 * c + 1];
              const int draft = k0 < 0 ? -1 : k0 + (lane & 15) - base;
              int i = (r0 + (warp & 3) * 32) % p.Sq;
#pragma unroll 8
              for (int r = 0; r < 32; ++r) {
                const bool see = draft >= 0 && decode_ancestor(p, x.b, drafts, i, draft);
                const uint32_t bits = __ballot_sync(0xffffffffu, see);
                if (lane == r) vis[c] |= bits;
                if (++i == p.Sq) i = 0;
              }
            }
          }
          if constexpr (!EIGHT) {
            // V of keys that no row sees may hold anything: its rows become 0 (P is 0 there), by each slot
            const int k0 = keys[row >> 4], k = k0 < 0 ? -1 : k0 + (row & 15);
            const int ld = 2 * tile + 1;
            if (!__all_sync(0xffffffffu, wait_bar(FULL(ld % NS), (ld / NS) & 1, wc))) {
              dead = true;
              break;
            }
            if (k < x.s.lo || k >= x.s.hi) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                for (int q = 0; q < 8; ++q)
                  st_shared_v4(sbase + SM::kRingOff + (ld % NS) * SM::kOp + c * (128 * 128) + row * 128 + q * 16, make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
          }
        }
        WideTileInfo info{1.f, 0.f, 1.f, 0};
        if constexpr (EIGHT) info = s_info[tile % kWideInfo];
        const float f = fac * info.k_scale;
        const uint8_t* vs = smem + SM::kScaleOff + (tile % kWideInfo) * 256 + 128;
        // scores in log2 units, the values' exponents added
        auto load = [&](int c, float (&s)[32]) {
          uint32_t u[32];
          tmem_ld32(tS + 32 * c, u);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = fmaf(__uint_as_float(u[i]), f, info.v_exp);
          if (EIGHT && info.each) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] += (float)((int)vs[32 * c + i] - 127);
          }
          if (!all) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((vis[c] >> i) & 1u)) s[i] = -INFINITY;
          }
        };
        if (j && j % kWideFlush == 0) {
          const float g = ex2_approx(m_acc - m);
          m_acc = m;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[32];
            tmem_ld32(tO + 32 * c, u);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              acc[8 * c + q] = plus(j == kWideFlush ? make_uint4(0, 0, 0, 0) : acc[8 * c + q], g, u + 4 * q);
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float s[32];
          load(c, s);
#pragma unroll
          for (int i = 0; i < 32; i += 2) top = fmaxf(top, fmaxf(s[i], s[i + 1]));     // (NaN is dropped)
        }
        if (__any_sync(0xffffffffu, top - m > kMaxOver + kLiftP)) {                    // references move up
          const float to = top - m > kMaxOver + kLiftP ? top - kLiftP : m;
          const float g = ex2_approx(m - to);
          m = to;
          l *= g;
          if (j % kWideFlush) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t u[32];
              tmem_ld32(tO + 32 * c, u);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * g);
              tmem_st32(tO + 32 * c, u);
            }
          }
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        // chunk c as P: 16 registers of hi, 16 of lo
        auto exps = [&](int c, uint32_t (&hi)[16], uint32_t (&lo)[16]) {
          float s[32];
          load(c, s);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float a = ex2_approx(s[i] - m), b = ex2_approx(s[i + 1] - m);
            if (EIGHT && info.each) {
              const uint32_t va = vs[32 * c + i], vb = vs[32 * c + i + 1];
              if (a > 0.f) sum[0] = fmaf(a, __uint_as_float((254u - va) << 23), sum[0]);
              if (b > 0.f) sum[1] = fmaf(b, __uint_as_float((254u - vb) << 23), sum[1]);
            } else {
              sum[(i >> 1) & 3] += a + b;
            }
            hi[i / 2] = kP16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
            if constexpr (!EIGHT) lo[i / 2] = pack_residual_x2(a, b, hi[i / 2], !kP16);
          }
        };
        uint32_t h0[16], h1[16], lo[16];
        if constexpr (EIGHT) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {      // (chunk c lies over chunk c / 2 of S, read by then)
            exps(c, h0, lo);
            tmem_st16(tS + 16 * c, h0);
          }
        } else {
          // lo of the upper half over the upper half of S, its hi once the lower half has been read
          exps(2, h0, lo);
          uint32_t lo2[16];
          exps(3, h1, lo2);
          tmem_st16(tS + 64 + 32, lo);
          tmem_st16(tS + 64 + 48, lo2);
          uint32_t h[16];
          exps(0, h, lo);
          tmem_st16(tS, h);
          tmem_st16(tS + 64, lo);
          exps(1, h, lo);
          tmem_st16(tS + 16, h);
          tmem_st16(tS + 64 + 16, lo);
          tmem_st16(tS + 32, h0);
          tmem_st16(tS + 48, h1);
        }
        const float all_sum = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        l = EIGHT && !info.each ? fmaf(all_sum, info.v_back, l) : l + all_sum;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(PREADY(t));
      }
      if (dead) break;
      // ---- the piece's answer
      if (!__all_sync(0xffffffffu, wait_bar(OFULL(t), piece & 1, wc))) break;
      ++piece;
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const float g = ex2_approx(m_acc - m);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t u[32];
        tmem_ld32(tO + 32 * c, u);
        tmem_wait_ld();
        if (x.d.nt > kWideFlush) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint4 y = plus(acc[8 * c + q], g, u + 4 * q);
            u[4 * q] = y.x, u[4 * q + 1] = y.y, u[4 * q + 2] = y.z, u[4 * q + 3] = y.w;
          }
        }
        if (direct) {
          if (mine) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + (at0 + row) * D + 32 * c);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = pack16x2<BF16>(__uint_as_float(u[8 * q + 2 * e]) * inv, __uint_as_float(u[8 * q + 2 * e + 1]) * inv);
              dst[q] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        } else if (mine) {
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[8 * c + q] = make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
        }
      }
      if (mine) {
        if (direct) p.lse[at0 + row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : INFINITY;
        else p.part_ml[part] = make_float2(m, l);
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 256 * SLOTS);
  }
}

}  // namespace fa
