// fa_decode_ext with many rows per KV head (a tree of drafts, a chunk of a prompt,
// large groups): the schedule, the pieces and the join of fa_decode.cuh with the
// tcgen05 tensor cores.
//
// Past about 32 rows the warp-level products of fa_decode_kernel take longer than
// the keys' bytes (1.4 us a row for 16 sequences of 4096 tokens on 8 KV heads).
// Here up to 128 rows are the lanes of one accumulator, a row per softmax thread,
// and a tile of 128 keys costs about 1000 cycles of the tensor cores whatever the
// rows (1500 where P is a pair), below the 2900 that its 64 KB take from memory (an
// 8-bit tile: 1450).
//
//   * One CTA per SM with two accumulators and two groups of softmax warps, which take
//     turns with the tensor cores.  A unit of up to 256 rows has 128 in each and shares
//     every key tile; with up to 128 rows (SPLIT) both have all rows and take every other
//     tile, and the first group joins the two at a piece's end.
//   * A producer warp, a warp that issues the MMAs, and over an 8-bit cache six converter
//     warps.  All hand-offs are mbarriers with bounded waits; no role waits for another in
//     any other way, so that an expired wait ends every role by the abort flag.
//   * Loads K(0), V(0), K(1), ... go through one ring of operand tiles (128 keys,
//     D / 64 chunks of 64 channels, 128-byte swizzle).  A 16-bit tile comes by TMA, a box
//     per page part and chunk; an 8-bit one comes as codes into a second ring, and
//     the converters write it as fp16 into the operand ring.
//   * The K codes of a tile are multiplied by 2^(e_k - E_k), E_k the largest exponent
//     of its seen keys, which leaves one factor per tile for the scores; values alike
//     with E_v, which joins the exponent of the probabilities as in fa_decode8.cuh.
//     That is exact where the tile's scales are within 2^15, of e5m2 2^8, of each other.
//     In other tiles (the keys', the values', or both) the codes stay and the softmax
//     threads take each key's exponent, which is slow.  A row of zeros (e = -80) beside
//     others makes a tile one of those, and so does a row that is not finite (a value's
//     also all of the piece's tiles behind it: nothing says how large its others are).
//   * The next S of a group is issued behind its P V, so that its commit says that O is at
//     rest: the softmax threads may then move their references and rescale O.
//   * P is written over S, as a hi + lo pair of the operands' type (64 + 64 columns) or, over an
//     8-bit cache with bf16 answers, as one fp16.
//   * Up to kWideFlush tiles of a piece add up in TMEM, where the adder cuts off what it adds
//     (about 2^-24 of the sum each 16 keys, always towards zero: 2^-15 over 8192 keys);
//     then the softmax threads add O to a place in scratch in fp32.
//
// Measured (32 query heads on 8 KV heads of 128, bf16, with the join): 16 trees of up to 12
// drafts over up to 8192 tokens (48 rows) 71 us, 41 of which are the bytes', over 32768 tokens
// each 348 us, 6.2 TB/s; 4 trees of up to 64 (256 rows) over an 8-bit cache of up to 16384
// tokens 70 us, over 65536 each 260 us, 1058 TF/s; the same over a 16-bit cache 70 and 291 us.
// A prompt's last 512 of 4096 tokens over an 8-bit cache 66 us, 521 TF/s.
// A unit costs about 13000 cycles beside its tiles (rows in, the last P V, the groups' join, the
// answer out); with 256 rows a group's chain (S 512 cycles, softmax 2500, P V 512) sets the step,
// 4000 cycles a tile, half of which the tensor cores work; with up to 128 rows over an 8-bit cache
// the conversion does (16 trees of 24 drafts, 96 rows, 103 us over up to 8192 tokens, 441 over 32768
// each): 96 KB a tile through shared memory, which the S products want too.  The code of all roles
// together is more than the instruction cache likes: what few tiles need has loops of its own.
// With every tile taken key by key (a row of zeros in each) the 4 trees take 254 us instead of
// 70, the 16 of 96 rows 231 instead of 103.
#pragma once
#include <type_traits>

#include "fa_decode8.cuh"

namespace fa {

constexpr int kWideTile = 128;
constexpr int kWideInfo = 8;       // tiles whose keys and scales are kept: the producer is at most seven ahead

// A unit's own cost in tiles: its rows, its ends, its answer.  (16 trees of up to 12 drafts over up to 8192
// tokens: 90 us at 2, 78 at 3, 70 at 5, 69 at 8; 4 of up to 64 over an 8-bit cache 88, 86, 87, 89.)
constexpr int kWideCharge = 6;
constexpr int kWideFlush = 64;     // tiles that add up in TMEM
constexpr int kWideDrafts = 64;    // drafts whose ancestors are kept as words; of larger trees they are looked up tile by tile

struct WideParams {
  DecodeCore c;
  const uint8_t* k_scale;          // 8-bit caches
  const uint8_t* v_scale;
  int e5m2;
  float* gone;                     // [ctas][groups][128][D]: sums that have left the accumulators
  CUtensorMap tm_k;                // 16-bit: (64 channels, slots, D / 64, heads, pages); 8-bit: (D, slots, heads, pages)
  CUtensorMap tm_v;
};

struct alignas(16) WideTileInfo {  // of an 8-bit tile
  float k_scale;                   // 2^E_k
  float v_exp;                     // E_v
  float v_back;                    // 2^-E_v
  int flags;                       // kWide..., and 256 times the largest scale byte of a value
};
constexpr int kWideEachV = 1;      // the values' exponents are taken key by key
constexpr int kWideNoneV = 2;      // (with kWideEachV) some are of rows that are not finite
constexpr int kWideEachK = 4;      // the keys' scales are taken key by key

template <int D, bool EIGHT, bool SPLIT>
struct WideSmem {
  static constexpr int kOp = 128 * D * 2;                        // an operand tile: 128 rows of Q, K or V
  static constexpr int kStages = D == 64 ? (EIGHT ? 4 : 10) : EIGHT ? (SPLIT ? 4 : 3) : SPLIT ? 6 : 5;
  static constexpr int kRawStages = !EIGHT ? 0 : D == 128 ? 3 : 8;
  static constexpr int kRaw = 128 * D;                           // codes of K or V of a tile
  // Barriers of a ring: one per stage, or two in turn where the stages are odd in number.  A wait on a phase's
  // parity also passes two phases too early, so that whoever waits has to have seen the phase before.  The
  // converters of K and those of V see every other load each, whose copies land in any order: with an even
  // number of barriers each of them belongs to one of the two kinds.
  static constexpr int kOpBars = EIGHT && kStages % 2 ? 2 * kStages : kStages;
  static constexpr int kRawBars = kRawStages % 2 ? 2 * kRawStages : kRawStages;
  static constexpr int kRingOff = (SPLIT ? 1 : 2) * kOp;         // (behind Q)
  static constexpr int kRawOff = kRingOff + kStages * kOp;
  static constexpr int kScaleOff = kRawOff + kRawStages * kRaw;  // bytes [kWideInfo][K, V with K, V with V][128]
  static constexpr int kMetaOff = kScaleOff + (EIGHT ? kWideInfo * 384 : 0);     // int [kWideInfo][8]
  static constexpr int kInfoOff = kMetaOff + kWideInfo * 32;     // WideTileInfo [kWideInfo]
  static constexpr int kMlOff = kInfoOff + kWideInfo * 16;       // float2 [128]: the second group's reference and sum
  static constexpr int kTreeOff = kMlOff + (SPLIT ? 1024 : 0);   // uint2 [2][kWideDrafts]: what each draft sees, per piece's parity
  static constexpr int kBarOff = kTreeOff + 16 * kWideDrafts;
  static constexpr int kBars = 2 * kOpBars + 2 * kRawBars + 9;
  static constexpr int kMiscOff = kBarOff + kBars * 8;
  static constexpr int kBytes = kMiscOff + 64;
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};
// Two groups of four softmax warps, producer, issuer, and six converters or two idle warps.
constexpr int kWideConverters = 3;      // of K, and as many of V
template <bool EIGHT>
constexpr int kWideThreads = EIGHT ? 512 : 384;
// Registers per thread at launch, and of the softmax warps and the others after they have traded.
template <bool EIGHT>
constexpr int kWideRegs = EIGHT ? 128 : 168;
template <bool EIGHT>
constexpr int kWideSoftmaxRegs = EIGHT ? 192 : 200;
template <bool EIGHT>
constexpr int kWideOtherRegs = EIGHT ? 64 : 104;
static_assert(256 * kWideSoftmaxRegs<true> + 256 * kWideOtherRegs<true> <= 512 * kWideRegs<true>, "what the CTA has");
static_assert(256 * kWideSoftmaxRegs<false> + 128 * kWideOtherRegs<false> <= 384 * kWideRegs<false>, "what the CTA has");

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

template <bool BF16, int D, bool EIGHT, bool SPLIT>
__global__ void __launch_bounds__(kWideThreads<EIGHT>, 1) fa_wide_kernel(const __grid_constant__ WideParams params) {
  const DecodeCore& p = params.c;
  using SM = WideSmem<D, EIGHT, SPLIT>;
  constexpr int ST = SM::kStages, NS = SM::kOpBars;   // load ld: stage ld % ST, barriers of ld % NS;
  constexpr int RS = EIGHT ? SM::kRawStages : 1, RB = EIGHT ? SM::kRawBars : 1;   // its codes alike
  constexpr int kRows = SPLIT ? 128 : 256;            // of a unit
  constexpr bool kP16 = EIGHT || !BF16;               // the type of P (and of Q, K and V as operands): fp16 or bf16
  constexpr bool kPair = !EIGHT || !BF16;             // P as hi + lo (fa_decode.cuh, fa_decode8.cuh)
  constexpr float kLiftP = kLift<!kP16>;
  constexpr int kProducer = 8, kIssuer = 9, kConvert = 10;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto BAR = [&](int i) { return sbase + SM::kBarOff + 8 * i; };
  auto FULL = [&](int s) { return BAR(s); };                       // an operand tile is there
  auto EMPTY = [&](int s) { return BAR(NS + s); };                 // its MMAs are done
  auto RFULL = [&](int s) { return BAR(2 * NS + s); };             // codes are there
  auto REMPTY = [&](int s) { return BAR(2 * NS + RB + s); };       // they are converted
  constexpr int kB = 2 * NS + 2 * SM::kRawBars;
  auto SFULL = [&](int t) { return BAR(kB + t); };                 // S of group t
  auto PREADY = [&](int t) { return BAR(kB + 2 + t); };            // P of group t, O rescaled
  auto OFULL = [&](int t) { return BAR(kB + 4 + t); };             // O of group t, at a piece's end
  const uint32_t QREADY = BAR(kB + 6), DRAIN = BAR(kB + 7), JOIN = BAR(kB + 8);
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
      mbar_init(FULL(s), EIGHT ? kWideConverters : 1);
      mbar_init(EMPTY(s), 1);
    }
    if constexpr (EIGHT)
      for (int s = 0; s < RB; ++s) {
        mbar_init(RFULL(s), 1);
        mbar_init(REMPTY(s), kWideConverters);
      }
    for (int t = 0; t < 2; ++t) {
      mbar_init(SFULL(t), 1);
      mbar_init(PREADY(t), 4);
      mbar_init(OFULL(t), 1);
    }
    mbar_init(QREADY, 8);
    mbar_init(DRAIN, 1);
    mbar_init(JOIN, 4);
    fence_mbar_init();
    *s_abort = 0;
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  // In this order: the join kernel may then read the lengths as soon as it runs.
  pdl_wait_prior();
  pdl_launch_dependents();
  if (warp == kProducer) decode_start<kWideTile, kWideCharge>(p, blockIdx.x, lane, s_walk, s_len);
  else if (blockIdx.x == 0 && warp < kDecWarps) decode_report(p);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  DecodeWalk walk = *s_walk;
  int next_len = *s_len;
  const WaitCtx wc{s_abort, p.status, p.timeout_ns};
  const int box_shift = min(p.page_shift, 7);     // slots per copy
  const int box = 1 << box_shift;
  // The next piece: its sequence, unit, span and tiles.
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
      x.d = decode_step<kWideCharge>(walk, x.s.n, p.units);
      if (walk.b != x.b && walk.left > 0) next_len = decode_len(p, walk.b);
      if (x.d.nt) return true;
    }
    return false;
  };
  Piece x;
  if (warp == kProducer) {
    // ============================================================ producer
    regs_dec<kWideOtherRegs<EIGHT>>();
    int tile = 0;                                     // of this CTA; its loads are 2 tile (K) and 2 tile + 1 (V)
    bool dead = false;
    const int nsub = kWideTile >> box_shift;
    constexpr int R = EIGHT ? RS : ST, B = EIGHT ? RB : NS;     // the ring that the copies go to
    auto there = [&](int ld) { return EIGHT ? RFULL(ld % B) : FULL(ld % B); };
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
          const int st = (ld + B - R) % B, n = (ld + B - R) / B;   // (the barrier of load ld - R, which had the stage)
          bool ok = true;
          if (lane == 0 && n > 0) ok = wait_bar(EIGHT ? REMPTY(st) : EMPTY(st), (n - 1) & 1, wc);
          if (!__shfl_sync(0xffffffffu, ok, 0)) {
            dead = true;
            // (the loads up to here land below; `tile` counts whole tiles, a K without its V is waited for here)
            if (kind == 1 && lane == 0) drain_bar(there(ld - 1), ((ld - 1) / B) & 1, wc.timeout);
            break;
          }
          // (the place of tile - kWideInfo: all its readers are done, see kWideInfo)
          if (kind == 0 && lane < 8) s_meta[at * 8 + lane] = first < 0 ? -1 : first + (off & (box - 1));
          __syncwarp();
          const uint32_t bar = there(ld), to = ld % R;
          const uint32_t each = EIGHT ? (uint32_t)box * D + (kind == 0 ? 2u * box : (uint32_t)box) : (uint32_t)box * D * 2;
          if (lane == 0) mbar_arrive_expect_tx(bar, each * __popc(live));
          __syncwarp();
          if (mine) {
            const void* tm = kind ? &params.tm_v : &params.tm_k;
            if constexpr (EIGHT) {
              tma_load_4d(sbase + SM::kRawOff + to * SM::kRaw + sub * box * D, tm, bar, slot, hk, id);
              // both scales with K, as the softmax needs the values' before V; theirs with V again
              const long long from = (((long long)id * p.Hkv + hk) << p.page_shift) + slot;
              const uint32_t scales = sbase + SM::kScaleOff + at * 384 + sub * box;
              if (kind == 0) bulk_load(scales, params.k_scale + from, box, bar);
              bulk_load(scales + (kind ? 256 : 128), params.v_scale + from, box, bar);
            } else {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_5d_chunk(sbase + SM::kRingOff + to * SM::kOp + c * (128 * 128) + sub * box * 128, tm, bar, slot, c, hk, id);
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
      const int end = 2 * tile;
      for (int i = max(0, end - R); i < end; ++i) drain_bar(there(i), (i / B) & 1, wc.timeout);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // ============================================================ MMA issue
    regs_dec<kWideOtherRegs<EIGHT>>();
    // (the whole warp runs the loop, one lane's MMAs count: their descriptors stay in uniform registers)
    {
      const uint32_t lead = elect_lane();
      constexpr uint32_t kIdescS = idesc_f16(128, 128, !kP16, false);
      constexpr uint32_t kIdescO = idesc_f16(128, D, !kP16, true);
      const uint64_t q0 = sw128_desc(sbase, 16, 1024);
      const uint64_t k0 = sw128_desc(sbase + SM::kRingOff, 16, 1024);
      const uint64_t v0 = sw128_desc(sbase + SM::kRingOff, 128 * 128, 1024);
      int tile = 0, piece = 0;
      uint32_t phases = 0;                             // bit t: the parity of group t's next P
      bool ok = true;
      // S of group t from the K of `tl`, whose stage is given back behind the last group that reads it
      auto scores = [&](int t, int tl, bool last) {
        const int ld = 2 * tl;
        const uint64_t a = q0 + (SPLIT ? 0 : (t * SM::kOp) >> 4), b = k0 + (((ld % ST) * SM::kOp) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
          mma_ss_if(tmem + 128 * t, a + off, b + off, kIdescS, kk > 0, lead);
        }
        mma_commit_if(SFULL(t), lead);
        if (last) mma_commit_if(EMPTY(ld % NS), lead);
      };
      auto values = [&](int t, int tl, int i, bool last) {     // i: the group's tiles of the piece before this one
        const int ld = 2 * tl + 1;
        const uint64_t b = v0 + (((ld % ST) * SM::kOp) >> 4);
        const uint32_t o = tmem + 256 + 128 * t, s = tmem + 128 * t;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_ts_if(o, s + 8 * kk, b + (kk * 2048 >> 4), kIdescO, i % kWideFlush || kk, lead);
        if constexpr (kPair) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_ts_if(o, s + 64 + 8 * kk, b + (kk * 2048 >> 4), kIdescO, 1, lead);
        }
        if (last) mma_commit_if(EMPTY(ld % NS), lead);
      };
      auto landed = [&](int ld) {
        const bool got = __all_sync(0xffffffffu, wait_bar(FULL(ld % NS), (ld / NS) & 1, wc));
        tc_fence_after();
        return got;
      };
      auto ready = [&](int t) {
        const bool got = __all_sync(0xffffffffu, wait_bar(PREADY(t), (phases >> t) & 1, wc));
        phases ^= 1u << t;
        tc_fence_after();
        return got;
      };
      while (ok && next_piece(x)) {
        const int nt = x.d.nt;
        ok = __all_sync(0xffffffffu, wait_bar(QREADY, piece & 1, wc));
        ok = ok && landed(2 * tile);
        if (!ok) break;
        if constexpr (SPLIT) {
          scores(0, tile, true);
          if (nt > 1) {
            ok = landed(2 * tile + 2);
            if (ok) scores(1, tile + 1, true);
          }
        } else {
          scores(0, tile, false);
          scores(1, tile, true);
        }
        for (int j = 0; j < nt && ok; ++j, ++tile) {
          ok = landed(2 * tile + 1);
          if constexpr (SPLIT) {
            const int t = j & 1;
            ok = ok && ready(t);
            if (!ok) break;
            values(t, tile, j >> 1, true);
            if (j + 2 < nt) {
              ok = landed(2 * tile + 4);
              if (ok) scores(t, tile + 2, true);
            } else {
              mma_commit_if(OFULL(t), lead);
            }
          } else {
            for (int t = 0; t < 2 && ok; ++t) {
              ok = ready(t);
              if (!ok) break;
              values(t, tile, j, t == 1);
              if (j + 1 < nt) {
                if (t == 0) ok = landed(2 * tile + 2);
                if (ok) scores(t, tile + 1, t == 1);
              } else {
                mma_commit_if(OFULL(t), lead);
              }
            }
          }
        }
        ++piece;
      }
      // whatever is in flight ends before the tensor memory and the tiles are given up
      mma_commit_if(DRAIN, lead);
      drain_bar(DRAIN, 0, wc.timeout);
    }
    __syncwarp();
  } else if (!EIGHT && warp >= kConvert) {
    regs_dec<kWideOtherRegs<EIGHT>>();               // (idle: registers are traded by groups of four warps)
  } else if (EIGHT && warp >= kConvert) {
    // ============================================================ converters
    // Half of them take the K tiles, half the V tiles: a tile's way through registers is latency (loads, two
    // conversions and a product deep, stores, the fence), so that two at a time go twice as fast.
    regs_dec<kWideOtherRegs<EIGHT>>();
    constexpr int kThreads = 32 * kWideConverters;
    const int tid = (threadIdx.x - 32 * kConvert) % kThreads, kind = (threadIdx.x - 32 * kConvert) / kThreads;
    int tile = 0;
    bool dead = false;
    while (!dead && next_piece(x)) {
      for (int j = 0; j < x.d.nt; ++j, ++tile) {
        const int at = tile % kWideInfo, ld = 2 * tile + kind, rs = ld % RS, st = ld % ST;
        if (!__all_sync(0xffffffffu, wait_bar(RFULL(ld % RB), (ld / RB) & 1, wc))) dead = true;
        if (!dead && ld >= ST && !__all_sync(0xffffffffu, wait_bar(EMPTY((ld - ST) % NS), ((ld - ST) / NS) & 1, wc))) dead = true;
        if (dead) break;
        const int* meta = s_meta + at * 8;
        auto seen = [&](int r) {
          const int k = meta[r >> 4] < 0 ? -1 : meta[r >> 4] + (r & 15);
          return k >= x.s.lo && k < x.s.hi;
        };
        // every warp for itself: the largest exponents of the seen keys, the values' least
        const uint8_t* scales = smem + SM::kScaleOff + at * 384;           // K's, V's as they came with K, with V
        int top_k = 0, low_k = 255, top_v = 0, low_v = 255;
        unsigned on = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * i + lane;
          if (!seen(r)) continue;
          ++on;
          const int ks = scales[r], vs = scales[(kind ? 256 : 128) + r];
          top_k = max(top_k, ks), low_k = min(low_k, ks), top_v = max(top_v, vs), low_v = min(low_v, vs);
        }
        top_v = __reduce_max_sync(0xffffffffu, top_v);
        low_v = __reduce_min_sync(0xffffffffu, low_v);
        const bool whole = __all_sync(0xffffffffu, on == 4);               // every key is seen
        const int apart = params.e5m2 ? 8 : 15;
        int flags = top_v << 8;
        if (top_v - low_v > apart || top_v == (int)kScaleNone) {
          flags |= top_v == (int)kScaleNone ? kWideEachV | kWideNoneV : kWideEachV;
          top_v = 0;                                                       // (0: the codes of V stay as they are)
        }
        int top = top_v;
        if (kind == 0) {
          top = __reduce_max_sync(0xffffffffu, top_k);
          low_k = __reduce_min_sync(0xffffffffu, low_k);
          if (top - low_k > apart || top == (int)kScaleNone) flags |= kWideEachK, top = 0;
          if (tid == 0)
            s_info[at] = WideTileInfo{flags & kWideEachK ? 1.f : scale_of(top), top_v ? (float)(top_v - 127) : 0.f,
                                      top_v ? __uint_as_float((uint32_t)(254 - top_v) << 23) : 1.f, flags};
        }
        // a thread keeps to one 16-byte chunk of codes and to the rows `row` + kStep i
        constexpr int kChunks = D / 16, kStep = kThreads / kChunks, kTurns = (127 + kStep) / kStep;
        static_assert(kStep % 8 == 0 || kStep % 8 == 4, "a row's place among a swizzled eight, and that of the next");
        const int c = tid % kChunks, row = tid / kChunks;
        const uint8_t* raw = smem + SM::kRawOff + rs * SM::kRaw + tid * 16;
        const uint8_t* scale = scales + (kind ? 256 : 0) + row;
        // (the two halves of a chunk, for the second 64 channels in the other order: no bank twice)
        const bool swap = (c >> 2) & 1;
        const uint32_t to = sbase + SM::kRingOff + st * SM::kOp + (c >> 2) * (128 * 128) + row * 128;
        const uint32_t first = to + (((2 * (c & 3) + swap) ^ (row & 7)) << 4);
        auto convert = [&](auto format, auto every) {
          constexpr bool E5M2 = decltype(format)::value;
#pragma unroll 1
          for (int y0 = 0; y0 < kTurns; y0 += 4) {
            uint4 w[4];                                // (four loads, then their stores: one order of memory for all)
            uint32_t f[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const bool there = row + kStep * (y0 + y) < 128;
              w[y] = there ? *reinterpret_cast<const uint4*>(raw + (y0 + y) * (kStep * D)) : make_uint4(0, 0, 0, 0);
              f[y] = there ? scale[kStep * (y0 + y)] : 0;
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              // 2^(e - E) as an fp16 pair, exactly down to 2^-24 (e <= E where the row is seen)
              const float z = top ? scale_of(max((int)f[y] - top, -100) + 127) : 1.f;
              f[y] = pack_f16x2(z, z);
              if (!decltype(every)::value && !seen(min(row + kStep * (y0 + y), 127))) w[y] = make_uint4(0, 0, 0, 0), f[y] = 0;
              if (D == 128 && swap) w[y] = make_uint4(w[y].z, w[y].w, w[y].x, w[y].y);
              uint32_t h[8];
              codes4<E5M2>(w[y].x, h[0], h[1]);
              codes4<E5M2>(w[y].y, h[2], h[3]);
              codes4<E5M2>(w[y].z, h[4], h[5]);
              codes4<E5M2>(w[y].w, h[6], h[7]);
#pragma unroll
              for (int q = 0; q < 8; ++q) h[q] = mul_f16x2(h[q], f[y]);
              if (row + kStep * (y0 + y) < 128) {
                const uint32_t p0 = (first + (y0 + y) * (kStep * 128)) ^ (kStep % 8 && (y & 1) ? 64u : 0u);
                st_shared_v4(p0, make_uint4(h[0], h[1], h[2], h[3]));
                st_shared_v4(p0 ^ 16u, make_uint4(h[4], h[5], h[6], h[7]));
              }
            }
          }
        };
        auto of = [&](auto format) {
          if (whole) convert(format, std::true_type{});
          else convert(format, std::false_type{});
        };
        if (params.e5m2) of(std::true_type{});
        else of(std::false_type{});
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(FULL(ld % NS));
          mbar_arrive(REMPTY(ld % RB));
        }
      }
    }
  } else {
    // ============================================================ softmax: a row per thread
    regs_inc<kWideSoftmaxRegs<EIGHT>>();
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;                 // of the group's 128
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 * t + lanes, tO = tmem + 256 + 128 * t + lanes;
    int tile0 = 0, made = 0, piece = 0, pieces = 0, joins = 0;   // the piece's first tile; tiles, pieces, pieces of this group
    bool dead = false;
    // fp32 numbers of scratch times g plus a row's 32 columns
    auto plus = [&](uint4 a, float g, const uint32_t* u) {
      return make_uint4(__float_as_uint(fmaf(__uint_as_float(a.x), g, __uint_as_float(u[0]))),
                        __float_as_uint(fmaf(__uint_as_float(a.y), g, __uint_as_float(u[1]))),
                        __float_as_uint(fmaf(__uint_as_float(a.z), g, __uint_as_float(u[2]))),
                        __float_as_uint(fmaf(__uint_as_float(a.w), g, __uint_as_float(u[3]))));
    };
    auto gone_of = [&](int group) {                    // this row's sum that has left group's accumulator
      return reinterpret_cast<uint4*>(params.gone + (((long long)blockIdx.x * 2 + group) * 128 + row) * D);
    };
    while (!dead && next_piece(x)) {
      const int hk = x.unit / p.groups, rg = x.unit % p.groups, nt = x.d.nt;
      const int r0 = rg * kRows + (SPLIT ? 0 : 128 * t);   // this group's first row of the KV head
      const long long at0 = ((long long)x.b * p.Hkv + hk) * p.rows + r0;
      const bool mine = r0 + row < p.rows;
      // The second group may have had no tile of the last piece: it stays at most one piece ahead of the first
      // (it would else stand for it at QREADY, and for its rows of Q).
      if (SPLIT && t == 1 && piece > 0 && !__all_sync(0xffffffffu, wait_bar(QREADY, (piece - 1) & 1, wc))) break;
      const int drafts = p.ancestors ? decode_drafts(p, x.b, x.len) : 0;
      const int base = x.len - drafts;                                        // a tree's first draft
      const bool small_tree = drafts > 0 && p.Sq <= kWideDrafts;
      uint2* s_tree = reinterpret_cast<uint2*>(smem + SM::kTreeOff) + (piece & 1) * kWideDrafts;
      ++piece;
      if (small_tree && (x.s.first + x.d.t0 + nt) * kWideTile > base) {       // the piece has drafts' keys
#pragma unroll
        for (int y = 0; y < kWideDrafts / 8; ++y) {                           // (a warp's drafts all at once)
          const int i = warp + 8 * y;
          const uint32_t a = __ballot_sync(0xffffffffu, decode_ancestor(p, x.b, drafts, i, lane));
          const uint32_t c = __ballot_sync(0xffffffffu, decode_ancestor(p, x.b, drafts, i, 32 + lane));
          if (lane == 0) s_tree[i] = make_uint2(a, c);
        }
      }
      // Q into its place (the last piece's S products of it are done), with the sign of the scale and, over an
      // 8-bit cache, as fp16 of a power of two times it: kLanes lanes per row, so that a load is whole lines
      float fac = fabsf(p.scale_log2);
      if (!SPLIT || t == 0 || (EIGHT && BF16)) {
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
        const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        const int c = lane % kLanes;
#pragma unroll
        for (int y0 = 0; y0 < kLanes; y0 += 8) {
          uint4 w[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int r = (warp & 3) * 32 + (y0 + y) * kAtOnce + lane / kLanes;
            w[y] = r0 + r < p.rows ? reinterpret_cast<const uint4*>(p.q + (at0 + r) * D)[c] : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int r = (warp & 3) * 32 + (y0 + y) * kAtOnce + lane / kLanes;
            if constexpr (EIGHT && BF16) {
              uint32_t top = max_u16x2(max_u16x2(w[y].x & 0x7FFF7FFFu, w[y].y & 0x7FFF7FFFu),
                                       max_u16x2(w[y].z & 0x7FFF7FFFu, w[y].w & 0x7FFF7FFFu));
              top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
              for (int q = 1; q < kLanes; q <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, q));
              const int e = max((int)(top >> 7), 127 - 100) - 127 - 14;       // as in fa_decode8_kernel
              const float f = __uint_as_float((uint32_t)(127 - e) << 23);
              auto half = [&](uint32_t u) { return pack_f16x2(lo16_f32<true>(u) * f, hi16_f32<true>(u) * f); };
              w[y] = make_uint4(half(w[y].x), half(w[y].y), half(w[y].z), half(w[y].w));
              // to the thread of the row
              const int its = __shfl_sync(0xffffffffu, e, (lane % kAtOnce) * kLanes);
              if (lane / kAtOnce == y0 + y) fac *= __uint_as_float((uint32_t)(127 + its) << 23);
            }
            if (!SPLIT || t == 0)
              st_shared_v4(sbase + t * SM::kOp + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           make_uint4(w[y].x ^ sign, w[y].y ^ sign, w[y].z ^ sign, w[y].w ^ sign));
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(QREADY);
      const int i_row = p.Sq == 1 ? 0 : (r0 + row) % p.Sq;
      const int tok = p.ancestors ? base - 1 : x.len - p.Sq + i_row;          // keys up to it are seen
      const int all_hi = p.ancestors ? base - 1 : x.len - p.Sq;               // by every row
      const int all_lo = p.pre_tokens >= 0 ? x.len - 1 - p.pre_tokens : 0;    // and from here on
      const int low = p.pre_tokens >= 0 ? tok - p.pre_tokens : 0;
      float m = kNoScore, l = 0.f, m_gone = kNoScore;  // m_gone: the reference of what has left the accumulator
      int n = 0;                                       // tiles of the piece in this group
      int v_high = 0;                                  // the largest scale byte of a value in them

#pragma unroll 1
      for (int j = SPLIT ? t : 0; j < nt; j += SPLIT ? 2 : 1, ++n) {
        const int tile = tile0 + j;
        if (!__all_sync(0xffffffffu, wait_bar(SFULL(t), made & 1, wc))) {
          dead = true;
          break;
        }
        ++made;
        tc_fence_after();
        const int* meta = s_meta + (tile % kWideInfo) * 8;
        // the keys of 32 that this row sees, from the first keys of both 16
        auto visible = [&](int ka, int kb) {
          auto group = [&](int k0) -> uint32_t {       // those before a tree
            if (k0 < 0) return 0;
            const int y = min(max(tok + 1 - k0, 0), 16), z = min(max(low - k0, 0), 16);
            return ((1u << y) - 1u) & ~((1u << z) - 1u);
          };
          uint32_t vis = group(ka) | group(kb) << 16;
          if (small_tree) {
            const uint2 y = s_tree[i_row];
            const unsigned long long w = y.x | (unsigned long long)y.y << 32;
            auto sees = [&](int k0) -> uint32_t {      // the drafts among 16 keys that this row sees
              const int d = k0 - base;
              if (k0 < 0 || d <= -16 || d >= kWideDrafts) return 0;
              return (uint32_t)(d < 0 ? w << -d : w >> d) & 0xFFFFu;
            };
            vis |= sees(ka) | sees(kb) << 16;
          } else if (p.ancestors && max(ka, kb) + 15 >= base) {
            // lane: one of the 32 keys; the warp's rows one by one
            const int k0 = lane < 16 ? ka : kb;
            const int draft = k0 < 0 ? -1 : k0 + (lane & 15) - base;
            int i = (r0 + (warp & 3) * 32) % p.Sq;
#pragma unroll 8
            for (int r = 0; r < 32; ++r) {
              const bool see = draft >= 0 && decode_ancestor(p, x.b, drafts, i, draft);
              const uint32_t bits = __ballot_sync(0xffffffffu, see);
              if (lane == r) vis |= bits;
              if (++i == p.Sq) i = 0;
            }
          }
          return vis;
        };
        if (n && n % kWideFlush == 0) {                // (O is at rest; the next P V starts from zero)
          const float g = ex2_approx(m_gone - m);
          m_gone = m;
          uint4* gone = gone_of(t);
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t u[16];
            tmem_ld16(tO + 16 * c, u);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q)
              gone[4 * c + q] = plus(n == kWideFlush ? make_uint4(0, 0, 0, 0) : gone[4 * c + q], g, u + 4 * q);
          }
        }
        auto move = [&](float top) {                   // references move up
          const float to = top - m > kMaxOver + kLiftP ? top - kLiftP : m;
          const float g = ex2_approx(m - to);
          if constexpr (EIGHT) {                       // (as in fa_decode8_kernel)
            const float a = ex2_floor(m - to);
            l *= ex2_approx(m - to - a);
            l *= ex2_approx(a);
          } else {
            l *= g;
          }
          m = to;
          if (n % kWideFlush) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t u[16];
              tmem_ld16(tO + 16 * c, u);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * g);
              tmem_st16(tO + 16 * c, u);
            }
          }
        };
        WideTileInfo info{1.f, 0.f, 1.f, 0};
        if constexpr (EIGHT) info = s_info[tile % kWideInfo];
        // a score in log2 units with its value's exponent is s f + v
        float f = fac * info.k_scale, v = info.v_exp;
        // taken key by key: what the converters say, and values far below others (kFarScales)
        const bool odd = EIGHT && ((info.flags & 255) || (info.flags >> 8) + kFarScales < v_high);
        if (EIGHT) v_high = max(v_high, info.flags >> 8);
        if (odd) {
          // Key by key, in tensor memory: the scores become what they are in log2 units, masked, the reference moves,
          // and the sum takes each without its value's exponent.  (In loops of their own: as part of the code
          // below they took 5 to 20 % of the time of the tiles that need none of it.)
          const uint8_t* ks = smem + SM::kScaleOff + (tile % kWideInfo) * 384;
          const bool each_k = info.flags & kWideEachK, each_v = info.flags & kWideEachV;
          // byte i, or what stands for the tile's one (a key's scale is in f then)
          auto k_byte = [&](int i) -> uint32_t { return each_k ? ks[i] : 127u; };
          auto v_byte = [&](int i) -> uint32_t { return each_v ? ks[128 + i] : (uint32_t)((int)info.v_exp + 127); };
          auto v_exp = [&](int i) { const uint32_t y = v_byte(i); return y == kScaleNone ? 0.f : (float)((int)y - 127); };
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            const uint32_t vis = visible(meta[c], -1);
            uint32_t u[16];
            tmem_ld16(tS + 16 * c, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              // (not finite: infinity times 0 of a key, of a value no exponent, so that it weighs as any other)
              const float y = (vis >> i) & 1u ? fmaf(__uint_as_float(u[i]) * f, scale_of(k_byte(16 * c + i)), v_exp(16 * c + i)) : -INFINITY;
              top = fmaxf(top, y);                     // (NaN is dropped)
              u[i] = __float_as_uint(y);
            }
            tmem_st16(tS + 16 * c, u);
          }
          tmem_wait_st();
          if (__any_sync(0xffffffffu, top - m > kMaxOver + kLiftP)) move(top);
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t u[16];
            tmem_ld16(tS + 16 * c, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float y = __uint_as_float(u[i]);
              l += ex2_approx(y - v_exp(16 * c + i) - m);
              if (v_byte(16 * c + i) == kScaleNone && y > -INFINITY) u[i] = 0x7FFFFFFFu;   // (its P is NaN)
            }
            tmem_st16(tS + 16 * c, u);
          }
          tmem_wait_st();
          f = 1.f, v = 0.f;
        }
        uint32_t su[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&su[32 * c]));
        const int4 ka = *reinterpret_cast<const int4*>(meta), kb = *reinterpret_cast<const int4*>(meta + 4);
        const int first = min(min(min(ka.x, ka.y), min(ka.z, ka.w)), min(min(kb.x, kb.y), min(kb.z, kb.w)));
        const int last = max(max(max(ka.x, ka.y), max(ka.z, ka.w)), max(max(kb.x, kb.y), max(kb.z, kb.w))) + 15;
        const bool all = first >= max(all_lo, 0) && last <= all_hi;
        tmem_wait_ld();
        float sv[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) sv[i] = __uint_as_float(su[i]);
        if (!all && !odd) {                            // (few tiles: a piece's ends)
          const int keys[8] = {ka.x, ka.y, ka.z, ka.w, kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t vis = visible(keys[2 * c], keys[2 * c + 1]);
#pragma unroll
            for (int i = 0; i < 32; ++i) sv[32 * c + i] = (vis >> i) & 1u ? fmaf(sv[32 * c + i], f, v) : -INFINITY;
          }
          f = 1.f, v = 0.f;
          if constexpr (!EIGHT) {
            // V of keys that no row sees may hold anything: its rows become 0 (P is 0 there), by each group
            const int k0 = meta[row >> 4], k = k0 < 0 ? -1 : k0 + (row & 15);
            const int ld = 2 * tile + 1;
            if (!__all_sync(0xffffffffu, wait_bar(FULL(ld % NS), (ld / NS) & 1, wc))) {
              dead = true;
              break;
            }
            if (k < x.s.lo || k >= x.s.hi || decode_blind_draft(p, x.b, drafts, k - base)) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  st_shared_v4(sbase + SM::kRingOff + (ld % ST) * SM::kOp + c * (128 * 128) + row * 128 + q * 16, make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
          }
        }
        const float top = fmaf(row_max(sv), f, v);     // (f >= 0; NaN is dropped)
        if (__any_sync(0xffffffffu, top - m > kMaxOver + kLiftP)) move(top);
        const float neg = v - m;
        const uint64_t f2 = f2_pack(f, f), neg2 = f2_pack(neg, neg);
        uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(sv[32 * c + 2 * i], sv[32 * c + 2 * i + 1]), f2, neg2), a, b);
            a = ex2_approx(a);
            b = ex2_approx(b);
            sum2[i & 1] = f2_add(sum2[i & 1], f2_pack(a, b));
            hi[i] = kP16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
            if constexpr (kPair) lo[i] = pack_residual_x2(a, b, hi[i], !kP16);
          }
          tmem_st16(tS + 16 * c, hi);
          if constexpr (kPair) tmem_st16(tS + 64 + 16 * c, lo);
        }
        if (!odd) {
          float a, b, c, d;
          f2_unpack(sum2[0], a, b);
          f2_unpack(sum2[1], c, d);
          l = fmaf((a + b) + (c + d), info.v_back, l);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(PREADY(t));
      }
      if (dead) break;
      tile0 += nt;
      // ---- the piece's answer
      const bool direct = x.d.t0 == 0 && nt == x.s.n;
      const long long part = (2LL * blockIdx.x + (x.d.t0 == 0 ? 1 : 0)) * kRows + (SPLIT ? 0 : 128 * t) + row;
      float2* s_ml = reinterpret_cast<float2*>(smem + SM::kMlOff);
      const bool other = SPLIT && nt > 1;              // the second group has tiles of the piece, too
      if (n) {
        if (!__all_sync(0xffffffffu, wait_bar(OFULL(t), pieces & 1, wc))) break;
        ++pieces;
        tc_fence_after();
      }
      if (SPLIT && t == 1) {                           // the first group joins the two
        if (!n) continue;
        s_ml[row] = make_float2(m, l);
        // what has left the accumulator comes back to this group's place in scratch as of m
        if (n > kWideFlush) {
          const float g = ex2_approx(m_gone - m);
          uint4* gone = gone_of(1);
          const uint32_t none[4] = {0, 0, 0, 0};
          for (int q = 0; q < D / 4; ++q) gone[q] = plus(gone[q], g, none);
          __threadfence_block();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(JOIN);
        continue;                                      // (O stays until the next piece's Q is ready)
      }
      float g0 = 1.f, g1 = 0.f;                        // the groups' weights
      bool gone1 = false;
      if (other) {
        if (!__all_sync(0xffffffffu, wait_bar(OFULL(1), joins & 1, wc) && wait_bar(JOIN, joins & 1, wc))) break;
        ++joins;
        tc_fence_after();
        const float2 ml = s_ml[row];
        const float to = fmaxf(m, ml.x);
        g0 = ex2_approx(m - to), g1 = ex2_approx(ml.x - to);
        const float a0 = ex2_floor(m - to), a1 = ex2_floor(ml.x - to);
        l = fmaf(l * ex2_approx(m - to - a0), ex2_approx(a0), ml.y * ex2_approx(ml.x - to - a1) * ex2_approx(a1));
        m_gone = m_gone - m;                           // (relative to this group's own reference)
        m = to;
        gone1 = (nt / 2) > kWideFlush;
      } else {
        m_gone = m_gone - m;
      }
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const float g = ex2_approx(m_gone) * g0;
      // 16 columns of the row: both groups' and what has left the accumulators
      auto answer = [&](int c, uint32_t (&u)[16]) {
        tmem_ld16(tO + 16 * c, u);
        if constexpr (SPLIT) {
          uint32_t u1[16];
          tmem_ld16(tO + 128 + 16 * c, u1);            // (whatever it is where the second group had no tile)
          tmem_wait_ld();
          if (other) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              u[i] = __float_as_uint(fmaf(__uint_as_float(u[i]), g0, __uint_as_float(u1[i]) * g1));
          }
        } else {
          tmem_wait_ld();
        }
        auto add = [&](const uint4* from, float f) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 y = plus(from[4 * c + q], f, u + 4 * q);
            u[4 * q] = y.x, u[4 * q + 1] = y.y, u[4 * q + 2] = y.z, u[4 * q + 3] = y.w;
          }
        };
        if (n > kWideFlush) add(gone_of(t), g);
        if (gone1) add(gone_of(1), g1);
      };
      // The warp's rows leave through where its rows of Q were (their last product is done; D / 64 areas of 128
      // bytes a row, 16-byte chunks turned by the row), so that the stores are whole lines.
      const uint32_t area = sbase + t * SM::kOp + ((warp & 3) * 32) * 128;
      auto stage = [&](int chunk, uint4 y) {           // the chunk-th 16 bytes of this row's D / 64 areas
        st_shared_v4(area + (chunk >> 3) * (128 * 128) + lane * 128 + (((chunk & 7) ^ (lane & 7)) << 4), y);
      };
      constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
      auto leave = [&](uint8_t* to, int pitch) {       // to: where this warp's first row begins
        __syncwarp();
#pragma unroll
        for (int y = 0; y < kLanes; ++y) {
          const int r = y * kAtOnce + lane / kLanes, c = lane % kLanes;
          const uint4 w = *reinterpret_cast<const uint4*>(smem + (area - sbase) + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          if (r0 + (warp & 3) * 32 + r < p.rows) *reinterpret_cast<uint4*>(to + (long long)r * pitch + c * 16) = w;
        }
        __syncwarp();
      };
      if (direct) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t u[16];
          answer(c, u);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = pack16x2<BF16>(__uint_as_float(u[8 * q + 2 * e]) * inv, __uint_as_float(u[8 * q + 2 * e + 1]) * inv);
            stage(2 * c + q, make_uint4(y[0], y[1], y[2], y[3]));
          }
        }
        leave(reinterpret_cast<uint8_t*>(p.o + (at0 + (warp & 3) * 32) * D), D * 2);
      } else {
        uint8_t* to = reinterpret_cast<uint8_t*>(p.part_o + (part - lane) * D);
#pragma unroll 1
        for (int z = 0; z < 2; ++z) {                  // (in fp32 half a row at a time)
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[16];
            answer(z * (D / 32) + c, u);
#pragma unroll
            for (int q = 0; q < 4; ++q) stage(4 * c + q, make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]));
          }
          leave(to + z * D * 2, D * 4);
        }
      }
      if (mine) {
        if (direct) p.lse[at0 + row] = l == 0.f ? INFINITY : (m + log2f(l)) * 0.6931471805599453f;   // (NaN stays)
        else p.part_ml[part] = make_float2(m, l);
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
