// fa_decode: attention of a sequence's newest tokens over its pages.
//
// Per KV head the G * Sq rows of a sequence (query heads of the group times new
// tokens) share every key, so that a key and its value are read once and used
// by all of them: 4 D flops per row against 4 D bytes, far below what the
// tensor cores need to be the limit.  The kernel is a stream of K and V tiles
// through shared memory at HBM speed with as little as possible beside it:
//
//   * a CTA is one producer warp and four consumer warps, two CTAs per SM: while
//     one waits at a barrier or ends a unit the other streams;
//   * the producer looks up pages and copies tiles of 64 keys (K and V, 64
//     channels x up to 64 slots x D / 64 halves per TMA box, 128-byte swizzle)
//     into a ring of 64 KB, 128 KB per SM, more than twice latency times
//     bandwidth (rings of 96 KB, or three CTAs: no faster);
//   * of every tile each consumer scores 16 keys against all rows, puts their P
//     into shared memory and then adds all 64 keys' values to its quarter of the
//     channels: O of 8 NT rows costs a thread 8 NT registers instead of 32 NT
//     with a whole O per warp, and nothing has to be joined at a unit's end but
//     the sums.  (The warps-by-keys form spilled at 24 rows, spent 2.4 us per
//     unit, and took 66 us against 48 us for five draft tokens in a window.)
//   * products are transposed, S^T = K Q^T and O^T = V^T P^T, with the keys (then
//     the channels) as the 16-row side of mma.m16n8k16 and the rows as its
//     8-column side: 4 rows of a common group waste 4 of 8 columns there, but
//     would waste 124 of the 128 lanes of a tcgen05 tile, whose accumulator
//     also costs a round trip through TMEM before every exponential.  Up to 32
//     rows the warp-level products stay behind the copies (launch_decode_rows
//     has the figures past that);
//   * P goes into the value product as hi + lo pairs of the cache's type (the
//     tensor cores are idle, and a single bf16 P would add an error as large as
//     the rounding of O).
//
// Work: a unit is one (sequence, KV head, group of up to 8 NT rows) with its
// tiles and a charge of kUnitTiles for what it costs by itself.  All units in a
// row are cut into equal ranges, one per CTA, so that ragged lengths and few
// long sequences fill the GPU alike; lengths are read on the device.  A unit
// inside one range is finished there; the pieces of a unit that several ranges
// share go to scratch (at most two per CTA, in fp32) and fa_decode_join_kernel
// joins them in the order of the keys.
//
// Measured (32 query heads on 8 KV heads of 128, bf16, both kernels): 8 sequences
// of 131072 tokens 599 us, 7.17 TB/s; 64 of mixed lengths up to 8192 167 us, 6.63
// TB/s; one of 517 tokens 5.6 us, of which 1.9 pass before the first tile is
// there (lengths, page ids, copies: three dependent trips to memory) and 1.4 are
// the join.  Calls of one token add 4 to 9 us to their bytes' time; five draft
// tokens in a window 12, 256 sequences of 60 tokens 19 (a unit's own 2 us each).
#pragma once
#include "fa_paged.cuh"
#include "fa_tiled.cuh"   // bounded waits

namespace fa {

constexpr int kDecTile = 64;                          // keys per tile
constexpr int kDecWarps = 4;                          // consumer warps, 16 keys of a tile each
constexpr int kDecCtasPerSm = 2;
constexpr int kDecThreads = 32 * (kDecWarps + 1);     // and the producer
constexpr int kUnitTiles = 2;                         // a unit's own cost, in tiles (0: ragged lengths 30 % slower)
// A row's reference (the subtrahend of its exponents) follows its maximum lazily: it stays while no
// score exceeds it by more than kMaxOver powers of two (beyond the lift below), so that the usual
// tile needs one vote and no shuffles; every sum is relative to the reference.  With fp16 the
// reference is set kLift below the maximum, so that the largest P lie between 2^7 and 2^15 and small
// ones keep an absolute error of 2^-25 / 2^7 of the largest instead of 2^-25 (fp16's subnormals);
// bf16 has fp32's range and needs none.
constexpr float kMaxOver = 8.f;
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;
constexpr float kNoScore = -3.402823466e38f;          // the reference before a row's first key

// What every warp needs, in as few lines of the parameter bank as it takes: the first touch of each
// is a miss, and the way to a CTA's first copy would pay them one after the other.
struct DecodeCore {
  const int32_t* kv_lens;
  const int32_t* table;
  long long table_stride;
  const int32_t* sel;          // [B, Hkv, max_sel] or null
  int max_len;                 // what a table row holds
  int num_pages, page_shift;   // page size = 1 << page_shift
  int max_sel;                 // entries of a list
  int B, Hkv;
  int rows;                    // G * Sq
  int groups;                  // row groups per KV head
  int units;                   // Hkv * groups
  int ctas;
  unsigned long long units_inv, ctas_inv;   // ceil(2^64 / x): quotients by a product's upper half
  int Sq;
  int pre_tokens;              // -1: unbounded
  int reach;                   // Sq + pre_tokens: the keys that some row sees are the last `reach`; -1: all
  float scale_log2;
  int* status;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  float* part_o;               // [2 * ctas][8 NT][D], unnormalised: slot 2 c + 1 begins its unit
  float2* part_ml;             // [2 * ctas][8 NT]: reference (log2 units), sum
  long long timeout_ns;
};
struct DecodeParams {
  DecodeCore c;
  CUtensorMap tm_k;   // (64 channels, slots, D / 64, heads, pages)
  CUtensorMap tm_v;
};

template <int D, int NT>
struct DecodeSmem {
  static constexpr int kHalf = kDecTile * D * 2;                 // K or V of a tile
  // The consumers take every tile, so that each has seen every earlier phase of a stage's barriers
  // (a wait on a phase's parity also passes two phases too early: teams that take turns would need
  // a stage count that leaves each stage with one of them).
  static constexpr int kStages = 2 * (128 / D);
  static constexpr bool kQShared = NT > 2;                       // Q in shared memory or in registers
  static constexpr int kPOff = kStages * 2 * kHalf;              // uint4 [4 x 16 keys][NT][lane]: P hi, lo
  static constexpr int kQOff = kPOff + kDecWarps * NT * 512;
  static constexpr int kMaxOff = kQOff + (kQShared ? NT * (D / 32) * 512 : 0);   // float [warps][8 NT]
  static constexpr int kSumOff = kMaxOff + kDecWarps * 8 * NT * 4;               // float [warps][8 NT]
  static constexpr int kMetaOff = kSumOff + kDecWarps * 8 * NT * 4;              // int4 [stages]
  static constexpr int kBarOff = kMetaOff + kStages * 16;
  static constexpr int kMiscOff = kBarOff + 2 * kStages * 8;     // range, abort flag
  static constexpr int kBytes = kMiscOff + 64;
  static_assert(kBytes <= 115712, "two CTAs must fit an SM's 228 KB, 1 KB of it reserved for each");
};

// Keys [lo, hi) that some row of a sequence sees, as tiles [first, first + n);
// an empty sequence counts one tile, whose CTA writes the empty answer.  Of a
// list as many entries count as the sequence has pages, so that short ones among
// long ones cost what they hold (64 of 100 tokens, lists of 64 pages, 8 KV heads:
// 11.7 us against 102 us with every slot of every list a tile's).
struct DecodeSpan {
  int lo, hi, first, n;
  int listed;      // entries of the list that count
};
__device__ __forceinline__ DecodeSpan decode_span(const DecodeCore& p, int len) {
  DecodeSpan s;
  s.hi = len;
  s.lo = p.reach >= 0 ? max(0, len - p.reach) : 0;
  s.first = p.sel ? 0 : s.lo / kDecTile;
  s.listed = min(p.max_sel, (len + (1 << p.page_shift) - 1) >> p.page_shift);
  const int keys = p.sel ? s.listed << p.page_shift : len;
  s.n = max(1, (keys + kDecTile - 1) / kDecTile - s.first);
  return s;
}
__device__ __forceinline__ int decode_len(const DecodeCore& p, int b) {
  // from L2: the join kernel may read lengths that this SM's L1 holds from an earlier call
  const int len = __ldcg(p.kv_lens + b);
  return len < 0 || len > p.max_len ? 0 : len;
}

// The lengths and charges of sequences base + 32 i + lane: eight independent loads.
constexpr int kChunks = 8;
__device__ __forceinline__ void decode_charges(const DecodeCore& p, int base, int lane, int (&len)[kChunks],
                                               int (&c)[kChunks]) {
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    len[i] = c[i] = 0;
    if (base + 32 * i < p.B) {         // (the same for the whole warp: a small batch pays for one chunk)
      const int b = base + 32 * i + lane;
      if (b < p.B) len[i] = decode_len(p, b);
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
    if (base + 32 * i + lane < p.B) c[i] = decode_span(p, len[i]).n + kUnitTiles;
}
// Sum over the warp of numbers below 2^59, in three pieces by the warp's reduction.
__device__ __forceinline__ long long warp_sum(long long x) {
  const unsigned m = 0xffffffu;
  const long long lo = __reduce_add_sync(0xffffffffu, (unsigned)x & m);
  const long long mid = __reduce_add_sync(0xffffffffu, (unsigned)(x >> 24) & m);
  const long long hi = __reduce_add_sync(0xffffffffu, (unsigned)(x >> 48));
  return lo + (mid << 24) + (hi << 48);
}
// Quotient of numbers >= 0; the schedule's fit 32 bits but for the longest, and it waits for them.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}
// a / d by inv = ceil(2^64 / d) (0 stands for d = 1): exact while a * d < 2^64.
__device__ __forceinline__ long long times_inverse(long long a, unsigned long long inv) {
  return inv ? (long long)__umul64hi((unsigned long long)a, inv) : a;
}
// CTAs that share `total` charged tiles, the start of CTA c's range, the CTA that has tile t.
__device__ __forceinline__ int decode_ctas(const DecodeCore& p, long long total) {
  return (int)min((long long)p.ctas, total);
}
__device__ __forceinline__ long long decode_first(const DecodeCore& p, long long total, int c) {
  return total <= p.ctas ? c : times_inverse(total * c, p.ctas_inv);
}
__device__ __forceinline__ int decode_owner(long long total, int n, long long t) {
  return (int)quotient((t + 1) * n - 1, total);
}
// A walk over the units of a CTA's range: unit `unit` (KV head, row group) of sequence b, from its
// charged tile `off`; `left` charged tiles to go.
struct DecodeWalk {
  int b, unit, off;
  long long left;
};
// The tiles [t0, t0 + nt) of a unit of n that the walk's next step holds.
struct DecodePiece {
  int t0, nt;
};
__device__ __forceinline__ DecodePiece decode_step(DecodeWalk& w, int n, int units) {
  DecodePiece d;
  const int charge = n + kUnitTiles;
  const int take = (int)min((long long)(charge - w.off), w.left);
  d.t0 = max(0, w.off - kUnitTiles);
  d.nt = max(0, w.off + take - kUnitTiles) - d.t0;
  w.left -= take;
  w.off = 0;                    // (whatever is left starts with a unit)
  if (++w.unit == units) w.unit = 0, ++w.b;
  return d;
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, uint32_t bar, int slot,
                                            int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(0), "r"(slot), "r"(head), "r"(page)
      : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 8x8 transpose of 16-bit values held two per lane
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// c (16 x 8, fp32) += a (16 x 16) b (16 x 8)
template <bool BF16>
__device__ __forceinline__ void mma_16x8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF16, int D, int NT>
__global__ void __launch_bounds__(kDecThreads, kDecCtasPerSm) fa_decode_kernel(const __grid_constant__ DecodeParams params) {
  const DecodeCore& p = params.c;
  using SM = DecodeSmem<D, NT>;
  constexpr int NS = SM::kStages;
  constexpr int KS = D / 16;                   // 16-channel steps
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto FULL = [&](int s) { return sbase + SM::kBarOff + 8 * s; };
  auto EMPTY = [&](int s) { return sbase + SM::kBarOff + 8 * (NS + s); };
  int* s_meta = reinterpret_cast<int*>(smem + SM::kMetaOff);   // per stage: first key of each 16, or -1
  DecodeWalk* s_walk = reinterpret_cast<DecodeWalk*>(smem + SM::kMiscOff);   // where this CTA starts,
  int* s_len = reinterpret_cast<int*>(smem + SM::kMiscOff + 24);             // the length there
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + SM::kMiscOff + 28);

  if (threadIdx.x == 0) {
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
  if (warp == kDecWarps) {   // this CTA's range of charged tiles, and the sequence it starts in
    int len[kChunks], c[kChunks];
    int mine = 0, my_len = 0, inc;           // of the sequence `at + lane`, its chunk of 32 summed up
    auto scan = [&](int x) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      return x;
    };
    long long total, start = 0, end = 0, first, before = 0;
    int at = 0;
    auto range = [&]() {
      if ((int)blockIdx.x < decode_ctas(p, total)) {
        start = decode_first(p, total, blockIdx.x);
        end = decode_first(p, total, blockIdx.x + 1);
      }
      // in charges of one unit per sequence: the sequence is the last with at most so many before it
      first = times_inverse(start, p.units_inv);
    };
    if (p.B <= 32) {
      if (lane < p.B) {
        my_len = decode_len(p, lane);
        mine = decode_span(p, my_len).n + kUnitTiles;
      }
      inc = scan(mine);
      total = (long long)__shfl_sync(0xffffffffu, inc, 31) * p.units;
      range();
    } else {
      long long sum = 0;
      for (int base = 32 * kChunks; base < p.B; base += 32 * kChunks) {
        decode_charges(p, base, lane, len, c);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) sum += c[i];
      }
      decode_charges(p, 0, lane, len, c);         // (kept for the search)
#pragma unroll
      for (int i = 0; i < kChunks; ++i) sum += c[i];
      total = warp_sum(sum) * p.units;
      range();
      at = -1;
      for (int base = 0; at < 0; base += 32 * kChunks) {
        if (base) decode_charges(p, base, lane, len, c);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          if (at >= 0) break;
          const int in = __reduce_add_sync(0xffffffffu, (unsigned)c[i]);   // (32 of at most 2^25 + 2)
          if (before + in > first || base + 32 * (i + 1) >= p.B) at = base + 32 * i, mine = c[i], my_len = len[i];
          else before += in;
        }
      }
      inc = scan(mine);
    }
    const unsigned here = __ballot_sync(0xffffffffu, mine > 0 && before + inc - mine <= first);
    if (lane == 31 - __clz(here)) {
      const long long off = start - (before + inc - mine) * p.units;
      const int unit = (int)quotient(off, mine);
      *s_walk = DecodeWalk{at + lane, unit, (int)(off - (long long)unit * mine), end - start};
      *s_len = my_len;
    }
  } else if (blockIdx.x == 0) {   // lengths that the tables cannot hold are reported once
    for (int i = threadIdx.x; i < p.B; i += 32 * kDecWarps) if (const int len = p.kv_lens[i]; len < 0 || len > p.max_len) atomicOr(p.status, fa_host::kStatusIndex);
  }
  __syncthreads();
  DecodeWalk walk = *s_walk;
  const WaitCtx wc{s_abort, p.status, p.timeout_ns};
  const int box_shift = min(p.page_shift, 6);     // slots per copy
  const int box = 1 << box_shift;

  if (warp == kDecWarps) {
    // ============================================================ producer
    int len = *s_len;
    int it = 0;
    bool dead = false;
    const int nsub = kDecTile >> box_shift;           // copies of K (and V) per tile
    const uint32_t sub_bytes = (uint32_t)box * D * 2;
    while (walk.left > 0 && !dead) {
      const DecodeSpan s = decode_span(p, len);
      const int b = walk.b, hk = walk.unit / p.groups;
      const DecodePiece d = decode_step(walk, s.n, p.units);
      if (walk.b != b && walk.left > 0) len = decode_len(p, walk.b);
      const int t0 = d.t0, nt = d.nt;
      const int n_pages = (s.hi + (1 << p.page_shift) - 1) >> p.page_shift;
      // Lane i looks up sub-block c0 + i of the unit (box keys each): page, first slot, first key.
      auto look_up = [&](int c, int& id, int& slot, int& key) {
        id = -1, slot = 0, key = -1;
        if (c >= (t0 + nt) * nsub) return;
        int page;
        if (p.sel) {
          const int spp = p.page_shift - box_shift;    // log2 sub-blocks per page
          const int at = c >> spp;
          if (at >= s.listed) return;
          page = p.sel[((long long)b * p.Hkv + hk) * p.max_sel + at];
          if (page < 0 || page >= n_pages) return;
          slot = (c & ((1 << spp) - 1)) << box_shift;
          key = (page << p.page_shift) + slot;
        } else {
          key = s.first * kDecTile + (c << box_shift);
          page = key >> p.page_shift;
          slot = key & ((1 << p.page_shift) - 1);
        }
        if (key >= s.hi || key + box <= s.lo) {           // (also any key of an empty sequence)
          key = -1;
          return;
        }
        id = p.table[(long long)b * p.table_stride + page];
        if (id < 0 || id >= p.num_pages) {
          atomicOr(p.status, fa_host::kStatusIndex);
          id = key = -1;
        }
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
        // lanes 0 to 3: the first key of each 16
        const int off = 16 * lane;
        const int first = __shfl_sync(0xffffffffu, key, in * nsub + ((off & (kDecTile - 1)) >> box_shift));
        if (lane < 4) s_meta[st * 4 + lane] = first < 0 ? -1 : first + (off & (box - 1));
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(FULL(st), 2u * sub_bytes * __popc(live));
        __syncwarp();
        if (mine) {
          const uint32_t dst = sbase + (uint32_t)st * 2 * SM::kHalf + (uint32_t)sub * sub_bytes;
          tma_load_5d(dst, &params.tm_k, FULL(st), slot, hk, id);
          tma_load_5d(dst + SM::kHalf, &params.tm_v, FULL(st), slot, hk, id);
        }
        // the next look-up, a look-up's tiles ahead of its use
        if (in == 0) look_up((t0 + j + per) * nsub + lane, id2, slot2, key2);
      }
    }
    // Every copy lands before the CTA ends, whether or not some wait expired: a consumer may give up
    // on a copy in flight after the producer's last wait.  (Where none did, the consumers wait for the
    // same phases.)
    if (lane == 0)
      for (int i = max(0, it - NS); i < it; ++i) drain_bar(FULL(i % NS), (i / NS) & 1, wc.timeout);
    return;
  }

  // ============================================================ consumers
  constexpr int DT = D / 64;                         // 16-channel steps of this warp's quarter of O
  const int g = lane >> 2, t4 = lane & 3;
  uint4* s_p = reinterpret_cast<uint4*>(smem + SM::kPOff);
  uint4* s_q = reinterpret_cast<uint4*>(smem + SM::kQOff);
  float* s_max = reinterpret_cast<float*>(smem + SM::kMaxOff);
  float* s_sum = reinterpret_cast<float*>(smem + SM::kSumOff);
  auto sync = [&]() { named_sync(1, 32 * kDecWarps); };
  // In a stage, 16 keys start at place(q) for q = 0 .. 3 (a copy is [D / 64][box][64]); a row of 64
  // channels is 128 bytes, its 16-byte chunk c at place c ^ (row & 7).
  const uint32_t half = (uint32_t)box * 128;
  auto place = [&](int q) {
    return (uint32_t)((16 * q) >> box_shift) * (uint32_t)box * D * 2 + (uint32_t)((16 * q) & (box - 1)) * 128;
  };
  // this lane's row of each ldmatrix: keys as stored for K; for V transposed, keys by 8, channels by 8
  const uint32_t klane = place(warp) + (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
  uint32_t vlane[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) {
    const int ch = 16 * (warp * DT + i);
    vlane[i] = SM::kHalf + (uint32_t)(ch >> 6) * half + ((lane & 7) + ((lane >> 4) << 3)) * 128 +
               ((((ch & 63) / 8 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
  }

  int next_len = *s_len;
  int it = 0;
  bool dead = false;
  auto first_row = [&](const DecodeWalk& w) {
    return ((long long)w.b * p.Hkv + w.unit / p.groups) * p.rows + (w.unit % p.groups) * 8 * NT;
  };
  while (walk.left > 0) {
    const int len = next_len, rg = walk.unit % p.groups, b = walk.b;
    const long long row0 = first_row(walk);
    const DecodeSpan s = decode_span(p, len);
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

    // Q as the B operand: lane (g, t4) holds row g, channels 2 t4, 2 t4 + 1 and + 8 of every step;
    // two steps per word
    uint4 qf[SM::kQShared ? 1 : NT][SM::kQShared ? 1 : KS / 2];
    auto load_q = [&](int n, int k2) {
      const int row = n * 8 + g;
      const uint32_t* x = reinterpret_cast<const uint32_t*>(p.q + (row0 + row) * D + k2 * 32) + t4;
      return row < rows ? make_uint4(x[0], x[4], x[8], x[12]) : make_uint4(0, 0, 0, 0);
    };
    if constexpr (SM::kQShared) {   // (the last unit's reads of it lie before its last barrier)
      for (int i = warp; i < NT * KS / 2; i += kDecWarps) s_q[i * 32 + lane] = load_q(i / (KS / 2), i % (KS / 2));
      sync();
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) qf[n][k2] = load_q(n, k2);
    }
    const int tok_min = len - p.Sq;                                       // the first row's token
    const int low_max = p.pre_tokens >= 0 ? len - 1 - p.pre_tokens : 0;   // lowest key that all rows see

    float o[NT][DT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = kNoScore;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < DT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

    for (int j = 0; j < d.nt; ++j, ++it) {
      const int st = it % NS;
      // (after an expired wait: the barriers below still see every warp, the answer is void)
      if (!dead) dead = !__all_sync(0xffffffffu, wait_bar(FULL(st), (it / NS) & 1, wc));
      const int4 keys = *reinterpret_cast<const int4*>(s_meta + 4 * st);
      const uint32_t base = sbase + (uint32_t)st * 2 * SM::kHalf;
      const int kq = warp == 0 ? keys.x : warp == 1 ? keys.y : warp == 2 ? keys.z : keys.w;
      // 16 keys that were not copied (their K is stale) lie past every row's token
      const int key0 = kq < 0 ? 0x7FFFFF00 : kq;
      float c[NT][4], c2[NT][4];       // (two chains of products: with few rows their latency shows)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[n][e] = c2[n][e] = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < KS / 2; ++k2) {
        uint32_t a0[4], a1[4];
        const uint32_t at = base + (klane ^ (uint32_t)((k2 & 1) << 6)) + (k2 >> 1) * half;
        ldmatrix4(at, a0);
        ldmatrix4(at ^ 32u, a1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 x = SM::kQShared ? s_q[(n * (KS / 2) + k2) * 32 + lane] : qf[SM::kQShared ? 0 : n][SM::kQShared ? 0 : k2];
          mma_16x8<BF16>(c[n], a0, x.x, x.y);
          mma_16x8<BF16>(NT > 2 ? c[n] : c2[n], a1, x.z, x.w);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[n][e] += c2[n][e];
      // scores in log2 units; lane (g, t4): keys g (c0, c1) and g + 8 (c2, c3), rows 2 t4, 2 t4 + 1
      float over = -INFINITY;        // the most that a score exceeds its row's reference by
      const bool all = key0 + 15 <= tok_min && key0 >= low_max;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[n][e] *= p.scale_log2;
      if (!all) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + g + 8 * (e >> 1);
            const int t = tok_min + (p.Sq == 1 ? 0 : (rg * 8 * NT + n * 8 + 2 * t4 + (e & 1)) % p.Sq);
            if (key > t || (p.pre_tokens >= 0 && key < t - p.pre_tokens)) c[n][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) over = fmaxf(over, c[n][e] - m[n][e & 1]);   // (NaN is dropped)
      if (named_or(2, 32 * kDecWarps, over > kMaxOver + kLift<BF16>)) {   // the references move up
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float mx[2] = {fmaxf(c[n][0], c[n][2]), fmaxf(c[n][1], c[n][3])};
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], w));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], w));
          }
          if (g == 0) *reinterpret_cast<float2*>(s_max + (warp * NT + n) * 8 + 2 * t4) = make_float2(mx[0], mx[1]);
        }
        sync();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float top[2] = {m[n][0], m[n][1]}, f[2];
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            const float2 x = *reinterpret_cast<const float2*>(s_max + (w * NT + n) * 8 + 2 * t4);
            top[0] = fmaxf(top[0], x.x - kLift<BF16>);
            top[1] = fmaxf(top[1], x.y - kLift<BF16>);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[e] = ex2_approx(m[n][e] - top[e]);
            m[n][e] = top[e];
            l[n][e] *= f[e];
          }
#pragma unroll
          for (int i = 0; i < DT; ++i) {
            o[n][i][0] *= f[0];
            o[n][i][1] *= f[1];
            o[n][i][2] *= f[0];
            o[n][i][3] *= f[1];
          }
        }
      }
      // this warp's channels of V: their way from shared memory is hidden by the exponentials (up to
      // 32 rows; with more O leaves no registers for it)
      uint32_t v[4][DT][4];
      auto load_v = [&](int q) {
#pragma unroll
        for (int i = 0; i < DT; ++i) ldmatrix4_trans(base + place(q) + vlane[i], v[q][i]);
      };
      if constexpr (NT <= 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) load_v(q);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float p0 = ex2_approx(c[n][0] - m[n][0]), p1 = ex2_approx(c[n][1] - m[n][1]);
        const float p2 = ex2_approx(c[n][2] - m[n][0]), p3 = ex2_approx(c[n][3] - m[n][1]);
        l[n][0] += p0 + p2;
        l[n][1] += p1 + p3;
        const uint32_t h0 = pack16x2<BF16>(p0, p1), h1 = pack16x2<BF16>(p2, p3);
        s_p[(warp * NT + n) * 32 + lane] =
            make_uint4(transpose8(h0), transpose8(h1), transpose8(pack_residual_x2(p0, p1, h0, BF16)),
                       transpose8(pack_residual_x2(p2, p3, h1, BF16)));
      }
      sync();
      // Keys that no row sees have P = 0, and their V may hold anything (or be stale): it becomes 0.
      const int4 hi4 = make_int4(keys.x + 16, keys.y + 16, keys.z + 16, keys.w + 16);
      const bool whole = min(min(keys.x, keys.y), min(keys.z, keys.w)) >= s.lo &&
                         max(max(hi4.x, hi4.y), max(hi4.z, hi4.w)) <= s.hi;
      auto keep_seen = [&](int q) {
        const int k0 = q == 0 ? keys.x : q == 1 ? keys.y : q == 2 ? keys.z : keys.w;
        auto seen = [&](int k) { return k0 >= 0 && k0 + k >= s.lo && k0 + k < s.hi; };
        // keys 2 t4, 2 t4 + 1 and + 8
        const uint32_t keep0 = (seen(2 * t4) ? 0xffffu : 0u) | (seen(2 * t4 + 1) ? 0xffff0000u : 0u);
        const uint32_t keep1 = (seen(2 * t4 + 8) ? 0xffffu : 0u) | (seen(2 * t4 + 9) ? 0xffff0000u : 0u);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          v[q][i][0] &= keep0;
          v[q][i][1] &= keep0;
          v[q][i][2] &= keep1;
          v[q][i][3] &= keep1;
        }
      };
      if constexpr (NT > 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) load_v(q);
      }
      if (!whole) {
#pragma unroll
        for (int q = 0; q < 4; ++q) keep_seen(q);
      }
      // The tile's sum starts from zero and is added to O by itself: the matrix instructions cut off what
      // they add (about 2^-24 of the sum so far each, always towards zero), and eight of them per tile on
      // a running O lost 8.6e-4 of it over 131072 keys of one CTA, four times an fp16 rounding.  Columns
      // of 8 rows are summed NB at a time, so that there are products that do not wait for each other.
      // (16 sequences of 4096 tokens, 8 KV heads of 128: on a running O 57.0 us at 32 rows and 81.5 at 48,
      // column by column 60.6 and 85, so 59.2 and 77.8; up to 24 rows all the same.)
      constexpr int NB = NT > 4 ? 3 : NT > 2 ? 2 : 1;
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += NB) {
        float sum[NB][DT][4];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int i = 0; i < DT; ++i) sum[j][i][0] = sum[j][i][1] = sum[j][i][2] = sum[j][i][3] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            if (n0 + j >= NT) break;
            const uint4 pp = s_p[(q * NT + n0 + j) * 32 + lane];
#pragma unroll
            for (int i = 0; i < DT; ++i) mma_16x8<BF16>(sum[j][i], v[q][i], pp.x, pp.y);
#pragma unroll
            for (int i = 0; i < DT; ++i) mma_16x8<BF16>(sum[j][i], v[q][i], pp.z, pp.w);
          }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          if (n0 + j >= NT) break;
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n0 + j][i][e] += sum[j][i][e];
        }
      }
      // A warp that gave up hands back no stage: its copy may still be in flight.  The producer's next
      // wait for that stage then fails too, so that no stage is armed before its last copy has landed.
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
    const long long part0 = (2LL * blockIdx.x + (d.t0 == 0 ? 1 : 0)) * (8 * NT);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float2 x = *reinterpret_cast<const float2*>(s_sum + (w * NT + n) * 8 + 2 * t4);
        sum[0] += x.x;
        sum[1] += x.y;
      }
      if (direct) {
        const float i0 = sum[0] > 0.f ? 1.f / sum[0] : 0.f, i1 = sum[1] > 0.f ? 1.f / sum[1] : 0.f;
        const int row = n * 8 + g;
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          // transposed back: lane (g, t4) gets row g, channels 2 t4 and 2 t4 + 1 (and + 8)
          const uint32_t x = transpose8(pack16x2<BF16>(o[n][i][0] * i0, o[n][i][1] * i1));
          const uint32_t y = transpose8(pack16x2<BF16>(o[n][i][2] * i0, o[n][i][3] * i1));
          if (row < rows) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (row0 + row) * D + 16 * (warp * DT + i)) + t4;
            dst[0] = x;
            dst[4] = y;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* dst = p.part_o + (part0 + n * 8 + 2 * t4 + e) * D + 16 * warp * DT + g;
#pragma unroll
          for (int i = 0; i < DT; ++i) {
            dst[16 * i] = o[n][i][e];
            dst[16 * i + 8] = o[n][i][e + 2];
          }
        }
      }
      if (warp == 0 && g == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = n * 8 + 2 * t4 + e;
          if (!direct) p.part_ml[part0 + row] = make_float2(m[n][e], sum[e]);
          else if (row < rows)
            p.lse[row0 + row] = sum[e] > 0.f ? (m[n][e] + log2f(sum[e])) * 0.6931471805599453f : INFINITY;
        }
      }
    }
  }
}

// Joins the pieces of the units that several CTAs shared: the schedule is
// computed anew from the lengths, the pieces summed in an order that depends on
// it alone (the same bits every time).  WPR warps per row: 1 where there are many
// rows, 8 where there are few, 32 where a unit may have so many pieces (one KV
// head over 131072 tokens has one per CTA, 304).
template <bool BF16, int D, int WPR>
__global__ void __launch_bounds__(WPR > 8 ? 32 * WPR : 256) fa_decode_join_kernel(const __grid_constant__ DecodeCore p, int rows8) {
  constexpr int kWarps = WPR > 8 ? WPR : 8;
  __shared__ __align__(16) float s_o[WPR][D];
  __shared__ float2 s_ml[WPR];
  // The schedule before the wait: by the time this kernel runs every CTA of the decode kernel has
  // seen the kernels before it finish, so that the lengths are final.
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kWarps / WPR) + warp / WPR;
  const int part = warp % WPR;
  const long long per_b = (long long)p.Hkv * p.rows;
  const bool none = row >= per_b * p.B;                  // (a row for all warps of a block where WPR > 1)
  const int b = none ? p.B - 1 : (int)(row / per_b);
  const int in_b = (int)(row % per_b);
  const int hk = in_b / p.rows, r = in_b % p.rows;
  const int rg = r / rows8, rr = r % rows8;
  long long total = 0, before = 0;
  auto add_up = [&](int base, int end) {                 // charges of 256 sequences, and of those before `end`
    int len[kChunks], c[kChunks];
    decode_charges(p, base, lane, len, c);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      total += c[i];
      if (base + 32 * i + lane < end) before += c[i];
    }
  };
  if (p.B <= 32 * kChunks) {
    add_up(0, b);
    total = warp_sum(total);
    before = warp_sum(before);
  } else {   // shared by the block's warps, up to the sequence of its first row; the few from there by each
    __shared__ long long s_sum[kWarps][2];
    const int b0 = (int)((long long)blockIdx.x * (kWarps / WPR) / per_b);
    for (int base = 32 * kChunks * warp; base < p.B; base += 32 * kChunks * kWarps) add_up(base, b0);
    total = warp_sum(total);
    before = warp_sum(before);
    if (lane == 0) s_sum[warp][0] = total, s_sum[warp][1] = before;
    __syncthreads();
    total = warp_sum(lane < kWarps ? s_sum[lane][0] : 0);
    before = (lane < kWarps ? s_sum[lane][1] : 0) + (b0 + lane < b ? decode_span(p, decode_len(p, b0 + lane)).n + kUnitTiles : 0);
    before = warp_sum(before);                           // (b - b0 is less than the block's 8 rows)
  }
  if (none) return;
  total *= p.units;
  const int ctas = decode_ctas(p, total);
  const int n = decode_span(p, decode_len(p, b)).n;
  const long long t0 = before * p.units + (long long)(hk * p.groups + rg) * (n + kUnitTiles) + kUnitTiles;
  const int c0 = decode_owner(total, ctas, t0), c1 = decode_owner(total, ctas, t0 + n - 1);
  pdl_wait_prior();
  if (c0 == c1) return;          // finished by its CTA
  auto at = [&](int c) { return (2LL * c + (c == c0 ? 1 : 0)) * rows8 + rr; };
  // Some pieces at a time: their loads wait for nothing but each other.
  constexpr int E = D / 32, kPieces = WPR > 1 ? 4 : 8;
  float m = kNoScore, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int cb = c0 + part; cb <= c1; cb += WPR * kPieces) {
    float2 ml[kPieces];
    float x[kPieces][E];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = cb + i * WPR;
      ml[i] = make_float2(kNoScore, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) x[i][e] = 0.f;
      if (c <= c1) {
        const long long a = at(c);
        ml[i] = p.part_ml[a];
        const float* src = p.part_o + a * D + E * lane;
        if constexpr (E == 4) {
          const float4 y = *reinterpret_cast<const float4*>(src);
          x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(src);
          x[i][0] = y.x, x[i][1] = y.y;
        }
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) top = fmaxf(top, ml[i].x);
    const float keep = ex2_approx(m - top);
    m = top;
    l *= keep;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const float f = ex2_approx(ml[i].x - top);     // (a piece that is none is all 0)
      l = fmaf(f, ml[i].y, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, x[i][e], o[e]);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[part][E * lane + e] = o[e];
    if (lane == 0) s_ml[part] = make_float2(m, l);
    __syncthreads();
    if (part) return;
    const float2 ml = lane < WPR ? s_ml[lane] : make_float2(kNoScore, 0.f);
    m = ml.x;
#pragma unroll
    for (int w = WPR / 2; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    m = __shfl_sync(0xffffffffu, m, 0);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 8
    for (int w = 0; w < WPR; ++w) {
      const float f = ex2_approx(s_ml[w].x - m);
      l = fmaf(f, s_ml[w].y, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, s_o[w][E * lane + e], o[e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D) + (E / 2) * lane;
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack16x2<BF16>(o[e] * inv, o[e + 1] * inv);
  if (lane == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : INFINITY;
}

}  // namespace fa
