// fa_kv_append: new keys (rotated) and values into their pages, rotated queries
// to q_out, page bounds brought up to date.
//
// Each thread owns 16 channels of a row as two 16-byte vectors A and B that
// hold whole pairs: with pairs (j, j + r/2) A and B are the same 8 channels of
// the two halves, with pairs (2j, 2j + 1), and past the rotated channels, they
// are neighbours.  A row is D / 16 threads, so a block of 256 threads takes 32
// (D 128) or 64 rows a step: `tp` tokens of one page times the heads that
// are left.  A block stays inside one page of one sequence, so that a page's
// bounds have one writer: no atomics, the same result every time.
//
// Bound by HBM: every row is read and written once.  Four prompts of up to 4096
// tokens, 32 + 2 * 8 heads of 128, bounds kept: 190 MB in 33.3 us, 5.71 TB/s.
// Four blocks of 64 registers per SM with two rows in flight per thread (five
// blocks 34.8 us, six spill, 46 us; one row in flight 37 us; queries and keys of
// both pairings in one kernel 35.4 us).  The lengths and the page id are a chain
// of three loads, of which the tokens wait for one only.  One token each of 128
// sequences: 2.3 us, a launch and that chain.
#pragma once
#include <type_traits>

#include "fa_paged.cuh"

namespace fa {

constexpr int kAppendThreads = 256;
constexpr int kAppendBlocks = 64;       // pieces per SM up to which each has a block of its own
constexpr int kAppendLoopBlocks = 32;   // blocks per SM past that
constexpr int kBatch = 2;      // rows per thread in flight (queries: heads, values: tokens)

struct AppendParams {
  PagedKv kv;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;
  uint16_t* qo;
  long long k_sb, k_sh, k_ss, v_sb, v_sh, v_ss, q_sb, q_sh, q_ss, o_sb, o_sh, o_ss;
  const float* cos;
  const float* sin;
  int rot_dim, max_pos;
  const int32_t* kv_lens;
  const int32_t* new_lens;
  int Hq, Hkv, Snew;
  int chunks;              // pages that one sequence's new tokens can touch
  int tp_shift;            // tokens per step = 1 << tp_shift
  int q_heads;             // heads per block of the Q blocks (the K and V blocks: those of one step)
  int k_items, q_items;    // blocks per page for K (V as many), for Q
  int* status;
};

// A piece of the work: one page of one sequence (`rest`), some heads (`item`) of its K, V or Q.  KIND: which
// of the three, or kAppendAny by the item (one way for all up to the tokens' loads: a copy for each kind
// takes a call of few tokens 0.1 us longer, on its way through the instruction cache).
constexpr int kAppendK = 0, kAppendV = 1, kAppendQ = 2, kAppendAny = 3;
template <bool BF16, int D, bool INTERLEAVED, int KIND>
__device__ __forceinline__ void append_piece(const AppendParams& p, int item, int rest) {
  constexpr int L = D / 16;                    // threads per row
  constexpr int kRows = kAppendThreads / L;    // rows per step
  __shared__ uint4 s_red[4][8][L];             // [min A, min B, max A, max B][warp][thread of the row]
  const int chunk = rest % p.chunks, b = rest / p.chunks;

  const int ps_shift = p.kv.page_shift, ps = 1 << ps_shift;
  const int n0 = p.new_lens ? p.new_lens[b] : p.Snew, len0 = p.kv_lens[b];
  const int n_new = min(max(n0, 0), p.Snew);
  if (n0 != n_new && threadIdx.x == 0) atomicOr(p.status, fa_host::kStatusIndex);
  if (n_new == 0) return;
  const int before = paged_len(p.kv, len0, p.status);
  if (before < 0) return;
  const int page = (before >> ps_shift) + chunk;
  // tokens [t0, t1) of the sequence, by position (64 bits: `before` may be near 2^31)
  const long long p0 = (long long)page << ps_shift;
  const long long end = min((long long)before + n_new, p0 + ps);
  if (max((long long)before, p0) >= end) return;
  if (page >= p.kv.max_pages) {
    if (threadIdx.x == 0) atomicOr(p.status, fa_host::kStatusIndex);
    return;
  }
  const int t0 = max(before, (int)p0);
  int t1 = (int)end;
  // (looked at only before the first store: the loads of the tokens do not wait for it)
  const int id = p.kv.table[(long long)b * p.kv.table_stride + page];
  auto no_page = [&]() {
    if (id >= 0 && id < p.kv.num_pages) return false;
    atomicOr(p.status, fa_host::kStatusIndex);
    return true;
  };
  if (p.rot_dim && t1 > p.max_pos) {
    if (threadIdx.x == 0) atomicOr(p.status, fa_host::kStatusIndex);
    t1 = p.max_pos;
    if (t0 >= t1) return;
  }

  const int part = threadIdx.x % L;
  const int row = threadIdx.x / L;
  const int tp = 1 << p.tp_shift;
  const int tl = row & (tp - 1), hl = row >> p.tp_shift, hp = kRows >> p.tp_shift;
  const bool turns = part < p.rot_dim / 16;
  const bool halves = turns && !INTERLEAVED;
  const int offA = halves ? 8 * part : 16 * part;
  const int offB = halves ? 8 * part + p.rot_dim / 2 : 16 * part + 8;
  const int half = p.rot_dim / 2;

  float c[8], s[8];
  auto angles = [&](int t) {
    if (!turns) return;
    const float4* cp = reinterpret_cast<const float4*>(p.cos + (long long)t * half + 8 * part);
    const float4* sp = reinterpret_cast<const float4*>(p.sin + (long long)t * half + 8 * part);
    const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
    c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
  };
  // in fp32, each channel rounded once to the cache's type
  auto rotate = [&](uint4& wa, uint4& wb) {
    if (!turns) return;
    float a[8], d[8];
    unpack8<BF16>(wa, a);
    unpack8<BF16>(wb, d);
    if constexpr (INTERLEAVED) {
      float x[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = a[j], x[8 + j] = d[j];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = x[2 * j], o = x[2 * j + 1];
        x[2 * j] = e * c[j] - o * s[j];
        x[2 * j + 1] = e * s[j] + o * c[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = x[j], d[j] = x[8 + j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = a[j], o = d[j];
        a[j] = e * c[j] - o * s[j];
        d[j] = e * s[j] + o * c[j];
      }
    }
    wa = pack8<BF16>(a);
    wb = pack8<BF16>(d);
  };
  // (no loads by the read-only path: the kernel may have started before the one that wrote its
  // inputs ended, and only ordinary loads are promised to see those writes after the wait)
  auto ld = [](const uint16_t* x) { return *reinterpret_cast<const uint4*>(x); };
  auto st = [](uint16_t* x, uint4 w) { *reinterpret_cast<uint4*>(x) = w; };

  if (KIND == kAppendQ || (KIND == kAppendAny && item >= 2 * p.k_items)) {   // ---------------- queries: one set of angles for all heads
    const int h0 = (item - 2 * p.k_items) * p.q_heads;
    const int h1 = min(p.Hq, h0 + p.q_heads);
    for (int t = t0 + tl; t < t1; t += tp) {
      const uint16_t* src = p.q + b * p.q_sb + (long long)(t - before) * p.q_ss;
      uint16_t* dst = p.qo + b * p.o_sb + (long long)(t - before) * p.o_ss;
      angles(t);
      for (int h = h0 + hl; h < h1; h += kBatch * hp) {
        uint4 wa[kBatch], wb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (h + i * hp >= h1) break;
          wa[i] = ld(src + (h + i * hp) * p.q_sh + offA);
          wb[i] = ld(src + (h + i * hp) * p.q_sh + offB);
        }
        if (no_page()) return;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (h + i * hp >= h1) break;
          rotate(wa[i], wb[i]);
          st(dst + (h + i * hp) * p.o_sh + offA, wa[i]);
          st(dst + (h + i * hp) * p.o_sh + offB, wb[i]);
        }
      }
    }
    return;
  }
  if (KIND == kAppendV || (KIND == kAppendAny && item >= p.k_items)) {       // ---------------- values: copied
    const int h = (item - p.k_items) * hp + hl;
    if (h >= p.Hkv) return;
    const uint16_t* src = p.v + b * p.v_sb + h * p.v_sh + 16 * part;
    for (int t = t0 + tl; t < t1; t += kBatch * tp) {
      uint4 wa[kBatch], wb[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (t + i * tp >= t1) break;
        const uint16_t* x = src + (long long)(t + i * tp - before) * p.v_ss;
        wa[i] = ld(x);
        wb[i] = ld(x + 8);
      }
      if (no_page()) return;
      uint16_t* dst = p.kv.v + (long long)id * p.kv.v_sp + h * p.kv.v_sh + 16 * part;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (t + i * tp >= t1) break;
        uint16_t* y = dst + (long long)((t + i * tp) & (ps - 1)) * p.kv.v_ss;
        st(y, wa[i]);
        st(y + 8, wb[i]);
      }
    }
    return;
  }
  // ---------------- keys: rotated; per page and channel the least and largest as stored
  const uint32_t kInf = BF16 ? 0x7F807F80u : 0x7C007C00u;
  const bool kept = (t0 & (ps - 1)) != 0;   // slot 0 holds an older key
  const int h = item * hp + hl;
  const bool on = h < p.Hkv;
  uint4 mn[2], mx[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    mn[j] = make_uint4(kInf, kInf, kInf, kInf);
    mx[j] = make_uint4(kInf | 0x80008000u, kInf | 0x80008000u, kInf | 0x80008000u, kInf | 0x80008000u);
  }
  auto widen = [&](int j, uint4 lo, uint4 hi) {
    mn[j] = make_uint4(min16x2<BF16>(mn[j].x, lo.x), min16x2<BF16>(mn[j].y, lo.y),
                       min16x2<BF16>(mn[j].z, lo.z), min16x2<BF16>(mn[j].w, lo.w));
    mx[j] = make_uint4(max16x2<BF16>(mx[j].x, hi.x), max16x2<BF16>(mx[j].y, hi.y),
                       max16x2<BF16>(mx[j].z, hi.z), max16x2<BF16>(mx[j].w, hi.w));
  };
  if (on) {
    const uint16_t* src = p.k + b * p.k_sb + h * p.k_sh;
    for (int t = t0 + tl; t < t1; t += tp) {
      const uint16_t* x = src + (long long)(t - before) * p.k_ss;
      uint4 wa = ld(x + offA), wb = ld(x + offB);
      angles(t);
      rotate(wa, wb);
      if (no_page()) break;
      uint16_t* y = p.kv.k + (long long)id * p.kv.k_sp + h * p.kv.k_sh + (long long)(t & (ps - 1)) * p.kv.k_ss;
      st(y + offA, wa);
      st(y + offB, wb);
      widen(0, wa, wa);
      widen(1, wb, wb);
    }
  }
  if (no_page()) return;   // (block-uniform)
  if (!p.kv.k_min) return;
  // join the tokens of a step: first the rows of the warp, then the warps.  With 2^x tokens
  // a step, rows that differ in the low x bits of their number hold the same head.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto other = [&](uint4 w, int m) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, w.x, m), __shfl_xor_sync(0xffffffffu, w.y, m),
                      __shfl_xor_sync(0xffffffffu, w.z, m), __shfl_xor_sync(0xffffffffu, w.w, m));
  };
  for (int m = L; m < 32 && m < (L << p.tp_shift); m <<= 1) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 lo = other(mn[j], m), hi = other(mx[j], m);
      widen(j, lo, hi);
    }
  }
  const int wpt = (L << p.tp_shift) >> 5;   // warps that share a head's tokens (0 or 1: none)
  if (wpt > 1) {                            // block-uniform
    if (lane < L) {
#pragma unroll
      for (int j = 0; j < 2; ++j) s_red[j][warp][lane] = mn[j], s_red[2 + j][warp][lane] = mx[j];
    }
    __syncthreads();
    if (lane < L && warp % wpt == 0) {
      for (int w = 1; w < wpt; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j) widen(j, s_red[j][warp + w][lane], s_red[2 + j][warp + w][lane]);
    }
  }
  if (on && tl == 0) {
    const long long at = ((long long)id * p.Hkv + h) * D;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int off = j ? offB : offA;
      uint4* lo = reinterpret_cast<uint4*>(p.kv.k_min + at + off);
      uint4* hi = reinterpret_cast<uint4*>(p.kv.k_max + at + off);
      if (kept) widen(j, *lo, *hi);
      *lo = mn[j];
      *hi = mx[j];
    }
  }
}

// A block per piece that Snew has room for, or, where that were more than kAppendBlocks per SM,
// kAppendLoopBlocks per SM (a multiple of the items) that each keep to one item and look at 32 of their
// pages at once for those that hold tokens: a padded batch may mix prompts with single tokens.  Each
// kind of piece has a loop of its own: one loop around all three needed 120 registers, spilled 150
// bytes at the 64 that four blocks per SM leave, and took 22 % longer over full pieces.  (8 prompts of
// 4096, pages of 64: 125.6 us, 6.41 TB/s, a block per piece 125.2; 32 sequences padded to 4096 tokens,
// pages of 16, one of them that long and the others one token: 24.5 and 117 us; all of one token 9.8
// and 104 us.  16 blocks per SM: 132, 24.2 and 8.0 us; 64: 127, 30.5 and 15.6.  Just below the limit a
// block per piece is ahead: the four prompts above 33.0 us, looping 34.2.)
template <bool BF16, int D, bool INTERLEAVED, bool MANY>
__global__ void __launch_bounds__(kAppendThreads, 4) fa_kv_append_kernel(const AppendParams p, int pieces) {
  pdl_launch_dependents();
  pdl_wait_prior();
  const unsigned items = 2 * p.k_items + p.q_items;
  const int item = (int)(blockIdx.x % items);
  if constexpr (!MANY) {
    append_piece<BF16, D, INTERLEAVED, kAppendAny>(p, item, (int)(blockIdx.x / items));
  } else {
    auto loop = [&](auto kind) {
      constexpr int KIND = decltype(kind)::value;
      const unsigned pages = (unsigned)pieces / items, step = gridDim.x / items;
#pragma unroll 1
      for (unsigned at0 = blockIdx.x / items; at0 < pages; at0 += 32 * step) {
        const unsigned at = at0 + step * (threadIdx.x & 31);
        bool some = false;
        if (at < pages) {
          const int chunk = at % p.chunks, b = at / p.chunks;
          const int n = p.new_lens ? min(p.new_lens[b], p.Snew) : p.Snew, len = p.kv_lens[b];
          // (whatever is to be reported, the piece of chunk 0 reports)
          some = chunk == 0 || (n > 0 && len >= 0 && (long long)len + n > ((long long)(len >> p.kv.page_shift) + chunk) << p.kv.page_shift);
        }
#pragma unroll 1
        for (unsigned live = __ballot_sync(0xffffffffu, some); live; live &= live - 1) {
          append_piece<BF16, D, INTERLEAVED, KIND>(p, item, (int)(at0 + step * (__ffs(live) - 1)));
          if constexpr (KIND == kAppendK) __syncthreads();   // (its shared memory)
        }
      }
    };
    if (item >= 2 * p.k_items) loop(std::integral_constant<int, kAppendQ>{});
    else if (item >= p.k_items) loop(std::integral_constant<int, kAppendV>{});
    else loop(std::integral_constant<int, kAppendK>{});
  }
}

}  // namespace fa
