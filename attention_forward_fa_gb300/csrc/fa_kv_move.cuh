// fa_kv_read: tokens out of their pages into dense 16-bit rows.
// fa_kv_keep: accepted drafts to the places behind the tokens before them.
//
// Both move rows and compute next to nothing: a row of an 8-bit cache is read as
// D bytes and a scale byte, and multiplied once; the rest is copied.
//
// Measured: two sequences of 65535 tokens, 16 KV heads of 64, fp16, pages of 16, read
// in 159 us, 6.7 TB/s; 8028 tokens of 8 heads of 128 out of 8 bits in 11.6 us, 4.1 TB/s
// (launch, three dependent loads, half of the issue slots).  Up to 12 drafts of each of 64
// sequences kept in 6.8 us, 4 of one in 2.9: a launch and five dependent loads.
#pragma once
#include <type_traits>

#include "fa_paged8.cuh"

namespace fa {

struct ReadParams {
  PagedKv kv;
  const uint8_t* k_scale;   // 8-bit caches
  const uint8_t* v_scale;
  uint16_t* k;
  uint16_t* v;
  long long k_sb, k_sh, k_ss, v_sb, v_sh, v_ss;
  const int32_t* starts;    // or null: 0
  const int32_t* lens;
  int Hkv, S;
  int chunks;               // runs of kReadTokens tokens that S has room for
  int e5m2;
  int* status;
};
constexpr int kReadThreads = 256;
constexpr int kReadTokens = 64;      // of one head, K and V, per block

// A block per (run of tokens, head, sequence), a thread 8 channels of a row, so that both the loads and the
// stores of a warp are whole lines (16 codes a thread, whose two stores fill half a sector each, took 13.9 us
// instead of 10.4 for 8028 tokens of 8 heads of 128); all of a block's loads are in flight at once, behind
// lengths and page ids.
template <bool BF16, int D, bool EIGHT>
__global__ void __launch_bounds__(kReadThreads) fa_kv_read_kernel(const ReadParams p) {
  constexpr int E = EIGHT ? 1 : 2;                     // bytes of an element
  using Word = std::conditional_t<EIGHT, uint2, uint4>;    // 8 channels, 16 bytes of the answer
  constexpr int L = D / 8;                             // threads per row
  constexpr int kRows = kReadThreads / L, kEach = kReadTokens / kRows;
  static_assert(kReadTokens % kRows == 0, "whole steps");
  pdl_launch_dependents();
  pdl_wait_prior();
  const int chunk = blockIdx.x % p.chunks;
  const int rest = blockIdx.x / p.chunks;
  const int h = rest % p.Hkv, b = rest / p.Hkv;
  const int n0 = p.lens[b], start = p.starts ? p.starts[b] : 0;
  const int n = min(max(n0, 0), p.S);
  const int room = p.kv.max_pages << p.kv.page_shift;
  const bool first = chunk == 0 && h == 0 && threadIdx.x == 0;
  if (n != n0 && first) atomicOr(p.status, fa_host::kStatusIndex);
  if (n == 0) return;
  if (start < 0 || start > room - n) {
    if (first) atomicOr(p.status, fa_host::kStatusIndex);
    return;
  }
  const int part = threadIdx.x % L, row = threadIdx.x / L;
  const int ps = 1 << p.kv.page_shift;
  Word k[kEach], v[kEach];
  uint32_t ks[kEach], vs[kEach];
  int id[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int t = chunk * kReadTokens + i * kRows + row;
    id[i] = t < n ? paged_id(p.kv, b, (start + t) >> p.kv.page_shift, p.status) : -1;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (id[i] < 0) continue;
    const int slot = (start + chunk * kReadTokens + i * kRows + row) & (ps - 1);
    const long long ka = (long long)id[i] * p.kv.k_sp + h * p.kv.k_sh + (long long)slot * p.kv.k_ss;
    const long long va = (long long)id[i] * p.kv.v_sp + h * p.kv.v_sh + (long long)slot * p.kv.v_ss;
    k[i] = *reinterpret_cast<const Word*>(reinterpret_cast<const uint8_t*>(p.kv.k) + (ka + 8 * part) * E);
    v[i] = *reinterpret_cast<const Word*>(reinterpret_cast<const uint8_t*>(p.kv.v) + (va + 8 * part) * E);
    if constexpr (EIGHT) {
      const long long at = (((long long)id[i] * p.Hkv + h) << p.kv.page_shift) + slot;
      ks[i] = p.k_scale[at];
      vs[i] = p.v_scale[at];
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (id[i] < 0) continue;
    const long long t = chunk * kReadTokens + i * kRows + row;
    uint4* ko = reinterpret_cast<uint4*>(p.k + b * p.k_sb + h * p.k_sh + t * p.k_ss + 8 * part);
    uint4* vo = reinterpret_cast<uint4*>(p.v + b * p.v_sb + h * p.v_sh + t * p.v_ss + 8 * part);
    if constexpr (EIGHT) {
      const float kf = scale_of(ks[i]), vf = scale_of(vs[i]);
      *ko = p.e5m2 ? read_codes<BF16, true>(k[i], kf) : read_codes<BF16, false>(k[i], kf);
      *vo = p.e5m2 ? read_codes<BF16, true>(v[i], vf) : read_codes<BF16, false>(v[i], vf);
    } else {
      *ko = k[i];
      *vo = v[i];
    }
  }
}

struct KeepParams {
  PagedKv kv;
  uint8_t* k_scale;
  uint8_t* v_scale;
  const int32_t* kv_lens;
  const int32_t* idx;        // [B, M]
  const int32_t* keep_lens;
  int Hkv, M;
  int parts;                 // blocks per sequence
  int e5m2;
  int* status;
};
constexpr int kKeepThreads = 256;

// A thread owns 16 bytes of one head's rows (of K or of V) and moves them token by token, eight in
// flight: a draft comes from its own place or from further back (idx ascending, so idx[i] >= i), which
// no earlier token of the walk was moved to; within eight the loads come before the stores.  So a
// path is compacted in place without a copy, and the page bounds have one writer per channel.
template <bool BF16, int D, bool EIGHT>
__global__ void __launch_bounds__(kKeepThreads) fa_kv_keep_kernel(const KeepParams p) {
  constexpr int E = EIGHT ? 1 : 2;
  constexpr int L = D * E / 16;
  constexpr int kBatchRows = 8;
  __shared__ int s_id[2][32], s_slot[2][32];      // where 32 tokens come from, and go to
  __shared__ int s_n;
  pdl_launch_dependents();
  pdl_wait_prior();
  const int b = blockIdx.x / p.parts, share = blockIdx.x % p.parts;
  const int n0 = p.keep_lens[b], len0 = p.kv_lens[b];
  const int n = min(max(n0, 0), p.M);
  if (n != n0 && share == 0 && threadIdx.x == 0) atomicOr(p.status, fa_host::kStatusIndex);
  if (n == 0) return;
  const int base = paged_len(p.kv, len0, p.status);
  if (base < 0) return;
  const int room = p.kv.max_pages << p.kv.page_shift, ps = 1 << p.kv.page_shift;
  const int col = share * kKeepThreads + threadIdx.x;
  const int part = col % L, h = (col / L) % p.Hkv, kind = col / (L * p.Hkv);      // kind 0: K, 1: V
  const bool on = kind < 2;
  const unsigned both = __ballot_sync(0xffffffffu, on);
  uint8_t* pool = reinterpret_cast<uint8_t*>(kind ? p.kv.v : p.kv.k);
  const long long sp = (kind ? p.kv.v_sp : p.kv.k_sp) * E, ss = (kind ? p.kv.v_ss : p.kv.k_ss) * E;
  const long long in_page = (kind ? p.kv.v_sh : p.kv.k_sh) * E * h + 16 * part;
  uint8_t* scales = kind ? p.v_scale : p.k_scale;
  const bool bounds = p.kv.k_min && on && kind == 0;
  constexpr int W = EIGHT ? 2 : 1;                // 8 channels each
  const uint32_t kInf = BF16 ? 0x7F807F80u : 0x7C007C00u;
  uint4 mn[W] = {}, mx[W] = {};
  int page = -1;                                  // whose bounds mn and mx are
  auto widen = [&](int j, uint4 lo, uint4 hi) {
    mn[j] = make_uint4(min16x2<BF16>(mn[j].x, lo.x), min16x2<BF16>(mn[j].y, lo.y),
                       min16x2<BF16>(mn[j].z, lo.z), min16x2<BF16>(mn[j].w, lo.w));
    mx[j] = make_uint4(max16x2<BF16>(mx[j].x, hi.x), max16x2<BF16>(mx[j].y, hi.y),
                       max16x2<BF16>(mx[j].z, hi.z), max16x2<BF16>(mx[j].w, hi.w));
  };
  auto bound_at = [&](uint16_t* x, int j) {
    return reinterpret_cast<uint4*>(x + ((long long)page * p.Hkv + h) * D + (EIGHT ? 16 : 8) * part + 8 * j);
  };
  auto flush = [&]() {
    if (page < 0) return;
#pragma unroll
    for (int j = 0; j < W; ++j) *bound_at(p.kv.k_min, j) = mn[j], *bound_at(p.kv.k_max, j) = mx[j];
  };

  for (int c0 = 0; c0 < n; c0 += 32) {
    __syncthreads();
    if (threadIdx.x < 32) {
      const int i = c0 + threadIdx.x;
      bool bad = false;
      int from = -1;
      if (i < n) {
        from = p.idx[(long long)b * p.M + i];
        const int prior = i ? p.idx[(long long)b * p.M + i - 1] : -1;
        // (ascending from >= 0 has from >= i; the sum is below 2^32: both are below 2^31)
        bad = from <= prior || from < i || (unsigned)base + (unsigned)from >= (unsigned)room;
        if (!bad) {
          const int s = base + from, d = base + i;
          s_id[0][threadIdx.x] = paged_id(p.kv, b, s >> p.kv.page_shift, p.status);
          s_id[1][threadIdx.x] = paged_id(p.kv, b, d >> p.kv.page_shift, p.status);
          s_slot[0][threadIdx.x] = s & (ps - 1);
          s_slot[1][threadIdx.x] = d & (ps - 1);
          bad = s_id[0][threadIdx.x] < 0 || s_id[1][threadIdx.x] < 0;
        }
      }
      const unsigned stop = __ballot_sync(0xffffffffu, bad);   // the first bad one ends the path
      if (bad && share == 0) atomicOr(p.status, fa_host::kStatusIndex);
      if (threadIdx.x == 0) s_n = stop ? __ffs(stop) - 1 : min(32, n - c0);
    }
    __syncthreads();
    const int here = s_n;
    if (on) {
      for (int i0 = 0; i0 < here; i0 += kBatchRows) {
        uint4 w[kBatchRows];
        uint32_t f[kBatchRows];
#pragma unroll
        for (int i = 0; i < kBatchRows; ++i) {
          if (i0 + i >= here) break;
          const int id = s_id[0][i0 + i], slot = s_slot[0][i0 + i];
          w[i] = *reinterpret_cast<const uint4*>(pool + id * sp + in_page + slot * ss);
          if constexpr (EIGHT) f[i] = scales[(((long long)id * p.Hkv + h) << p.kv.page_shift) + slot];
        }
        if constexpr (EIGHT) __syncwarp(both);     // (a row's lanes all read its scale byte, one writes it)
#pragma unroll
        for (int i = 0; i < kBatchRows; ++i) {
          if (i0 + i >= here) break;
          const int id = s_id[1][i0 + i], slot = s_slot[1][i0 + i];
          if (id == s_id[0][i0 + i] && slot == s_slot[0][i0 + i]) continue;      // in its place already
          *reinterpret_cast<uint4*>(pool + id * sp + in_page + slot * ss) = w[i];
          if constexpr (EIGHT) {
            if (part == 0) scales[(((long long)id * p.Hkv + h) << p.kv.page_shift) + slot] = (uint8_t)f[i];
          }
          if (bounds) {
            if (id != page) {
              flush();
              page = id;
#pragma unroll
              for (int j = 0; j < W; ++j) mn[j] = *bound_at(p.kv.k_min, j), mx[j] = *bound_at(p.kv.k_max, j);
            }
            if (slot == 0) {
#pragma unroll
              for (int j = 0; j < W; ++j) {
                mn[j] = make_uint4(kInf, kInf, kInf, kInf);
                mx[j] = make_uint4(kInf | 0x80008000u, kInf | 0x80008000u, kInf | 0x80008000u, kInf | 0x80008000u);
              }
            }
            if constexpr (EIGHT) {
              uint4 lo, hi;
              const uint2 c0 = make_uint2(w[i].x, w[i].y), c1 = make_uint2(w[i].z, w[i].w);
              p.e5m2 ? stored_bounds<BF16, true>(c0, f[i], lo, hi) : stored_bounds<BF16, false>(c0, f[i], lo, hi);
              widen(0, lo, hi);
              p.e5m2 ? stored_bounds<BF16, true>(c1, f[i], lo, hi) : stored_bounds<BF16, false>(c1, f[i], lo, hi);
              widen(1, lo, hi);
            } else {
              widen(0, w[i], w[i]);
            }
          }
        }
      }
    }
    if (here < min(32, n - c0)) break;
  }
  if (bounds) flush();
}

}  // namespace fa
