// What the kernels over a paged key-value cache share: the cache as the device
// sees it and the 16-bit element helpers.
#pragma once
#include <cstdint>

#include "fa_host.h"
#include "fa_ptx.cuh"

namespace fa {

struct PagedKv {
  uint16_t* k;
  uint16_t* v;
  long long k_sp, k_sh, k_ss;   // page, head, slot strides (elements)
  long long v_sp, v_sh, v_ss;
  uint16_t* k_min;              // [num_pages, Hkv, D] or null
  uint16_t* k_max;
  const int32_t* table;
  long long table_stride;
  int max_pages, num_pages, page_shift;   // page size = 1 << page_shift
};

// Tokens of a sequence; -1 (reported) where the table cannot hold so many.
__device__ __forceinline__ int paged_len(const PagedKv& c, int len, int* status) {
  if (len < 0 || len > (c.max_pages << c.page_shift)) {
    atomicOr(status, fa_host::kStatusIndex);
    return -1;
  }
  return len;
}

// Page of column p of sequence b's table row; -1 (reported) where the entry is no page.
__device__ __forceinline__ int paged_id(const PagedKv& c, int b, int p, int* status) {
  const int id = c.table[(long long)b * c.table_stride + p];
  if (id < 0 || id >= c.num_pages) {
    atomicOr(status, fa_host::kStatusIndex);
    return -1;
  }
  return id;
}

template <bool BF16>
__device__ __forceinline__ float lo16_f32(uint32_t w) {
  return BF16 ? __uint_as_float(w << 16) : f16_lo_to_f32(w);
}
template <bool BF16>
__device__ __forceinline__ float hi16_f32(uint32_t w) {
  return BF16 ? __uint_as_float(w & 0xFFFF0000u) : f16_hi_to_f32(w);
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}
template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = lo16_f32<BF16>(u[j]);
    x[2 * j + 1] = hi16_f32<BF16>(u[j]);
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack16x2<BF16>(x[0], x[1]), pack16x2<BF16>(x[2], x[3]),
                    pack16x2<BF16>(x[4], x[5]), pack16x2<BF16>(x[6], x[7]));
}
// per-half minimum / maximum of pairs (a number where one of the two is NaN)
template <bool BF16>
__device__ __forceinline__ uint32_t min16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace fa
