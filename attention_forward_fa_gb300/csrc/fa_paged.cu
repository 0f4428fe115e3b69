// Host side of the operators over a paged key-value cache (include/fa_fwd.h):
// argument checks, variant selection and launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include "../../include/fa_fwd.h"
#include "fa_decode.cuh"
#include "fa_host.h"
#include "fa_kv_append.cuh"
#include "fa_select.cuh"

namespace {

using fa_host::cuda_fail;
using fa_host::launch_dependent;

constexpr long long kMostTokens = (1LL << 31) - 65536;   // of one sequence: positions are 32-bit
constexpr long long kMostRows = (1LL << 31) - 65536;     // of a call (B * heads * tokens), counted in 32 bits
constexpr int kMostSel = 1 << 20;                        // listed pages of one KV head

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Checks of what the three entry points share; nothing is launched.
int validate_cache(const fa_paged_kv_t* kv, int B, int Hq, int Hkv, int S, int D, int mask_mode) {
  if (!kv || !kv->page_table) return FA_ERR_NULL;
  if (mask_mode & ~FA_DTYPE_FP16) return FA_ERR_SHAPE;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || S <= 0 || D <= 0 || Hq % Hkv) return FA_ERR_SHAPE;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  const int ps = kv->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1))) return FA_ERR_SHAPE;
  if (kv->num_pages <= 0 || kv->max_pages <= 0 || kv->table_stride < 0) return FA_ERR_SHAPE;
  if ((long long)kv->max_pages * ps > kMostTokens) return FA_ERR_SHAPE;
  if ((kv->k_min == nullptr) != (kv->k_max == nullptr)) return FA_ERR_NULL;
  if (!aligned(kv->page_table, 4) || !aligned(kv->k_min, 16) || !aligned(kv->k_max, 16))
    return FA_ERR_ALIGN;
  return FA_OK;
}

// A stride that steps over `n` things: refused where negative, 0 (things would share memory) or not
// a multiple of 8; of no meaning, and any, where there is one thing only.
int validate_stride(int64_t s, int64_t n, bool may_share) {
  if (n <= 1) return FA_OK;
  if (s < 0 || s >= (1LL << 38) || (s == 0 && !may_share)) return FA_ERR_SHAPE;
  return s % 8 ? FA_ERR_ALIGN : FA_OK;
}

// The pools: bases and strides.
int validate_pools(const fa_paged_kv_t* kv, int Hkv) {
  if (!kv->k || !kv->v) return FA_ERR_NULL;
  int rc = FA_OK;
  for (const auto& [s, n] : {std::pair<int64_t, int64_t>{kv->k_stride_page, kv->num_pages}, {kv->v_stride_page, kv->num_pages},
                             {kv->k_stride_head, Hkv}, {kv->v_stride_head, Hkv},
                             {kv->k_stride_slot, kv->page_size}, {kv->v_stride_slot, kv->page_size}})
    if (rc == FA_OK) rc = validate_stride(s, n, false);
  if (rc != FA_OK) return rc;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return FA_ERR_ALIGN;
  return FA_OK;
}

fa::PagedKv device_cache(const fa_paged_kv_t* kv) {
  fa::PagedKv c;
  c.k = static_cast<uint16_t*>(kv->k);
  c.v = static_cast<uint16_t*>(kv->v);
  c.k_sp = kv->k_stride_page;
  c.k_sh = kv->k_stride_head;
  c.k_ss = kv->k_stride_slot;
  c.v_sp = kv->v_stride_page;
  c.v_sh = kv->v_stride_head;
  c.v_ss = kv->v_stride_slot;
  c.k_min = static_cast<uint16_t*>(kv->k_min);
  c.k_max = static_cast<uint16_t*>(kv->k_max);
  c.table = kv->page_table;
  c.table_stride = kv->table_stride;
  c.max_pages = kv->max_pages;
  c.num_pages = kv->num_pages;
  c.page_shift = 0;
  while ((1 << c.page_shift) < kv->page_size) ++c.page_shift;
  return c;
}

template <bool BF16, int D, bool INTERLEAVED>
cudaError_t launch_append(const fa::AppendParams& p, long long pieces, cudaStream_t st) {
  const int sms = fa_host::sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long long items = 2LL * p.k_items + p.q_items;
  const long long loop = std::max(1LL, (long long)fa::kAppendLoopBlocks * sms / items) * items;   // (an item per block)
  return pieces > (long long)fa::kAppendBlocks * sms
             ? launch_dependent(fa::fa_kv_append_kernel<BF16, D, INTERLEAVED, true>, (unsigned)loop,
                                fa::kAppendThreads, 0, st, p, (int)pieces)
             : launch_dependent(fa::fa_kv_append_kernel<BF16, D, INTERLEAVED, false>, (unsigned)pieces,
                                fa::kAppendThreads, 0, st, p, (int)pieces);
}
template <bool BF16, int D>
cudaError_t launch_append(const fa::AppendParams& p, bool interleaved, long long pieces, cudaStream_t st) {
  return interleaved ? launch_append<BF16, D, true>(p, pieces, st) : launch_append<BF16, D, false>(p, pieces, st);
}

// 5-D view (64 channels, slots, D / 64, heads, pages) of a pool, in boxes of
// one page's and head's `box` slots with all channels, 128-byte swizzle: in
// shared memory [D / 64][box][64].
bool encode_pool(CUtensorMap* tm, const void* base, bool fp16, int D, int Hkv, const fa_paged_kv_t* kv,
                 int64_t s_page, int64_t s_head, int64_t s_slot, int box) {
  auto enc = fa_host::tensor_map_encoder();
  if (!enc) return false;
  // a stride over a single head or page is never stepped; for the map it has to be valid
  if (Hkv == 1) s_head = 64;
  if (kv->num_pages == 1) s_page = 64;
  cuuint64_t dims[5] = {64, (cuuint64_t)kv->page_size, (cuuint64_t)(D / 64), (cuuint64_t)Hkv,
                        (cuuint64_t)kv->num_pages};
  cuuint64_t strides[4] = {(cuuint64_t)s_slot * 2, 128, (cuuint64_t)s_head * 2, (cuuint64_t)s_page * 2};
  cuuint32_t boxes[5] = {64, (cuuint32_t)box, (cuuint32_t)(D / 64), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(tm, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
             const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int D, int NT>
int launch_decode(fa::DecodeParams& p, long long most_tiles, cudaStream_t st) {
  auto kern = fa::fa_decode_kernel<BF16, D, NT>;
  constexpr int smem = fa::DecodeSmem<D, NT>::kBytes;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  std::call_once(once[dev & 63], [&] {
    attr_err[dev & 63] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr_err[dev & 63] != cudaSuccess) return cuda_fail(attr_err[dev & 63]);
  const int sms = fa_host::sm_count();
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice);
  p.c.ctas = (int)std::min<long long>(fa::kDecCtasPerSm * sms, most_tiles);
  auto inverse = [](unsigned long long d) { return d == 1 ? 0ull : ~0ull / d + 1; };   // ceil(2^64 / d)
  p.c.ctas_inv = inverse(p.c.ctas);
  p.c.units_inv = inverse(p.c.units);
  const size_t o_bytes = (size_t)2 * p.c.ctas * 8 * NT * D * 4;
  void* scratch = fa_host::scratch_alloc(o_bytes + (size_t)2 * p.c.ctas * 8 * NT * 8, st);
  if (!scratch) return cuda_fail(cudaGetLastError());
  p.c.part_o = static_cast<float*>(scratch);
  p.c.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(scratch) + o_bytes);
  cudaError_t e = launch_dependent(kern, (unsigned)p.c.ctas, fa::kDecThreads, smem, st, p);
  if (e == cudaSuccess) {
    const long long rows = (long long)p.c.B * p.c.Hkv * p.c.rows;
    if (rows > 8LL * sms)   // more than one wave of blocks of a row each
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 1>, (unsigned)((rows + 7) / 8), 256, 0, st, p.c, 8 * NT);
    else if (p.c.ctas / ((long long)p.c.B * p.c.units) < 32)   // pieces of a unit, nearly
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 8>, (unsigned)rows, 256, 0, st, p.c, 8 * NT);
    else
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 32>, (unsigned)rows, 1024, 0, st, p.c, 8 * NT);
  }
  cudaFreeAsync(scratch, st);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

template <bool BF16, int D>
int launch_decode_rows(fa::DecodeParams& p, long long tiles_per_unit, cudaStream_t st) {
  // As few passes over the keys as 48 rows each allow, and as few columns of 8 as then hold a pass's
  // rows.  Up to 32 rows the time is that of the keys, past that the matrix instructions', about 1.4
  // us a row whatever the split (16 sequences of 4096 tokens, 8 KV heads of 128, bf16: 46 us at 4
  // rows, 59 at 32, 68 at 40, 78 at 48, 105 at 64, 143 at 96; with 128 channels the passes of 40 and 48
  // rows spill 4 and 12 bytes, one of 64 rows spilled far more and took 127 us).
  fa::DecodeCore& c = p.c;
  const int passes = (c.rows + 47) / 48;
  const int nt = ((c.rows + passes - 1) / passes + 7) / 8;
  c.groups = (c.rows + 8 * nt - 1) / (8 * nt);
  if ((long long)c.Hkv * c.groups > 0x7FFFFFFFLL) return FA_ERR_SHAPE;
  c.units = c.Hkv * c.groups;
  const long long most = (tiles_per_unit + fa::kUnitTiles) * c.B * c.units;
  switch (nt) {
    case 1: return launch_decode<BF16, D, 1>(p, most, st);
    case 2: return launch_decode<BF16, D, 2>(p, most, st);
    case 3: return launch_decode<BF16, D, 3>(p, most, st);
    case 4: return launch_decode<BF16, D, 4>(p, most, st);
    case 5: return launch_decode<BF16, D, 5>(p, most, st);
    default: return launch_decode<BF16, D, 6>(p, most, st);
  }
}

template <bool BF16, int D>
int launch_select(fa::SelectParams& p, long long units, cudaStream_t st) {
  const int sms = fa_host::sm_count();
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice);
  const size_t pages = (size_t)units * p.kv.max_pages;
  uint8_t* scratch = static_cast<uint8_t*>(fa_host::scratch_alloc(pages * 24, st));
  if (!scratch) return cuda_fail(cudaGetLastError());
  p.score = reinterpret_cast<float2*>(scratch);
  p.exact = reinterpret_cast<unsigned long long*>(scratch + pages * 8);
  p.near = reinterpret_cast<int32_t*>(scratch + pages * 16);
  p.mark = reinterpret_cast<uint32_t*>(scratch + pages * 20);
  const long long runs = units * p.chunks, most = (long long)fa::kScoreBlocks * sms;
  cudaError_t e = runs > most ? launch_dependent(fa::fa_page_score_kernel<BF16, D, true>, (unsigned)most, 32, 0, st, p)
                              : launch_dependent(fa::fa_page_score_kernel<BF16, D, false>, (unsigned)runs, 32, 0, st, p);
  if (e == cudaSuccess)
    e = launch_dependent(fa::fa_select_kernel<BF16, D>, (unsigned)units, fa::kSelectThreads, 0, st, p);
  cudaFreeAsync(scratch, st);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

int fa_kv_append(const fa_paged_kv_t* kv, const fa_kv_new_t* x, int B, int Hq, int Hkv, int Snew,
                 int D, int mask_mode, const int32_t* kv_lens, const int32_t* new_lens,
                 void* stream) {
  if (!x) return FA_ERR_NULL;
  int rc = validate_cache(kv, B, Hq, Hkv, Snew, D, mask_mode);
  if (rc == FA_OK) rc = validate_pools(kv, Hkv);
  if (rc != FA_OK) return rc;
  if ((long long)B * (x->q ? Hq : Hkv) > kMostRows / Snew) return FA_ERR_SHAPE;
  if (!x->k || !x->v || !kv_lens || (x->q == nullptr) != (x->q_out == nullptr)) return FA_ERR_NULL;
  if (x->rot_dim < 0 || x->rot_dim > D || x->rot_dim % 16 || x->interleaved < 0 || x->interleaved > 1)
    return FA_ERR_SHAPE;
  if (x->rot_dim && (!x->cos || !x->sin)) return FA_ERR_NULL;
  if (x->rot_dim && x->max_pos <= 0) return FA_ERR_SHAPE;
  rc = FA_OK;
  auto strides = [&](int64_t sb, int64_t sh, int64_t ss, int heads, bool may_share) {
    for (const auto& [s, n] : {std::pair<int64_t, int64_t>{sb, B}, {sh, heads}, {ss, Snew}})
      if (rc == FA_OK) rc = validate_stride(s, n, may_share);
  };
  strides(x->k_stride_b, x->k_stride_h, x->k_stride_s, Hkv, true);
  strides(x->v_stride_b, x->v_stride_h, x->v_stride_s, Hkv, true);
  if (x->q) {
    strides(x->q_stride_b, x->q_stride_h, x->q_stride_s, Hq, true);
    strides(x->qo_stride_b, x->qo_stride_h, x->qo_stride_s, Hq, false);
  }
  if (rc != FA_OK) return rc;
  if (x->q && x->q == x->q_out &&   // in place only row onto row
      ((B > 1 && x->q_stride_b != x->qo_stride_b) || (Hq > 1 && x->q_stride_h != x->qo_stride_h) ||
       (Snew > 1 && x->q_stride_s != x->qo_stride_s)))
    return FA_ERR_SHAPE;
  if (!aligned(x->k, 16) || !aligned(x->v, 16) || !aligned(x->q, 16) || !aligned(x->q_out, 16) ||
      (x->rot_dim && (!aligned(x->cos, 16) || !aligned(x->sin, 16))) || !aligned(kv_lens, 4) ||
      !aligned(new_lens, 4))
    return FA_ERR_ALIGN;

  fa::AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.kv = device_cache(kv);
  p.k = static_cast<const uint16_t*>(x->k);
  p.v = static_cast<const uint16_t*>(x->v);
  p.q = static_cast<const uint16_t*>(x->q);
  p.qo = static_cast<uint16_t*>(x->q_out);
  p.k_sb = x->k_stride_b, p.k_sh = x->k_stride_h, p.k_ss = x->k_stride_s;
  p.v_sb = x->v_stride_b, p.v_sh = x->v_stride_h, p.v_ss = x->v_stride_s;
  p.q_sb = x->q_stride_b, p.q_sh = x->q_stride_h, p.q_ss = x->q_stride_s;
  p.o_sb = x->qo_stride_b, p.o_sh = x->qo_stride_h, p.o_ss = x->qo_stride_s;
  p.cos = x->cos;
  p.sin = x->sin;
  p.rot_dim = x->rot_dim;
  p.max_pos = x->max_pos;
  p.kv_lens = kv_lens;
  p.new_lens = new_lens;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Snew = Snew;
  const int ps = kv->page_size;
  p.chunks = (int)(((long long)Snew + ps - 2) / ps) + 1;
  const int rows = fa::kAppendThreads / (D / 16);
  while ((1 << p.tp_shift) < rows && (1 << p.tp_shift) < std::min(Snew, ps)) ++p.tp_shift;
  const int hp = rows >> p.tp_shift;
  p.q_heads = 2 * fa::kBatch * hp;
  p.k_items = (Hkv + hp - 1) / hp;
  p.q_items = x->q ? (Hq + p.q_heads - 1) / p.q_heads : 0;
  const long long per_b = (long long)p.chunks * (2 * p.k_items + p.q_items);
  if (per_b > kMostRows / B) return FA_ERR_SHAPE;
  const long long pieces = per_b * B;
  p.status = fa_host::status_ptr();
  if (!p.status) return cuda_fail(cudaGetLastError());
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool fp16 = (mask_mode & FA_DTYPE_FP16) != 0;
  const bool il = x->interleaved != 0;
  const cudaError_t e =
      D == 128 ? (fp16 ? launch_append<false, 128>(p, il, pieces, st) : launch_append<true, 128>(p, il, pieces, st))
               : (fp16 ? launch_append<false, 64>(p, il, pieces, st) : launch_append<true, 64>(p, il, pieces, st));
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

int fa_decode(const void* q, const fa_paged_kv_t* kv, void* o, float* lse, int B, int Hq, int Hkv,
              int Sq, int D, float scale, int mask_mode, const int32_t* kv_lens, int pre_tokens,
              const int32_t* page_idx, int max_sel, void* stream) {
  int rc = validate_cache(kv, B, Hq, Hkv, Sq, D, mask_mode);
  if (rc == FA_OK) rc = validate_pools(kv, Hkv);
  if (rc != FA_OK) return rc;
  if (!q || !o || !lse || !kv_lens) return FA_ERR_NULL;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!std::isfinite(scale) || !std::isfinite(scale_log2) || pre_tokens < -1) return FA_ERR_SHAPE;
  if (page_idx && (max_sel <= 0 || max_sel > kMostSel)) return FA_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(kv_lens, 4) || !aligned(page_idx, 4))
    return FA_ERR_ALIGN;
  if ((long long)B * Hq > kMostRows / Sq) return FA_ERR_SHAPE;
  fa::DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  const bool fp16 = (mask_mode & FA_DTYPE_FP16) != 0;
  const int box = std::min(kv->page_size, fa::kDecTile);
  if (!encode_pool(&p.tm_k, kv->k, fp16, D, Hkv, kv, kv->k_stride_page, kv->k_stride_head, kv->k_stride_slot, box) ||
      !encode_pool(&p.tm_v, kv->v, fp16, D, Hkv, kv, kv->v_stride_page, kv->v_stride_head, kv->v_stride_slot, box))
    return cuda_fail(cudaErrorInvalidValue);
  fa::DecodeCore& c = p.c;
  c.kv_lens = kv_lens;
  c.table = kv->page_table;
  c.table_stride = kv->table_stride;
  c.sel = page_idx;
  c.max_len = kv->max_pages * kv->page_size;
  c.num_pages = kv->num_pages;
  c.page_shift = device_cache(kv).page_shift;
  c.max_sel = max_sel;
  c.B = B;
  c.Hkv = Hkv;
  c.rows = Hq / Hkv * Sq;
  c.Sq = Sq;
  c.pre_tokens = pre_tokens;
  c.reach = pre_tokens < 0 ? -1 : (int)std::min<long long>((long long)Sq + pre_tokens, 0x7FFFFFFF);
  c.scale_log2 = scale_log2;
  c.q = static_cast<const uint16_t*>(q);
  c.o = static_cast<uint16_t*>(o);
  c.lse = lse;
  c.timeout_ns = fa_host::wait_timeout_ns();
  c.status = fa_host::status_ptr();
  if (!c.status) return cuda_fail(cudaGetLastError());
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // the most tiles that a unit can have: the lengths are known on the device only
  const long long keys = (long long)(page_idx ? std::min(max_sel, kv->max_pages) : kv->max_pages) * kv->page_size;
  const long long tiles = (keys + fa::kDecTile - 1) / fa::kDecTile;
  if (D == 128)
    return fp16 ? launch_decode_rows<false, 128>(p, tiles, st) : launch_decode_rows<true, 128>(p, tiles, st);
  return fp16 ? launch_decode_rows<false, 64>(p, tiles, st) : launch_decode_rows<true, 64>(p, tiles, st);
}

int fa_select_pages(const void* q, const fa_paged_kv_t* kv, int32_t* page_idx, int B, int Hq,
                    int Hkv, int Sq, int D, int mask_mode, const int32_t* kv_lens, int max_sel,
                    int first, int last, void* stream) {
  const int rc = validate_cache(kv, B, Hq, Hkv, Sq, D, mask_mode);
  if (rc != FA_OK) return rc;
  if (!q || !page_idx || !kv_lens || !kv->k_min) return FA_ERR_NULL;
  if (max_sel <= 0 || max_sel > kMostSel || first < 0 || last < 0 ||
      (long long)first + last > max_sel)
    return FA_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(page_idx, 4) || !aligned(kv_lens, 4)) return FA_ERR_ALIGN;
  if ((long long)B * Hq > kMostRows / Sq) return FA_ERR_SHAPE;
  const long long units = (long long)B * Hkv;
  fa::SelectParams p;
  std::memset(&p, 0, sizeof(p));
  p.kv = device_cache(kv);
  p.q = static_cast<const uint16_t*>(q);
  p.out = page_idx;
  p.kv_lens = kv_lens;
  p.B = B;
  p.Hkv = Hkv;
  p.rows = Hq / Hkv * Sq;
  p.max_sel = max_sel;
  p.first = first;
  p.last = last;
  p.chunks = (kv->max_pages + fa::kScorePages - 1) / fa::kScorePages;
  if (units * p.chunks > 0x7FFFFFFFLL) return FA_ERR_SHAPE;
  p.status = fa_host::status_ptr();
  if (!p.status) return cuda_fail(cudaGetLastError());
  const bool fp16 = (mask_mode & FA_DTYPE_FP16) != 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return D == 128 ? (fp16 ? launch_select<false, 128>(p, units, st) : launch_select<true, 128>(p, units, st))
                  : (fp16 ? launch_select<false, 64>(p, units, st) : launch_select<true, 64>(p, units, st));
}

}  // extern "C"
