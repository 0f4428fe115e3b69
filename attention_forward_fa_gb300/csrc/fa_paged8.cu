// Kernels of the paged operators over an 8-bit cache and of drafting, and their
// launches (arguments are checked in fa_paged.cu).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "../../include/fa_fwd.h"
#include "fa_paged_launch.h"

namespace fa_host {

static_assert(kStatusRange == fa::kStatusRange, "one word");

cudaError_t launch_append_placed(const fa::AppendParams& p, bool fp16, int D, bool interleaved, long long pieces, cudaStream_t st) {
  return launch_append<fa::kAppendPlaced>(p, fp16, D, interleaved, pieces, st);
}
cudaError_t launch_append8(const fa::AppendParams& p, bool fp16, int D, bool interleaved, long long pieces, cudaStream_t st) {
  return launch_append<fa::kAppend8>(p, fp16, D, interleaved, pieces, st);
}

cudaError_t launch_read(const fa::ReadParams& p, bool fp16, int D, bool eight, unsigned blocks, cudaStream_t st) {
  auto go = [&](auto kern) { return launch_dependent(kern, blocks, fa::kReadThreads, 0, st, p); };
  if (!eight) return D == 128 ? go(fa::fa_kv_read_kernel<true, 128, false>) : go(fa::fa_kv_read_kernel<true, 64, false>);   // (copied)
  if (D == 128) return fp16 ? go(fa::fa_kv_read_kernel<false, 128, true>) : go(fa::fa_kv_read_kernel<true, 128, true>);
  return fp16 ? go(fa::fa_kv_read_kernel<false, 64, true>) : go(fa::fa_kv_read_kernel<true, 64, true>);
}

cudaError_t launch_keep(const fa::KeepParams& p, bool fp16, int D, bool eight, unsigned blocks, cudaStream_t st) {
  auto go = [&](auto kern) { return launch_dependent(kern, blocks, fa::kKeepThreads, 0, st, p); };
  if (D == 128) {
    if (eight) return fp16 ? go(fa::fa_kv_keep_kernel<false, 128, true>) : go(fa::fa_kv_keep_kernel<true, 128, true>);
    return fp16 ? go(fa::fa_kv_keep_kernel<false, 128, false>) : go(fa::fa_kv_keep_kernel<true, 128, false>);
  }
  if (eight) return fp16 ? go(fa::fa_kv_keep_kernel<false, 64, true>) : go(fa::fa_kv_keep_kernel<true, 64, true>);
  return fp16 ? go(fa::fa_kv_keep_kernel<false, 64, false>) : go(fa::fa_kv_keep_kernel<true, 64, false>);
}

namespace {

template <bool BF16, int D, int NT, bool E5M2>
int launch_decode8_rows(fa::Decode8Params& p, long long most_tiles, cudaStream_t st) {
  auto kern = fa::fa_decode8_kernel<BF16, D, NT, E5M2>;
  constexpr int smem = fa::Decode8Smem<BF16, D, NT>::kBytes;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  std::call_once(once[dev & 63], [&] {
    attr_err[dev & 63] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr_err[dev & 63] != cudaSuccess) return cuda_fail(attr_err[dev & 63]);
  const int sms = sm_count();
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice);
  p.c.ctas = (int)std::min<long long>(fa::kDec8Teams<BF16, NT> * sms, most_tiles);
  auto inverse = [](unsigned long long d) { return d == 1 ? 0ull : ~0ull / d + 1; };   // ceil(2^64 / d)
  p.c.ctas_inv = inverse(p.c.ctas);
  p.c.units_inv = inverse(p.c.units);
  const size_t o_bytes = (size_t)2 * p.c.ctas * 8 * NT * D * 4;
  void* scratch = scratch_alloc(o_bytes + (size_t)2 * p.c.ctas * 8 * NT * 8, st);
  if (!scratch) return cuda_fail(cudaGetLastError());
  p.c.part_o = static_cast<float*>(scratch);
  p.c.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(scratch) + o_bytes);
  const unsigned grid = (unsigned)std::min(p.c.ctas, sms);
  cudaError_t e = launch_dependent(kern, grid, fa::kDecThreads * fa::kDec8Teams<BF16, NT>, smem, st, p);
  if (e == cudaSuccess) {   // (as for a 16-bit cache)
    const long long rows = (long long)p.c.B * p.c.Hkv * p.c.rows;
    constexpr int T = fa::kDec8Tile;
    if (rows > 8LL * sms)
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 1, T>, (unsigned)((rows + 7) / 8), 256, 0, st, p.c, 8 * NT);
    else if (p.c.ctas / ((long long)p.c.B * p.c.units) < 32)
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 8, T>, (unsigned)rows, 256, 0, st, p.c, 8 * NT);
    else
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 32, T>, (unsigned)rows, 1024, 0, st, p.c, 8 * NT);
  }
  cudaFreeAsync(scratch, st);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

template <bool BF16, int D, bool E5M2>
int launch_decode8_groups(fa::Decode8Params& p, long long keys, cudaStream_t st) {
  fa::DecodeCore& c = p.c;
  // (passes of up to 32 rows: at 40 and 48 one of all rows spills 118 and 342 bytes)
  const int passes = (c.rows + 31) / 32, nt = ((c.rows + passes - 1) / passes + 7) / 8;   // (more rows: launch_wide)
  c.groups = (c.rows + 8 * nt - 1) / (8 * nt);
  if ((long long)c.Hkv * c.groups > 0x7FFFFFFFLL) return FA_ERR_SHAPE;
  c.units = c.Hkv * c.groups;
  const long long most = ((keys + fa::kDec8Tile - 1) / fa::kDec8Tile + fa::kUnitTiles) * c.B * c.units;
  switch (nt) {
    case 1: return launch_decode8_rows<BF16, D, 1, E5M2>(p, most, st);
    case 2: return launch_decode8_rows<BF16, D, 2, E5M2>(p, most, st);
    case 3: return launch_decode8_rows<BF16, D, 3, E5M2>(p, most, st);
    default: return launch_decode8_rows<BF16, D, 4, E5M2>(p, most, st);
  }
}
template <bool BF16, int D>
int launch_decode8_format(fa::Decode8Params& p, long long keys, cudaStream_t st) {
  return p.e5m2 ? launch_decode8_groups<BF16, D, true>(p, keys, st) : launch_decode8_groups<BF16, D, false>(p, keys, st);
}

}  // namespace

namespace {

template <bool BF16, int D, bool EIGHT, bool SPLIT>
int launch_wide_rows(fa::WideParams& p, long long keys, cudaStream_t st) {
  auto kern = fa::fa_wide_kernel<BF16, D, EIGHT, SPLIT>;
  constexpr int smem = fa::WideSmem<D, EIGHT, SPLIT>::kBytes, rows8 = SPLIT ? 128 : 256;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  std::call_once(once[dev & 63], [&] {
    cudaError_t& e = attr_err[dev & 63];
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    // The warps trade registers with setmaxnreg, which would wait forever for more than the launch gave.
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kern);
    if (e == cudaSuccess && a.numRegs < fa::kWideRegs<EIGHT>) e = cudaErrorInvalidConfiguration;
  });
  if (attr_err[dev & 63] != cudaSuccess) return cuda_fail(attr_err[dev & 63]);
  const int sms = sm_count();
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice);
  fa::DecodeCore& c = p.c;
  c.groups = (int)(((long long)c.rows + rows8 - 1) / rows8);
  if ((long long)c.Hkv * c.groups > 0x7FFFFFFFLL) return FA_ERR_SHAPE;
  c.units = c.Hkv * c.groups;
  const long long most = ((keys + fa::kWideTile - 1) / fa::kWideTile + fa::kWideCharge) * c.B * c.units;
  c.ctas = (int)std::min<long long>(sms, most);
  auto inverse = [](unsigned long long d) { return d == 1 ? 0ull : ~0ull / d + 1; };   // ceil(2^64 / d)
  c.ctas_inv = inverse(c.ctas);
  c.units_inv = inverse(c.units);
  const size_t o_bytes = (size_t)2 * c.ctas * rows8 * D * 4;
  const size_t ml_bytes = (size_t)2 * c.ctas * rows8 * 8;
  void* scratch = scratch_alloc(o_bytes + ml_bytes + (size_t)2 * c.ctas * 128 * D * 4, st);
  if (!scratch) return cuda_fail(cudaGetLastError());
  c.part_o = static_cast<float*>(scratch);
  c.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(scratch) + o_bytes);
  p.gone = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + o_bytes + ml_bytes);
  cudaError_t e = launch_dependent(kern, (unsigned)c.ctas, fa::kWideThreads<EIGHT>, smem, st, p);
  if (e == cudaSuccess) {   // (as fa_paged.cu joins)
    const long long rows = (long long)c.B * c.Hkv * c.rows;
    constexpr int T = fa::kWideTile, C = fa::kWideCharge;
    if (rows > 8LL * sms)
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 1, T, C>, (unsigned)((rows + 7) / 8), 256, 0, st, c, rows8);
    else if (c.ctas / ((long long)c.B * c.units) < 32)
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 8, T, C>, (unsigned)rows, 256, 0, st, c, rows8);
    else
      e = launch_dependent(fa::fa_decode_join_kernel<BF16, D, 32, T, C>, (unsigned)rows, 1024, 0, st, c, rows8);
  }
  cudaFreeAsync(scratch, st);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}
template <bool BF16, int D>
int launch_wide_type(fa::WideParams& p, bool eight, long long keys, cudaStream_t st) {
  const bool split = p.c.rows <= 128;
  if (eight) return split ? launch_wide_rows<BF16, D, true, true>(p, keys, st) : launch_wide_rows<BF16, D, true, false>(p, keys, st);
  return split ? launch_wide_rows<BF16, D, false, true>(p, keys, st) : launch_wide_rows<BF16, D, false, false>(p, keys, st);
}

}  // namespace

int launch_wide(fa::WideParams& p, bool fp16, int D, bool eight, long long keys, cudaStream_t st) {
  if (D == 128) return fp16 ? launch_wide_type<false, 128>(p, eight, keys, st) : launch_wide_type<true, 128>(p, eight, keys, st);
  return fp16 ? launch_wide_type<false, 64>(p, eight, keys, st) : launch_wide_type<true, 64>(p, eight, keys, st);
}

int launch_decode8(fa::Decode8Params& p, bool fp16, int D, long long keys, cudaStream_t st) {
  if (D == 128) return fp16 ? launch_decode8_format<false, 128>(p, keys, st) : launch_decode8_format<true, 128>(p, keys, st);
  return fp16 ? launch_decode8_format<false, 64>(p, keys, st) : launch_decode8_format<true, 64>(p, keys, st);
}

}  // namespace fa_host
