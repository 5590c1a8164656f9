// What the two attention kernels share: the cache's tensor maps, lengths, conversions and the
// layout of partial results.
#pragma once

#include <algorithm>
#include <mutex>
#include <cudaTypedefs.h>

#include "chain.cuh"
#include "fge_device.cuh"

namespace fge {

namespace {

constexpr int kTile = 128;  // tokens of a tile

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}

// Four e4m3 codes as two fp16 pairs, exactly.
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of tile row r in the TMA's swizzled layout (128-byte swizzle
// for 128-byte rows, 64-byte swizzle for 64-byte rows).
template <int D>
__device__ __forceinline__ int swizzled(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ int clamp_length(int n, int64_t width, const KvCacheArgs& c,
                                            int32_t* status) {
  const int64_t cap = width << c.page_shift;
  if (n >= 0 && n <= cap) return n;
  set_device_error(status, FGE_ERR_BAD_INDEX);
  return n < 0 ? 0 : static_cast<int>(cap);
}

// The same without a report.
__device__ __forceinline__ int quiet_length(int n, int64_t width, int page_shift) {
  const int64_t cap = width << page_shift;
  return n < 0 ? 0 : static_cast<int>(n < cap ? n : cap);
}

// Tiles of that many tokens; unsigned, as lengths go up to 2^31 - 1.
__host__ __device__ constexpr int tile_count(int len) {
  return static_cast<int>((static_cast<uint32_t>(len) + kTile - 1) / kTile);
}

// A partial result of `rows` query rows: their maxima (base 2), sums, and outputs before the
// division, [rows, head_dim].
__host__ __device__ constexpr int partial_floats(int rows, int head_dim) {
  return rows * (head_dim + 2);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The cache's codes as rows of head_dim bytes, boxes of one page (at most a tile) of rows.
bool code_map(CUtensorMap* m, const void* base, const KvCacheArgs& c) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.head_dim),
                              static_cast<cuuint64_t>(c.n_pages) * c.n_kv * c.page_size};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.head_dim)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(c.head_dim),
                             static_cast<cuuint32_t>(std::min(c.page_size, kTile))};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The shared prefix's part of the attention of many rows on tcgen05 (attention_prefix.cu):
// partial results [n_kv * groups][max(splits, last)] of kPrefixTcRows query rows, those of the
// whole batch; splits runs of the token tiles for two groups together, last for an odd last one.
constexpr int kPrefixTcRows = 128;
cudaError_t launch_prefix_tc(const AttentionArgs& a, int groups, int splits, int last,
                             float* partials, cudaStream_t s);

}  // namespace fge
