// prefix_common.cuh — pieces shared by the two kernels of the shared prefix:
// a compact bounded wait, predicated tcgen05 issue, 4-D TMA, and the host side
// of tensor maps and dependent launches.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "kernel_common.cuh"
#include "mla_decode.h"

namespace mla {
namespace prefix {

constexpr int kMaxRows = 1 << 30;  // of a prefix, and query tokens (row counts are rounded up in 32 bits)

// 4-D tiled load (x: dim within a 64-dim chunk, y: row, z: chunk, w: head).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// tma_load_4d into this CTA's shared memory, completing on an mbarrier of
// either CTA of the pair (cluster address).
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int w,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar_cluster)
      : "memory");
}

// Predicated forms for a warp of which one lane issues: D (+)= A B^T with A
// in shared or in tensor memory, and the commit.
__device__ __forceinline__ void umma_ss_if(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue) : "memory");
}
__device__ __forceinline__ void umma_ts_if(uint32_t issue, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue) : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint32_t issue, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
      ::"r"(bar), "r"(issue) : "memory");
}

// The same for a pair of SMs, and the commit that arrives in every CTA of `mask`.
__device__ __forceinline__ void umma_pair_ss_if(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue) : "memory");
}
__device__ __forceinline__ void umma_pair_ts_if(uint32_t issue, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue) : "memory");
}
__device__ __forceinline__ void umma_commit_pair_if(uint32_t issue, uint32_t bar, uint16_t mask) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}"
      ::"r"(bar), "h"(mask), "r"(issue) : "memory");
}

// wait_bar with a rolled loop: these kernels wait in many places, and the
// unrolled form made the attention's code 110 KB, which the instruction caches
// do not hold.
template <bool kCluster = false>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Ctl& c) {
  if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!(kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) {
    if (*c.abort) return false;
    if (globaltimer_ns() - t0 > kTimeoutNs) {
      raise_timeout(c);
      return false;
    }
  }
  return true;
}

// The same for a whole warp, with one answer: what depends on it stays
// warp-uniform (an MMA takes its operands from uniform registers; issued from
// code that may have diverged, each one first moves them there).
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait_uniform(uint32_t bar, uint32_t parity, const Ctl& c) {
  return __all_sync(0xffffffffu, wait<kCluster>(bar, parity, c));
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// 4 x 4 transpose of 16-byte pieces over four lanes: piece i of lane q becomes
// piece q of lane i.
__device__ __forceinline__ void quad_transpose(uint4 (&c)[4], int lane) {
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
    const bool up = (lane & b) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & b) continue;
      uint4& lo = c[i];
      uint4& hi = c[i | b];
      uint4 v = up ? lo : hi;
      v.x = __shfl_xor_sync(0xffffffffu, v.x, b);
      v.y = __shfl_xor_sync(0xffffffffu, v.y, b);
      v.z = __shfl_xor_sync(0xffffffffu, v.z, b);
      v.w = __shfl_xor_sync(0xffffffffu, v.w, b);
      if (up)
        lo = v;
      else
        hi = v;
    }
  }
}

// ---------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

inline bool encode(CUtensorMap* m, bool fp16, int rank, const void* base, const cuuint64_t* size, const cuuint64_t* strides,
            const cuuint32_t* box) {
  EncodeTiledFn fn = encode_tiled();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn && fn(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                  const_cast<void*>(base), size, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Keys or values [heads, head_rows, 128] as boxes of {64 dims, `rows` rows, `chunks` 64-dim chunks, 1 head};
// rows from prefix_len on read as zeros and are not written.
inline bool encode_kv(CUtensorMap* m, bool fp16, const void* base, int prefix_len, int64_t head_rows, int heads,
                      uint32_t rows, uint32_t chunks) {
  const cuuint64_t size[4] = {64, static_cast<cuuint64_t>(prefix_len), 2, static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[3] = {256, 128, static_cast<cuuint64_t>(head_rows) * 256};
  const cuuint32_t box[4] = {64u, rows, chunks, 1u};
  return encode(m, fp16, 4, base, size, strides, box);
}

// Launch as a programmatic dependent of the kernel before it on the stream,
// in clusters of `cluster` CTAs.
template <typename... A>
int launch_dependent(void (*kernel)(A...), dim3 grid, dim3 block, int smem, int cluster, mla_stream_t stream,
                     const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

// Whether [rows][width] floats at a, and [rows][other_width] at b, share memory (rows at their strides; the strides of
// one row say nothing).
inline bool share(const float* a, int64_t a_stride, int64_t width, const float* b, int64_t b_stride, int64_t other_width,
                  int64_t rows) {
  if (!a || !b || width <= 0 || other_width <= 0 || rows <= 0) return false;
  const int64_t d = (reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) / static_cast<int64_t>(sizeof(float));
  const int64_t a_all = (rows - 1) * a_stride + width, b_all = (rows - 1) * b_stride + other_width;
  if (d >= a_all || -d >= b_all) return false;
  if (rows == 1 || a_stride != b_stride) return true;
  const int64_t at = (d % a_stride + a_stride) % a_stride;  // columns beside each other in rows of one stride
  return at < width || at + other_width > a_stride;
}

inline bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace prefix
}  // namespace mla
