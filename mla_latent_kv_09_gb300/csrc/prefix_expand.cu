// prefix_expand.cu — per-head keys and values of a shared prefix, from its
// cached latents, with the C ABI (include/mla_prefix.h).
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kernel_common.cuh"
#include "mla_prefix.h"

namespace mla {
namespace {

constexpr int kLatent = 512;
constexpr int kHeadDim = 128;
constexpr int kRope = 64;
constexpr int kFp8Row = MLA_FP8_ROW_BYTES;
constexpr int kRowsPerCta = 16;

struct ExpandParams {
  const uint8_t* cache;
  long long num_pages;
  const int* block_table;
  int prefix_len, num_heads, fp8;
  const uint16_t* w_uk;
  const uint16_t* w_uv;
  uint16_t* k_nope;
  uint16_t* v;
  long long head_rows;
  uint16_t* k_pe;
  int* status;
};

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// One CTA: 16 rows of one head; thread d sums K's and V's dim d of each.
__global__ void __launch_bounds__(kHeadDim) mla_prefix_expand_kernel(const __grid_constant__ ExpandParams p) {
  __shared__ float lat[kRowsPerCta][kLatent];
  const int h = blockIdx.y, r0 = blockIdx.x * kRowsPerCta, d = threadIdx.x;
  const long long row_bytes = p.fp8 ? kFp8Row : 2 * kDqk;
  grid_dependency_wait();
  for (int r = 0; r < kRowsPerCta; ++r) {
    const int pos = r0 + r;
    const long long page = pos < p.prefix_len ? p.block_table[pos / kPage] : -1;
    const bool ok = page >= 0 && page < p.num_pages;
    if (!ok && pos < p.prefix_len && d == 0) atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
    const uint8_t* row = p.cache + (ok ? (page * kPage + pos % kPage) * row_bytes : 0);
    for (int c = d; c < kLatent; c += kHeadDim) {
      float x = 0.f;
      if (ok && !p.fp8) x = bf(reinterpret_cast<const uint16_t*>(row)[c]);
      if (ok && p.fp8) {
        __nv_fp8_e4m3 q;
        q.__x = row[c];
        x = static_cast<float>(q) * exp2f(static_cast<float>(row[kLatent + c / 128]) - 127.f);
      }
      lat[r][c] = x;
    }
    if (h == 0 && d < kRope && pos < p.prefix_len)
      p.k_pe[static_cast<long long>(pos) * kRope + d] =
          ok ? reinterpret_cast<const uint16_t*>(row + (p.fp8 ? 528 : 2 * kLatent))[d] : 0;
  }
  __syncthreads();
  float k[kRowsPerCta] = {}, v[kRowsPerCta] = {};
  const uint16_t* wk = p.w_uk + static_cast<long long>(h) * kLatent * kHeadDim + d;
  const uint16_t* wv = p.w_uv + static_cast<long long>(h) * kLatent * kHeadDim + d;
  for (int c = 0; c < kLatent; ++c) {
    const float a = bf(wk[c * kHeadDim]), b = bf(wv[c * kHeadDim]);
#pragma unroll
    for (int r = 0; r < kRowsPerCta; ++r) {
      k[r] = fmaf(lat[r][c], a, k[r]);
      v[r] = fmaf(lat[r][c], b, v[r]);
    }
  }
  for (int r = 0; r < kRowsPerCta; ++r) {
    if (r0 + r >= p.prefix_len) break;
    const long long at = (h * p.head_rows + r0 + r) * kHeadDim + d;
    p.k_nope[at] = __bfloat16_as_ushort(__float2bfloat16_rn(k[r]));
    p.v[at] = __half_as_ushort(__float2half_rn(v[r]));
    if (!(fabsf(v[r]) < 65520.f)) atomicCAS(p.status, 0, static_cast<int>(kStValueRange));
  }
}

constexpr int kMaxDev = 64;
struct ExpandDevice {
  std::once_flag once;
  int status = MLA_OK;
};
ExpandDevice g_expand_dev[kMaxDev];

int expand_device_ready() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return MLA_ERR_DEVICE;
  ExpandDevice& st = g_expand_dev[dev];
  std::call_once(st.once, [&st, dev] {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess || major != 10 ||
        minor != 3)
      st.status = MLA_ERR_DEVICE;
  });
  return st.status;
}

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_prefix_expand_workspace_size(int prefix_len, unsigned flags) {
  if (prefix_len < 1 || !(flags & MLA_FLAG_KV_FP8)) return 0;
  return static_cast<size_t>(prefix_len) * kLatent * 2;
}

int mla_prefix_expand(const void* kv_cache, int64_t num_pages, const int32_t* block_table, int prefix_len,
                      const void* w_uk, const void* w_uv, int num_heads, unsigned flags, void* k_nope, void* v,
                      int64_t head_rows, void* k_pe, void* workspace, size_t ws_bytes, int* status,
                      mla_stream_t stream) {
  if (!kv_cache || !block_table || !w_uk || !w_uv || !k_nope || !v || !k_pe || !status) return MLA_ERR_INVALID_ARG;
  if (!al(kv_cache, 16) || !al(block_table, 4) || !al(w_uk, 16) || !al(w_uv, 16) || !al(k_nope, 16) || !al(v, 16) ||
      !al(k_pe, 16) || !al(workspace, 16) || !al(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_pages < 1 || prefix_len < 0 || head_rows < prefix_len) return MLA_ERR_INVALID_ARG;
  if (flags & ~static_cast<unsigned>(MLA_FLAG_KV_FP8)) return MLA_ERR_INVALID_ARG;
  if (num_heads < 1 || num_heads > kHeads) return MLA_ERR_UNSUPPORTED;
  if (num_pages > (INT32_MAX / kPage) - 1 || head_rows > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  const size_t need = mla_prefix_expand_workspace_size(prefix_len, flags);
  if (need > 0 && !workspace) return MLA_ERR_INVALID_ARG;
  if (ws_bytes < need) return MLA_ERR_WORKSPACE;
  const int rc = expand_device_ready();
  if (rc != MLA_OK) return rc;
  if (prefix_len == 0) return MLA_OK;
  ExpandParams p;
  p.cache = static_cast<const uint8_t*>(kv_cache);
  p.num_pages = num_pages;
  p.block_table = block_table;
  p.prefix_len = prefix_len;
  p.num_heads = num_heads;
  p.fp8 = (flags & MLA_FLAG_KV_FP8) != 0;
  p.w_uk = static_cast<const uint16_t*>(w_uk);
  p.w_uv = static_cast<const uint16_t*>(w_uv);
  p.k_nope = static_cast<uint16_t*>(k_nope);
  p.v = static_cast<uint16_t*>(v);
  p.head_rows = head_rows;
  p.k_pe = static_cast<uint16_t*>(k_pe);
  p.status = status;
  const dim3 grid((prefix_len + kRowsPerCta - 1) / kRowsPerCta, num_heads);
  mla_prefix_expand_kernel<<<grid, kHeadDim, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
