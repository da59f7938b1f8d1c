// weights_kernel.cu — the attention weight that every cached row received, with
// its C ABI (include/mla_evict.h).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "kernel_common.cuh"
#include "mla_evict.h"

namespace mla {
namespace {

struct WeightsParams {
  const uint16_t* q;
  const float* lse;
  const uint8_t* kv;
  long long num_pages;
  const int* table;
  long long bt_stride;
  const int* lens;
  int max_len;
  const int* starts;
  int requests, tokens, causal, fp8;
  float scale_log2, decay;
  const float* weights;
  long long w_stride;
  float* out;
  long long out_stride;
  int* status;
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ int start_of(const WeightsParams& p, int b) {
  if (!p.starts) return b * (p.tokens / p.requests);
  return min(max(__ldg(p.starts + b), 0), p.tokens);
}

// A warp a row: its dims in registers, a dot product with every head of every
// token that sees it.
__global__ void __launch_bounds__(256) mla_attention_weights_kernel(const __grid_constant__ WeightsParams p) {
  const int lane = threadIdx.x & 31;
  for (int b = blockIdx.y; b < p.requests; b += gridDim.y) {
    const int given = p.lens[b], len = min(max(given, 0), p.max_len);
    const int first = start_of(p, b), n = start_of(p, b + 1) - first;
    if (blockIdx.x == 0 && threadIdx.x == 0 &&
        (given != len || (p.starts && (p.starts[b] < 0 || p.starts[b + 1] < p.starts[b] || p.starts[b + 1] > p.tokens))))
      atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
    if (n <= 0) continue;
    for (int j = blockIdx.x * 8 + (threadIdx.x >> 5); j < len; j += gridDim.x * 8) {
      const int page = p.table[b * p.bt_stride + j / kPage];
      float k[18] = {};
      if (page >= 0 && page < p.num_pages) {
        const long long at = static_cast<long long>(page) * kPage + j % kPage;
#pragma unroll
        for (int i = 0; i < 18; ++i) {
          const int d = 32 * i + lane;
          if (!p.fp8 || d >= 512) {
            const uint16_t* row = reinterpret_cast<const uint16_t*>(p.kv + at * (p.fp8 ? 656 : 1152)) + (p.fp8 ? -248 : 0);
            k[i] = __uint_as_float(static_cast<uint32_t>(row[d]) << 16);
          } else {
            const uint8_t* row = p.kv + at * 656;
            const uint32_t c = row[d], e = row[512 + d / 128];
            const uint32_t m = c & 0x7fu;
            float v = m == 0x7fu ? __int_as_float(0x7fffffff) : __uint_as_float(m << 20) * 0x1p120f;
            v *= __uint_as_float(e == 255 ? 0x7fffffffu : e ? e << 23 : 0x00400000u);
            k[i] = c & 0x80u ? -v : v;
          }
        }
      } else if (lane == 0) {
        atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
      }
      float sum = 0.f;
      for (int t = p.causal ? max(0, j - (len - n)) : 0; t < n; ++t) {
        for (int h = 0; h < kHeads; ++h) {
          const long long qh = static_cast<long long>(first + t) * kHeads + h;
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < 18; ++i)
            s = fmaf(k[i], __uint_as_float(static_cast<uint32_t>(p.q[qh * kDqk + 32 * i + lane]) << 16), s);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          const float lse = p.lse[qh];
          if (lse != -INFINITY) sum += exp2f(fmaf(s, p.scale_log2, -lse * kLog2e));
        }
      }
      if (lane == 0) {
        const float old = p.decay != 0.f ? p.decay * p.weights[b * p.w_stride + j] : 0.f;
        p.out[b * p.out_stride + j] = old + sum;
      }
    }
  }
}

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int weights_device_ready() {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_DEVICE;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  return major == 10 && minor == 3 ? MLA_OK : MLA_ERR_DEVICE;
}

int check_sizes(int num_tokens, int num_requests, int max_len, unsigned flags) {
  if (num_tokens < 0 || num_requests < 1 || max_len < 1) return MLA_ERR_INVALID_ARG;
  if (flags & ~static_cast<unsigned>(MLA_FLAG_CAUSAL | MLA_FLAG_KV_FP8)) return MLA_ERR_INVALID_ARG;
  if ((static_cast<int64_t>(num_tokens) + 1) * kHeads > INT32_MAX || max_len > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_attention_weights_workspace_size(int num_tokens, int num_requests, int max_len, unsigned flags, int* err) {
  const int rc = check_sizes(num_tokens, num_requests, max_len, flags);
  if (err) *err = rc;
  return rc == MLA_OK ? 256 : 0;
}

int mla_attention_weights(const void* q, const float* lse, const void* kv_cache, int64_t num_pages,
                          const int32_t* block_table, int64_t bt_stride, const int32_t* cache_lens, int max_len,
                          const int32_t* token_starts, int num_requests, int num_tokens, int num_heads,
                          float softmax_scale, float decay, const float* weights, int64_t weights_stride,
                          unsigned flags, void* workspace, size_t ws_bytes, float* out, int64_t out_stride,
                          int* status, mla_stream_t stream) {
  if (!q || !lse || !kv_cache || !block_table || !cache_lens || !out || !status || !workspace) return MLA_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(kv_cache, 16) || !al(lse, 4) || !al(block_table, 4) || !al(cache_lens, 4) || !al(token_starts, 4) ||
      !al(weights, 4) || !al(out, 4) || !al(status, 4) || !al(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (num_heads != kHeads) return MLA_ERR_UNSUPPORTED;
  int rc = check_sizes(num_tokens, num_requests, max_len, flags);
  if (rc != MLA_OK) return rc;
  if (num_pages < 1 || bt_stride < 1 || (!token_starts && num_tokens % num_requests)) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f) || !std::isfinite(decay)) return MLA_ERR_INVALID_ARG;
  if (decay != 0.f && !weights) return MLA_ERR_INVALID_ARG;
  if (num_requests > 1 && (bt_stride < (static_cast<int64_t>(max_len) + kPage - 1) / kPage || out_stride < max_len ||
                           (decay != 0.f && weights_stride < max_len)))
    return MLA_ERR_INVALID_ARG;
  if (out == weights && num_requests > 1 && out_stride != weights_stride) return MLA_ERR_INVALID_ARG;
  if (num_pages > (INT32_MAX / kPage) - 1) return MLA_ERR_UNSUPPORTED;
  if (ws_bytes < mla_attention_weights_workspace_size(num_tokens, num_requests, max_len, flags, nullptr))
    return MLA_ERR_WORKSPACE;
  if ((rc = weights_device_ready()) != MLA_OK) return rc;
  if (num_tokens == 0) return MLA_OK;
  WeightsParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.lse = lse;
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.num_pages = num_pages;
  p.table = block_table;
  p.bt_stride = bt_stride;
  p.lens = cache_lens;
  p.max_len = max_len;
  p.starts = token_starts;
  p.requests = num_requests;
  p.tokens = num_tokens;
  p.causal = (flags & MLA_FLAG_CAUSAL) ? 1 : 0;
  p.fp8 = (flags & MLA_FLAG_KV_FP8) ? 1 : 0;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  p.decay = decay;
  p.weights = weights;
  p.w_stride = weights_stride;
  p.out = out;
  p.out_stride = out_stride;
  p.status = status;
  const int x = (max_len + 7) / 8;
  mla_attention_weights_kernel<<<dim3(x < 4096 ? x : 4096, num_requests < 65535 ? num_requests : 65535), 256, 0,
                                 static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
