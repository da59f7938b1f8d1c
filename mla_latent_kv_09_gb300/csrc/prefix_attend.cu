// prefix_attend.cu — attention of a batch's query tokens over a shared,
// expanded prefix, with the C ABI (include/mla_prefix.h).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernel_common.cuh"
#include "mla_prefix.h"

namespace mla {
namespace {

constexpr int kHeadDim = 128;
constexpr int kRope = 64;
constexpr int kKeys = 128;  // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttendParams {
  const uint16_t* q_nope;
  const uint16_t* q_pe;
  long long q_stride;
  const uint16_t* k_nope;
  const uint16_t* v;
  long long head_rows;
  const uint16_t* k_pe;
  int prefix_len;
  const int* visible;
  int num_tokens, num_heads;
  float scale_log2;
  const uint16_t* suffix_out;
  const float* suffix_lse;
  int out_fp32;
  void* out;
  float* lse;
};

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// One CTA: one (token, head).  Thread j scores key j of each tile of 128, then
// sums dim j of the values; one pass with a running maximum and sum.
__global__ void __launch_bounds__(kKeys) mla_prefix_attend_kernel(const __grid_constant__ AttendParams p) {
  __shared__ float q[kHeadDim + kRope], w[kKeys], red[4];
  const int h = blockIdx.x, t = blockIdx.y, j = threadIdx.x, warp = j >> 5;
  grid_dependency_wait();
  const long long row = static_cast<long long>(t) * p.num_heads + h;
  q[j] = bf(p.q_nope[row * p.q_stride + j]);
  if (j < kRope) q[kHeadDim + j] = bf(p.q_pe[row * p.q_stride + j]);
  const int seen = p.visible ? max(0, min(p.visible[t], p.prefix_len)) : p.prefix_len;
  float m = -INFINITY, total = 0.f, used = 0.f, o = 0.f;  // exponents in the base 2
  for (int k0 = 0; k0 < seen; k0 += kKeys) {
    __syncthreads();
    float s = -INFINITY;
    if (k0 + j < seen) {
      const uint16_t* kr = p.k_nope + (h * p.head_rows + k0 + j) * kHeadDim;
      const uint16_t* pr = p.k_pe + static_cast<long long>(k0 + j) * kRope;
      s = 0.f;
      for (int d = 0; d < kHeadDim; ++d) s = fmaf(q[d], bf(kr[d]), s);
      for (int d = 0; d < kRope; ++d) s = fmaf(q[kHeadDim + d], bf(pr[d]), s);
      s *= p.scale_log2;
    }
    float top = s;
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    if ((j & 31) == 0) red[warp] = top;
    __syncthreads();
    const float next = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float e = exp2f(s - next), keep = exp2f(m - next);
    total = total * keep + e;  // this thread's keys only; joined at the end
    const float r = __half2float(__float2half_rn(e));
    used = used * keep + r;
    w[j] = r;
    m = next;
    o *= keep;
    __syncthreads();
    const int n = min(kKeys, seen - k0);
    const uint16_t* vr = p.v + (h * p.head_rows + k0) * kHeadDim + j;
    for (int i = 0; i < n; ++i) o = fmaf(w[i], __half2float(__ushort_as_half(vr[i * kHeadDim])), o);
  }
  for (int pass = 0; pass < 2; ++pass) {
    float x = pass ? used : total;
    for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    __syncthreads();
    if ((j & 31) == 0) red[warp] = x;
    __syncthreads();
    (pass ? used : total) = red[0] + red[1] + red[2] + red[3];
  }
  float lse = seen > 0 ? m * kLn2 + logf(total) : -INFINITY;
  o = seen > 0 ? o / used : 0.f;
  if (p.suffix_out) {
    const float other = p.suffix_lse[row];
    const float top = fmaxf(lse, other);
    if (top == -INFINITY) {
      o = 0.f;
    } else {
      const float a = exp2f((lse - top) * kLog2e), b = exp2f((other - top) * kLog2e);
      const float x = b > 0.f ? bf(p.suffix_out[row * kHeadDim + j]) * b : 0.f;
      o = (o * a + x) / (a + b);
      lse = top + logf(a + b);
    }
  }
  __syncthreads();
  if (p.out_fp32)
    static_cast<float*>(p.out)[row * kHeadDim + j] = o;
  else
    static_cast<uint16_t*>(p.out)[row * kHeadDim + j] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
  if (j == 0) p.lse[row] = lse;
}

constexpr int kMaxDev = 64;
struct AttendDevice {
  std::once_flag once;
  int status = MLA_OK;
  int sms = 0;
};
AttendDevice g_attend_dev[kMaxDev];

int attend_device_ready(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return MLA_ERR_DEVICE;
  AttendDevice& st = g_attend_dev[dev];
  std::call_once(st.once, [&st, dev] {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess || major != 10 ||
        minor != 3 || cudaDeviceGetAttribute(&st.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      st.status = MLA_ERR_DEVICE;
  });
  *sms = st.sms;
  return st.status;
}

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_prefix_attend_workspace_size(int num_tokens, int num_heads, int prefix_len, int* err) {
  int sms = 0;
  int rc = num_tokens < 0 || prefix_len < 0 ? MLA_ERR_INVALID_ARG
           : num_heads < 1 || num_heads > kHeads ? MLA_ERR_UNSUPPORTED : attend_device_ready(&sms);
  if (err) *err = rc;
  if (rc != MLA_OK) return 0;
  return 256;
}

int mla_prefix_attend(const void* q_nope, const void* q_pe, int64_t q_stride, const void* k_nope, const void* v,
                      int64_t head_rows, const void* k_pe, int prefix_len, const int32_t* visible, int num_tokens,
                      int num_heads, float softmax_scale, const void* suffix_out, const float* suffix_lse,
                      unsigned flags, void* workspace, size_t ws_bytes, void* out, float* lse, int* status,
                      mla_stream_t stream) {
  if (!q_nope || !q_pe || !workspace || !out || !lse || !status) return MLA_ERR_INVALID_ARG;
  if (prefix_len != 0 && (!k_nope || !v || !k_pe)) return MLA_ERR_INVALID_ARG;
  if (!al(q_nope, 16) || !al(q_pe, 16) || !al(k_nope, 16) || !al(v, 16) || !al(k_pe, 16) || !al(visible, 4) ||
      !al(suffix_out, 16) || !al(suffix_lse, 4) || !al(workspace, 256) || !al(out, 16) || !al(lse, 4) ||
      !al(status, 4))
    return MLA_ERR_INVALID_ARG;
  if ((suffix_out == nullptr) != (suffix_lse == nullptr)) return MLA_ERR_INVALID_ARG;
  if (num_tokens < 0 || prefix_len < 0 || head_rows < prefix_len) return MLA_ERR_INVALID_ARG;
  if (q_stride < kHeadDim || (q_stride & 7) != 0 || q_stride > (int64_t{1} << 30)) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  if (flags & ~static_cast<unsigned>(MLA_FLAG_OUT_FP32)) return MLA_ERR_INVALID_ARG;
  if (out == suffix_out && (flags & MLA_FLAG_OUT_FP32)) return MLA_ERR_INVALID_ARG;
  if (num_heads < 1 || num_heads > kHeads) return MLA_ERR_UNSUPPORTED;
  if (head_rows > INT32_MAX || static_cast<int64_t>(num_tokens) * num_heads > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  int sms = 0;
  const int rc = attend_device_ready(&sms);
  if (rc != MLA_OK) return rc;
  if (ws_bytes < mla_prefix_attend_workspace_size(num_tokens, num_heads, prefix_len, nullptr))
    return MLA_ERR_WORKSPACE;
  if (num_tokens == 0) return MLA_OK;
  AttendParams p;
  p.q_nope = static_cast<const uint16_t*>(q_nope);
  p.q_pe = static_cast<const uint16_t*>(q_pe);
  p.q_stride = q_stride;
  p.k_nope = static_cast<const uint16_t*>(k_nope);
  p.v = static_cast<const uint16_t*>(v);
  p.head_rows = head_rows;
  p.k_pe = static_cast<const uint16_t*>(k_pe);
  p.prefix_len = prefix_len;
  p.visible = visible;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.scale_log2 = softmax_scale * kLog2e;
  p.suffix_out = static_cast<const uint16_t*>(suffix_out);
  p.suffix_lse = suffix_lse;
  p.out_fp32 = (flags & MLA_FLAG_OUT_FP32) != 0;
  p.out = out;
  p.lse = lse;
  for (int t0 = 0; t0 < num_tokens; t0 += 65535) {  // grid.y's limit
    AttendParams part = p;
    const long long rows = static_cast<long long>(t0) * num_heads;
    part.q_nope += rows * q_stride;
    part.q_pe += rows * q_stride;
    if (visible) part.visible += t0;
    if (suffix_out) part.suffix_out += rows * kHeadDim;
    if (suffix_lse) part.suffix_lse += rows;
    part.out = static_cast<char*>(out) + rows * kHeadDim * (p.out_fp32 ? 4 : 2);
    part.lse += rows;
    const int n = num_tokens - t0 < 65535 ? num_tokens - t0 : 65535;
    mla_prefix_attend_kernel<<<dim3(num_heads, n), kKeys, 0, static_cast<cudaStream_t>(stream)>>>(part);
  }
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
