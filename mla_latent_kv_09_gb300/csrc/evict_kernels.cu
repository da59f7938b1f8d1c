// evict_kernels.cu — the choice of the rows that a cache keeps and their move
// to pages of their own, with their C ABI (include/mla_evict.h).
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "kernel_common.cuh"
#include "mla_evict.h"

namespace mla {
namespace {

// ------------------------------------------------------------------ select
// A cluster of CTAs per request, a slice of its rows each, which stays in
// shared memory where it fits.  Weights map to order-preserving 32-bit keys;
// three histogram passes over the cluster (11, 11, 10 bits) find the key T of
// the last row to keep among those that are not protected, and how many of the
// keys equal to T to keep; an ordered pass (ballots within a warp's run of
// rows, prefix sums over warps and CTAs) then writes the kept rows in order.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSelRows = 49152;  // rows of a slice that shared memory holds; the rest is read again in every pass

struct SelectParams {
  const float* weights;
  long long stride;
  const int* lens;
  int max_len, keep, sinks, recent, cluster;
  int smem_rows;  // of a slice, in dynamic shared memory
  int* kept;
  int* new_lens;
  float* new_weights;
  long long new_stride;
  int new_width;
  int* status;
};

// Larger weight -> larger key; the two zeros are one key, NaN is -inf's.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -__int_as_float(0x7f800000);
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa(smem_u32(p), rank)) : "memory");
  return v;
}

// Inclusive scan over a block of one value per thread (warp sums in s[32]); the caller syncs before s is used again.
__device__ __forceinline__ int block_scan(int v, int* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) s[warp] = v;
  __syncthreads();
  int before = lane < warp ? s[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  return v + before;
}

__global__ void __launch_bounds__(kSelThreads) mla_evict_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ float s_rows[];
  __shared__ int s_hist[2][2048];  // this CTA's counts, by pass parity
  __shared__ int s_sum[kSelWarps], s_found[2], s_count[2], s_warp[2][kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
  const int given = p.lens[b];
  const int len = min(max(given, 0), p.max_len);
  if (tid == 0 && rank == 0) {
    if (given != len) atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
    p.new_lens[b] = min(len, p.keep);
  }
  const float* row = p.weights + b * p.stride;
  int* kept = p.kept + static_cast<long long>(b) * p.keep;
  float* out = p.new_weights ? p.new_weights + b * p.new_stride : nullptr;
  const int all = rank * kSelThreads + tid, step = p.cluster * kSelThreads;
  const int stay = min(len, p.keep);
  for (int i = stay + all; i < p.keep; i += step) kept[i] = -1;
  if (out)
    for (int i = stay + all; i < p.new_width; i += step) out[i] = 0.f;
  if (len <= p.keep) {  // (the whole cluster: the same len)
    for (int i = all; i < len; i += step) {
      kept[i] = i;
      if (out) out[i] = row[i];
    }
    return;
  }

  // slices are multiples of 32 rows, so that a warp's ballots do not straddle them
  const int slice = ((len + p.cluster - 1) / p.cluster + 31) / 32 * 32;
  const int j0 = min(rank * slice, len), n = min(slice, len - j0);
  for (int i = tid; i < min(n, p.smem_rows); i += kSelThreads) s_rows[i] = row[j0 + i];
  auto weight = [&](int i) { return i < p.smem_rows ? s_rows[i] : __ldg(row + j0 + i); };
  const int old_end = len - p.recent;
  auto fixed = [&](int i) { return j0 + i < p.sinks || j0 + i >= old_end; };

  // ---- the key of the last row to keep
  uint32_t prefix = 0, mask = 0;
  int left = p.keep - p.sinks - p.recent;  // rows still to be taken among the keys that match the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    int* hist = s_hist[pass & 1];
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t key = weight_key(weight(i));
      if ((key & mask) == prefix && !fixed(i)) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
    }
    if (p.cluster > 1)
      cluster_sync();
    else
      __syncthreads();
    // bins from the largest down, two a thread
    int c[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int bin = bins - 1 - (2 * tid + e);
      if (bin < 0) continue;
      if (p.cluster == 1)
        c[e] = hist[bin];
      else
        for (int r = 0; r < p.cluster; ++r) c[e] += ld_cluster(&hist[bin], r);
    }
    const int upto = block_scan(c[0] + c[1], s_sum), before = upto - c[0] - c[1];
    if (before < left && left <= upto) {
      const int e = left <= before + c[0] ? 0 : 1;
      s_found[0] = bins - 1 - (2 * tid + e);
      s_found[1] = before + (e ? c[0] : 0);
    }
    __syncthreads();
    if (left > 0) {  // (left = 0: no bin was found, and none is needed)
      prefix |= static_cast<uint32_t>(s_found[0]) << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      left -= s_found[1];
    }
    __syncthreads();
  }
  const bool some = p.keep > p.sinks + p.recent;
  // 2: stays, 1: stays if there is room for it, 0: goes
  auto grade = [&](int i) {
    if (i >= n) return 0;
    if (fixed(i)) return 2;
    const uint32_t key = weight_key(weight(i));
    return !some || key < prefix ? 0 : key > prefix ? 2 : 1;
  };

  // ---- the kept rows in order: a run of 32-row groups per warp
  const int groups = (n + 31) / 32, per = (groups + kSelWarps - 1) / kSelWarps;
  const int g0 = min(warp * per, groups), g1 = min(g0 + per, groups);
  int sure = 0, maybe = 0;
  for (int g = g0; g < g1; ++g) {
    const int a = grade(32 * g + lane);
    sure += __popc(__ballot_sync(0xffffffffu, a == 2));
    maybe += __popc(__ballot_sync(0xffffffffu, a == 1));
  }
  if (lane == 0) {
    s_warp[0][warp] = sure;
    s_warp[1][warp] = maybe;
  }
  __syncthreads();
  int sure_before = lane < warp ? s_warp[0][lane] : 0, maybe_before = lane < warp ? s_warp[1][lane] : 0;
  int sure_all = s_warp[0][lane], maybe_all = s_warp[1][lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sure_before += __shfl_xor_sync(0xffffffffu, sure_before, o);
    maybe_before += __shfl_xor_sync(0xffffffffu, maybe_before, o);
    sure_all += __shfl_xor_sync(0xffffffffu, sure_all, o);
    maybe_all += __shfl_xor_sync(0xffffffffu, maybe_all, o);
  }
  if (p.cluster > 1) {
    if (tid == 0) {
      s_count[0] = sure_all;
      s_count[1] = maybe_all;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      sure_before += ld_cluster(&s_count[0], r);
      maybe_before += ld_cluster(&s_count[1], r);
    }
  }
  const uint32_t lower = (1u << lane) - 1u;
  for (int g = g0; g < g1; ++g) {
    const int i = 32 * g + lane, a = grade(i);
    const uint32_t s = __ballot_sync(0xffffffffu, a == 2), m = __ballot_sync(0xffffffffu, a == 1);
    const int maybe_at = maybe_before + __popc(m & lower);
    const int place = sure_before + __popc(s & lower) + min(maybe_at, left);
    if (a == 2 || (a == 1 && maybe_at < left)) {
      kept[place] = j0 + i;
      if (out) out[place] = weight(i);
    }
    sure_before += __popc(s);
    maybe_before += __popc(m);
  }
  if (p.cluster > 1) cluster_sync();  // no CTA's counts go away while another reads them
}

// ------------------------------------------------------------------ compact
// A CTA moves kMoveRows rows of a request: where they lie and where they go is
// looked up once, then every thread copies 16-byte units, kMoveDepth of them in
// flight.  HBM-bound: a row is read once and written once.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;

struct MoveParams {
  uint4* cache;
  long long num_pages;
  const int* table;
  long long bt_stride;
  int bt_width;
  const int* kept;
  long long kept_stride;
  int kept_width;
  const int* lens;
  const int* out_table;
  long long out_stride;
  int out_width, requests;
  int* status;
};

template <int kUnits>
__global__ void __launch_bounds__(kMoveThreads) mla_cache_compact_kernel(const __grid_constant__ MoveParams p) {
  __shared__ long long s_src[kMoveRows], s_dst[kMoveRows];
  constexpr int kItems = kMoveRows * kUnits;
  constexpr int kDepth = (kItems + kMoveThreads - 1) / kMoveThreads;
  for (int b = blockIdx.y; b < p.requests; b += gridDim.y) {
    const int given = p.lens[b];
    const int len = min(max(given, 0), p.kept_width);
    if (given != len && blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
    for (int i0 = blockIdx.x * kMoveRows; i0 < len; i0 += gridDim.x * kMoveRows) {
      if (threadIdx.x < kMoveRows) {
        const int i = i0 + threadIdx.x;
        long long src = -1, dst = -1;
        if (i < len) {
          const int j = p.kept[b * p.kept_stride + i];
          if (j < 0 || j / kPage >= p.bt_width) {
            atomicCAS(p.status, 0, static_cast<int>(kStBadIndex));
          } else {
            const int from = p.table[b * p.bt_stride + j / kPage];
            const int to = i / kPage < p.out_width ? p.out_table[b * p.out_stride + i / kPage] : -1;
            if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
              atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
            } else {
              src = (static_cast<long long>(from) * kPage + j % kPage) * kUnits;
              dst = (static_cast<long long>(to) * kPage + i % kPage) * kUnits;
            }
          }
        }
        s_src[threadIdx.x] = src;
        s_dst[threadIdx.x] = dst;
      }
      __syncthreads();
      uint4 v[kDepth];
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        const int at = k * kMoveThreads + threadIdx.x, r = at / kUnits;
        if (at < kItems && s_src[r] >= 0) v[k] = p.cache[s_src[r] + at % kUnits];
      }
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        const int at = k * kMoveThreads + threadIdx.x, r = at / kUnits;
        if (at < kItems && s_src[r] >= 0) p.cache[s_dst[r] + at % kUnits] = v[k];
      }
      __syncthreads();
    }
  }
}

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Device check and the selection's shared memory, once per device.
int evict_device_ready() {
  static std::once_flag once[64];
  static int state[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MLA_ERR_DEVICE;
  std::call_once(once[dev], [dev] {
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (major != 10 || minor != 3) {
      state[dev] = MLA_ERR_DEVICE;
      return;
    }
    state[dev] = cudaFuncSetAttribute(mla_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kSelRows * 4) == cudaSuccess
                     ? MLA_OK
                     : MLA_ERR_CUDA;
    cudaGetLastError();
  });
  return state[dev];
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int mla_evict_select(const float* weights, int64_t weights_stride, const int32_t* cache_lens, int num_requests,
                     int max_len, int keep, int sinks, int recent, int32_t* kept, int32_t* new_lens,
                     float* new_weights, int64_t new_weights_stride, int new_width, int* status,
                     mla_stream_t stream) {
  if (!weights || !cache_lens || !kept || !new_lens || !status || !al(weights, 4) || !al(cache_lens, 4) || !al(kept, 4) ||
      !al(new_lens, 4) || !al(status, 4) || !al(new_weights, 4) || weights == new_weights)
    return MLA_ERR_INVALID_ARG;
  if (num_requests < 0 || max_len < 1 || keep < 1 || sinks < 0 || recent < 0 || sinks > keep || recent > keep - sinks)
    return MLA_ERR_INVALID_ARG;
  if (num_requests > 1 && weights_stride < max_len) return MLA_ERR_INVALID_ARG;
  if (new_weights && (new_width < (keep < max_len ? keep : max_len) || (num_requests > 1 && new_weights_stride < new_width)))
    return MLA_ERR_INVALID_ARG;
  // rows are numbered in 32 bits, beyond the end by a grid's step
  if (max_len > (1 << 30) || keep > (1 << 30) || new_width > (1 << 30) || num_requests > INT32_MAX / kMaxCluster)
    return MLA_ERR_UNSUPPORTED;
  const int rc = evict_device_ready();
  if (rc != MLA_OK) return rc;
  if (num_requests == 0) return MLA_OK;
  SelectParams p;
  p.weights = weights;
  p.stride = weights_stride;
  p.lens = cache_lens;
  p.max_len = max_len;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.cluster = 1;
  while (p.cluster < kMaxCluster && static_cast<int64_t>(p.cluster) * 4096 < max_len) p.cluster *= 2;
  const int slice = ((max_len + p.cluster - 1) / p.cluster + 31) / 32 * 32;
  p.smem_rows = slice < kSelRows ? slice : kSelRows;
  p.kept = kept;
  p.new_lens = new_lens;
  p.new_weights = new_weights;
  p.new_stride = new_weights_stride;
  p.new_width = new_weights ? new_width : 0;
  p.status = status;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_requests) * p.cluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.smem_rows) * 4;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, mla_evict_select_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

int mla_cache_compact(void* cache, int64_t num_pages, int row_bytes, const int32_t* block_table, int64_t bt_stride,
                      int bt_width, const int32_t* kept, int64_t kept_stride, int kept_width, const int32_t* lens,
                      int num_requests, const int32_t* out_table, int64_t out_stride, int out_width, int* status,
                      mla_stream_t stream) {
  if (!cache || !block_table || !kept || !lens || !out_table || !status || !al(cache, 16) || !al(block_table, 4) ||
      !al(kept, 4) || !al(lens, 4) || !al(out_table, 4) || !al(status, 4) || block_table == out_table)
    return MLA_ERR_INVALID_ARG;
  if (num_pages < 1 || num_requests < 0 || bt_width < 1 || kept_width < 0 || out_width < 1) return MLA_ERR_INVALID_ARG;
  if (num_requests > 1 && (bt_stride < bt_width || kept_stride < kept_width || out_stride < out_width))
    return MLA_ERR_INVALID_ARG;
  if (row_bytes != 1152 && row_bytes != MLA_FP8_ROW_BYTES && row_bytes != 256) return MLA_ERR_UNSUPPORTED;
  if (kept_width > (1 << 30) || num_pages > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  const int rc = evict_device_ready();
  if (rc != MLA_OK) return rc;
  if (num_requests == 0 || kept_width == 0) return MLA_OK;
  MoveParams p;
  p.cache = static_cast<uint4*>(cache);
  p.num_pages = num_pages;
  p.table = block_table;
  p.bt_stride = bt_stride;
  p.bt_width = bt_width;
  p.kept = kept;
  p.kept_stride = kept_stride;
  p.kept_width = kept_width;
  p.lens = lens;
  p.out_table = out_table;
  p.out_stride = out_stride;
  p.out_width = out_width;
  p.requests = num_requests;
  p.status = status;
  const int x = (kept_width + kMoveRows - 1) / kMoveRows;
  const dim3 grid(x, num_requests < 65535 ? num_requests : 65535);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (row_bytes == 1152)
    mla_cache_compact_kernel<72><<<grid, kMoveThreads, 0, s>>>(p);
  else if (row_bytes == 256)
    mla_cache_compact_kernel<16><<<grid, kMoveThreads, 0, s>>>(p);
  else
    mla_cache_compact_kernel<41><<<grid, kMoveThreads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

}  // extern "C"
