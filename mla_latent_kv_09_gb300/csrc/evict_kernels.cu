// evict_kernels.cu — the choice of the rows that a cache keeps and their move
// to pages of their own, with their C ABI (include/mla_evict.h).
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "mla_evict.h"
#include "prefix_common.cuh"

namespace mla {
namespace {

using prefix::al;
using prefix::launch_dependent;
using prefix::share;

// ------------------------------------------------------------------ select
// A cluster of CTAs per request, a slice of its rows each, which stays in shared
// memory where it fits.  Weights map to order-preserving 32-bit keys; histogram
// passes over the cluster (11, 11, 10 bits) find the key of the last row to keep
// among those that are not protected, and how many of the keys equal to it to
// keep.  They end as soon as a bin is taken whole, which saves the third one
// wherever few keys share 22 bits.  An ordered pass (ballots within a group of 32
// rows, prefix sums over warps and CTAs) then writes the kept rows in order.
// Bound by latency: a load, two or three passes of three meetings each, the
// ordered pass.  Loops are rolled: with the weights in registers and everything
// unrolled, fetching the instructions took longer than running them (one request
// of 8192 rows 15 us on one CTA).  A dependent launch: calls one after the other,
// 64 x 8192 rows, 10.4 us each instead of 13.6.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
static_assert(kSelWarps == 32, "the ordered pass adds the warps' counts a lane each");
constexpr int kMaxCluster = 16;  // (more than 8 as a permission asks)
constexpr int kSelRows = 4096;   // of a CTA, before the request gets further ones
constexpr int kRoomRows = 49152;  // of a slice that shared memory holds; others are read again in every pass

struct SelectParams {
  const float* weights;
  long long stride;
  const int* lens;
  int max_len, keep, sinks, recent, cluster;
  int room;  // rows of a slice in dynamic shared memory (a multiple of 32)
  int* kept;
  int* new_lens;
  float* new_weights;
  long long new_stride;
  int new_width;
  int* status;
};

// Larger weight -> larger key, none of them 0 or kProtected; the two zeros are one key, NaN is -inf's.
constexpr uint32_t kProtected = 0xffffffffu, kZero = 0x80000000u, kLowest = 0x007fffffu;
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

__device__ __forceinline__ int warp_scan(int v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

__global__ void __launch_bounds__(kSelThreads) mla_evict_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ uint32_t s_keys[];
  __shared__ int s_hist[3][2048];  // this CTA's counts, per pass
  __shared__ int s_coarse[3][64];  // ... of 32 bins together
  __shared__ int s_found[3], s_count[2], s_warp[2][kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
  const int given = p.lens[b];
  const int len = min(max(given, 0), p.max_len);
  if (p.new_lens == p.lens) {  // written below: the whole cluster has read it
    if (p.cluster > 1)
      cluster_sync();
    else
      __syncthreads();
  }
  const float* row = p.weights + b * p.stride;
  int* kept = p.kept + static_cast<long long>(b) * p.keep;
  float* out = p.new_weights ? p.new_weights + b * p.new_stride : nullptr;

  if (tid == 0 && rank == 0) {
    if (given != len) atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
    p.new_lens[b] = min(len, p.keep);
  }
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
  // this CTA's slice, in groups of 32 rows; a run of them per warp
  const int slice = ((len + p.cluster - 1) / p.cluster + 31) / 32, j0 = min(rank * slice * 32, len);
  const int n = min(slice * 32, len - j0), per = (slice + kSelWarps - 1) / kSelWarps;
  // of the slice, rows [free0, free1) are not protected
  const int free0 = max(p.sinks - j0, 0), free1 = min(len - p.recent - j0, n);
  auto key_of = [&](int i, float x) { return i < free0 || i >= free1 ? kProtected : weight_key(x); };
#pragma unroll 4
  for (int i = tid; i < min(n, p.room); i += kSelThreads) s_keys[i] = key_of(i, __ldg(row + j0 + i));
  for (int i = tid; i < 3 * 2048; i += kSelThreads) s_hist[0][i] = 0;
  __syncthreads();
  const int i0 = min(32 * warp * per, n), i1 = min(32 * (warp + 1) * per, n);  // this warp's rows of the slice

  // f(row of the slice, its key) for every lane's row of every group of the warp (0 for rows from i1 on)
  auto each = [&](auto f) {
#pragma unroll 2
    for (int i = i0 + lane; i - lane < min(i1, p.room); i += 32) f(i, i < i1 ? s_keys[i] : 0u);
#pragma unroll 1
    for (int i = max(i0, p.room) + lane; i - lane < i1; i += 32) f(i, i < i1 ? key_of(i, __ldg(row + j0 + i)) : 0u);
  };

  // ---- the key of the last row to keep
  uint32_t prefix = 0, mask = 0;
  int left = p.keep - p.sinks - p.recent;  // rows still to be taken among the keys that match the prefix
  const bool some = left > 0;
#pragma unroll 1
  for (int pass = 0; some && pass < 3; ++pass) {
    int* hist = s_hist[pass];
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
    each([&](int, uint32_t key) {
      if (key - 1u < kProtected - 1u && ((key ^ prefix) & mask) == 0) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
    });
    __syncthreads();
    for (int i = warp; i < bins / 32; i += kSelWarps) {
      const int sum = __reduce_add_sync(0xffffffffu, hist[32 * i + lane]);
      if (lane == 0) s_coarse[pass][i] = sum;
    }
    if (p.cluster > 1)
      cluster_sync();
    else
      __syncthreads();
    // One warp looks for the bin, from the largest down: among 64 sums of 32 bins
    // (two a lane), then among those 32.  Every bin of every CTA read by every
    // CTA cost 2,500 cycles a pass with eight of them.
    if (warp == 0) {
      int c[2] = {0, 0};
      const int top = bins / 32 - 1 - 2 * lane;
      if (top > 0)
        for (int r = 0; r < p.cluster; ++r) {
          c[0] += ld_cluster(&s_coarse[pass][top], r);
          c[1] += ld_cluster(&s_coarse[pass][top - 1], r);
        }
      int upto = warp_scan(c[0] + c[1]), before = upto - c[0] - c[1];
      const int e = left <= before + c[0] ? 0 : 1;
      const uint32_t here = __ballot_sync(0xffffffffu, before < left && left <= upto);
      const int from = __ffs(here) - 1;  // (one lane: `left` is between 1 and the number of keys)
      const int block = __shfl_sync(0xffffffffu, top - e, from);
      const int above = __shfl_sync(0xffffffffu, before + (e ? c[0] : 0), from);
      const int bin = 32 * block + 31 - lane;
      int mine = 0;
      for (int r = 0; r < p.cluster; ++r) mine += ld_cluster(&hist[bin], r);
      upto = above + warp_scan(mine);
      if (upto - mine < left && left <= upto) {
        s_found[0] = bin;
        s_found[1] = upto - mine;
        s_found[2] = mine;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_found[0]) << shift;
    mask |= static_cast<uint32_t>(bins - 1) << shift;
    left -= s_found[1];
    if (left == s_found[2]) break;  // (the next pass writes s_found behind two more meetings)
  }
  if (!some) {  // the protected ones only
    prefix = kProtected - 1u;
    mask = kProtected;
  }

  // ---- the kept rows in order
  int sure = 0, maybe = 0;
  each([&](int, uint32_t key) {
    sure += __popc(__ballot_sync(0xffffffffu, (key & mask) > prefix));
    maybe += __popc(__ballot_sync(0xffffffffu, (key & mask) == prefix));
  });
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
  each([&](int i, uint32_t key) {
    const bool stays = (key & mask) > prefix, may = (key & mask) == prefix;
    const uint32_t s = __ballot_sync(0xffffffffu, stays), m = __ballot_sync(0xffffffffu, may);
    const int maybe_at = maybe_before + __popc(m & lower);
    if (stays || (may && maybe_at < left)) {
      const int place = sure_before + __popc(s & lower) + min(maybe_at, left);
      // (rows read again in every pass may change meanwhile, by a caller's mistake: not outside the list)
      if (place < p.keep) kept[place] = j0 + i;
      // a key says what the weight was, but for zeros' signs, NaN and protected rows
      if (out && place < p.keep)
        out[place] = key == kZero || key == kLowest || key == kProtected ? __ldg(row + j0 + i)
                     : __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
    }
    sure_before += __popc(s);
    maybe_before += __popc(m);
  });
  if (p.cluster > 1) cluster_sync();  // no CTA's counts go away while another reads them
}

// ------------------------------------------------------------------ compact
// A CTA moves kMoveRows rows of a request: where they lie and where they go is
// looked up once, then every thread copies 16-byte units, all of its loads in
// flight together.  HBM-bound: a row is read once and written once.  Small CTAs,
// so that one's lookups run beside others' copies, and streaming loads and stores:
// 64 requests x 4096 of up to 8192 rows (553 MB) 84.7 us, 6.5 TB/s, near a device
// copy's rate; 110 us with 256 threads and 32 rows a CTA, 104.5 without streaming.
constexpr int kMoveThreads = 128;
constexpr int kMoveRows = 16;

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
  grid_launch_dependents();
  grid_dependency_wait();
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
        if (at < kItems && s_src[r] >= 0) v[k] = ld_global_nc_v4(p.cache + s_src[r] + at % kUnits);
      }
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        const int at = k * kMoveThreads + threadIdx.x, r = at / kUnits;
        if (at < kItems && s_src[r] >= 0) __stcs(p.cache + s_dst[r] + at % kUnits, v[k]);
      }
      __syncthreads();
    }
  }
}

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
                                      kRoomRows * 4) == cudaSuccess &&
                         cudaFuncSetAttribute(mla_evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                              1) == cudaSuccess
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
      !al(new_lens, 4) || !al(status, 4) || !al(new_weights, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_requests < 0 || max_len < 1 || keep < 1 || sinks < 0 || recent < 0 || sinks > keep || recent > keep - sinks)
    return MLA_ERR_INVALID_ARG;
  if (num_requests > 1 && weights_stride < max_len) return MLA_ERR_INVALID_ARG;
  if (new_weights && (new_width < (keep < max_len ? keep : max_len) || (num_requests > 1 && new_weights_stride < new_width)))
    return MLA_ERR_INVALID_ARG;
  // rows are numbered in 32 bits, beyond the end by a grid's step
  if (max_len > (1 << 30) || keep > (1 << 30) || new_width > (1 << 30) || num_requests > INT32_MAX / kMaxCluster)
    return MLA_ERR_UNSUPPORTED;
  const int64_t apart = static_cast<int64_t>(reinterpret_cast<intptr_t>(new_lens) - reinterpret_cast<intptr_t>(cache_lens)) / 4;
  if (apart != 0 && apart < num_requests && -apart < num_requests) return MLA_ERR_INVALID_ARG;  // another request's length
  if (share(weights, weights_stride, max_len, new_weights, new_weights_stride, new_width, num_requests))
    return MLA_ERR_INVALID_ARG;
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
  while (p.cluster < kMaxCluster && static_cast<int64_t>(p.cluster) * kSelRows < max_len) p.cluster *= 2;
  const int rows = ((max_len + p.cluster - 1) / p.cluster + 31) / 32 * 32;
  p.room = rows < kRoomRows ? rows : kRoomRows;
  p.kept = kept;
  p.new_lens = new_lens;
  p.new_weights = new_weights;
  p.new_stride = new_weights_stride;
  p.new_width = new_weights ? new_width : 0;
  p.status = status;
  return launch_dependent(mla_evict_select_kernel, dim3(static_cast<unsigned>(num_requests) * p.cluster), dim3(kSelThreads),
                          p.room * 4, p.cluster, stream, p);
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
  return launch_dependent(row_bytes == 1152 ? mla_cache_compact_kernel<72>
                          : row_bytes == 256 ? mla_cache_compact_kernel<16>
                                             : mla_cache_compact_kernel<41>,
                          grid, dim3(kMoveThreads), 0, 1, stream, p);
}

}  // extern "C"
