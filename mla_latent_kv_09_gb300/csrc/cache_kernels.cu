// cache_kernels.cu — rotary positions and the append to the paged latent
// cache, with their C ABI (include/mla_cache.h).
//
// Both are streams: every element is read once and written once, a few
// operations each, so HBM bounds the long calls and launch latency the short
// ones.  Measured: rotation of 8192 tokens x 128 heads x 192 dims 117.6 us (805
// MB at 6.85 TB/s, a copy's rate; half layout 121), 1332 x 64 x 128 in the half
// layout 6.9 us where the rows lie in L2, 9.3 from the HBM (44 MB), 64 x 128 x 64
// 2.0 us; append of 8192 tokens 4.7 us (19 MB), of 64 tokens 2.2 us.
//
// Angles.  Pair i at position p turns by p * f_i radians.  In fp32 that loses
// the angle at far positions (at p = 2^20 one ulp is 1/16 radian), and fp64
// is slow on this chip.  A rotation only needs the angle modulo one turn, and
// p is whole: with F = f_i / 2 pi as a 64-bit fixed-point fraction of a turn,
// p * F mod 2^64 IS the angle modulo one turn, exact in F's last bit, in one
// integer product.  F comes in whole numbers too, as f_i's 53-bit mantissa times
// the 128 bits of 1 / 2 pi that its exponent picks: off by less than 2 2^-64
// turns, so the angle by 2^-32 turns at most, whatever the frequency (an fp64
// product f_i * (1 / 2 pi) is off by 2^-53 of itself: 2e-5 radians for f = 100
// at p = 2^31).  The top 32 bits as a signed fraction in [-1/2, 1/2) go through
// sincospif.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "kernel_common.cuh"
#include "mla_cache.h"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeItems = 4;     // 16-byte units per thread and turn, all loads in flight together
constexpr int kRopeCtas = 8 * 152;  // CTAs wanted before a token's heads stay in one CTA
constexpr int kLatent = 512;
constexpr int kRopeDim = 64;
constexpr int kFp8Row = MLA_FP8_ROW_BYTES;
constexpr int kAppendWarps = 4;

__device__ __forceinline__ float2 turn(double f, int pos, bool inverse, float scale) {
  // f = m 2^(e - 1075), so turns a position times 2^64, modulo 2^64 (positions are
  // whole: whole turns drop out), are m times (1 / 2 pi) 2^(e - 1011): its 64 bits
  // ahead of the point and the 64 behind it, from the first 128 bits of 1 / 2 pi.
  constexpr unsigned long long kTurn0 = 0x28be60db9391054aull, kTurn1 = 0x7f09d5f47d4d3770ull;
  const long long bits = __double_as_longlong(f);
  const int e = static_cast<int>(bits >> 52) & 2047;
  const unsigned long long m = (bits & 0xfffffffffffffll) | (e != 0 ? 0x10000000000000ll : 0ll);
  const int up = min(e - 1011, 63);  // (frequencies of 2^52 and more turn by no angle in particular)
  unsigned long long ahead = 0, behind = up > -64 ? kTurn0 >> (-up & 63) : 0;
  if (up > 0) {
    ahead = kTurn0 >> (64 - up);
    behind = kTurn0 << up | kTurn1 >> (64 - up);
  }
  unsigned long long fix = m * ahead + __umul64hi(m, behind);
  if (bits < 0) fix = 0 - fix;
  const unsigned long long a = fix * static_cast<unsigned long long>(static_cast<long long>(pos));
  const float half_turns = static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * scale, (inverse ? -s : s) * scale);
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

struct RopeParams {
  const uint16_t* x;
  long long x_ts, x_hs;
  const int* positions;
  int tokens, heads, offset, rope;
  int units;     // 16-byte units per head that a thread handles (rotated ones, and copied ones out of place)
  int per_turn;  // heads of a token that a CTA's threads cover side by side
  int together;  // tokens of a CTA
  int copy;      // dims outside the rotated range are copied
  const double* inv_freq;
  float scale;
  int inverse;
  uint16_t* out;
  long long out_ts, out_hs;
};

// One CTA: one token, its heads in turns of per_turn * kRopeItems, or several
// tokens of few heads (8192 tokens x 1 head x 64 dims 22 us with a CTA each,
// 4.0 so).  A unit is 8 contiguous dims: 4 interleaved pairs, or 8 copied dims; a warp's units are
// neighbours in memory.  A thread keeps one unit for all its heads: its cosines
// and sines stay in registers, and nothing is divided in the loop.  In the half
// layout a unit's 8 dims need their 8 partners: there the two threads of a unit
// and its partner's each take both for half of the heads, so that every thread
// has the same four loads in flight (a thread with two loads a head and its
// copying neighbours with one: 8192 tokens x 128 heads x 192 dims 168 us
// instead of 122).  The first turn's loads are issued before the angles are
// computed (once a token, through shared memory), which hides sincospif and the
// position's load behind them.
template <bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, kHalf ? 4 : 5) mla_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[4 * kRopeThreads];   // [token][pair]: a token has at least rope / 8 threads
  const bool wide = p.units > kRopeThreads;  // a head is more than a CTA: units in blocks of kRopeThreads
  const int u = wide ? blockIdx.z * kRopeThreads + threadIdx.x : threadIdx.x % p.units;
  const int place = wide ? 0 : threadIdx.x / p.units;  // (token, head) of those side by side
  const int token = place / p.per_turn, h0 = place - token * p.per_turn;
  const long long t = static_cast<long long>(blockIdx.x) * p.together + token;
  const bool mine = (wide ? u < p.units : token < p.together) && t < p.tokens;
  const int before = p.copy ? p.offset / 8 : 0;     // copied units ahead of the rotated ones
  const int r = u - before;
  const bool turns = r >= 0 && r < p.rope / 8;
  const int second = kHalf && turns && r >= p.rope / 16 ? 1 : 0;  // takes the second half of the heads
  const int unit = second ? r - p.rope / 16 : r;
  const int dim = turns ? p.offset + 8 * unit : (r < 0 ? 8 * u : p.offset + p.rope + 8 * (r - p.rope / 8));
  const int pair = turns ? (kHalf ? 8 * unit : 4 * unit) : 0;
  const int step = p.per_turn * kRopeItems;
  grid_dependency_wait();
  const uint16_t* src = p.x + t * p.x_ts + dim;
  uint16_t* dst = p.out + t * p.out_ts + dim;
  const bool both = kHalf && turns;  // items are a unit and its partner of two heads, not a unit of four
  uint4 v[kRopeItems] = {};
  auto head = [&](int base, int i) { return base + h0 + (both ? 2 * second + (i >> 1) : i) * p.per_turn; };
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kRopeItems; ++i) {
      const int h = head(base, i);
      if (!mine || h >= p.heads) continue;
      v[i] = *reinterpret_cast<const uint4*>(src + h * p.x_hs + (both && (i & 1) ? p.rope / 2 : 0));
    }
  };
  int base = blockIdx.y * step;
  load(base);
  for (int i = threadIdx.x; i < p.together * (p.rope / 2); i += kRopeThreads) {
    const int of = i / (p.rope / 2);
    const long long at = static_cast<long long>(blockIdx.x) * p.together + of;
    if (at < p.tokens) cs[i] = turn(p.inv_freq[i - of * (p.rope / 2)], p.positions[at], p.inverse != 0, p.scale);
  }
  __syncthreads();
  float2 c[kHalf ? 8 : 4];
#pragma unroll
  for (int j = 0; j < (kHalf ? 8 : 4); ++j) c[j] = cs[mine ? token * (p.rope / 2) + pair + j : 0];
#pragma unroll 1
  while (base < p.heads) {
    if (kHalf && turns) {
#pragma unroll
      for (int i = 0; i < kRopeItems; i += 2) {
        uint32_t* x = reinterpret_cast<uint32_t*>(&v[i]);
        uint32_t* y = reinterpret_cast<uint32_t*>(&v[i + 1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 c0 = c[2 * j], c1 = c[2 * j + 1];
          const float x0 = lo_f(x[j]), x1 = hi_f(x[j]), y0 = lo_f(y[j]), y1 = hi_f(y[j]);
          x[j] = pack_bf16x2(x0 * c0.x - y0 * c0.y, x1 * c1.x - y1 * c1.y);
          y[j] = pack_bf16x2(x0 * c0.y + y0 * c0.x, x1 * c1.y + y1 * c1.x);
        }
      }
    } else if (turns) {
#pragma unroll
      for (int i = 0; i < kRopeItems; ++i) {
        uint32_t* x = reinterpret_cast<uint32_t*>(&v[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = lo_f(x[j]), x1 = hi_f(x[j]);
          x[j] = pack_bf16x2(x0 * c[j].x - x1 * c[j].y, x0 * c[j].y + x1 * c[j].x);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRopeItems; ++i) {
      const int h = head(base, i);
      if (!mine || h >= p.heads) continue;
      *reinterpret_cast<uint4*>(dst + h * p.out_hs + (both && (i & 1) ? p.rope / 2 : 0)) = v[i];
    }
    base += gridDim.y * step;
    if (base < p.heads) load(base);
  }
}

struct AppendParams {
  const uint16_t* latent;
  long long latent_stride;
  const uint16_t* k_pe;
  long long k_pe_stride;
  const uint16_t* weight;
  float eps;
  const double* inv_freq;
  float rope_scale;
  const int* positions;
  const int* request_ids;
  int num_tokens, per_request;
  const int* block_table;
  long long bt_stride;
  int bt_width;
  int num_requests;
  uint8_t* cache;
  long long num_pages;
  int* status;
};

// Two fp32 values to a pair of E4M3 codes, nearest even; what is not finite
// becomes NaN (the conversion alone would saturate an infinity to 448).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  const float nan = __int_as_float(0x7fffffff);
  lo = isfinite(lo) ? lo : nan;
  hi = isfinite(hi) ? hi : nan;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// One warp per token.  Lane l holds latent dims [8 l, 8 l + 8) and 256 on, so
// that both loads and both stores of the warp are contiguous, and a 128-dim
// FP8 group is 16 lanes of one half; it turns pair l of the RoPE dims, whose
// angle it computes itself.  Nothing goes through shared memory, so tokens
// only share the SM's latency.
template <bool kFp8, bool kHalf>
__global__ void __launch_bounds__(32 * kAppendWarps) mla_append_kernel(const __grid_constant__ AppendParams p) {
  const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  if (t >= p.num_tokens) return;
  const int pos = p.positions[t];
  if (pos < 0) return;
  const int req = p.request_ids ? p.request_ids[t] : t / p.per_request;
  uint4 v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v[i] = *reinterpret_cast<const uint4*>(p.latent + t * p.latent_stride + 256 * i + 8 * lane);
  const uint16_t* pe = p.k_pe + t * p.k_pe_stride;
  float pa, pb;  // the lane's pair
  if (kHalf) {
    pa = __uint_as_float(static_cast<uint32_t>(pe[lane]) << 16);
    pb = __uint_as_float(static_cast<uint32_t>(pe[lane + 32]) << 16);
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(pe + 2 * lane);
    pa = lo_f(w);
    pb = hi_f(w);
  }
  // the row; a request, position or page out of range skips the token
  bool ok = req >= 0 && req < p.num_requests && pos / kPage < p.bt_width;
  long long page = -1;
  if (ok) page = p.block_table[req * p.bt_stride + pos / kPage];
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
    return;
  }
  const long long row = page * kPage + pos % kPage;

  float x[16];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = lo_f(w[j]);
      x[8 * i + 2 * j + 1] = hi_f(w[j]);
    }
  }
  if (p.weight) {
    auto squares = [&x] {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      return ss;
    };
    float mean = squares() * (1.0f / kLatent), eps = p.eps;
    // Squares beyond fp32's range, at either end, where eps does not outweigh
    // them: again with the latent times a power of two, which the norm drops
    // (2^-70 keeps the sum of 512 squares finite; 2^100 brings the least bf16
    // number, 2^-133, to where its square is a normal one).
    if (!(mean + eps < INFINITY) || mean + eps < 1e-30f) {
      const float by = mean < 1.f ? 0x1p100f : 0x1p-70f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= by;
      mean = squares() * (1.0f / kLatent);
      eps = eps * by * by;
    }
    const float r = 1.0f / sqrtf(mean + eps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 wv = *reinterpret_cast<const uint4*>(p.weight + 256 * i + 8 * lane);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&wv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = x[8 * i + 2 * j] * r * lo_f(w[j]);
        x[8 * i + 2 * j + 1] = x[8 * i + 2 * j + 1] * r * hi_f(w[j]);
      }
    }
  }
  if (p.inv_freq) {
    const float2 c = turn(p.inv_freq[lane], pos, false, p.rope_scale);
    const float a = pa * c.x - pb * c.y, b = pa * c.y + pb * c.x;
    pa = a;
    pb = b;
  }

  uint8_t* dst = p.cache + row * (kFp8 ? kFp8Row : 2 * kDqk);
  if (!kFp8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 o;
      o.x = pack_bf16x2(x[8 * i + 0], x[8 * i + 1]);
      o.y = pack_bf16x2(x[8 * i + 2], x[8 * i + 3]);
      o.z = pack_bf16x2(x[8 * i + 4], x[8 * i + 5]);
      o.w = pack_bf16x2(x[8 * i + 6], x[8 * i + 7]);
      *reinterpret_cast<uint4*>(dst + 512 * i + 16 * lane) = o;
    }
  } else {
    // Group scale 2^e, the smallest with amax <= 448 * 2^e = 1.75 * 2^(e + 8):
    // read off amax's exponent and mantissa, exactly.
    uint32_t scales = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = fabsf(x[8 * i + j]);
        m = isfinite(a) ? fmaxf(m, a) : m;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int bits = __float_as_int(m);
      int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
      e = m == 0.f ? 0 : (e < -127 ? -127 : e);
      // 2^-e with e in [-127, 120]: a normal fp32 (exponent field 127 - e in [7, 254])
      const float inv = __int_as_float((127 - e) << 23);
      uint2 o;
      o.x = e4m3x2(x[8 * i + 0] * inv, x[8 * i + 1] * inv) | e4m3x2(x[8 * i + 2] * inv, x[8 * i + 3] * inv) << 16;
      o.y = e4m3x2(x[8 * i + 4] * inv, x[8 * i + 5] * inv) | e4m3x2(x[8 * i + 6] * inv, x[8 * i + 7] * inv) << 16;
      *reinterpret_cast<uint2*>(dst + 256 * i + 8 * lane) = o;
      const uint32_t mine = static_cast<uint32_t>(e + 127);
      scales |= (__shfl_sync(0xffffffffu, mine, 0) | __shfl_sync(0xffffffffu, mine, 16) << 8) << (16 * i);
    }
    if (lane == 0) *reinterpret_cast<uint4*>(dst + kLatent) = make_uint4(scales, 0u, 0u, 0u);
  }
  uint16_t* dpe = reinterpret_cast<uint16_t*>(dst + (kFp8 ? 528 : 2 * kLatent));
  const uint32_t w = pack_bf16x2(pa, pb);
  if (kHalf) {
    dpe[lane] = static_cast<uint16_t>(w);
    dpe[lane + 32] = static_cast<uint16_t>(w >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(dpe + 2 * lane) = w;
  }
}

// ============================================================ host side
constexpr int kMaxDev = 64;
struct CacheDevice {
  std::once_flag once;
  int status = MLA_OK;
};
CacheDevice g_cache_dev[kMaxDev];

int cache_device_ready() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return MLA_ERR_DEVICE;
  CacheDevice& st = g_cache_dev[dev];
  std::call_once(st.once, [&st, dev] {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess || major != 10 ||
        minor != 3)
      st.status = MLA_ERR_DEVICE;
  });
  return st.status;
}

template <typename P>
int launch_dependent(void (*kernel)(P), dim3 grid, dim3 block, mla_stream_t stream, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool row_stride_ok(int64_t s, int64_t min) { return s >= min && (s & 7) == 0 && s <= (int64_t{1} << 30); }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int mla_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
             int num_tokens, int num_heads, int head_dim, int rope_offset, int rope_dim, const double* inv_freq,
             float scale, unsigned flags, void* out, int64_t out_token_stride, int64_t out_head_stride,
             mla_stream_t stream) {
  if (!x || !positions || !inv_freq || !out || !al(x, 16) || !al(out, 16) || !al(positions, 4) || !al(inv_freq, 8))
    return MLA_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_heads < 1 || head_dim < 8 || rope_offset < 0 || rope_dim < 2) return MLA_ERR_INVALID_ARG;
  if (flags & ~static_cast<unsigned>(MLA_FLAG_ROPE_HALF | MLA_FLAG_ROPE_INVERSE)) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return MLA_ERR_INVALID_ARG;
  if (head_dim % 8 || rope_offset % 8 || rope_dim % 16 || rope_dim > MLA_MAX_ROPE_DIM || head_dim > (1 << 16) ||
      num_heads > (1 << 30))
    return MLA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(rope_offset) + rope_dim > head_dim) return MLA_ERR_INVALID_ARG;
  if (!row_stride_ok(x_token_stride, 0) || !row_stride_ok(x_head_stride, 0) || !row_stride_ok(out_token_stride, 0) ||
      !row_stride_ok(out_head_stride, 0))
    return MLA_ERR_INVALID_ARG;
  // rows of the output are distinct: all heads of a token lie between two tokens, or the other way round
  if ((num_heads > 1 && out_head_stride < head_dim) || (num_tokens > 1 && out_token_stride < head_dim))
    return MLA_ERR_INVALID_ARG;
  if (num_heads > 1 && num_tokens > 1 && out_token_stride < (num_heads - 1) * out_head_stride + head_dim &&
      out_head_stride < (num_tokens - 1) * out_token_stride + head_dim)
    return MLA_ERR_INVALID_ARG;
  const bool in_place = x == out;
  if (in_place && ((num_tokens > 1 && x_token_stride != out_token_stride) ||
                   (num_heads > 1 && x_head_stride != out_head_stride)))
    return MLA_ERR_INVALID_ARG;
  const bool half = (flags & MLA_FLAG_ROPE_HALF) != 0;
  RopeParams p;
  p.x = static_cast<const uint16_t*>(x);
  p.x_ts = x_token_stride;
  p.x_hs = x_head_stride;
  p.positions = positions;
  p.tokens = num_tokens;
  p.heads = num_heads;
  p.offset = rope_offset;
  p.rope = rope_dim;
  p.copy = in_place ? 0 : 1;
  p.units = (in_place ? rope_dim : head_dim) / 8;
  p.inv_freq = inv_freq;
  p.scale = scale;
  p.inverse = (flags & MLA_FLAG_ROPE_INVERSE) != 0;
  p.out = static_cast<uint16_t*>(out);
  p.out_ts = out_token_stride;
  p.out_hs = out_head_stride;
  // heads side by side, no more than a turn takes; the room left goes to further
  // tokens, once there are more of them than CTAs to keep the SMs busy (64 tokens
  // x 1 head together 4.1 us, apart 1.9)
  const int room = p.units < kRopeThreads ? kRopeThreads / p.units : 1, need = (num_heads + kRopeItems - 1) / kRopeItems;
  p.per_turn = room < need ? room : need;
  const int64_t spread = (static_cast<int64_t>(num_tokens) + kRopeCtas / 2 - 1) / (kRopeCtas / 2);
  p.together = room / p.per_turn;
  if (p.together > spread) p.together = spread > 1 ? static_cast<int>(spread) : 1;
  const int rc = cache_device_ready();
  if (rc != MLA_OK) return rc;
  if (num_tokens == 0) return MLA_OK;
  // few tokens: their heads spread over CTAs; many: a CTA takes all of a token's
  const int64_t x_blocks = (static_cast<int64_t>(num_tokens) + p.together - 1) / p.together;
  const int64_t blocks = (static_cast<int64_t>(num_heads) + p.per_turn * kRopeItems - 1) / (p.per_turn * kRopeItems);
  int64_t y = (kRopeCtas + x_blocks - 1) / x_blocks;
  if (y > blocks) y = blocks;
  const dim3 grid(static_cast<unsigned>(x_blocks), static_cast<unsigned>(y), (p.units + kRopeThreads - 1) / kRopeThreads);
  return launch_dependent(half ? mla_rope_kernel<true> : mla_rope_kernel<false>, grid, dim3(kRopeThreads), stream, p);
}

int mla_cache_append(const void* latent, int64_t latent_stride, const void* k_pe, int64_t k_pe_stride,
                     const void* norm_weight, float eps, const double* inv_freq, float rope_scale,
                     const int32_t* positions, const int32_t* request_ids, int num_tokens,
                     const int32_t* block_table, int64_t bt_stride, int bt_width, int num_requests, void* kv_cache,
                     int64_t num_pages, unsigned flags, int* status, mla_stream_t stream) {
  if (!latent || !k_pe || !positions || !block_table || !kv_cache || !status) return MLA_ERR_INVALID_ARG;
  if (!al(latent, 16) || !al(k_pe, 16) || !al(norm_weight, 16) || !al(inv_freq, 8) || !al(positions, 4) ||
      !al(request_ids, 4) || !al(block_table, 4) || !al(kv_cache, 16) || !al(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_requests < 1 || bt_width < 1 || bt_stride < bt_width || num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (flags & ~static_cast<unsigned>(MLA_FLAG_KV_FP8 | MLA_FLAG_ROPE_HALF)) return MLA_ERR_INVALID_ARG;
  if (!row_stride_ok(latent_stride, kLatent) || !row_stride_ok(k_pe_stride, kRopeDim)) return MLA_ERR_INVALID_ARG;
  if (norm_weight && !(eps >= 0.f && std::isfinite(eps))) return MLA_ERR_INVALID_ARG;
  if (inv_freq && !std::isfinite(rope_scale)) return MLA_ERR_INVALID_ARG;
  if (!request_ids && num_tokens % num_requests != 0) return MLA_ERR_INVALID_ARG;
  if (num_pages > (INT32_MAX / kPage) - 1 || num_tokens > INT32_MAX - kAppendWarps) return MLA_ERR_UNSUPPORTED;
  const int rc = cache_device_ready();
  if (rc != MLA_OK) return rc;
  if (num_tokens == 0) return MLA_OK;
  AppendParams p;
  p.latent = static_cast<const uint16_t*>(latent);
  p.latent_stride = latent_stride;
  p.k_pe = static_cast<const uint16_t*>(k_pe);
  p.k_pe_stride = k_pe_stride;
  p.weight = static_cast<const uint16_t*>(norm_weight);
  p.eps = eps;
  p.inv_freq = inv_freq;
  p.rope_scale = rope_scale;
  p.positions = positions;
  p.request_ids = request_ids;
  p.num_tokens = num_tokens;
  p.per_request = request_ids ? 1 : num_tokens / num_requests;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.bt_width = bt_width;
  p.num_requests = num_requests;
  p.cache = static_cast<uint8_t*>(kv_cache);
  p.num_pages = num_pages;
  p.status = status;
  const dim3 grid((num_tokens + kAppendWarps - 1) / kAppendWarps), block(32 * kAppendWarps);
  const bool fp8 = (flags & MLA_FLAG_KV_FP8) != 0, half = (flags & MLA_FLAG_ROPE_HALF) != 0;
  return launch_dependent(fp8 ? (half ? mla_append_kernel<true, true> : mla_append_kernel<true, false>)
                              : (half ? mla_append_kernel<false, true> : mla_append_kernel<false, false>),
                          grid, block, stream, p);
}

}  // extern "C"
