// prefix_attend.cuh — what the two attention kernels over a shared prefix have
// in common: the work split and its walk, a softmax step on 32 scores, and the
// join with a suffix's result.
#pragma once
#include <cmath>
#include <cstdint>

#include "prefix_common.cuh"

namespace mla {
namespace prefix {

constexpr int kHeadDim = 128;
constexpr int kRope = 64;
constexpr int kTile = 128;                  // query rows of a row tile, keys of a key tile
constexpr int kQChunks = 3;                 // 64-dim chunks of a query or key row
constexpr int kQTile = kQChunks * 16384;    // 48 KiB: 128 query rows
constexpr int kSoftmaxWarps = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2 by which a score must beat the running maximum to move it: weights stay
// below 2^14, which fp16 (up to 65504) holds with its 11 bits.  At 8, peaked
// scores moved some row of a warp in 40 % of the tiles, and each time the warp
// rescaled O.
constexpr float kLazy = 14.0f;

// ---- work split
struct Plan {
  int nk;         // key tiles
  int blocks;     // row blocks of 256
  int width;      // row blocks worked on side by side by the CTAs of a group
  int groups;     // CTA groups, each with a range of the line
  int passes;     // ceil(blocks / width)
  long long line; // passes * heads * nk steps
};

struct AttendParams {
  const int* visible;
  int num_tokens, num_heads, prefix_len;
  float scale_log2;
  const uint16_t* suffix_out;
  const float* suffix_lse;
  int out_fp32;
  void* out;
  float* lse;
  float* part_o;    // [2 * units][rows][128], normalised
  float* part_lse;  // [2 * units][rows], log2
  int part_rows;
  Plan plan;
  int* status;
};

// x / n, x >= 0, n > 0: almost always in 32 bits (a 64-bit division is a hundred instructions).
__host__ __device__ __forceinline__ long long quotient(long long x, long long n) {
  return (x | n) >> 32 ? x / n : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(n));
}
__host__ __device__ __forceinline__ long long cut(const Plan& w, int g) { return quotient(w.line * g, w.groups); }

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 lanes x 16 consecutive 32-bit columns (the store of tmem_ld16).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Two fp32 in a 64-bit register, and the packed operations on them.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---- a softmax step on 32 consecutive scores of a row
// Scores `limit` and up become -inf.
__device__ __forceinline__ void mask32(uint32_t (&x)[32], int limit) {
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (k >= limit) x[k] = 0xff800000u;
}

// The largest of three, NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The largest score, NaN if one is no number.
__device__ __forceinline__ float max32(const uint32_t (&x)[32]) {
  float a = __uint_as_float(x[0]), b = __uint_as_float(x[1]);
#pragma unroll
  for (int k = 2; k < 30; k += 4) {
    a = max3_nan(a, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
    b = max3_nan(b, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
  }
  return max3_nan(max3_nan(a, b, __uint_as_float(x[30])), __uint_as_float(x[31]), -INFINITY);
}

// Whether a row that sees none of these keys has a score among them whose
// weight 2^(score * scale - inf) would not be zero: +inf, or no number (finite
// keys may overflow, and a padded token's query may hold anything).  Without
// `visible` only rows behind the prefix are hidden, which read as zeros.
__device__ __forceinline__ bool hidden_overflow(int limit, float top) { return limit <= 0 && !(top < INFINITY); }

// Weights 2^(x * scale - base) to 16 columns of tensor memory in fp16, and
// their sums: of the fp32 values, and of the fp16 ones that the value product
// takes (each widened exactly).
__device__ __forceinline__ void weights32(const uint32_t (&x)[32], float scale, float base, uint32_t taddr, float& total,
                                          float& used) {
  const uint64_t scale2 = pack_f32x2(scale, scale), base2 = pack_f32x2(-base, -base);
  uint32_t w[16];
  uint64_t t2 = 0;
  float u0 = 0.f, u1 = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float a0, a1;
    unpack_f32x2(
        fma_f32x2(pack_f32x2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), scale2, base2), a0, a1);
    a0 = ex2_approx(a0);
    a1 = ex2_approx(a1);
    t2 = add_f32x2(t2, pack_f32x2(a0, a1));
    w[k] = pack_f16x2(a0, a1);
    if (k & 1)
      u1 = add_f16x2_halves(u1, w[k]);
    else
      u0 = add_f16x2_halves(u0, w[k]);
  }
  tmem_st16(taddr, w);
  float t0, t1;
  unpack_f32x2(t2, t0, t1);
  total += t0 + t1;
  used += u0 + u1;
}

// 16 consecutive columns of O times `keep`.
__device__ __forceinline__ void rescale16(uint32_t taddr, float keep) {
  uint32_t o[16];
  tmem_ld16(taddr, o);
  tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
  tmem_st16(taddr, o);
}

// One segment of a CTA's range: key tiles [k0, k1) of head h for row block `block`.
struct Segment {
  int h, block, k0, k1, rows;
  bool first, whole;
};

struct SegmentIter {
  const Plan& w;
  int num_tokens, num_heads, lane_block, unit, k0;
  long long left;
  bool first;
  // `unit_id`: the CTA's number, or the pair's
  __device__ SegmentIter(const AttendParams& p, int unit_id)
      : w(p.plan), num_tokens(p.num_tokens), num_heads(p.num_heads) {
    const int g = unit_id / w.width;
    lane_block = unit_id % w.width;
    const long long begin = cut(w, g);
    left = cut(w, g + 1) - begin;
    unit = static_cast<int>(quotient(begin, w.nk));
    k0 = static_cast<int>(begin - static_cast<long long>(unit) * w.nk);
    first = true;
  }
  __device__ bool next(Segment& s) {
    if (left <= 0) return false;
    s.block = unit / num_heads * w.width + lane_block;
    if (s.block >= w.blocks) return false;  // blocks grow along the line
    s.h = unit % num_heads;
    s.k0 = k0;
    s.k1 = left < w.nk - k0 ? k0 + static_cast<int>(left) : w.nk;
    s.whole = s.k1 - k0 == w.nk;
    s.first = first;
    const int rows = num_tokens - s.block * 2 * kTile;
    s.rows = rows < 2 * kTile ? rows : 2 * kTile;
    left -= s.k1 - k0;
    k0 = 0;
    ++unit;
    first = false;
    return true;
  }
};

// Weights of the prefix's and the suffix's result in their join, and the joined LSE (log2).
struct Join {
  float mine, other, lse2;
};
__device__ __forceinline__ Join join(float lse2, float other2) {
  Join j;
  const float top = fmaxf(lse2, other2);
  const float base = top == -INFINITY ? 0.f : top;
  const float a = ex2_approx(lse2 - base), b = ex2_approx(other2 - base);
  const float sum = a + b;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
  j.mine = a * inv;
  j.other = b * inv;
  j.lse2 = sum == 0.f ? -INFINITY : base + lg2(sum);
  return j;
}

// 8 result columns of a row: their share of the join with the suffix's 8.
__device__ __forceinline__ void join8(float* x, const Join& j, const uint4& suffix) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= j.mine;
  if (j.other != 0.f) {  // a suffix without a share is not read as numbers
    const uint32_t w[4] = {suffix.x, suffix.y, suffix.z, suffix.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = fmaf(__uint_as_float(w[i] << 16), j.other, x[2 * i]);
      x[2 * i + 1] = fmaf(__uint_as_float(w[i] & 0xffff0000u), j.other, x[2 * i + 1]);
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint4 pack4(const float* x) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// Joins and writes 8 columns of a row (16-byte pieces).
__device__ __forceinline__ void write8(const AttendParams& p, long long row, int col, const float* o, const Join& j) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = o[i];
  const long long at = row * kHeadDim + col;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (p.suffix_out) v = *reinterpret_cast<const uint4*>(p.suffix_out + at);
  join8(x, j, v);
  if (p.out_fp32) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(p.out) + at);
    dst[0] = pack4(x);
    dst[1] = pack4(x + 4);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) = pack8(x);
  }
}

// The same for 4 columns.
__device__ __forceinline__ void write4(const AttendParams& p, long long row, int col, const float4& o, const Join& j) {
  float x[4] = {o.x * j.mine, o.y * j.mine, o.z * j.mine, o.w * j.mine};
  const long long at = row * kHeadDim + col;
  if (p.suffix_out && j.other != 0.f) {  // a suffix without a share is not read as numbers
    const uint2 s = *reinterpret_cast<const uint2*>(p.suffix_out + at);
    x[0] = fmaf(__uint_as_float(s.x << 16), j.other, x[0]);
    x[1] = fmaf(__uint_as_float(s.x & 0xffff0000u), j.other, x[1]);
    x[2] = fmaf(__uint_as_float(s.y << 16), j.other, x[2]);
    x[3] = fmaf(__uint_as_float(s.y & 0xffff0000u), j.other, x[3]);
  }
  if (p.out_fp32)
    *reinterpret_cast<uint4*>(static_cast<float*>(p.out) + at) = pack4(x);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// The segment epilogue of a warp: 32 rows (one a lane), 32 columns from `col`.
// Rows lie heads * 256 bytes apart, so that a warp that stored its rows as it
// holds them would touch 32 lines with every 16-byte store (7,000 cycles for
// a CTA's 128 rows); transposed over four lanes, 64 bytes of 8 rows, it
// touches 8.  (Up to 128 tokens the plain stores are as fast or faster: few of
// the rows are real, and the code is shorter.)
struct RowOut {
  long long quad_row;  // first of the quad's four rows, in the result or among the partial rows
  int step;            // rows between them
  int left;            // rows from the first on that are real
  bool whole;
};

// The suffix's columns, four lanes to a row (asked for early; see write32).
__device__ __forceinline__ void load_suffix(const AttendParams& p, const RowOut& w, uint32_t col, int lane, uint4 (&c)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.suffix_out && w.whole && i < w.left)
      c[i] = *reinterpret_cast<const uint4*>(p.suffix_out + (w.quad_row + static_cast<long long>(i) * w.step) * kHeadDim +
                                             col + 8 * (lane & 3));
  }
}

// `read16(h, o)` gives columns col + 16 h .. of the lane's row.
template <typename F>
__device__ __forceinline__ void write32(const AttendParams& p, const RowOut& w, uint32_t col, int lane, const Join& j,
                                        uint4 (&c)[4], F read16) {
  const bool joined = p.suffix_out && w.whole, fp32 = !w.whole || p.out_fp32;
  float* dst32 = w.whole ? static_cast<float*>(p.out) : p.part_o;
  const long long at = w.quad_row * kHeadDim + col, step = static_cast<long long>(w.step) * kHeadDim;
  if (joined) quad_transpose(c, lane);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float o[16];
    read16(h, o);
    if (joined) {
      join8(o, j, c[2 * h]);
      join8(o + 8, j, c[2 * h + 1]);
    }
    if (!fp32) {
      c[2 * h] = pack8(o);
      c[2 * h + 1] = pack8(o + 8);
    } else {
      uint4 d[4] = {pack4(o), pack4(o + 4), pack4(o + 8), pack4(o + 12)};
      quad_transpose(d, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < w.left) *reinterpret_cast<uint4*>(dst32 + at + i * step + 16 * h + 4 * (lane & 3)) = d[i];
    }
  }
  if (!fp32) {
    quad_transpose(c, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < w.left) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at + i * step + 8 * (lane & 3)) = c[i];
  }
}

// The kernel for more than 128 tokens (prefix_attend_pair.cu).
cudaError_t attend_pair_set_attrs();
int attend_pair_launch(int pairs, mla_stream_t stream, const AttendParams& p, const CUtensorMap& qn,
                       const CUtensorMap& qp, const CUtensorMap& k, const CUtensorMap& kp, const CUtensorMap& v);

}  // namespace prefix
}  // namespace mla
