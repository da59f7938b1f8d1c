// weights_kernel.cu — the attention weight that every cached row received, with
// its C ABI (include/mla_evict.h).
//
// w[j] = sum over the tokens that see row j, and over 128 heads, of
// exp(q . row_j * scale - lse): the scores are products of rows and heads with
// K = 576, and what comes of them is one number a row.  So rows are the MMA's M
// and a token's heads its N: every thread of the epilogue holds a row's scores
// with 64 heads, and the sum over heads needs no other lane.
//
// A pair of SMs takes tiles of 256 rows (four pages) and runs a token's 128
// heads over each: M256 N128 tcgen05 operations over the pair, each CTA holding
// half of the rows and half of the heads.  Rows stay in shared memory for all
// tokens of their request and a token's query for all tiles until the next
// token's comes: one step a request (decode) streams rows past a resident query,
// bound by HBM; many tokens (an observation window) stream queries past resident
// rows, bound by the tensor cores.  Both operands lie in four groups of 64-dim
// chunks, each given back as soon as its last product is done, so that the next
// one's load runs behind the other groups' products.
//
// A step's K is cut into two accumulators, chunks 0-4 and 5-8 (FP8 0-3 and 4-8),
// that eight warps add in fp32 (four lane quarters, two halves of the heads).  A tensor core
// truncates when it accumulates, so that a score comes out too small by about
// half a step for each of its K / 16 additions, and the sum over heads and tokens
// does not average that away: 32 tokens x 16384 rows were off by 1.5e-6 with one
// accumulator, 7e-7 with two.  And each accumulator has a thread of its own to
// issue its products: one thread alone issues more slowly than they execute (32 x
// 16384 75 us against 55, before the steps below).
//
// Work: the (tile, token) steps of all requests lie on a line that is cut into
// equal ranges, one a pair.  A range that begins inside a tile's tokens writes
// that tile's part to the workspace, and a second kernel adds the parts in the
// line's order: no atomics, equal calls give equal bits.
//
// FP8 rows come as codes by TMA and are widened in place by eight further warps, a
// chain (codes 2 us, widening 0.8, hand-over to the pair 0.5, products 0.6) that
// one tile in shared memory lets run once a tile and so bounds one or two tokens
// a request: 64 x 8192 114 us (3.0 TB/s; bf16 100, 6.1 TB/s), 33 x 2 x 2560 35
// (29), 64 x 2 x 8192 161 (125).  Many tokens: 32 x 16384 55 (52), 64 x 65536 341
// (343: 1.8 PFLOP/s).  The next tile's pages asked into L2 did not shorten it.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "mla_evict.h"
#include "prefix_common.cuh"

namespace mla {
namespace {

using namespace prefix;

constexpr int kRows = 128;                    // of a CTA's half of a tile
constexpr int kTileRows = 2 * kRows;
constexpr int kKChunk = kRows * 128;          // 16 KiB: 128 rows x 64 dims
constexpr int kQChunk = 64 * 128;             // 8 KiB: 64 heads x 64 dims
// Chunks lie in groups that land and are given back together (a commit a chunk
// made 32 x 16384 107 us instead of the 55 of then).  An FP8 cache's codes come two chunks at
// a time; bf16 rows with these groups: 64 x 2 x 8192 143 us against 131.
constexpr int kGroups = 4;
template <bool kFp8>
__host__ __device__ constexpr int group_begin(int g) {  // 0, 3, 5, 7, 9; FP8 0, 2, 4, 6, 9
  return kFp8 ? (g < 4 ? 2 * g : 9) : (g < 2 ? 3 * g : 2 * g + 1);
}
// The two issuers take a half of the groups each and go through them side by
// side: groups land 0, 2, 1, 3, as they are given back (0, 1, 2, 3: 64 x 8192
// 102.6 us against 99.7, 64 tokens x 65536 361 against 352).
__device__ __forceinline__ int group_turn(int i) { return (i & 1) << 1 | i >> 1; }
static_assert(group_begin<false>(kGroups) == kNumChunks && group_begin<true>(kGroups) == kNumChunks, "all chunks");
constexpr int kUnits = 76;                    // SM pairs
constexpr int kOffQ = kNumChunks * kKChunk;
constexpr int kOffLse = kOffQ + kNumChunks * kQChunk;      // float[8 warps][64]
constexpr int kOffHalf = kOffLse + 8 * 64 * 4;             // float[2][128]: the other half's sums
constexpr int kOffWalk = kOffHalf + 2 * kRows * 4;         // where this unit's range begins
constexpr int kOffBar = kOffWalk + 64;
enum Bar {
  kKF = 0,                    // [4] rank 0: a group of the rows landed in both CTAs
  kKE = kKF + kGroups,        // [4] its last product is done
  kQF = kKE + kGroups,        // [4] rank 0: a group of the query landed in both CTAs
  kQE = kQF + kGroups,        // [4] its last product is done
  kAF = kQE + kGroups,        // [2] both accumulators of a step complete
  kAE = kAF + 2,              // [2] rank 0: ... and read by the sixteen warps of both CTAs
  kRaw = kAE + 2,             // [4] FP8 rows: a group's codes landed in this CTA
  kWide = kRaw + kGroups,     // [4] rank 1, FP8 rows: widened (for the relay)
  kDrain = kWide + kGroups,   // [2] per issuer
  kNumBars = kDrain + 2
};
constexpr int kSlack = 1024;
constexpr int kSmem = kOffBar + kNumBars * 8 + 16 + kSlack;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kEpiWarp = 4;                   // eight warps (a multiple of four: lane quarters)
constexpr int kFillWarp = 12;                 // eight further warps, FP8 rows only
constexpr int kPeAt = 264;                    // an FP8 row's position dims, in bf16 elements
constexpr int kThreads = 32 * 12, kThreadsFp8 = 32 * 20;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdesc = idesc_bf16(256, 128, 0);
constexpr float kLog2e = 1.4426950408889634f;

struct WeightsParams {
  const uint8_t* kv;
  long long num_pages;
  const float* lse;
  const int* table;
  long long bt_stride;
  const int* lens;
  int max_len;
  const int* starts;
  int requests, tokens, causal;
  float scale_log2, decay;
  const float* weights;
  long long w_stride;
  float* out;
  long long out_stride;
  int4* begins;  // [kUnits] {request, tile, first token in it, 0}; request -1: no work
  float* parts;  // [kUnits][kTileRows]
  int* status;
};

__device__ __forceinline__ int start_of(const WeightsParams& p, int b) {
  if (!p.starts) return b * (p.tokens / p.requests);
  return min(max(__ldg(p.starts + b), 0), p.tokens);
}
__device__ __forceinline__ int len_of(const WeightsParams& p, int b) {
  return min(max(__ldg(p.lens + b), 0), p.max_len);
}

// A unit's visits to tiles, in the line's order.
struct Visit {
  int b, tile, t0, t1;    // steps [t0, t1) of the tile
  int first, n, len;      // the request's first token, its tokens and rows
  // Those of its steps whose token sees a row of the tile: how many, the first
  // one's token of the batch, and the way on.  Tokens take their turns over odd
  // tiles backwards, so that a tile begins with the query that the last one ended with.
  int steps, q0, way;
};
__device__ __forceinline__ int limit(const Visit& v, int q, int causal) {  // rows that token q of the batch sees
  return causal ? max(0, v.len - v.n + q - v.first + 1) : v.len;
}
struct Walk {
  const WeightsParams& p;
  int b, tile, tok;
  long long left;
  int first, n, len;
  __device__ Walk(const WeightsParams& params, const int* begin) : p(params) {
    b = begin[0];
    tile = begin[1];
    tok = begin[2];
    left = static_cast<long long>(static_cast<uint32_t>(begin[4])) | static_cast<long long>(begin[5]) << 32;
    if (left > 0) request();
  }
  __device__ void request() {
    first = start_of(p, b);
    n = start_of(p, b + 1) - first;
    len = len_of(p, b);
  }
  __device__ bool next(Visit& v) {
    if (left <= 0) return false;
    while (n <= 0 || tile * kTileRows >= len) {  // (`left` says that there is a further request)
      if (++b >= p.requests) return false;
      tile = 0;
      request();
    }
    v.b = b;
    v.tile = tile;
    v.t0 = tok;
    v.t1 = left < n - tok ? tok + static_cast<int>(left) : n;
    v.first = first;
    v.n = n;
    v.len = len;
    const int blind = p.causal ? max(0, tile * kTileRows - (len - n)) : 0;  // tokens that see nothing of it
    const int s0 = tile & 1 ? v.t0 : max(v.t0, blind);
    v.steps = (tile & 1 ? min(v.t1, n - blind) : v.t1) - s0;
    v.q0 = first + (tile & 1 ? n - 1 - s0 : s0);
    v.way = tile & 1 ? -1 : 1;
    left -= v.t1 - tok;
    tok = v.t1;
    if (tok == n) {
      tok = 0;
      ++tile;
    }
    return true;
  }
  // the next visit with a token that sees some of the tile
  __device__ bool next_live(Visit& v) {
    while (next(v))
      if (v.steps > 0) return true;
    return false;
  }
};

// Where the range of every unit begins: a CTA finds its own, over all threads.
template <int kThreadCount>
__device__ void find_begin(const WeightsParams& p, int unit, int* begin) {
  __shared__ long long s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto steps_of = [&](int b) -> long long {
    if (b >= p.requests) return 0;
    const int n = start_of(p, b + 1) - start_of(p, b);
    return n <= 0 ? 0 : static_cast<long long>((len_of(p, b) + kTileRows - 1) / kTileRows) * n;
  };
  if (threadIdx.x == 0) {
    begin[0] = -1;
    begin[1] = begin[2] = begin[4] = begin[5] = 0;
  }
  const long long mine = steps_of(threadIdx.x);  // (of the first kThreadCount requests)
  long long total = 0;
  for (int b = threadIdx.x + kThreadCount; b < p.requests; b += kThreadCount) total += steps_of(b);
  total += mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_warp[warp] = total;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kThreadCount / 32; ++w) total += s_warp[w];
  const long long s0 = total * unit / kUnits, s1 = total * (unit + 1) / kUnits;
  long long carry = 0;
  for (int base = 0; base < p.requests; base += kThreadCount) {
    const int b = base + threadIdx.x;
    const long long own = base == 0 ? mine : steps_of(b);
    long long upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    __syncthreads();  // s_warp has been read
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    long long chunk = 0;
    for (int w = 0; w < kThreadCount / 32; ++w) {
      if (w == warp) upto += carry + chunk;
      chunk += s_warp[w];
    }
    if (s1 > s0 && upto - own <= s0 && s0 < upto) {
      const int n = start_of(p, b + 1) - start_of(p, b);
      const long long at = s0 - (upto - own), left = s1 - s0;
      begin[0] = b;
      begin[1] = static_cast<int>(at / n);
      begin[2] = static_cast<int>(at % n);
      begin[4] = static_cast<int>(static_cast<uint32_t>(left));
      begin[5] = static_cast<int>(left >> 32);
    }
    carry += chunk;
  }
}

// Place i of a visit's block table, asked for ahead, and the pool's page that it
// names; pages outside the pool are reported and read as zeros.
__device__ __forceinline__ int ask_page(const WeightsParams& p, const Visit& v, int i) {
  return i * kPage < v.len ? __ldg(p.table + v.b * p.bt_stride + i) : 0;
}
__device__ __forceinline__ int page_of(const WeightsParams& p, const Visit& v, int i, int page) {
  if (i * kPage >= v.len) return -1;
  if (page >= 0 && page < p.num_pages) return page;
  atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
  return -1;
}

// Two neighbouring E4M3 codes of a word as bf16 times 2^-120: a code beside its
// sign's copies (prmt makes both), four bits higher, without the copies between
// sign and exponent.
template <int kHigh>
__device__ __forceinline__ uint32_t place2(uint32_t codes) {
  uint32_t w;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(w) : "r"(codes), "n"(kHigh ? 0xB3A2 : 0x9180));
  return (w << 4) & 0x87f087f0u;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 8 codes as bf16 times `factor` * 2^-120 (two copies of 2^(e - 7) for a scale of
// 2^(e - 127)): exact (powers of two) while they are in bf16's range.
__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b, uint32_t factor) {
  return make_uint4(mul_bf16x2(place2<0>(a), factor), mul_bf16x2(place2<1>(a), factor), mul_bf16x2(place2<0>(b), factor),
                    mul_bf16x2(place2<1>(b), factor));
}
// The same for any code and scale byte: NaN codes (S.1111.111), and scales of 2^8
// and more, whose 2^(e - 7) bf16 does not hold.
__device__ __noinline__ uint4 widen8_any(uint32_t a, uint32_t b, uint32_t e) {
  const uint32_t s = e == 255 ? 0x7fffu : e ? e << 7 : 0x0040u;
  const uint32_t w[4] = {place2<0>(a), place2<1>(a), place2<0>(b), place2<1>(b)};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool lo = (w[k] & 0x7f0u) == 0x7f0u, hi = (w[k] & 0x7f00000u) == 0x7f00000u;
    o[k] = mul_bf16x2(mul_bf16x2(w[k], 0x7b807b80u), s | s << 16) | (lo ? 0x7fffu : 0u) | (hi ? 0x7fff0000u : 0u);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool kFp8>
__global__ void __launch_bounds__(kFp8 ? kThreadsFp8 : kThreads, 1) __cluster_dims__(2, 1, 1)
mla_attention_weights_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ CUtensorMap tm_q,
                             const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_pe) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t mis = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + mis;
  const uint32_t sbase = smem_u32(smem);
  const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = uniform(cluster_ctarank());
  const int unit = blockIdx.x >> 1;
  int* begin = reinterpret_cast<int*>(smem + kOffWalk);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + kNumBars * 8);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + kNumBars * 8 + 4);

  if (threadIdx.x == 0) {
    for (int g = 0; g < kGroups; ++g) {
      mbar_init(bar(kKF + g), kFp8 ? 9 : 1);  // FP8: rank 0's fill warps and rank 1's relay
      mbar_init(bar(kKE + g), 1);
      mbar_init(bar(kQF + g), 1);
      mbar_init(bar(kQE + g), 1);
      mbar_init(bar(kRaw + g), 1);
      mbar_init(bar(kWide + g), 8);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar(kAF + a), 2);  // both issuers
      mbar_init(bar(kAE + a), 16);
      mbar_init(bar(kDrain + a), 1);
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  grid_launch_dependents();  // (the join waits for this grid)
  grid_dependency_wait();
  find_begin<kFp8 ? kThreadsFp8 : kThreads>(p, unit, begin);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote operation
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  Ctl ctl;
  ctl.abort = abort_flag;
  ctl.n_remote = 1;
  ctl.abort_remote[0] = mapa(smem_u32(const_cast<uint32_t*>(abort_flag)), rank ^ 1u);
  ctl.status = p.status;

  if (threadIdx.x == 0 && rank == 0) {
    p.begins[unit] = make_int4(begin[0], begin[1], begin[2], 0);
    for (int b = unit; b < p.requests; b += kUnits) {
      const int L = p.lens[b];
      bool bad = L < 0 || L > p.max_len;
      if (p.starts) bad = bad || p.starts[b] < 0 || p.starts[b + 1] < p.starts[b] || p.starts[b + 1] > p.tokens;
      if (bad) atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
    }
  }

  // The producers' and issuers' warps walk whole, one lane issues.  Every copy
  // completes on rank 0's barriers, which rank 0 arms with the bytes of both CTAs.
  auto landing_time = [&]() {  // after a failed wait: copies in flight land before the CTA goes away
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kDrainNs / 8) {
    }
  };
  if (warp == 0) {
    // ================================================= rows, by TMA
    // FP8: the codes of a group's two chunks go to the second one's slot, for this
    // CTA's fill warps to widen in place; the position dims to theirs at once.
    const uint32_t rk = mapa(bar(kKF), 0);
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      if (kFp8) tma_prefetch_desc(&tm_pe);
    }
    Walk walk(p, begin);
    Visit v, after;
    // (a lane a page, a visit ahead)
    auto place = [&](const Visit& s) { return s.tile * 4 + static_cast<int>(rank) * 2 + (lane & 1); };
    bool ok = true, more = walk.next_live(v);
    int asked = more ? ask_page(p, v, place(v)) : 0;
    for (uint32_t nk = 0; ok && more; ++nk) {
      const int page = page_of(p, v, place(v), asked);
      if ((more = walk.next_live(after))) asked = ask_page(p, after, place(after));
      v = after;
      int y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int mine = __shfl_sync(0xffffffffu, page, e);
        y[e] = (mine >= 0 ? mine : static_cast<int>(p.num_pages)) * kPage;
      }
      for (int i = 0; i < kGroups; ++i) {
        const int g = group_turn(i);
        if (nk > 0 && !(ok = warp_wait_uniform<true>(bar(kKE + g), (nk - 1) & 1, ctl))) break;
        if (lane == 0) {
          const int c0 = group_begin<kFp8>(g), c1 = group_begin<kFp8>(g + 1);
          if (kFp8) {
            mbar_arrive_expect_tx_relaxed(bar(kRaw + g), (c1 - c0 - 1) * kKChunk);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              tma_load_2d(sbase + (c0 + 1) * kKChunk + e * (kKChunk / 2), &tm_k, 64 * c0, y[e], bar(kRaw + g));
              if (c1 == kNumChunks)
                tma_load_2d(sbase + 8 * kKChunk + e * (kKChunk / 2), &tm_pe, kPeAt, y[e], bar(kRaw + g));
            }
            continue;
          }
          if (rank == 0) mbar_arrive_expect_tx_relaxed(bar(kKF + g), (c1 - c0) * 2 * kKChunk);
          for (int c = c0; c < c1; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              tma_load_2d_pair(sbase + c * kKChunk + e * (kKChunk / 2), &tm_k, 64 * c, y[e], rk + 8u * g);
        }
      }
    }
    if (!ok && lane == 0) landing_time();
    __syncwarp();
  } else if (warp == 2) {
    // ================================================= queries, by TMA
    const uint32_t rq = mapa(bar(kQF), 0);
    if (lane == 0) tma_prefetch_desc(&tm_q);
    Walk walk(p, begin);
    Visit v;
    uint32_t nq = 0;
    int last_q = -1;
    bool ok = true;
    while (ok && walk.next_live(v)) {
      for (int i = v.steps, q = v.q0; ok && i > 0; --i, q += v.way) {
        if (q == last_q) continue;
        last_q = q;
        for (int j = 0; j < kGroups; ++j) {
          const int g = group_turn(j);
          if (nq > 0 && !(ok = warp_wait_uniform<true>(bar(kQE + g), (nq - 1) & 1, ctl))) break;
          if (lane == 0) {
            const int c0 = group_begin<kFp8>(g), c1 = group_begin<kFp8>(g + 1);
            if (rank == 0) mbar_arrive_expect_tx_relaxed(bar(kQF + g), (c1 - c0) * 2 * kQChunk);
            for (int c = c0; c < c1; ++c)
              tma_load_2d_pair(sbase + kOffQ + c * kQChunk, &tm_q, 64 * c, last_q * kHeads + static_cast<int>(rank) * 64,
                               rq + 8u * g);
          }
        }
        ++nq;
      }
    }
    if (!ok && lane == 0) landing_time();
    __syncwarp();
  } else if ((warp == 1 || warp == 3) && rank == 0) {
    // ================================================= MMA issue: warp 1 the first accumulator, warp 3 the second
    const uint32_t leader = lane == 0 ? 1u : 0u;
    const int which = warp >> 1;
    const uint64_t kd = smem_desc(sbase, 16u, 1024u), qd = smem_desc(sbase + kOffQ, 16u, 1024u);
    Walk walk(p, begin);
    Visit v, after;
    uint32_t nk = 0, nq = 0, step = 0;
    int last_q = -1;
    bool ok = true, more = walk.next_live(v);
    auto issue = [&](auto first, auto end) {  // groups [first, end) of every step
      while (ok && more) {
        more = walk.next_live(after);
        // (values that the compiler knows to be a warp's keep the operations' descriptors in
        // uniform registers: 64 tokens x 65536 FP8 337 us against 369)
        const int steps = uniform(v.steps), way = uniform(v.way), then = uniform(more ? after.q0 : -1);
        int q = uniform(v.q0);
        for (int i = steps; ok && i > 0; --i, q += way, ++step) {
          const bool new_k = i == steps, new_q = q != last_q, last = i == 1;
          const bool q_goes = !last || (then >= 0 && then != q);
          const uint32_t buf = step & 1, d = tmem + 256u * buf + kHeads * which;
          if (step >= 2) ok = warp_wait_uniform<true>(bar(kAE + buf), ((step >> 1) - 1) & 1, ctl);
          if (new_q) ++nq;
          last_q = q;
#pragma unroll
          for (int g = first; g < end; ++g) {
            if (new_k) ok = ok && warp_wait_uniform<true>(bar(kKF + g), nk & 1, ctl);
            if (new_q) ok = ok && warp_wait_uniform<true>(bar(kQF + g), (nq - 1) & 1, ctl);
            if (!ok) break;
            tc_fence_after();
            // (rolled: 20 warps of six kinds share the instruction cache; unrolled 64 tokens x
            // 65536 FP8 392 us against 345, bf16 356 / 344)
#pragma unroll 1
            for (int c = group_begin<kFp8>(g); c < group_begin<kFp8>(g + 1); ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_pair_ss_if(leader, d, kd + static_cast<uint64_t>((c * kKChunk + 32 * kk) >> 4),
                                qd + static_cast<uint64_t>((c * kQChunk + 32 * kk) >> 4), kIdesc,
                                (c != 0 && c != group_begin<kFp8>(kGroups / 2)) || kk > 0 ? 1u : 0u);
            if (last) umma_commit_pair_if(leader, bar(kKE + g), 3);
            if (q_goes) umma_commit_pair_if(leader, bar(kQE + g), 3);
          }
          if (!ok) break;
          umma_commit_pair_if(leader, bar(kAF + buf), 3);
        }
        ++nk;
        v = after;
      }
    };
    if (which == 0)
      issue(std::integral_constant<int, 0>(), std::integral_constant<int, kGroups / 2>());
    else
      issue(std::integral_constant<int, kGroups / 2>(), std::integral_constant<int, kGroups>());
    umma_commit_pair_if(leader, bar(kDrain + which), 1);  // arrives once every MMA issued above has completed
    drain_bar(bar(kDrain + which), 0u);
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // Rank 1 has nothing to issue.  With an FP8 cache these threads relay its fill
    // warps' arrivals to rank 0, whose MMAs read this CTA's rows too: the warps
    // release to their own CTA, a thread without stores of its own to the cluster
    // (a release to the cluster by each of them waits for its earlier stores).
    if (kFp8 && lane == 0) {
      const uint32_t rk = mapa(bar(kKF), 0);
      Walk walk(p, begin);
      Visit v;
      bool ok = true;
      for (uint32_t nk = 0; ok && walk.next_live(v); ++nk)
        for (int i = 0; ok && i < kGroups / 2; ++i) {
          const int g = kGroups / 2 * (warp >> 1) + i;
          if ((ok = wait(bar(kWide + g), nk & 1, ctl))) mbar_arrive_remote(rk + 8u * g);
        }
    }
    __syncwarp();
  } else if (warp >= kEpiWarp && warp < kEpiWarp + 8) {
    // ================================================= sums over heads and tokens
    // Warp (quarter, half): rows 32 quarter .. of the CTA's 128, one a lane, heads 64 half .. +63.
    const int quarter = warp & 3, half = (warp - kEpiWarp) >> 2;
    const int r = 32 * quarter + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 64u * half;
    const uint32_t s_lse = sbase + kOffLse + 256u * (warp - kEpiWarp);  // this warp's own
    float2* my_lse = reinterpret_cast<float2*>(smem + kOffLse + 256 * (warp - kEpiWarp)) + lane;
    float* s_half = reinterpret_cast<float*>(smem + kOffHalf);
    const uint32_t racc = mapa(bar(kAE), 0);
    Walk walk(p, begin);
    Visit v, after;
    uint32_t step = 0;
    // a visit's older weight and its first token's lse are asked for a visit ahead
    float old = 0.f, next_old = 0.f;
    float2 l2 = make_float2(0.f, 0.f), next_l2 = l2;
    auto lse_of = [&](int q) {
      return reinterpret_cast<const float2*>(p.lse + static_cast<long long>(q) * kHeads + 64 * half) + lane;
    };
    auto row_of = [&](const Visit& s) { return s.tile * kTileRows + static_cast<int>(rank) * kRows + r; };
    auto ask = [&](const Visit& s, float& o, float2& l) {
      if (half == 0 && s.t0 == 0 && row_of(s) < s.len && p.decay != 0.f) o = p.weights[s.b * p.w_stride + row_of(s)];
      if (s.steps > 0) l = __ldg(lse_of(s.q0));
    };
    bool more = walk.next(v);
    if (more) ask(v, old, l2);
    for (uint32_t visit = 0; more; ++visit) {
      more = walk.next(after);
      if (more) ask(after, next_old, next_l2);
      const int pos = row_of(v);
      float sum = 0.f;
      bool ok = true;
      for (int i = v.steps, q = v.q0; i > 0; --i, q += v.way, ++step) {
        const uint32_t buf = step & 1;
        // a head without a result (-inf) weighs nothing: 2^(s - inf), and where there are
        // such heads their scores, which may be no numbers, are left out
        auto log2_of = [](float x) { return x == -INFINITY ? -INFINITY : -x * kLog2e; };
        const bool empty = __any_sync(0xffffffffu, l2.x == -INFINITY || l2.y == -INFINITY);
        *my_lse = make_float2(log2_of(l2.x), log2_of(l2.y));
        if (i > 1) l2 = __ldg(lse_of(q + v.way));
        __syncwarp();
        ok = warp_wait_uniform<true>(bar(kAF + buf), (step >> 1) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        float e[4] = {0.f, 0.f, 0.f, 0.f};
        constexpr int kCols = kFp8 ? 16 : 32;  // (registers: 20 warps have 96 a thread)
#pragma unroll 1
        for (int h = 0; h < 64 / kCols; ++h) {
          uint32_t x[2][kCols];
          for (int a = 0; a < 2; ++a) {
            const uint32_t at = tl + 256u * buf + kHeads * a + kCols * h;
            if constexpr (kFp8)
              tmem_ld16(at, x[a]);
            else
              tmem_ld32(at, x[a]);
          }
          tmem_wait_ld();
          if (h == 64 / kCols - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(racc + 8u * buf);
          }
          auto add = [&](auto some) {
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
              const float4 l = ld_shared_v4f(s_lse + 4u * (kCols * h + c));
              const float bias[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float w =
                    ex2_approx(fmaf(__uint_as_float(x[0][c + i]) + __uint_as_float(x[1][c + i]), p.scale_log2, bias[i]));
                e[i] += some && bias[i] == -INFINITY ? 0.f : w;
              }
            }
          };
          if (empty)
            add(std::true_type());
          else
            add(std::false_type());
        }
        __syncwarp();  // the warp's lse has been read
        if (pos < limit(v, q, p.causal)) sum += (e[0] + e[1]) + (e[2] + e[3]);  // hidden rows may hold anything
      }
      // the two halves of the heads meet; the buffer of the visit before the last is free again
      if (half == 1) s_half[(visit & 1) * kRows + r] = sum;
      if (!named_bar_all(1 + quarter, 64, ok)) break;
      if (half == 0) {
        sum += s_half[(visit & 1) * kRows + r];
        if (v.t0 != 0)
          p.parts[unit * kTileRows + static_cast<int>(rank) * kRows + r] = sum;
        else if (pos < v.len)
          p.out[v.b * p.out_stride + pos] = (p.decay != 0.f ? p.decay * old : 0.f) + sum;
      }
      v = after;
      old = next_old;
      l2 = next_l2;
    }
  } else if (kFp8 && warp >= kFillWarp) {
    // ================================================= FP8 rows: codes widened in place
    // Warp w has rows 16 w .. +15 (all of one page).  A row's codes of two chunks
    // lie in the 128 bytes that its second chunk's dims take, so that a warp that
    // holds its rows' codes waits for no other before it writes.  Four lanes a row
    // take 16 bytes each: odd rows the other chunk's first, so that eight lanes
    // meet all banks, reading and writing.  (Boxes of one chunk's codes, 64 bytes a
    // row: 33 x 2 x 2560 42.7 us, 64 x 1 x 8192 128; rows read from global memory
    // by these warps, three turns of loads in flight: 64 x 2 x 8192 245, bound by
    // their latency, where the TMA holds a whole tile in flight.)
    const int w = warp - kFillWarp;
    Walk walk(p, begin);
    Visit v;
    uint32_t nk = 0;
    const int row0 = lane >> 2, unit16 = lane & 3;
    auto place = [&](const Visit& s) { return s.tile * 4 + static_cast<int>(rank) * 2 + (w >> 2); };
    // the scale bytes of the lane's two rows of a visit
    auto scales_of = [&](const Visit& s, int asked) {
      const int page = page_of(p, s, place(s), asked);
      if (page < 0) return make_uint2(0u, 0u);
      const uint8_t* row = p.kv + (static_cast<long long>(page) * kPage + 16 * (w & 3) + row0) * MLA_FP8_ROW_BYTES + 512;
      return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(row)),
                        __ldg(reinterpret_cast<const uint32_t*>(row + 8 * MLA_FP8_ROW_BYTES)));
    };
    // scales are asked for a visit ahead, pages two
    bool ok = true, more = walk.next_live(v);
    uint2 scales = more ? scales_of(v, ask_page(p, v, place(v))) : make_uint2(0u, 0u);
    bool next = more && walk.next_live(v);
    int asked = next ? ask_page(p, v, place(v)) : 0;
    const uint32_t rows = sbase + (16 * w + row0) * 128, sw = row0;  // (row & 7, for both of the rows)
    const uint32_t at0 = ((2u * unit16) ^ sw) << 4, at1 = ((2u * unit16 + 1u) ^ sw) << 4;
    while (ok && more) {
      const uint2 next_scales = next ? scales_of(v, asked) : make_uint2(0u, 0u);
      more = next;
      if (next && (next = walk.next_live(v))) asked = ask_page(p, v, place(v));
      // no byte above 134
      const bool small = __vcmpgtu4(scales.x, 0x86868686u) == 0 && __vcmpgtu4(scales.y, 0x86868686u) == 0;
#pragma unroll 1
      for (int i = 0; i < kGroups; ++i) {
        const int g = group_turn(i);
        if (!(ok = warp_wait_uniform(bar(kRaw + g), nk & 1, ctl))) break;
        const uint32_t pair = rows + 2 * g * kKChunk;
        uint4 x[2][2];
        uint32_t nan = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint4 v4 = x[t][r] = ld_shared_v4u(pair + kKChunk + 1024u * r + 64u * (t ^ (row0 & 1)) + 16u * unit16);
            nan |= ((v4.x & 0x7f7f7f7fu) + 0x01010101u) | ((v4.y & 0x7f7f7f7fu) + 0x01010101u) |
                   ((v4.z & 0x7f7f7f7fu) + 0x01010101u) | ((v4.w & 0x7f7f7f7fu) + 0x01010101u);
          }
        __syncwarp();  // the warp holds its codes, and writes over them
        // (one question for a whole group: asked for every 8 codes, it took as long as they)
        const bool plain = (nan & 0x80808080u) == 0 && small;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t dst = pair + kKChunk * (t ^ (row0 & 1)) + 1024u * r;
            const uint32_t e = ((r ? scales.y : scales.x) >> (8 * g)) & 255u;
            const uint4 v4 = x[t][r];
            uint4 o0, o1;
            if (plain) {
              const uint32_t f = (e + 120) << 7, factor = f | f << 16;
              o0 = widen8(v4.x, v4.y, factor);
              o1 = widen8(v4.z, v4.w, factor);
            } else {
              o0 = widen8_any(v4.x, v4.y, e);
              o1 = widen8_any(v4.z, v4.w, e);
            }
            st_shared_v4(dst + at0, o0.x, o0.y, o0.z, o0.w);
            st_shared_v4(dst + at1, o1.x, o1.y, o1.z, o1.w);
          }
        fence_proxy_async_smem();  // generic writes, read next by the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(bar((rank == 0 ? kKF : kWide) + g));
      }
      scales = next_scales;
      ++nk;
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA touches another's shared memory after this
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Adds the parts of tiles that several units share, in the line's order: block u
// does so for the tile in whose tokens unit u begins, if no unit before it does.
// The parts are added before they meet the older weight, which may be far larger
// and would be rounded at each of them.
__global__ void __launch_bounds__(kTileRows) mla_attention_weights_join_kernel(const __grid_constant__ WeightsParams p) {
  grid_dependency_wait();
  const int u = blockIdx.x;
  const int4 mine = p.begins[u];
  if (mine.x < 0 || mine.z == 0) return;
  auto same = [&](const int4& o) { return o.x == mine.x && o.y == mine.y && o.z > 0; };
  for (int v = u - 1; v >= 0; --v) {
    const int4 o = p.begins[v];
    if (o.x < 0) continue;
    if (same(o)) return;
    break;
  }
  const int pos = mine.y * kTileRows + static_cast<int>(threadIdx.x);
  if (pos >= len_of(p, mine.x)) return;
  float sum = p.parts[u * kTileRows + threadIdx.x];
  for (int v = u + 1; v < kUnits; ++v) {
    const int4 o = p.begins[v];
    if (o.x < 0) continue;
    if (!same(o)) break;
    sum += p.parts[v * kTileRows + threadIdx.x];
  }
  p.out[mine.x * p.out_stride + pos] += sum;
}

// Device check and kernel attributes, once per device.
int weights_device_ready() {
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
    state[dev] = MLA_OK;
    for (auto* kernel : {mla_attention_weights_kernel<false>, mla_attention_weights_kernel<true>})
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
        state[dev] = MLA_ERR_CUDA;
    cudaGetLastError();
  });
  return state[dev];
}

// The codes of an FP8 cache's rows as boxes of two chunks x 64 rows, as they are.
bool encode_codes(CUtensorMap* m, const void* base, uint64_t rows) {
  EncodeTiledFn fn = encode_tiled();
  const cuuint64_t size[2] = {512, rows}, strides[1] = {MLA_FP8_ROW_BYTES};
  const cuuint32_t box[2] = {128, 64}, one[2] = {1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), size, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Their position dims as boxes of 64 dims x 64 rows.
bool encode_position(CUtensorMap* m, const void* base, uint64_t rows) {
  const cuuint64_t size[2] = {MLA_FP8_ROW_BYTES / 2, rows}, strides[1] = {MLA_FP8_ROW_BYTES};
  const cuuint32_t box[2] = {64, 64};
  return encode(m, false, 2, base, size, strides, box);
}

// Rows of 576 dims as boxes of 64 dims x 64 rows.
bool encode_rows(CUtensorMap* m, const void* base, uint64_t rows) {
  const cuuint64_t size[2] = {kDqk, rows}, strides[1] = {kDqk * 2};
  const cuuint32_t box[2] = {64, 64};
  return encode(m, false, 2, base, size, strides, box);
}

int check_sizes(int num_tokens, int num_requests, int max_len, unsigned flags) {
  if (num_tokens < 0 || num_requests < 1 || max_len < 1) return MLA_ERR_INVALID_ARG;
  if (flags & ~static_cast<unsigned>(MLA_FLAG_CAUSAL | MLA_FLAG_KV_FP8)) return MLA_ERR_INVALID_ARG;
  if ((static_cast<int64_t>(num_tokens) + 1) * kHeads > INT32_MAX || max_len > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

constexpr size_t kBeginBytes = (kUnits * sizeof(int4) + 255) / 256 * 256;
constexpr size_t kWorkspace = kBeginBytes + kUnits * kTileRows * sizeof(float);

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_attention_weights_workspace_size(int num_tokens, int num_requests, int max_len, unsigned flags, int* err) {
  const int rc = check_sizes(num_tokens, num_requests, max_len, flags);
  if (err) *err = rc;
  return rc == MLA_OK ? kWorkspace : 0;
}

int mla_attention_weights(const void* q, const float* lse, const void* kv_cache, int64_t num_pages,
                          const int32_t* block_table, int64_t bt_stride, const int32_t* cache_lens, int max_len,
                          const int32_t* token_starts, int num_requests, int num_tokens, int num_heads,
                          float softmax_scale, float decay, const float* weights, int64_t weights_stride,
                          unsigned flags, void* workspace, size_t ws_bytes, float* out, int64_t out_stride,
                          int* status, mla_stream_t stream) {
  if (!q || !lse || !kv_cache || !block_table || !cache_lens || !out || !status || !workspace) return MLA_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(kv_cache, 16) || !al(lse, 16) || !al(block_table, 4) || !al(cache_lens, 4) || !al(token_starts, 4) ||
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
  if (decay != 0.f && (out != weights || (num_requests > 1 && out_stride != weights_stride)) &&
      share(out, out_stride, max_len, weights, weights_stride, max_len, num_requests))
    return MLA_ERR_INVALID_ARG;
  if (num_pages > (INT32_MAX / kPage) - 1) return MLA_ERR_UNSUPPORTED;
  if (ws_bytes < kWorkspace) return MLA_ERR_WORKSPACE;
  if ((rc = weights_device_ready()) != MLA_OK) return rc;
  if (num_tokens == 0) return MLA_OK;
  const bool fp8 = (flags & MLA_FLAG_KV_FP8) != 0;
  WeightsParams p;
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.num_pages = num_pages;
  p.lse = lse;
  p.table = block_table;
  p.bt_stride = bt_stride;
  p.lens = cache_lens;
  p.max_len = max_len;
  p.starts = token_starts;
  p.requests = num_requests;
  p.tokens = num_tokens;
  p.causal = (flags & MLA_FLAG_CAUSAL) ? 1 : 0;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  p.decay = decay;
  p.weights = weights;
  p.w_stride = weights_stride;
  p.out = out;
  p.out_stride = out_stride;
  p.begins = static_cast<int4*>(workspace);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kBeginBytes);
  p.status = status;
  CUtensorMap tm_q, tm_k, tm_pe = {};
  const uint64_t rows = static_cast<uint64_t>(num_pages) * kPage;
  if (!encode_rows(&tm_q, q, static_cast<uint64_t>(num_tokens) * kHeads)) return MLA_ERR_CUDA;
  if (fp8 ? !encode_codes(&tm_k, kv_cache, rows) || !encode_position(&tm_pe, kv_cache, rows)
          : !encode_rows(&tm_k, kv_cache, rows))
    return MLA_ERR_CUDA;
  rc = fp8 ? launch_dependent(mla_attention_weights_kernel<true>, dim3(2 * kUnits), dim3(kThreadsFp8), kSmem, 1, stream, p,
                              tm_q, tm_k, tm_pe)
           : launch_dependent(mla_attention_weights_kernel<false>, dim3(2 * kUnits), dim3(kThreads), kSmem, 1, stream, p,
                              tm_q, tm_k, tm_pe);
  if (rc != MLA_OK) return rc;
  if (!token_starts && num_tokens == num_requests) return MLA_OK;  // one step a tile: no tile is shared
  return launch_dependent(mla_attention_weights_join_kernel, dim3(kUnits), dim3(kTileRows), 0, 1, stream, p);
}

}  // extern "C"
