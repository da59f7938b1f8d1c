// prefix_expand.cu — per-head keys and values of a shared prefix, from its
// cached latents, with the C ABI (include/mla_prefix.h).
//
// K[h] = L W_UK[h] and V[h] = L W_UV[h] for the prefix's latents L [P, 512]:
// one product of [P, 512] by [512, heads * 256], bound by the tensor cores
// (4 * 512 * 128 operations a (row, head) for 512 bytes written).
//
// A pair of SMs computes 256 rows of one head's keys and values at a time
// (tcgen05.mma.cta_group::2, M256 N256 K16): each CTA holds 128 rows of L and
// one of the weights (rank 0 W_UK, rank 1 W_UV), and receives both products of
// its rows, 128 key and 128 value columns, in its tensor memory.  The weights
// stay in shared memory (128 KiB a CTA) over all row tiles of a head and are
// replaced stage by stage under the last one; the latents stream through a
// ring of 6 chunks of 64 dims, read from the cache's pages by TMA (they lie
// in L2: every pair reads the same rows).  Two accumulators, so that a tile is
// drained under the next one's products.  (row tile, head) items form one
// line, head by head, cut into equal ranges, one per pair.
//
// Measured: 8192 rows x 128 heads 163 to 167 us (1.67 PFLOP/s, 3.25 TB/s written;
// called for seconds on end 187 to 194, as the power limit, 1,378 W, then holds the clock
// at 1.5 GHz).  The rest was measured with two issuing warps, 157 to 163 us.
// Without its stores the kernel took 133 us, with half of its products 156: the
// results' way out (shuffles and stores share the data
// path that the MMAs read their operands on) and the products get in each
// other's way.  Streaming stores, 64 bytes a row over four lanes, are the best of
// those tried: not streaming 165 to 170, 128 bytes over eight lanes 161, 32-byte
// stores 171, through shared memory and TMA more.  Not kept either: the weights
// as A operand in tensor memory (dims come out as rows and have to be transposed
// on their way: 197 us with 4-byte stores, 253 with shuffles, 263 through shared
// memory); keys and values as two N = 128 products that share A (184).
//
//   warp 0     TMA: latents and weights
//   warp 1     MMA issue (rank 0, for both CTAs)
//   warps 2-9  drain: tensor memory -> bf16 / fp16 -> global memory, 64 columns
//              at a time; keys and values by four warps each
//   warp 10    copies the RoPE dims and checks the block table
//
//   warps 12-19  (FP8 cache only) widen the latents: TMA brings a chunk's codes
//              into the upper half of its slot, bf16 replaces them
//   warps 1, 11  of rank 1 (FP8 cache only) pass its converters' arrivals on to
//              rank 0's warp 1
//
// FP8 rows are widened on their way into shared memory (exactly: 4 significant
// bits and a power of two), by every pair for every head, so that a prefix needs
// one launch and no workspace.  Against a kernel that widens the prefix once, in
// a workspace, for the bf16 product: 100 rows x 16 heads 8.4 / 9.0 us, 1000 x 16
// 10.2 / 10.9 (and 9 us less of the host's time), 4000 x 64 65 / 52.3, 8192 x 128
// 238 / 165: there the widening (890 cycles a chunk) and the way to the other
// SM's issuer hold up the products' 690.  Not kept (measured while rank 1's
// converters released to their own CTA only, which orders nothing for an issuer
// in the other; 205 us so): four warps 274 us, six or three warps with a chunk
// each 277 and 375, the next chunk's codes read ahead 322, integer widening 219.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "mla_prefix.h"
#include "prefix_common.cuh"

namespace mla {
namespace {

using namespace prefix;

constexpr int kLatent = 512;
constexpr int kRope = 64;
constexpr int kHeadDim = 128;
constexpr int kFp8Row = MLA_FP8_ROW_BYTES;

constexpr int kRows = 128;                   // rows of a CTA's tile
constexpr int kStages = kLatent / 64;        // 64 latent dims each
constexpr int kChunk = 16384;                // 128 rows x 64 dims, or 64 dims x 128 columns of a weight
constexpr int kSlots = 6;
constexpr int kOffW = 0;
constexpr int kOffRing = kStages * kChunk;                // 128 KiB
constexpr int kOffBar = kOffRing + kSlots * kChunk;       // 224 KiB
constexpr int kNumBars = 4 * kSlots + 2 * kStages + 4 + 1;
constexpr int kSlack = 1024;                 // re-aligned to 1024 B (128-byte swizzle atoms)
constexpr int kSmem = kOffBar + kNumBars * 8 + 16 + kSlack;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kThreads = 352;
constexpr int kRelayWarp = 11;               // further warps, FP8 cache only: the relay of odd chunks,
constexpr int kConverterWarp = 12;           // and two groups of four
constexpr int kConverters = 8;
static_assert(kSlots % 2 == 0, "a slot's chunks are one group's");
constexpr int kThreadsFp8 = 32 * (kConverterWarp + kConverters);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdesc = idesc_bf16(256, 256, 1);

struct ExpandParams {
  const uint8_t* cache;      // the pool (RoPE dims, FP8 rows)
  int row_bytes, rope_byte;  // of a pool row
  long long num_pages;
  const int* block_table;
  int prefix_len, num_heads;
  uint16_t* k_nope;
  uint16_t* v;
  long long head_rows;
  uint16_t* k_pe;
  int* status;
};

template <bool kFp8>
__global__ void __launch_bounds__(kFp8 ? kThreadsFp8 : kThreads, 1) __cluster_dims__(2, 1, 1)
mla_prefix_expand_kernel(const __grid_constant__ ExpandParams p, const __grid_constant__ CUtensorMap tm_lat,
                         const __grid_constant__ CUtensorMap tm_wk, const __grid_constant__ CUtensorMap tm_wv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t mis = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + mis;
  const uint32_t sbase = smem_u32(smem);
  const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = uniform(cluster_ctarank());
  const int tiles = (p.prefix_len + 2 * kRows - 1) / (2 * kRows);
  const long long items = static_cast<long long>(tiles) * p.num_heads;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const long long i0 = items * pair / pairs, i1 = items * (pair + 1) / pairs;
  const int n = static_cast<int>(i1 - i0);
  const int h0 = static_cast<int>(i0 / tiles), m0 = static_cast<int>(i0 % tiles);

  const uint32_t bar0 = sbase + kOffBar;
  auto a_full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto a_empty = [&](uint32_t s) { return bar0 + 8u * (kSlots + s); };
  auto w_full = [&](uint32_t s) { return bar0 + 8u * (2 * kSlots + s); };
  auto w_empty = [&](uint32_t s) { return bar0 + 8u * (2 * kSlots + kStages + s); };
  auto acc_full = [&](uint32_t s) { return bar0 + 8u * (2 * kSlots + 2 * kStages + s); };
  auto acc_empty = [&](uint32_t s) { return bar0 + 8u * (2 * kSlots + 2 * kStages + 2 + s); };
  auto raw_full = [&](uint32_t s) { return bar0 + 8u * (2 * kSlots + 2 * kStages + 4 + s); };  // codes (FP8 cache)
  auto widened = [&](uint32_t s) { return bar0 + 8u * (3 * kSlots + 2 * kStages + 4 + s); };  // bf16 (FP8 cache, rank 1)
  const uint32_t bar_drain = bar0 + 8u * (kNumBars - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + kNumBars * 8);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + kNumBars * 8 + 4);

  if (threadIdx.x == 0) {
    // each once: to initialise a barrier that is one already is undefined
    for (uint32_t s = 0; s < kSlots; ++s) {
      mbar_init(a_full(s), kFp8 ? kConverters / 2 + 1 : 1);  // FP8: rank 0's group, and rank 1's relay
      mbar_init(a_empty(s), 1);
      mbar_init(raw_full(s), 1);
      mbar_init(widened(s), kConverters / 2);
    }
    for (uint32_t k = 0; k < kStages; ++k) {
      mbar_init(w_full(k), 1);
      mbar_init(w_empty(k), 1);
    }
    for (uint32_t s = 0; s < 2; ++s) {
      mbar_init(acc_full(s), 1);
      mbar_init(acc_empty(s), 16);  // the drain warps of both CTAs
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
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

  grid_dependency_wait();

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_lat);
      tma_prefetch_desc(rank == 0 ? &tm_wk : &tm_wv);
      const CUtensorMap* tw = rank == 0 ? &tm_wk : &tm_wv;
      const int pages = (p.prefix_len + kPage - 1) / kPage;
      // Every copy completes on rank 0's barriers, which rank 0 arms with the bytes of both CTAs.
      const uint32_t ra = mapa(a_full(0), 0), rw = mapa(w_full(0), 0);
      uint32_t chunk = 0, heads = 0;
      int h = h0, m = m0;
      bool ok = true;
      for (int i = 0; ok && i < n; ++i) {
        // the tile's two pages; a page that is not there reads as zeros
        int z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pg = (m * 2 + static_cast<int>(rank)) * 2 + e;
          const int id = pg < pages ? p.block_table[pg] : -1;
          z[e] = id >= 0 && id < p.num_pages ? id : static_cast<int>(p.num_pages);
        }
        const bool new_head = i == 0 || m == 0;
        for (uint32_t k = 0; ok && k < kStages; ++k, ++chunk) {
          if (new_head) {
            if (heads > 0 && !(ok = wait<true>(w_empty(k), (heads - 1) & 1, ctl))) break;
            if (rank == 0) mbar_arrive_expect_tx(w_full(k), 2 * kChunk);
            const uint32_t dst = sbase + kOffW + k * kChunk;
            tma_load_2d_pair(dst, tw, 0, h * kLatent + 64 * k, rw + 8u * k);
            tma_load_2d_pair(dst + kChunk / 2, tw, 64, h * kLatent + 64 * k, rw + 8u * k);
          }
          const uint32_t s = chunk % kSlots;
          if (chunk >= kSlots && !(ok = wait<true>(a_empty(s), ((chunk / kSlots) - 1) & 1, ctl))) break;
          const uint32_t dst = sbase + kOffRing + s * kChunk;
          if (kFp8) {  // codes, for this CTA's own converters
            mbar_arrive_expect_tx(raw_full(s), kChunk / 2);
            tma_load_3d(dst + kChunk / 2, &tm_lat, 64 * k, 0, z[0], raw_full(s));
            tma_load_3d(dst + kChunk / 2 + kChunk / 4, &tm_lat, 64 * k, 0, z[1], raw_full(s));
            continue;
          }
          if (rank == 0) mbar_arrive_expect_tx(a_full(s), 2 * kChunk);
          tma_load_3d_pair(dst, &tm_lat, 64 * k, 0, z[0], ra + 8u * s);
          tma_load_3d_pair(dst + kChunk / 2, &tm_lat, 64 * k, 0, z[1], ra + 8u * s);
        }
        if (new_head) ++heads;
        if (++m == tiles) {
          m = 0;
          ++h;
        }
      }
      grid_launch_dependents();
      if (!ok) {  // let copies in flight land before the CTA goes away
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kDrainNs / 8) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // One thread issues all products, in the order of their sum.  Two warps with
    // a stage each in turns fill the gaps in which a commit and a wait let the
    // tensor core run dry (8192 x 128 in 160 us instead of 165), but a token that
    // passes between them does not keep their MMAs in order: once in a thousand
    // calls a value's last bit differed.  The whole warp runs, one lane issues
    // (uniform operands).  Commits or waits between a stage's MMAs: 171 to 185.
    const uint32_t leader = lane == 0 ? 1u : 0u;
    const uint64_t wd = smem_desc(sbase + kOffW, kChunk / 2, 1024u);   // MN-major: 64-column halves kChunk / 2 apart
    const uint64_t ad = smem_desc(sbase + kOffRing, 16u, 1024u);
    uint32_t heads = 0, chunk = 0;
    int m = m0;
    bool ok = true;
    for (int i = 0; ok && i < n; ++i) {
      const uint32_t buf = i & 1, d = tmem + 256u * buf;
      const bool new_head = i == 0 || m == 0, last = m == tiles - 1;
      if (i >= 2) ok = warp_wait_uniform<true>(acc_empty(buf), ((i >> 1) - 1) & 1, ctl);
#pragma unroll
      for (uint32_t k = 0; k < kStages; ++k, ++chunk) {
        const uint32_t s = chunk % kSlots;
        if (new_head) ok = ok && warp_wait_uniform<true>(w_full(k), heads & 1, ctl);
        ok = ok && warp_wait_uniform<true>(a_full(s), (chunk / kSlots) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_pair_ss_if(leader, d, ad + static_cast<uint64_t>((s * kChunk + 32 * kk) >> 4),
                          wd + static_cast<uint64_t>((k * kChunk + 2048 * kk) >> 4), kIdesc,
                          (k | kk) != 0 ? 1u : 0u);
        umma_commit_pair_if(leader, a_empty(s), 3);
        if (last) umma_commit_pair_if(leader, w_empty(k), 3);
      }
      if (!ok) break;
      umma_commit_pair_if(leader, acc_full(buf), 3);
      if (new_head) ++heads;
      m = last ? 0 : m + 1;
    }
    umma_commit_pair_if(leader, bar_drain, 1);  // arrives once every MMA issued above has completed
    drain_bar(bar_drain, 0u);
    __syncwarp();
  } else if (warp == 1 || warp == kRelayWarp) {
    // Rank 1 has nothing to issue.  With an FP8 cache two of its warps relay its
    // converters' arrivals to rank 0, whose MMAs read this CTA's rows too.  The
    // converters release to their own CTA; a thread without stores of its own,
    // which has acquired their rows, releases to the cluster.  That is slow beside
    // the drain's stores (a third relay gains 2 %, but then no warp is left for
    // rank 1's RoPE rows; the converters releasing to the cluster themselves take
    // 8192 x 128 from 236 us to 337).
    if (kFp8 && rank == 1 && lane == 0) {
      const uint32_t ra = mapa(a_full(0), 0), chunks = static_cast<uint32_t>(n) * kStages;
      for (uint32_t chunk = warp == 1 ? 0u : 1u; chunk < chunks; chunk += 2) {
        const uint32_t s = chunk % kSlots;
        if (!wait(widened(s), (chunk / kSlots) & 1, ctl)) break;
        mbar_arrive_remote(ra + 8u * s);
      }
    }
    __syncwarp();
  } else if (warp < 10) {
    const int q = warp & 3;  // tensor-memory lanes 32 q .. +31: those rows of the tile
    const bool keys = warp < 6;
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + (keys ? 0u : 128u);
    const uint32_t racc = mapa(acc_empty(0), 0);
    uint16_t* out = keys ? p.k_nope : p.v;
    const uint32_t one = keys ? 0x00800080u : 0x04000400u;  // one in the exponents of a bf16 or an fp16 pair
    const int quad = lane & 3;
    int h = h0, m = m0;
    for (int i = 0; i < n; ++i) {
      const uint32_t buf = i & 1;
      const int row0 = (m * 2 + static_cast<int>(rank)) * kRows + 32 * q;
      if (!__all_sync(0xffffffffu, wait<true>(acc_full(buf), (i >> 1) & 1, ctl))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t x[2][32];
        tmem_ld32(tl + 256u * buf + 64u * c, x[0]);
        tmem_ld32(tl + 256u * buf + 64u * c + 32u, x[1]);
        tmem_wait_ld();
        if (c == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(racc + 8u * buf);  // the accumulator may take the tile after next
        }
        // A value that its type does not hold shows as exponent bits all ones
        // after the rounding: adding one to the exponent carries out of them.
        uint32_t w[32], carry = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float lo = __uint_as_float(x[k >> 4][2 * (k & 15)]), hi = __uint_as_float(x[k >> 4][2 * (k & 15) + 1]);
          w[k] = keys ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
          carry |= (w[k] & 0x7fff7fffu) + one;
        }
        // rows behind the prefix may hold anything
        if ((carry & 0x80008000u) != 0 && row0 + lane < p.prefix_len)
          atomicCAS(p.status, 0, static_cast<int>(kStValueRange));
        // four lanes to 64 bytes of a row (the rows, as threads hold them, lie 256
        // bytes apart), streaming: most of a long prefix leaves the L2 before it is read
        const int first = row0 + lane - quad;
        uint16_t* dst = out + (h * p.head_rows + first) * kHeadDim + 64 * c + 8 * quad;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint4 piece[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            piece[j] = make_uint4(w[16 * g + 4 * j], w[16 * g + 4 * j + 1], w[16 * g + 4 * j + 2], w[16 * g + 4 * j + 3]);
          quad_transpose(piece, lane);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (first + j < p.prefix_len) __stcs(reinterpret_cast<uint4*>(dst + j * kHeadDim + 32 * g), piece[j]);
        }
      }
      if (++m == tiles) {
        m = 0;
        ++h;
      }
    }
  } else if (kFp8 && warp >= kConverterWarp) {
    // Latents from FP8 rows: a chunk's codes (8 KiB) land in the upper half of
    // its slot, each thread of four warps takes 4 x 16 of them (4 lanes a row, 8
    // rows of the warp's 32 at a time), and when all have, bf16 replaces them.
    // That is 1,180 cycles a chunk, most of them latency beside the MMAs' reads
    // of shared memory; two groups of warps, each with every second chunk
    // (always of the same slots, so that it sees all their phases), hide it.
    const uint32_t g = static_cast<uint32_t>(warp - kConverterWarp) >> 2;
    const int w = warp & 3, sub = lane >> 2, u = lane & 3;
    const uint32_t done = rank == 0 ? a_full(0) : widened(0);
    const uint32_t in = sbase + kOffRing + kChunk / 2 + static_cast<uint32_t>(32 * w) * 64u + static_cast<uint32_t>(lane) * 16u;
    // the lane's two 16-byte pieces of a row, swizzled (the row's number modulo 8 is sub)
    const uint32_t out = sbase + kOffRing + static_cast<uint32_t>(32 * w + sub) * 128u;
    const uint32_t c0 = static_cast<uint32_t>((2 * u) ^ sub) << 4, c1 = static_cast<uint32_t>((2 * u + 1) ^ sub) << 4;
    // the four groups' scales of the thread's rows in tile m (what is not there reads as zeros)
    auto load_scales = [&](int m, uint32_t (&scales)[4]) {
      const int row0 = (m * 2 + static_cast<int>(rank)) * kRows + 32 * w;
      const long long page = row0 < p.prefix_len ? p.block_table[row0 / kPage] : -1;
      const int rows = page >= 0 && page < p.num_pages ? p.prefix_len - row0 - sub : 0;
      const uint8_t* src = p.cache + ((rows > 0 ? page * kPage : 0) + row0 % kPage + sub) * kFp8Row + kLatent;
#pragma unroll
      for (int r = 0; r < 4; ++r) scales[r] = 8 * r < rows ? *reinterpret_cast<const uint32_t*>(src + 8 * r * kFp8Row) : 0u;
    };
    uint32_t chunk = g, next[4];
    int m = m0;
    bool ok = true;
    if (n > 0) load_scales(m, next);
    for (int i = 0; ok && i < n; ++i) {
      uint32_t scales[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) scales[r] = next[r];
      if (++m == tiles) m = 0;
      if (i + 1 < n) load_scales(m, next);
#pragma unroll 1
      for (int k = 0; k < kStages; k += 2, chunk += 2) {
        const uint32_t s = chunk % kSlots;
        ok = warp_wait_uniform(raw_full(s), (chunk / kSlots) & 1, ctl);
        uint4 code[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) code[r] = ld_shared_v4u(in + s * kChunk + 512u * r);
        ok = named_bar_all(1 + g, 128, ok);  // all codes are in registers (and votes: a wait that ran out ends the four)
        if (!ok) break;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // 2^(e - 127); the scale byte 0 is 2^-127, 255 is NaN
          const uint32_t e = (scales[r] >> (4 * k)) & 255u;
          const float scale = __uint_as_float(e == 0 ? 0x00400000u : (e == 255 ? 0x7fc00000u : e << 23));
          const uint32_t words[4] = {code[r].x, code[r].y, code[r].z, code[r].w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(words[j >> 1] >> (16 * (j & 1)))));
            float a, b;
            asm("{\n .reg .f16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}" : "=f"(a), "=f"(b) : "r"(h2));
            o[j] = pack_bf16x2(a * scale, b * scale);
          }
          const uint32_t dst = out + s * kChunk + 1024u * r;
          st_shared_v4(dst + c0, o[0], o[1], o[2], o[3]);
          st_shared_v4(dst + c1, o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(done + 8u * s);
      }
    }
  } else {
    // RoPE dims, 8 lanes a row, and the pages' check, over the whole grid; eight
    // rows a lane in flight (one by one, 1000 rows x 1 head took 11.5 us)
    constexpr int kFlight = 8;
    for (long long r0 = blockIdx.x * (4ll * kFlight) + (lane >> 3); r0 < p.prefix_len; r0 += gridDim.x * (4ll * kFlight)) {
      long long page[kFlight];
      uint4 v[kFlight];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) page[j] = r0 + 4 * j < p.prefix_len ? p.block_table[(r0 + 4 * j) / kPage] : 0;
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const long long r = r0 + 4 * j;
        const bool ok = page[j] >= 0 && page[j] < p.num_pages;
        if (!ok && (lane & 7) == 0) atomicCAS(p.status, 0, static_cast<int>(kStBadTable));
        v[j] = make_uint4(0u, 0u, 0u, 0u);
        if (ok && r < p.prefix_len)
          v[j] = *reinterpret_cast<const uint4*>(p.cache + (page[j] * kPage + r % kPage) * p.row_bytes + p.rope_byte + 16 * (lane & 7));
      }
#pragma unroll
      for (int j = 0; j < kFlight; ++j)
        if (r0 + 4 * j < p.prefix_len) *reinterpret_cast<uint4*>(p.k_pe + (r0 + 4 * j) * kRope + 8 * (lane & 7)) = v[j];
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA touches another's shared memory after this
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ============================================================ host side
constexpr int kMaxDev = 64;
struct ExpandDevice {
  std::once_flag once;
  int status = MLA_OK;
  int sms = 0;
};
ExpandDevice g_expand_dev[kMaxDev];

int expand_device_ready(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return MLA_ERR_DEVICE;
  ExpandDevice& st = g_expand_dev[dev];
  std::call_once(st.once, [&st, dev] {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess || major != 10 ||
        minor != 3 || cudaDeviceGetAttribute(&st.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        st.sms < 2) {
      st.status = MLA_ERR_DEVICE;
      return;
    }
    if (cudaFuncSetAttribute(mla_prefix_expand_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(mla_prefix_expand_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
            cudaSuccess) {
      cudaGetLastError();
      st.status = MLA_ERR_CUDA;
    }
  });
  *sms = st.sms;
  return st.status;
}

// A weight [H, 512, 128] as 2-D [H * 512 rows, 128 columns], boxes of 64 x 64.
bool encode_weight(CUtensorMap* m, const void* base, int heads) {
  const cuuint64_t size[2] = {128, static_cast<cuuint64_t>(heads) * kLatent};
  const cuuint64_t strides[1] = {256};
  const cuuint32_t box[2] = {64u, 64u};
  return encode(m, false, 2, base, size, strides, box);
}

// Latents as {dim, row of a page, page} of the pool, boxes of 64 dims of a page's
// rows: bf16, swizzled as the MMA takes them, or codes, as they are.
bool encode_latents(CUtensorMap* m, const void* base, int64_t num_pages, bool fp8) {
  const cuuint64_t row = fp8 ? kFp8Row : 2 * kDqk;
  const cuuint64_t size[3] = {fp8 ? cuuint64_t{kLatent} : cuuint64_t{kDqk}, kPage, static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[2] = {row, row * kPage};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(kPage), 1u}, one[3] = {1, 1, 1};
  if (!fp8) return encode(m, false, 3, base, size, strides, box);
  EncodeTiledFn fn = encode_tiled();
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), size, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int mla_prefix_expand(const void* kv_cache, int64_t num_pages, const int32_t* block_table, int prefix_len,
                      const void* w_uk, const void* w_uv, int num_heads, unsigned flags, void* k_nope, void* v,
                      int64_t head_rows, void* k_pe, int* status, mla_stream_t stream) {
  if (!kv_cache || !block_table || !w_uk || !w_uv || !k_nope || !v || !k_pe || !status) return MLA_ERR_INVALID_ARG;
  if (!al(kv_cache, 16) || !al(block_table, 4) || !al(w_uk, 16) || !al(w_uv, 16) || !al(k_nope, 16) || !al(v, 16) ||
      !al(k_pe, 16) || !al(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_pages < 1 || prefix_len < 0 || head_rows < prefix_len) return MLA_ERR_INVALID_ARG;
  if (flags & ~static_cast<unsigned>(MLA_FLAG_KV_FP8)) return MLA_ERR_INVALID_ARG;
  if (num_heads < 1 || num_heads > kHeads) return MLA_ERR_UNSUPPORTED;
  if (num_pages > (INT32_MAX / kPage) - 1 || head_rows > kMaxRows) return MLA_ERR_UNSUPPORTED;
  int sms = 0;
  const int rc = expand_device_ready(&sms);
  if (rc != MLA_OK) return rc;
  if (prefix_len == 0) return MLA_OK;
  const bool fp8 = (flags & MLA_FLAG_KV_FP8) != 0;
  ExpandParams p;
  p.cache = static_cast<const uint8_t*>(kv_cache);
  p.row_bytes = fp8 ? kFp8Row : 2 * kDqk;
  p.rope_byte = fp8 ? 528 : 2 * kLatent;
  p.num_pages = num_pages;
  p.block_table = block_table;
  p.prefix_len = prefix_len;
  p.num_heads = num_heads;
  p.k_nope = static_cast<uint16_t*>(k_nope);
  p.v = static_cast<uint16_t*>(v);
  p.head_rows = head_rows;
  p.k_pe = static_cast<uint16_t*>(k_pe);
  p.status = status;
  CUtensorMap lat, wk, wv;
  if (!encode_latents(&lat, kv_cache, num_pages, fp8) || !encode_weight(&wk, w_uk, num_heads) ||
      !encode_weight(&wv, w_uv, num_heads))
    return MLA_ERR_CUDA;
  const long long items = static_cast<long long>((prefix_len + 2 * kRows - 1) / (2 * kRows)) * num_heads;
  const int pairs = static_cast<int>(items < sms / 2 ? items : sms / 2);
  return launch_dependent(fp8 ? mla_prefix_expand_kernel<true> : mla_prefix_expand_kernel<false>, dim3(2 * pairs),
                          dim3(fp8 ? kThreadsFp8 : kThreads), kSmem, 1, stream, p, lat, wk, wv);
}

}  // extern "C"
