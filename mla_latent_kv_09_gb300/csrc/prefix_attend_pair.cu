// prefix_attend_pair.cu — attention over a shared, expanded prefix for more
// than 128 query tokens.
//
// Above about 270 tokens a head the tensor cores bound the call (see
// prefix_attend.cu), so the design feeds them: a pair of SMs works on 256
// query rows of one head, 128 a CTA, as one M = 256 operand of
// tcgen05.mma.cta_group::2.  Each CTA holds half of every key tile (64 of its
// 128 keys) and of every value tile (64 of the 128 dims), which halves the
// shared memory, its reads and the L2 traffic of a tile against two CTAs of
// their own, and leaves room for four tiles in flight.
//
// Tensor memory of a CTA: O (128 columns) and three score buffers (128 each).
// Tile j's scores S(j) lie in buffer j % 3; its weights P(j) replace them in
// fp16.  In the steady state the tensor cores run PV(j), QK(j + 2), PV(j + 1),
// QK(j + 3) ..: the buffer that QK(j + 2) overwrites is that of P(j - 1), two
// products back, so nothing waits on a product just issued, and two tiles are
// in the softmax at a time.
//
//   warps 0-7, 8-15 softmax of even and odd tiles: two threads a query row,
//                   64 scores each
//   warp 16         TMA
//   warps 17, 18    tcgen05.mma (rank 0, for both CTAs): scores, value products.
//                   One warp issuing both lost 830 of a tile's 2,370 cycles
//                   to its waits (the tensor core queues few MMAs); each now
//                   waits under the other's products
//
// The running maximum passes from tile to tile, from one group of warps to the
// other, through shared memory (a barrier for each 32 rows); it is lazy, so
// that O is rarely rescaled, by the group that moves it, once PV of the tile
// before is done.  Each thread keeps its own sums, against the maximum it last
// saw.
//
// Measured, whole calls: 256 tokens x 16384 rows x 128 heads 226 us (4.8 TB/s,
// 1.5 PFLOP/s; 246 to 252 with scores that move the maximum late, 281 of them for
// seconds on end, at the 1.7 GHz that the power limit leaves), 2048 x 4096 x 16 58
// us (1.48 PFLOP/s).  A key tile takes a pair about 1,950 cycles, of which
// the products are 1,550 (an MMA with A in shared memory takes 83 cycles, with
// A in tensor memory 69, of the 64 that M = 256 N = 128 K = 16 would need); the
// rest are waits along the chain scores -> softmax -> value product.  Two row
// tiles in one CTA (two streams with their own O and one score buffer each,
// whose chain is as long as both streams' products) took 307 and 102 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "prefix_attend.cuh"

namespace mla {
namespace prefix {
namespace {

constexpr uint32_t kStagesKV = 4;
constexpr int kKStage = 3 * 8192;           // 64 keys x 192 dims, as 64-dim chunks
constexpr int kVStage = 16384;              // 128 keys x 64 dims
constexpr int kOffK = kQTile;               // 48 KiB of queries first
constexpr int kOffV = kOffK + kStagesKV * kKStage;
constexpr int kOffMax = kOffV + kStagesKV * kVStage;    // 208 KiB: [group][2][half][row] maxima
constexpr int kOffRef = kOffMax + 8 * kTile * 4;        // [tile & 1][row] the running maximum
constexpr int kOffXchg = kOffRef + 2 * kTile * 4;           // [group][half][maximum, two sums][row]
constexpr int kOffBar = kOffXchg + 12 * kTile * 4;
// q_full q_empty o_free drain; by stage k_full v_full s_full pv; p_full[4][2]; m_done[2][4]
constexpr int kNumBars = 4 + 4 * kStagesKV + 8 + 8;
constexpr int kSlack = 1024;                // re-aligned to 1024 B (128-byte swizzle atoms)
constexpr int kSmem = kOffBar + kNumBars * 8 + 16 + kSlack;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kThreads = 608;
constexpr int kTmaWarp = 16, kQkWarp = 17;  // and 18 for the value products
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 128;  // + 128 * buffer
constexpr uint32_t kIdescQK = idesc_bf16(256, 128, 0);
// fp16 A (weights, tensor memory) and B (values, MN-major): formats 0
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((256u >> 4) << 24);
constexpr uint16_t kBoth = 3;

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
mla_prefix_attend_pair_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap tm_qn,
                              const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_k,
                              const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t mis = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + mis;
  const uint32_t sbase = smem_u32(smem);
  const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = uniform(cluster_ctarank());
  const int pair = blockIdx.x >> 1;

  const uint32_t bar0 = sbase + kOffBar;
  const uint32_t bar_q_full = bar0, bar_q_empty = bar0 + 8u, bar_o_free = bar0 + 16u, bar_drain = bar0 + 24u;
  // Of the pair's tile q (counted over its whole run), in rank 0: landed.  In
  // both CTAs: scores done (its keys may be replaced), value product done (its
  // values may be).  A stage's barriers move on only after TMA has refilled it.
  auto k_full = [&](uint32_t q) { return bar0 + 32u + 8u * (q & 3u); };
  auto v_full = [&](uint32_t q) { return bar0 + 64u + 8u * (q & 3u); };
  auto bar_s = [&](uint32_t q) { return bar0 + 96u + 8u * (q & 3u); };
  auto bar_pv = [&](uint32_t q) { return bar0 + 128u + 8u * (q & 3u); };
  // Weights of tile q's first and second 64 keys (rank 0).  Scores of tile q +
  // 2 may come while a slower warp of the group still works on tile q, those
  // of q + 4 not (they need PV(q + 1)): four barriers, and two buffers for
  // what a group's warps exchange.
  auto p_full = [&](uint32_t q, uint32_t half) { return bar0 + 160u + 16u * (q & 3u) + 8u * half; };
  // the running maximum after tile q, of 32 rows
  auto m_done = [&](uint32_t q, int quarter) { return bar0 + 224u + 32u * (q & 1u) + 8u * quarter; };
  auto par4 = [](uint32_t q) { return (q >> 2) & 1u; };
  auto par2 = [](uint32_t q) { return (q >> 1) & 1u; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + kNumBars * 8);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + kNumBars * 8 + 4);

  if (threadIdx.x == 0) {
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_empty, 1);
    mbar_init(bar_o_free, 2 * kSoftmaxWarps);
    mbar_init(bar_drain, 2);
    for (uint32_t q = 0; q < kStagesKV; ++q) {
      mbar_init(k_full(q), 1);
      mbar_init(v_full(q), 1);
      mbar_init(bar_s(q), 1);
      mbar_init(bar_pv(q), 1);
    }
    for (uint32_t q = 0; q < 4; ++q)
      for (uint32_t half = 0; half < 2; ++half) mbar_init(p_full(q, half), kSoftmaxWarps);  // 8 warps of both CTAs
    for (uint32_t q = 0; q < 2; ++q) {
      for (int quarter = 0; quarter < 4; ++quarter) mbar_init(m_done(q, quarter), 2);
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kQkWarp) {
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
  SegmentIter it(p, pair);
  Segment sg{};

  if (warp == kTmaWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_qn);
      tma_prefetch_desc(&tm_qp);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_kp);
      tma_prefetch_desc(&tm_v);
      // Every copy completes on rank 0's barriers, which rank 0 arms with the bytes of both CTAs.
      const uint32_t rq = mapa(bar_q_full, 0), rk = mapa(k_full(0), 0), rv = mapa(v_full(0), 0);
      uint32_t q = 0, seg = 0;
      bool ok = true;
      while (ok && it.next(sg)) {
        if (seg > 0 && !(ok = wait<true>(bar_q_empty, (seg - 1) & 1, ctl))) break;
        if (rank == 0) mbar_arrive_expect_tx(bar_q_full, 2 * kQTile);
        const int t0 = (2 * sg.block + static_cast<int>(rank)) * kTile;
        tma_load_3d_pair(sbase, &tm_qn, 0, sg.h, t0, rq);
        tma_load_3d_pair(sbase + 16384u, &tm_qn, 64, sg.h, t0, rq);
        tma_load_3d_pair(sbase + 32768u, &tm_qp, 0, sg.h, t0, rq);
        for (int j = sg.k0; j < sg.k1; ++j, ++q) {
          const uint32_t st = q & 3u;
          if (q >= kStagesKV && !(ok = wait<true>(bar_s(q), par4(q - kStagesKV), ctl))) break;
          if (rank == 0) mbar_arrive_expect_tx(k_full(q), 2 * kKStage);
          const uint32_t kd = sbase + kOffK + st * kKStage;
          const int key = j * kTile + 64 * static_cast<int>(rank);
          tma_load_4d_pair(kd, &tm_k, 0, key, 0, sg.h, rk + 8u * st);
          tma_load_4d_pair(kd + 8192u, &tm_k, 0, key, 1, sg.h, rk + 8u * st);
          tma_load_2d_pair(kd + 16384u, &tm_kp, 0, key, rk + 8u * st);
          if (q >= kStagesKV && !(ok = wait<true>(bar_pv(q), par4(q - kStagesKV), ctl))) break;
          if (rank == 0) mbar_arrive_expect_tx(v_full(q), 2 * kVStage);
          tma_load_4d_pair(sbase + kOffV + st * kVStage, &tm_v, 0, j * kTile, static_cast<int>(rank), sg.h, rv + 8u * st);
        }
        ++seg;
      }
      grid_launch_dependents();
      if (!ok) {  // let copies in flight land before the CTA goes away
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kDrainNs / 8) {
        }
      }
    }
    __syncwarp();
  } else if (warp >= kQkWarp) {
    if (rank == 0) {
      // the whole warp runs, one lane issues (uniform operands)
      const uint32_t leader = lane == 0 ? 1u : 0u;
      uint32_t q0 = 0, seg = 0;  // the segment's first tile
      bool ok = true;
      if (warp == kQkWarp) {
        const uint64_t ad = smem_desc(sbase, 16u, 1024u), kd = smem_desc(sbase + kOffK, 16u, 1024u);
        while (ok && it.next(sg)) {
          const uint32_t q1 = q0 + static_cast<uint32_t>(sg.k1 - sg.k0);
          ok = warp_wait_uniform<true>(bar_q_full, seg & 1, ctl);
          for (uint32_t q = q0; ok && q < q1; ++q) {
            // its score buffer last held the weights of tile q - 3
            ok = warp_wait_uniform<true>(k_full(q), par4(q), ctl) && (q < 3 || warp_wait_uniform<true>(bar_pv(q - 3), par4(q - 3), ctl));
            if (!ok) break;
            tc_fence_after();
            const uint64_t bd = kd + static_cast<uint64_t>((q & 3u) * (kKStage >> 4));
            const uint32_t d = tmem + kColS + 128u * (q % 3u);
#pragma unroll
            for (int c = 0; c < kQChunks; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_pair_ss_if(leader, d, ad + ((c * 16384 + 32 * kk) >> 4), bd + ((c * 8192 + 32 * kk) >> 4), kIdescQK,
                                (c | kk) != 0 ? 1u : 0u);
            umma_commit_pair_if(leader, bar_s(q), kBoth);
          }
          umma_commit_pair_if(leader, bar_q_empty, kBoth);
          q0 = q1;
          ++seg;
        }
      } else {
        const uint64_t vd = smem_desc(sbase + kOffV, 16384u, 1024u);
        while (ok && it.next(sg)) {
          const uint32_t q1 = q0 + static_cast<uint32_t>(sg.k1 - sg.k0);
          // O of the segment before has been read
          if (seg > 0) ok = warp_wait_uniform<true>(bar_o_free, (seg - 1) & 1, ctl);
          for (uint32_t q = q0; ok && q < q1; ++q) {
            ok = warp_wait_uniform<true>(v_full(q), par4(q), ctl);
            const uint64_t bd = vd + static_cast<uint64_t>((q & 3u) * (kVStage >> 4));
            const uint32_t a = tmem + kColS + 128u * (q % 3u);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && warp_wait_uniform<true>(p_full(q, half), par4(q), ctl);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_pair_ts_if(leader, tmem + kColO, a + 32u * half + 8u * kk, bd + ((8192 * half + 2048 * kk) >> 4),
                                kIdescPV, q == q0 && (half | kk) == 0 ? 0u : 1u);
            }
            if (!ok) break;
            umma_commit_pair_if(leader, bar_pv(q), kBoth);
          }
          q0 = q1;
          ++seg;
        }
      }
      umma_commit_pair_if(leader, bar_drain, 1);  // arrives once every MMA issued above has completed
      drain_bar(bar_drain, 0u);
      __syncwarp();
    }
  } else {
    const uint32_t g = warp >> 3;                     // group: tiles of this parity
    const int hf = (warp >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane;                // row of the CTA's 128, lane of tensor memory
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t to = tmem + lane_base + kColO;
    float* xmax2 = reinterpret_cast<float*>(smem + kOffMax) + g * 4 * kTile + r;
    float* ref = reinterpret_cast<float*>(smem + kOffRef) + r;
    float* xchg = reinterpret_cast<float*>(smem + kOffXchg) + r;
    const int pair_bar = 1 + static_cast<int>(g) * 4 + quarter;  // the two warps that share rows of a tile
    const uint32_t rp0 = mapa(p_full(0, 0), 0), ro = mapa(bar_o_free, 0);
    uint32_t q0 = 0;
    bool ok = true;  // cleared by a wait that ran out, and voted on at the next meeting of the warps
    while (it.next(sg)) {
      const uint32_t n = static_cast<uint32_t>(sg.k1 - sg.k0), q1 = q0 + n;
      const int brow = static_cast<int>(rank) * kTile + r;
      const bool real = brow < sg.rows;
      int seen = p.prefix_len;
      if (p.visible) seen = real ? max(0, min(p.visible[sg.block * 2 * kTile + brow], p.prefix_len)) : 0;
      float m = -INFINITY;                            // running maximum (log2) as of this thread's last tile
      float total = 0.f, used = 0.f;                  // this thread's sums of the weights and of the rounded ones
      for (uint32_t q = q0 + ((q0 ^ g) & 1u); q < q1; q += 2) {
        const int key0 = (sg.k0 + static_cast<int>(q - q0)) * kTile;
        const uint32_t ts = tmem + lane_base + kColS + 128u * (q % 3u);
        ok = __all_sync(0xffffffffu, wait<true>(bar_s(q), par4(q), ctl)) && ok;
        tc_fence_after();
        // Keys [32 hf, 32 hf + 32) of the tile's first 64 and of its second,
        // which is read twice: held across the step, it would push the thread
        // over its registers, into local memory.
        const int limit = seen - key0 - 32 * hf;      // keys of this tile the row sees
        // only rows that end in this tile need masks (a row that sees none of it
        // gets zeros below, unless its scores overflow)
        const bool ragged = __any_sync(0xffffffffu, limit > 0 && limit < 96);
        uint32_t x[32];
        float top;
        {
          uint32_t y[32];
          tmem_ld32(ts + 32u * hf, x);
          tmem_ld32(ts + 64u + 32u * hf, y);
          tmem_wait_ld();
          if (ragged) {
            mask32(x, limit);
            mask32(y, limit - 64);
          }
          top = max3_nan(max32(x), max32(y), -INFINITY);
        }
        const bool overflow = p.visible && __any_sync(0xffffffffu, hidden_overflow(limit, top));
        if (overflow) mask32(x, limit);
        if (limit <= 0) top = -INFINITY;
        float* xmax = xmax2 + ((q >> 1) & 1u) * 2 * kTile;
        xmax[hf * kTile] = top;
        ok = named_bar_all(pair_bar, 64, ok);         // votes: a wait that ran out in one warp ends both
        if (!ok) break;
        top = fmaxf(top, xmax[(hf ^ 1) * kTile]) * p.scale_log2;
        // the maximum that the tile before left
        if (q > 0) ok = __all_sync(0xffffffffu, wait(m_done(q - 1, quarter), par2(q - 1), ctl)) && ok;
        const float old = q == q0 ? -INFINITY : ref[((q - 1) & 1u) * kTile];
        const bool move = top > old + kLazy;
        const float now = move ? top : old;
        bool at_rest = true;
        if (q > q0 && __any_sync(0xffffffffu, move)) {
          // O is rescaled once the product before is done, half of the columns by each of the row's threads
          at_rest = __all_sync(0xffffffffu, wait<true>(bar_pv(q - 1), par4(q - 1), ctl));
          tc_fence_after();
          const float keep = move ? ex2_approx(old - top) : 1.f;
#pragma unroll 1
          for (uint32_t c = 0; c < 64u; c += 16u) rescale16(to + 64u * hf + c, keep);
          tmem_wait_st();
        }
        // (both of the row's threads have read the old maximum before the next
        // tile's may write over it)
        if (hf == 0) ref[(q & 1u) * kTile] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(m_done(q, quarter));
        if (now != m) {
          const float keep = ex2_approx(m - now);     // 0 from the first tile's -inf
          total *= keep;
          used *= keep;
          m = now;
        }
        ok = ok && at_rest;
        // +inf makes every weight of a row that sees none of these keys zero, 0 those of one that saw none yet
        const float base = limit <= 0 ? INFINITY : (m == -INFINITY ? 0.f : m);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 1) {
            tmem_ld32(ts + 64u + 32u * hf, x);
            tmem_wait_ld();
            if (ragged || overflow) mask32(x, limit - 64);
          }
          weights32(x, p.scale_log2, base, ts + 32u * c + 16u * hf, total, used);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          // (orders tensor-memory accesses only, which tcgen05.wait has completed)
          if (lane == 0) mbar_arrive_remote_relaxed(rp0 + 16u * (q & 3u) + 8u * c);
        }
      }
      q0 = q1;
      const long long row = static_cast<long long>(sg.block * 2 * kTile + brow) * p.num_heads + sg.h;
      float other2 = -INFINITY;
      if (p.suffix_lse && real && sg.whole) other2 = p.suffix_lse[row] * kLog2e;
      const long long prow = (2ll * pair + (sg.first ? 0 : 1)) * p.part_rows + brow;
      const int quad = lane & 3;
      const RowOut w = {sg.whole ? row - static_cast<long long>(quad) * p.num_heads : prow - quad,
                        sg.whole ? p.num_heads : 1, sg.rows - (brow - quad), sg.whole};
      const uint32_t c0 = 64u * g + 32u * hf;         // a quarter of the columns
      uint4 suffix[4];
      load_suffix(p, w, c0, lane, suffix);
      if (ok) ok = __all_sync(0xffffffffu, wait<true>(bar_pv(q1 - 1), par4(q1 - 1), ctl));
      // The row's result: the sums of its four threads, against the last
      // maximum.  All softmax warps vote, so that a wait that ran out in one
      // ends them all.
      float* mine = xchg + (g * 2 + hf) * 3 * kTile;
      mine[0] = m;
      mine[kTile] = total;
      mine[2 * kTile] = used;
      ok = named_bar_all(9, kSoftmaxWarps * 32, ok);
      if (!ok) break;
      const float last = ref[((q1 - 1) & 1u) * kTile], base = last == -INFINITY ? 0.f : last;  // O's own
      float sum = 0.f, u = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = ex2_approx(xchg[3 * i * kTile] - base);
        sum = fmaf(xchg[(3 * i + 1) * kTile], f, sum);
        u = fmaf(xchg[(3 * i + 2) * kTile], f, u);
      }
      const float f0 = u == 0.f ? 0.f : 1.f / u;
      const float lse2 = sum == 0.f ? -INFINITY : base + lg2(sum);
      named_bar_sync(9, kSoftmaxWarps * 32);          // the exchange and the maximum may be written again
      tc_fence_after();
      Join j = {1.f, 0.f, lse2};
      if (p.suffix_lse && sg.whole) j = join(lse2, other2);
      write32(p, w, c0, lane, j, suffix, [&](int h, float (&o)[16]) {
        uint32_t a[16];
        tmem_ld16(to + c0 + 16u * h, a);
        tmem_wait_ld();
        // an accumulator that took nothing is not read as a number
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = f0 == 0.f ? 0.f : __uint_as_float(a[k]) * f0;
      });
      if (real && hf == 0 && g == 0) {
        if (sg.whole)
          p.lse[row] = j.lse2 * kLn2;
        else
          p.part_lse[prow] = lse2;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(ro);
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA touches another's shared memory after this
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t attend_pair_set_attrs() {
  return cudaFuncSetAttribute(mla_prefix_attend_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

int attend_pair_launch(int pairs, mla_stream_t stream, const AttendParams& p, const CUtensorMap& qn,
                       const CUtensorMap& qp, const CUtensorMap& k, const CUtensorMap& kp, const CUtensorMap& v) {
  return launch_dependent(mla_prefix_attend_pair_kernel, dim3(2 * pairs), dim3(kThreads), kSmem, 1, stream, p, qn, qp,
                          k, kp, v);
}

}  // namespace prefix
}  // namespace mla
