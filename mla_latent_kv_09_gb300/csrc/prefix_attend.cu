// prefix_attend.cu — attention of a batch's query tokens over a shared,
// expanded prefix: the kernel for up to 128 tokens, the join of cut heads, and
// the C ABI (include/mla_prefix.h).
//
// One head is ordinary attention: T query rows of 192 dims, P keys of 192 (128
// of the head's, 64 RoPE dims shared by all heads), P values of 128.  A key
// tile of 128 rows is 64 KiB from HBM for 128 * 2 * 320 operations a query
// row: up to about 270 tokens the HBM bounds the call, above it the tensor
// cores do.
//
// This kernel (a CTA per SM, one row tile of up to 128 query rows, the rest of
// the tile zeros) is bound by the HBM: the tensor cores need 1,280 of the
// 2,850 cycles that a tile takes to arrive.  Its two streams take alternate
// key tiles, each with its own scores S and output O in tensor memory (2 * (128
// + 128) columns, all of it), and are joined at the end.
//
//   warps 0-7, 8-15 softmax of stream 0, 1: two threads own a query row, each
//                   64 of its 128 scores, which it reads from tensor memory;
//                   they agree on the running maximum, keep their own sums
//                   and write the weights in fp16 over the scores, where the
//                   value product reads them as its A operand
//   warp 16         TMA: the queries (48 KiB), then key and value chunks of
//                   16 KiB through a ring of 10 slots
//   warps 17, 18    tcgen05.mma for stream 0, 1: S = Q K^T (12 steps of M128
//                   N128 K16, bf16), O += P V (8 steps, fp16).  The tensor
//                   core takes an MMA every 64 cycles and queues few, so a
//                   wait of the issuing thread (100 to 250 cycles) is time
//                   lost; two issuers fill each other's
//
// The weights are handed over in two halves of 64 keys: the value product of
// the first runs under the exponentials of the second.
//
// The running maximum is lazy: it moves only when a score beats it by 2^14, so
// that O is rarely rescaled.  O is normalised by the sum of the rounded weights
// that the value product used, so that a weight's rounding acts on v_j - O and
// not on v_j; the LSE takes the sum of the unrounded ones.  fp16 for the weights
// and values: 11 bits, against bf16's 8; a weight below 2^-25 of the running
// maximum's rounds to zero, so P rows lose at most P 2^-25 of their sum.
//
// Work split: all (head, key tile) steps of a row block form one line, cut
// into equal ranges, one per CTA or pair (see plan()).  A range that covers a
// head's whole prefix writes the result; a head cut in pieces leaves
// normalised fp32 partial rows and their LSE, which the combine kernel joins.
//
// Measured, whole calls: 64 tokens x 8192 rows x 128 heads 93.5 us (545 MB, 5.8
// TB/s), 1 x 777 x 128 14.3 us (51 MB, of which 6 us are the launch, the first
// tile's way in and the last one's way out).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "mla_prefix.h"
#include "prefix_attend.cuh"

namespace mla {
namespace {

using namespace prefix;

constexpr int kSlot = 16384;                // a key chunk (128 keys x 64 dims) or half a value tile (64 keys x 128 dims)
constexpr uint32_t kSlots = 10;             // two key and two value tiles
constexpr int kOffXchg = kQTile;            // the threads of a row exchange their sums here
constexpr int kOffRing = kQTile + kSlot;
constexpr int kOffBar = kOffRing + kSlots * kSlot;      // 224 KiB
constexpr int kNumBars = 8 + 12;
constexpr int kOffMax = kOffBar + kNumBars * 8 + 16;    // [stream][half][row]: exchange between a row's two threads
constexpr int kSmem = kOffMax + 4 * kTile * 4;          // no room to re-align: the base must lie on 1024 B (checked)
static_assert(kSmem <= 232448, "shared memory");
constexpr int kThreads = 608;
constexpr int kTmaWarp = 16, kMmaWarp = 17;  // and 18, for the second stream
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;  // + 128 * stream
constexpr uint32_t kIdescQK = idesc_bf16(128, 128, 0);
// fp16 A (weights, tensor memory) and B (values, MN-major): formats 0
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

// kPartial: the call has `visible`.  Without it only rows behind the prefix are
// hidden, and the code for hidden scores that overflow is left out (its size
// alone, with no such scores: 1 x 777 x 128 14.8 us against 14.4, 64 x 8192 x 128
// 94.4 against 93.6).
template <bool kPartial>
__global__ void __launch_bounds__(kThreads, 1)
mla_prefix_attend_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap tm_qn,
                         const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sbase = smem_u32(smem);
  const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if ((sbase & 1023u) != 0) {  // the swizzled tiles need it; the kernel has no static shared memory ahead of it
    if (threadIdx.x == 0) atomicCAS(p.status, 0, static_cast<int>(MLA_ERR_CUDA));
    return;
  }

  const uint32_t bar0 = sbase + kOffBar;
  // key (value) tile q of the CTA's run, by q & 1: landed, and used by every stream that uses it
  auto k_full = [&](uint32_t q) { return bar0 + 8u * (q & 1u); };
  auto k_empty = [&](uint32_t q) { return bar0 + 16u + 8u * (q & 1u); };
  auto v_full = [&](uint32_t q) { return bar0 + 32u + 8u * (q & 1u); };
  auto v_empty = [&](uint32_t q) { return bar0 + 48u + 8u * (q & 1u); };
  const uint32_t bar_q_full = bar0 + 64u, bar_q_empty = bar_q_full + 8u;
  auto bar_s_full = [&](int s) { return bar_q_full + 8u * (2 + s); };  // scores of a stream are in tensor memory
  auto bar_p_full = [&](int s, int half) { return bar_q_full + 8u * (4 + 2 * s + half); };  // its weights are
  auto bar_pv = [&](int s) { return bar_q_full + 8u * (8 + s); };      // its value product is done
  const uint32_t bar_o_free = bar_q_full + 8u * 10, bar_drain = bar_q_full + 8u * 11;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + kNumBars * 8);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + kNumBars * 8 + 4);
  auto slot_addr = [&](uint32_t n) { return sbase + kOffRing + (n % kSlots) * kSlot; };

  if (threadIdx.x == 0) {
    for (uint32_t q = 0; q < 2; ++q) {
      mbar_init(k_full(q), 1);
      mbar_init(k_empty(q), 1);
      mbar_init(v_full(q), 1);
      mbar_init(v_empty(q), 1);
    }
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_empty, 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_s_full(s), 1);
      mbar_init(bar_p_full(s, 0), kSoftmaxWarps / 2);
      mbar_init(bar_p_full(s, 1), kSoftmaxWarps / 2);
      mbar_init(bar_pv(s), 1);
    }
    mbar_init(bar_o_free, kSoftmaxWarps);
    mbar_init(bar_drain, 2);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);

  Ctl ctl;
  ctl.abort = abort_flag;
  ctl.n_remote = 0;
  ctl.status = p.status;

  grid_dependency_wait();
  SegmentIter it(p, blockIdx.x);
  Segment sg{};

  // Tiles enter the ring in the order the MMAs use them: K0 K1 V0 K2 V1 K3 ..
  // A key tile is three chunks, a value tile two; these are the places of tile
  // j's first chunk in a segment of n tiles.  At most two key and two value
  // tiles are in the ring at a time, hence two barriers for each.
  auto place_k = [](int j) { return j < 2 ? 3 * j : 5 * j - 2; };
  auto place_v = [](int j, int n) { return j == n - 1 ? 5 * n - 2 : 5 * j + 6; };

  uint32_t issued = 0, k_issued = 0, v_issued = 0;  // chunks and tiles requested so far (TMA warp)
  int q_loads = 0;
  if (warp == kTmaWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_qn);
      tma_prefetch_desc(&tm_qp);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_kp);
      tma_prefetch_desc(&tm_v);
      bool ok = true;
      // tiles in the ring: the oldest one's first chunk, how many of each kind
      // have left, and their kinds in order (bit 0 the oldest, 1 = value)
      uint32_t oldest = 0, k_left = 0, v_left = 0, kinds = 0, held = 0;
      auto make_room = [&](uint32_t chunks, const uint32_t& requested, const uint32_t& left) -> bool {
        while (held > 0 && (oldest + kSlots < issued + chunks || requested - left >= 2)) {
          if (kinds & 1u) {
            if (!wait(v_empty(v_left), (v_left >> 1) & 1, ctl)) return false;
            ++v_left;
            oldest += 2;
          } else {
            if (!wait(k_empty(k_left), (k_left >> 1) & 1, ctl)) return false;
            ++k_left;
            oldest += 3;
          }
          kinds >>= 1;
          --held;
        }
        return true;
      };
      auto load_k = [&](int tile) -> bool {
        if (!make_room(3, k_issued, k_left)) return false;
        const uint32_t bar = k_full(k_issued);
        mbar_arrive_expect_tx(bar, kQTile);
        tma_load_4d(slot_addr(issued), &tm_k, 0, tile * kTile, 0, sg.h, bar);
        tma_load_4d(slot_addr(issued + 1), &tm_k, 0, tile * kTile, 1, sg.h, bar);
        tma_load_2d(slot_addr(issued + 2), &tm_kp, 0, tile * kTile, bar);
        issued += 3;
        ++k_issued;
        ++held;
        return true;
      };
      auto load_v = [&](int tile) -> bool {
        if (!make_room(2, v_issued, v_left)) return false;
        const uint32_t bar = v_full(v_issued);
        mbar_arrive_expect_tx(bar, 2 * kSlot);
        tma_load_4d(slot_addr(issued), &tm_v, 0, tile * kTile, 0, sg.h, bar);
        tma_load_4d(slot_addr(issued + 1), &tm_v, 0, tile * kTile + 64, 0, sg.h, bar);
        issued += 2;
        ++v_issued;
        kinds |= 1u << held;
        ++held;
        return true;
      };
      while (ok && it.next(sg)) {
        if (q_loads > 0 && !wait(bar_q_empty, (q_loads - 1) & 1, ctl)) break;
        mbar_arrive_expect_tx(bar_q_full, kQTile);
        tma_load_3d(sbase, &tm_qn, 0, sg.h, 0, bar_q_full);
        tma_load_3d(sbase + kSlot, &tm_qn, 64, sg.h, 0, bar_q_full);
        tma_load_3d(sbase + 2 * kSlot, &tm_qp, 0, sg.h, 0, bar_q_full);
        ++q_loads;
        ok = load_k(sg.k0);
        if (ok && sg.k0 + 1 < sg.k1) ok = load_k(sg.k0 + 1);
        for (int j = sg.k0; ok && j < sg.k1; ++j) {
          ok = load_v(j);
          if (ok && j + 2 < sg.k1) ok = load_k(j + 2);
        }
      }
      grid_launch_dependents();
    }
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // The whole warp runs this loop and one lane issues, by predicates: the
    // operands stay warp-uniform, and so in uniform registers.  (Issued from a
    // divergent branch, with the counters in local memory, the 20 MMAs of a
    // step took 3,600 cycles against the tensor cores' 1,280.)
    const uint32_t leader = lane == 0 ? 1u : 0u;
    const uint32_t s = warp - kMmaWarp;  // stream
    const uint64_t ring_k = smem_desc(sbase + kOffRing, 16u, 1024u), ring_v = smem_desc(sbase + kOffRing, 8192u, 1024u);
    const uint32_t t_s = tmem + kColS + 128u * s, t_o = tmem + kColO + 128u * s;
    uint32_t base = 0, tiles = 0;  // chunks, key tiles of the segments before this one
    uint32_t n_pv = 0;             // value products issued
    uint32_t seg = 0;
    bool ok = true;
    auto slot_off = [](uint32_t c) { return static_cast<uint64_t>(c % kSlots) * (kSlot >> 4); };
    // Waits for the last value product and gives its tile back: a commit per
    // tile cost 125 cycles of the issuing thread each, an arrive 20.
    uint32_t v_held = 0;           // its barrier, 0: given back
    auto release_v = [&]() -> bool {
      if (v_held == 0) return true;
      if (!warp_wait_uniform(bar_pv(s), (n_pv - 1) & 1, ctl)) return false;
      if (leader) mbar_arrive(v_held);
      v_held = 0;
      return true;
    };
    while (ok && it.next(sg)) {
      const int n = sg.k1 - sg.k0;
      const int steps = (n + 1 - static_cast<int>(s)) / 2;
      const uint64_t ad = smem_desc(sbase, 16u, 1024u);
      // Scores of key tile j.  S holds the weights of the step before until
      // its value product is done.
      auto issue_qk = [&](int j) -> bool {
        const uint32_t c0 = base + place_k(j), q = tiles + j;
        if (!warp_wait_uniform(k_full(q), (q >> 1) & 1, ctl)) return false;
        if (!release_v()) return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kQChunks; ++c) {
          const uint64_t bd = ring_k + slot_off(c0 + c);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss_if(leader, t_s, ad + ((c * kSlot + 32 * kk) >> 4), bd + ((32 * kk) >> 4), kIdescQK,
                       (c | kk) != 0 ? 1u : 0u);
        }
        umma_commit_if(leader, bar_s_full(s));
        return true;
      };
      ok = warp_wait_uniform(bar_q_full, seg & 1, ctl) && (steps == 0 || issue_qk(s));
      if (steps <= 1) umma_commit_if(leader, bar_q_empty);
      // O of the segment before has been read
      if (ok && seg > 0) ok = warp_wait_uniform(bar_o_free, (seg - 1) & 1, ctl);
      for (int i = 0; ok && i < steps; ++i) {
        const int j = 2 * i + static_cast<int>(s);
        const uint32_t c0 = base + place_v(j, n), q = tiles + j;
        ok = warp_wait_uniform(v_full(q), (q >> 1) & 1, ctl);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          ok = ok && warp_wait_uniform(bar_p_full(s, c), n_pv & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bd = ring_v + slot_off(c0 + c);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ts_if(leader, t_o, t_s + 32u * c + 8u * kk, bd + ((2048 * kk) >> 4), kIdescPV,
                       i == 0 && (c | kk) == 0 ? 0u : 1u);
        }
        if (!ok) break;
        umma_commit_if(leader, bar_pv(s));
        v_held = v_empty(q);
        ++n_pv;
        if (i + 1 < steps) {
          ok = issue_qk(j + 2);
          if (i + 2 == steps) umma_commit_if(leader, bar_q_empty);  // the segment's last scores
        }
      }
      ok = ok && release_v();
      base += 5u * n;
      tiles += n;
      ++seg;
    }
    umma_commit_if(leader, bar_drain);  // arrives once every MMA issued above has completed
    __syncwarp();
  } else {
    const int s = warp >> 3, hf = (warp >> 2) & 1;    // stream, and which half of a row's scores
    const int r = (warp & 3) * 32 + lane;             // row of the tile, lane of tensor memory
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + kColS + 128u * s;
    const uint32_t to = tmem + lane_base + kColO;
    float* xmax = reinterpret_cast<float*>(smem + kOffMax) + s * 2 * kTile + r;
    float* xchg = reinterpret_cast<float*>(smem + kOffXchg);
    const int pair_bar = 1 + s * 4 + (warp & 3);      // the two warps that share rows
    uint32_t n_s = 0;    // score tiles taken
    uint32_t tiles = 0;  // key tiles of the segments before this one
    bool ok = true;
    while (it.next(sg)) {
      const int n = sg.k1 - sg.k0;
      const int steps = (n + 1 - s) / 2;
      const bool real = r < sg.rows;
      int seen = p.prefix_len;
      if (kPartial) seen = real ? max(0, min(p.visible[r], p.prefix_len)) : 0;
      float m = -INFINITY;                            // running maximum (log2)
      float total = 0.f, used = 0.f;                  // this thread's sums of the weights and of the rounded ones
      for (int i = 0; i < steps; ++i) {
        const int key0 = (sg.k0 + 2 * i + s) * kTile;
        ok = __all_sync(0xffffffffu, wait(bar_s_full(s), n_s & 1, ctl));
        ++n_s;
        tc_fence_after();
        // the key tile has been read: its slots may be filled again
        if (lane == 0 && (warp & 7) == 0) mbar_arrive(k_empty(tiles + 2 * i + s));
        // Keys [32 hf, 32 hf + 32) of the tile's first 64 and of its second.
        // The second part is read twice: held across the step, it would push
        // the thread over its 96 registers, into local memory.
        const int limit = seen - key0 - 32 * hf;      // keys of this tile the row sees
        // A row that sees none of them needs no masks (its weights become
        // zeros below) unless its scores overflow: only rows that end in this
        // tile do.
        const bool ragged = __any_sync(0xffffffffu, limit > 0 && limit < 96);
        uint32_t x[32];
        tmem_ld32(ts + 64u + 32u * hf, x);
        tmem_wait_ld();
        if (ragged) mask32(x, limit - 64);
        float top = max32(x);
        tmem_ld32(ts + 32u * hf, x);
        tmem_wait_ld();
        if (ragged) mask32(x, limit);
        bool overflow = false;
        if (kPartial) {
          top = max3_nan(top, max32(x), -INFINITY);
          overflow = __any_sync(0xffffffffu, hidden_overflow(limit, top));
          if (overflow) mask32(x, limit);
          if (limit <= 0) top = -INFINITY;
        } else {
          top = limit <= 0 ? -INFINITY : fmaxf(top, max32(x));
        }
        // The partner cannot write its next maximum before this one is read:
        // its next scores wait for this warp's weights.
        xmax[hf * kTile] = top;
        ok = named_bar_all(pair_bar, 64, ok);         // votes: a wait that ran out in one warp ends both
        if (!ok) break;
        top = fmaxf(top, xmax[(hf ^ 1) * kTile]) * p.scale_log2;
        const bool move = top > m + kLazy;
        // This step's scores were issued after the value product of the step
        // before had completed: O is at rest and may be rescaled here, half
        // of its columns by each of the row's threads.
        if (__any_sync(0xffffffffu, move)) {
          const float keep = move ? ex2_approx(m - top) : 1.f;
          if (move) m = top;
          total *= keep;
          used *= keep;
          if (i > 0) {
#pragma unroll 1
            for (uint32_t c = 0; c < 64u; c += 16u) rescale16(to + 128u * s + 64u * hf + c, keep);
          }
        }
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
          if (lane == 0) mbar_arrive(bar_p_full(s, c));
        }
      }
      tiles += n;
      const long long row = static_cast<long long>(r) * p.num_heads + sg.h;
      float other2 = -INFINITY;
      if (p.suffix_lse && real && sg.whole) other2 = p.suffix_lse[row] * kLog2e;
      // every value product of the stream in this segment (n_s counts them too)
      if (ok && steps > 0) ok = __all_sync(0xffffffffu, wait(bar_pv(s), (n_s - 1) & 1, ctl));
      // The row's result: the sums of its four threads; the streams' maxima
      // differ.  All softmax warps vote, so that a wait that ran out in one
      // ends them all.
      float* mine = xchg + (s * 2 + hf) * 3 * kTile + r;
      mine[0] = m;
      mine[kTile] = total;
      mine[2 * kTile] = used;
      ok = named_bar_all(9, kSoftmaxWarps * 32, ok);
      if (!ok) break;
      const float m0 = xchg[r], m1 = xchg[6 * kTile + r];
      const float top = fmaxf(m0, m1), base = top == -INFINITY ? 0.f : top;
      const float a0 = ex2_approx(m0 - base), a1 = ex2_approx(m1 - base);
      const float sum = (xchg[kTile + r] + xchg[4 * kTile + r]) * a0 + (xchg[7 * kTile + r] + xchg[10 * kTile + r]) * a1;
      const float u = (xchg[2 * kTile + r] + xchg[5 * kTile + r]) * a0 + (xchg[8 * kTile + r] + xchg[11 * kTile + r]) * a1;
      const float inv = u == 0.f ? 0.f : 1.f / u;
      const float f0 = a0 * inv, f1 = a1 * inv;       // scale of each stream's O in the row's result
      const float lse2 = sum == 0.f ? -INFINITY : base + lg2(sum);
      named_bar_sync(9, kSoftmaxWarps * 32);          // the exchange may be written again
      tc_fence_after();
      Join j = {1.f, 0.f, lse2};
      if (p.suffix_lse && sg.whole) j = join(lse2, other2);
      const long long prow = (2ll * blockIdx.x + (sg.first ? 0 : 1)) * p.part_rows + r;
      // both streams' O, a quarter of the columns each
      const uint32_t c0 = 64u * s + 32u * hf;
      const bool second = n > 1;
#pragma unroll 1
      for (uint32_t c = c0; c < c0 + 32u; c += 16u) {
        uint32_t a[16], b[16];
        __syncwarp();  // lanes without a row have gone round sooner; the loads are the whole warp's
        tmem_ld16(to + c, a);
        if (second) tmem_ld16(to + 128u + c, b);
        tmem_wait_ld();
        if (!real) continue;
        float o[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          o[k] = f0 == 0.f ? 0.f : __uint_as_float(a[k]) * f0;  // an accumulator that took nothing is not read as a number
          if (second && f1 != 0.f) o[k] = fmaf(__uint_as_float(b[k]), f1, o[k]);
        }
        if (sg.whole) {
          write8(p, row, c, o, j);
          write8(p, row, c + 8, o + 8, j);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + prow * kHeadDim + c);
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if (real && hf == 0 && s == 0) {
        if (sg.whole)
          p.lse[row] = j.lse2 * kLn2;
        else
          p.part_lse[prow] = lse2;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_o_free);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == kMmaWarp * 32) drain_bar(bar_drain, 0u);  // MMAs finish before TMEM is released
  if (threadIdx.x == kTmaWarp * 32 && *abort_flag) {
    // teardown after a wait ran out: loads still in flight land before the CTA exits
    for (uint32_t q = k_issued > 2 ? k_issued - 2 : 0; q < k_issued; ++q) drain_bar(k_full(q), (q >> 1) & 1);
    for (uint32_t q = v_issued > 2 ? v_issued - 2 : 0; q < v_issued; ++q) drain_bar(v_full(q), (q >> 1) & 1);
    if (q_loads > 0) drain_bar(bar_q_full, (q_loads - 1) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partial rows of the (row block, head)s that were cut.  Block (x,
// lane block, chunk) takes one of them: unit x of the line if there are fewer
// units than ranges, else the unit that range x + 1 starts inside of, if no
// earlier range does; and of it kCombineRows rows a warp (kWide = false, up to
// 8 pieces: lane l takes the LSE of row l / 8 and piece l % 8, and all four
// rows' loads are in flight together) or one row (kWide: a thread takes the LSE
// of a piece, a warp every eighth piece, eight loads in flight).  Four columns
// a lane.  Latency is all it costs, so loads do not wait for one another: one
// row a warp, its LSEs first, took 13.4 us for 75 heads of 256 rows (9.5 so),
// and for one row of 118 pieces 25 us.
constexpr int kCombineWarps = 8, kCombineRows = 4;
__host__ __device__ __forceinline__ bool few_units(const Plan& w, int num_heads) {
  return static_cast<long long>(w.passes) * num_heads < w.groups;
}
template <bool kWide>
__global__ void __launch_bounds__(32 * kCombineWarps) mla_prefix_combine_kernel(const __grid_constant__ AttendParams p) {
  __shared__ float4 acc[kWide ? kCombineWarps : 1][32];
  constexpr int kRowsWarp = kWide ? 1 : kCombineRows;
  const Plan& w = p.plan;
  // Every block waits, those without work too: what follows on the stream
  // waits for this kernel, and this kernel's end must not come before the end
  // of the one that wrote the pieces.
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lane_block = blockIdx.y;
  int unit, g0;  // g0: the range that holds the unit's first step, as its first segment or, after another, its second
  if (few_units(w, p.num_heads)) {
    unit = blockIdx.x;
    g0 = static_cast<int>(quotient((static_cast<long long>(unit) * w.nk + 1) * w.groups - 1, w.line));
  } else {
    g0 = blockIdx.x;
    unit = static_cast<int>(quotient(cut(w, g0 + 1), w.nk));
  }
  const long long start = static_cast<long long>(unit) * w.nk, end = start + w.nk;
  const long long before = cut(w, g0), at = cut(w, g0 + 1);
  if (before > start || at <= start || at >= end) return;  // not the range of the unit's first step, or the unit is whole
  const int block = unit / p.num_heads * w.width + lane_block, h = unit % p.num_heads;
  if (block >= w.blocks) return;
  const int odd = before < start ? 1 : 0;
  const int n = static_cast<int>(quotient(end * w.groups - 1, w.line)) - g0 + 1;  // up to the range of its last step
  const int brow = kWide ? blockIdx.z : (blockIdx.z * kCombineWarps + warp) * kRowsWarp;
  const int left = min(p.part_rows - brow, p.num_tokens - block * 2 * kTile - brow);  // real rows from brow on
  if (left <= 0) return;  // (kWide: the block's warps all have the same row)
  const long long row0 = static_cast<long long>(block * 2 * kTile + brow) * p.num_heads + h;
  auto piece = [&](int i) {  // first row of piece i among the partial rows
    const int slot = 2 * ((g0 + i) * w.width + lane_block) + (i == 0 ? odd : 0);
    return static_cast<long long>(slot) * p.part_rows + brow;
  };
  const float4* part_o = reinterpret_cast<const float4*>(p.part_o) + lane;
  float4 o[kRowsWarp];
  float lse2, f;  // of the lane's row; the share of its piece
  float other2 = -INFINITY;
  if (!kWide) {
    const int r = min(lane >> 3, left - 1);
    if (p.suffix_lse) other2 = p.suffix_lse[row0 + static_cast<long long>(r) * p.num_heads] * kLog2e;
    const float mine = (lane & 7) < n ? p.part_lse[piece(lane & 7) + r] : -INFINITY;
    float top = mine;
#pragma unroll
    for (int i = 4; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float base = top == -INFINITY ? 0.f : top;
    f = ex2_approx(mine - base);
    float sum = f;
#pragma unroll
    for (int i = 4; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    f *= sum == 0.f ? 0.f : 1.f / sum;
    lse2 = sum == 0.f ? -INFINITY : base + lg2(sum);
#pragma unroll
    for (int k = 0; k < kRowsWarp; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const long long from = piece(i);
      float4 v[kRowsWarp];
#pragma unroll
      for (int k = 0; k < kRowsWarp; ++k)
        v[k] = k < left ? part_o[(from + k) * (kHeadDim / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kRowsWarp; ++k) {
        const float share = __shfl_sync(0xffffffffu, f, 8 * k + i);
        o[k].x = fmaf(v[k].x, share, o[k].x);
        o[k].y = fmaf(v[k].y, share, o[k].y);
        o[k].z = fmaf(v[k].z, share, o[k].z);
        o[k].w = fmaf(v[k].w, share, o[k].w);
      }
    }
  } else {
    // thread i: the LSE of piece i; a warp's first eight pieces come under them
    __shared__ float red[2][kCombineWarps], share[32 * kCombineWarps];
    if (p.suffix_lse) other2 = p.suffix_lse[row0] * kLog2e;
    const int i0 = threadIdx.x;
    const float mine = i0 < n ? p.part_lse[piece(i0)] : -INFINITY;
    auto load = [&](int first, float4 (&v)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = first + k * kCombineWarps;
        v[k] = i < n ? part_o[piece(i) * (kHeadDim / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    float4 v[8];
    load(warp, v);
    float top = mine;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    red[0][warp] = top;
    __syncthreads();
    top = red[0][lane & 7];
#pragma unroll
    for (int i = 4; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float base = top == -INFINITY ? 0.f : top;
    f = ex2_approx(mine - base);
    float sum = f;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    red[1][warp] = sum;
    share[i0] = f;
    __syncthreads();
    sum = red[1][lane & 7];
#pragma unroll
    for (int i = 4; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    lse2 = sum == 0.f ? -INFINITY : base + lg2(sum);
    o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int first = warp; first < n; first += 8 * kCombineWarps) {
      if (first != warp) load(first, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = first + k * kCombineWarps;
        const float part = i < n ? share[i] * inv : 0.f;
        o[0].x = fmaf(v[k].x, part, o[0].x);
        o[0].y = fmaf(v[k].y, part, o[0].y);
        o[0].z = fmaf(v[k].z, part, o[0].z);
        o[0].w = fmaf(v[k].w, part, o[0].w);
      }
    }
    acc[warp][lane] = o[0];
    __syncthreads();
    if (warp != 0) return;
    for (int i = 1; i < kCombineWarps; ++i) {
      const float4 v = acc[i][lane];
      o[0].x += v.x;
      o[0].y += v.y;
      o[0].z += v.z;
      o[0].w += v.w;
    }
  }
  Join j = {1.f, 0.f, lse2};
  if (p.suffix_lse) j = join(lse2, other2);
  __syncwarp();  // lse may be suffix_lse: all lanes have read it
  if (kWide ? lane == 0 : (lane & 7) == 0 && (lane >> 3) < left)
    p.lse[row0 + static_cast<long long>(kWide ? 0 : lane >> 3) * p.num_heads] = j.lse2 * kLn2;
#pragma unroll
  for (int k = 0; k < kRowsWarp; ++k) {
    const Join of = {__shfl_sync(0xffffffffu, j.mine, 8 * k), __shfl_sync(0xffffffffu, j.other, 8 * k), 0.f};
    if (k < left) write4(p, row0 + static_cast<long long>(k) * p.num_heads, 4 * lane, o[k], of);
  }
}

// Nothing to attend to in the prefix: the suffix's result, or zeros.
__global__ void __launch_bounds__(128) mla_prefix_empty_kernel(const __grid_constant__ AttendParams p) {
  grid_dependency_wait();
  const long long at = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x;
  const long long row = at / (kHeadDim / 8);
  const bool real = row < static_cast<long long>(p.num_tokens) * p.num_heads;
  const int col = static_cast<int>(at % (kHeadDim / 8)) * 8;
  const float other = real && p.suffix_lse ? p.suffix_lse[row] : -INFINITY;
  const float zero[8] = {};
  if (real) write8(p, row, col, zero, join(-INFINITY, other * kLog2e));
  // 16 threads of one warp share the row: the one that writes its LSE, which may
  // be the suffix's, does so after all have read it
  __syncwarp();
  if (real && col == 0) p.lse[row] = other;
}

// ============================================================ host side
// Query rows as boxes of {64 dims, 1 head, 128 tokens}.
bool encode_q(CUtensorMap* m, const void* base, int dims, int64_t stride, int heads, int tokens) {
  const cuuint64_t size[3] = {static_cast<cuuint64_t>(dims), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride) * 2,
                                 static_cast<cuuint64_t>(stride) * 2 * static_cast<cuuint64_t>(heads)};
  const cuuint32_t box[3] = {64u, 1u, static_cast<cuuint32_t>(kTile)};
  return encode(m, false, 3, base, size, strides, box);
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
        minor != 3 || cudaDeviceGetAttribute(&st.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        st.sms < 1) {
      st.status = MLA_ERR_DEVICE;
      return;
    }
    if (cudaFuncSetAttribute(mla_prefix_attend_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(mla_prefix_attend_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
            cudaSuccess ||
        attend_pair_set_attrs() != cudaSuccess) {
      cudaGetLastError();
      st.status = MLA_ERR_CUDA;
    }
  });
  *sms = st.sms;
  return st.status;
}

// Units: up to 128 tokens CTAs, above pairs of SMs, which take 256 rows.
// Row blocks of a head that are worked on side by side read each key tile
// from HBM once and from L2 after that, so a batch of several blocks wants
// them side by side; but `width` must leave few units idle (units / width
// groups) and few blocks over in the last pass.  And the groups either share
// the line equally, cutting heads, or take whole heads, some groups staying
// idle.  The cost of a choice, in cycles, is that of the steps of the longest
// range and of the join.  A step takes a pair 600 cycles besides the tensor
// cores' 1,280 or, when all groups stream different tiles, their share of the
// HBM (64 KiB a group at 3.5 KB a cycle: 18.6 a group); a CTA 2,500 or that
// share, so that 128 CTAs with a head each are as fast as 152.  A join takes
// 5,000 and 0.75 for each partial row (written, read and summed by the next
// kernel).  Measured, cut / whole: 1 token x 777 rows x 128 heads 16.8 / 14.2
// us, 128 x 4096 x 128 65.5 / 54.2, 64 x 8192 x 128 93 / 93.5, 8 x 4096 x 64
// 31.7 / 45.4, 256 x 500 x 128 31.2 / 20.1.
Plan plan(int num_tokens, int num_heads, int prefix_len, int sms) {
  Plan w;
  const bool pairs = num_tokens > kTile;
  // (the join gives each piece of a head a thread)
  const int units = min(pairs ? sms / 2 : sms, 32 * kCombineWarps), rows = num_tokens < 2 * kTile ? num_tokens : 2 * kTile;
  w.nk = (prefix_len + kTile - 1) / kTile;
  w.blocks = (num_tokens + 2 * kTile - 1) / (2 * kTile);
  double best = 0;
  bool any = false;
  auto take = [&](int width, int passes, long long groups, double cost) {
    if (any && cost >= 0.99 * best) return;
    any = true;
    best = cost;
    w.width = width;
    w.groups = static_cast<int>(groups);
    w.passes = passes;
  };
  auto step = [pairs](long long groups) {
    const double hbm = 18.6 * static_cast<double>(groups);
    return pairs ? 600.0 + fmax(1280.0, hbm) : fmax(2500.0, hbm);
  };
  for (int width = 1; width <= w.blocks && width <= units && width <= 16; ++width) {
    const int passes = (w.blocks + width - 1) / width;
    const long long heads = static_cast<long long>(passes) * num_heads, line = heads * w.nk;
    const long long most = units / width, whole = (heads + most - 1) / most;  // heads a group
    if (w.nk == 1) {  // heads of a single tile cannot be cut
      const long long groups = most < heads ? most : heads;
      take(width, passes, groups, static_cast<double>(whole) * step(groups));
      continue;
    }
    if (heads % whole == 0)
      take(width, passes, heads / whole, static_cast<double>(whole * w.nk) * step(heads / whole));
    // at least two steps a range, one for each stream
    const long long groups = most < (line + 1) / 2 ? most : (line + 1) / 2;
    take(width, passes, groups, static_cast<double>((line + groups - 1) / groups) * step(groups) + 5000.0 +
             0.75 * static_cast<double>(groups * width * rows));
  }
  w.line = static_cast<long long>(w.passes) * num_heads * w.nk;
  return w;
}

// Heads are cut wherever a range does not end with one (one of a single tile cannot be).
bool cuts_heads(const Plan& w) { return w.nk > 1 && (w.line / w.nk) % w.groups != 0; }

struct AttendWs {
  size_t lse, total;
  int rows;  // of a unit's two partial tiles
};
AttendWs attend_ws(const Plan& w, int num_tokens) {
  AttendWs l;
  l.rows = num_tokens < 2 * kTile ? num_tokens : 2 * kTile;
  const size_t slots = cuts_heads(w) ? 2 * static_cast<size_t>(w.groups) * w.width * l.rows : 0;
  l.lse = align256(slots * kHeadDim * sizeof(float));
  l.total = l.lse + align256(slots * sizeof(float));
  return l;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_prefix_attend_workspace_size(int num_tokens, int num_heads, int prefix_len, int* err) {
  int sms = 0;
  int rc = num_tokens < 0 || prefix_len < 0 ? MLA_ERR_INVALID_ARG
           : num_heads < 1 || num_heads > kHeads || num_tokens > kMaxRows || prefix_len > kMaxRows
               ? MLA_ERR_UNSUPPORTED
               : attend_device_ready(&sms);
  if (err) *err = rc;
  if (rc != MLA_OK) return 0;
  if (num_tokens == 0 || prefix_len == 0) return 0;
  return attend_ws(plan(num_tokens, num_heads, prefix_len, sms), num_tokens).total;
}

int mla_prefix_attend(const void* q_nope, const void* q_pe, int64_t q_stride, const void* k_nope, const void* v,
                      int64_t head_rows, const void* k_pe, int prefix_len, const int32_t* visible, int num_tokens,
                      int num_heads, float softmax_scale, const void* suffix_out, const float* suffix_lse,
                      unsigned flags, void* workspace, size_t ws_bytes, void* out, float* lse, int* status,
                      mla_stream_t stream) {
  if (!q_nope || !q_pe || !out || !lse || !status) return MLA_ERR_INVALID_ARG;
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
  if (head_rows > kMaxRows || num_tokens > kMaxRows || static_cast<int64_t>(num_tokens) * num_heads > INT32_MAX)
    return MLA_ERR_UNSUPPORTED;
  int sms = 0;
  int rc = attend_device_ready(&sms);
  if (rc != MLA_OK) return rc;
  const size_t need = mla_prefix_attend_workspace_size(num_tokens, num_heads, prefix_len, nullptr);
  if (need > 0 && !workspace) return MLA_ERR_INVALID_ARG;
  if (ws_bytes < need) return MLA_ERR_WORKSPACE;
  if (num_tokens == 0) return MLA_OK;
  AttendParams p = {};
  p.visible = visible;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.prefix_len = prefix_len;
  p.scale_log2 = softmax_scale * kLog2e;
  p.suffix_out = static_cast<const uint16_t*>(suffix_out);
  p.suffix_lse = suffix_lse;
  p.out_fp32 = (flags & MLA_FLAG_OUT_FP32) != 0;
  p.out = out;
  p.lse = lse;
  p.status = status;
  if (prefix_len == 0) {
    const long long threads = static_cast<long long>(num_tokens) * num_heads * (kHeadDim / 8);
    return launch_dependent(mla_prefix_empty_kernel, dim3(static_cast<unsigned>((threads + 127) / 128)), dim3(128), 0,
                            1, stream, p);
  }
  p.plan = plan(num_tokens, num_heads, prefix_len, sms);
  const AttendWs l = attend_ws(p.plan, num_tokens);
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.lse);
  p.part_rows = l.rows;
  const bool small = num_tokens <= kTile;
  const cuuint32_t half = kTile / 2;
  CUtensorMap qn, qp, k, kp, vm;
  const cuuint64_t pe_size[2] = {kRope, static_cast<cuuint64_t>(prefix_len)};
  const cuuint64_t pe_stride[1] = {kRope * 2};
  const cuuint32_t pe_box[2] = {kRope, small ? kTile : half};
  // boxes: keys {64 dims, 128 rows} or a rank's 64 of them; values {64 dims,
  // 64 rows, both chunks} or {64 dims, 128 rows} of a rank's chunk
  if (!encode_q(&qn, q_nope, kHeadDim, q_stride, num_heads, num_tokens) ||
      !encode_q(&qp, q_pe, kRope, q_stride, num_heads, num_tokens) ||
      !encode_kv(&k, false, k_nope, prefix_len, head_rows, num_heads, small ? kTile : half, 1) ||
      !encode(&kp, false, 2, k_pe, pe_size, pe_stride, pe_box) ||
      !encode_kv(&vm, true, v, prefix_len, head_rows, num_heads, small ? half : kTile, small ? 2 : 1))
    return MLA_ERR_CUDA;
  const int units = p.plan.groups * p.plan.width;
  rc = small ? launch_dependent(visible ? mla_prefix_attend_kernel<true> : mla_prefix_attend_kernel<false>, dim3(units),
                                dim3(kThreads), kSmem, 1, stream, p, qn, qp, k, kp, vm)
             : attend_pair_launch(units, stream, p, qn, qp, k, kp, vm);
  if (rc != MLA_OK || !cuts_heads(p.plan)) return rc;
  // pieces a head can be cut in: the ranges that overlap its nk steps
  const bool few = p.plan.nk / (p.plan.line / p.plan.groups) + 2 <= 8;
  const int rows = l.rows, block_rows = few ? kCombineWarps * kCombineRows : 1;
  return launch_dependent(few ? mla_prefix_combine_kernel<false> : mla_prefix_combine_kernel<true>,
                          dim3(few_units(p.plan, num_heads) ? p.plan.passes * num_heads : p.plan.groups - 1, p.plan.width,
                               (rows + block_rows - 1) / block_rows),
                          dim3(32 * kCombineWarps), 0, 1, stream, p);
}

}  // extern "C"
