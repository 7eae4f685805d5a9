// Ragged grouped products on SM pairs (tcgen05 cta_group::2): forward, dgrad
// and wgrad for segments of many rows (the formulas, the tile cut and the
// epilogue stores are in ragged.cuh; the one-SM form is ragged_one.cuh).
//
//  * a cluster of two CTAs computes 256 weights x up to 256 tokens (wgrad: 256
//    rows x 256 columns of one expert's dw).  Each CTA stages its own 128
//    weights and half of the tokens, 32 KB for a 64-deep step against 48 KB of
//    the one-SM form for the same work an SM; the tensor core reads the other
//    half of the tokens from the peer's shared memory.
//  * six stages a CTA; both CTAs' copies complete on the leader's barrier, the
//    leader's MMA warp issues M = 256, N = the tile's tokens rounded up to 32,
//    K = 16 into one of two accumulators, and its commits reach both CTAs.
//  * each CTA's epilogue warps drain their own 128 accumulator rows: four, or
//    eight where a tile has two accumulators' worth of work (double tiles) or its
//    output goes out through boxes in shared memory (wgrad).
//  * long segments: two weight tiles together against the same tokens (MT = 2,
//    512 x up to 256), one in each accumulator.  A step then takes in 48 KB for
//    1024 cycles of MMAs instead of 32 KB for 512: an SM gets some 50 to 56 bytes
//    a cycle from L2, so single tiles wait for their operands at full clock.
//  * wgrad's last step of a segment that ends inside the 16 rows of an
//    instruction: each CTA's copies complete on a barrier of its own, a further
//    warp zeroes the rows behind the segment and signals the leader's issuer.
//  * every wait is bounded; the final cluster barrier is reached by both CTAs
//    after their bounded loops, and after tail waits for every signal that the
//    peer sends to a barrier of this CTA: one that arrives at a CTA that has ended
//    is lost, or keeps its sender from ending.
//
// 8 experts of 1024 rows each, in short bursts: forward 4096 -> 28672 1050 us (1830
// TFLOP/s), dgrad 4096 -> 14336 533 us (1807), wgrad of the same 582 us (1654); in
// long runs at the power limit 1208, 607 and 658 us.  Forward of uneven segments
// (900 to 1100 rows) 1140 and 1313 us: tiles round up to 32 rows, and 5.9% of the
// MMAs' columns are no row's.
// wgrad of segments that end inside 16 rows (1025, 1030 or 1039) takes 677 us in
// bursts and 721 in long runs, of 1040 rows 604 and 679: the hand-off to the
// zeroing warp at each tile's end costs some 12% there, which more rows hide.
// wgrad without it is bound by what the SMs take in from L2: 64 bytes a cycle at
// the tensor cores' full rate.
#pragma once

#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "pdl.cuh"
#include "ragged.cuh"
#include "ragged_epi.cuh"
#include "ragged_maps.h"

namespace moe {

namespace {

constexpr int BK = 64, MAX_STAGES = 6;
constexpr int A_BYTES = 128 * BK * 2, B_BYTES = 128 * BK * 2;   // this CTA's halves
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int SMALL_BOX = 32 * BK * 2;
constexpr int TMEM_COLS = 512;
// Epilogue warps: four; wgrad and the fused epilogues two for each quadrant of the
// accumulator's rows, a double tile four for each accumulator.
constexpr int epi_warps(int op, int mt, int epi) {
  return op == RAG_WGRAD || epi != EPI_PLAIN ? 8 : 4 * mt;
}
// producer, MMA, epilogue warps; wgrad has one more, which zeroes
constexpr int num_threads(int op, int mt, int epi) {
  return 64 + 32 * epi_warps(op, mt, epi) + (op == RAG_WGRAD ? 32 : 0);
}
constexpr int BAR_BYTES = 256;
constexpr int BOXES = 1;                      // store boxes of each epilogue warp (wgrad)
static_assert(epi_warps(RAG_WGRAD, 1, EPI_PLAIN) * BOXES * 4096 <= STAGE_BYTES, "store boxes");
constexpr int SMEM_BYTES = MAX_STAGES * STAGE_BYTES + 1024 + BAR_BYTES + kRagSchedBytes;
static_assert(SMEM_BYTES <= 232448, "shared memory");

// tmC: forward and dgrad: the tokens in boxes of 32 rows; wgrad: the output.
// MT: tiles of 256 weights that a pair computes together (forward, dgrad).
template <int OP, typename T, int MT, int EPI>
__global__ void __launch_bounds__(num_threads(OP, MT, EPI), 1)
    k_ragged_2sm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmC, const RagArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + MAX_STAGES * STAGE_BYTES);
  // full[S], empty[S], tail[S], zeroed[S], tfull[2], tempty[2], drain
  constexpr int NBARS = 4 * MAX_STAGES + 5;
  static_assert(8 * NBARS + 8 <= BAR_BYTES, "barrier area");
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_sched = reinterpret_cast<int*>(smem + MAX_STAGES * STAGE_BYTES + BAR_BYTES);
  // a stage: MT x 16 KB of weights, 16 KB of tokens; wgrad gives one stage's
  // space to the store boxes
  constexpr int STEP_BYTES = MT * A_BYTES + B_BYTES;
  constexpr int STAGES = OP == RAG_WGRAD ? MAX_STAGES - 1 : MAX_STAGES * STAGE_BYTES / STEP_BYTES;
  constexpr int EPI_WARPS = epi_warps(OP, MT, EPI);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t bar_base = smem_u32(bars);
  const uint32_t box_base = smem_base + (MAX_STAGES - 1) * STAGE_BYTES;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto tail_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + s); };
  auto zeroed_bar = [&](int s) { return bar_base + 8u * (3 * STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (4 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (4 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar_base + 8u * (4 * STAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 3 * STAGES; ++s) mbar_init(bar_base + 8u * s, 1);
    for (int s = 0; s < STAGES; ++s) mbar_init(zeroed_bar(s), 2);   // one warp of each CTA
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      // an accumulator's warps in both CTAs (the leader's barrier is used)
      mbar_init(tempty_bar(a), MT == 2 ? 8 : 2 * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc_pair(smem_u32(tmem_holder), TMEM_COLS);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();        // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  RagSched sched{};
  if constexpr (EPI != EPI_DENSE)
    sched = rag_sched_build<32>(args, s_sched, reinterpret_cast<int*>(smem));
  const int2* s_rows = OP == RAG_WGRAD
                           ? rag_rows_by_expert(sched, args.E, s_sched, reinterpret_cast<int2*>(smem))
                           : nullptr;
  const int total = OP == RAG_WGRAD    ? args.E * args.e_tiles.d
                    : EPI == EPI_DENSE ? args.E * args.dense.e_tiles.d
                                       : sched.tile0[sched.nseg] * args.w_tiles.d;

  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    return mbar_wait_bounded(bar, parity, abort_flag, args.limit_ns, args.err);
  };
  auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {   // the whole warp
    return __all_sync(0xffffffffu, wait(bar, parity));
  };
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;   // this pair's tiles

  // wgrad's producer is one lane: the whole warp measured slower there (605
  // against 574 us in turn, in bursts: 8 experts of 1024 rows, 4096 x 14336), faster
  // in the others (68 against 81 us for 32 rows, 256 x 16384)
  constexpr bool LONE = OP == RAG_WGRAD;
  if (warp == 0 && (!LONE || lane == 0)) {
    // ------------------------------------------------------------ producers
    const uint64_t pol_w = l2_policy(0), pol_t = l2_policy(1);
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_parity = 0, tail_mask = 0, tail_parity = 0;
    bool skip_first = leader && args.never_arrive != 0;
    for (int t = first; t < total; t += stride) {
      RagTile D{};
      RagWTile V{};
      int kb_n = args.num_kb, row0, tail_kb = -1, b_bytes = B_BYTES, a_tiles = 1;
      if (OP == RAG_WGRAD) {
        V = rag_wtile(args, t);
        const int2 rows = s_rows[V.e];
        row0 = rows.x;
        kb_n = (rows.y + BK - 1) / BK;
        if (rows.y % 16) tail_kb = kb_n - 1;
      } else {
        D = rag_any_tile<EPI, 32>(sched, args, t);
        // this CTA's half of the token operand: one box of 128 rows, or as many
        // of 32 as it has (a decode step's few rows then move little beside the
        // weights)
        const int own = (D.rows + 31) / 32 * 16;
        row0 = D.row0 + (leader ? 0 : own);
        if (own <= 64) b_bytes = (own + 31) / 32 * SMALL_BOX;
        a_tiles = rag_second_tile<MT>(args, D.w_tile) ? 2 : 1;
      }
      bool ok = true;
      // EPI_DENSE: hi x hi, hi x lo and lo x hi parts one after the other
      int seg = 0, seg_k = 0;
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!(LONE ? wait(empty_bar(stage), phase ^ 1) : warp_wait(empty_bar(stage), phase ^ 1))) {
          ok = false;
          break;
        }
        if (skip_first) {
          skip_first = false;   // watchdog test: leave this stage unarmed
        } else {
          const uint32_t sa = smem_base + stage * STEP_BYTES, sb = sa + MT * A_BYTES;
          uint32_t bar = mapa_shared(full_bar(stage), 0);
          const bool tail = OP == RAG_WGRAD && kb == tail_kb;
          if (tail) {
            // copies of a step to be zeroed behind: counted on this CTA's own barrier
            bar = mapa_shared(tail_bar(stage), rank);
            tail_parity ^= 1u << stage;     // bit: parity of the next use's phase
            tail_mask |= 1u << stage;
          }
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          const bool one = LONE || elect_one();
          if (one && tail) {
            if (leader) mbar_arrive(full_bar(stage));
            mbar_arrive_expect_tx(tail_bar(stage), STAGE_BYTES);
          } else if (one && leader) {
            mbar_arrive_expect_tx(full_bar(stage), 2 * (a_tiles * A_BYTES + b_bytes));
          }
          if (one && OP == RAG_WGRAD) {
            const int n0 = V.n_tile * 256 + rank * 128, k0 = V.k_tile * 256 + rank * 128;
            const int r0 = row0 + kb * BK;
            if (args.wide_a) {
              tma_load_4d_pair(sa, &tmA, bar, 0, r0, n0 / 64, 0, pol_t);
            } else {
              tma_load_2d_pair(sa, &tmA, bar, n0, r0, pol_t);
              tma_load_2d_pair(sa + 8192, &tmA, bar, n0 + 64, r0, pol_t);
            }
            if (args.wide_b) {
              tma_load_4d_pair(sb, &tmB, bar, 0, r0, k0 / 64, 0, pol_t);
            } else {
              tma_load_2d_pair(sb, &tmB, bar, k0, r0, pol_t);
              tma_load_2d_pair(sb + 8192, &tmB, bar, k0 + 64, r0, pol_t);
            }
          } else if (one) {
            const int k0 = (EPI == EPI_DENSE ? seg_k : kb) * BK;
            const int a_lo = seg == 1 ? args.dense.a_lo : 0, b_lo = seg == 2 ? args.dense.b_lo : 0;
            for (int i = 0; i < a_tiles; ++i) {
              const int w0 = (D.w_tile * MT + i) * 256 + rank * 128;
              const uint32_t s_a = sa + i * A_BYTES;
              if (EPI == EPI_GATED) {
                tma_load_5d_pair(s_a, &tmA, bar, k0, w0 / 16, D.e, pol_w);
              } else if (OP == RAG_FWD) {
                tma_load_3d_pair(s_a, &tmA, bar, k0 + a_lo, w0, D.e, pol_w);
              } else if (args.wide_a) {
                tma_load_4d_pair(s_a, &tmA, bar, 0, k0, (w0 + a_lo) / 64, D.e, pol_w);
              } else {
                tma_load_3d_pair(s_a, &tmA, bar, w0, k0, D.e, pol_w);
                tma_load_3d_pair(s_a + 8192, &tmA, bar, w0 + 64, k0, D.e, pol_w);
              }
            }
            if (b_bytes == B_BYTES) {
              tma_load_2d_pair(sb, &tmB, bar, k0 + b_lo, row0, pol_t);
            } else {
              tma_load_2d_pair(sb, &tmC, bar, k0 + b_lo, row0, pol_t);
              if (b_bytes > SMALL_BOX)
                tma_load_2d_pair(sb + SMALL_BOX, &tmC, bar, k0 + b_lo, row0 + 32, pol_t);
            }
          }
        }
        if (EPI == EPI_DENSE && ++seg_k == args.dense.seg_kb) {
          seg_k = 0;
          ++seg;
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
    }
    // tail wait: the leader's commits signal this CTA's barriers, and nothing else
    // waits for the last ones; they have to land before the CTA ends
    for (int s = 0; lane == 0 && s < STAGES; ++s)
      if ((issued_mask & (1u << s)) && !wait(empty_bar(s), (issued_parity >> s) & 1)) break;
    // the leader's barrier counts both CTAs' copies: once its issued phases
    // (and the own barrier's) complete, every copy has landed
    for (int s = 0; lane == 0 && s < STAGES; ++s) {
      if (leader && (issued_mask & (1u << s)))
        mbar_wait_bounded(full_bar(s), (issued_parity >> s) & 1, nullptr, args.limit_ns, args.err);
      if (tail_mask & (1u << s))
        mbar_wait_bounded(tail_bar(s), ((tail_parity >> s) & 1) ^ 1, nullptr, args.limit_ns,
                          args.err);
    }
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t major = (OP != RAG_FWD ? kIdescAMn : 0u) | (OP == RAG_WGRAD ? kIdescBMn : 0u);
    constexpr uint32_t a_step = OP != RAG_FWD ? 128 : 2, b_step = OP == RAG_WGRAD ? 128 : 2;
    int stage = 0;
    uint32_t phase = 0, tail_parity = 0;
    int local = 0, second = 0;     // tiles so far, and those with a second half
    // rows of tile t (wgrad: of its expert); the next tile's are looked up while
    // this one's MMAs run
    bool two_next = false;        // the next tile's second half exists (MT == 2)
    auto rows_of = [&](int t) -> int {
      if (t >= total) return 0;
      if (OP == RAG_WGRAD) return s_rows[rag_wtile(args, t).e].y;
      const RagTile D = rag_any_tile<EPI, 32>(sched, args, t);
      two_next = rag_second_tile<MT>(args, D.w_tile);
      return D.rows;
    };
    int rows_next = rows_of(first);
    for (int t = first; t < total; t += stride) {
      const int cnt = rows_next;
      const bool two = two_next;
      const int kb_n = OP == RAG_WGRAD ? (cnt + BK - 1) / BK : args.num_kb;
      const int n = OP == RAG_WGRAD ? 256 : (cnt + 31) / 32 * 32;
      if (kb_n == 0) {
        rows_next = rows_of(t + stride);
        continue;
      }
      const uint32_t idesc = make_idesc(Half16<T>::kFmt, Half16<T>::kFmt, 256, n) | major;
      // one tile in turn in the two accumulators, or a double tile in both
      const int acc = MT == 2 ? 0 : local & 1;
      const uint32_t acc_phase = (MT == 2 ? local : local >> 1) & 1;
      if (!warp_wait(tempty_bar(acc), acc_phase ^ 1)) break;
      tc_fence_after();
      bool ok = true;
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!warp_wait(full_bar(stage), phase)) {
          ok = false;
          break;
        }
        const uint32_t sa = smem_base + stage * STEP_BYTES;
        int steps = BK / 16;
        if (OP == RAG_WGRAD && kb == kb_n - 1) {
          const int rem = cnt - kb * BK;
          steps = (rem + 15) / 16;
          if (rem % 16) {          // the rows behind the segment are zeros in both CTAs
            const uint32_t par = (tail_parity >> stage) & 1;
            tail_parity ^= 1u << stage;
            if (!__all_sync(0xffffffffu,
                            mbar_wait_bounded<true>(zeroed_bar(stage), par, abort_flag,
                                                    args.limit_ns, args.err))) {
              ok = false;
              break;
            }
          }
        }
        tc_fence_after();
        const uint64_t adesc = OP != RAG_FWD ? sdesc_mn_sw128(sa) : sdesc_k_sw128(sa);
        const uint64_t bdesc = OP == RAG_WGRAD ? sdesc_mn_sw128(sa + A_BYTES)
                                               : sdesc_k_sw128(sa + MT * A_BYTES);
        const bool one = elect_one();
        if (one)
          for (int k = 0; k < steps; ++k)
            umma_f16_pair(tmem_base + acc * 256, adesc + a_step * k, bdesc + b_step * k, idesc,
                          (kb | k) != 0);
        if (MT == 2) {
          // the first half is complete while the second's last MMAs still run
          if (kb == kb_n - 1 && one) tc_commit_pair(tfull_bar(0), 0x3);
          if (two) {
            if (kb == 0) {
              if (!warp_wait(tempty_bar(1), (second & 1) ^ 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
            }
            if (one)
              for (int k = 0; k < steps; ++k)
                umma_f16_pair(tmem_base + 256, adesc + A_BYTES / 16 + a_step * k,
                              bdesc + b_step * k, idesc, (kb | k) != 0);
          }
        }
        if (one) tc_commit_pair(empty_bar(stage), 0x3);
        if (kb == 0) rows_next = rows_of(t + stride);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      const bool one = elect_one();
      if (MT == 1 && one) tc_commit_pair(tfull_bar(acc), 0x3);
      if (two) {
        if (one) tc_commit_pair(tfull_bar(1), 0x3);
        ++second;
      }
      ++local;
    }
    if (elect_one()) tc_commit_pair(drain_bar, 0x1);
    if (lane == 0) {
      mbar_wait_bounded(drain_bar, 0, nullptr, args.limit_ns, args.err);
      // tail wait: for the last signals of both CTAs' epilogues
      for (int a = 0; a < 2; ++a) {
        const int uses = MT == 1 ? (local + 1 - a) >> 1 : a == 0 ? local : second;
        if (uses > 0 && !wait(tempty_bar(a), (uses - 1) & 1)) break;
      }
    }
  } else if (OP == RAG_WGRAD && warp == 2 + EPI_WARPS) {
    // ------------------------------------------------------------ zeroing warp
    // As soon as the copies of a segment's last step have landed in this CTA,
    // well before the MMA issuer gets there (done by the issuer itself, the
    // round trip to the peer cost 2000 cycles a tile).
    int stage = 0;
    uint32_t tail_parity = 0;
    for (int t = first; t < total; t += stride) {
      const int cnt = s_rows[rag_wtile(args, t).e].y;
      const int kb_n = (cnt + BK - 1) / BK;
      if (cnt % 16) {
        const int s = (stage + kb_n - 1) % STAGES;      // stage of the last step
        const uint32_t par = (tail_parity >> s) & 1;
        tail_parity ^= 1u << s;
        if (!__all_sync(0xffffffffu, wait(tail_bar(s), par))) break;
        const int rem = cnt - (kb_n - 1) * BK;
        rag_zero_rows<4>(smem_base + s * STEP_BYTES, rem, (rem + 15) / 16 * 16, lane);
        if (lane == 0) mbar_arrive_cluster(mapa_shared(zeroed_bar(s), 0));
      }
      stage = (stage + kb_n) % STAGES;
    }
  } else if (MT == 2 && warp >= 2) {
    // ------------------------------------------------------------ epilogue, double tile
    // Four warps an accumulator.  Both are in use until a tile's end, so each
    // warp first reads its 32 x 256 sums as packed pairs of tokens, hands the
    // accumulator back, and stores while the next tile's MMAs run.  (With its 128
    // pairs a thread needs 12 words more than the 168 registers it can have.)
    const int q = warp & 3, half = (warp - 2) >> 2;
    int local = 0;
    for (int t = first; t < total; t += stride) {
      const RagTile D = rag_any_tile<EPI, 32>(sched, args, t);
      if (half == 1 && !rag_second_tile<MT>(args, D.w_tile)) continue;
      int ok = 0;
      if (lane == 0) ok = wait(tfull_bar(half), local & 1);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + half * 256;
      const int w = (D.w_tile * MT + half) * 256 + rank * 128 + q * 32 + lane;
      float bias = 0.0f;
      if (OP == RAG_FWD && args.bias != nullptr && w < args.W)
        bias = Half16<T>::value(static_cast<const uint16_t*>(args.bias)[(size_t)D.e * args.W + w]);
      uint32_t pk[128];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (32 * c < D.rows) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + 32 * c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            pk[16 * c + j] = Half16<T>::pack(__uint_as_float(r[2 * j]) + bias,
                                             __uint_as_float(r[2 * j + 1]) + bias);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar(half), 0));
      ++local;
      uint16_t* out = static_cast<uint16_t*>(args.out) + D.row0 * args.ldo + w;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (32 * c < D.rows)
          rag_store_packed32(pk + 16 * c, out + 32 * c * args.ldo, args.ldo, D.rows - 32 * c, w,
                             args.W, lane);
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    [[maybe_unused]] const bool clamp = args.gated.limit < __int_as_float(0x7f800000);
    int local = 0, turn = 0;
    for (int t = first; t < total; t += stride) {
      RagTile D{};
      RagWTile V{};
      bool empty = false;
      if (OP == RAG_WGRAD) {
        V = rag_wtile(args, t);
        empty = s_rows[V.e].y == 0;
        if (empty && args.accumulate) continue;
      } else {
        D = rag_any_tile<EPI, 32>(sched, args, t);
      }
      if (empty) {
        rag_zero_expert(args, V.e, 2 * (t - V.e * args.e_tiles.d) + rank, 2 * args.e_tiles.d,
                        threadIdx.x - 64, 32 * EPI_WARPS);
        continue;
      }
      const int acc = local & 1;
      // what the epilogue reads beside the sums, while they are computed
      [[maybe_unused]] Words16 next;
      [[maybe_unused]] const bool loads =
          (EPI == EPI_GATED_GRAD || (EPI == EPI_DENSE && args.dense.mat != nullptr));
      [[maybe_unused]] const int part = (warp - 2) >> 2;
      if constexpr (EPI == EPI_GATED_GRAD || EPI == EPI_DENSE) {
        const int w = D.w_tile * 256 + rank * 128 + q * 32 + lane;
        if (loads && 16 * part < D.rows) {
          if constexpr (EPI == EPI_DENSE)
            rag_dense_load(args, D, next, 16 * part, w, lane);
          else
            rag_gated_load(args, D, next, 16 * part, w, lane);
        }
      }
      int ok = 0;
      if (lane == 0) ok = wait(tfull_bar(acc), (local >> 1) & 1);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
      auto release = [&] {           // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        // carries no data through memory; the releasing form would wait for this
        // warp's output stores
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar(acc), 0));
        ++local;
      };
      if (OP == RAG_WGRAD) {
        const int half = (warp - 2) >> 2;
        rag_wgrad_epilogue<T, BOXES, 128>(args, &tmC, box_base + (warp - 2) * BOXES * 4096, turn,
                                          taddr + half * 128, V.e,
                                          V.n_tile * 256 + rank * 128 + q * 32,
                                          V.k_tile * 256 + half * 128, lane, release);
      } else if constexpr (EPI != EPI_PLAIN) {
        const int w = D.w_tile * 256 + rank * 128 + q * 32 + lane;
        float bias = 0.0f;
        if (EPI == EPI_GATED && args.bias != nullptr && w < args.W)
          bias = Half16<T>::value(
              static_cast<const uint16_t*>(args.bias)[(size_t)D.e * args.W +
                                                      ((w >> 3) & 1) * args.gated.inter +
                                                      gated_col(w)]);
        constexpr int STEP = 4 * EPI_WARPS;
#pragma unroll 1
        for (int c = 16 * part; c < D.rows; c += STEP) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(taddr + c, r);
          [[maybe_unused]] Words16 h;
          if constexpr (EPI != EPI_GATED) h = next;
          tmem_ld_wait();
          if constexpr (EPI == EPI_GATED) {
            if (clamp)
              rag_gated_tokens16<T, true>(args, r, bias, D.row0 + c, D.rows - c, w, lane);
            else
              rag_gated_tokens16<T, false>(args, r, bias, D.row0 + c, D.rows - c, w, lane);
          } else if constexpr (EPI == EPI_GATED_GRAD) {
            if (c + STEP < D.rows) rag_gated_load(args, D, next, c + STEP, w, lane);
            if (clamp)
              rag_gated_grad_tokens16<T, true>(args, r, h, D.row0 + c, D.rows - c, w, lane);
            else
              rag_gated_grad_tokens16<T, false>(args, r, h, D.row0 + c, D.rows - c, w, lane);
          } else {
            if (loads && c + STEP < D.rows) rag_dense_load(args, D, next, c + STEP, w, lane);
            // the symmetric products are the forward ones
            rag_dense_store16<OP == RAG_FWD>(args, D, r, h, loads, D.tok * args.dense.per + c,
                                             D.rows - c, w, lane);
          }
          __syncwarp();
        }
        release();
      } else {
        const int w = D.w_tile * 256 + rank * 128 + q * 32 + lane;
        float bias = 0.0f;
        if (OP == RAG_FWD && args.bias != nullptr && w < args.W)
          bias = Half16<T>::value(
              static_cast<const uint16_t*>(args.bias)[(size_t)D.e * args.W + w]);
#pragma unroll 1
        for (int c = 0; c < D.rows; c += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + c, r);
          tmem_ld_wait();
          rag_store_tokens32<T>(r, OP == RAG_FWD && args.bias != nullptr, bias,
                                static_cast<uint16_t*>(args.out) + (D.row0 + c) * args.ldo + w,
                                args.ldo, D.rows - c, w, args.W, lane);
        }
        release();
      }
    }
    if (OP == RAG_WGRAD && lane == 0) tma_store_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {
    // after a timeout, give copies the other CTA may still have in flight
    // into this CTA's shared memory time to land before the pair exits
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

template <int OP, typename T, int MT, int EPI = EPI_PLAIN>
cudaError_t launch_pair(const CUtensorMap& tmA, const CUtensorMap& tmB,
                      const CUtensorMap& tmC, const RagArgs& a,
                        long long tiles, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(num_threads(OP, MT, EPI), 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  static DeviceOnce setup;
  static int max_pairs[kMaxDevices];
  const int dev = device_index();
  const cudaError_t es = setup.call([&] {
    cudaError_t e = cudaFuncSetAttribute(k_ragged_2sm<OP, T, MT, EPI>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(num_sms(), 1, 1);
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, k_ragged_2sm<OP, T, MT, EPI>, &cfg);
    if (e != cudaSuccess) return e;
    max_pairs[dev] = n;
    return cudaSuccess;
  });
  if (es != cudaSuccess) return es;
  if (max_pairs[dev] <= 0) return cudaErrorInvalidConfiguration;
  return launch_dependent(k_ragged_2sm<OP, T, MT, EPI>, 2 * (unsigned)std::min<long long>(max_pairs[dev], tiles),
                          num_threads(OP, MT, EPI), SMEM_BYTES, stream, 2, tmA, tmB, tmC, a);
}
inline bool pair_args(const RaggedProblem& p, RagArgs& a) {
  a.offsets = p.offsets;
  a.R = p.R;
  a.E = p.E;
  a.tile_rows = 256;
  a.group_max = 8;
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  return a.err != nullptr;
}

}  // namespace

}  // namespace moe
