// Ragged grouped products on one SM per tile (forward, dgrad, wgrad; the
// formulas and the tile cut are in ragged.cuh), bf16 or fp16 operands, fp32
// accumulation in tensor memory.
//
//  * persistent CTAs, one per SM; tiles of 128 weights x up to 256 tokens
//    (wgrad: 128 rows x 256 columns of one expert's dw);
//  * warp 0: TMA producer into a ring of 64-deep steps.  The token
//    operand comes in boxes of 32 rows, only as many as the tile has, so a
//    decode step (a few rows an expert) moves little beside the weights;
//  * warp 1: tcgen05.mma (M = 128, N = the tile's rows rounded up to 16,
//    K = 16) into one of two 256-column accumulators.  Both warps run their loops
//    whole and issue from an elected lane: a loop inside a one-lane branch took
//    some 600 cycles a step to issue four MMAs;
//  * warps 2-5 (wgrad 2-9): epilogue from the other accumulator.
//  * dgrad reads w[e] with the reduction along its rows: the same boxes in the
//    MMA's MN-major form, so no transposed copy of the weights exists.
//  * wgrad reduces over an expert's rows, both operands MN-major.  Its last
//    step may end inside the 16 rows of an instruction: a further
//    warp then writes zeros over the rows behind the segment in both operands
//    (in one alone, an infinity or NaN of the next expert's rows would enter the
//    sums as 0 x inf).
//  * fewer tiles than half the SMs (few experts, narrow outputs): a cluster of
//    2, 4 or 8 CTAs takes one tile, each a slice of the reduction; the fp32 sums
//    go to the workspace (they stay in L2), and after a cluster barrier each CTA
//    adds and rounds its share of the tile's tokens (wgrad: rows), in the order
//    of the slices.
//  * every wait is bounded (wall clock); on a timeout the kernel records the
//    error, drains its own copies and MMAs, frees tensor memory and returns.
//
// Few rows are bound by the weights' bytes: forward of 128 rows to 8 experts,
// 7168 -> 4096 a projection of 470 MB, runs at HBM's rate (8 experts of 28672 x
// 4096, 1.88 GB: 279 us, 6.8 TB/s); two rows of one small expert by launch and
// latency (4.6 us in a graph, 1.5 of them an empty kernel's).  wgrad of segments
// up to some 200 rows is bound by writing dw: 64 experts of 64 rows, 4096 x 4096
// (2.15 GB), 393 us, 5.5 TB/s (a plain fill of dw: 532 us).
#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "pdl.cuh"
#include "ragged.cuh"
#include "ragged_maps.h"

namespace moe {

namespace {

constexpr int BK = 64, MAX_STAGES = 9;
constexpr int A_BYTES = 128 * BK * 2;
constexpr int RING_BYTES = 196608, BAR_BYTES = 384;
// Epilogue warps: one for each quadrant of the accumulator's rows, wgrad two (of
// 128 columns each).
constexpr int epi_warps(int op) { return op == RAG_WGRAD ? 8 : 4; }
// producer, MMA, epilogue warps; wgrad has one more, which zeroes
constexpr int num_threads(int op) { return 64 + 32 * epi_warps(op) + (op == RAG_WGRAD ? 32 : 0); }
constexpr int TMEM_COLS = 512;
// wgrad: three stages and two store boxes for each epilogue warp, a tile's
// output, in the ring's space and 16 KB more.
constexpr int W_STAGES = 3, BOXES = 2;
constexpr int W_STAGE_BYTES = A_BYTES + 256 * BK * 2;
constexpr int OPERAND_BYTES = W_STAGES * W_STAGE_BYTES + epi_warps(RAG_WGRAD) * BOXES * 4096;
static_assert(OPERAND_BYTES >= RING_BYTES, "operand space");
constexpr int SMEM_BYTES = OPERAND_BYTES + 1024 + BAR_BYTES + kRagSchedBytes;
static_assert(SMEM_BYTES <= 232448, "shared memory");
static_assert(8 * (4 * MAX_STAGES + 5) + 8 <= BAR_BYTES, "barrier area");

template <int OP, typename T>
__global__ void __launch_bounds__(num_threads(OP), 1)
    k_ragged(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
             const __grid_constant__ CUtensorMap tmD, const RagArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OPERAND_BYTES);
  // full[S], empty[S], tfull[2], tempty[2], drain, tail[S], zeroed[S]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 4 * MAX_STAGES + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_sched = reinterpret_cast<int*>(smem + OPERAND_BYTES + BAR_BYTES);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t bar_base = smem_u32(bars);
  const uint32_t box_base = smem_base + W_STAGES * W_STAGE_BYTES;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (MAX_STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * MAX_STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar_base + 8u * (2 * MAX_STAGES + 4);
  auto tail_bar = [&](int s) { return bar_base + 8u * (2 * MAX_STAGES + 5 + s); };
  auto zeroed_bar = [&](int s) { return bar_base + 8u * (3 * MAX_STAGES + 5 + s); };

  if (args.splits == 1) griddep_launch();      // (pdl.cuh)
  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(tail_bar(s), 1);
      mbar_init(zeroed_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), epi_warps(OP));
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
    tmem_alloc(smem_u32(tmem_holder), TMEM_COLS);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  griddep_wait();
  const RagSched sched = rag_sched_build<16>(args, s_sched, reinterpret_cast<int*>(smem));
  const int2* s_rows = OP == RAG_WGRAD
                           ? rag_rows_by_expert(sched, args.E, s_sched, reinterpret_cast<int2*>(smem))
                           : nullptr;
  const int total = OP == RAG_WGRAD ? args.E * args.e_tiles.d
                                    : sched.tile0[sched.nseg] * args.w_tiles.d;
  const int stages = args.stages;
  // the CTAs of a cluster share a tile (splits > 1: one tile each cluster)
  const int splits = args.splits;
  const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
  const int first = blockIdx.x / splits, stride = gridDim.x / splits;
  // this CTA's steps [kb0, kb1) of a reduction of n
  auto slice0 = [&](int n) { return n * rank / splits; };
  auto slice1 = [&](int n) { return n * (rank + 1) / splits; };
  const int kb0 = slice0(args.num_kb), kb1 = slice1(args.num_kb);
  const int stage_bytes = A_BYTES + (OP == RAG_WGRAD ? 256 : args.tile_rows) * BK * 2;

  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    return mbar_wait_bounded(bar, parity, abort_flag, args.limit_ns, args.err);
  };
  auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {   // the whole warp
    return __all_sync(0xffffffffu, wait(bar, parity));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol_w = l2_policy(0);
    const uint64_t pol_t = l2_policy(1);     // tokens: re-read for every weight tile
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_parity = 0, tail_mask = 0, tail_parity = 0;
    bool skip_first = args.never_arrive != 0;
    for (int t = first; t < total; t += stride) {
      RagTile D{};
      RagWTile V{};
      int kb_n = kb1 - kb0, boxes = 4, row0 = 0, tail_kb = -1;
      if (OP == RAG_WGRAD) {
        V = rag_wtile(args, t);
        const int cnt = s_rows[V.e].y, n = (cnt + BK - 1) / BK;
        kb_n = slice1(n) - slice0(n);
        row0 = s_rows[V.e].x + slice0(n) * BK;
        if (cnt % 16 && slice1(n) == n) tail_kb = kb_n - 1;
      } else {
        D = rag_tile<16>(sched, args, t);
        boxes = (D.rows + 31) / 32;
      }
      bool ok = true;
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!warp_wait(empty_bar(stage), phase ^ 1)) {
          ok = false;
          break;
        }
        if (skip_first) {
          skip_first = false;   // watchdog test: leave this stage unarmed
        } else {
          const uint32_t sa = smem_base + stage * stage_bytes, sb = sa + A_BYTES;
          uint32_t bar = full_bar(stage);
          const bool one = elect_one();
          if (OP == RAG_WGRAD && kb == tail_kb) {
            // copies of a step to be zeroed behind: counted on their own barrier
            if (one) mbar_arrive(bar);
            bar = tail_bar(stage);
            tail_parity ^= 1u << stage;       // bit: parity of the next use's phase
            tail_mask |= 1u << stage;
          }
          if (one && OP == RAG_WGRAD) {
            mbar_arrive_expect_tx(bar, A_BYTES + 256 * BK * 2);
            const int r0 = row0 + kb * BK;
            if (args.wide_a) {
              tma_load_4d(sa, &tmA, bar, 0, r0, V.n_tile * 2, 0, pol_t);
            } else {
              for (int j = 0; j < 2; ++j)
                tma_load_2d(sa + j * 8192, &tmA, bar, V.n_tile * 128 + 64 * j, r0, pol_t);
            }
            if (args.wide_b) {
              tma_load_4d(sb, &tmB, bar, 0, r0, V.k_tile * 4, 0, pol_t);
            } else {
              for (int j = 0; j < 4; ++j)
                tma_load_2d(sb + j * 8192, &tmB, bar, V.k_tile * 256 + 64 * j, r0, pol_t);
            }
          } else if (one) {
            mbar_arrive_expect_tx(bar, A_BYTES + boxes * 32 * BK * 2);
            const int k0 = (kb0 + kb) * BK;
            if (OP == RAG_FWD) {
              tma_load_3d(sa, &tmA, bar, k0, D.w_tile * 128, D.e, pol_w);
            } else if (args.wide_a) {
              tma_load_4d(sa, &tmA, bar, 0, k0, D.w_tile * 2, D.e, pol_w);
            } else {
              tma_load_3d(sa, &tmA, bar, D.w_tile * 128, k0, D.e, pol_w);
              tma_load_3d(sa + 8192, &tmA, bar, D.w_tile * 128 + 64, k0, D.e, pol_w);
            }
            for (int j = 0; j < boxes; ++j)
              tma_load_2d(sb + j * 32 * BK * 2, &tmB, bar, k0, D.row0 + 32 * j, pol_t);
          }
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
    }
    for (int s = 0; lane == 0 && s < stages; ++s) {
      if (issued_mask & (1u << s))
        mbar_wait_bounded(full_bar(s), (issued_parity >> s) & 1, nullptr, args.limit_ns, args.err);
      if (tail_mask & (1u << s))
        mbar_wait_bounded(tail_bar(s), ((tail_parity >> s) & 1) ^ 1, nullptr, args.limit_ns,
                          args.err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t major = (OP != RAG_FWD ? kIdescAMn : 0u) | (OP == RAG_WGRAD ? kIdescBMn : 0u);
    constexpr uint32_t a_step = OP != RAG_FWD ? 128 : 2, b_step = OP == RAG_WGRAD ? 128 : 2;
    int stage = 0;
    uint32_t phase = 0, tail_parity = 0;
    int local = 0;
    // rows of tile t (wgrad: of its expert); the next tile's are looked up while
    // this one's MMAs run
    auto rows_of = [&](int t) -> int {
      if (t >= total) return 0;
      return OP == RAG_WGRAD ? s_rows[rag_wtile(args, t).e].y : rag_tile<16>(sched, args, t).rows;
    };
    int rows_next = rows_of(first);
    for (int t = first; t < total; t += stride) {
      const int cnt = rows_next;
      const int all = (cnt + BK - 1) / BK;      // wgrad: steps of all slices
      const int kb_n = OP == RAG_WGRAD ? slice1(all) - slice0(all) : kb1 - kb0;
      const int n = OP == RAG_WGRAD ? 256 : (cnt + 15) / 16 * 16;
      if (kb_n == 0) {
        rows_next = rows_of(t + stride);
        continue;
      }
      const uint32_t idesc = make_idesc(Half16<T>::kFmt, Half16<T>::kFmt, 128, n) | major;
      const int acc = local & 1;
      if (!warp_wait(tempty_bar(acc), ((local >> 1) & 1) ^ 1)) break;
      tc_fence_after();
      bool ok = true;
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!warp_wait(full_bar(stage), phase)) {
          ok = false;
          break;
        }
        int steps = BK / 16;
        if (OP == RAG_WGRAD && slice0(all) + kb == all - 1) {
          const int rem = cnt - (all - 1) * BK;
          steps = (rem + 15) / 16;
          if (rem % 16) {               // the rows behind the segment are zeros
            const uint32_t par = (tail_parity >> stage) & 1;
            tail_parity ^= 1u << stage;
            if (!warp_wait(zeroed_bar(stage), par)) {
              ok = false;
              break;
            }
          }
        }
        tc_fence_after();
        const uint32_t sa = smem_base + stage * stage_bytes;
        const uint64_t adesc = OP != RAG_FWD ? sdesc_mn_sw128(sa) : sdesc_k_sw128(sa);
        const uint64_t bdesc = OP == RAG_WGRAD ? sdesc_mn_sw128(sa + A_BYTES)
                                               : sdesc_k_sw128(sa + A_BYTES);
        if (elect_one()) {
          for (int k = 0; k < steps; ++k)
            umma_f16(tmem_base + acc * 256, adesc + a_step * k, bdesc + b_step * k, idesc,
                     (kb | k) != 0);
          tc_commit(empty_bar(stage));
        }
        if (kb == 0) rows_next = rows_of(t + stride);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(tfull_bar(acc));
      ++local;
    }
    if (elect_one()) tc_commit(drain_bar);
    if (lane == 0) mbar_wait_bounded(drain_bar, 0, nullptr, args.limit_ns, args.err);
  } else if (OP == RAG_WGRAD && warp == 2 + epi_warps(OP)) {
    // ------------------------------------------------------------ zeroing warp
    int stage = 0;
    uint32_t tail_parity = 0;
    for (int t = first; t < total; t += stride) {
      const int cnt = s_rows[rag_wtile(args, t).e].y, n = (cnt + BK - 1) / BK;
      const int kb_n = slice1(n) - slice0(n);
      if (cnt % 16 && kb_n > 0 && slice1(n) == n) {
        const int s = (stage + kb_n - 1) % stages;      // stage of the last step
        const uint32_t par = (tail_parity >> s) & 1;
        tail_parity ^= 1u << s;
        if (!__all_sync(0xffffffffu, wait(tail_bar(s), par))) break;
        const int rem = cnt - (n - 1) * BK;
        rag_zero_rows<6>(smem_base + s * stage_bytes, rem, (rem + 15) / 16 * 16, lane);
        if (lane == 0) mbar_arrive(zeroed_bar(s));
      }
      stage = (stage + kb_n) % stages;
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    int local = 0, turn = 0;
    for (int t = first; t < total; t += stride) {
      RagTile D{};
      RagWTile V{};
      bool empty = false;
      if (OP == RAG_WGRAD) {
        V = rag_wtile(args, t);
        const int n = (s_rows[V.e].y + BK - 1) / BK;
        empty = slice1(n) == slice0(n);
        if (empty && (args.accumulate || splits > 1)) continue;
      } else {
        D = rag_tile<16>(sched, args, t);
      }
      if (empty) {
        rag_zero_expert(args, V.e, t - V.e * args.e_tiles.d, args.e_tiles.d, threadIdx.x - 64,
                        32 * epi_warps(OP));
        continue;
      }
      const int acc = local & 1;
      int ok = 0;
      if (lane == 0) ok = wait(tfull_bar(acc), (local >> 1) & 1);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
      auto release = [&] {           // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
        ++local;
      };
      if (OP == RAG_WGRAD) {
        const int half = (warp - 2) >> 2;
        if (splits > 1) {
          float* p = args.part + (((size_t)t * splits + rank) * 128 + q * 32 + lane) * 256 + half * 128;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(taddr + half * 128 + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(p + c + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
          }
          release();
          continue;
        }
        rag_wgrad_epilogue<T, BOXES, 128>(args, &tmD, box_base + (warp - 2) * BOXES * 4096, turn,
                                          taddr + half * 128, V.e,
                                          V.n_tile * 128 + q * 32, V.k_tile * 256 + half * 128,
                                          lane, release);
      } else {
        const int w = D.w_tile * 128 + q * 32 + lane;
        float bias = 0.0f;
        if (OP == RAG_FWD && args.bias != nullptr && w < args.W)
          bias = Half16<T>::value(
              static_cast<const uint16_t*>(args.bias)[(size_t)D.e * args.W + w]);
#pragma unroll 1
        for (int c = 0; c < D.rows; c += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + c, r);
          tmem_ld_wait();
          if (splits > 1) {
            rag_store_part(args, r, t, rank, c, D.rows, q * 32 + lane);
            continue;
          }
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
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
  if (splits > 1) {
    // join: the cluster's sums are in the workspace
    cluster_sync();
    constexpr int WARPS = num_threads(OP) / 32;
    if (OP == RAG_WGRAD && first < total) {
      // a lane takes eight columns of a row
      const RagWTile V = rag_wtile(args, first);
      const int steps = (s_rows[V.e].y + BK - 1) / BK, k = V.k_tile * 256 + 8 * lane;
      const float* p = args.part + (size_t)first * splits * 128 * 256 + 8 * lane;
      for (int j = rank * WARPS + warp; j < 128; j += splits * WARPS) {
        const int n = V.n_tile * 128 + j;
        if (n >= args.N || k >= args.K || (steps == 0 && args.accumulate)) continue;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
        for (int s = 0; s < splits; ++s) {
          if (steps * (s + 1) / splits == steps * s / splits) continue;   // nothing was summed
          const float4* v = reinterpret_cast<const float4*>(p + ((size_t)s * 128 + j) * 256);
          a = make_float4(a.x + v[0].x, a.y + v[0].y, a.z + v[0].z, a.w + v[0].w);
          b = make_float4(b.x + v[1].x, b.y + v[1].y, b.z + v[1].z, b.w + v[1].w);
        }
        const size_t at = ((size_t)V.e * args.N + n) * args.K + k;
        if (args.out_f32) {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(args.out) + at);
          if (args.accumulate) {
            const float4 x = d[0], y = d[1];
            a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
            b = make_float4(b.x + y.x, b.y + y.y, b.z + y.z, b.w + y.w);
          }
          d[0] = a;
          d[1] = b;
        } else {
          uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.out) + at);
          if (args.accumulate) {
            const uint4 o = *d;
            a = make_float4(a.x + Half16<T>::value((uint16_t)(o.x & 0xFFFFu)),
                            a.y + Half16<T>::value((uint16_t)(o.x >> 16)),
                            a.z + Half16<T>::value((uint16_t)(o.y & 0xFFFFu)),
                            a.w + Half16<T>::value((uint16_t)(o.y >> 16)));
            b = make_float4(b.x + Half16<T>::value((uint16_t)(o.z & 0xFFFFu)),
                            b.y + Half16<T>::value((uint16_t)(o.z >> 16)),
                            b.z + Half16<T>::value((uint16_t)(o.w & 0xFFFFu)),
                            b.w + Half16<T>::value((uint16_t)(o.w >> 16)));
          }
          *d = make_uint4(Half16<T>::pack(a.x, a.y), Half16<T>::pack(a.z, a.w),
                          Half16<T>::pack(b.x, b.y), Half16<T>::pack(b.z, b.w));
        }
      }
    }
    if (OP != RAG_WGRAD && first < total)
      rag_join_tokens<T, OP == RAG_FWD>(args, rag_tile<16>(sched, args, first), first, rank,
                                        warp, WARPS, lane);
  }
}

template <int OP, typename T>
cudaError_t launch_one(const CUtensorMap& tmA, const CUtensorMap& tmB,
                      const CUtensorMap& tmD, const RagArgs& a, int grid,
                       cudaStream_t stream) {
  static DeviceOnce attr;
  const cudaError_t e = attr.call([] {
    return cudaFuncSetAttribute(k_ragged<OP, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SMEM_BYTES);
  });
  if (e != cudaSuccess) return e;
  return launch_dependent(k_ragged<OP, T>, grid, num_threads(OP), SMEM_BYTES, stream,
                          std::max(1, a.splits), tmA, tmB, tmD, a);
}
template <int OP>
cudaError_t launch_op(bool half, const CUtensorMap& tmA, const CUtensorMap& tmB,
                      const CUtensorMap& tmD, const RagArgs& a,
                      int grid, cudaStream_t stream) {
  return half ? launch_one<OP, __half>(tmA, tmB, tmD, a, grid, stream)
              : launch_one<OP, __nv_bfloat16>(tmA, tmB, tmD, a, grid, stream);
}

}  // namespace

constexpr int kLeastSteps = 8;     // of a slice of a reduction

// Tiles and splits of the rows' products on one SM.
struct RowsPlan {
  int tile_rows, w_tiles, splits;
  long long tiles;      // at most, whatever the segments
};
static RowsPlan rows_plan(int R, int E, int width, int red) {
  RowsPlan r;
  // Token tiles of about twice the rows an expert has on average: a narrower
  // ring stage leaves room for more of them, and so for more weight bytes in
  // flight (256 experts of 64 rows, 7168 x 2048: dgrad 1188 us with 128 rows,
  // 1260 with 256); a longer segment takes more tiles.
  const int want = std::min(R, 2 * ((R + E - 1) / E));
  r.tile_rows = want <= 32 ? 32 : want <= 64 ? 64 : want <= 128 ? 128 : 256;
  r.w_tiles = (width + 127) / 128;
  r.tiles = ((long long)std::min(E, R) + R / r.tile_rows) * r.w_tiles;
  // Slices, by the tiles that even segments make (a 100 x 4096 x 4096 product of
  // one expert: 13 us in four slices, 28 us in one).  The grid and the workspace
  // take the tiles that any segments can make.
  const int segs = std::max(1, std::min(E, R));
  const long long even =
      segs * (((R + segs - 1) / segs + r.tile_rows - 1ll) / r.tile_rows) * r.w_tiles;
  r.splits = rag_slices(even, (red + BK - 1) / BK, kLeastSteps);
  return r;
}
int ragged_wgrad_splits(int R, int N, int K, int E) {
  return rag_slices((long long)E * ((N + 127) / 128) * ((K + 255) / 256), R / E / BK, kLeastSteps);
}
size_t ragged_wgrad_bytes(int R, int N, int K, int E) {
  const int s = ragged_wgrad_splits(R, N, K, E);
  return s > 1 ? (size_t)E * ((N + 127) / 128) * ((K + 255) / 256) * s * 128 * 256 * sizeof(float)
               : 0;
}
int ragged_rows_splits(int R, int E, int width, int red) {
  return rows_plan(R, E, width, red).splits;
}
size_t ragged_split_bytes(int R, int E, int width, int red) {
  const RowsPlan r = rows_plan(R, E, width, red);
  return rag_part_bytes(R, E, r.w_tiles, (red + BK - 1) / BK, kLeastSteps, r.tile_rows);
}

cudaError_t launch_ragged_rows(const RaggedProblem& p, int op, const void* rows, const void* w,
                               const void* bias, void* out, void* workspace,
                               cudaStream_t stream) {
  const bool fwd = op == RAG_FWD;
  CUtensorMap tmA, tmB;
  const int red = fwd ? p.K : p.N;
  const bool wide = !fwd && p.K % 64 == 0;
  if (!(wide ? make_tmap_rag_wide(&tmA, w, p.half, p.N, p.K, p.E, p.K, 2)
             : make_tmap_rag(&tmA, w, p.half, 3, p.K, p.N, p.E, p.K, fwd ? 128 : 64)) ||
      !make_tmap_rag(&tmB, rows, p.half, 2, red, p.R, 0, fwd ? p.ldx : p.ldy, 32))
    return cudaErrorInvalidValue;
  RagArgs a{};
  a.offsets = p.offsets;
  a.R = p.R;
  a.E = p.E;
  a.W = fwd ? p.N : p.K;
  a.num_kb = (red + BK - 1) / BK;
  const RowsPlan r = rows_plan(p.R, p.E, a.W, red);
  a.tile_rows = r.tile_rows;
  a.w_tiles = fast_div(r.w_tiles);
  a.splits = r.splits;
  a.part = static_cast<float*>(workspace);
  a.stages = std::min(MAX_STAGES, RING_BYTES / (A_BYTES + a.tile_rows * BK * 2));
  a.group_max = 8;
  a.wide_a = wide;
  a.out = out;
  a.ldo = fwd ? p.ldy : p.ldx;
  a.bias = bias;
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  const int grid = a.splits > 1 ? (int)r.tiles * a.splits
                                : (int)std::min<long long>(num_sms(), r.tiles);
  return fwd ? launch_op<RAG_FWD>(p.half, tmA, tmB, tmB, a, grid, stream)
             : launch_op<RAG_DGRAD>(p.half, tmA, tmB, tmB, a, grid, stream);
}

cudaError_t launch_ragged_wgrad(const RaggedProblem& p, const void* dy, const void* x, void* dw,
                                bool out_f32, bool accumulate, void* workspace,
                                cudaStream_t stream) {
  CUtensorMap tmA, tmB, tmD;
  const bool wide_a = p.N % 64 == 0, wide_b = p.K % 64 == 0;
  if (!(wide_a ? make_tmap_rag_wide(&tmA, dy, p.half, p.R, p.N, 1, p.ldy, 2)
               : make_tmap_rag(&tmA, dy, p.half, 2, p.N, p.R, 0, p.ldy, 64)) ||
      !(wide_b ? make_tmap_rag_wide(&tmB, x, p.half, p.R, p.K, 1, p.ldx, 4)
               : make_tmap_rag(&tmB, x, p.half, 2, p.K, p.R, 0, p.ldx, 64)) ||
      !make_tmap_rag_store(&tmD, dw, out_f32 ? 2 : p.half ? 1 : 0, p.K, p.N, p.E))
    return cudaErrorInvalidValue;
  RagArgs a{};
  a.offsets = p.offsets;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.K = p.K;
  a.w_tiles = fast_div((p.N + 127) / 128);
  a.k_tiles = fast_div((p.K + 255) / 256);
  a.e_tiles = fast_div(a.w_tiles.d * a.k_tiles.d);
  a.tile_rows = 256;
  a.stages = W_STAGES;
  a.wide_a = wide_a;
  a.wide_b = wide_b;
  a.out = dw;
  a.out_f32 = out_f32;
  a.accumulate = accumulate;
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  a.splits = ragged_wgrad_splits(p.R, p.N, p.K, p.E);
  a.part = static_cast<float*>(workspace);
  const long long tiles = (long long)p.E * a.e_tiles.d;
  const int grid = a.splits > 1 ? (int)tiles * a.splits
                                : (int)std::min<long long>(num_sms(), tiles);
  return launch_op<RAG_WGRAD>(p.half, tmA, tmB, tmD, a, grid, stream);
}

}  // namespace moe
