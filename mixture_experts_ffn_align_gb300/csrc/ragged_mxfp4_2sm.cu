// Ragged grouped product of 4-bit operands on SM pairs (tcgen05 cta_group::2),
// for segments of many rows; the formula and the scales' way are in
// ragged_mxfp4.cu, which is the one-SM form.
//
//  * tiles of 256 weights x up to 256 tokens over a cluster of two CTAs.  At the
//    4-bit rate a one-SM tile of 128 x 256 takes in 51 KB a step of 256 in the
//    time of 512 MMA cycles, about twice what an SM gets from L2; a pair's CTA
//    takes 35 KB (its 128 weights, half of the tokens, and scales).
//  * each CTA's tensor memory holds the scales of its own 128 weights and of all
//    the tile's tokens; the leader's tcgen05.cp.cta_group::2 copies each CTA's
//    slot into its own tensor memory.  The scales come by tensor copies (blocks
//    of 128 words), whose completion may count on the leader's barrier.
//  * short segments (on average at most 64 rows): tiles of up to 128 tokens in
//    two accumulators in turn.
//  * else one accumulator of 256 columns, beside it the four slots' places: eight
//    epilogue warps first read it whole, as packed 16-bit pairs, hand it back,
//    and store while the next tile's MMAs run.
//  * fixed tile order, bounded waits and teardown as in ragged_gemm_2sm.cu.
//
// 8192 rows, 8 experts, 4096 -> 28672: 363 us in bursts, 377 in long runs (5.1
// PFLOP/s).  The tensor pipe is busy 55% of the time, for two reasons: a tile's MMAs
// wait for the one accumulator to be read, and a step of 512 cycles of MMAs takes
// in 35 KB, 70 bytes a cycle where an SM gets about 50 from L2.
#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "pdl.cuh"
#include "ragged_maps.h"
#include "ragged_mx.cuh"

namespace moe {

namespace {

constexpr int BK = 256, STAGES = 4;
constexpr int A_BYTES = 128 * BK / 2, B_BYTES = 128 * BK / 2;   // this CTA's halves
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int SMALL_BOX = 32 * BK / 2;
constexpr int SLOT_BYTES = 1024 + 2048;      // A: 2 words x 512; B: 2 words x 2 x 512
constexpr int SF_COL0 = 256, SF_SLOT = 64;   // A word 0, A word 1, B word 0, B word 1: 16 each
constexpr int TMEM_COLS = 512;
constexpr int EPI_WARP0 = 3, EPI_WARPS = 8;
constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int SMEM_BYTES = STAGES * (STAGE_BYTES + SLOT_BYTES) + 1024 + 256 + kRagSchedBytes;
static_assert(SMEM_BYTES <= 232448, "shared memory");
static_assert(SF_COL0 + STAGES * SF_SLOT <= TMEM_COLS, "tensor memory");

__device__ __forceinline__ void umma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

template <typename T>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_ragged_mxfp4_2sm(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmB32,
                       const __grid_constant__ CUtensorMap tmSA,
                       const __grid_constant__ CUtensorMap tmSB, const Mx44Args margs) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const RagArgs& args = margs.r;
  uint8_t* slots = smem + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(slots + STAGES * SLOT_BYTES);
  // full[S], empty[S], sfull[S], sready[S], tfull[2], tempty[2], drain, cdrain
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 4 * STAGES + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_sched = reinterpret_cast<int*>(slots + STAGES * SLOT_BYTES + 256);
  static_assert(8 * (4 * STAGES + 6) + 8 <= 256, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t smem_base = smem_u32(smem), slot_base = smem_u32(slots);
  const uint32_t bar_base = smem_u32(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto sfull_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + s); };
  auto sready_bar = [&](int s) { return bar_base + 8u * (3 * STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (4 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (4 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar_base + 8u * (4 * STAGES + 4);
  const uint32_t cdrain_bar = bar_base + 8u * (4 * STAGES + 5);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4 * STAGES; ++s) mbar_init(bar_base + 8u * s, 1);
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * EPI_WARPS);   // both CTAs' (leader's is used)
    }
    mbar_init(drain_bar, 1);
    mbar_init(cdrain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
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

  const RagSched sched = rag_sched_build<32>(args, s_sched, reinterpret_cast<int*>(smem));
  const int total = sched.tile0[sched.nseg] * args.w_tiles.d;
  const int kb128 = margs.K / 128;
  const int groups = tile_groups(args.tile_rows);
  // accumulators: two of 128 columns when tiles are no wider, else one of 256
  const bool twin = groups == 1;
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;   // this pair's tiles
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    return mbar_wait_bounded(bar, parity, abort_flag, args.limit_ns, args.err);
  };
  auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {   // the whole warp
    return __all_sync(0xffffffffu, wait(bar, parity));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producers
    const uint64_t pol_w = l2_policy(0), pol_t = l2_policy(1);
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
    bool skip_first = leader && args.never_arrive != 0;
    for (int t = first; t < total; t += stride) {
      const RagTile D = rag_tile<32>(sched, args, t);
      // this CTA's half of the tokens: one box of 128 rows, or one or two of 32
      const int own = (D.rows + 31) / 32 * 16;
      const int row0 = D.row0 + (leader ? 0 : own);
      const int b_bytes = own <= 64 ? (own + 31) / 32 * SMALL_BOX : B_BYTES;
      const int w0 = D.w_tile * 256 + rank * 128;
      bool ok = true;
      for (int kb = 0; kb < args.num_kb; ++kb) {
        if (!warp_wait(empty_bar(stage), phase ^ 1)) {
          ok = false;
          break;
        }
        if (skip_first) {
          skip_first = false;   // watchdog test: leave this stage unarmed
        } else {
          const uint32_t slot = slot_base + stage * SLOT_BYTES;
          const uint32_t sa = smem_base + stage * STAGE_BYTES;
          const uint32_t sbar = mapa_shared(sfull_bar(stage), 0);
          const uint32_t bar = mapa_shared(full_bar(stage), 0);
          const uint32_t sb = sa + A_BYTES;
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (elect_one()) {
            if (leader) {
              mbar_arrive_expect_tx(sfull_bar(stage), 2 * (1024 + 1024 * groups));
              mbar_arrive_expect_tx(full_bar(stage), 2 * (A_BYTES + b_bytes));
            }
            // the second word of a last step of 128 is not used
            tma_load_3d_pair(slot, &tmSA, sbar, 0, w0 / 128, D.e * kb128 + 2 * kb, pol_w);
            tma_load_2d_pair(slot + 1024, &tmSB, sbar, 0, (D.tok * kb128 + 2 * kb) * groups, pol_t);
            tma_load_3d_pair(sa, &tmA, bar, kb * (BK / 2), w0, D.e, pol_w);
            if (b_bytes == B_BYTES) {
              tma_load_2d_pair(sb, &tmB, bar, kb * (BK / 2), row0, pol_t);
            } else {
              tma_load_2d_pair(sb, &tmB32, bar, kb * (BK / 2), row0, pol_t);
              if (b_bytes > SMALL_BOX)
                tma_load_2d_pair(sb + SMALL_BOX, &tmB32, bar, kb * (BK / 2), row0 + 32, pol_t);
            }
          }
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
    }
    // tail wait, as in ragged_gemm_2sm.cu
    for (int s = 0; lane == 0 && s < STAGES; ++s)
      if ((issued_mask & (1u << s)) && !wait(empty_bar(s), (issued_parity >> s) & 1)) break;
    // the leader's barriers count both CTAs' copies
    if (leader)
      for (int s = 0; lane == 0 && s < STAGES; ++s)
        if (issued_mask & (1u << s)) {
          mbar_wait_bounded(full_bar(s), (issued_parity >> s) & 1, nullptr, args.limit_ns, args.err);
          mbar_wait_bounded(sfull_bar(s), (issued_parity >> s) & 1, nullptr, args.limit_ns,
                            args.err);
        }
  } else if (warp == 2 && leader) {
    // ------------------------------------------------------------ scale copier
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += stride) {
      for (int kb = 0; kb < args.num_kb; ++kb) {
        if (!warp_wait(sfull_bar(stage), phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t src = slot_base + stage * SLOT_BYTES;
        const uint32_t dst = tmem_base + SF_COL0 + SF_SLOT * stage;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tmem_cp_pair_32x128b_x4(dst + 16 * j, sdesc_rows16(src + 512 * j));
            tmem_cp_pair_32x128b_x4(dst + 32 + 16 * j, sdesc_rows16(src + 1024 + 512 * groups * j));
            if (!twin)
              tmem_cp_pair_32x128b_x4(dst + 36 + 16 * j, sdesc_rows16(src + 1536 + 1024 * j));
          }
          tc_commit_pair(sready_bar(stage), 0x1);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (elect_one()) tc_commit_pair(cdrain_bar, 0x1);
    if (lane == 0) mbar_wait_bounded(cdrain_bar, 0, nullptr, args.limit_ns, args.err);
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------ MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    int local = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += stride) {
      const int n = (rag_tile<32>(sched, args, t).rows + 31) / 32 * 32;
      const uint32_t id0 = make_idesc_block_scaled(kFmtMxf4, kFmtMxf4, 256, n, 0);
      const uint32_t id2 = make_idesc_block_scaled(kFmtMxf4, kFmtMxf4, 256, n, 2);
      const int acc = twin ? local & 1 : 0;
      const uint32_t d_tmem = tmem_base + 128 * acc;
      if (!warp_wait(tempty_bar(acc), ((twin ? local >> 1 : local) & 1) ^ 1)) break;
      tc_fence_after();
      for (int kb = 0; kb < args.num_kb; ++kb) {
        if (!warp_wait(full_bar(stage), phase) || !warp_wait(sready_bar(stage), phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = smem_base + stage * STAGE_BYTES;
        const uint64_t adesc = sdesc_k_sw128(sa), bdesc = sdesc_k_sw128(sa + A_BYTES);
        const uint32_t sf = tmem_base + SF_COL0 + SF_SLOT * stage;
        const int words = min(2, kb128 - 2 * kb);
        if (elect_one()) {
          for (int j = 0; j < words; ++j) {
            umma_mxf4_pair(d_tmem, adesc + 4 * j, bdesc + 4 * j, id0, sf + 16 * j, sf + 32 + 16 * j,
                           (kb | j) != 0);
            umma_mxf4_pair(d_tmem, adesc + 4 * j + 2, bdesc + 4 * j + 2, id2, sf + 16 * j,
                           sf + 32 + 16 * j, 1);
          }
          tc_commit_pair(empty_bar(stage), 0x3);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) tc_commit_pair(tfull_bar(acc), 0x3);
      ++local;
    }
    if (elect_one()) tc_commit_pair(drain_bar, 0x1);
    if (lane == 0) {
      mbar_wait_bounded(drain_bar, 0, nullptr, args.limit_ns, args.err);
      for (int a = 0; a < 2; ++a) {
        const int uses = twin ? (local + 1 - a) >> 1 : a == 0 ? local : 0;
        if (uses > 0 && !wait(tempty_bar(a), (uses - 1) & 1)) break;
      }
    }
  } else if (warp >= EPI_WARP0) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - EPI_WARP0) >> 2;   // 128 of the 256 columns
    int local = 0;
    for (int t = first; t < total; t += stride) {
      const RagTile D = rag_tile<32>(sched, args, t);
      int ok = 0;
      const int acc = twin ? local & 1 : 0;
      if (lane == 0) ok = wait(tfull_bar(acc), (twin ? local >> 1 : local) & 1);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (half + acc) * 128;
      const int live = D.rows - half * 128;
      uint32_t pk[64];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (32 * c < live) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + 32 * c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            pk[16 * c + j] = Half16<T>::pack(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar(acc), 0));
      ++local;
      const int w = D.w_tile * 256 + rank * 128 + q * 32 + lane;
      uint16_t* out = static_cast<uint16_t*>(args.out) + (D.row0 + half * 128) * args.ldo + w;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (32 * c < live)
          rag_store_packed32(pk + 16 * c, out + 32 * c * args.ldo, args.ldo, live - 32 * c, w,
                             args.W, lane);
    }
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

template <typename T>
cudaError_t launch_mx_pair(const CUtensorMap (&tm)[5], const Mx44Args& a, long long tiles,
                           cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  static DeviceOnce setup;
  static int max_pairs[kMaxDevices];
  const int dev = device_index();
  const cudaError_t es = setup.call([&] {
    cudaError_t e = cudaFuncSetAttribute(k_ragged_mxfp4_2sm<T>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(num_sms(), 1, 1);
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, k_ragged_mxfp4_2sm<T>, &cfg);
    if (e != cudaSuccess) return e;
    max_pairs[dev] = n;
    return cudaSuccess;
  });
  if (es != cudaSuccess) return es;
  if (max_pairs[dev] <= 0) return cudaErrorInvalidConfiguration;
  return launch_dependent(k_ragged_mxfp4_2sm<T>, 2 * (unsigned)std::min<long long>(max_pairs[dev], tiles),
                          NUM_THREADS, SMEM_BYTES, stream, 2, tm[0], tm[1], tm[4], tm[2], tm[3], a);
}

}  // namespace

cudaError_t launch_ragged_mxfp4_2sm(const RaggedProblem& p, const void* xq, const uint8_t* x_scale,
                                    const void* wq, const void* w_scale_packed, void* y,
                                    void* workspace, cudaStream_t stream) {
  const int tile_rows = ragged_mxfp4_tile_rows(p.R, p.E);
  const int groups = tile_groups(tile_rows);
  const long long tok = most_token_tiles(p.R, p.E, tile_rows);
  CUtensorMap tm[5];
  if (!make_tmap_rag_fp4(&tm[0], wq, 3, p.K, p.N, p.E, 128) ||
      !make_tmap_rag_fp4(&tm[1], xq, 2, p.K, p.R, 0, 128) ||
      !make_tmap_rag_fp4(&tm[4], xq, 2, p.K, p.R, 0, 32) ||
      !make_tmap_scale_blocks(&tm[2], w_scale_packed, 3, p.N / 128, (uint64_t)p.E * (p.K / 128), 1,
                              2) ||
      !make_tmap_scale_blocks(&tm[3], workspace, 2, (uint64_t)tok * (p.K / 128) * groups, 0,
                              2 * groups, 1))
    return cudaErrorInvalidValue;
  Mx44Args a{};
  a.r.offsets = p.offsets;
  a.r.R = p.R;
  a.r.E = p.E;
  a.r.W = p.N;
  a.r.num_kb = (p.K + BK - 1) / BK;
  a.r.tile_rows = tile_rows;
  a.r.group_max = 8;
  a.r.out = y;
  a.r.ldo = p.ldy;
  watchdog_params(&a.r.limit_ns, &a.r.never_arrive);
  a.r.err = dev_error_word();
  if (a.r.err == nullptr) return cudaErrorInvalidDevice;
  a.x_scale = x_scale;
  a.x_packed = static_cast<uint8_t*>(workspace);
  a.K = p.K;
  const cudaError_t e = launch_pack_token_scales<32>(a, tok, stream);
  if (e != cudaSuccess) return e;
  a.r.w_tiles = fast_div((p.N + 255) / 256);
  return p.half ? launch_mx_pair<__half>(tm, a, tok * a.r.w_tiles.d, stream)
                : launch_mx_pair<__nv_bfloat16>(tm, a, tok * a.r.w_tiles.d, stream);
}

}  // namespace moe
