// Ragged grouped product of 4-bit operands (MXFP4 x MXFP4, "W4A4"):
//   y[r, n] = sum_k xq[r, k] 2^(sx[r, k/32]) * wq[e, n, k] 2^(sw[e, n, k/32])
// for the rows r of expert e, E2M1 values, fp32 accumulation, 16-bit output.
// Segments and tiles as in ragged.cuh, weights in the MMA's M, tokens in its N.
//
// tcgen05.mma kind::mxf4.block_scale.scale_vec::2X takes both operands packed
// (two values a byte, K = 64 an instruction) and applies both operands' E8M0
// scales, so the whole reduction stays in one tensor-memory accumulator.
//
//  * warp 0: TMA producer, a ring of 256-deep steps (128 bytes a row),
//    and bulk copies of the step's scale operands into a slot of their own
//    barrier, so the scales' way into tensor memory runs ahead of the codes;
//  * warp 2: copies each slot into tensor memory (tcgen05.cp);
//  * warp 1: MMAs, four of K = 64 a step;
//  * warps 3-6: epilogue.
//  * Weight scales come packed as moe_mxfp4_pack_scales writes them, 512-byte
//    blocks of 128 rows x 128 columns in the form tcgen05.cp takes.  The
//    tokens' scales are brought into that form for this call's tiles by
//    k_pack_token_scales: segments begin at any row, and a block has to begin
//    at the tile's.  (Doing it beside the product would need a warp that
//    gathers 2 KB of scales every ~500 cycles.)
//  * A slot holds a 32-bit word (four scales, 128 of K) for each row: for two
//    such words an operand has two 16-column places in tensor memory, and MMA j
//    of a step takes word j / 2 and its bytes 2 (j % 2) and 2 (j % 2) + 1.
//  * every wait is bounded, as in ragged_one.cuh.
//
// Few rows are bound by the weights' 0.53 bytes a value: 512 rows, 64 experts,
// 7168 -> 4096, 1.0 GB: 180 us here and on SM pairs.  8192 rows, 8 experts, 4096 ->
// 28672: 478 us, bound by what an SM takes in from L2 (on pairs 377).
#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "pdl.cuh"
#include "ragged_maps.h"
#include "ragged_mx.cuh"

namespace moe {

namespace {

constexpr int BK = 256, STAGES = 4;
constexpr int A_BYTES = 128 * BK / 2;
constexpr int B_BYTES = 256 * BK / 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int SLOT_BYTES = 1024 + 2048;      // A: 2 words x 512; B: 2 words x up to 2 x 512
constexpr int SF_COL0 = 256;                 // scale places after the accumulator(s)
constexpr int SF_SLOT = 64;                  // A word 0, A word 1, B word 0, B word 1: 16 each
constexpr int TMEM_COLS = 512;
constexpr int NUM_THREADS = 224;
constexpr int SMEM_BYTES = STAGES * (STAGE_BYTES + SLOT_BYTES) + 1024 + 256 + kRagSchedBytes;
static_assert(SMEM_BYTES <= 232448, "shared memory");
static_assert(SF_COL0 + STAGES * SF_SLOT <= TMEM_COLS, "tensor memory");

__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// One block per token tile and trip: 16 bytes (4 rows' words) a thread.  Rows
// past the tile get 2^0: their columns are not stored.
template <int G>
__global__ void __launch_bounds__(256) k_pack_token_scales(const Mx44Args args) {
  __shared__ int s_mem[kRagSchedBytes / 4];
  __shared__ int s_scratch[kRagMaxExperts + 1];
  griddep_launch();
  griddep_wait();
  const RagSched sched = rag_sched_build<G>(args.r, s_mem, s_scratch);
  const int tiles = sched.tile0[sched.nseg];
  const int groups = tile_groups(args.r.tile_rows), kb_n = args.K / 128, KQ = args.K / 32;
  const int per_tile = kb_n * groups * 32;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const RagTile T = rag_tile<G>(sched, args.r, t);   // with w_tiles == 1: token tile t
    uint4* dst = reinterpret_cast<uint4*>(args.x_packed + T.tok * tile_scale_bytes(args.r.tile_rows, args.K));
    for (int i = threadIdx.x; i < per_tile; i += blockDim.x) {
      // neighbouring threads take neighbouring K words of one row
      const int kb = i % kb_n, l = (i / kb_n) % 32, g = i / (kb_n * 32);
      uint32_t w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int row = g * 128 + 32 * c + l;
        w[c] = row < T.rows
                   ? __ldg(reinterpret_cast<const uint32_t*>(args.x_scale + (size_t)(T.row0 + row) * KQ) + kb)
                   : 0x7F7F7F7Fu;
      }
      dst[(kb * groups + g) * 32 + l] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_ragged_mxfp4(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const Mx44Args margs) {
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

  if (args.splits == 1) griddep_launch();      // (pdl.cuh)
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4 * STAGES; ++s) mbar_init(bar_base + 8u * s, 1);
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    mbar_init(drain_bar, 1);
    mbar_init(cdrain_bar, 1);
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
  const int total = sched.tile0[sched.nseg] * args.w_tiles.d;
  const int groups = tile_groups(args.tile_rows);
  const int kb128 = margs.K / 128;
  // accumulators: two of 128 columns when tiles are no wider, else one of 256
  const int accs = groups == 1 ? 2 : 1;
  // the CTAs of a cluster share a tile (splits > 1: one tile each cluster)
  const int splits = args.splits;
  const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
  const int first = blockIdx.x / splits, stride = gridDim.x / splits;
  const int kb0 = args.num_kb * rank / splits, kb1 = args.num_kb * (rank + 1) / splits;

  auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {   // the whole warp
    return __all_sync(0xffffffffu,
                      mbar_wait_bounded(bar, parity, abort_flag, args.limit_ns, args.err));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol_w = l2_policy(0), pol_t = l2_policy(1);
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
    bool skip_first = args.never_arrive != 0;
    for (int t = first; t < total; t += stride) {
      const RagTile T = rag_tile<16>(sched, args, t);
      const int boxes = (T.rows + 31) / 32;
      const uint8_t* wsc = margs.w_packed +
                           ((size_t)T.e * kb128 * args.w_tiles.d + T.w_tile) * 512;
      const uint8_t* xsc = margs.x_packed + T.tok * tile_scale_bytes(args.tile_rows, margs.K);
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait(empty_bar(stage), phase ^ 1)) {
          ok = false;
          break;
        }
        if (skip_first) {
          skip_first = false;
        } else {
          const int words = min(2, kb128 - 2 * kb);
          const uint32_t slot = slot_base + stage * SLOT_BYTES;
          const uint32_t sa = smem_base + stage * STAGE_BYTES;
          if (elect_one()) {
            mbar_arrive_expect_tx(sfull_bar(stage), words * 512 * (1 + groups));
            for (int j = 0; j < words; ++j)
              bulk_load(slot + 512 * j, wsc + (size_t)(2 * kb + j) * args.w_tiles.d * 512, 512,
                        sfull_bar(stage));
            bulk_load(slot + 1024, xsc + (size_t)(2 * kb) * groups * 512, words * groups * 512,
                      sfull_bar(stage));
            mbar_arrive_expect_tx(full_bar(stage), A_BYTES + boxes * 32 * (BK / 2));
            tma_load_3d(sa, &tmA, full_bar(stage), kb * (BK / 2), T.w_tile * 128, T.e, pol_w);
            for (int j = 0; j < boxes; ++j)
              tma_load_2d(sa + A_BYTES + j * 32 * (BK / 2), &tmB, full_bar(stage), kb * (BK / 2),
                          T.row0 + 32 * j, pol_t);
          }
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
    }
    for (int s = 0; lane == 0 && s < STAGES; ++s)
      if (issued_mask & (1u << s)) {
        mbar_wait_bounded(full_bar(s), (issued_parity >> s) & 1, nullptr, args.limit_ns, args.err);
        mbar_wait_bounded(sfull_bar(s), (issued_parity >> s) & 1, nullptr, args.limit_ns, args.err);
      }
  } else if (warp == 2) {
    // ------------------------------------------------------------ scale copier
    // The place of slot s in tensor memory is free: the slot was refilled only
    // after the MMAs of its last step completed.
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += stride) {
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait(sfull_bar(stage), phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int words = min(2, kb128 - 2 * kb);
        const uint32_t src = slot_base + stage * SLOT_BYTES;
        const uint32_t dst = tmem_base + SF_COL0 + SF_SLOT * stage;
        if (elect_one()) {
          for (int j = 0; j < words; ++j) {
            tmem_cp_32x128b_x4(dst + 16 * j, sdesc_rows16(src + 512 * j));
            for (int g = 0; g < groups; ++g)
              tmem_cp_32x128b_x4(dst + 32 + 16 * j + 4 * g,
                                 sdesc_rows16(src + 1024 + (j * groups + g) * 512));
          }
          tc_commit(sready_bar(stage));
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (elect_one()) tc_commit(cdrain_bar);
    if (lane == 0) mbar_wait_bounded(cdrain_bar, 0, nullptr, args.limit_ns, args.err);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    int local = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += stride) {
      const int n = (rag_tile<16>(sched, args, t).rows + 15) / 16 * 16;
      const uint32_t id0 = make_idesc_block_scaled(kFmtMxf4, kFmtMxf4, 128, n, 0);
      const uint32_t id2 = make_idesc_block_scaled(kFmtMxf4, kFmtMxf4, 128, n, 2);
      const int acc = accs == 2 ? local & 1 : 0;
      const int use = accs == 2 ? local >> 1 : local;
      if (!warp_wait(tempty_bar(acc), (use & 1) ^ 1)) break;
      tc_fence_after();
      for (int kb = kb0; kb < kb1; ++kb) {
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
            umma_mxf4(tmem_base + acc * 128, adesc + 4 * j, bdesc + 4 * j, id0, sf + 16 * j,
                      sf + 32 + 16 * j, kb != kb0 || j != 0);
            umma_mxf4(tmem_base + acc * 128, adesc + 4 * j + 2, bdesc + 4 * j + 2, id2,
                      sf + 16 * j, sf + 32 + 16 * j, 1);
          }
          tc_commit(empty_bar(stage));
        }
        if (++stage == STAGES) {
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
  } else if (warp >= 3) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    int local = 0;
    for (int t = first; t < total; t += stride) {
      const RagTile V = rag_tile<16>(sched, args, t);
      const int acc = accs == 2 ? local & 1 : 0;
      const int use = accs == 2 ? local >> 1 : local;
      int ok = 0;
      if (lane == 0)
        ok = mbar_wait_bounded(tfull_bar(acc), use & 1, abort_flag, args.limit_ns, args.err);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 128;
      const int w = V.w_tile * 128 + q * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < V.rows; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(taddr + c, r);
        tmem_ld_wait();
        if (splits > 1) {
          rag_store_part(args, r, t, rank, c, V.rows, q * 32 + lane);
          continue;
        }
        rag_store_tokens32<T>(r, false, 0.0f,
                              static_cast<uint16_t*>(args.out) + (V.row0 + c) * args.ldo + w,
                              args.ldo, V.rows - c, w, args.W, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
      ++local;
    }
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
    cluster_sync();       // the cluster's sums are in the workspace
    if (first < total)
      rag_join_tokens<T, false>(args, rag_tile<16>(sched, args, first), first, rank, warp,
                                NUM_THREADS / 32, lane);
  }
}

template <typename T>
cudaError_t launch_mx(const CUtensorMap& tmA, const CUtensorMap& tmB, const Mx44Args& a, int grid,
                      cudaStream_t stream) {
  static DeviceOnce attr;
  const cudaError_t e = attr.call([] {
    return cudaFuncSetAttribute(k_ragged_mxfp4<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SMEM_BYTES);
  });
  if (e != cudaSuccess) return e;
  return launch_dependent(k_ragged_mxfp4<T>, grid, NUM_THREADS, SMEM_BYTES, stream, std::max(1, a.r.splits),
                          tmA, tmB, a);
}

}  // namespace

// Rows of the token tiles: at 128 and below two accumulators fit beside the
// scales' places, and a tile's end is hidden; long segments take wide tiles,
// which read the weights less often.
int ragged_mxfp4_tile_rows(int R, int E) { return R <= 64ll * E || R <= 128 ? 128 : 256; }

template <int G>
cudaError_t launch_pack_token_scales(const Mx44Args& args, long long most_tiles,
                                     cudaStream_t stream) {
  Mx44Args a = args;
  a.r.w_tiles = fast_div(1);          // tile numbers are token tiles
  return launch_dependent(k_pack_token_scales<G>, (unsigned)std::min<long long>(most_tiles, 4 * num_sms()),
                          256, 0, stream, 1, a);
}
template cudaError_t launch_pack_token_scales<32>(const Mx44Args&, long long, cudaStream_t);

constexpr int kLeastSteps = 4;     // of a slice of the reduction
int ragged_mxfp4_splits(int R, int N, int K, int E) {
  const int tr = ragged_mxfp4_tile_rows(R, E);
  const int segs = std::max(1, std::min(E, R));
  const long long even = segs * (((R + segs - 1) / segs + tr - 1ll) / tr) * (N / 128);
  return rag_slices(even, (K + BK - 1) / BK, kLeastSteps);
}
static size_t scale_bytes(int R, int K, int E) {
  const int tr = ragged_mxfp4_tile_rows(R, E);
  return (size_t)most_token_tiles(R, E, tr) * tile_scale_bytes(tr, K);
}
size_t ragged_mxfp4_bytes(int R, int N, int K, int E) {
  return scale_bytes(R, K, E) + rag_part_bytes(R, E, N / 128, (K + BK - 1) / BK, kLeastSteps,
                                               ragged_mxfp4_tile_rows(R, E));
}

cudaError_t launch_ragged_mxfp4(const RaggedProblem& p, const void* xq, const uint8_t* x_scale,
                                const void* wq, const void* w_scale_packed, void* y,
                                void* workspace, cudaStream_t stream) {
  CUtensorMap tmA, tmB;
  if (!make_tmap_rag_fp4(&tmA, wq, 3, p.K, p.N, p.E, 128) ||
      !make_tmap_rag_fp4(&tmB, xq, 2, p.K, p.R, 0, 32))
    return cudaErrorInvalidValue;
  Mx44Args a{};
  a.r.offsets = p.offsets;
  a.r.R = p.R;
  a.r.E = p.E;
  a.r.W = p.N;
  a.r.num_kb = (p.K + BK - 1) / BK;
  a.r.tile_rows = ragged_mxfp4_tile_rows(p.R, p.E);
  a.r.group_max = 8;
  a.r.out = y;
  a.r.ldo = p.ldy;
  watchdog_params(&a.r.limit_ns, &a.r.never_arrive);
  a.r.err = dev_error_word();
  if (a.r.err == nullptr) return cudaErrorInvalidDevice;
  a.x_scale = x_scale;
  a.w_packed = static_cast<const uint8_t*>(w_scale_packed);
  a.x_packed = static_cast<uint8_t*>(workspace);
  a.K = p.K;
  const long long tok = most_token_tiles(p.R, p.E, a.r.tile_rows);
  const cudaError_t e = launch_pack_token_scales<16>(a, tok, stream);
  if (e != cudaSuccess) return e;
  a.r.w_tiles = fast_div(p.N / 128);
  a.r.splits = ragged_mxfp4_splits(p.R, p.N, p.K, p.E);
  a.r.part = reinterpret_cast<float*>(a.x_packed + scale_bytes(p.R, p.K, p.E));
  const int grid = a.r.splits > 1 ? (int)(tok * a.r.w_tiles.d) * a.r.splits
                                  : (int)std::min<long long>(num_sms(), tok * a.r.w_tiles.d);
  return p.half ? launch_mx<__half>(tmA, tmB, a, grid, stream)
                : launch_mx<__nv_bfloat16>(tmA, tmB, a, grid, stream);
}

}  // namespace moe
