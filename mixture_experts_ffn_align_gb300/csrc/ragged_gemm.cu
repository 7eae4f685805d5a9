// Ragged grouped products on one SM per tile (forward, dgrad, wgrad; the
// formulas and the tile cut are in ragged.cuh), bf16 or fp16 operands, fp32
// accumulation in tensor memory.
//
//  * persistent CTAs, one per SM; tiles of 128 weights x up to 256 tokens
//    (wgrad: 128 rows x 256 columns of one expert's dw);
//  * warp 0 lane 0: TMA producer into a ring of 64-deep steps.  The token
//    operand comes in boxes of 32 rows, only as many as the tile has, so a
//    decode step (a few rows an expert) moves little beside the weights;
//  * warp 1 lane 0: tcgen05.mma (M = 128, N = the tile's rows rounded up to 16,
//    K = 16) into one of two 256-column accumulators;
//  * warps 2-5: epilogue from the other accumulator.
//  * dgrad reads w[e] with the reduction along its rows: the same boxes in the
//    MMA's MN-major form, so no transposed copy of the weights exists.
//  * wgrad reduces over an expert's rows, both operands MN-major.  Its last
//    step ends inside the segment: the tensor maps it loads through are cut to
//    the expert's rows (k_ragged_maps below writes them), so the rows behind
//    come in as zeros, and an infinity or NaN of the next expert's rows
//    cannot enter a sum as 0 x inf.
//  * every wait is bounded (wall clock); on a timeout the kernel records the
//    error, drains its own copies and MMAs, frees tensor memory and returns.
#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "ragged.cuh"

namespace moe {

bool make_tmap_rag(CUtensorMap* map, const void* base, bool half, int rank, uint64_t d0,
                   uint64_t d1, uint64_t d2, uint64_t ld, uint32_t box1);

namespace {

constexpr int BK = 64, MAX_STAGES = 9;
constexpr int A_BYTES = 128 * BK * 2;
constexpr int RING_BYTES = 196608;
constexpr int TMEM_COLS = 512;
constexpr int NUM_THREADS = 192;
constexpr int SMEM_BYTES = RING_BYTES + 1024 + 256 + kRagSchedBytes;
static_assert(SMEM_BYTES <= 232448, "shared memory");
static_assert(8 * (2 * MAX_STAGES + 5) + 8 <= 256, "barrier area");

template <int OP, typename T>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_ragged(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
             const RagArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + RING_BYTES);
  // full[S], empty[S], tfull[2], tempty[2], drain
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * MAX_STAGES + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_sched = reinterpret_cast<int*>(smem + RING_BYTES + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t bar_base = smem_u32(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (MAX_STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * MAX_STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar_base + 8u * (2 * MAX_STAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (OP != RAG_WGRAD && warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(smem_u32(tmem_holder), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  const RagSched sched = rag_sched_build<16>(args, s_sched, reinterpret_cast<int*>(smem));
  int* s_cnt = s_sched + 4;     // wgrad: rows of each expert, over the table just built
  if (OP == RAG_WGRAD) {
    // the table lists experts with rows only; wgrad visits every expert
    int* by_e = reinterpret_cast<int*>(smem);
    for (int e = threadIdx.x; e < args.E; e += blockDim.x) by_e[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < sched.nseg; s += blockDim.x) by_e[sched.exp[s]] = sched.cnt[s];
    __syncthreads();
    for (int e = threadIdx.x; e < args.E; e += blockDim.x) s_cnt[e] = by_e[e];
    fence_proxy_async_smem();   // by_e lies where TMA writes next
    __syncthreads();
  }
  const int total = OP == RAG_WGRAD ? args.E * args.w_tiles * args.k_tiles
                                    : sched.tile0[sched.nseg] * args.w_tiles;
  const int stages = args.stages;
  const int stage_bytes = A_BYTES + (OP == RAG_WGRAD ? 256 : args.tile_rows) * BK * 2;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol_w = l2_policy(0);
    const uint64_t pol_t = l2_policy(1);     // tokens: re-read for every weight tile
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
    bool skip_first = args.never_arrive != 0;
    int last_e = -1;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      RagTile D{};
      RagWTile V{};
      const CUtensorMap *mdy = nullptr, *mx = nullptr;
      int kb_n = args.num_kb, boxes = 4;
      if (OP == RAG_WGRAD) {
        V = rag_wtile(args, t);
        kb_n = (s_cnt[V.e] + BK - 1) / BK;
        mdy = args.maps + 2 * V.e;
        mx = mdy + 1;
        if (V.e != last_e && kb_n > 0) {
          tensormap_acquire(mdy);
          tensormap_acquire(mx);
          last_e = V.e;
        }
      } else {
        D = rag_tile<16>(sched, args, t);
        boxes = (D.rows + 31) / 32;
      }
      bool ok = true;
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1, abort_flag, args.limit_ns, args.err)) {
          ok = false;
          break;
        }
        if (skip_first) {
          skip_first = false;   // watchdog test: leave this stage unarmed
        } else {
          const uint32_t sa = smem_base + stage * stage_bytes, sb = sa + A_BYTES;
          const uint32_t bar = full_bar(stage);
          if (OP == RAG_WGRAD) {
            mbar_arrive_expect_tx(bar, A_BYTES + 256 * BK * 2);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_2d(sa + j * 8192, mdy, bar, V.n_tile * 128 + 64 * j, kb * BK, pol_t);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tma_load_2d(sb + j * 8192, mx, bar, V.k_tile * 256 + 64 * j, kb * BK, pol_t);
          } else {
            mbar_arrive_expect_tx(bar, A_BYTES + boxes * 32 * BK * 2);
            if (OP == RAG_FWD) {
              tma_load_3d(sa, &tmA, bar, kb * BK, D.w_tile * 128, D.e, pol_w);
            } else {
              tma_load_3d(sa, &tmA, bar, D.w_tile * 128, kb * BK, D.e, pol_w);
              tma_load_3d(sa + 8192, &tmA, bar, D.w_tile * 128 + 64, kb * BK, D.e, pol_w);
            }
            for (int j = 0; j < boxes; ++j)
              tma_load_2d(sb + j * 32 * BK * 2, &tmB, bar, kb * BK, D.row0 + 32 * j, pol_t);
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
    for (int s = 0; s < stages; ++s)
      if (issued_mask & (1u << s))
        mbar_wait_bounded(full_bar(s), (issued_parity >> s) & 1, nullptr, args.limit_ns, args.err);
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t major = (OP != RAG_FWD ? kIdescAMn : 0u) | (OP == RAG_WGRAD ? kIdescBMn : 0u);
    constexpr uint32_t a_step = OP != RAG_FWD ? 128 : 2, b_step = OP == RAG_WGRAD ? 128 : 2;
    int stage = 0;
    uint32_t phase = 0;
    int local = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      int kb_n = args.num_kb, n = 256;
      if (OP == RAG_WGRAD) {
        kb_n = (s_cnt[rag_wtile(args, t).e] + BK - 1) / BK;
        if (kb_n == 0) continue;
      } else {
        n = (rag_tile<16>(sched, args, t).rows + 15) / 16 * 16;
      }
      const uint32_t idesc = make_idesc(Half16<T>::kFmt, Half16<T>::kFmt, 128, n) | major;
      const int acc = local & 1;
      if (!mbar_wait_bounded(tempty_bar(acc), ((local >> 1) & 1) ^ 1, abort_flag, args.limit_ns,
                             args.err))
        break;
      tc_fence_after();
      bool ok = true;
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!mbar_wait_bounded(full_bar(stage), phase, abort_flag, args.limit_ns, args.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = smem_base + stage * stage_bytes;
        const uint64_t adesc = OP != RAG_FWD ? sdesc_mn_sw128(sa) : sdesc_k_sw128(sa);
        const uint64_t bdesc = OP == RAG_WGRAD ? sdesc_mn_sw128(sa + A_BYTES)
                                               : sdesc_k_sw128(sa + A_BYTES);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)
          umma_f16(tmem_base + acc * 256, adesc + a_step * k, bdesc + b_step * k, idesc,
                   (kb | k) != 0);
        tc_commit(empty_bar(stage));
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      tc_commit(tfull_bar(acc));
      ++local;
    }
    tc_commit(drain_bar);
    mbar_wait_bounded(drain_bar, 0, nullptr, args.limit_ns, args.err);
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    int local = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      RagTile D{};
      RagWTile V{};
      bool empty = false;
      if (OP == RAG_WGRAD) {
        V = rag_wtile(args, t);
        empty = s_cnt[V.e] == 0;
        if (empty && args.accumulate) continue;
      } else {
        D = rag_tile<16>(sched, args, t);
      }
      const int acc = local & 1;
      if (!empty) {
        int ok = 0;
        if (lane == 0)
          ok = mbar_wait_bounded(tfull_bar(acc), (local >> 1) & 1, abort_flag, args.limit_ns,
                                 args.err);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
      if (OP == RAG_WGRAD) {
        const int n = V.n_tile * 128 + q * 32 + lane, k0 = V.k_tile * 256;
        const size_t at = ((size_t)V.e * args.N + n) * args.K + k0;
#pragma unroll 1
        for (int c = 0; c < 256 && k0 + c < args.K; c += 32) {
          uint32_t r[32];
          if (empty) {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = 0;
          } else {
            tmem_ld_32x32b_x32(taddr + c, r);
            tmem_ld_wait();
          }
          if (n >= args.N) continue;
          if (args.out_f32)
            rag_store_row32_f32(r, static_cast<float*>(args.out) + at + c, args.K - k0 - c,
                                args.accumulate);
          else
            rag_store_row32<T>(r, static_cast<uint16_t*>(args.out) + at + c, args.K - k0 - c,
                               args.accumulate);
        }
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
          rag_store_tokens32<T>(r, bias,
                                static_cast<uint16_t*>(args.out) + (D.row0 + c) * args.ldo + w,
                                args.ldo, D.rows - c, w, args.W, lane);
        }
      }
      if (!empty) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
        ++local;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// Tensor maps of dy and x cut to each expert's rows: the whole tensors' maps
// with the base moved to the expert's first row and the row count replaced.
// One warp per map; offsets clamped as in rag_sched_build.
__global__ void k_ragged_maps(const __grid_constant__ CUtensorMap tmDy,
                              const __grid_constant__ CUtensorMap tmX, const void* dy,
                              const void* x, long long ld_dy_bytes, long long ld_x_bytes,
                              const int32_t* offsets, int R, int E, CUtensorMap* maps) {
  const int id = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int e = id >> 1;
  if (e >= E) return;
  // first row: the largest clamped offset up to e, as the running maximum gives it
  int top = 0;
  for (int i = lane; i <= e; i += 32) top = max(top, min(max(offsets[i], 0), R));
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int end = max(top, min(max(offsets[e + 1], 0), R));
  const CUtensorMap* src = (id & 1) ? &tmX : &tmDy;
  CUtensorMap* dst = maps + id;
  reinterpret_cast<uint32_t*>(dst)[lane] = reinterpret_cast<const uint32_t*>(src)[lane];
  __syncwarp();
  if (lane == 0) {
    const char* base = static_cast<const char*>((id & 1) ? x : dy) +
                       (long long)top * ((id & 1) ? ld_x_bytes : ld_dy_bytes);
    const uint64_t m = reinterpret_cast<uint64_t>(dst);
    asm volatile("tensormap.replace.tile.global_address.global.b1024.b64 [%0], %1;" ::"l"(m),
                 "l"(reinterpret_cast<uint64_t>(base))
                 : "memory");
    asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(m),
                 "r"(max(end - top, 1))
                 : "memory");
    asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
  }
}

template <int OP, typename T>
cudaError_t launch_one(const CUtensorMap& tmA, const CUtensorMap& tmB, const RagArgs& a, int grid,
                       cudaStream_t stream) {
  static DeviceOnce attr;
  const cudaError_t e = attr.call([] {
    return cudaFuncSetAttribute(k_ragged<OP, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SMEM_BYTES);
  });
  if (e != cudaSuccess) return e;
  k_ragged<OP, T><<<grid, NUM_THREADS, SMEM_BYTES, stream>>>(tmA, tmB, a);
  return cudaGetLastError();
}
template <int OP>
cudaError_t launch_op(bool half, const CUtensorMap& tmA, const CUtensorMap& tmB, const RagArgs& a,
                      int grid, cudaStream_t stream) {
  return half ? launch_one<OP, __half>(tmA, tmB, a, grid, stream)
              : launch_one<OP, __nv_bfloat16>(tmA, tmB, a, grid, stream);
}

}  // namespace

size_t ragged_maps_bytes(int E) { return (size_t)E * 2 * sizeof(CUtensorMap); }

cudaError_t launch_ragged_maps(const RaggedProblem& p, const void* dy, const void* x,
                               void* workspace, cudaStream_t stream) {
  CUtensorMap tmDy, tmX;
  if (!make_tmap_rag(&tmDy, dy, p.half, 2, p.N, p.R, 0, p.ldy, 64) ||
      !make_tmap_rag(&tmX, x, p.half, 2, p.K, p.R, 0, p.ldx, 64))
    return cudaErrorInvalidValue;
  k_ragged_maps<<<(2 * p.E + 7) / 8, 256, 0, stream>>>(tmDy, tmX, dy, x, p.ldy * 2, p.ldx * 2,
                                                       p.offsets, p.R, p.E,
                                                       static_cast<CUtensorMap*>(workspace));
  return cudaGetLastError();
}

cudaError_t launch_ragged_rows(const RaggedProblem& p, int op, const void* rows, const void* w,
                               const void* bias, void* out, cudaStream_t stream) {
  const bool fwd = op == RAG_FWD;
  CUtensorMap tmA, tmB;
  const int red = fwd ? p.K : p.N;
  if (!make_tmap_rag(&tmA, w, p.half, 3, p.K, p.N, p.E, p.K, fwd ? 128 : 64) ||
      !make_tmap_rag(&tmB, rows, p.half, 2, red, p.R, 0, fwd ? p.ldx : p.ldy, 32))
    return cudaErrorInvalidValue;
  RagArgs a{};
  a.offsets = p.offsets;
  a.R = p.R;
  a.E = p.E;
  a.W = fwd ? p.N : p.K;
  a.num_kb = (red + BK - 1) / BK;
  a.w_tiles = (a.W + 127) / 128;
  // token tiles no wider than the rows there are: a narrower ring stage leaves
  // room for more stages, and so for more weight bytes in flight
  a.tile_rows = p.R <= 32 ? 32 : p.R <= 64 ? 64 : p.R <= 128 ? 128 : 256;
  a.stages = std::min(MAX_STAGES, RING_BYTES / (A_BYTES + a.tile_rows * BK * 2));
  a.group_max = 8;
  a.out = out;
  a.ldo = fwd ? p.ldy : p.ldx;
  a.bias = bias;
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  const long long most =
      ((long long)std::min(p.E, p.R) + p.R / a.tile_rows) * a.w_tiles;   // tiles at most
  const int grid = (int)std::min<long long>(num_sms(), most);
  return fwd ? launch_op<RAG_FWD>(p.half, tmA, tmB, a, grid, stream)
             : launch_op<RAG_DGRAD>(p.half, tmA, tmB, a, grid, stream);
}

cudaError_t launch_ragged_wgrad(const RaggedProblem& p, const void* maps, void* dw, bool out_f32,
                                bool accumulate, cudaStream_t stream) {
  RagArgs a{};
  a.offsets = p.offsets;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.K = p.K;
  a.w_tiles = (p.N + 127) / 128;
  a.k_tiles = (p.K + 255) / 256;
  a.tile_rows = 256;
  a.stages = RING_BYTES / (A_BYTES + 256 * BK * 2);
  a.group_max = 8;
  a.out = dw;
  a.out_f32 = out_f32;
  a.accumulate = accumulate;
  a.maps = static_cast<const CUtensorMap*>(maps);
  watchdog_params(&a.limit_ns, &a.never_arrive);
  a.err = dev_error_word();
  if (a.err == nullptr) return cudaErrorInvalidDevice;
  const long long tiles = (long long)p.E * a.w_tiles * a.k_tiles;
  const int grid = (int)std::min<long long>(num_sms(), tiles);
  CUtensorMap none{};
  return launch_op<RAG_WGRAD>(p.half, none, none, a, grid, stream);
}

}  // namespace moe
