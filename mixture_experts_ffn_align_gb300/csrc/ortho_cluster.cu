// All steps of the orthogonalised update (orthogonalize.cu has the formulas) in one
// launch.  Two forms of one kernel:
//
// Clusters, for small matrices: a cluster of 1 to 8 CTAs takes a matrix and goes through
// the products A = X X^T, B = a I + b A + c A^2, X = B X of every step, with a cluster
// barrier between them.  Small products are bound by latency: as launches of their own
// they take 4.7 us each (a launch's end and start, cold instructions, the first copies),
// 15 of them for five steps; here 3.1 us, for the barrier, the first copies and the last
// tile's epilogue (8 x 64 x 64 in five steps: 78 and 57 us with the norm and the scaling).
// Matrices and sums stay in L2.
//
// The whole grid, for matrices of some tiles (GRID): the tiles of all products of all
// matrices stand in one order, step by step, product by product, matrix by matrix, and
// CTA i of n takes the tiles i, i + n, ...  A tile waits until its matrix's products
// before are finished, which it counts in the workspace; other matrices' tiles fill the
// time.  A tile waits for earlier ones only, every CTA goes through its own in order and
// all run at once (a cooperative launch), so the earliest unfinished tile can always go
// on.  Against launches of their own no launch's end is waited for and no partly filled
// round is left between products, only after the last: 8 x 1024 x 1024 313 and 238 us,
// 16 x 517 x 1031 270 and 213, 64 x 512 x 1024 677 and 548.  Long sums in few tiles (no
// slices here) and tiles of 256 x 256 on SM pairs stay ahead as launches of their own.
//
// orthogonalize.cu compares the forms by modelled cycles.
//
// Roles, tiles, epilogue and slices of a reduction are those of ragged_one.cuh's
// EPI_DENSE (128 columns x up to 256 rows, fp32 sums in tensor memory, slices joined
// through the workspace in their order).  What a product's epilogue writes, the next
// product's copies read through the asynchronous proxy: a proxy fence stands on both
// sides of the barrier or flag.  Every wait is bounded; a CTA whose wait ran out skips the
// rest of its work but keeps to the cluster's barriers.
#include <algorithm>

#include "dense_gemm.h"
#include "moe_common.cuh"
#include "ortho_cluster.h"
#include "pdl.cuh"
#include "ragged_epi.cuh"
#include "ragged_maps.h"

namespace moe {
namespace {

constexpr int BK = 64, MAX_STAGES = 9;
constexpr int A_BYTES = 128 * BK * 2, RING_BYTES = 196608, BAR_BYTES = 256;
// 12 over the whole grid measured 5% slower where sums are long (8 x 1536 x 1536: 639 and
// 607 us) and 6% faster where they are short (64 x 256 x 2048: 423 and 449); 16 spill.
// (8 take 168 registers, with 16 bytes spilled in clusters, 4 over the grid.)
constexpr int EPI_WARPS = 8;
// producer, MMA, epilogue warps; whole grid: one that tells it of finished tiles
constexpr int threads(bool grid) { return 64 + 32 * EPI_WARPS + (grid ? 32 : 0); }
constexpr int TMEM_COLS = 512;
constexpr int SMEM_BYTES = RING_BYTES + 1024 + BAR_BYTES;

// Orders this thread's generic accesses to global memory with the asynchronous ones.
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

struct Maps {
  CUtensorMap x_nt[2], x_mn[2], x_rows[2], a_nt, a_rows, b_rows;
};
struct Args {
  OrthoClusterPlan plan;
  int E, m, M, mp, Mp, parts, steps, transposed, kept;
  __half *x[2], *lo, *a, *b;
  __nv_bfloat16* out;
  float* part;
  uint32_t* done;
  float c_gram, c_apply, c_last;                 // c_acc of the products
  float coef[3 * MOE_MAX_ORTHOGONALIZE_STEPS];   // a or c_diag, c_mat and c_acc of B
  uint64_t limit_ns;
  int never_arrive;
  int* err;
};

// One product: its tiles and slices, operands, and the epilogue's arguments.
struct Phase {
  int per, tok_tiles, tiles, splits, log_splits, seg_kb, segs, rows_end;
  bool nt, tri;
  const CUtensorMap *w, *rows;
};
__device__ __forceinline__ Phase phase_of(const Maps& maps, const Args& q, int p, RagArgs& a) {
  const int step = p / 3, type = p - 3 * step, cur = step & 1;
  const bool last = type == 2 && step == q.steps - 1;
  const OrthoTiles& t = q.plan.t[type];
  Phase f;
  f.per = t.per;
  f.tok_tiles = t.tok_tiles;
  f.tiles = t.tiles;
  f.tri = t.tri;
  f.splits = t.splits;
  f.log_splits = t.splits == 1 ? 0 : t.splits == 2 ? 1 : t.splits == 4 ? 2 : 3;
  f.segs = q.parts == 2 ? 3 : 1;
  f.nt = type != 2;
  f.rows_end = type == 2 ? q.m : q.mp;
  f.seg_kb = (type == 0 ? q.Mp : q.mp) / BK;
  f.w = type == 0 ? &maps.x_nt[cur] : type == 1 ? &maps.a_nt : &maps.x_mn[cur];
  f.rows = type == 0 ? &maps.x_rows[cur] : type == 1 ? &maps.a_rows : &maps.b_rows;
  a.W = type == 2 ? (last ? q.M : q.Mp) : q.mp;
  a.out = type == 0 ? q.a : type == 1 ? q.b : q.x[cur ^ 1];
  a.ldo = (type == 2 ? q.Mp : q.mp) * q.parts;
  a.splits = t.splits;
  a.tile_rows = t.per;
  a.part = q.part;
  RagDense& d = a.dense;
  d.m = q.m;
  d.sym = type != 2;
  d.mp = q.mp;
  d.tri = t.tri;
  d.per = t.per;
  d.c_acc = type == 0 ? q.c_gram : type == 1 ? q.coef[3 * step + 2] : last ? q.c_last : q.c_apply;
  const bool kept = step < q.kept;
  const long long part_lo = q.parts == 2 ? (type == 2 ? q.Mp : q.mp) : 0;
  d.c_mat = q.coef[3 * step + (type == 2 ? 0 : 1)];
  d.c_diag = type == 1 && !kept ? q.coef[3 * step] : 0.0f;
  d.mat = type == 1 ? q.a : type == 2 && kept ? q.x[cur] : nullptr;
  d.mat_lo = type == 2 && kept ? q.lo - q.x[cur] : part_lo;
  d.out_lo = type == 2 && step + 1 < q.kept ? q.lo - q.x[cur ^ 1] : part_lo;
  d.final_out = last ? q.out : nullptr;
  d.transposed = q.transposed;
  return f;
}
// Item i of a phase: a tile, and a slice of its reduction.
struct Item {
  RagTile tile;
  int t, slice, kb0, kb1;
};
__device__ __forceinline__ Item item_of(const Phase& f, const Args& q, int e, int i) {
  Item r;
  r.t = i >> f.log_splits;
  r.slice = i - (r.t << f.log_splits);
  r.tile.e = e;
  if (f.tri) {
    rag_triangle(r.t, r.tile);
  } else {
    r.tile.w_tile = f.tok_tiles == 1 ? r.t : r.t / f.tok_tiles;
    r.tile.tok = r.t - r.tile.w_tile * f.tok_tiles;
  }
  r.tile.row0 = e * q.m + r.tile.tok * f.per;
  r.tile.rows = min(f.per, f.rows_end - r.tile.tok * f.per);
  const int n = f.segs * f.seg_kb;
  r.kb0 = n * r.slice >> f.log_splits;
  r.kb1 = n * (r.slice + 1) >> f.log_splits;
  return r;
}

// Tiles of matrix e that are finished, with all that their CTAs wrote before.
__device__ __forceinline__ uint32_t done_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void done_release(uint32_t* p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}
// Tiles of this CTA whose matrix's products before are finished: its producer's count
// for the epilogue's warps, which load A or X before the sums are complete (eight warps
// more that read the grid's counter in L2 cost 1 to 4%).
__device__ __forceinline__ uint32_t ready_acquire(uint32_t p) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ void ready_release(uint32_t p, uint32_t v) {
  asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(p), "r"(v) : "memory");
}

template <bool GRID>
__global__ void __launch_bounds__(threads(GRID), 1)
    k_ortho_cluster(const __grid_constant__ Maps maps, const __grid_constant__ Args args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + RING_BYTES);
  // full[S], empty[S], tfull[2], tempty[2], drain, stored[2], told[2]
  constexpr int NBARS = 2 * MAX_STAGES + 9;
  static_assert(8 * NBARS + 12 <= BAR_BYTES, "barrier area");
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const uint32_t ready = smem_u32(tmem_holder + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem), bar_base = smem_u32(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (MAX_STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * MAX_STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar_base + 8u * (2 * MAX_STAGES + 4);
  auto stored_bar = [&](int b) { return bar_base + 8u * (2 * MAX_STAGES + 5 + b); };
  auto told_bar = [&](int b) { return bar_base + 8u * (2 * MAX_STAGES + 7 + b); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), EPI_WARPS);
      mbar_init(stored_bar(a), EPI_WARPS);
      mbar_init(told_bar(a), 1);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    tmem_holder[2] = 0;
    fence_barrier_init();
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

  const int ctas = GRID ? (int)gridDim.x : args.plan.ctas;
  const int stages = args.plan.stages, stage_bytes = args.plan.stage_bytes;
  const int rank = GRID ? (int)blockIdx.x : blockIdx.x % ctas, e = GRID ? 0 : blockIdx.x / ctas;
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    return mbar_wait_bounded(bar, parity, abort_flag, args.limit_ns, args.err);
  };
  auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(bar, parity));
  };
  const uint64_t pol = l2_policy(0);
  int stage = 0, local = 0;
  uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
  bool ok = true, skip_first = args.never_arrive != 0;

  // GRID: until get() is at least `need`, by the whole warp
  auto wait_count = [&](auto get, uint32_t need) -> bool {
    int got = 1;
    if (lane == 0 && need != 0) {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t it = 1; get() < need; ++it) {
        if ((it & 15) != 0) continue;
        if (*abort_flag || globaltimer_ns() - t0 > args.limit_ns) {
          if (!*abort_flag) set_dev_error(args.err, kDevErrTimeout);
          *abort_flag = 1;
          got = 0;
          break;
        }
      }
    }
    got = __shfl_sync(0xffffffffu, got, 0);
    __syncwarp();
    return got != 0;
  };
  // item i of a product
  auto at = [&](const Phase& f, int i) -> Item {
    if (!GRID) return item_of(f, args, e, i);
    const int m = i / f.tiles;
    return item_of(f, args, m, i - m * f.tiles);
  };

  RagArgs a;
  Phase f = phase_of(maps, args, 0, a);
  Item first{};
  if (!GRID) first = item_of(f, args, e, rank);
  int begin = rank;               // GRID: this CTA's next item, counted from the product's first
  uint32_t before = 0;            // GRID: tiles of a matrix in the products before
  for (int p = 0; p < 3 * args.steps; ++p) {
    // Arguments and the first item: the producer and the MMA issuer have them before
    // the barrier opens, the epilogue's warps find them while the sums are computed.
    if ((GRID || warp >= 2) && p > 0) {
      f = phase_of(maps, args, p, a);
      if (!GRID) first = item_of(f, args, e, rank);
    }
    const int items = GRID ? args.E * f.tiles : f.tiles * f.splits;
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      for (int i = begin; ok && i < items; i += ctas) {
        const Item it = !GRID && i == rank ? first : at(f, i);
        const int boxes = (it.tile.rows + 31) / 32;
        if (GRID) {
          const uint32_t* done = args.done + it.tile.e;
          if (!wait_count([&] { return done_acquire(done); }, before)) {
            ok = false;
            break;
          }
          if (lane == 0) ready_release(ready, ++local);
          fence_proxy_async_global();
        }
        int seg = it.kb0 >= 2 * f.seg_kb ? 2 : it.kb0 >= f.seg_kb ? 1 : 0;
        int seg_k = it.kb0 - seg * f.seg_kb;
        const int w_lo = f.nt ? (f.seg_kb * BK) : args.Mp, rows_lo = f.seg_kb * BK;
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!warp_wait(empty_bar(stage), phase ^ 1)) {
            ok = false;
            break;
          }
          if (skip_first) {
            skip_first = false;      // watchdog test: leave this stage unarmed
          } else {
            const uint32_t sa = smem_base + stage * stage_bytes, sb = sa + A_BYTES;
            const uint32_t bar = full_bar(stage);
            if (elect_one()) {
              mbar_arrive_expect_tx(bar, A_BYTES + boxes * 32 * BK * 2);
              const int k0 = seg_k * BK, a_lo = seg == 1 ? w_lo : 0, b_lo = seg == 2 ? rows_lo : 0;
              if (f.nt)
                tma_load_3d(sa, f.w, bar, k0 + a_lo, it.tile.w_tile * 128, it.tile.e, pol);
              else
                tma_load_4d(sa, f.w, bar, 0, k0, it.tile.w_tile * 2 + a_lo / 64, it.tile.e,
                            pol);
              for (int j = 0; j < boxes; ++j)
                tma_load_2d(sb + j * 32 * BK * 2, f.rows, bar, k0 + b_lo, it.tile.row0 + 32 * j,
                            pol);
            }
            issued_mask |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          }
          if (++seg_k == f.seg_kb) {
            seg_k = 0;
            ++seg;
          }
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t major = f.nt ? 0u : kIdescAMn, a_step = f.nt ? 2 : 128;
      for (int i = begin; ok && i < items; i += ctas) {
        const Item it = !GRID && i == rank ? first : at(f, i);
        const int n = (it.tile.rows + 15) / 16 * 16;
        const uint32_t idesc = make_idesc(Half16<__half>::kFmt, Half16<__half>::kFmt, 128, n) | major;
        const int acc = local & 1;
        if (!warp_wait(tempty_bar(acc), ((local >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!warp_wait(full_bar(stage), phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_base + stage * stage_bytes;
          const uint64_t adesc = f.nt ? sdesc_k_sw128(sa) : sdesc_mn_sw128(sa);
          const uint64_t bdesc = sdesc_k_sw128(sa + A_BYTES);
          if (elect_one()) {
            for (int k = 0; k < BK / 16; ++k)
              umma_f16(tmem_base + acc * 256, adesc + a_step * k, bdesc + 2 * k, idesc,
                       kb != it.kb0 || k != 0);
            tc_commit(empty_bar(stage));
          }
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (elect_one()) tc_commit(tfull_bar(acc));
        ++local;
      }
    } else if (GRID && warp == 2 + EPI_WARPS) {
      // ---------------------------------------------------------- flags
      // Tells the grid of a tile when its stores are done: the fences wait for all of
      // them (some 2000 cycles), the epilogue's warps go on with the next tile.
      for (int i = begin; ok && i < items; i += ctas) {
        if (!warp_wait(stored_bar(local & 1), (local >> 1) & 1)) {
          ok = false;
          break;
        }
        fence_proxy_async_global();
        __threadfence();
        if (lane == 0) {
          done_release(args.done + i / f.tiles);
          mbar_arrive(told_bar(local & 1));
        }
        __syncwarp();
        ++local;
      }
    } else {
      // ---------------------------------------------------------- epilogue
      const int q = warp & 3;
      const bool loads = f.splits == 1 && a.dense.mat != nullptr;
      const int part = (warp - 2) >> 2;
      constexpr int STEP = 4 * EPI_WARPS;
      for (int i = begin; ok && i < items; i += ctas) {
        const Item it = !GRID && i == rank ? first : at(f, i);
        const int acc = local & 1, w = it.tile.w_tile * 128 + q * 32 + lane;
        Words16 mat_next;
        if (GRID && loads && !wait_count([&] { return ready_acquire(ready); }, local + 1)) {
          ok = false;
          break;
        }
        if (loads && 16 * part < it.tile.rows)
          rag_dense_load(a, it.tile, mat_next, 16 * part, w, lane);
        int got = 0;
        if (lane == 0) got = wait(tfull_bar(acc), (local >> 1) & 1);
        ok = __shfl_sync(0xffffffffu, got, 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
#pragma unroll 1
        for (int c = 16 * part; c < it.tile.rows; c += STEP) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(taddr + c, r);
          const Words16 h = mat_next;
          tmem_ld_wait();
          const int tok = it.tile.tok * f.per + c, left = it.tile.rows - c;
          if (loads && c + STEP < it.tile.rows) rag_dense_load(a, it.tile, mat_next, c + STEP, w, lane);
          if (!GRID && f.splits > 1)
            rag_store_part(a, r, e * f.tiles + it.t, it.slice, c, it.tile.rows, q * 32 + lane);
          else if (f.nt)
            rag_dense_store16<true>(a, it.tile, r, h, loads, tok, left, w, lane);
          else
            rag_dense_store16<false>(a, it.tile, r, h, loads, tok, left, w, lane);
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
        ++local;
        if (GRID) {                 // (the tile two before has been told)
          const int n = local - 1;
          if (!warp_wait(told_bar(n & 1), ((n >> 1) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive(stored_bar(n & 1));
        }
      }
    }
    if (GRID) {
      const int mine = begin < items ? (items - begin + ctas - 1) / ctas : 0;
      begin += mine * ctas - items;
      before += f.tiles;
      continue;
    }
    if (f.splits > 1) {
      cluster_sync();
      if (*abort_flag == 0) {
        for (int t = 0; t < f.tiles; ++t) {
          const RagTile D = item_of(f, args, e, t * f.splits).tile;
          rag_join_fused<EPI_DENSE, __half>(a, D, e * f.tiles + t, rank, ctas, warp,
                                            threads(false) / 32, lane);
        }
      }
    }
    if (f.splits > 1 || warp >= 2) fence_proxy_async_global();
    if (warp < 2 && p + 1 < 3 * args.steps) {
      f = phase_of(maps, args, p + 1, a);
      first = item_of(f, args, e, rank);
    }
    cluster_sync();
    if (warp == 0) fence_proxy_async_global();
  }

  // copies and MMAs still in flight after a wait that ran out
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < stages; ++s)
      if (issued_mask & (1u << s))
        mbar_wait_bounded(full_bar(s), (issued_parity >> s) & 1, nullptr, args.limit_ns, args.err);
  } else if (warp == 1) {
    if (elect_one()) tc_commit(drain_bar);
    if (lane == 0) mbar_wait_bounded(drain_bar, 0, nullptr, args.limit_ns, args.err);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

}  // namespace

// Of each size of cluster the tiles and slices of least time, and of these the size.
// Cycles as dense_gemm.cu's model has them, with a barrier and the first copies in
// place of a launch.
OrthoClusterPlan ortho_cluster_plan(int E, int m, int mp, int M, int Mp, int parts, int steps) {
  OrthoClusterPlan best{};
  const int segs = parts == 2 ? 3 : 1;
  for (int ctas = 1; ctas <= 8; ctas *= 2) {
    OrthoClusterPlan r{};
    r.ctas = ctas;
    long long step_cycles = 0;
    int widest = 32;
    for (int type = 0; type < 3; ++type) {
      const int width = type == 2 ? Mp : mp, rows = type == 2 ? m : mp;
      const int kb = segs * (type == 0 ? Mp : mp) / BK, unit = type == 2 ? 16 : 32;
      long long least = 0;
      for (int tile = 32; tile <= 256; tile *= 2) {
        if (tile > 32 && tile >= 2 * rows) break;
        for (int splits = 1; splits <= ctas; splits *= 2) {
          OrthoTiles t{};
          t.splits = splits;
          t.w_tiles = (width + 127) / 128;
          t.tok_tiles = (rows + tile - 1) / tile;
          t.per = ((rows + t.tok_tiles - 1) / t.tok_tiles + unit - 1) / unit * unit;
          t.tiles = t.w_tiles * t.tok_tiles;
          const long long items = (long long)t.tiles * splits;
          if (splits > 1 && (items > ctas || kb < 2 * splits)) continue;
          const long long k = (kb + splits - 1) / splits;
          const long long step = std::max((16384 + (t.per + 31) / 32 * 4096) / 55, 53 * t.per / 20);
          const long long epilogue = (type == 2 ? 1000 : 1500) * ((t.per + 63) / 64);
          const long long c =
              splits > 1 ? 8000 + k * step + 600 * ((t.per + 63) / 64)
                         : 3500 + (items + ctas - 1) / ctas * std::max(k * step, epilogue) + epilogue;
          if (least == 0 || c < least) {
            least = c;
            r.t[type] = t;
          }
        }
      }
      step_cycles += least;
      widest = std::max(widest, (r.t[type].per + 31) / 32 * 32);
    }
    r.stage_bytes = A_BYTES + widest * BK * 2;
    r.stages = std::min(MAX_STAGES, RING_BYTES / r.stage_bytes);
    const int at_once = ctas == 1 ? 152 : kRagClusters[ctas == 8 ? 0 : ctas == 4 ? 1 : 2];
    r.cycles = (long long)((E + at_once - 1) / at_once) * (steps * step_cycles + 5000) + 5000;
    if (best.cycles == 0 || r.cycles < best.cycles) best = r;
  }
  return best;
}

// For the whole grid: tiles of least time.  A product takes its tiles' share of the
// SMs, or what stands between one matrix's products: the flag and its fences, the first
// copies, a tile.  Between unlike forms (`cycles`) the latter counts more than between
// tiles, as measured: its operands were just written by other SMs.  The last product
// takes what its epilogue moves of X's two parts.
OrthoClusterPlan ortho_grid_plan(int E, int m, int mp, int M, int Mp, int parts, int steps) {
  OrthoClusterPlan r{};
  const int segs = parts == 2 ? 3 : 1;
  int widest = 32;
  for (int type = 0; type < 3; ++type) {
    const int width = type == 2 ? Mp : mp, rows = type == 2 ? m : mp;
    const int kb = segs * (type == 0 ? Mp : mp) / BK, unit = type == 2 ? 16 : 32;
    long long least = 0, cycles = 0;
    for (int tile = 32; tile <= 256; tile *= 2) {
      if (tile > 32 && tile >= 2 * rows) break;
      for (int tri = 0; tri < 2; ++tri) {
        if (tri && (type == 2 || tile != 128)) continue;
        OrthoTiles t{};
        t.splits = 1;
        t.tri = tri;
        t.w_tiles = (width + 127) / 128;
        t.tok_tiles = (rows + tile - 1) / tile;
        t.per = tri ? tile : ((rows + t.tok_tiles - 1) / t.tok_tiles + unit - 1) / unit * unit;
        t.tiles = tri ? t.w_tiles * (t.w_tiles + 1) / 2 : t.w_tiles * t.tok_tiles;
        const long long step = std::max((16384 + (t.per + 31) / 32 * 4096) / 55, 53 * t.per / 20);
        const long long epilogue = (tri ? 1700 : 1400) * ((t.per + 31) / 32);
        const long long each = std::max(kb * step, epilogue);
        const long long share = ((long long)E * t.tiles + 151) / 152 * (each + 1200);
        const long long c = std::max(share, 6000 + kb * step + epilogue);
        if (least == 0 || c < least) {
          least = c;
          cycles = std::max(share, 8000 + 6 * kb * step / 5 + epilogue);
          r.t[type] = t;
        }
      }
    }
    if (type == 2 && parts == 1) cycles = std::max(cycles, 8ll * E * m * Mp / 2100);
    r.cycles += steps * cycles;
    widest = std::max(widest, (r.t[type].per + 31) / 32 * 32);
  }
  r.stage_bytes = A_BYTES + widest * BK * 2;
  r.stages = std::min(MAX_STAGES, RING_BYTES / r.stage_bytes);
  return r;
}

size_t ortho_cluster_part_bytes(const OrthoClusterPlan& p, int E) {
  size_t most = 0;
  for (const OrthoTiles& t : p.t)
    if (t.splits > 1)
      most = std::max(most, (size_t)E * t.w_tiles * t.tok_tiles * t.splits * t.per * 128 * sizeof(float));
  return most;
}

cudaError_t launch_ortho_cluster(const OrthoClusterProblem& d, cudaStream_t stream) {
  Maps maps;
  Args q{};
  q.plan = d.plan;
  const int ldx = d.parts * d.Mp, lda = d.parts * d.mp;
  const uint64_t rows = (uint64_t)d.E * d.m;
  for (int i = 0; i < 2; ++i) {
    if (!make_tmap_rag(&maps.x_nt[i], d.x[i], true, 3, ldx, d.m, d.E, ldx, 128) ||
        !make_tmap_rag_wide(&maps.x_mn[i], d.x[i], true, d.m, ldx, d.E, ldx, 2) ||
        !make_tmap_rag(&maps.x_rows[i], d.x[i], true, 2, ldx, rows, 0, ldx, 32))
      return cudaErrorInvalidValue;
    q.x[i] = static_cast<__half*>(d.x[i]);
  }
  if (!make_tmap_rag(&maps.a_nt, d.a, true, 3, lda, d.m, d.E, lda, 128) ||
      !make_tmap_rag(&maps.a_rows, d.a, true, 2, lda, rows, 0, lda, 32) ||
      !make_tmap_rag(&maps.b_rows, d.b, true, 2, lda, rows, 0, lda, 32))
    return cudaErrorInvalidValue;
  q.E = d.E;
  q.m = d.m;
  q.M = d.M;
  q.mp = d.mp;
  q.Mp = d.Mp;
  q.parts = d.parts;
  q.steps = d.steps;
  q.transposed = d.transposed;
  q.kept = d.kept;
  q.lo = static_cast<__half*>(d.lo);
  q.a = static_cast<__half*>(d.a);
  q.b = static_cast<__half*>(d.b);
  q.out = static_cast<__nv_bfloat16*>(d.out);
  q.part = static_cast<float*>(d.part);
  q.c_gram = d.c_gram;
  q.c_apply = d.c_apply;
  q.c_last = d.c_last;
  for (int i = 0; i < 3 * d.steps; ++i) q.coef[i] = d.coef[i];
  watchdog_params(&q.limit_ns, &q.never_arrive);
  q.err = dev_error_word();
  if (q.err == nullptr) return cudaErrorInvalidDevice;
  static DeviceOnce attr;
  const cudaError_t e = attr.call([] {
    const cudaError_t r = cudaFuncSetAttribute(
        k_ortho_cluster<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(k_ortho_cluster<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SMEM_BYTES);
  });
  if (e != cudaSuccess) return e;
  if (d.plan.ctas == 0) {          // all CTAs at the same time: one an SM
    q.done = d.done;
    int most = 0;
    for (const OrthoTiles& t : d.plan.t) most = std::max(most, t.tiles);
    cudaLaunchAttribute coop;
    coop.id = cudaLaunchAttributeCooperative;
    coop.val.cooperative = 1;
    cudaLaunchConfig_t cfg = {};
    const int ctas = ortho_grid_ctas() > 0 ? ortho_grid_ctas() : num_sms();
    cfg.gridDim = dim3((unsigned)std::min<long long>(ctas, (long long)d.E * most), 1, 1);
    if ((int)cfg.gridDim.x > num_sms()) {      // a refusal inside a capture would end it
      cudaStreamCaptureStatus status;
      const cudaError_t c = cudaStreamIsCapturing(stream, &status);
      if (c != cudaSuccess) return c;
      if (status != cudaStreamCaptureStatusNone) return cudaErrorCooperativeLaunchTooLarge;
    }
    cfg.blockDim = dim3(threads(true), 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = &coop;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_ortho_cluster<true>, maps, q);
  }
  return launch_dependent(k_ortho_cluster<false>, (unsigned)(d.E * d.plan.ctas), threads(false),
                          SMEM_BYTES, stream, d.plan.ctas, maps, q);
}

}  // namespace moe
