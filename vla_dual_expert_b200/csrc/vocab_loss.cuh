// Softmax cross entropy over a vocabulary, without keeping the logits, and its gradient.
//
//   z_iv = h_i . W_v                     lse_i = log sum_v exp(z_iv)
//   loss_i = lse_i - z_{i, t_i}          (0 where t_i < 0)
//   G_iv = (exp(z_iv - lse_i) - [v = t_i]) dloss_i      dh = G W      dW = G^T h
//
// One tcgen05 kernel does all four products; its mode sets the operands' majors and the epilogue:
//   kVgStats  z tile -> the row's (max, sum of exp) of its columns, and z_{i, t_i}
//   kVgGrad   z tile again -> G / s in bf16, one piece of the vocabulary at a time
//   kVgBack   both products with the piece's G, in one launch:
//             dh += G W:  A = G (K-major), B = W read along H (MN-major), fp32 sums
//             dW = G^T h: A = G read along V (MN-major), B = h read along H (MN-major)
//
// s = max |dloss_i|, of the finite ones of the tokens with a target: G / s is what is rounded to bf16 (half a step:
// 2^-8 of the value) and s multiplies the fp32 results, so the factor 1 / tokens of a mean, the same in every row,
// takes no part in the rounding (a constant dloss that is no power of two would otherwise put one and the same
// relative error into every entry -dloss of the targets, which no sum averages out).
//
// G lies in panels of 64 columns, [panel][token][64], so that every box of it, 64 columns x some tokens, is one
// stretch of memory; as [token][column] a box's rows lay 2 x piece bytes apart, a power of two (both gradients of
// 256 tokens x 131072 x 2048: 505 -> 490 us).
//
// The products are bound by the tensor cores for many tokens, under load by the power limit: the loss of 4096
// tokens x 131072 x 2048 takes 1.67 ms one after another, 1320 TFLOP/s (the library's bf16 product that writes those
// logits 1.74 ms), the gradients of 8192 tokens 10.5 ms, 1260 TFLOP/s (the library's three products 10.0 ms).  With
// few tokens they are bound by HBM: the loss reads W once (7 tokens: 91 us alone, 103 among calls with other
// weights, 82 at the rate of a copy); the gradient twice, once for the logits and once for dh, in launches of their own,
// and dW is written (7 tokens: 294 to 318 us between one B200 and another, 245 at that rate; with one reading it would
// be 164, as lse is given and a tile's G is known with its logits).  dW in fp32 passes through shared memory and plain
// stores: 412 us, 986 where it is added to what is there (327 and 491 at that rate).
#pragma once
#include "attention_tc.cuh"   // sw128_mnmajor_desc, tmem_st32
#include "embedding.cuh"
#include "gemm.cuh"           // band_tile, resid_swz, bf2
#include "residual_norm.cuh"  // store4

namespace dm0 {

enum VgMode : int { kVgStats = 0, kVgGrad = 1, kVgBack = 2 };

struct VgArgs {
  int M, N, K;          // of this product (rows of A, rows of B, contraction)
  int mt, nt, splits, kb_per_split;
  int band;             // raster: m-tiles per band (1: n fastest)
  int b_y0;             // offset of B's first row in its map: vocabulary row of the piece
  // Bytes of A's and B's k-block per CTA.  Rows that a box takes beyond its tensor cost the copy engine as much as
  // others, so with few tokens the boxes have only theirs: as rows of A, the tile's others are then whatever lies
  // in shared memory (rows of a product do not mix; theirs are not stored); as the contraction of dW, to the next
  // multiple of 16, and ksteps instructions of 16 take no more.
  uint32_t a_bytes, b_bytes;
  int ksteps;
  int* err;
  // statistics and G
  Ids targets;
  int vocab, v0;        // whole vocabulary; first column of the piece
  int valid_n;          // columns of this product that are vocabulary entries
  float2* part;         // (max, sum): [2 nt][part_ld] of each tile half; with one m-tile, where a worker's tiles
                        // have the same rows, [2 workers][part_ld] of its halves of all of them
  int part_ld;
  float* zt;            // [tokens] logit of the target
  const float *lse, *dloss;
  float* scale;         // scale[0] = s: found by the first piece's kVgGrad, read by the others
  // dh: fp32 sums of the splits, [split][tokens][H]; dW: rows of the piece
  float* dh;
  int add;              // add to what is there (dh: from the second piece on; dW: accumulate)
  float* dw;            // [vocab][H] in fp32; null: bf16 through the map
};

constexpr int kVgBackStretch = 256;   // k-blocks of the gradients' products added in the accumulator

// Tile of a CTA pair (cta_group::2): 256 rows of A times 256 rows of B, of which each CTA stages half.  Tile of
// one CTA, for up to 128 tokens, where a product is one read of W: 128 x 128, narrow so that the tiles of a
// vocabulary spread evenly (131072 columns, 148 SMs: 7 rounds of 128, 99% busy, against 4 of 256, 86%).
template <bool PAIR>
struct VgTile {
  static constexpr int kM = PAIR ? 256 : 128, kN = PAIR ? 256 : 128;
  static constexpr int kBRows = 128;   // of B, per CTA
  static constexpr int kStages = 6;
  static constexpr int kBufs = 512 / kN;   // accumulators in TMEM
  static constexpr int kStretch = PAIR ? 16 : 8;   // k-blocks of logits added in the accumulator
  static constexpr uint32_t kA = 128 * 128, kB = kBRows * 128, kStage = kA + kB, kPipe = kStages * kStage;
  static constexpr uint32_t kScr = kPipe;                 // 8 x 4 KB
  static constexpr uint32_t kBar = kScr + 8 * 4096;
  static constexpr uint32_t kBytes = kBar + 256 + 1024;   // barriers, alignment slack
  static_assert(kBytes <= 232448, "shared memory of one CTA");
};

// Copy of a box from shared memory to a tensor (rows and columns outside it are not written), its group, and the
// waits for the groups' reads and for their writes; by one lane of a warp.
__device__ __forceinline__ void vg_copy_out(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void vg_copy_out_panel(const CUtensorMap* map, const void* src, int row, int panel) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(0), "r"(row), "r"(panel)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void vg_scratch_free() {
  if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
// 32 rows x 64 bf16 (values of one lane: its row's 64 columns) through the warp's 4 KB of scratch, in the layout of
// a 128-byte-swizzled box, and from there by one copy.  The tiles of few tokens are all epilogue, two warps to a
// scheduler, so its instructions count: addresses by one exclusive or, paired multiplications, one accumulator load
// per chunk, and no loads and stores of the rows by the warp.
template <bool PANEL>
__device__ __forceinline__ void vg_store_bf16(uint8_t* scr, const float (&v)[64], const CUtensorMap* map, int x, int y,
                                              int rows, int place = -1, float at = 0.f) {
  const int lane = threadIdx.x & 31;
  vg_scratch_free();
  const uint32_t w = smem_u32(scr) + lane * 128 + ((lane & 7) << 4);   // scr is 1024-byte aligned
#pragma unroll
  for (int j = 0; j < 8; ++j)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(w ^ (j << 4)), "r"(bf2(v[8 * j], v[8 * j + 1])),
                 "r"(bf2(v[8 * j + 2], v[8 * j + 3])), "r"(bf2(v[8 * j + 4], v[8 * j + 5])),
                 "r"(bf2(v[8 * j + 6], v[8 * j + 7]))
                 : "memory");
  if (place >= 0)   // this row's value there is another
    asm volatile("st.shared.b16 [%0], %1;" ::"r"((w ^ ((place >> 3) << 4)) + 2 * (place & 7)),
                 "h"(static_cast<uint16_t>(bf2(at, 0.f)))
                 : "memory");
  fence_async_smem();
  __syncwarp();
  if (lane == 0 && rows > 0) {
    if (PANEL)
      vg_copy_out_panel(map, scr, y, x >> 6);
    else
      vg_copy_out(map, scr, x, y);
  }
}
// 32 rows x 32 fp32, added to what is there if `add`
__device__ __forceinline__ void vg_store_f32(uint8_t* scr, const float* v, float* dst, int64_t ld, int rows,
                                             bool add) {
  const int lane = threadIdx.x & 31;
  const int qr = lane >> 3, qc = lane & 7;
  float4 old[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + qr;
    old[i] = add && r < rows ? *reinterpret_cast<const float4*>(dst + r * ld + qc * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(scr + resid_swz(lane, j)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + qr;
    float4 x = *reinterpret_cast<const float4*>(scr + resid_swz(r, qc));
    if (add) x = make_float4(x.x + old[i].x, x.y + old[i].y, x.z + old[i].z, x.w + old[i].w);
    if (r < rows) *reinterpret_cast<float4*>(dst + r * ld + qc * 4) = x;
  }
  __syncwarp();
}

constexpr float kLog2e = 1.4426950408889634f;

// The tensor cores' fp32 accumulator drops the bits below its last place instead of rounding them, so a long
// sum loses up to that at each of its K / 16 steps, always toward zero.  The logits are therefore added in
// stretches of VgTile::kStretch k-blocks, each from zero, and the stretches in fp32 registers.  Error of lse for 4096
// tokens x 131072 x 2048: 1.7e-6 in one stretch, 0.9e-6 in stretches of 1024 (1.67 ms both), 0.4e-6 in stretches of
// 512 (1.76 ms; up to 128 tokens, bound by HBM, it costs nothing).
// The gradient builds the same logits bit for bit.  Of a target that the model is sure of, exp(z - lse) - 1 is all
// cancellation: there the logit's error has to be the one that lse has, and the difference one function, expm1 (in one
// stretch and as a difference, rows of dhidden were off by up to 23% at 1 - p from 1e-4 to 1e-3, and by three times
// themselves below).
// The gradients' products take stretches of kVgBackStretch k-blocks: a split of dh is at most one, dW of more than
// 16384 tokens several (LONG; 2^17 tokens of one sign in one stretch: 8e-4 off).

// Warp 0: TMA; warp 1: TMEM and, in a pair's first CTA, MMA; warps 2..9: epilogue, two per TMEM lane quarter
// (column halves; sixteen warps on quarters, with stores of 64 instead of 128 bytes a row, made the gradients of
// 8192 tokens 10.9 ms instead of 10.0).  Persistent: one CTA per SM, or one pair per two, walks the tiles; the
// accumulator is buffered (two of a pair, four of a CTA), and free again as soon as it is in registers.  In a pair
// the copies of both CTAs count on the first one's `full`, its MMAs free both CTAs' stages and fill both
// accumulators, and both epilogues free its `tempty`.
//
// kVgBack's tiles: dh's first, then dW's, each product with its own operands.
struct VgMaps {
  CUtensorMap a, b, out;   // operands, and a bf16 result: boxes of 64 columns x 32 rows
};
template <int MODE, bool PAIR, bool LONG>
__device__ __forceinline__ void vocab_gemm(const VgMaps& m0, const VgArgs& a0, const VgMaps& m1, const VgArgs& a1) {
  using L = VgTile<PAIR>;
  constexpr int kStages = L::kStages, kN = L::kN, kBufs = L::kBufs;
  constexpr int kStretch = MODE == kVgBack ? kVgBackStretch : L::kStretch;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* drain = tempty + kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* red = reinterpret_cast<float*>(tmem_slot + 2);   // [8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_rank()) : 0;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x, workers = PAIR ? gridDim.x >> 1 : gridDim.x;
  int* const err = a0.err;
  const int tiles0 = a0.mt * a0.nt * a0.splits;
  const int ntiles = MODE == kVgBack ? tiles0 + a1.mt * a1.nt * a1.splits : tiles0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], PAIR ? 16 : 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, kBufs * kN);
    } else {
      tmem_alloc(tmem_slot, kBufs * kN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();   // the other CTA's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  struct Tile {
    bool second;   // of kVgBack: a tile of dW
    int m, n, kb0, kb1, split;
  };
  const int mine = worker < ntiles ? (ntiles - 1 - worker) / workers + 1 : 0;   // tiles of this worker
  auto tile_at = [&](int q) {
    int t = worker + q * workers;
    Tile w;
    w.second = MODE == kVgBack && t >= tiles0;
    const VgArgs& a = w.second ? a1 : a0;
    if (w.second) t -= tiles0;
    const int plane = a.mt * a.nt;
    w.split = t / plane;
    band_tile(t - w.split * plane, a.mt, a.nt, a.band, w.m, w.n);
    w.kb0 = w.split * a.kb_per_split;
    w.kb1 = min((a.K + 63) >> 6, w.kb0 + a.kb_per_split);
    return w;
  };
  auto stretch_end = [&](int kb, int kb1) { return LONG ? min(kb1, kb + kStretch) : kb1; };

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&m0.a);
      tma_prefetch_desc(&m0.b);
      if (MODE == kVgBack) {
        tma_prefetch_desc(&m1.a);
        tma_prefetch_desc(&m1.b);
      }
      const uint64_t keep = policy_evict_last();
      int it = 0;
      for (int q = 0; q < mine && !*abort_flag; ++q) {
        const Tile w = tile_at(q);
        const VgArgs& a = w.second ? a1 : a0;
        const VgMaps& maps = w.second ? m1 : m0;
        const bool a_mn = w.second, b_mn = MODE == kVgBack;
        const int ra = w.m * L::kM + rank * 128, rb = w.n * kN + rank * L::kBRows;
        const uint32_t bytes = (PAIR ? 2 : 1) * (a.a_bytes + a.b_bytes);
        const int by0 = a.b_y0;
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
          const int s = it % kStages;
          if (it >= kStages && !mbar_wait(&empty[s], ((it / kStages) - 1) & 1, abort_flag)) {
            *abort_flag = 1;
            raise_error(err, kErrTimeoutProducer);
            break;
          }
          uint8_t* sa = smem + s * L::kStage;
          uint8_t* sb = sa + L::kA;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          const uint32_t bar = PAIR ? cluster_addr(&full[s], 0) : 0;
          auto load = [&](uint8_t* dst, const CUtensorMap& map, int x, int y) {
            if constexpr (PAIR)
              tma_load_2d_pair(dst, &map, bar, x, y, keep);
            else
              tma_load_2d(dst, &map, &full[s], x, y, keep);
          };
          auto load_panel = [&](uint8_t* dst, int row, int panel) {   // of G
            if constexpr (PAIR)
              tma_load_3d_pair(dst, &maps.a, bar, 0, row, panel, keep);
            else
              tma_load_3d(dst, &maps.a, &full[s], 0, row, panel, keep);
          };
          if (a_mn) {
#pragma unroll
            for (int j = 0; j < 2; ++j) load_panel(sa + 8192 * j, kb * 64, (ra >> 6) + j);
          } else if (MODE == kVgBack) {
            load_panel(sa, ra, kb);
          } else {
            load(sa, maps.a, kb * 64, ra);
          }
          if (b_mn) {
#pragma unroll
            for (int j = 0; j < L::kBRows / 64; ++j) load(sb + 8192 * j, maps.b, rb + 64 * j, by0 + kb * 64);
          } else {
            load(sb, maps.b, kb * 64, by0 + rb);
          }
        }
      }
      // copies in flight land before the CTA exits (a pair's, both CTAs': the first one waits for them, the
      // other for it)
      if (rank == 0)
        for (int i = it - kStages; i < it; ++i) {
          if (i < 0) continue;
          if (!mbar_wait(&full[i % kStages], (i / kStages) & 1, nullptr, kDrainTimeoutNs)) raise_error(err, kErrDrain);
        }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      auto commit = [&](uint64_t* bar) {
        if constexpr (PAIR)
          umma_commit_pair(bar);
        else
          umma_commit(bar);
      };
      int it = 0, local = 0;
      bool ok = true;
      for (int q = 0; ok && q < mine; ++q) {
        const Tile w = tile_at(q);
        const bool a_mn = w.second;
        constexpr bool b_mn = MODE == kVgBack;
        const int ksteps = (w.second ? a1 : a0).ksteps;
        const uint32_t idesc = idesc_bf16_f32(L::kM, kN) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
        for (int ks = w.kb0; ok && ks < w.kb1; ++local) {
          const int ke = stretch_end(ks, w.kb1), buf = local % kBufs;
          const uint32_t freed = (local / kBufs - 1) & 1;
          if (local >= kBufs && !(PAIR ? mbar_wait_cluster(&tempty[buf], freed, abort_flag)
                                   : mbar_wait(&tempty[buf], freed, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int kb = ks; kb < ke; ++kb, ++it) {
            const int s = it % kStages;
            if (!mbar_wait(&full[s], (it / kStages) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t aa = smem_u32(smem + s * L::kStage), bb = aa + L::kA;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (MODE == kVgBack && kk >= ksteps) break;
              const uint64_t da = a_mn ? sw128_mnmajor_desc(aa + 2048 * kk, 8192) : sw128_kmajor_desc(aa + 32 * kk);
              const uint64_t db = b_mn ? sw128_mnmajor_desc(bb + 2048 * kk, 8192) : sw128_kmajor_desc(bb + 32 * kk);
              const uint32_t acc = (kb > ks || kk != 0) ? 1u : 0u;
              if constexpr (PAIR)
                umma_bf16_pair(tmem + buf * kN, da, db, idesc, acc);
              else
                umma_bf16(tmem + buf * kN, da, db, idesc, acc);
            }
            commit(&empty[s]);
          }
          if (ok) commit(&tfull[buf]);
          ks = ke;
        }
      }
      if (!ok) {
        *abort_flag = 1;
        raise_error(err, kErrTimeoutMma);
      }
      commit(drain);
      if (!mbar_wait(drain, 0, nullptr, kWaitTimeoutNs + kDrainTimeoutNs)) raise_error(err, kErrDrain);
    }
  } else {
    const int lane_base = (warp & 3) * 32, half = (warp - 2) >> 2;
    uint8_t* scr = smem + L::kScr + (warp - 2) * 4096;
    constexpr int kCols = kN / 2;   // columns of this warp
    float s = 1.f;
    if constexpr (MODE == kVgGrad) {
      if (a0.v0 == 0) {   // s, by every CTA beside its first tile's products; the first one keeps it
        float mx = 0.f;
        bool bad = false;
        for (int i = threadIdx.x - 64; i < a0.M; i += 256) {
          const int t = a0.targets.get(i);
          bad |= t >= a0.vocab;
          const float d = fabsf(a0.dloss[i]);
          if (t >= 0 && t < a0.vocab && d <= 3.402823466e38f) mx = fmaxf(mx, d);   // infinities and NaN stay in their rows
        }
        if (bad && blockIdx.x == 0) raise_error(err, kErrBounds);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        if (lane == 0) red[warp - 2] = mx;
        named_bar_sync(1, 256);
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = fmaxf(mx, red[k]);
        s = mx > 0.f ? mx : 1.f;
        if (blockIdx.x == 0 && threadIdx.x == 64) a0.scale[0] = s;
      } else {
        s = a0.scale[0];
      }
    }
    if constexpr (MODE == kVgBack) s = a0.scale[0];
    int local = 0;
    auto ready = [&]() {   // the next accumulator of this CTA is complete
      if (mbar_wait(&tfull[local % kBufs], (local / kBufs) & 1, abort_flag)) {
        tc_fence_after();
        return true;
      }
      *abort_flag = 1;
      raise_error(err, kErrTimeoutEpilogue);
      return false;
    };
    auto release = [&]() {   // and read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_cluster(cluster_addr(&tempty[local % kBufs], 0));
        else
          mbar_arrive(&tempty[local % kBufs]);
      }
      ++local;
    };
    const uint32_t tm0 = tmem + (static_cast<uint32_t>(lane_base) << 16) + half * kCols;
    // The next accumulator holds the tile's whole sum: those of more stretches are added in registers, and go back to the
    // last one's place, from where all tiles are read alike, a few columns at a time.
    auto whole = [&](const Tile& w) {
      if (!ready()) return false;
      if (!LONG || w.kb1 - w.kb0 <= kStretch) return true;
      float v[kCols / 32][32];
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) tmem_ld32(tm0 + (local % kBufs) * kN + 32 * c, v[c]);
      release();
      for (int ks = stretch_end(w.kb0, w.kb1);; ks = stretch_end(ks, w.kb1)) {
        if (!ready()) return false;
        const bool last = ks + kStretch >= w.kb1;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          const uint32_t at = tm0 + (local % kBufs) * kN + 32 * c;
          float x[32];
          tmem_ld32(at, x);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[c][j] += x[j];
          if (last) tmem_st32(at, v[c]);
        }
        if (last) {
          tmem_wait_st();
          return true;
        }
        release();
      }
    };
    bool go = true;
    float run_mx = -INFINITY, run_sum = 0.f;   // of kVgStats with one m-tile
    for (int q = 0; go && q < mine; ++q) {
      const Tile w = tile_at(q);
      const VgArgs& a = w.second ? a1 : a0;
      const int row0 = w.m * L::kM + rank * 128 + lane_base, row = row0 + lane;
      const int col0 = w.n * kN + half * kCols;
      const int rows = min(32, a.M - row0);   // rows of this warp to store (may be <= 0)
      // what the epilogue knows of its row, requested while the products run
      int tgt = -1;
      float row_lse = 0.f, row_dloss = 0.f;
      if (MODE != kVgBack && row < a.M) {
        tgt = a.targets.get(row);
        if (tgt >= a.vocab) tgt = -1;
        if (MODE == kVgGrad) row_lse = a.lse[row], row_dloss = a.dloss[row];
      }
      if constexpr (MODE == kVgStats) {
        float v[kCols / 32][32];
        for (int ks = w.kb0; ks < w.kb1; ks = stretch_end(ks, w.kb1)) {
          if (!ready()) {
            go = false;
            break;
          }
          const uint32_t tm = tm0 + (local % kBufs) * kN;
          if (ks == w.kb0) {
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) tmem_ld32(tm + 32 * c, v[c]);
          } else {
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) {
              float x[32];
              tmem_ld32(tm + 32 * c, x);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[c][j] += x[j];
            }
          }
          release();
        }
        if (!go) break;
        if (col0 + kCols > a.valid_n) {
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col0 + 32 * c + j >= a.valid_n) v[c][j] = -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 2) mx = max3f(mx, v[c][j], v[c][j + 1]);
        if (tgt >= 0 && static_cast<unsigned>(tgt - col0) < static_cast<unsigned>(kCols)) {
          float z = 0.f;
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) z = tgt - col0 == 32 * c + j ? v[c][j] : z;
          a.zt[row] = z;
        }
        mx = fmaxf(mx, run_mx);
        // The exponents are v log2 e against ref, log2 e times the maximum rounded: the sum comes out 2^(mx log2 e - ref)
        // times too large, up to half a unit of ref in the exponent, and is put right once.  The sum of the tiles before
        // is taken over as it is while the maximum stays; a factor that is only nearly one would be there again with every
        // tile (2^20 entries, 56 tiles a worker, lse 45: 3.7e-5 off; so 2.4e-6, of which 1.9e-6 is its last rounding).
        const float top = mx == -INFINITY ? 0.f : mx;
        const float ref = __fmul_rn(top, kLog2e);
        const float fix = ex2_fast(-fmaf(top, kLog2e, -ref));
        float2 sum[2] = {};
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 x = ffma2(make_float2(v[c][j], v[c][j + 1]), make_float2(kLog2e, kLog2e), make_float2(-ref, -ref));
            sum[(j >> 1) & 1] = fadd2(sum[(j >> 1) & 1], make_float2(ex2_fast(x.x), ex2_fast(x.y)));
          }
        const float before = mx == run_mx ? run_sum : run_sum * ex2_fast((run_mx - mx) * kLog2e);
        const float2 now = make_float2(mx, fmaf((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y), fix, before));
        if (a.mt > 1) {
          if (row < a.M) a.part[static_cast<int64_t>(2 * w.n + half) * a.part_ld + row] = now;
        } else {
          run_mx = now.x, run_sum = now.y;
          if (q + 1 == mine && row < a.M) a.part[static_cast<int64_t>(2 * worker + half) * a.part_ld + row] = now;
        }
      } else {
        if (!whole(w)) break;
        const uint32_t tm = tm0 + (local % kBufs) * kN;
        if constexpr (MODE == kVgGrad) {
          const float l2 = row_lse * kLog2e, gi = row_dloss / s;
          const int rel = tgt - a.v0;   // column of the target in this piece (maybe outside)
#pragma unroll 1
          for (int c = 0; c < kCols / 64; ++c) {
            float v[64];
            tmem_ld64(tm + 64 * c, v);
            if (c + 1 == kCols / 64) release();
            const int cc = col0 + 64 * c;
            const bool here = static_cast<unsigned>(rel - cc) < 64u;
            float at = 0.f;   // the target's value
            if (here) {
#pragma unroll
              for (int j = 0; j < 64; ++j) at = rel - cc == j ? v[j] : at;
              at = expm1f(at - row_lse) * gi;
            }
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
              const float2 x = ffma2(make_float2(v[j], v[j + 1]), make_float2(kLog2e, kLog2e), make_float2(-l2, -l2));
              const float2 p = fmul2(make_float2(ex2_fast(x.x), ex2_fast(x.y)), make_float2(gi, gi));
              v[j] = p.x, v[j + 1] = p.y;
            }
            if (tgt < 0 || cc + 64 > a.valid_n) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (tgt < 0 || cc + j >= a.valid_n) v[j] = 0.f;
            }
            vg_store_bf16<true>(scr, v, &m0.out, cc, row0, rows, here ? rel - cc : -1, at);
          }
        } else if (!w.second) {
          vg_scratch_free();
          float* dst = a.dh + (static_cast<int64_t>(w.split) * a.M + row0) * a.N + col0;
#pragma unroll 1
          for (int c = 0; c < kCols / 32; ++c) {
            float v[32];
            tmem_ld32(tm + 32 * c, v);
            if (c + 1 == kCols / 32) release();
            if (col0 + 32 * c < a.N) vg_store_f32(scr, v, dst + 32 * c, a.N, rows, a.add != 0);
          }
        } else {
          const int64_t at = static_cast<int64_t>(a.v0 + row0) * a.N + col0;
#pragma unroll 1
          for (int c = 0; c < kCols / 64; ++c) {
            float v[64];
            tmem_ld64(tm + 64 * c, v);
            if (c + 1 == kCols / 64) release();
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
              const float2 x = fmul2(make_float2(v[j], v[j + 1]), make_float2(s, s));
              v[j] = x.x, v[j + 1] = x.y;
            }
            if (col0 + 64 * c >= a.N) continue;
            if (a.dw) {
              float* dst = a.dw + at + 64 * c;
              vg_store_f32(scr, v, dst, a.N, rows, a.add != 0);
              vg_store_f32(scr, v + 32, dst + 32, a.N, rows, a.add != 0);
            } else {
              vg_store_bf16<false>(scr, v, &m1.out, col0 + 64 * c, a.v0 + row0, rows);
            }
          }
        }
      }
    }
    if (MODE != kVgStats && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // results written
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();   // no arrival or copy for the other CTA is outstanding
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, kBufs * kN);
    else
      tmem_dealloc(tmem, kBufs * kN);
  }
}

template <int MODE, bool LONG>
__global__ void __launch_bounds__(320, 1)
    vocab_gemm_kernel(const __grid_constant__ VgMaps m, const __grid_constant__ VgArgs a) {
  vocab_gemm<MODE, false, LONG>(m, a, m, a);
}
template <int MODE, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(320, 1)
    vocab_gemm_pair_kernel(const __grid_constant__ VgMaps m, const __grid_constant__ VgArgs a) {
  vocab_gemm<MODE, true, LONG>(m, a, m, a);
}
__global__ void __launch_bounds__(320, 1)
    vocab_back_kernel(const __grid_constant__ VgMaps mh, const __grid_constant__ VgArgs ah,
                      const __grid_constant__ VgMaps mw, const __grid_constant__ VgArgs aw) {
  vocab_gemm<kVgBack, false, false>(mh, ah, mw, aw);
}
template <bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(320, 1)
    vocab_back_pair_kernel(const __grid_constant__ VgMaps mh, const __grid_constant__ VgArgs ah,
                           const __grid_constant__ VgMaps mw, const __grid_constant__ VgArgs aw) {
  vocab_gemm<kVgBack, true, LONG>(mh, ah, mw, aw);
}

// The tiles' (max, sum) joined: a block has 4 tokens (one 32-byte sector of `part` a tile) x 128 lanes of tiles,
// so that a few tokens' thousand tiles are read in a few steps (7 tokens: 34 us with 16 lanes, 6 with 128).
__global__ void __launch_bounds__(512) vocab_loss_kernel(const float2* part, int parts, int part_ld, const float* zt,
                                                         Ids targets, int tokens, int vocab, float* loss, float* lse,
                                                         int* err) {
  __shared__ float2 red[16][4];
  const int tl = threadIdx.x & 3, g = threadIdx.x >> 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 4 + tl;
  const bool in = i < tokens;
  const int t = in ? targets.get(i) : -1;
  pdl_wait();
  const bool held = t >= 0 && t < vocab;
  const float z = held && threadIdx.x < 4 ? zt[i] : 0.f;
  float mx = -INFINITY, sum = 0.f;
  auto join = [&](float2 p) {
    const float m = fmaxf(mx, p.x);
    const float ref = m == -INFINITY ? 0.f : m;
    sum = sum * expf(mx - ref) + p.y * expf(p.x - ref);
    mx = m;
  };
  auto join_lanes = [&]() {   // lanes l and l + d hold the same token
#pragma unroll
    for (int d = 16; d >= 4; d >>= 1) {
      float2 q;
      q.x = __shfl_down_sync(0xffffffffu, mx, d);
      q.y = __shfl_down_sync(0xffffffffu, sum, d);
      join(q);
    }
  };
  if (in) {
#pragma unroll 8
    for (int p = g; p < parts; p += 128) join(part[static_cast<int64_t>(p) * part_ld + i]);
  }
  join_lanes();
  if (lane < 4) red[warp][lane] = make_float2(mx, sum);
  __syncthreads();
  if (warp != 0) return;
  mx = -INFINITY, sum = 0.f;
  join(red[lane >> 2][tl]);
  join(red[8 + (lane >> 2)][tl]);
  join_lanes();
  if (lane >= 4 || !in) return;
  const float l = mx + logf(sum);
  if (t >= vocab) raise_error(err, kErrBounds);
  lse[i] = l;
  // mx - z is exact near the target's logit, so a loss near zero keeps its own bits instead of those of lse; below zero
  // it is rounding
  const float nll = (mx - z) + logf(sum);
  loss[i] = !held ? 0.f : nll < 0.f ? 0.f : nll;
}

// dh = s * the sum of the splits, in order; four values a thread, sixteen splits requested together
template <typename To>
__global__ void __launch_bounds__(256) vocab_hidden_kernel(const float* part, int splits, int64_t n, const float* scale,
                                                           To* dh) {
  pdl_wait();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const float s = scale[0];
  float f[4] = {};
#pragma unroll 16
  for (int k = 0; k < splits; ++k) {
    const float4 p = *reinterpret_cast<const float4*>(part + k * n + i);
    f[0] += p.x, f[1] += p.y, f[2] += p.z, f[3] += p.w;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] *= s;
  store4(dh + i, f);
}

}  // namespace dm0
