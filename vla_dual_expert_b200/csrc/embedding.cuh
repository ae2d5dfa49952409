// Token embedding rows and their gradient.
//
//   forward   out[r] = scale * E[id_r]                    (id_r < 0: a zero row)
//   gradient  dE[v]  = scale * sum over { r : id_r = v } of dout[r], r ascending
//
// The gradient adds in an order that the ids alone fix, without float atomics: the positions are sorted
// by id (stable, so ascending within an id), the sorted list is cut into tiles of kEmbTile positions,
// each tile adds its rows segment by segment in fp32, and a segment that crosses tiles leaves one
// partial per tile, which a second pass adds in tile order.
#pragma once
#include "ptx.cuh"

namespace dm0 {

// Values that an earlier kernel of the same call wrote are read with plain loads: a read-only load may be
// moved above griddepcontrol.wait.

// row `r` of a [B][T][H] tensor with batch and token strides (elements)
struct RowsView {
  int64_t batch_stride, row_stride;
  int tokens;   // T
  __device__ __forceinline__ int64_t off(int r) const {
    const int b = r / tokens;
    return b * batch_stride + (r - b * tokens) * row_stride;
  }
};

struct Ids {
  const void* p;
  int wide;   // 1: int64, 0: int32
  // ids outside int32 keep their meaning: negative stays negative, too large stays too large
  __device__ __forceinline__ int get(int64_t i) const {
    if (!wide) return __ldg(static_cast<const int*>(p) + i);
    const long long v = __ldg(static_cast<const long long*>(p) + i);
    return v < 0 ? -1 : (v > 0x7fffffffll ? 0x7fffffff : static_cast<int>(v));
  }
};

__device__ __forceinline__ void bf8_to_f32(const uint4& q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 f32_to_bf8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// eight consecutive values of a bf16 or fp32 row as fp32
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  bf8_to_f32(__ldg(reinterpret_cast<const uint4*>(p)), f);
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
// the same for memory that this launch or an overlapping one writes (no read-only path)
__device__ __forceinline__ void load8_rw(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = f32_to_bf8(f);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// One warp per row; a lane's 16-byte pieces of the row are requested together.  Bound by HBM: 32768 rows of 2048 in
// 38 us, 7.0 TB/s of rows read and written (some of the frequent rows come from L2); one row by the launch, 4 us.
template <typename To>
__global__ void __launch_bounds__(256) embed_kernel(const __nv_bfloat16* table, Ids ids, int n, int vocab, int H,
                                                    float scale, To* out, RowsView ov, int* err) {
  pdl_wait();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= n) return;
  const int id = ids.get(r);
  if (id >= vocab && lane == 0) raise_error(err, kErrBounds);
  const bool held = id >= 0 && id < vocab;
  const __nv_bfloat16* src = table + static_cast<int64_t>(held ? id : 0) * H;
  To* dst = out + ov.off(r);
  for (int c0 = lane * 8; c0 < H; c0 += 8 * 256) {
    uint4 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + 256 * i;
      q[i] = held && c < H ? __ldg(reinterpret_cast<const uint4*>(src + c)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + 256 * i;
      if (c >= H) continue;
      float f[8];
      bf8_to_f32(q[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = held ? f[j] * scale : 0.f;   // a missing row is +0 for any scale
      store8(dst + c, f);
    }
  }
}

// ---------------------------------------------------------------- gradient: positions sorted by id
constexpr int kEmbTile = 32;        // sorted positions per tile of the sums; a longer segment is cut at tiles
constexpr int kSortWarps = 16;
constexpr int kSortMaxRows = 1600;  // vocabulary rows of one sorting CTA: 16 warps x 1600 counters = 100 KB
constexpr int kSortList = 512;      // of its own ids, that a warp keeps between the passes
constexpr int kSortZero = 1 << 16;  // bytes that one of the sort's zeroing CTAs writes

// Scratch of one gradient.  Sorted place i holds position perm[i] of id row_of[i]; seg[v] is the range of
// places of id v; total[0] the number of places; long_row[t] the id whose segment of more than kEmbTile
// places begins in tile t, or -1 (there is at most one: it reaches behind the tile).
struct EmbScratch {
  int *perm, *row_of, *total, *long_row;
  int2* seg;
  float* part;   // [tile][2][H]: the tile's sums of a cut segment that began before it, and of one that begins in it
};

// Each of G CTAs (a power of two) owns the ids v with v mod G = its index, so that neighbouring frequent ids
// fall to different CTAs.  Each reads every id: it counts those of smaller owners (its place in the sorted list,
// so the CTAs need no exchange) and its own per (warp, row), warp w taking the w-th stretch of positions and
// listing its own; after a scan it writes the listed positions in (row, position) order (a warp with more than
// kSortList of them reads its stretch again).  The ids come from L2, G times.  An entry's rank among equal ids of
// its 32 is counted over the lanes.  32768 tokens x 131072 rows, 6% of the tokens one id: 25 us; 37 with every id
// read and tested in both passes, and match.any for the ranks took 10 us more.
// The sort leaves HBM idle, so the CTAs behind the first G write zeros meanwhile: `zero_bytes` of the gradient
// from `zero`, the rows of the highest ids, whether their ids occur or not (the sums come later).
template <typename Id>
__global__ void __launch_bounds__(kSortWarps * 32, 2) embed_sort_kernel(const Id* ids, int n, int vocab, int log_g, int rows,
                                                                        EmbScratch o, uint8_t* zero,
                                                                        int64_t zero_bytes, int* err) {
  extern __shared__ int cnt[];   // [kSortWarps][rows], then the lists
  __shared__ int warp_tot[kSortWarps], below_tot[kSortWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int own = blockIdx.x, mask = (1 << log_g) - 1;
  if (own > mask) {
    pdl_wait();
    int64_t at = static_cast<int64_t>(own - mask - 1) * kSortZero + tid * 16;
#pragma unroll
    for (int k = 0; k < kSortZero / (kSortWarps * 32 * 16); ++k, at += kSortWarps * 32 * 16)
      if (at < zero_bytes) __stcs(reinterpret_cast<float4*>(zero + at), make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  const int nb = (vocab - own + mask) >> log_g;   // ids own, own + G, ... below vocab
  for (int i = tid; i < kSortWarps * rows; i += blockDim.x) cnt[i] = 0;
  pdl_wait();
  __syncthreads();
  const int chunk = (((n + kSortWarps - 1) / kSortWarps) + 31) & ~31;
  // the CTAs start at different stretches, or all would ask the same L2 slices at once
  const int stretch = (warp + own) % kSortWarps;
  const int p0 = min(n, stretch * chunk), p1 = min(n, p0 + chunk);
  int* mine = cnt + stretch * rows;
  int* list = cnt + kSortWarps * rows + warp * kSortList;   // this warp's own ids: place in the stretch, row (11 bits)
  int below = 0, listed = 0;
  bool bad = false;
  // 1024 positions of a warp at a time, sixteen requested together.  -1: not a token
  constexpr int U = 32;
  int id[U];
  auto fetch = [&](int b) {
#pragma unroll
    for (int u0 = 0; u0 < U; u0 += 16) {
      if (b + 32 * u0 >= p1) break;
      Id raw[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int p = b + 32 * (u0 + u) + lane;
        raw[u] = p < p1 ? __ldg(ids + p) : Id(-1);
      }
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        bad |= raw[u] >= vocab;
        id[u0 + u] = raw[u] >= 0 && raw[u] < vocab ? static_cast<int>(raw[u]) : -1;
      }
    }
  };
  for (int b = p0; b < p1; b += 32 * U) {
    fetch(b);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + 32 * u >= p1) break;
      const int k = id[u] & mask;
      if (id[u] >= 0) below += k < own;
      const bool in = id[u] >= 0 && k == own;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (!act) continue;
      const int at = listed + __popc(act & ((1u << lane) - 1u));
      listed += __popc(act);
      if (!in) continue;
      atomicAdd(&mine[id[u] >> log_g], 1);
      if (at < kSortList) list[at] = ((b + 32 * u + lane - p0) << 11) | (id[u] >> log_g);
    }
  }
  if (bad && blockIdx.x == 0) raise_error(err, kErrBounds);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) below += __shfl_xor_sync(0xffffffffu, below, d);
  if (lane == 0) below_tot[warp] = below;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) base += below_tot[w];
  // exclusive scan over (row, warp), a row per thread at a time
  int carry = base;
  for (int r0 = 0; r0 < nb; r0 += kSortWarps * 32) {
    const int r = r0 + tid;
    int tot = 0;
    if (r < nb) {
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) tot += cnt[w * rows + r];
    }
    int inc = tot;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int pre = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      pre += w < warp ? warp_tot[w] : 0;
      all += warp_tot[w];
    }
    if (r < nb) {
      int at = carry + pre + inc - tot;
      o.seg[(static_cast<int64_t>(r) << log_g) + own] = make_int2(at, at + tot);
      if (tot)
        for (int w = 0; w < kSortWarps; ++w) {
          const int k = cnt[w * rows + r];
          cnt[w * rows + r] = at;
          at += k;
        }
    }
    carry += all;
    __syncthreads();
  }
  if (tid == 0 && own == mask) o.total[0] = carry;
  if (carry == base) return;   // none of its ids occurs
  // places within a row, 32 entries of the stretch at a time
  auto place = [&](bool in, int bin, int position) {
    int rank = 0, same = 0;
    for (unsigned rest = __ballot_sync(0xffffffffu, in); rest; rest &= rest - 1) {
      const int l = __ffs(rest) - 1;
      const bool eq = __shfl_sync(0xffffffffu, bin, l) == bin;
      same += eq;
      rank += eq && l < lane;
    }
    if (in) {
      const int at = mine[bin] + rank;
      o.perm[at] = position;
      o.row_of[at] = (bin << log_g) + own;
    }
    __syncwarp();
    if (in && rank == 0) mine[bin] += same;
    __syncwarp();
  };
  if (listed <= kSortList) {
    for (int b = 0; b < listed; b += 32) {
      const bool in = b + lane < listed;
      const int e = in ? list[b + lane] : 0;
      place(in, in ? e & 2047 : -1, p0 + (e >> 11));
    }
    return;
  }
  for (int b = p0; b < p1; b += 32 * U) {   // too many for the list: the ids once more
    fetch(b);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + 32 * u >= p1) break;
      const bool in = id[u] >= 0 && (id[u] & mask) == own;
      if (__ballot_sync(0xffffffffu, in)) place(in, in ? id[u] >> log_g : -1, b + 32 * u + lane);
    }
  }
}

// eight values as they were loaded, so that a batch of rows waits in half the registers when they are bf16
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&f)[8]) const { bf8_to_f32(q, f); }
};
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = v[k];
  }
};

// Sums of the sorted rows.  A summing block has one tile x 2048 columns, a thread owning 8 columns and
// walking the tile's rows, eight requested ahead.  A segment of up to kEmbTile places belongs whole to the tile
// where it begins (at most 63 rows a tile); a longer one is cut at the tiles and leaves partial sums.  The
// other blocks write the zero rows of ids below zero_rows that never occur (none when the gradient is added to).
// Bound by HBM: 32768 tokens of 2048 in bf16 into 131072 fp32 rows, 154 us for 0.93 GB at 6.0 TB/s (215 us with the
// zeroing blocks behind the summing ones and tiles of 64 places at half the blocks per SM).
constexpr int kEmbCols = 2048;   // columns of one block: 256 threads x 8
constexpr int kEmbZeroRows = 16;
template <typename Td>
__global__ void __launch_bounds__(256, sizeof(Td) == 2 ? 4 : 3) embed_sum_kernel(EmbScratch o, const Td* dout, RowsView dv, int H,
                                                        float scale, float* grad, int accumulate, int tiles,
                                                        int slices, int zero_rows) {
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  // three zeroing blocks behind each summing one, so that the stores of the ones fill the latencies of the others
  // and no sum begins late
  const int sums = tiles * slices, b = blockIdx.x;
  const int step = min(4, static_cast<int>(gridDim.x) / sums);
  if (b % step != 0 || b / step >= sums) {
    const int v0 = (b - min(sums, b / step + 1)) * kEmbZeroRows;
    const int my = v0 + (tid & 31);
    const bool none = (tid & 31) < kEmbZeroRows && my < zero_rows && o.seg[my].x == o.seg[my].y;
    for (unsigned todo = __ballot_sync(0xffffffffu, none); todo; todo &= todo - 1) {
      float4* dst = reinterpret_cast<float4*>(grad + static_cast<int64_t>(v0 + __ffs(todo) - 1) * H);
      for (int c = tid; c < H / 4; c += blockDim.x) __stcs(dst + c, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    return;
  }
  const int tile = b / step / slices, slice = b / step - tile * slices;
  const int m = o.total[0];
  const int i0 = tile * kEmbTile;
  __shared__ int64_t src[2 * kEmbTile];
  __shared__ int row[2 * kEmbTile];
  __shared__ int range[2], cut[2];   // places of this tile; whether its first / last segment is cut
  if (tid == 0) {
    int a = i0, z = min(m, i0 + kEmbTile), first = 0, last = 0, lrow = -1;
    if (a < z) {
      const int2 g0 = o.seg[o.row_of[a]];
      first = g0.y - g0.x > kEmbTile && g0.x < a;           // goes on from an earlier tile
      if (!first && g0.x < a) a = g0.y;                     // whole in an earlier tile
      const int v1 = o.row_of[z - 1];
      const int2 g1 = o.seg[v1];
      if (g1.y - g1.x > kEmbTile) {
        if (g1.x >= i0) last = 1, lrow = v1;                // begins here, goes on behind
      } else if (g1.x >= i0) {
        z = g1.y;
      }
    }
    range[0] = a, range[1] = z, cut[0] = first, cut[1] = last;
    if (slice == 0) o.long_row[tile] = lrow;
  }
  __syncthreads();
  const int b0 = range[0], cnt = range[1] - b0;
  if (cnt <= 0) return;
  if (tid < cnt) {
    src[tid] = dv.off(o.perm[b0 + tid]);
    row[tid] = o.row_of[b0 + tid];
  }
  __syncthreads();
  const int c = slice * kEmbCols + tid * 8;
  if (c >= H) return;
  float acc[8] = {};
  for (int j0 = 0; j0 < cnt; j0 += 8) {
    Raw8<Td> raw[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j0 + u < cnt) raw[u].load(dout + src[j0 + u] + c);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u;
      if (j >= cnt) break;
      float f[8];
      raw[u].get(f);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += f[k];
      if (j + 1 < cnt && row[j + 1] == row[j]) continue;
      // the sum of row[j] in this tile is complete
      const bool head = cut[0] && row[j] == row[0], tail = cut[1] && j + 1 == cnt;
      if (head || tail) {
        store8(o.part + (static_cast<int64_t>(tile) * 2 + (head ? 0 : 1)) * H + c, acc);
      } else {
        float* dst = grad + static_cast<int64_t>(row[j]) * H + c;
        float d[8] = {};
        if (accumulate) load8_rw(dst, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = accumulate ? d[k] + scale * acc[k] : scale * acc[k];
        store8(dst, d);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    }
  }
}

// The cut segments: for each that begins in one of the block's 32 tiles, its partials are added in tile order,
// by four groups of 64 lanes that take stretches of the tiles, then the groups' sums in order.
constexpr int kFixCols = 256;   // columns of one block: 64 lanes x 4
constexpr int kFixTiles = 32;
__global__ void __launch_bounds__(256) embed_join_kernel(EmbScratch o, int tiles, int H, float scale, float* grad,
                                                         int accumulate) {
  pdl_wait();
  const int t0 = blockIdx.x * kFixTiles;
  const int l = threadIdx.x & 31;
  const int my = t0 + l < tiles ? o.long_row[t0 + l] : -1;
  const int g = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = blockIdx.y * kFixCols + lane * 4;
  __shared__ float4 sum[4][64];
  for (unsigned todo = __ballot_sync(0xffffffffu, my >= 0); todo; todo &= todo - 1) {   // the same in every warp
    const int at = __ffs(todo) - 1;
    const int v = __shfl_sync(0xffffffffu, my, at), tile = t0 + at;
    const int cnt = (o.seg[v].y - 1) / kEmbTile - tile + 1;   // partials [tile][1], [tile + 1 ...][0]
    const int per = (cnt + 3) / 4, k0 = g * per, k1 = min(cnt, k0 + per);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < H) {
#pragma unroll 8
      for (int k = k0; k < k1; ++k) {
        const int64_t slot = static_cast<int64_t>(tile + k) * 2 + (k == 0 ? 1 : 0);
        const float4 p = *reinterpret_cast<const float4*>(o.part + slot * H + c);
        s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
      }
    }
    sum[g][lane] = s;
    __syncthreads();
    if (g == 0 && c < H) {
      for (int k = 1; k < 4; ++k) {
        const float4 p = sum[k][lane];
        s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
      }
      float4* dst = reinterpret_cast<float4*>(grad + static_cast<int64_t>(v) * H + c);
      float4 d = make_float4(scale * s.x, scale * s.y, scale * s.z, scale * s.w);
      if (accumulate) {
        const float4 old = *dst;
        d = make_float4(d.x + old.x, d.y + old.y, d.z + old.z, d.w + old.w);
      }
      *dst = d;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- gradient of few tokens in one launch
// The same sums for up to kEmbFew tokens: each owner lists its tokens in order (their places among the list's equal
// ids by comparing with the entries before, of which there are n / G as a rule), adds them, and writes the zero
// rows of its own ids, so that nothing waits for another launch.  A warp adds up to kEmbTile rows of one id and 256
// columns; a longer segment is cut as above and its partials joined by the same block.
// One launch against three, at 4500 rows of 1232 (32003 of 1024): 48 tokens 8 against 18 us (23 against 27), 256
// tokens 12 against 18 (23 against 27).  The price is one block's bandwidth for a frequent id: 256 tokens of one
// id 33 against 18 us (41 against 29), 512 already 55 (59), so more tokens take the three launches.
constexpr int kEmbFew = 256;
template <typename Id, typename Td>
__global__ void __launch_bounds__(512, 1) embed_few_kernel(const Id* ids, int n, int vocab, int log_g, int rows,
                                                           const Td* dout, RowsView dv, int H, float scale, float* grad,
                                                           int accumulate, float* part, int* err) {
  extern __shared__ int bins[];   // [rows + 1] first places
  __shared__ int2 listed[kEmbFew], sorted[kEmbFew];   // (row, position)
  __shared__ int piece[kEmbFew], pieces;              // places where a piece begins, and their number
  __shared__ int warp_n[16], below_n[16], scan[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int own = blockIdx.x, mask = (1 << log_g) - 1;
  const int nb = max(0, (vocab - own + mask) >> log_g);
  for (int i = tid; i <= rows; i += 512) bins[i] = 0;
  pdl_wait();
  const Id raw = tid < n ? __ldg(ids + tid) : Id(-1);   // a position per thread
  const bool bad = raw >= vocab;
  const int v = raw >= 0 && raw < vocab ? static_cast<int>(raw) : -1;
  int below = v >= 0 && (v & mask) < own;
  const int id = v >= 0 && (v & mask) == own ? v >> log_g : -1;
  const unsigned act = __ballot_sync(0xffffffffu, id >= 0);
  if (bad && own == 0) raise_error(err, kErrBounds);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) below += __shfl_xor_sync(0xffffffffu, below, d);
  if (lane == 0) warp_n[warp] = __popc(act), below_n[warp] = below;
  __syncthreads();
  int base = 0, at = 0, m = 0;   // places of smaller owners; this warp's first entry; entries
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    base += below_n[w];
    at += w < warp ? warp_n[w] : 0;
    m += warp_n[w];
  }
  if (id >= 0) {
    listed[at + __popc(act & ((1u << lane) - 1u))] = make_int2(id, tid);
    atomicAdd(&bins[id], 1);
  }
  __syncthreads();
  // bins: counts -> first places, kept beside the next row's as the segment's end
  int carry = 0;
  for (int r0 = 0; r0 < nb; r0 += 512) {
    const int r = r0 + tid, k = r < nb ? bins[r] : 0;
    int inc = k;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int pre = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      pre += w < warp ? scan[w] : 0;
      all += scan[w];
    }
    if (r < nb) bins[r] = carry + pre + inc - k;
    carry += all;
    __syncthreads();
  }
  if (tid == 0) bins[nb] = m;
  if (tid < m) {
    const int2 e = listed[tid];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < tid; ++j) rank += listed[j].x == e.x;
    sorted[bins[e.x] + rank] = e;
  }
  __syncthreads();
  // the pieces: at each segment's first place and every kEmbTile places on
  const bool begins = tid < m && (tid - bins[sorted[tid].x]) % kEmbTile == 0;
  const unsigned beg = __ballot_sync(0xffffffffu, begins);
  if (lane == 0) warp_n[warp] = __popc(beg);
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) before += w < warp ? warp_n[w] : 0;
  if (begins) piece[before + __popc(beg & ((1u << lane) - 1u))] = tid;
  if (tid == 511) pieces = before + __popc(beg);
  __syncthreads();
  const int chunks = (H + 255) / 256;
  auto slot = [&](int i) {   // of the cut piece that begins at place i: segments are told apart by their first piece
    return static_cast<int64_t>((base + i) / kEmbTile) * 2 + (i == bins[sorted[i].x] ? 1 : 0);
  };
  for (int t = warp; t < pieces * chunks; t += 16) {
    const int k0 = t / chunks, c = (t - k0 * chunks) * 256 + lane * 8;
    if (c >= H) continue;
    const int i = piece[k0], r = sorted[i].x, len = min(kEmbTile, bins[r + 1] - i);
    const bool whole = bins[r + 1] - bins[r] <= kEmbTile;
    float acc[8] = {};
    for (int j0 = 0; j0 < len; j0 += 8) {
      Raw8<Td> raw8[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < len) raw8[u].load(dout + dv.off(sorted[i + j0 + u].y) + c);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (j0 + u >= len) break;
        float f[8];
        raw8[u].get(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += f[k];
      }
    }
    if (whole) {
      float* dst = grad + ((static_cast<int64_t>(r) << log_g) + own) * H + c;
      float d[8] = {};
      if (accumulate) load8_rw(dst, d);
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = accumulate ? d[k] + scale * acc[k] : scale * acc[k];
      store8(dst, d);
    } else {
      store8(part + slot(i) * H + c, acc);
    }
  }
  if (!accumulate)
    for (int r = warp; r < nb; r += 16) {
      if (bins[r] != bins[r + 1]) continue;
      float4* dst = reinterpret_cast<float4*>(grad + ((static_cast<int64_t>(r) << log_g) + own) * H);
      for (int c = lane; c < H / 4; c += 32) __stcs(dst + c, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  if (m <= kEmbTile) return;   // nothing was cut
  __syncthreads();
  for (int i = 0; i < m;) {
    const int r = sorted[i].x, end = bins[r + 1];
    if (end - i > kEmbTile)
      for (int c = tid * 4; c < H; c += 2048) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int j = i; j < end; j += kEmbTile) {
          const float4 p = *reinterpret_cast<const float4*>(part + slot(j) * H + c);
          s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
        }
        float4* dst = reinterpret_cast<float4*>(grad + ((static_cast<int64_t>(r) << log_g) + own) * H + c);
        float4 d = make_float4(scale * s.x, scale * s.y, scale * s.z, scale * s.w);
        if (accumulate) {
          const float4 old = *dst;
          d = make_float4(d.x + old.x, d.y + old.y, d.z + old.z, d.w + old.w);
        }
        *dst = d;
      }
    i = end;
  }
}

}  // namespace dm0
