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

// One warp per row; a lane's 16-byte pieces of the row are requested together.  Bound by HBM.
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
constexpr int kEmbTile = 64;        // sorted positions per tile of the sums
constexpr int kSortWarps = 32;
constexpr int kSortMaxRows = 1600;  // vocabulary rows of one sorting CTA: 32 warps x 1600 counters = 200 KB

// Each CTA owns `rows` consecutive vocabulary rows and reads every id: it counts the ids below its range
// (its place in the sorted list, so the CTAs need no exchange), counts its own ids per (warp, row) with
// warp w taking the w-th stretch of positions, and writes the positions in (row, position) order.  Ids are
// read from L2 by every CTA: 148 x n x 8 bytes, 2 x 39 MB at 32768 tokens.
//   perm[i], row_of[i]: position and id of sorted place i;  start[v]: first place of row v;
//   start[vocab]: number of positions with a token.
__global__ void __launch_bounds__(kSortWarps * 32) embed_sort_kernel(Ids ids, int n, int vocab, int rows, int* perm,
                                                                     int* row_of, int* start, int* err) {
  extern __shared__ int cnt[];   // [kSortWarps][rows], then the scan's warp totals
  __shared__ int warp_tot[kSortWarps], below_tot[kSortWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = blockIdx.x * rows, nb = min(rows, vocab - v0);
  for (int i = tid; i < kSortWarps * rows; i += blockDim.x) cnt[i] = 0;
  pdl_wait();
  __syncthreads();
  const int chunk = (((n + kSortWarps - 1) / kSortWarps) + 31) & ~31;
  const int p0 = min(n, warp * chunk), p1 = min(n, p0 + chunk);
  int* mine = cnt + warp * rows;
  int below = 0;
  bool bad = false;
  constexpr int U = 8;
  for (int b = p0; b < p1; b += 32 * U) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = b + 32 * u + lane;
      id[u] = p < p1 ? ids.get(p) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bad |= id[u] >= vocab;
      below += id[u] >= 0 && id[u] < v0;
      const unsigned bin = static_cast<unsigned>(id[u] - v0);
      const bool in = id[u] >= 0 && bin < static_cast<unsigned>(nb);
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        const unsigned peers = __match_any_sync(act, bin);
        if (lane == __ffs(peers) - 1) mine[bin] += __popc(peers);
      }
      __syncwarp();
    }
  }
  if (bad && blockIdx.x == 0) raise_error(err, kErrBounds);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 0) below_tot[warp] = below;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < kSortWarps; ++w) base += below_tot[w];
  // exclusive scan over (row, warp), rows in blocks of 1024
  int carry = base;
  for (int r0 = 0; r0 < nb; r0 += kSortWarps * 32) {
    const int r = r0 + tid;
    int tot = 0;
    if (r < nb)
      for (int w = 0; w < kSortWarps; ++w) tot += cnt[w * rows + r];
    int inc = tot;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int pre = 0, all = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      pre += w < warp ? warp_tot[w] : 0;
      all += warp_tot[w];
    }
    if (r < nb) {
      int at = carry + pre + inc - tot;
      start[v0 + r] = at;
      for (int w = 0; w < kSortWarps; ++w) {
        const int k = cnt[w * rows + r];
        cnt[w * rows + r] = at;
        at += k;
      }
    }
    carry += all;
    __syncthreads();
  }
  if (tid == 0 && v0 + nb == vocab) start[vocab] = carry;
  for (int b = p0; b < p1; b += 32 * U) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = b + 32 * u + lane;
      id[u] = p < p1 ? ids.get(p) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned bin = static_cast<unsigned>(id[u] - v0);
      const bool in = id[u] >= 0 && bin < static_cast<unsigned>(nb);
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        const unsigned peers = __match_any_sync(act, bin);
        const int lead = __ffs(peers) - 1;
        int at = 0;
        if (lane == lead) {
          at = mine[bin];
          mine[bin] = at + __popc(peers);
        }
        at = __shfl_sync(peers, at, lead) + __popc(peers & ((1u << lane) - 1u));
        perm[at] = b + 32 * u + lane;
        row_of[at] = id[u];
      }
      __syncwarp();
    }
  }
}

// Sums of the sorted rows.  Blocks [0, tiles * slices): one tile of sorted positions x 2048 columns, a
// thread owning 8 columns and walking the tile's rows, eight requested ahead.  The remaining blocks write
// the zero rows of ids that never occur (only when the gradient is written, not added to).
//   part[tile][0]: the tile's sum of a segment that began before it; part[tile][1]: of one that goes on
//   behind it.
constexpr int kEmbCols = 2048;   // columns of one block: 256 threads x 8
constexpr int kEmbZeroRows = 16;
template <typename Td>
__global__ void __launch_bounds__(256) embed_sum_kernel(const int* perm, const int* row_of, const int* start,
                                                        const Td* dout, RowsView dv, int n, int vocab, int H,
                                                        float scale, float* grad, int accumulate, float* part,
                                                        int tiles, int slices) {
  pdl_wait();
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) >= tiles * slices) {
    const int v0 = (blockIdx.x - tiles * slices) * kEmbZeroRows;
    for (int v = v0; v < min(vocab, v0 + kEmbZeroRows); ++v) {
      if (start[v] != start[v + 1]) continue;
      float4* dst = reinterpret_cast<float4*>(grad + static_cast<int64_t>(v) * H);
      for (int c = tid; c < H / 4; c += blockDim.x) __stcs(dst + c, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    return;
  }
  const int tile = blockIdx.x / slices, slice = blockIdx.x - tile * slices;
  const int m = start[vocab];
  const int i0 = tile * kEmbTile, i1 = min(m, i0 + kEmbTile);
  if (i0 >= i1) return;
  __shared__ int64_t src[kEmbTile];
  __shared__ int row[kEmbTile + 1], beg, end;
  if (tid < kEmbTile) {
    const int i = i0 + tid;
    src[tid] = i < i1 ? dv.off(perm[i]) : 0;
    row[tid] = i < i1 ? row_of[i] : -1;
  }
  if (tid == 0) {
    row[kEmbTile] = -1;
    beg = start[row_of[i0]];          // where the tile's first segment begins
    end = start[row_of[i1 - 1] + 1];  // where its last one ends
  }
  __syncthreads();
  const int c = slice * kEmbCols + tid * 8;
  if (c >= H) return;
  float acc[8] = {};
  const int cnt = i1 - i0;
  for (int j0 = 0; j0 < cnt; j0 += 8) {
    float f[8][8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j0 + u < cnt) load8(dout + src[j0 + u] + c, f[u]);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u;
      if (j >= cnt) break;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += f[u][k];
      if (j + 1 < cnt && row[j + 1] == row[j]) continue;
      // the segment of row[j] ends in this tile, or the tile ends
      const bool first = row[j] == row[0], last = j + 1 == cnt;
      const bool opened = first && beg < i0, open = last && end > i0 + kEmbTile;
      float* dst;
      if (opened || open) {
        dst = part + (static_cast<int64_t>(tile) * 2 + (opened ? 0 : 1)) * H + c;
        store8(dst, acc);
      } else {
        dst = grad + static_cast<int64_t>(row[j]) * H + c;
        float o[8] = {};
        if (accumulate) load8_rw(dst, o);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = accumulate ? o[k] + scale * acc[k] : scale * acc[k];
        store8(dst, o);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    }
  }
}

// The segments that cross tiles: the block of the tile where one begins adds its partials in tile order.
// Eight groups of 32 lanes take stretches of the tiles, then the groups' sums are added in order.
constexpr int kFixCols = 128;   // columns of one block: 32 lanes x 4
__global__ void __launch_bounds__(256) embed_join_kernel(const int* row_of, const int* start, int vocab, int H,
                                                         float scale, float* grad, int accumulate, const float* part) {
  pdl_wait();
  const int tile = blockIdx.x;
  const int m = start[vocab];
  const int i1 = (tile + 1) * kEmbTile;
  if (i1 >= m) return;   // the last tile: nothing goes on behind it
  const int v = row_of[i1 - 1];
  const int beg = start[v], end = start[v + 1];
  if (beg < tile * kEmbTile || end <= i1) return;   // begins elsewhere, or ends here
  const int t1 = (end - 1) / kEmbTile;              // last tile of the segment
  const int cnt = t1 - tile + 1;                    // partials: [tile][1], then [tile + 1 .. t1][0]
  const int g = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.y * kFixCols + lane * 4;
  const int per = (cnt + 7) / 8, k0 = g * per, k1 = min(cnt, k0 + per);
  __shared__ float4 sum[8][32];
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H) {
#pragma unroll 8
    for (int k = k0; k < k1; ++k) {
      const int64_t slot = static_cast<int64_t>(tile + k) * 2 + (k == 0 ? 1 : 0);
      const float4 p = *reinterpret_cast<const float4*>(part + slot * H + c);
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
  }
  sum[g][lane] = s;
  __syncthreads();
  if (g != 0 || c >= H) return;
  for (int k = 1; k < 8; ++k) {
    const float4 p = sum[k][lane];
    s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
  }
  float4* dst = reinterpret_cast<float4*>(grad + static_cast<int64_t>(v) * H + c);
  float4 o = make_float4(scale * s.x, scale * s.y, scale * s.z, scale * s.w);
  if (accumulate) {
    const float4 d = *dst;
    o = make_float4(o.x + d.x, o.y + d.y, o.z + d.z, o.w + d.w);
  }
  *dst = o;
}

}  // namespace dm0
