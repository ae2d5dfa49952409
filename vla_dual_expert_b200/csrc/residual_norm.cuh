// The boundary between two blocks of a layer: the norm behind a block, its gate, the scaled residual, and
// the norm before the next block, in one pass over the rows.
//
//   u  = y r_post g_post            r_post = 1 / sqrt(mean(y^2) + eps)     (u = y without a post gain)
//   h' = alpha h + gate_s u
//   n  = h' r_pre g_pre (1 + scale_s) + shift_s                            r_pre = 1 / sqrt(mean(h'^2) + eps)
//
// gate, scale and shift are per sample s, or one row for all.  With x = h' r_pre, z = y r_post and
// a = g_pre (1 + scale_s) the adjoint is
//
//   dH  = dh' + r_pre (a dn - x mean(a dn x))          dh = alpha dH
//   dy  = r_post (w dH - z mean(w dH z)),              w = gate g_post    (dy = gate dH without a post gain)
//   A_s = sum dn x,  B_s = sum dn,  C_s = sum dH z     over the sample's rows:
//   dscale_s = g_pre A_s, dshift_s = B_s, dgate_s = g_post C_s,
//   dg_pre = sum_s (1 + scale_s) A_s, dg_post = sum_s gate_s C_s
//
// Bound by HBM: 12 bytes per value forward (fp32 h, bf16 y and n) and 18 backward.
#pragma once
#include "embedding.cuh"
#include "gemm.cuh"   // bf2

namespace dm0 {

constexpr int kRnMaxHidden = 8192;

struct RnArgs {
  int rows, H;
  int rows_per_sample;          // rows of one sample (per-sample vectors); >= 1
  float alpha, eps;
  const float *post_gain, *pre_gain;                  // [H] or null
  const float *gate, *mod_scale, *mod_shift;          // rows of [H], or null
  int gate_ld, mod_ld;          // elements between two samples' rows; 0: one row for all
};

// four consecutive values as fp32; a warp's pieces of four are adjacent, so its loads and stores are whole
// lines for both types
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&f)[4]) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(q.x << 16), f[1] = __uint_as_float(q.x & 0xffff0000u);
  f[2] = __uint_as_float(q.y << 16), f[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&f)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf2(f[0], f[1]), bf2(f[2], f[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// Forward: W warps per row, 16 values per thread in registers between the two norms.  Small blocks, so that
// many are resident and one row's loads overlap another's reductions and stores: 32768 x 2048 (fp32 h, bf16 y) in
// 124 us, 6.5 TB/s (264 us with a warp per row and 64 values a lane: one block per SM, loads and stores by turns).
template <typename Th, typename Ty, int W>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128) residual_norm_kernel(const Th* h, const Ty* y, RnArgs a,
                                                                            Th* h_out, __nv_bfloat16* n_out,
                                                                            float* r_post_out, float* r_pre_out) {
  pdl_wait();
  constexpr int NP = 4, kRows = W > 4 ? 1 : 4 / W, kT = 32 * W;
  __shared__ float red[2][kRows][W];
  const int rl = threadIdx.x / kT, t = threadIdx.x - rl * kT, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kRows + rl;
  if (row >= a.rows) return;   // whole groups of W warps, which share no barrier with the others
  const int64_t base = static_cast<int64_t>(row) * a.H;
  const float inv_h = 1.f / a.H;
  auto total = [&](float v, int which) {
    v = warp_sum(v);
    if (W == 1) return v;
    if (lane == 0) red[which][rl][t >> 5] = v;
    named_bar_sync(1 + rl, kT);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) s += red[which][rl][k];
    return s;
  };
  float v[NP][4], u[NP][4];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = (t + kT * i) * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[i][k] = u[i][k] = 0.f;
    if (c < a.H) {
      load4(h + base + c, v[i]);
      if (y) load4(y + base + c, u[i]);
    }
  }
  const int sample = row / a.rows_per_sample;
  if (y) {
    float rp = 1.f;
    if (a.post_gain) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) ss += u[i][k] * u[i][k];
      rp = rsqrtf(total(ss, 0) * inv_h + a.eps);
      if (t == 0) r_post_out[row] = rp;
    }
    const float* gate = a.gate ? a.gate + static_cast<int64_t>(sample) * a.gate_ld : nullptr;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = (t + kT * i) * 4;
      if (c >= a.H) continue;
      float g[4];
      if (a.post_gain) {
        load4(a.post_gain + c, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[i][k] *= rp * g[k];
      }
      if (gate) {
        load4(gate + c, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[i][k] *= g[k];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[i][k] = fmaf(a.alpha, v[i][k], u[i][k]);
      ss += v[i][k] * v[i][k];
    }
  const float r = rsqrtf(total(ss, 1) * inv_h + a.eps);
  if (t == 0) r_pre_out[row] = r;
  const int64_t mod = static_cast<int64_t>(sample) * a.mod_ld;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = (t + kT * i) * 4;
    if (c >= a.H) continue;
    store4(h_out + base + c, v[i]);
    float g[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[i][k] *= r;
    if (a.pre_gain) {
      load4(a.pre_gain + c, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] *= g[k];
    }
    if (a.mod_scale) {
      load4(a.mod_scale + mod + c, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] *= 1.f + g[k];
    }
    if (a.mod_shift) {
      load4(a.mod_shift + mod + c, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] += g[k];
    }
    store4(n_out + base + c, v[i]);
  }
}

// Backward over a stripe of one sample's rows: a thread owns 8 columns and keeps their sums A, B, C; the
// row's three sums (of a dn x, of w z (dh' + r a dn), of w z x, from which both means follow) take one block
// reduction.  The rows come by bulk copies into a ring of `stages` rows in shared memory, so the reads of
// later rows go on through a row's reduction and stores: 32768 x 2048 in 189 us at 6.2 TB/s and 10 us for the sums
// of the stripes (276 us in all with loads into registers, a row at a time).
//   part[stripe][3][H]: the stripe's A, B, C.
constexpr int kRnMaxStages = 4;
struct RnGradArgs {
  RnArgs f;
  const float *r_post, *r_pre;
  int stripes, per;     // stripes per sample, rows of a stripe
  int stages;
  float* part;
  int* err;
};

template <typename Tn, typename Th, typename Ty, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 2 : 1)
    residual_norm_grad_kernel(const Tn* dn, const Th* dh_out, const Th* h_out, const Ty* y, RnGradArgs a, Th* dh,
                              Ty* dy) {
  extern __shared__ __align__(16) uint8_t ring[];   // [stages][h_out | dh_out | dn | y] rows
  __shared__ uint64_t full[kRnMaxStages];
  __shared__ float4 red[2][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
  const int H = a.f.H;
  const int s = blockIdx.x / a.stripes, q = blockIdx.x - s * a.stripes;
  const int T = a.f.rows_per_sample;
  const int t0 = min(T, q * a.per), t1 = min(T, t0 + a.per);
  const float inv_h = 1.f / H;
  const uint32_t bh = H * sizeof(Th), bn = H * sizeof(Tn), by = y ? H * sizeof(Ty) : 0, bu = dh_out ? bh : 0;
  const uint32_t stage = bh + bu + bn + by;
  if (tid == 0) {
    for (int k = 0; k < a.stages; ++k) mbar_init(&full[k], 1);
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  auto fetch = [&](int t) {   // by thread 0
    const int k = (t - t0) % a.stages;
    uint8_t* d = ring + static_cast<size_t>(k) * stage;
    const int64_t at = static_cast<int64_t>(s * T + t) * H;
    mbar_arrive_expect_tx(&full[k], stage);
    bulk_load(d, h_out + at, bh, &full[k]);
    if (bu) bulk_load(d + bh, dh_out + at, bh, &full[k]);
    bulk_load(d + bh + bu, dn + at, bn, &full[k]);
    if (by) bulk_load(d + bh + bu + bn, y + at, by, &full[k]);
  };
  if (tid == 0)
    for (int t = t0; t < min(t1, t0 + a.stages); ++t) fetch(t);
  // a = g_pre (1 + scale), w = gate g_post of this thread's columns
  float ga[2][4], w[2][4];
  int col[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = col[i] = (tid + static_cast<int>(blockDim.x) * i) * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) ga[i][k] = w[i][k] = 1.f;
    if (c >= H) continue;
    float g[4];
    if (a.f.pre_gain) load4(a.f.pre_gain + c, ga[i]);
    if (a.f.mod_scale) {
      load4(a.f.mod_scale + static_cast<int64_t>(s) * a.f.mod_ld + c, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) ga[i][k] *= 1.f + g[k];
    }
    if (a.f.post_gain) load4(a.f.post_gain + c, w[i]);
    if (a.f.gate) {
      load4(a.f.gate + static_cast<int64_t>(s) * a.f.gate_ld + c, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[i][k] *= g[k];
    }
  }
  float A[2][4] = {}, B[2][4] = {}, C[2][4] = {};
  const bool post = a.f.post_gain != nullptr;
  bool ok = true;
  for (int t = t0; t < t1; ++t) {
    const int k0 = (t - t0) % a.stages;
    const int row = s * T + t;
    const float r = a.r_pre[row], rp = post ? a.r_post[row] : 1.f;
    if (ok && !mbar_wait(&full[k0], ((t - t0) / a.stages) & 1, nullptr)) {
      ok = false;   // the remaining rows are not waited for: the results are void and the error word says so
      raise_error(a.err, kErrTimeoutProducer);
    }
    const uint8_t* d0 = ring + static_cast<size_t>(k0) * stage;
    float d[2][4] = {}, x[2][4] = {}, z[2][4] = {};
    float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = col[i];
      if (c >= H) continue;
      float n[4];
      load4(reinterpret_cast<const Th*>(d0) + c, x[i]);
      if (bu) load4(reinterpret_cast<const Th*>(d0 + bh) + c, d[i]);
      load4(reinterpret_cast<const Tn*>(d0 + bh + bu) + c, n);
      if (by) load4(reinterpret_cast<const Ty*>(d0 + bh + bu + bn) + c, z[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[i][k] *= r;
        A[i][k] += n[k] * x[i][k];
        B[i][k] += n[k];
        const float dx = n[k] * ga[i][k];
        s1 += dx * x[i][k];
        d[i][k] += r * dx;   // dH without its mean term
        z[i][k] *= rp;
        if (post) {
          s2 += w[i][k] * z[i][k] * d[i][k];
          s3 += w[i][k] * z[i][k] * x[i][k];
        }
      }
    }
    float4* rd = red[t & 1];
    s1 = warp_sum(s1);
    if (post) s2 = warp_sum(s2), s3 = warp_sum(s3);
    if (lane == 0) rd[warp] = make_float4(s1, s2, s3, 0.f);
    __syncthreads();   // every thread has read the row's slot
    if (tid == 0 && ok && t + a.stages < t1) fetch(t + a.stages);
    s1 = s2 = s3 = 0.f;
    for (int k = 0; k < nw; ++k) {
      const float4 p = rd[k];
      s1 += p.x, s2 += p.y, s3 += p.z;
    }
    const float m1 = r * s1 * inv_h;
    const float m2 = (s2 - m1 * s3) * inv_h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = col[i];
      if (c >= H) continue;
      const int64_t at = static_cast<int64_t>(row) * H + c;
      float o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        d[i][k] -= m1 * x[i][k];
        o[k] = a.f.alpha * d[i][k];
        C[i][k] += d[i][k] * z[i][k];
      }
      store4(dh + at, o);
      if (by) {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = post ? rp * (w[i][k] * d[i][k] - z[i][k] * m2) : w[i][k] * d[i][k];
        store4(dy + at, o);
      }
    }
  }
  if (!ok)   // copies in flight land before the block's shared memory is released
    for (int k = 0; k < a.stages; ++k)
      if (!mbar_wait(&full[k], 0, nullptr, kDrainTimeoutNs)) mbar_wait(&full[k], 1, nullptr, kDrainTimeoutNs);
  if (!a.part) return;
  float* p = a.part + static_cast<int64_t>(blockIdx.x) * 3 * H;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (col[i] >= H) continue;
    store4(p + col[i], A[i]);
    store4(p + H + col[i], B[i]);
    store4(p + 2 * H + col[i], C[i]);
  }
}

// Sums of the stripes in a fixed order, per sample and over the samples.  Block: 32 columns x 32 groups; up to
// 32 samples at a time, 32 / samples groups sharing a sample's stripes.
struct RnSumArgs {
  RnArgs f;
  int samples, stripes;
  const float* part;
  float *d_post, *d_gate, *d_pre, *d_scale, *d_shift;   // null: not wanted
};
__global__ void __launch_bounds__(1024) residual_norm_sum_kernel(RnSumArgs a) {
  pdl_wait();
  __shared__ float red[5][32][33];
  const int cl = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int H = a.f.H, c = blockIdx.x * 32 + cl;
  const bool in = c < H;
  const float gp = in && a.f.pre_gain ? a.f.pre_gain[c] : 1.f;
  const float gq = in && a.f.post_gain ? a.f.post_gain[c] : 1.f;
  const int at_once = min(32, a.samples), parts = 32 / at_once;
  const int sl = g / parts, part = g - sl * parts;   // (sl >= at_once: idle)
  float all[5] = {};   // of this group's samples: pre gain, post gain, shared gate, scale, shift
  for (int s0 = 0; s0 < a.samples; s0 += at_once) {
    const int s = s0 + sl;
    const bool mine = in && sl < at_once && s < a.samples;
    float t[3] = {};
    if (mine) {
#pragma unroll 4
      for (int q = part; q < a.stripes; q += parts) {
        const float* p = a.part + (static_cast<int64_t>(s) * a.stripes + q) * 3 * H + c;
        t[0] += p[0], t[1] += p[H], t[2] += p[2 * H];
      }
    }
    if (parts > 1) {
      __syncthreads();
      for (int k = 0; k < 3; ++k) red[k][g][cl] = t[k];
      __syncthreads();
      if (mine && part == 0)
        for (int j = 1; j < parts; ++j)
          for (int k = 0; k < 3; ++k) t[k] += red[k][g + j][cl];
    }
    if (mine && part == 0) {
      const float A = t[0], B = t[1], C = t[2];
      const float ms = a.f.mod_scale ? 1.f + a.f.mod_scale[static_cast<int64_t>(s) * a.f.mod_ld + c] : 1.f;
      const float gt = a.f.gate ? a.f.gate[static_cast<int64_t>(s) * a.f.gate_ld + c] : 1.f;
      all[0] += ms * A;
      all[1] += gt * C;
      all[2] += gq * C;
      all[3] += gp * A;
      all[4] += B;
      if (a.d_scale && a.f.mod_ld) a.d_scale[static_cast<int64_t>(s) * H + c] = gp * A;
      if (a.d_shift && a.f.mod_ld) a.d_shift[static_cast<int64_t>(s) * H + c] = B;
      if (a.d_gate && a.f.gate_ld) a.d_gate[static_cast<int64_t>(s) * H + c] = gq * C;
    }
  }
  __syncthreads();
  for (int k = 0; k < 5; ++k) red[k][g][cl] = all[k];
  __syncthreads();
  if (g >= 5 || !in) return;
  float v = 0.f;   // one group per vector; idle groups hold zeros
  for (int k = 0; k < 32; ++k) v += red[g][k][cl];
  float* dst = g == 0 ? a.d_pre : g == 1 ? a.d_post : g == 2 ? (a.f.gate_ld ? nullptr : a.d_gate)
             : a.f.mod_ld ? nullptr : g == 3 ? a.d_scale : a.d_shift;
  if (dst) dst[c] = v;
}

}  // namespace dm0
