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

// Forward, W warps per row, each lane NP pieces of 8 values kept in registers between the two norms.
template <typename Th, typename Ty, int NP, int W>
__global__ void __launch_bounds__(256) residual_norm_kernel(const Th* h, const Ty* y, RnArgs a, Th* h_out,
                                                            __nv_bfloat16* n_out, float* r_post_out,
                                                            float* r_pre_out) {
  pdl_wait();
  constexpr int kRows = 8 / W;   // rows of a block
  __shared__ float red[2][kRows][W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rl = warp / W, wi = warp - rl * W;
  const int row = blockIdx.x * kRows + rl;
  const bool live = row < a.rows;
  if (W == 1 && !live) return;
  const int64_t base = static_cast<int64_t>(live ? row : 0) * a.H;
  const float inv_h = 1.f / a.H;
  auto col = [&](int i) { return (lane + 32 * (i + NP * wi)) * 8; };
  auto total = [&](float v, int which) {
    v = warp_sum(v);
    if (W == 1) return v;
    if (lane == 0) red[which][rl][wi] = v;
    __syncthreads();
    float t = 0.f;
    for (int k = 0; k < W; ++k) t += red[which][rl][k];
    return t;
  };
  float v[NP][8], u[NP][8];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = col(i);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] = u[i][k] = 0.f;
    if (live && c < a.H) {
      load8(h + base + c, v[i]);
      if (y) load8(y + base + c, u[i]);
    }
  }
  if (y) {
    float rp = 1.f;
    if (a.post_gain) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) ss += u[i][k] * u[i][k];
      rp = rsqrtf(total(ss, 0) * inv_h + a.eps);
      if (live && lane == 0 && wi == 0) r_post_out[row] = rp;
    }
    const float* gate = a.gate ? a.gate + static_cast<int64_t>(live ? row / a.rows_per_sample : 0) * a.gate_ld : nullptr;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = col(i);
      if (c >= a.H) continue;
      float g[8];
      if (a.post_gain) {
        load8(a.post_gain + c, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[i][k] *= rp * g[k];
      }
      if (gate) {
        load8(gate + c, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[i][k] *= g[k];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[i][k] = fmaf(a.alpha, v[i][k], u[i][k]);
      ss += v[i][k] * v[i][k];
    }
  const float r = rsqrtf(total(ss, 1) * inv_h + a.eps);
  if (!live) return;
  if (lane == 0 && wi == 0) r_pre_out[row] = r;
  const int64_t mod = static_cast<int64_t>(row / a.rows_per_sample) * a.mod_ld;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = col(i);
    if (c >= a.H) continue;
    store8(h_out + base + c, v[i]);
    float g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] *= r;
    if (a.pre_gain) {
      load8(a.pre_gain + c, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] *= g[k];
    }
    if (a.mod_scale) {
      load8(a.mod_scale + mod + c, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] *= 1.f + g[k];
    }
    if (a.mod_shift) {
      load8(a.mod_shift + mod + c, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] += g[k];
    }
    store8(n_out + base + c, v[i]);
  }
}

// Backward over a stripe of one sample's rows: a thread owns 8 columns and keeps their sums A, B, C; the
// row's three sums (of a dn x, of w z (dh' + r a dn), of w z x, from which both means follow) take one block
// reduction.
//   part[stripe][3][H]: the stripe's A, B, C.
struct RnGradArgs {
  RnArgs f;
  const float *r_post, *r_pre;
  int stripes;          // per sample
  float* part;
};

template <typename Tn, typename Th, typename Ty, int THREADS>
__global__ void __launch_bounds__(THREADS) residual_norm_grad_kernel(const Tn* dn, const Th* dh_out, const Th* h_out,
                                                                  const Ty* y, RnGradArgs a, Th* dh, Ty* dy) {
  pdl_wait();
  __shared__ float red[2][3][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
  const int H = a.f.H;
  const int c = tid * 8;
  const bool in = c < H;
  const int s = blockIdx.x / a.stripes, q = blockIdx.x - s * a.stripes;
  const int T = a.f.rows_per_sample;
  const int per = (T + a.stripes - 1) / a.stripes;
  const int t0 = min(T, q * per), t1 = min(T, t0 + per);
  const float inv_h = 1.f / H;
  float ga[8], w[8];   // a = g_pre (1 + scale), w = gate g_post
#pragma unroll
  for (int k = 0; k < 8; ++k) ga[k] = w[k] = 1.f;
  if (in) {
    float g[8];
    if (a.f.pre_gain) load8(a.f.pre_gain + c, ga);
    if (a.f.mod_scale) {
      load8(a.f.mod_scale + static_cast<int64_t>(s) * a.f.mod_ld + c, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) ga[k] *= 1.f + g[k];
    }
    if (a.f.post_gain) load8(a.f.post_gain + c, w);
    if (a.f.gate) {
      load8(a.f.gate + static_cast<int64_t>(s) * a.f.gate_ld + c, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] *= g[k];
    }
  }
  float A[8] = {}, B[8] = {}, C[8] = {};
  const bool post = a.f.post_gain != nullptr;
  for (int t = t0; t < t1; ++t) {
    const int row = s * T + t;
    const int64_t at = static_cast<int64_t>(row) * H + c;
    float n[8] = {}, d[8] = {}, x[8] = {}, z[8] = {};
    if (in) {
      load8(dn + at, n);
      load8(h_out + at, x);
      if (dh_out) load8(dh_out + at, d);
      if (y) load8(y + at, z);
    }
    const float r = a.r_pre[row], rp = post ? a.r_post[row] : 1.f;
    float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] *= r;
      A[k] += n[k] * x[k];
      B[k] += n[k];
      const float dx = n[k] * ga[k];
      s1 += dx * x[k];
      d[k] += r * dx;   // dH without its mean term
      z[k] *= rp;
      if (post) {
        s2 += w[k] * z[k] * d[k];
        s3 += w[k] * z[k] * x[k];
      }
    }
    float(*rd)[32] = red[t & 1];
    s1 = warp_sum(s1);
    if (post) s2 = warp_sum(s2), s3 = warp_sum(s3);
    if (lane == 0) rd[0][warp] = s1, rd[1][warp] = s2, rd[2][warp] = s3;
    __syncthreads();
    s1 = s2 = s3 = 0.f;
    for (int k = 0; k < nw; ++k) s1 += rd[0][k], s2 += rd[1][k], s3 += rd[2][k];
    const float m1 = r * s1 * inv_h;
    const float m2 = (s2 - m1 * s3) * inv_h;
    if (in) {
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        d[k] -= m1 * x[k];
        o[k] = a.f.alpha * d[k];
        C[k] += d[k] * z[k];
      }
      store8(dh + at, o);
      if (y) {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = post ? rp * (w[k] * d[k] - z[k] * m2) : w[k] * d[k];
        store8(dy + at, o);
      }
    }
  }
  if (in && a.part) {
    float* p = a.part + static_cast<int64_t>(blockIdx.x) * 3 * H + c;
    store8(p, A);
    store8(p + H, B);
    store8(p + 2 * H, C);
  }
}

// Sums of the stripes in order, per sample and over the samples.  Block: 32 columns x 32 lanes of stripes.
struct RnSumArgs {
  RnArgs f;
  int samples, stripes;
  const float* part;
  float *d_post, *d_gate, *d_pre, *d_scale, *d_shift;   // null: not wanted
};
__global__ void __launch_bounds__(1024) residual_norm_sum_kernel(RnSumArgs a) {
  pdl_wait();
  __shared__ float red[3][32][33];
  const int cl = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int H = a.f.H, c = blockIdx.x * 32 + cl;
  const bool in = c < H;
  const float gp = in && a.f.pre_gain ? a.f.pre_gain[c] : 1.f;
  const float gq = in && a.f.post_gain ? a.f.post_gain[c] : 1.f;
  float pre = 0.f, post = 0.f, gate = 0.f, sc = 0.f, sh = 0.f;   // sums over the samples
  for (int s = 0; s < a.samples; ++s) {
    float t[3] = {};
    if (in)
      for (int q = g; q < a.stripes; q += 32) {
        const float* p = a.part + (static_cast<int64_t>(s) * a.stripes + q) * 3 * H + c;
        t[0] += p[0], t[1] += p[H], t[2] += p[2 * H];
      }
    for (int k = 0; k < 3; ++k) red[k][g][cl] = t[k];
    __syncthreads();
    if (g < 3) {   // one warp per sum
      float v = 0.f;
      for (int k = 0; k < 32; ++k) v += red[g][k][cl];
      red[g][0][cl] = v;
    }
    __syncthreads();
    if (g == 0 && in) {
      const float A = red[0][0][cl], B = red[1][0][cl], C = red[2][0][cl];
      const float ms = a.f.mod_scale ? 1.f + a.f.mod_scale[static_cast<int64_t>(s) * a.f.mod_ld + c] : 1.f;
      const float gt = a.f.gate ? a.f.gate[static_cast<int64_t>(s) * a.f.gate_ld + c] : 1.f;
      pre += ms * A;
      post += gt * C;
      gate += gq * C;
      sc += gp * A;
      sh += B;
      if (a.d_scale && a.f.mod_ld) a.d_scale[static_cast<int64_t>(s) * H + c] = gp * A;
      if (a.d_shift && a.f.mod_ld) a.d_shift[static_cast<int64_t>(s) * H + c] = B;
      if (a.d_gate && a.f.gate_ld) a.d_gate[static_cast<int64_t>(s) * H + c] = gq * C;
    }
    __syncthreads();
  }
  if (g != 0 || !in) return;
  if (a.d_pre) a.d_pre[c] = pre;
  if (a.d_post) a.d_post[c] = post;
  if (a.d_scale && !a.f.mod_ld) a.d_scale[c] = sc;
  if (a.d_shift && !a.f.mod_ld) a.d_shift[c] = sh;
  if (a.d_gate && !a.f.gate_ld) a.d_gate[c] = gate;
}

}  // namespace dm0
