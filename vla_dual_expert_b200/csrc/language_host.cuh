// Host side of the language operators (dm0_embed, dm0_residual_norm, dm0_vocab_loss and their gradients):
// argument checks, workspace layouts, TMA maps and launches.  Included by dm0.cu after its dispatch
// helpers (launch, fail, ...), whose definitions it uses.  All scratch is the caller's workspace, so calls on
// different streams and captured graphs share nothing inside the context.
#pragma once

namespace {

constexpr int kLangMaxTokens = 1 << 24, kLangMaxVocab = 1 << 22, kLangMaxHidden = 1 << 16;
constexpr int kLangSms = 148;   // plans depend on sizes alone, so a workspace size holds for every context

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The context part of every entry's checks: its device must be the current one.
dm0_status lang_enter(dm0_ctx* c) {
  if (!c) return fail(c, DM0_EINVAL, "null context");
  int dev = -1;
  CK(cudaGetDevice(&dev));
  if (dev != c->device)
    return fail(c, DM0_EINVAL, "the context belongs to device " + std::to_string(c->device) + ", the current one is " +
                                   std::to_string(dev));
  c->pdl_ok = false;   // the first kernel follows foreign work
  return DM0_OK;
}

bool lang_tokens_ok(int B, int T) {
  return B >= 1 && T >= 1 && static_cast<int64_t>(B) * T <= kLangMaxTokens;
}

// ---------------------------------------------------------------- embedding
// (every call's size checks, which its workspace function shares)
dm0_status embed_sizes_ok(dm0_ctx* c, int B, int T, int vocab, int hidden) {
  if (!lang_tokens_ok(B, T) || vocab < 1 || vocab > kLangMaxVocab) return fail(c, DM0_ESHAPE, "bad batch, tokens or vocab");
  if (hidden < 8 || hidden % 8 != 0 || hidden > kLangMaxHidden)
    return fail(c, DM0_ESHAPE, "hidden must be a multiple of 8, at most 65536");
  return DM0_OK;
}

dm0_status rows_ok(dm0_ctx* c, const void* p, int f32, int T, int H, int64_t batch, int64_t row) {
  const int vec = f32 ? 4 : 8;
  if (row < H || batch < 0 || row % vec != 0 || batch % vec != 0 || !aligned16(p))
    return fail(c, DM0_EINVAL, "rows must be 16-byte aligned, their strides multiples of 16 bytes, row stride >= hidden");
  return DM0_OK;
}

struct EmbGradPlan {
  int log_g, rows, tiles, slices;
  size_t row_of, seg, total, long_row, part, bytes;
};
EmbGradPlan emb_grad_plan(int n, int vocab, int H) {
  EmbGradPlan p{};
  for (p.log_g = 7; (vocab + (1 << p.log_g) - 1) >> p.log_g > dm0::kSortMaxRows; ++p.log_g) {}
  p.rows = (vocab + (1 << p.log_g) - 1) >> p.log_g;
  p.tiles = (n + dm0::kEmbTile - 1) / dm0::kEmbTile;
  p.slices = (H + dm0::kEmbCols - 1) / dm0::kEmbCols;
  p.row_of = align256(sizeof(int) * static_cast<size_t>(n));
  p.seg = 2 * p.row_of;
  p.total = p.seg + align256(sizeof(int2) * static_cast<size_t>(vocab));
  p.long_row = p.total + 256;
  p.part = p.long_row + align256(sizeof(int) * static_cast<size_t>(p.tiles));
  p.bytes = p.part + align256(sizeof(float) * 2 * p.tiles * static_cast<size_t>(H));
  return p;
}

template <typename Td>
dm0_status embed_grad_run(dm0_ctx* c, cudaStream_t s, dm0::Ids ids, int n, const dm0::RowsView& v, int vocab, int H,
                          float scale, const Td* dout, float* grad, int accumulate, uint8_t* ws) {
  const EmbGradPlan p = emb_grad_plan(n, vocab, H);
  dm0::EmbScratch o{};
  o.perm = reinterpret_cast<int*>(ws);
  o.row_of = reinterpret_cast<int*>(ws + p.row_of);
  o.seg = reinterpret_cast<int2*>(ws + p.seg);
  o.total = reinterpret_cast<int*>(ws + p.total);
  o.long_row = reinterpret_cast<int*>(ws + p.long_row);
  o.part = reinterpret_cast<float*>(ws + p.part);
  if (n <= dm0::kEmbFew) {
    auto few = [&](auto kernel, auto typed) {
      return launch(c, s, kernel, dim3(1 << p.log_g), dim3(512), sizeof(int) * (p.rows + 1), typed, n, vocab, p.log_g, p.rows,
                    dout, v, H, scale, grad, accumulate, o.part, c->d_err);
    };
    return ids.wide ? few(dm0::embed_few_kernel<long long, Td>, static_cast<const long long*>(ids.p))
                    : few(dm0::embed_few_kernel<int, Td>, static_cast<const int*>(ids.p));
  }
  // rows that the sort's shadow has time to zero: about 3 us and 1.6 ns a token, at 5 TB/s
  const double shadow = (3e-6 + 1.6e-9 * n) * 5e12;
  const int early = accumulate ? 0 : static_cast<int>(std::min<double>(vocab, shadow / (4.0 * H)));
  const int64_t zero_bytes = 4ll * H * early;
  const int zero_rows = accumulate ? 0 : vocab - early;
  auto sort = [&](auto kernel, auto typed) {
    return launch(c, s, kernel,
                  dim3((1 << p.log_g) + static_cast<unsigned>((zero_bytes + dm0::kSortZero - 1) / dm0::kSortZero)),
                  dim3(dm0::kSortWarps * 32), sizeof(int) * dm0::kSortWarps * (p.rows + dm0::kSortList), typed, n, vocab, p.log_g, p.rows,
                  o, reinterpret_cast<uint8_t*>(grad + static_cast<int64_t>(zero_rows) * H), zero_bytes, c->d_err);
  };
  TRY(ids.wide ? sort(dm0::embed_sort_kernel<long long>, static_cast<const long long*>(ids.p))
               : sort(dm0::embed_sort_kernel<int>, static_cast<const int*>(ids.p)));
  const int zero_ctas = (zero_rows + dm0::kEmbZeroRows - 1) / dm0::kEmbZeroRows;
  TRY(launch(c, s, dm0::embed_sum_kernel<Td>, dim3(p.tiles * p.slices + zero_ctas), dim3(256), 0, o, dout, v, H, scale,
             grad, accumulate, p.tiles, p.slices, zero_rows));
  return launch(c, s, dm0::embed_join_kernel,
                dim3((p.tiles + dm0::kFixTiles - 1) / dm0::kFixTiles, (H + dm0::kFixCols - 1) / dm0::kFixCols),
                dim3(256), 0, o, p.tiles, H, scale, grad, accumulate);
}

// ---------------------------------------------------------------- residual norms
dm0_status norm_ok(dm0_ctx* c, const dm0_norm* a) {
  if (!a) return fail(c, DM0_EINVAL, "null argument");
  if (!lang_tokens_ok(a->batch, a->tokens)) return fail(c, DM0_ESHAPE, "bad batch or tokens");
  if (a->hidden < 8 || a->hidden % 8 != 0 || a->hidden > dm0::kRnMaxHidden)
    return fail(c, DM0_ESHAPE, "the norms take hidden sizes of 8..8192, multiples of 8");
  if (!std::isfinite(a->scale)) return fail(c, DM0_EINVAL, "the residual scale must be finite");
  for (int ld : {a->gate_stride, a->mod_stride})
    if (ld != 0 && (ld < a->hidden || ld % 4 != 0))
      return fail(c, DM0_EINVAL, "per-sample strides are 0 or at least hidden, multiples of 4");
  for (const float* p : {a->post_gain, a->pre_gain, a->gate, a->mod_scale, a->mod_shift})
    if (!aligned16(p)) return fail(c, DM0_EINVAL, "gain, gate and modulation vectors must be 16-byte aligned");
  return DM0_OK;
}
// rows_per_sample collapses to all rows where no vector is per sample
dm0::RnArgs norm_args(const dm0_ctx* c, const dm0_norm* a) {
  dm0::RnArgs r{};
  r.rows = a->batch * a->tokens;
  r.H = a->hidden;
  r.gate_ld = a->gate ? a->gate_stride : 0;
  r.mod_ld = a->mod_scale || a->mod_shift ? a->mod_stride : 0;
  r.rows_per_sample = r.gate_ld || r.mod_ld ? a->tokens : r.rows;
  r.alpha = a->scale;
  r.eps = c->cfg.rms_eps;
  r.post_gain = a->post_gain;
  r.pre_gain = a->pre_gain;
  r.gate = a->gate;
  r.mod_scale = a->mod_scale;
  r.mod_shift = a->mod_shift;
  return r;
}

template <typename Th, typename Ty>
dm0_status norm_run(dm0_ctx* c, cudaStream_t s, const dm0::RnArgs& a, const Th* h, const Ty* y, Th* h_out, bf16* n_out,
                    float* r_post, float* r_pre) {
  auto go = [&](auto kernel, int warps) {
    const int rows = warps > 4 ? 1 : 4 / warps;
    return launch(c, s, kernel, dim3((a.rows + rows - 1) / rows), dim3(32 * warps * rows), 0, h, y, a, h_out, n_out,
                  r_post, r_pre);
  };
  if (a.H <= 512) return go(dm0::residual_norm_kernel<Th, Ty, 1>, 1);
  if (a.H <= 1024) return go(dm0::residual_norm_kernel<Th, Ty, 2>, 2);
  if (a.H <= 2048) return go(dm0::residual_norm_kernel<Th, Ty, 4>, 4);
  if (a.H <= 4096) return go(dm0::residual_norm_kernel<Th, Ty, 8>, 8);
  return go(dm0::residual_norm_kernel<Th, Ty, 16>, 16);
}

int norm_grad_threads(int H) { return (H / 8 + 31) / 32 * 32; }
// Stripes per sample of the backward pass: the blocks that are resident at once (512 threads per SM), at
// least one row each; `per` rows a stripe.
int norm_stripes(int samples, int rows_per_sample, int H, int* per) {
  const int resident = kLangSms * std::max(1, std::min(8, 512 / norm_grad_threads(H)));
  const int want = std::min(rows_per_sample, std::max(1, resident / samples));
  *per = (rows_per_sample + want - 1) / want;
  return (rows_per_sample + *per - 1) / *per;
}
int norm_samples(const dm0_norm* a) {
  return (a->gate && a->gate_stride) || ((a->mod_scale || a->mod_shift) && a->mod_stride) ? a->batch : 1;
}
size_t norm_grad_bytes(const dm0_norm* a) {
  const int samples = norm_samples(a), T = samples == 1 ? a->batch * a->tokens : a->tokens;
  int per = 0;
  return align256(sizeof(float) * 3 * a->hidden * static_cast<size_t>(samples) * norm_stripes(samples, T, a->hidden, &per));
}

template <typename Tn, typename Th, typename Ty>
dm0_status norm_grad_run(dm0_ctx* c, cudaStream_t s, dm0::RnGradArgs a, int samples, const Tn* dn,
                         const Th* dh_out, const Th* h_out, const Ty* y, Th* dh, Ty* dy) {
  const int threads = norm_grad_threads(a.f.H);
  const size_t row = static_cast<size_t>(a.f.H) * (sizeof(Tn) + (dh_out ? 2 : 1) * sizeof(Th) + (y ? sizeof(Ty) : 0));
  // rows in the ring: four, or as many as leave room for the other resident blocks (at most 128 KB a row)
  const size_t room = threads <= 256 ? size_t(200) * 1024 / std::min(8, 512 / threads) : size_t(200) * 1024;
  a.stages = static_cast<int>(std::max<size_t>(1, std::min<size_t>(dm0::kRnMaxStages, room / row)));
  auto go = [&](auto kernel) {
    return launch(c, s, kernel, dim3(samples * a.stripes), dim3(threads), a.stages * row, dn, dh_out, h_out, y, a, dh, dy);
  };
  if (threads <= 256) return go(dm0::residual_norm_grad_kernel<Tn, Th, Ty, 256>);
  if (threads <= 512) return go(dm0::residual_norm_grad_kernel<Tn, Th, Ty, 512>);
  return go(dm0::residual_norm_grad_kernel<Tn, Th, Ty, 1024>);
}

template <typename Tn, typename Th, typename Ty>
bool norm_grad_setup() {
  auto attr = [&](auto kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  return attr(dm0::residual_norm_grad_kernel<Tn, Th, Ty, 256>, 128 * 1024) &&
         attr(dm0::residual_norm_grad_kernel<Tn, Th, Ty, 512>, 200 * 1024) &&
         attr(dm0::residual_norm_grad_kernel<Tn, Th, Ty, 1024>, 200 * 1024);
}

// ---------------------------------------------------------------- vocabulary loss
constexpr int kVgPieceElems = 1 << 27;   // entries of G held at a time: 256 MB of workspace

// bf16 [rows][cols] map of 64-column boxes of `box` rows, 128-byte swizzle (nothing is kept by address)
dm0_status vg_tmap(dm0_ctx* c, CUtensorMap* m, const void* p, uint64_t rows, uint64_t cols, uint32_t box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(c, DM0_ECUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * 2};
  cuuint32_t boxd[2] = {64, box}, estr[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, boxd, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DM0_OK : fail(c, DM0_ECUDA, "cuTensorMapEncodeTiled failed (" + std::to_string(r) + ")");
}

// G's map: [panels][tokens][64] bf16, boxes of one panel's `box` tokens
dm0_status vg_panel_tmap(dm0_ctx* c, CUtensorMap* m, const void* p, uint64_t tokens, uint64_t panels, uint32_t box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(c, DM0_ECUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {64, tokens, panels}, strides[2] = {128, 128 * tokens};
  cuuint32_t boxd[3] = {64, box, 1}, estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, boxd, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DM0_OK : fail(c, DM0_ECUDA, "cuTensorMapEncodeTiled failed (" + std::to_string(r) + ")");
}

// More than 128 tokens: pairs of CTAs on 256 x 256 tiles; up to 128: one CTA on 128 x 128, where a pair's
// second half of the rows would be padding.
bool vocab_pairs(int tokens) { return tokens > 128; }
// token rows of an A k-block's box
int vocab_a_rows(int tokens) { return std::min(128, (tokens + 7) / 8 * 8); }
int vocab_tile(int tokens) { return vocab_pairs(tokens) ? 256 : 128; }   // rows and columns

struct VocabLossPlan {
  int mt, nt, part_ld;
  size_t part, zt, bytes;
};
VocabLossPlan vocab_loss_plan(int tokens, int vocab) {
  VocabLossPlan p{};
  const int tile = vocab_tile(tokens);
  p.mt = (tokens + tile - 1) / tile;
  p.nt = (vocab + tile - 1) / tile;
  p.part_ld = (tokens + 31) / 32 * 32;
  p.part = 0;
  p.zt = align256(sizeof(float2) * 2 * p.nt * static_cast<size_t>(p.part_ld));
  p.bytes = p.zt + align256(sizeof(float) * static_cast<size_t>(tokens));
  return p;
}

struct VocabGradPlan {
  int piece, splits, kb_per_split;
  size_t scale, g, dh, bytes;
};
VocabGradPlan vocab_grad_plan(int tokens, int vocab, int H) {
  VocabGradPlan p{};
  const int vr = (vocab + 255) / 256 * 256;
  const int most = std::min(vr, std::max(256, kVgPieceElems / tokens / 256 * 256));
  const int pieces = (vr + most - 1) / most;
  p.piece = ((vr + pieces - 1) / pieces + 255) / 256 * 256;
  // splits of dh's contraction over the piece: the time of the busiest worker, whose tiles of dh and dW come in
  // turn (0.28 us a k-block, 1 us a tile: of a pair's 256 x 256; the 128 x 128 of up to 128 tokens, which HBM bounds, go
  // by the same), against the traffic of the fp32 sums
  const int tile = vocab_tile(tokens), workers = vocab_pairs(tokens) ? kLangSms / 2 : kLangSms;
  const int cols = std::min(p.piece, vocab);
  const int64_t ht = (H + tile - 1) / tile, th = (tokens + tile - 1) / tile * ht, tw = (cols + tile - 1) / tile * ht;
  const int KB = (cols + 63) / 64, KW = (tokens + 63) / 64;   // of the first piece, whose splits all write
  // (a split is one stretch of the accumulator: at most kVgBackStretch k-blocks)
  double best = 0;
  const int least = (KB + dm0::kVgBackStretch - 1) / dm0::kVgBackStretch;
  for (int S = least; S <= std::max(least, std::min(KB, 64)); ++S) {
    const int per = (KB + S - 1) / S, used = (KB + per - 1) / per;
    if (used != S) continue;
    double busiest = 0;
    // worker 0 has the most tiles of both; the first one with a tile of dh less may have one of dW more
    for (int64_t w : {int64_t(0), th * S % workers}) {
      const int64_t mine = (th * S + workers - 1 - w) / workers;
      const int64_t all = (th * S + tw + workers - 1 - w) / workers;
      busiest = std::max(busiest, mine * (per * 0.28 + 1.0) + (all - mine) * (KW * 0.28 + 1.0));
    }
    const double t = busiest + S * 8.0 * tokens * H / 6.0e6;
    if (!p.splits || t < best) best = t, p.splits = S, p.kb_per_split = per;
  }
  p.scale = 0;
  p.g = 256;
  p.dh = p.g + align256(sizeof(bf16) * static_cast<size_t>(tokens) * p.piece);
  p.bytes = p.dh + align256(sizeof(float) * p.splits * static_cast<size_t>(tokens) * H);
  return p;
}

dm0_status vocab_sizes_ok(dm0_ctx* c, int tokens, int vocab, int H) {
  if (tokens < 1 || tokens > kLangMaxTokens || vocab < 1 || vocab > kLangMaxVocab)
    return fail(c, DM0_ESHAPE, "tokens or vocab out of range");
  if (H < 64 || H % 64 != 0 || H > kLangMaxHidden) return fail(c, DM0_ESHAPE, "hidden must be a multiple of 64");
  return DM0_OK;
}
dm0_status vocab_ok(dm0_ctx* c, const void* h, const void* w, const void* t, int tokens, int vocab, int H) {
  if (!h || !w || !t) return fail(c, DM0_EINVAL, "null argument");
  TRY(vocab_sizes_ok(c, tokens, vocab, H));
  if (!aligned16(h) || !aligned16(w)) return fail(c, DM0_EINVAL, "hidden states and weights must be 16-byte aligned");
  return DM0_OK;
}

// grid of a product's `tiles`: one CTA per SM, or one pair per two
dm0_status vocab_grid(dm0_ctx* c, bool pairs, int64_t tiles, dim3* grid) {
  if (tiles > 0x3fffffff) return fail(c, DM0_ESHAPE, "too many tiles");
  *grid = pairs ? dim3(2 * static_cast<unsigned>(std::min<int64_t>(tiles, c->num_sms / 2)))
                : dim3(static_cast<unsigned>(std::min<int64_t>(tiles, c->num_sms)));
  return DM0_OK;
}
bool vocab_long(bool pairs, int H) {
  return H > 64 * (pairs ? dm0::VgTile<true>::kStretch : dm0::VgTile<false>::kStretch);
}
int64_t vocab_tiles(const dm0::VgArgs& a) { return static_cast<int64_t>(a.mt) * a.nt * a.splits; }

// LONG: the contraction takes more than one stretch of the accumulator
template <int MODE, bool LONG>
dm0_status vocab_gemm(dm0_ctx* c, cudaStream_t s, bool pairs, const dm0::VgMaps& m, const dm0::VgArgs& a) {
  dim3 grid;
  TRY(vocab_grid(c, pairs, vocab_tiles(a), &grid));
  if (pairs) return launch(c, s, dm0::vocab_gemm_pair_kernel<MODE, LONG>, grid, dim3(320), dm0::VgTile<true>::kBytes, m, a);
  return launch(c, s, dm0::vocab_gemm_kernel<MODE, LONG>, grid, dim3(320), dm0::VgTile<false>::kBytes, m, a);
}

dm0_status vocab_loss_run(dm0_ctx* c, cudaStream_t s, const bf16* h, const bf16* w, dm0::Ids tgt, int tokens, int vocab,
                          int H, float* loss, float* lse, uint8_t* ws) {
  const VocabLossPlan p = vocab_loss_plan(tokens, vocab);
  dm0::VgMaps m{};
  const bool pairs = vocab_pairs(tokens);
  TRY(vg_tmap(c, &m.a, h, tokens, H, vocab_a_rows(tokens)));
  TRY(vg_tmap(c, &m.b, w, vocab, H, 128));
  dm0::VgArgs a{};
  a.M = tokens;
  a.N = vocab;
  a.K = H;
  a.mt = p.mt;
  a.nt = p.nt;
  a.splits = 1;
  a.kb_per_split = H / 64;
  a.a_bytes = 128u * vocab_a_rows(tokens);
  a.b_bytes = 128u * 128u;
  a.ksteps = 4;
  a.err = c->d_err;
  a.targets = tgt;
  a.vocab = vocab;
  a.valid_n = vocab;
  a.part = reinterpret_cast<float2*>(ws + p.part);
  a.part_ld = p.part_ld;
  a.zt = reinterpret_cast<float*>(ws + p.zt);
  TRY((vocab_gemm<dm0::kVgStats, true>(c, s, pairs, m, a)));
  const int parts = 2 * (p.mt > 1 ? p.nt : std::min(p.nt, pairs ? c->num_sms / 2 : c->num_sms));
  return launch(c, s, dm0::vocab_loss_kernel, dim3((tokens + 3) / 4), dim3(512), 0,
                static_cast<const float2*>(a.part), parts, p.part_ld, static_cast<const float*>(a.zt), tgt, tokens,
                vocab, loss, lse, c->d_err);
}

dm0_status vocab_grad_run(dm0_ctx* c, cudaStream_t s, const bf16* h, const bf16* w, dm0::Ids tgt, const float* lse,
                          const float* dloss, int tokens, int vocab, int H, void* dh, int dh_f32, void* dw, int dw_f32,
                          int accumulate, uint8_t* ws) {
  const VocabGradPlan p = vocab_grad_plan(tokens, vocab, H);
  float* scale = reinterpret_cast<float*>(ws + p.scale);
  bf16* g = reinterpret_cast<bf16*>(ws + p.g);
  float* part = reinterpret_cast<float*>(ws + p.dh);
  const bool pairs = vocab_pairs(tokens);
  const int tile = vocab_tile(tokens);
  dm0::VgMaps mg{}, mh{}, mw{};   // of G, dh and dW
  TRY(vg_tmap(c, &mg.a, h, tokens, H, vocab_a_rows(tokens)));
  TRY(vg_tmap(c, &mg.b, w, vocab, H, 128));
  TRY(vg_panel_tmap(c, &mg.out, g, tokens, p.piece / 64, 32));
  if (dw && !dw_f32) TRY(vg_tmap(c, &mw.out, dw, vocab, H, 32));
  TRY(vg_panel_tmap(c, &mh.a, g, tokens, p.piece / 64, vocab_a_rows(tokens)));
  TRY(vg_tmap(c, &mh.b, w, vocab, H, 64));
  const int kbox = std::min(64, (tokens + 15) / 16 * 16);   // tokens of a k-block of dW
  TRY(vg_panel_tmap(c, &mw.a, g, tokens, p.piece / 64, kbox));
  TRY(vg_tmap(c, &mw.b, h, tokens, H, kbox));
  const int mt = (tokens + tile - 1) / tile, ht = (H + tile - 1) / tile;
  for (int v0 = 0; v0 < vocab; v0 += p.piece) {
    const int cols = std::min(p.piece, vocab - v0);
    dm0::VgArgs a{};   // G of the piece
    a.err = c->d_err;
    a.a_bytes = 128u * vocab_a_rows(tokens);
    a.b_bytes = 128u * 128u;
    a.ksteps = 4;
    a.scale = scale;
    a.vocab = vocab;
    a.v0 = v0;
    a.M = tokens;
    a.N = cols;
    a.K = H;
    a.mt = mt;
    a.nt = (cols + tile - 1) / tile;
    a.splits = 1;
    a.kb_per_split = H / 64;
    a.b_y0 = v0;
    a.targets = tgt;
    a.valid_n = cols;
    a.lse = lse;
    a.dloss = dloss;
    TRY((vocab_long(pairs, H) ? vocab_gemm<dm0::kVgGrad, true>(c, s, pairs, mg, a)
                              : vocab_gemm<dm0::kVgGrad, false>(c, s, pairs, mg, a)));
    dm0::VgArgs ah = a, aw = a;
    ah.N = H;
    ah.K = cols;
    ah.nt = dh ? ht : 0;
    ah.kb_per_split = p.kb_per_split;
    ah.splits = ((cols + 63) / 64 + p.kb_per_split - 1) / p.kb_per_split;
    ah.band = 1;
    ah.dh = part;
    ah.add = v0 > 0;
    aw.M = cols;
    aw.N = H;
    aw.K = tokens;
    aw.a_bytes = aw.b_bytes = 2u * 128u * kbox;   // two boxes of 64 columns
    aw.ksteps = kbox / 16;
    aw.mt = (cols + tile - 1) / tile;
    aw.nt = dw ? ht : 0;
    aw.kb_per_split = (tokens + 63) / 64;
    aw.band = 1;
    aw.b_y0 = 0;
    aw.add = accumulate;
    aw.dw = dw_f32 ? static_cast<float*>(dw) : nullptr;
    dim3 grid;
    TRY(vocab_grid(c, pairs, vocab_tiles(ah) + vocab_tiles(aw), &grid));
    const bool many = tokens > 64 * dm0::kVgBackStretch;   // so dW takes several stretches
    if (pairs)
      TRY(launch(c, s, many ? dm0::vocab_back_pair_kernel<true> : dm0::vocab_back_pair_kernel<false>, grid, dim3(320),
                 dm0::VgTile<true>::kBytes, mh, ah, mw, aw));
    else
      TRY(launch(c, s, dm0::vocab_back_kernel, grid, dim3(320), dm0::VgTile<false>::kBytes, mh, ah, mw, aw));
  }
  if (!dh) return DM0_OK;
  const int64_t n = static_cast<int64_t>(tokens) * H;
  const dim3 grid(static_cast<unsigned>((n / 4 + 255) / 256));
  // the splits of the first piece; the last piece may have used fewer
  const int splits = p.splits;
  if (dh_f32)
    return launch(c, s, dm0::vocab_hidden_kernel<float>, grid, dim3(256), 0, static_cast<const float*>(part), splits, n,
                  static_cast<const float*>(scale), static_cast<float*>(dh));
  return launch(c, s, dm0::vocab_hidden_kernel<bf16>, grid, dim3(256), 0, static_cast<const float*>(part), splits, n,
                static_cast<const float*>(scale), static_cast<bf16*>(dh));
}

// shared-memory limits of these kernels (dm0_create)
bool lang_setup() {
  auto attr = [](auto kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  typedef float f;
  return norm_grad_setup<f, f, f>() && norm_grad_setup<f, f, bf16>() && norm_grad_setup<f, bf16, f>() &&
         norm_grad_setup<f, bf16, bf16>() && norm_grad_setup<bf16, f, f>() && norm_grad_setup<bf16, f, bf16>() &&
         norm_grad_setup<bf16, bf16, f>() && norm_grad_setup<bf16, bf16, bf16>() &&
         attr(dm0::embed_sort_kernel<int>, 4 * dm0::kSortWarps * (dm0::kSortMaxRows + dm0::kSortList)) &&
         attr(dm0::embed_sort_kernel<long long>, 4 * dm0::kSortWarps * (dm0::kSortMaxRows + dm0::kSortList)) &&
         attr(dm0::vocab_gemm_kernel<dm0::kVgStats, true>, dm0::VgTile<false>::kBytes) &&
         attr(dm0::vocab_gemm_kernel<dm0::kVgGrad, false>, dm0::VgTile<false>::kBytes) &&
         attr(dm0::vocab_gemm_kernel<dm0::kVgGrad, true>, dm0::VgTile<false>::kBytes) &&
         attr(dm0::vocab_back_kernel, dm0::VgTile<false>::kBytes) &&
         attr(dm0::vocab_gemm_pair_kernel<dm0::kVgStats, true>, dm0::VgTile<true>::kBytes) &&
         attr(dm0::vocab_gemm_pair_kernel<dm0::kVgGrad, false>, dm0::VgTile<true>::kBytes) &&
         attr(dm0::vocab_gemm_pair_kernel<dm0::kVgGrad, true>, dm0::VgTile<true>::kBytes) &&
         attr(dm0::vocab_back_pair_kernel<false>, dm0::VgTile<true>::kBytes) &&
         attr(dm0::vocab_back_pair_kernel<true>, dm0::VgTile<true>::kBytes);
}
}  // namespace

// Runs a callable with a typed null pointer for each of (fp32, bf16)
#define DM0_BY_TYPE(f32, T, ...)                \
  [&]() -> dm0_status {                         \
    if (f32) {                                  \
      using T = float;                          \
      return [&]() -> dm0_status __VA_ARGS__(); \
    }                                           \
    using T = bf16;                             \
    return [&]() -> dm0_status __VA_ARGS__();   \
  }()

extern "C" {

dm0_status dm0_embed(dm0_ctx* c, const void* table, const void* ids, int ids_i64, int B, int T, int vocab, int hidden,
                     float scale, void* out, int out_f32, int64_t batch_stride, int64_t row_stride, void* stream) {
  if (!table || !ids || !out) return fail(c, DM0_EINVAL, "null argument");
  TRY(embed_sizes_ok(c, B, T, vocab, hidden));
  if (!aligned16(table)) return fail(c, DM0_EINVAL, "the table must be 16-byte aligned");
  TRY(rows_ok(c, out, out_f32, T, hidden, batch_stride, row_stride));
  if (B > 1 && batch_stride < (T - 1) * row_stride + hidden && (batch_stride < hidden || row_stride < (B - 1) * batch_stride + hidden))
    return fail(c, DM0_EINVAL, "the rows of out overlap");
  TRY(lang_enter(c));
  const int n = B * T;
  const dm0::Ids id{ids, ids_i64};
  const dm0::RowsView v{batch_stride, row_stride, T};
  return DM0_BY_TYPE(out_f32, To, {
    return launch(c, static_cast<cudaStream_t>(stream), dm0::embed_kernel<To>, dim3((n + 7) / 8), dim3(256), 0,
                  static_cast<const bf16*>(table), id, n, vocab, hidden, scale, static_cast<To*>(out), v, c->d_err);
  });
}

size_t dm0_embed_grad_workspace(int B, int T, int vocab, int hidden) {
  if (embed_sizes_ok(nullptr, B, T, vocab, hidden) != DM0_OK) return 0;
  return emb_grad_plan(B * T, vocab, hidden).bytes;
}

dm0_status dm0_embed_grad(dm0_ctx* c, const void* ids, int ids_i64, int B, int T, int vocab, int hidden, float scale,
                          const void* dout, int dout_f32, int64_t batch_stride, int64_t row_stride, float* grad,
                          int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (!ids || !dout || !grad || !workspace) return fail(c, DM0_EINVAL, "null argument");
  TRY(embed_sizes_ok(c, B, T, vocab, hidden));
  if (!aligned16(grad) || !aligned16(workspace)) return fail(c, DM0_EINVAL, "grad and workspace must be 16-byte aligned");
  TRY(rows_ok(c, dout, dout_f32, T, hidden, batch_stride, row_stride));
  if (workspace_bytes < emb_grad_plan(B * T, vocab, hidden).bytes) return fail(c, DM0_EINVAL, "workspace too small");
  TRY(lang_enter(c));
  const dm0::Ids id{ids, ids_i64};
  const dm0::RowsView v{batch_stride, row_stride, T};
  return DM0_BY_TYPE(dout_f32, Td, {
    return embed_grad_run(c, static_cast<cudaStream_t>(stream), id, B * T, v, vocab, hidden, scale,
                          static_cast<const Td*>(dout), grad, accumulate, static_cast<uint8_t*>(workspace));
  });
}

dm0_status dm0_residual_norm(dm0_ctx* c, const dm0_norm* a, const void* h, const void* y, void* h_out, void* n_out,
                             float* r_post, float* r_pre, void* stream) {
  TRY(norm_ok(c, a));
  if (!h || !h_out || !n_out || !r_pre || (y && a->post_gain && !r_post)) return fail(c, DM0_EINVAL, "null argument");
  if (!y && (a->post_gain || a->gate)) return fail(c, DM0_EINVAL, "a post gain or gate needs a block output");
  for (const void* p : {h, y, static_cast<const void*>(h_out), static_cast<const void*>(n_out)})
    if (!aligned16(p)) return fail(c, DM0_EINVAL, "row tensors must be 16-byte aligned");
  TRY(lang_enter(c));
  const dm0::RnArgs r = norm_args(c, a);
  return DM0_BY_TYPE(a->h_f32, Th, {
    return DM0_BY_TYPE(a->y_f32, Ty, {
      return norm_run(c, static_cast<cudaStream_t>(stream), r, static_cast<const Th*>(h), static_cast<const Ty*>(y),
                      static_cast<Th*>(h_out), static_cast<bf16*>(n_out), r_post, r_pre);
    });
  });
}

size_t dm0_residual_norm_grad_workspace(const dm0_norm* a) {
  return norm_ok(nullptr, a) == DM0_OK ? norm_grad_bytes(a) : 0;
}

dm0_status dm0_residual_norm_grad(dm0_ctx* c, const dm0_norm* a, const void* dn, int dn_f32, const void* dh_out,
                                  const void* h_out, const void* y, const float* r_post, const float* r_pre, void* dh,
                                  void* dy, const dm0_norm_grads* g, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  TRY(norm_ok(c, a));
  if (!dn || !h_out || !r_pre || !dh || !g || !workspace || (y && (!dy || (a->post_gain && !r_post))))
    return fail(c, DM0_EINVAL, "null argument");
  if (!y && (a->post_gain || a->gate)) return fail(c, DM0_EINVAL, "a post gain or gate needs a block output");
  if ((g->post_gain && !a->post_gain) || (g->pre_gain && !a->pre_gain) || (g->gate && !a->gate) ||
      (g->mod_scale && !a->mod_scale) || (g->mod_shift && !a->mod_shift))
    return fail(c, DM0_EINVAL, "a gradient was asked for a vector that is not there");
  for (const void* p : {dn, dh_out, h_out, y, static_cast<const void*>(dh), static_cast<const void*>(dy),
                        static_cast<const void*>(workspace)})
    if (!aligned16(p)) return fail(c, DM0_EINVAL, "row tensors and workspace must be 16-byte aligned");
  if (workspace_bytes < norm_grad_bytes(a)) return fail(c, DM0_EINVAL, "workspace too small");
  TRY(lang_enter(c));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int samples = norm_samples(a);
  const bool sums = g->post_gain || g->pre_gain || g->gate || g->mod_scale || g->mod_shift;
  dm0::RnGradArgs r{};
  r.f = norm_args(c, a);
  r.r_post = r_post;
  r.r_pre = r_pre;
  r.stripes = norm_stripes(samples, r.f.rows_per_sample, a->hidden, &r.per);
  r.err = c->d_err;
  r.part = sums ? static_cast<float*>(workspace) : nullptr;
  TRY(DM0_BY_TYPE(dn_f32, Tn, {
    return DM0_BY_TYPE(a->h_f32, Th, {
      return DM0_BY_TYPE(a->y_f32, Ty, {
        return norm_grad_run(c, s, r, samples, static_cast<const Tn*>(dn), static_cast<const Th*>(dh_out),
                             static_cast<const Th*>(h_out), static_cast<const Ty*>(y), static_cast<Th*>(dh),
                             static_cast<Ty*>(dy));
      });
    });
  }));
  if (!sums) return DM0_OK;
  dm0::RnSumArgs t{};
  t.f = r.f;
  t.samples = samples;
  t.stripes = r.stripes;
  t.part = r.part;
  t.d_post = g->post_gain;
  t.d_gate = g->gate;
  t.d_pre = g->pre_gain;
  t.d_scale = g->mod_scale;
  t.d_shift = g->mod_shift;
  return launch(c, s, dm0::residual_norm_sum_kernel, dim3((a->hidden + 31) / 32), dim3(1024), 0, t);
}

size_t dm0_vocab_loss_workspace(int tokens, int vocab, int hidden) {
  if (vocab_sizes_ok(nullptr, tokens, vocab, hidden) != DM0_OK) return 0;
  return vocab_loss_plan(tokens, vocab).bytes;
}

dm0_status dm0_vocab_loss(dm0_ctx* c, const void* hidden_states, const void* weight, const void* targets,
                          int targets_i64, int tokens, int vocab, int hidden, float* loss, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  TRY(vocab_ok(c, hidden_states, weight, targets, tokens, vocab, hidden));
  if (!loss || !lse || !workspace) return fail(c, DM0_EINVAL, "null argument");
  if (!aligned16(workspace)) return fail(c, DM0_EINVAL, "the workspace must be 16-byte aligned");
  if (workspace_bytes < vocab_loss_plan(tokens, vocab).bytes) return fail(c, DM0_EINVAL, "workspace too small");
  TRY(lang_enter(c));
  return vocab_loss_run(c, static_cast<cudaStream_t>(stream), static_cast<const bf16*>(hidden_states),
                        static_cast<const bf16*>(weight), dm0::Ids{targets, targets_i64}, tokens, vocab, hidden, loss,
                        lse, static_cast<uint8_t*>(workspace));
}

size_t dm0_vocab_loss_grad_workspace(int tokens, int vocab, int hidden) {
  if (vocab_sizes_ok(nullptr, tokens, vocab, hidden) != DM0_OK) return 0;
  return vocab_grad_plan(tokens, vocab, hidden).bytes;
}

dm0_status dm0_vocab_loss_grad(dm0_ctx* c, const void* hidden_states, const void* weight, const void* targets,
                               int targets_i64, const float* lse, const float* dloss, int tokens, int vocab, int hidden,
                               void* dhidden, int dhidden_f32, void* dweight, int dweight_f32, int accumulate,
                               void* workspace, size_t workspace_bytes, void* stream) {
  TRY(vocab_ok(c, hidden_states, weight, targets, tokens, vocab, hidden));
  if (!lse || !dloss || !workspace || (!dhidden && !dweight)) return fail(c, DM0_EINVAL, "null argument");
  if (!aligned16(dhidden) || !aligned16(dweight) || !aligned16(workspace))
    return fail(c, DM0_EINVAL, "gradients and workspace must be 16-byte aligned");
  if (accumulate && dweight && !dweight_f32)
    return fail(c, DM0_EINVAL, "only an fp32 weight gradient accumulates: a bf16 sum would be rounded at every call");
  if (workspace_bytes < vocab_grad_plan(tokens, vocab, hidden).bytes) return fail(c, DM0_EINVAL, "workspace too small");
  TRY(lang_enter(c));
  return vocab_grad_run(c, static_cast<cudaStream_t>(stream), static_cast<const bf16*>(hidden_states),
                        static_cast<const bf16*>(weight), dm0::Ids{targets, targets_i64}, lse, dloss, tokens, vocab,
                        hidden, dhidden, dhidden_f32, dweight, dweight_f32, accumulate,
                        static_cast<uint8_t*>(workspace));
}

}  // extern "C"
#undef DM0_BY_TYPE
