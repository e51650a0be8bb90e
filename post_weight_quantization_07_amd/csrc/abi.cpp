// C ABI of the GPTQ layer solve: argument checks, workspace sizing and the
// launch sequence of each call.  Declarations and contracts: include/gptq.h.
#include "../../include/gptq.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gptq_internal.h"

namespace {

constexpr int kBlock = 128;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

int device_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 256;
  return cus;
}

gptq_status from_hip(hipError_t e) { return e == hipSuccess ? GPTQ_OK : GPTQ_ERR_HIP; }

bool bits_ok(int32_t b) { return b == 2 || b == 3 || b == 4 || b == 8; }

// size limits of every call: channels and output rows up to 2^20 (an H of
// that size would take 4 TiB), tokens up to 2^40; beyond them no size
// computation of the library can overflow
constexpr int64_t kMaxDim = int64_t{1} << 20;
constexpr int64_t kMaxTokens = int64_t{1} << 40;
bool dim_ok(int64_t v) { return v > 0 && v <= kMaxDim; }
bool tokens_ok(int64_t n) { return n >= 0 && n <= kMaxTokens; }

// d_in % (32 / bits) == 0, and d_in % 32 == 0 for 3 bits: whole words per row
bool packable(int64_t d_in, int32_t bits) {
  if (!bits_ok(bits) || d_in <= 0) return false;
  const int64_t m = (bits == 3) ? 32 : 32 / bits;
  return d_in % m == 0;
}

// the serving calls: rows (tokens) of one call, and a product of sizes that
// stays below 2^31
constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int64_t kMaxIntDim = int64_t{1} << 16;  // 32-bit sums of int8 products stay exact
bool rows_ok(int64_t n) { return n >= 0 && n <= kMaxRows; }

bool cache_shape(const gptq_cache* c, gptq::CacheShape* out) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return false;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scales) || !aligned16(c->v_scales))
    return false;
  if (c->bits != 4 && c->bits != 8) return false;
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0) return false;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0) return false;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 65536 || c->n_pages < 1 || c->n_pages > (int64_t{1} << 31) - 1) return false;
  *out = gptq::CacheShape{c->n_pages, c->page_size, c->n_kv_heads, c->head_dim, c->bits};
  return true;
}

// A launch has fewer than 2^32 threads along x; the cache kernels give each row of
// head_dim values, rounded up to a power of two P, P / 8 lanes for every four rows.
bool cache_rows_ok(const gptq::CacheShape& c, int64_t n_tokens) {
  int64_t p = 16;
  while (p < c.hd) p *= 2;
  return n_tokens * c.n_kv * p <= (int64_t{1} << 37) - (int64_t{1} << 13);  // n_tokens <= 2^30, n_kv <= 2^16: no overflow
}

}  // namespace

extern "C" {

const char* gptq_status_string(int32_t s) {
  switch (s) {
    case GPTQ_OK: return "ok";
    case GPTQ_ERR_INVALID_ARG: return "invalid argument";
    case GPTQ_ERR_NOT_SPD: return "damped Hessian is not positive definite";
    case GPTQ_ERR_HIP: return "HIP runtime error";
    case GPTQ_ERR_WORKSPACE: return "workspace missing, too small or misaligned";
    case GPTQ_ERR_TOO_LARGE: return "the call needs more scratch memory than the library's fixed buffer holds";
  }
  return "unknown status";
}

gptq_status gptq_config_validate(const gptq_config* c) {
  if (!c) return GPTQ_ERR_INVALID_ARG;
  if (!bits_ok(c->bits)) return GPTQ_ERR_INVALID_ARG;
  if (!(c->group_size == -1 || c->group_size > 0)) return GPTQ_ERR_INVALID_ARG;
  if (!(c->damp_percent > 0.0f && c->damp_percent < 1.0f)) return GPTQ_ERR_INVALID_ARG;
  if (c->block_size != kBlock) return GPTQ_ERR_INVALID_ARG;
  if (c->group_size > 0 && !(kBlock % c->group_size == 0 || c->group_size % kBlock == 0))
    return GPTQ_ERR_INVALID_ARG;
  return GPTQ_OK;
}

size_t gptq_hessian_workspace_size(int64_t d_in, int64_t n_tokens, int32_t xt) {
  if (!dim_ok(d_in) || !tokens_ok(n_tokens) || (xt != GPTQ_F32 && xt != GPTQ_BF16)) return 0;
  return gptq::hessian_plan(d_in, n_tokens, xt == GPTQ_BF16, device_cus()).ws_bytes;
}

gptq_status gptq_hessian_accumulate(float* S, int64_t d_in, const void* X, int32_t xt, int64_t n_tokens,
                                    int64_t ldx, void* ws, size_t ws_bytes, void* stream) {
  if (!S || !dim_ok(d_in) || !tokens_ok(n_tokens) || (xt != GPTQ_F32 && xt != GPTQ_BF16)) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return GPTQ_OK;
  const bool bf16 = (xt == GPTQ_BF16);
  const int64_t vec = bf16 ? 8 : 4;
  if (!X || d_in % vec != 0 || ldx < d_in || ldx % vec != 0 || !aligned16(X) || !aligned16(S))
    return GPTQ_ERR_INVALID_ARG;
  if (ldx > (int64_t{1} << 24)) return GPTQ_ERR_INVALID_ARG;  // 32-bit in-stage offsets
  const gptq::HessPlan plan = gptq::hessian_plan(d_in, n_tokens, bf16, device_cus());
  if (!ws || ws_bytes < plan.ws_bytes || !aligned256(ws)) return GPTQ_ERR_WORKSPACE;
  return from_hip(gptq::hessian_launch(plan, S, d_in, X, bf16, n_tokens, ldx, ws,
                                       static_cast<hipStream_t>(stream)));
}

size_t gptq_prepare_workspace_size(int64_t d_in) {
  if (!dim_ok(d_in)) return 0;
  return gptq::prepare_layout(d_in).ws_bytes;
}

gptq_status gptq_prepare_hinv(float* S_to_H, int64_t d_in, int64_t n_total, const gptq_config* cfg, float* U,
                              int32_t* perm, int32_t* info_dev, void* ws, size_t ws_bytes, void* stream) {
  if (!S_to_H || !U || !perm || !info_dev || !dim_ok(d_in) || n_total <= 0) return GPTQ_ERR_INVALID_ARG;
  if (gptq_config_validate(cfg) != GPTQ_OK) return GPTQ_ERR_INVALID_ARG;
  if (d_in % 4 != 0 || !aligned16(S_to_H) || !aligned16(U)) return GPTQ_ERR_INVALID_ARG;
  const gptq::PrepLayout lay = gptq::prepare_layout(d_in);
  if (!ws || ws_bytes < lay.ws_bytes || !aligned256(ws)) return GPTQ_ERR_WORKSPACE;
  return from_hip(gptq::prepare_launch(S_to_H, d_in, n_total, cfg->damp_percent, cfg->desc_act != 0, U, perm,
                                       info_dev, ws, static_cast<hipStream_t>(stream)));
}

size_t gptq_workspace_size(int64_t d_out, int64_t d_in, const gptq_config* cfg) {
  if (!dim_ok(d_out) || !dim_ok(d_in) || gptq_config_validate(cfg) != GPTQ_OK) return 0;
  return gptq::quant_layout(d_out, d_in, gptq::quant_planes(cfg->group_size, cfg->static_groups != 0)).ws_bytes;
}

gptq_status gptq_quantize_layer(const void* W, int32_t wt, int64_t d_out, int64_t d_in, const float* U,
                                const int32_t* perm, const gptq_config* cfg, uint8_t* codes, float* scales,
                                int32_t* zeros, int32_t* g_idx, float* Q_or_null, float* row_loss_or_null,
                                void* ws, size_t ws_bytes, void* stream) {
  if (gptq_config_validate(cfg) != GPTQ_OK) return GPTQ_ERR_INVALID_ARG;
  if (!W || !U || !codes || !scales || !zeros || !g_idx || !dim_ok(d_out) || !dim_ok(d_in)) return GPTQ_ERR_INVALID_ARG;
  if (wt != GPTQ_F32 && wt != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (cfg->desc_act && !perm) return GPTQ_ERR_INVALID_ARG;
  if (!packable(d_in, cfg->bits)) return GPTQ_ERR_INVALID_ARG;
  if (!aligned16(U) || !aligned16(codes) || (Q_or_null && !aligned16(Q_or_null))) return GPTQ_ERR_INVALID_ARG;
  const gptq::QuantLayout lay =
      gptq::quant_layout(d_out, d_in, gptq::quant_planes(cfg->group_size, cfg->static_groups != 0));
  if (!ws || ws_bytes < lay.ws_bytes || !aligned256(ws)) return GPTQ_ERR_WORKSPACE;
  return from_hip(gptq::quantize_launch(W, wt == GPTQ_BF16, d_out, d_in, U, perm, cfg->bits, cfg->group_size,
                                        cfg->sym != 0, cfg->static_groups != 0, codes, scales, zeros, g_idx,
                                        Q_or_null, row_loss_or_null, ws, static_cast<hipStream_t>(stream),
                                        cfg->desc_act == 0));
}

gptq_status gptq_pack(const uint8_t* codes, int64_t d_out, int64_t d_in, int32_t bits, int32_t* qweight,
                      void* stream) {
  if (!codes || !qweight || !dim_ok(d_out) || !dim_ok(d_in)) return GPTQ_ERR_INVALID_ARG;
  if (!packable(d_in, bits)) return GPTQ_ERR_INVALID_ARG;
  return from_hip(gptq::pack_launch(codes, d_out, d_in, bits, qweight, static_cast<hipStream_t>(stream)));
}

size_t gptq_dequant_workspace_size(int64_t m, int64_t d_in, int64_t d_out) {
  if (m <= 0 || !tokens_ok(m) || !dim_ok(d_in) || !dim_ok(d_out) || d_in % 32 != 0) return 0;
  return gptq::dequant_workspace_bytes(m, d_in, d_out);
}

gptq_status gptq_dequant_matmul(const void* x, int32_t xt, int64_t m, int64_t d_in, const int32_t* qweight,
                                const float* scales, const int32_t* zeros, const int32_t* g_idx, int32_t bits,
                                int64_t d_out, int32_t n_groups, float* y, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!x || !qweight || !scales || !zeros || !g_idx || !y) return GPTQ_ERR_INVALID_ARG;
  if (m <= 0 || !tokens_ok(m) || !dim_ok(d_out) || !dim_ok(d_in) || d_in % 32 != 0 || n_groups <= 0)
    return GPTQ_ERR_INVALID_ARG;
  if (!bits_ok(bits) || (xt != GPTQ_F32 && xt != GPTQ_BF16)) return GPTQ_ERR_INVALID_ARG;
  // qweight and scales / zeros are addressed with 32-bit byte offsets
  if (d_in / 32 * bits * d_out * 4 >= (int64_t{1} << 31) || int64_t{n_groups} * d_out * 4 >= (int64_t{1} << 31))
    return GPTQ_ERR_INVALID_ARG;
  const size_t need = gptq::dequant_workspace_bytes(m, d_in, d_out);
  if (need > 0 && (!ws || ws_bytes < need || !aligned256(ws))) return GPTQ_ERR_WORKSPACE;
  return from_hip(gptq::dequant_matmul_launch(x, xt == GPTQ_BF16, m, d_in, qweight, scales, zeros, g_idx, bits, d_out,
                                              n_groups, y, ws, static_cast<hipStream_t>(stream)));
}

size_t gptq_dequant_scratch_bytes(void) { return gptq::kDequantScratchBytes; }

size_t gptq_dequant_noalloc_need(int64_t m, int32_t xt, int64_t d_in, int32_t bits, int64_t d_out) {
  if (m <= 0 || !tokens_ok(m) || !dim_ok(d_in) || !dim_ok(d_out) || d_in % 32 != 0 || !bits_ok(bits)) return 0;
  if (xt != GPTQ_F32 && xt != GPTQ_BF16) return 0;
  return gptq::dequant_partial_bytes(m, d_in, d_out, xt == GPTQ_BF16, bits);
}

gptq_status gptq_dequant_matmul_noalloc(const void* x, int32_t xt, int64_t m, int64_t d_in,
                                        const int32_t* qweight, const float* scales, const int32_t* zeros,
                                        const int32_t* g_idx, int32_t bits, int64_t d_out, int32_t n_groups,
                                        float* y, void* stream) {
  if (!x || !qweight || !scales || !zeros || !g_idx || !y) return GPTQ_ERR_INVALID_ARG;
  if (m <= 0 || !tokens_ok(m) || !dim_ok(d_out) || !dim_ok(d_in) || d_in % 32 != 0 || n_groups <= 0)
    return GPTQ_ERR_INVALID_ARG;
  if (!bits_ok(bits) || (xt != GPTQ_F32 && xt != GPTQ_BF16)) return GPTQ_ERR_INVALID_ARG;
  if (d_in / 32 * bits * d_out * 4 >= (int64_t{1} << 31) || int64_t{n_groups} * d_out * 4 >= (int64_t{1} << 31))
    return GPTQ_ERR_INVALID_ARG;
  if (gptq::dequant_partial_bytes(m, d_in, d_out, xt == GPTQ_BF16, bits) > gptq::kDequantScratchBytes)
    return GPTQ_ERR_TOO_LARGE;
  void* ws = nullptr;
  const gptq_status st = from_hip(gptq::dequant_scratch(&ws));
  if (st != GPTQ_OK) return st;
  return from_hip(gptq::dequant_matmul_launch(x, xt == GPTQ_BF16, m, d_in, qweight, scales, zeros, g_idx, bits, d_out,
                                              n_groups, y, ws, static_cast<hipStream_t>(stream)));
}

gptq_status gptq_dequant_order(const int32_t* qweight, const int32_t* g_idx, int32_t bits, int64_t d_in,
                               int64_t d_out, int32_t* qweight_out, int32_t* g_idx_out, int32_t* order,
                               void* stream) {
  if (!qweight || !g_idx || !qweight_out || !g_idx_out || !order) return GPTQ_ERR_INVALID_ARG;
  if (!dim_ok(d_out) || !dim_ok(d_in) || d_in % 32 != 0 || !bits_ok(bits)) return GPTQ_ERR_INVALID_ARG;
  if (d_in / 32 * bits * d_out * 4 >= (int64_t{1} << 31)) return GPTQ_ERR_INVALID_ARG;
  return from_hip(gptq::dequant_order_launch(qweight, g_idx, bits, d_in, d_out, qweight_out, g_idx_out, order,
                                             static_cast<hipStream_t>(stream)));
}

size_t gptq_dequant_ordered_workspace_size(int64_t m, int64_t d_in, int64_t d_out) {
  if (m <= 0 || !tokens_ok(m) || !dim_ok(d_in) || !dim_ok(d_out) || d_in % 32 != 0) return 0;
  return gptq::dequant_ordered_workspace_bytes(m, d_in, d_out);
}

gptq_status gptq_dequant_matmul_ordered(const void* x, int32_t xt, int64_t m, int64_t d_in,
                                        const int32_t* qweight, const float* scales, const int32_t* zeros,
                                        const int32_t* g_idx, const int32_t* order, int32_t bits, int64_t d_out,
                                        int32_t n_groups, float* y, void* ws, size_t ws_bytes, void* stream) {
  if (!x || !qweight || !scales || !zeros || !g_idx || !order || !y) return GPTQ_ERR_INVALID_ARG;
  if (m <= 0 || !tokens_ok(m) || !dim_ok(d_out) || !dim_ok(d_in) || d_in % 32 != 0 || n_groups <= 0)
    return GPTQ_ERR_INVALID_ARG;
  if (!bits_ok(bits) || (xt != GPTQ_F32 && xt != GPTQ_BF16)) return GPTQ_ERR_INVALID_ARG;
  if (d_in / 32 * bits * d_out * 4 >= (int64_t{1} << 31) || int64_t{n_groups} * d_out * 4 >= (int64_t{1} << 31))
    return GPTQ_ERR_INVALID_ARG;
  const size_t need = gptq::dequant_ordered_workspace_bytes(m, d_in, d_out);
  if (!ws || ws_bytes < need || !aligned256(ws)) return GPTQ_ERR_WORKSPACE;
  return from_hip(gptq::dequant_matmul_ordered_launch(x, xt == GPTQ_BF16, m, d_in, qweight, scales, zeros, g_idx,
                                                      order, bits, d_out, n_groups, y, ws,
                                                      static_cast<hipStream_t>(stream)));
}

gptq_status gptq_quantize_tokens(const void* x, int32_t xt, int64_t n_tokens, int64_t d_in, int64_t ldx, int8_t* codes,
                                 float* scales, int32_t* sums_or_null, void* stream) {
  if ((xt != GPTQ_F32 && xt != GPTQ_BF16) || !rows_ok(n_tokens) || !dim_ok(d_in) || ldx < d_in) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return GPTQ_OK;
  if (!x || !codes || !scales) return GPTQ_ERR_INVALID_ARG;
  return from_hip(gptq::token_codes_launch(x, xt == GPTQ_BF16, n_tokens, d_in, ldx, codes, scales, sums_or_null,
                                           static_cast<hipStream_t>(stream)));
}

gptq_status gptq_integer_weight(const int32_t* qweight, const int32_t* zeros, int32_t bits, int64_t d_in, int64_t d_out,
                                int8_t* w, int32_t* offsets, void* stream) {
  if (!qweight || !zeros || !w || !offsets || !bits_ok(bits)) return GPTQ_ERR_INVALID_ARG;
  if (!dim_ok(d_in) || !dim_ok(d_out) || d_in % 32 != 0 || !aligned16(w)) return GPTQ_ERR_INVALID_ARG;
  return from_hip(gptq::integer_weight_launch(qweight, zeros, bits, d_in, d_out, w, offsets,
                                              static_cast<hipStream_t>(stream)));
}

size_t gptq_integer_workspace_size(int64_t m, int32_t xt, int64_t d_in, int64_t d_out) {
  if (m <= 0 || !rows_ok(m) || !dim_ok(d_in) || !dim_ok(d_out) || d_in % 32 != 0 || d_in > kMaxIntDim) return 0;
  if (xt != GPTQ_F32 && xt != GPTQ_BF16 && xt != GPTQ_I8) return 0;
  return gptq::integer_matmul_workspace(m, d_in, d_out, xt == GPTQ_I8, device_cus());
}

gptq_status gptq_integer_matmul(const void* x, int32_t xt, const float* x_scales, const int32_t* x_sums, int64_t m,
                                int64_t d_in, int64_t ldx, const int8_t* w, const float* w_scales,
                                const int32_t* w_offsets_or_null, int64_t d_out, void* y, int32_t yt, void* ws,
                                size_t ws_bytes, void* stream) {
  if ((xt != GPTQ_F32 && xt != GPTQ_BF16 && xt != GPTQ_I8) || (yt != GPTQ_F32 && yt != GPTQ_BF16))
    return GPTQ_ERR_INVALID_ARG;
  if (!rows_ok(m) || !dim_ok(d_in) || !dim_ok(d_out) || d_in % 32 != 0 || d_in > kMaxIntDim || ldx < d_in)
    return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!x || !w || !w_scales || !y || !aligned16(w)) return GPTQ_ERR_INVALID_ARG;
  if (xt == GPTQ_I8) {
    if (!x_scales || (w_offsets_or_null && !x_sums) || ldx % 16 != 0 || ldx > (int64_t{1} << 22) || !aligned16(x))
      return GPTQ_ERR_INVALID_ARG;
  }
  const int cus = device_cus();
  const size_t need = gptq::integer_matmul_workspace(m, d_in, d_out, xt == GPTQ_I8, cus);
  if (need > 0 && (!ws || ws_bytes < need || !aligned256(ws))) return GPTQ_ERR_WORKSPACE;
  return from_hip(gptq::integer_matmul_launch(x, xt, x_scales, x_sums, m, d_in, ldx, w, w_scales, w_offsets_or_null,
                                              d_out, y, yt == GPTQ_BF16, ws, cus, static_cast<hipStream_t>(stream)));
}

gptq_status gptq_cache_write(const gptq_cache* cache, const void* k, const void* v, int32_t xt, int64_t n_tokens,
                             int64_t ldk, int64_t ldv, const int64_t* slots, void* stream) {
  gptq::CacheShape c;
  if (!cache_shape(cache, &c) || (xt != GPTQ_F32 && xt != GPTQ_BF16) || !rows_ok(n_tokens)) return GPTQ_ERR_INVALID_ARG;
  const int64_t vec = (xt == GPTQ_BF16) ? 8 : 4, width = int64_t{c.n_kv} * c.hd;
  if (ldk < width || ldv < width || ldk % vec != 0 || ldv % vec != 0 || !cache_rows_ok(c, n_tokens))
    return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return GPTQ_OK;
  if (!k || !v || !slots || !aligned16(k) || !aligned16(v)) return GPTQ_ERR_INVALID_ARG;
  return from_hip(gptq::cache_write_launch(c, cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales, k, v,
                                           xt == GPTQ_BF16, n_tokens, ldk, ldv, slots,
                                           static_cast<hipStream_t>(stream)));
}

gptq_status gptq_cache_read(const gptq_cache* cache, const int64_t* slots, int64_t n_tokens, void* k, void* v, int32_t yt,
                            void* stream) {
  gptq::CacheShape c;
  if (!cache_shape(cache, &c) || (yt != GPTQ_F32 && yt != GPTQ_BF16) || !rows_ok(n_tokens)) return GPTQ_ERR_INVALID_ARG;
  if (!cache_rows_ok(c, n_tokens)) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return GPTQ_OK;
  if (!k || !v || !slots || !aligned16(k) || !aligned16(v)) return GPTQ_ERR_INVALID_ARG;
  return from_hip(gptq::cache_read_launch(c, cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales, slots,
                                          n_tokens, k, v, yt == GPTQ_BF16, static_cast<hipStream_t>(stream)));
}

namespace {
// The plan of a call within the header's limits whose launch has fewer than 2^32
// threads: of up to 64 rows a (sequence, key head) there are at most 64 / 16 + 1 tiles (heads
// wider than 128; 64 / 32 + 1 otherwise), which 2^21 of those keep below it, and
// of more rows tiles of 128, fewer than 2^23 + 2^21.
bool attention_plan_of(const gptq::CacheShape& c, int64_t n_tokens, int32_t n_heads, int32_t n_seq, int64_t pages_per_seq,
                       gptq::AttnPlan* plan) {
  if (n_heads < 1 || n_heads % c.n_kv != 0 || !rows_ok(n_tokens) || n_tokens * n_heads >= (int64_t{1} << 30) || n_seq < 0 ||
      n_seq > (1 << 20) || int64_t{n_seq} * c.n_kv > (int64_t{1} << 21) || pages_per_seq < 1 ||
      pages_per_seq > (int64_t{1} << 30) / c.page)
    return false;
  *plan = gptq::AttnPlan{};
  if (n_tokens == 0 || n_seq == 0) return true;
  *plan = gptq::attention_plan(c, n_tokens, n_heads, n_seq, pages_per_seq, device_cus());
  return plan->blocks * 256 < (int64_t{1} << 32);
}
}  // namespace

size_t gptq_attention_workspace_size(const gptq_cache* cache, int64_t n_tokens, int32_t n_heads, int32_t n_seq,
                                     int64_t pages_per_seq) {
  gptq::CacheShape c;
  gptq::AttnPlan plan;
  if (!cache_shape(cache, &c) || !attention_plan_of(c, n_tokens, n_heads, n_seq, pages_per_seq, &plan)) return 0;
  return plan.ws_bytes;
}

gptq_status gptq_cache_attention(const gptq_cache* cache, const void* q, int32_t qt, int64_t n_tokens, int64_t ldq,
                                 int32_t n_heads, const int32_t* page_table, int64_t pages_per_seq,
                                 const int32_t* q_starts, const int32_t* kv_lens, int32_t n_seq, float scale, void* out,
                                 int64_t ldo, void* ws, size_t ws_bytes, void* stream) {
  gptq::CacheShape c;
  if (!cache_shape(cache, &c) || qt != GPTQ_BF16 || !(scale > 0.0f && scale <= 3.402823466e38f))
    return GPTQ_ERR_INVALID_ARG;
  gptq::AttnPlan plan;
  if (!attention_plan_of(c, n_tokens, n_heads, n_seq, pages_per_seq, &plan)) return GPTQ_ERR_INVALID_ARG;
  const int64_t width = int64_t{n_heads} * c.hd;
  if (ldq < width || ldo < width || ldq % 8 != 0 || ldo % 8 != 0) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_seq == 0) return GPTQ_OK;
  if (!q || !out || !page_table || !q_starts || !kv_lens || !aligned16(q) || !aligned16(out)) return GPTQ_ERR_INVALID_ARG;
  if (plan.ws_bytes > 0 && (!ws || ws_bytes < plan.ws_bytes || !aligned256(ws))) return GPTQ_ERR_WORKSPACE;
  return from_hip(gptq::attention_launch(plan, c, q, ldq, n_tokens, n_heads, cache->k_codes, cache->v_codes,
                                         cache->k_scales, cache->v_scales, page_table, pages_per_seq, q_starts, kv_lens,
                                         n_seq, scale, out, ldo, ws, static_cast<hipStream_t>(stream)));
}

gptq_status gptq_phase_timing(int32_t enable) { return from_hip(gptq::phase_timing_set(enable != 0)); }

int32_t gptq_phase_count(void) { return gptq::kNumPhases; }

const char* gptq_phase_name(int32_t phase) { return gptq::phase_name(phase); }

gptq_status gptq_phase_read(float* ms, int32_t* launches, int32_t n) {
  if (!ms || !launches || n <= 0) return GPTQ_ERR_INVALID_ARG;
  return from_hip(gptq::phase_timing_read(ms, launches, n));
}

}  // extern "C"
