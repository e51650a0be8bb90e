// The paged key/value cache in 8- or 4-bit codes: writing tokens into it and
// reading them back.
//
// A row (one head of one token's key or value) is held as integer codes and
// one fp32 scale (quant_row.h): codes [n_pages][n_kv_heads][page_size][head_dim]
// so that the keys of one head lie together, as attention walks them.
// Both kernels move each row once; they are bound by HBM.  L lanes share a
// row, eight values (16 bytes of bf16) each, so a 64-lane wave covers 64 / L
// rows, the heads of one token next to each other in k and v.
#include "gptq_common.h"
#include "gptq_internal.h"
#include "quant_row.h"

namespace gptq {
namespace {

struct CacheRows {
  const void* x[2];   // k, v: write reads them, read writes them
  void* y[2];
  uint8_t* codes[2];
  float* scales[2];
  const int64_t* slots;
  int64_t ldx[2];     // elements between tokens
  int64_t rows;       // n_tokens * n_kv
  int64_t n_slots;    // n_pages * page_size
  int32_t n_kv, hd, page_shift, bits;
};

// index of the row of slot s, head h in the cache, or -1
GPTQ_DEV int64_t cache_row(const CacheRows& p, int64_t s, int h) {
  if (s < 0 || s >= p.n_slots) return -1;
  const int64_t page = s >> p.page_shift, tok = s & ((int64_t{1} << p.page_shift) - 1);
  return ((page * p.n_kv + h) << p.page_shift) + tok;
}

template <int L, bool BF16, int BITS>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheRows p) {
  constexpr int kTop = BITS == 8 ? 127 : 7;
  const int sub = threadIdx.x % L;
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / L;
  if (r >= p.rows) return;  // whole groups of L lanes
  const int which = blockIdx.y;
  const int64_t t = r / p.n_kv;
  const int h = static_cast<int>(r - t * p.n_kv);
  const int64_t at = cache_row(p, p.slots[t], h);
  float v[8];
  const bool live = sub * 8 < p.hd;
  if (live) {
    load8<BF16>(p.x[which], t * p.ldx[which] + static_cast<int64_t>(h) * p.hd + sub * 8, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
  uint32_t am = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = max(am, abs_bits(v[i]));
  am = group_max<L>(am);
  if (at < 0 || !live) return;
  const RowScale rs = row_scale(am, static_cast<float>(kTop));
  int c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = static_cast<int>(row_code<kTop>(v[i], rs));
  if (BITS == 8) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= (static_cast<uint32_t>(c[i]) & 0xFFu) << (8 * (i & 3));
    *reinterpret_cast<uint2*>(p.codes[which] + at * p.hd + sub * 8) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= static_cast<uint32_t>(c[i] + 8) << (4 * i);
    *reinterpret_cast<uint32_t*>(p.codes[which] + at * (p.hd / 2) + sub * 4) = w;
  }
  if (sub == 0) p.scales[which][at] = rs.scale;
}

template <int L, bool BF16, int BITS>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheRows p) {
  const int sub = threadIdx.x % L;
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / L;
  if (r >= p.rows || sub * 8 >= p.hd) return;
  const int which = blockIdx.y;
  const int64_t t = r / p.n_kv;
  const int h = static_cast<int>(r - t * p.n_kv);
  const int64_t at = cache_row(p, p.slots[t], h);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (at >= 0) {
    const float s = p.scales[which][at];
    if (BITS == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(p.codes[which] + at * p.hd + sub * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = s * static_cast<float>(static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3))));
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p.codes[which] + at * (p.hd / 2) + sub * 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = s * static_cast<float>(static_cast<int>((w >> (4 * i)) & 15u) - 8);
    }
  }
  const int64_t e = r * p.hd + sub * 8;  // contiguous [n_tokens, n_kv, hd]
  if (BF16) {
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = f32_to_bf16(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.y[which]) + e) = o;
  } else {
    f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(p.y[which]) + e);
    o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  }
}

template <int L, bool BF16, int BITS>
void rows_go(const CacheRows& p, bool write, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((p.rows * L + 255) / 256), 2);
  if (write) cache_write_kernel<L, BF16, BITS><<<grid, 256, 0, st>>>(p);
  else cache_read_kernel<L, BF16, BITS><<<grid, 256, 0, st>>>(p);
}

template <int L>
void rows_go_l(const CacheRows& p, bool bf16, bool write, hipStream_t st) {
  if (bf16 && p.bits == 8) rows_go<L, true, 8>(p, write, st);
  else if (bf16) rows_go<L, true, 4>(p, write, st);
  else if (p.bits == 8) rows_go<L, false, 8>(p, write, st);
  else rows_go<L, false, 4>(p, write, st);
}

hipError_t rows_launch(const CacheRows& p, bool bf16, bool write, hipStream_t st) {
  if (p.hd <= 16) rows_go_l<2>(p, bf16, write, st);
  else if (p.hd <= 32) rows_go_l<4>(p, bf16, write, st);
  else if (p.hd <= 64) rows_go_l<8>(p, bf16, write, st);
  else if (p.hd <= 128) rows_go_l<16>(p, bf16, write, st);
  else rows_go_l<32>(p, bf16, write, st);
  return hipGetLastError();
}

CacheRows rows_of(const CacheShape& c, void* kc, void* vc, float* ks, float* vs, const int64_t* slots, int64_t n) {
  CacheRows p{};
  p.codes[0] = static_cast<uint8_t*>(kc);
  p.codes[1] = static_cast<uint8_t*>(vc);
  p.scales[0] = ks;
  p.scales[1] = vs;
  p.slots = slots;
  p.rows = n * c.n_kv;
  p.n_slots = c.n_pages * c.page;
  p.n_kv = c.n_kv;
  p.hd = c.hd;
  p.bits = c.bits;
  p.page_shift = __builtin_ctz(static_cast<unsigned>(c.page));
  return p;
}

}  // namespace

hipError_t cache_write_launch(const CacheShape& c, void* kc, void* vc, float* ks, float* vs, const void* k,
                              const void* v, bool bf16, int64_t n, int64_t ldk, int64_t ldv, const int64_t* slots,
                              hipStream_t st) {
  CacheRows p = rows_of(c, kc, vc, ks, vs, slots, n);
  p.x[0] = k;
  p.x[1] = v;
  p.ldx[0] = ldk;
  p.ldx[1] = ldv;
  return rows_launch(p, bf16, true, st);
}

hipError_t cache_read_launch(const CacheShape& c, const void* kc, const void* vc, const float* ks, const float* vs,
                             const int64_t* slots, int64_t n, void* k, void* v, bool bf16, hipStream_t st) {
  CacheRows p = rows_of(c, const_cast<void*>(kc), const_cast<void*>(vc), const_cast<float*>(ks),
                        const_cast<float*>(vs), slots, n);
  p.y[0] = k;
  p.y[1] = v;
  return rows_launch(p, bf16, false, st);
}

}  // namespace gptq
