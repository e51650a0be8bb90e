// The paged key/value cache in 8- or 4-bit codes: writing tokens into it and
// reading them back.
//
// A row (one head of one token's key or value) is held as integer codes and
// one fp32 scale (quant_row.h): codes [n_pages][n_kv_heads][page_size][head_dim]
// so that the keys of one head lie together, as attention walks them.
// Both kernels move each row once; they are bound by HBM.  L lanes share a
// row, eight values (16 bytes of bf16) each, so a 64-lane wave covers 64 / L
// rows, the heads of one token next to each other in k and v.  Once that fills
// the card, a group of lanes takes four rows and loads them together: 16384
// tokens of 32 heads x 128 in bf16 to int8 codes at scattered slots are written
// in 100 us and read in 95 us, 4.1 and 4.3 TB/s (one row a group 117 and 116 us;
// two rows 102 and 104; eight 115 and 90).  64 tokens of 8 heads: 3.6 and 3.0 us,
// a launch and two dependent loads.
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

// The U rows of one group of L lanes: row(i) is 256 / L rows after row(i - 1),
// so that a workgroup's lanes cover neighbouring rows at each i.
template <int L, int U>
struct RowWalk {
  int64_t t[U];
  int h[U];
  bool in[U];
  GPTQ_DEV explicit RowWalk(const CacheRows& p) {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 / L * U);
    const int64_t t0 = first / p.n_kv;  // of the workgroup; the lanes' divisions are of small numbers
    const uint32_t h0 = static_cast<uint32_t>(first - t0 * p.n_kv), n = static_cast<uint32_t>(p.n_kv);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t off = i * (256 / L) + threadIdx.x / L;
      const uint32_t d = (h0 + off) / n;
      in[i] = first + off < p.rows;
      t[i] = in[i] ? t0 + d : 0;
      h[i] = in[i] ? static_cast<int>(h0 + off - d * n) : 0;
    }
  }
};

template <int L, int U, bool BF16, int BITS>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheRows p) {
  constexpr int kTop = BITS == 8 ? 127 : 7;
  const int sub = threadIdx.x % L, which = blockIdx.y;
  const bool live = sub * 8 < p.hd;
  const RowWalk<L, U> row(p);
  int64_t at[U];
  float v[U][8];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    at[i] = p.slots[row.t[i]];
    load8<BF16>(p.x[which], row.t[i] * p.ldx[which] + static_cast<int64_t>(row.h[i]) * p.hd + (live ? sub * 8 : 0), v[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    at[i] = row.in[i] ? cache_row(p, at[i], row.h[i]) : -1;
    uint32_t am = 0u;  // lanes past the row hold its first values again
#pragma unroll
    for (int j = 0; j < 8; ++j) am = max(am, abs_bits(v[i][j]));
    am = group_max<L>(am);
    if (at[i] < 0 || !live) continue;
    const RowScale rs = row_scale(am, static_cast<float>(kTop));
    uint32_t w[2];
    if (BITS == 8) {
      row_codes<kTop, 0>(v[i], rs, w);
      *reinterpret_cast<uint2*>(p.codes[which] + at[i] * p.hd + sub * 8) = make_uint2(w[0], w[1]);
    } else {
      row_codes<kTop, 8>(v[i], rs, w);  // bytes of 1 .. 15: two to a byte, four in each word's low half
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        w[j] = (w[j] | (w[j] >> 4)) & 0x00FF00FFu;
        w[j] |= w[j] >> 8;
      }
      *reinterpret_cast<uint32_t*>(p.codes[which] + at[i] * (p.hd / 2) + sub * 4) = (w[0] & 0xFFFFu) | (w[1] << 16);
    }
    if (sub == 0) p.scales[which][at[i]] = rs.scale;
  }
}

template <int L, int U, bool BF16, int BITS>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheRows p) {
  const int sub = threadIdx.x % L, which = blockIdx.y;
  if (sub * 8 >= p.hd) return;
  const RowWalk<L, U> row(p);
  int64_t at[U];
  float s[U];
  uint2 w[U];
#pragma unroll
  for (int i = 0; i < U; ++i) at[i] = cache_row(p, p.slots[row.t[i]], row.h[i]);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t a = at[i] < 0 ? 0 : at[i];  // a cache has a row 0
    s[i] = p.scales[which][a];
    if (BITS == 8) w[i] = *reinterpret_cast<const uint2*>(p.codes[which] + a * p.hd + sub * 8);
    else w[i].x = *reinterpret_cast<const uint32_t*>(p.codes[which] + a * (p.hd / 2) + sub * 4);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (!row.in[i]) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (BITS == 8) v[j] = s[i] * static_cast<float>(static_cast<int8_t>((j < 4 ? w[i].x : w[i].y) >> (8 * (j & 3))));
      else v[j] = s[i] * static_cast<float>(static_cast<int>((w[i].x >> (4 * j)) & 15u) - 8);
      v[j] = at[i] < 0 ? 0.f : v[j];
    }
    const int64_t e = (row.t[i] * p.n_kv + row.h[i]) * p.hd + sub * 8;  // contiguous [n_tokens, n_kv, hd]
    if (BF16) {
      u32x4_t o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = f32_to_bf16(v[2 * j]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * j + 1])) << 16);
      *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.y[which]) + e) = o;
    } else {
      f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(p.y[which]) + e);
      o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
      o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    }
  }
}

template <int L, int U, bool BF16, int BITS>
void rows_go_u(const CacheRows& p, bool write, hipStream_t st) {
  constexpr int kRows = 256 / L * U;
  const dim3 grid(static_cast<unsigned>((p.rows + kRows - 1) / kRows), 2);
  if (write) cache_write_kernel<L, U, BF16, BITS><<<grid, 256, 0, st>>>(p);
  else cache_read_kernel<L, U, BF16, BITS><<<grid, 256, 0, st>>>(p);
}

template <int L, bool BF16, int BITS>
void rows_go(const CacheRows& p, bool write, hipStream_t st) {
  // four rows a group while that leaves four workgroups a CU and tensor (1024 of them)
  if (p.rows >= 256 / L * 4 * 1024ll) rows_go_u<L, 4, BF16, BITS>(p, write, st);
  else rows_go_u<L, 1, BF16, BITS>(p, write, st);
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
