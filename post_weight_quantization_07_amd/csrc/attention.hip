// Attention of new tokens over the paged quantized cache (cache.hip).
//
// For a new token at position a of its sequence (a = length - n_new + i), head
// h and its key head, over the keys j <= a:
//   s_j = scale (q . ck_j) sk_j,  p = softmax(s),  out = sum_j p_j sv_j cv_j
// in one pass over the keys with the running maximum and sum of the softmax.
// The integer codes are exact in bf16 and enter the matrix cores as they are;
// the key scale multiplies the score in fp32 and the value scale multiplies
// p_j before its one rounding to bf16 (2^-9 relative, at most), so the scales
// cost no precision and the products and sums are fp32.
//
// The query heads that share a key head are rows of one tile: row r of a
// sequence is token r / G, head r % G of its group, and M rows make a tile.
// The work list is (sequence, row tile, key split, key head); its lengths are
// known on the device only, so every workgroup finds its entry from q_starts
// and kv_lens with a scan by one wave (find_work).
#include "gptq_common.h"
#include "gptq_internal.h"
#include "quant_row.h"

#include <algorithm>

namespace gptq {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr int kUnit = 64;  // keys per unit of the work split

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* codes[2];
  const float* scales[2];
  const int32_t* table;
  const int32_t* starts;
  const int32_t* lens;
  float* partial;
  int64_t ldq, ldo, ld_table;
  int64_t n_tokens, n_pages, max_slots;
  int32_t n_seq, n_kv, group, hd, page_shift;
  int32_t tile_rows;   // M
  int32_t target;      // workgroups the keys are split for
  int32_t min_units;   // fewest units of a split
  float scale_log2e;
};

struct Seq {
  int q0, n, len, tiles, units;
};

// everything read from the caller's device arrays is clamped, so that no value
// in them makes an access leave its buffer
GPTQ_DEV Seq seq_info(const AttnParams& p, int i) {
  Seq s;
  const int64_t total = p.n_tokens;
  const int64_t a = min(max(static_cast<int64_t>(p.starts[i]), int64_t{0}), total);
  const int64_t b = min(max(static_cast<int64_t>(p.starts[i + 1]), a), total);
  const int64_t cap = p.ld_table << p.page_shift;
  s.q0 = static_cast<int>(a);
  s.n = static_cast<int>(b - a);
  s.len = static_cast<int>(min(max(static_cast<int64_t>(p.lens[i]), int64_t{0}), cap));
  s.tiles = s.n > 0 ? (s.n * p.group - 1) / p.tile_rows + 1 : 0;
  s.units = s.len > 0 ? (s.len - 1) / kUnit + 1 : 1;
  return s;
}

GPTQ_DEV int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

struct Work {
  Seq s;
  int seq, tile, split, n_split;
  int64_t slot;  // of the unit's first split (for this key head: times n_kv, plus h)
};

// Entry u of the list (SPLITS: of (tile, split) pairs; otherwise of tiles).
// The keys of a sequence are split so that a split has at least `per` units,
// per = (all units) / target: a batch with enough tiles is not split, a long
// sequence among short ones is.
template <bool SPLITS>
GPTQ_DEV bool find_work(const AttnParams& p, int64_t u, Work& w) {
  const int lane = lane_id();
  int64_t total = 0;
  for (int i0 = 0; i0 < p.n_seq; i0 += 64) {
    int64_t v = 0;
    if (i0 + lane < p.n_seq) {
      const Seq s = seq_info(p, i0 + lane);
      v = static_cast<int64_t>(s.tiles) * s.units;
    }
    total += __shfl(wave_scan(v, lane), 63);
  }
  const int64_t all = total * p.n_kv;
  const int64_t per = max((all + p.target - 1) / p.target, static_cast<int64_t>(p.min_units));
  int64_t base = 0, slots = 0;
  for (int i0 = 0; i0 < p.n_seq; i0 += 64) {
    Seq s{};
    int64_t cnt = 0, slot = 0;
    int n_split = 1;
    if (i0 + lane < p.n_seq) {
      s = seq_info(p, i0 + lane);
      n_split = static_cast<int>((s.units + per - 1) / per);
      slot = n_split > 1 ? static_cast<int64_t>(s.tiles) * n_split : 0;
      cnt = SPLITS ? static_cast<int64_t>(s.tiles) * n_split : s.tiles;
    }
    const int64_t end = base + wave_scan(cnt, lane);
    const int64_t slot_end = slots + wave_scan(slot, lane);
    const uint64_t hit = __ballot(u < end);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      w.seq = i0 + l;
      w.s.q0 = __shfl(s.q0, l);
      w.s.n = __shfl(s.n, l);
      w.s.len = __shfl(s.len, l);
      w.s.tiles = __shfl(s.tiles, l);
      w.s.units = __shfl(s.units, l);
      w.n_split = __shfl(n_split, l);
      const int64_t local = u - __shfl(end - cnt, l);
      w.slot = __shfl(slot_end - slot, l);
      if (SPLITS) {
        w.tile = static_cast<int>(local / w.n_split);
        w.split = static_cast<int>(local % w.n_split);
      } else {
        w.tile = static_cast<int>(local);
        w.split = 0;
      }
      w.slot += static_cast<int64_t>(w.tile) * w.n_split;
      return true;
    }
    base = __shfl(end, 63);
    slots = __shfl(slot_end, 63);
  }
  return false;
}

// v_exp_f32: 2^x within an ulp; -inf gives 0 (results below the normal range flush to 0)
GPTQ_DEV float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

GPTQ_DEV float max_over_groups(float v) {  // lanes l, l ^ 16, l ^ 32, l ^ 48
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
GPTQ_DEV float sum_over_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

GPTQ_DEV uint32_t pack_hi(float lo, float hi) {  // two values exact in bf16
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
GPTQ_DEV uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("v_cvt_pk_bf16_f32 %0, %1, %2" : "=v"(r) : "v"(lo), "v"(hi));
  return r;
}
template <int B>
GPTQ_DEV float sbyte(uint32_t w) {
  return static_cast<float>(static_cast<int8_t>(w >> (8 * B)));
}

// 8 codes of one row, 8 bits: two words -> bf16 in the order of the bytes
GPTQ_DEV bf16x8_t row8(uint32_t a, uint32_t b) {
  const u32x4_t v = {pack_hi(sbyte<0>(a), sbyte<1>(a)), pack_hi(sbyte<2>(a), sbyte<3>(a)),
                     pack_hi(sbyte<0>(b), sbyte<1>(b)), pack_hi(sbyte<2>(b), sbyte<3>(b))};
  return __builtin_bit_cast(bf16x8_t, v);
}
// 8 codes of one row, 4 bits, as 24 + code (16 + nibble: 0x4180 | nibble << 3,
// exact), in the order 0 4 1 5 2 6 3 7 that a shift and a mask give
constexpr uint32_t kNibMask = 0x00780078u, kNibOne = 0x41804180u;
GPTQ_DEV bf16x8_t row4(uint32_t a) {
  const u32x4_t v = {((a << 3) & kNibMask) | kNibOne, ((a >> 1) & kNibMask) | kNibOne,
                     ((a >> 5) & kNibMask) | kNibOne, ((a >> 9) & kNibMask) | kNibOne};
  return __builtin_bit_cast(bf16x8_t, v);
}
// byte B of eight keys' words
template <int B>
GPTQ_DEV bf16x8_t col8(const uint32_t (&w)[8]) {
  const u32x4_t v = {pack_hi(sbyte<B>(w[0]), sbyte<B>(w[1])), pack_hi(sbyte<B>(w[2]), sbyte<B>(w[3])),
                     pack_hi(sbyte<B>(w[4]), sbyte<B>(w[5])), pack_hi(sbyte<B>(w[6]), sbyte<B>(w[7]))};
  return __builtin_bit_cast(bf16x8_t, v);
}
// both nibbles of byte B of eight keys' words, as 24 + code
template <int B>
GPTQ_DEV void col4(const uint32_t (&w)[8], bf16x8_t& lo, bf16x8_t& hi) {
  u32x4_t a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x0C000C00u | ((4u + B) << 16) | B);
    a[i] = ((t << 3) & kNibMask) | kNibOne;
    b[i] = ((t >> 1) & kNibMask) | kNibOne;
  }
  lo = __builtin_bit_cast(bf16x8_t, a);
  hi = __builtin_bit_cast(bf16x8_t, b);
}

// ---------------------------------------------------- keys split over waves --
// A workgroup owns 16 MT rows of one (sequence, key head) and one key split;
// its NW waves take turns of 32 keys, straight from global memory into the
// operands, and their results meet in LDS at the end.
//
// Scores are computed transposed, S^T = K Q^T (16x16x32): lane l holds key
// l % 16's codes at the 8 BPL dims of its group g = l / 16, and its results
// are keys 4 g + r (r < 4) for query row l % 16.  Two such tiles (32 keys) are,
// without any exchange between lanes, the P^T operand of O^T = V^T P^T, when
// the sum over keys runs in that order; so lane l reads V at keys 4 g + r and
// 16 + 4 g + r, dims (l % 16) HDP / 16 + t, and byte t of its eight words
// makes the operand of output tile t.  Lane l then ends up with query row
// l % 16, dims g HDP / 4 ... in order.
template <int HDP, int BITS, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void attn_split_kernel(AttnParams p) {
  constexpr int kKW = HDP * BITS / 128;        // words of K a lane holds per key: HDP / 4 dims
  constexpr int kVB = HDP * BITS / 128;        // bytes of V a lane holds per key: HDP / 16 dims
  constexpr int kVW = (kVB + 3) / 4;
  constexpr int kSteps = HDP / 32;             // products of a 16-key score tile
  constexpr int kTiles = HDP / 16;             // output tiles
  constexpr int kM = 16 * MT;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.n_kv));
  Work w;
  if (!find_work<true>(p, blockIdx.x / static_cast<unsigned>(p.n_kv), w)) return;
  const int rows = w.s.n * p.group;
  const int r0 = w.tile * kM;
  const int first = w.s.len - w.s.n + r0 / p.group;                              // last key of the tile's first row
  const int vis = w.s.len - w.s.n + (min(r0 + kM, rows) - 1) / p.group + 1;       // keys any of its rows sees
  const int units = vis > 0 ? (vis - 1) / kUnit + 1 : 0;
  const int per = (units + w.n_split - 1) / w.n_split;
  const int key0 = w.split * per * kUnit, key1 = min(vis, (w.split + 1) * per * kUnit);

  // query operands, their sums (4 bits), and each row's last key
  bf16x8_t q[MT][kSteps];
  float bias[MT];
  int lim[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = r0 + 16 * i + c;
    const bool live = r < rows;
    const int tok = live ? r / p.group : 0;
    lim[i] = live ? w.s.len - w.s.n + tok : -1;
    const uint16_t* src = p.q + static_cast<int64_t>(w.s.q0 + tok) * p.ldq +
                          static_cast<int64_t>(h * p.group + (live ? r % p.group : 0)) * p.hd;
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = g * (HDP / 4) + 8 * s;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (live && d < p.hd) v = *reinterpret_cast<const u32x4_t*>(src + d);
      if (BITS == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += __uint_as_float(v[e] << 16) + __uint_as_float(v[e] & 0xFFFF0000u);
        // dims 0..7 -> 0 4 1 5 2 6 3 7
        v = u32x4_t{(v[0] & 0xFFFFu) | (v[2] << 16), (v[0] >> 16) | (v[2] & 0xFFFF0000u),
                    (v[1] & 0xFFFFu) | (v[3] << 16), (v[1] >> 16) | (v[3] & 0xFFFF0000u)};
      }
      q[i][s] = __builtin_bit_cast(bf16x8_t, v);
    }
    bias[i] = BITS == 4 ? -24.f * sum_over_groups(sum) : 0.f;
  }

  f32x4_t acc[MT][kTiles];
  float m[MT], l[MT], psum[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
    psum[i] = 0.f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  const int row_bytes = p.hd * BITS / 8;
  const int page_mask = (1 << p.page_shift) - 1;
  const int32_t* table = p.table + static_cast<int64_t>(w.seq) * p.ld_table;
  for (int k0 = key0 + 32 * wave; k0 < key1; k0 += 32 * NW) {
    uint32_t kw[2][kKW], vw[kVW][8];
    f32x4_t ks[2], vs[2];
    bool ok[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int k = k0 + 16 * b;
      const int page = (k < key1) ? table[k >> p.page_shift] : -1;
      ok[b] = page >= 0 && page < p.n_pages;
      const int64_t row = ((static_cast<int64_t>(ok[b] ? page : 0) * p.n_kv + h) << p.page_shift) + (k & page_mask);
      const uint8_t* kp = p.codes[0] + (row + c) * row_bytes + g * (kKW * 4);
#pragma unroll
      for (int e = 0; e < kKW; e += (BITS == 8 ? 2 : 1)) {
        const bool in = g * (HDP / 4) + e * (32 / BITS) < p.hd;
        if (BITS == 8) {
          const uint2 v = in ? *reinterpret_cast<const uint2*>(kp + 4 * e) : make_uint2(0u, 0u);
          kw[b][e] = v.x;
          kw[b][e + 1] = v.y;
        } else {
          kw[b][e] = in ? *reinterpret_cast<const uint32_t*>(kp + 4 * e) : 0u;
        }
      }
      const bool vin = c * (HDP / 16) < p.hd;
      const uint8_t* vp = p.codes[1] + (row + 4 * g) * row_bytes + c * kVB;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint8_t* one = vp + r * row_bytes;
        if (kVB == 2) vw[0][4 * b + r] = vin ? *reinterpret_cast<const uint16_t*>(one) : 0u;
        if (kVB >= 4) {
#pragma unroll
          for (int e = 0; e < kVW; ++e) vw[e][4 * b + r] = vin ? *reinterpret_cast<const uint32_t*>(one + 4 * e) : 0u;
        }
      }
      ks[b] = *reinterpret_cast<const f32x4_t*>(p.scales[0] + row + 4 * g);
      vs[b] = *reinterpret_cast<const f32x4_t*>(p.scales[1] + row + 4 * g);
    }
    const bool masked = k0 + 31 > first || !ok[0] || !ok[1];

    float s[MT][8];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      bf16x8_t kop[kSteps];
#pragma unroll
      for (int e = 0; e < kSteps; ++e) kop[e] = BITS == 8 ? row8(kw[b][2 * e % kKW], kw[b][(2 * e + 1) % kKW]) : row4(kw[b][e % kKW]);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        f32x4_t a = {bias[i], bias[i], bias[i], bias[i]};
#pragma unroll
        for (int e = 0; e < kSteps; ++e) a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kop[e], q[i][e], a, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) s[i][4 * b + r] = a[r] * (ks[b][r] * p.scale_log2e);
      }
    }
    bf16x8_t pop[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      bool see[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) see[j] = true;
      if (masked) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          see[j] = ok[j >> 2] && k0 + 16 * (j >> 2) + 4 * g + (j & 3) <= lim[i];
          if (!see[j]) s[i][j] = kNegInf;
        }
      }
      float mx = s[i][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mx = fmaxf(mx, s[i][j]);
      mx = max_over_groups(mx);
      if (__any(mx > m[i])) {
        const float mn = fmaxf(m[i], mx);
        const float alpha = fast_exp2(m[i] - (mn == kNegInf ? 0.f : mn));
        m[i] = mn;
        l[i] *= alpha;
        psum[i] *= alpha;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][t][r] *= alpha;
      }
      const float mm = m[i] == kNegInf ? 0.f : m[i];
      float pv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = fast_exp2(s[i][j] - mm);
        l[i] += e;
        pv[j] = e * vs[j >> 2][j & 3];
        if (masked && !see[j]) pv[j] = 0.f;  // the scale of a key that is not there may be anything
      }
      const u32x4_t pk = {pack_bf16(pv[0], pv[1]), pack_bf16(pv[2], pv[3]), pack_bf16(pv[4], pv[5]),
                          pack_bf16(pv[6], pv[7])};
      if (BITS == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) psum[i] += __uint_as_float(pk[e] << 16) + __uint_as_float(pk[e] & 0xFFFF0000u);
      }
      pop[i] = __builtin_bit_cast(bf16x8_t, pk);
    }
#pragma unroll
    for (int e = 0; e < kVW; ++e) {
      bf16x8_t vop[8];
      if (BITS == 8) {
        vop[0] = col8<0>(vw[e]);
        vop[1] = col8<1>(vw[e]);
        vop[2] = col8<2>(vw[e]);
        vop[3] = col8<3>(vw[e]);
      } else {
        col4<0>(vw[e], vop[0], vop[1]);
        col4<1>(vw[e], vop[2], vop[3]);
        if (kVB >= 4) {
          col4<2>(vw[e], vop[4], vop[5]);
          col4<3>(vw[e], vop[6], vop[7]);
        }
      }
      constexpr int kPer = BITS == 8 ? 4 : (kVB >= 4 ? 8 : 4);
#pragma unroll
      for (int t = 0; t < kPer; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i][e * kPer + t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vop[t], pop[i], acc[i][e * kPer + t], 0, 0, 0);
    }
  }

  // the waves' results
  __shared__ float wm[NW][kM], wl[NW][kM];
  __shared__ __attribute__((aligned(16))) float wo[NW][16][HDP + 4];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    l[i] = sum_over_groups(l[i]);
    if (BITS == 4) psum[i] = sum_over_groups(psum[i]);
    if (g == 0) {
      wm[wave][16 * i + c] = m[i];
      wl[wave][16 * i + c] = l[i];
    }
  }
  __syncthreads();
  const int64_t slot = (w.slot + w.split) * p.n_kv + h;
  const bool whole = w.n_split == 1;
  if (!whole && slot >= p.max_slots) return;  // the whole workgroup
  float* part = p.partial + slot * (kM * (HDP + 2));
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    float top = kNegInf;
#pragma unroll
    for (int v = 0; v < NW; ++v) top = fmaxf(top, wm[v][16 * i + c]);
    const float f = fast_exp2(m[i] - (top == kNegInf ? 0.f : top));
    // lane l: dims g HDP / 4 + r HDP / 16 + t
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int t = 0; t < kTiles; t += 4) {
        f32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = f * (acc[i][t + e][r] - (BITS == 4 ? 24.f * psum[i] : 0.f));
        *reinterpret_cast<f32x4_t*>(&wo[wave][c][g * (HDP / 4) + r * (HDP / 16) + t]) = v;
      }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * HDP / 4; e += 64 * NW) {
      const int row = e / (HDP / 4), d = (e % (HDP / 4)) * 4;
      const int r = r0 + 16 * i + row;
      float t2 = kNegInf;
#pragma unroll
      for (int v = 0; v < NW; ++v) t2 = fmaxf(t2, wm[v][16 * i + row]);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < NW; ++v) sum += wl[v][16 * i + row] * fast_exp2(wm[v][16 * i + row] - (t2 == kNegInf ? 0.f : t2));
      f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(&wo[v][row][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += a[j];
      }
      if (!whole) {
        *reinterpret_cast<f32x4_t*>(part + (16 * i + row) * HDP + d) = o;
        if (d == 0) {
          part[kM * HDP + 16 * i + row] = t2;
          part[kM * HDP + kM + 16 * i + row] = sum;
        }
      } else if (r < rows && d < p.hd) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint2 b;
        b.x = f32_to_bf16(o[0] * inv) | (static_cast<uint32_t>(f32_to_bf16(o[1] * inv)) << 16);
        b.y = f32_to_bf16(o[2] * inv) | (static_cast<uint32_t>(f32_to_bf16(o[3] * inv)) << 16);
        *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(w.s.q0 + r / p.group) * p.ldo +
                                  static_cast<int64_t>(h * p.group + r % p.group) * p.hd + d) = b;
      }
    }
    __syncthreads();
  }
}

// Joins the splits of a tile, in their order.  One workgroup per (tile, key
// head); tiles that were not split were written by the kernel above.
template <int HDP, int MT>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p) {
  constexpr int kM = 16 * MT;
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.n_kv));
  Work w;
  if (!find_work<false>(p, blockIdx.x / static_cast<unsigned>(p.n_kv), w) || w.n_split == 1) return;
  const int rows = w.s.n * p.group, r0 = w.tile * kM;
  if ((w.slot + w.n_split - 1) * p.n_kv + h >= p.max_slots) return;
  const int64_t step = static_cast<int64_t>(p.n_kv) * (kM * (HDP + 2));
  const float* part = p.partial + (w.slot * p.n_kv + h) * (kM * (HDP + 2));
  for (int e = threadIdx.x; e < kM * HDP / 4; e += 256) {
    const int row = e / (HDP / 4), d = (e % (HDP / 4)) * 4;
    const int r = r0 + row;
    if (r >= rows || d >= p.hd) continue;
    float top = kNegInf;
    for (int s = 0; s < w.n_split; ++s) top = fmaxf(top, part[s * step + kM * HDP + row]);
    const float safe = top == kNegInf ? 0.f : top;
    float sum = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < w.n_split; ++s) {
      const float f = fast_exp2(part[s * step + kM * HDP + row] - safe);
      sum += f * part[s * step + kM * HDP + kM + row];
      const f32x4_t a = *reinterpret_cast<const f32x4_t*>(part + s * step + row * HDP + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] += f * a[j];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint2 b;
    b.x = f32_to_bf16(o[0] * inv) | (static_cast<uint32_t>(f32_to_bf16(o[1] * inv)) << 16);
    b.y = f32_to_bf16(o[2] * inv) | (static_cast<uint32_t>(f32_to_bf16(o[3] * inv)) << 16);
    *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(w.s.q0 + r / p.group) * p.ldo +
                              static_cast<int64_t>(h * p.group + r % p.group) * p.hd + d) = b;
  }
}

int head_pad(int hd) { return hd <= 64 ? 64 : hd <= 128 ? 128 : 256; }

template <int HDP, int BITS>
void attn_go(const AttnParams& p, unsigned blocks, unsigned joins, hipStream_t st) {
  attn_split_kernel<HDP, BITS, 1, 8><<<blocks, 512, 0, st>>>(p);
  if (joins) attn_join_kernel<HDP, 1><<<joins, 256, 0, st>>>(p);
}

}  // namespace

AttnPlan attention_plan(const CacheShape& c, int64_t n_tokens, int32_t n_heads, int32_t n_seq, int64_t ld_table, int n_cu) {
  AttnPlan a{};
  a.tile_rows = 16;
  a.target = 2 * n_cu;
  a.min_units = 4;
  const int64_t group = n_heads / c.n_kv;
  const int64_t tiles = (n_tokens * group) / a.tile_rows + std::min<int64_t>(n_seq, n_tokens);
  a.joins = tiles * c.n_kv;
  a.blocks = a.joins + a.target;
  // no sequence can have more units than one split holds: nothing to join
  const int64_t most = (ld_table * c.page + kUnit - 1) / kUnit;
  if (most <= a.min_units) {
    a.joins = 0;
    a.blocks = tiles * c.n_kv;
  } else {
    a.slots = 2 * static_cast<int64_t>(a.target);
    a.ws_bytes = static_cast<size_t>(a.slots) * a.tile_rows * (head_pad(c.hd) + 2) * 4;
  }
  return a;
}

hipError_t attention_launch(const AttnPlan& plan, const CacheShape& c, const void* q, int64_t ldq, int64_t n_tokens,
                            int32_t n_heads, const void* kc, const void* vc, const float* ks, const float* vs,
                            const int32_t* table, int64_t ld_table, const int32_t* starts, const int32_t* lens,
                            int32_t n_seq, float scale, void* out, int64_t ldo, void* ws, hipStream_t st) {
  AttnParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.codes[0] = static_cast<const uint8_t*>(kc);
  p.codes[1] = static_cast<const uint8_t*>(vc);
  p.scales[0] = ks;
  p.scales[1] = vs;
  p.table = table;
  p.starts = starts;
  p.lens = lens;
  p.partial = static_cast<float*>(ws);
  p.ldq = ldq;
  p.ldo = ldo;
  p.ld_table = ld_table;
  p.n_tokens = n_tokens;
  p.n_pages = c.n_pages;
  p.max_slots = plan.slots;
  p.n_seq = n_seq;
  p.n_kv = c.n_kv;
  p.group = n_heads / c.n_kv;
  p.hd = c.hd;
  p.page_shift = __builtin_ctz(static_cast<unsigned>(c.page));
  p.tile_rows = plan.tile_rows;
  p.target = plan.target;
  p.min_units = plan.min_units;
  p.scale_log2e = scale * 1.4426950408889634f;
  const unsigned b = static_cast<unsigned>(plan.blocks), j = static_cast<unsigned>(plan.joins);
  const int hp = head_pad(c.hd);
  if (c.bits == 8) {
    if (hp == 64) attn_go<64, 8>(p, b, j, st);
    else if (hp == 128) attn_go<128, 8>(p, b, j, st);
    else attn_go<256, 8>(p, b, j, st);
  } else {
    if (hp == 64) attn_go<64, 4>(p, b, j, st);
    else if (hp == 128) attn_go<128, 4>(p, b, j, st);
    else attn_go<256, 4>(p, b, j, st);
  }
  return hipGetLastError();
}

}  // namespace gptq
