// Attention of new tokens over the paged quantized cache (cache.hip).
//
// For a new token at position a of its sequence (a = length - n_new + i), head
// h and its key head, over the keys j <= a:
//   s_j = scale (q . ck_j) sk_j,  p = softmax(s),  out = sum_j p_j sv_j cv_j
// in one pass over the keys with the running maximum and sum of the softmax.
// Scores: q and the key codes are exact in bf16, their products are summed in
// fp32 and the key scale multiplies the sum in fp32.  Output: the second
// product runs in fp16, whose 11 bits round eight times finer than bf16's 8: an
// operand is off by 2^-11 relative.  fp16's range is narrow, and a key may have any
// weight and any value scale.  So what it holds is taken relative to the largest
// weight times value scale that a row has seen (ProductUnit), which is held above
// 2^8, and what falls below fp16's normal range is off by 2^-33 of that a key at
// most; where a kernel keeps weight and scale apart (the tile kernel, while the
// scales are within 2^8 of each other), by less than 2^-24.
//
// The query heads that share a key head are rows of one tile: row r of a
// sequence is token r / G, head r % G of its group, and M rows make a tile.
// The work list is (sequence, row tile, key split, key head); its lengths are
// known on the device only, so every workgroup finds its entry from q_starts
// and kv_lens with a scan by one wave (find_work).
#include "gptq_common.h"
#include "gptq_internal.h"
#include "key_lanes.h"
#include "quant_row.h"

#include <algorithm>
#include <type_traits>

namespace gptq {
namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4_t;
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef u32x4_t u32x4_at8_t __attribute__((aligned(8)));
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;

constexpr float kNegInf = -__builtin_inff();
constexpr float kNoMax = -3.402823466e38f;  // running maximum before any key: below every score, and finite, so that differences stay defined
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
  int32_t tile_rows, tile_shift;    // M, a power of two
  int32_t max_len;                  // keys that a row of the table can name
  float inv_target;                 // n_kv / the workgroups the keys are split for
  float min_units;                  // fewest units of a split,
  float few;                        // or two while there are no more (tile, unit) pairs than this
  uint32_t group_mul, group_shift;  // division by group
  uint32_t kv_mul, kv_shift;        // division by n_kv
  float scale_log2e;
};

// What becomes of a score z (of scale q . k) before the softmax, in flags of a
// kernel's S, since each costs instructions a score; any S but kAsIs takes a prefix.
//   kCap     cap tanh(z / cap) = cap - 2 cap / (1 + e^(2 z / cap)), off by 2^-20 cap:
//            1 + e, its reciprocal r and e are off by 2^-24, 2^-23 and 2^-23 relative, and r <= 1
//   kWide    (with kCap) for caps past 2^8, where that would be half of what the weights'
//            fp16 rounds: |z| < 0.3 cap by tanh's series up to x^9, all off by 2^-19 relative
//   kBias    then less slope_h |a - j|
// Two prompts of 2048 tokens, 32/16 heads of 128, 8 bits: as they are 115 us, with slopes 113 (154 with the
// keys taken from the first one), capped 136; 48 ragged sequences of single tokens 57, with slopes 59.
enum { kAsIs = 0, kBias = 1, kCap = 2, kWide = 4, kPrefix = 8 };
constexpr float kWideCap = 256.f;
constexpr float kLog2e = 1.4426950408889634f;
template <int S>
struct Shape {
  const float* slopes;      // [n_heads], or null: zeros
  const int32_t* prefixes;  // [n_seq], or null: keys of a sequence that all its tokens see
  float cap;                // cap log2(e): scores are exponents of 2 here
  float twice;              // 2 / cap: what turns z log2(e) into the exponent above
};
template <>
struct Shape<kAsIs> {};

template <int S>
GPTQ_DEV int prefix_of(const Shape<S>& sh, int i, int len) {
  if constexpr (S != kAsIs) {
    if (sh.prefixes) return min(max(sh.prefixes[i], 0), len);
  }
  return 0;
}
template <int S>
GPTQ_DEV float slope_of(const Shape<S>& sh, int head) {
  if constexpr ((S & kBias) != 0) {
    if (sh.slopes) return sh.slopes[head] * kLog2e;
  }
  return 0.f;
}
// The factor of a key's products: its scale, the score's and, before a cap, twice.
// Where a small cap takes a finite scale past fp32, the largest: tanh is 1 there, for products from 2^-122 on.
template <int S>
GPTQ_DEV float key_factor(const Shape<S>& sh, float ks, float scale_log2e) {
  const float v = ks * scale_log2e;
  if constexpr ((S & kCap) != 0) {
    const float w = v * sh.twice;
    return fabsf(w) == __builtin_inff() && fabsf(v) < __builtin_inff() ? copysignf(3.402823466e38f, w) : w;
  }
  return v;
}
// rest + the capped score of a product that has its factor (kCap), or rest + itself; rest
// has cap in it already unless kWide
template <int S>
GPTQ_DEV float capped(const Shape<S>& sh, float product, float factor, float rest) {
  if constexpr ((S & kCap) == 0) return fmaf(product, factor, rest);
  if constexpr ((S & kCap) != 0) {
    const float y = product * factor, r = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(y));
    if constexpr ((S & kWide) == 0) return fmaf(-2.f * sh.cap, r, rest);
    const float x = y * 0.34657359f, x2 = x * x;  // ln 2 / 2
    const float near = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), x);
    return fmaf(sh.cap, fabsf(x) < 0.3f ? near : fmaf(-2.f, r, 1.f), rest);
  }
}
template <int S>
GPTQ_DEV float cap_rest(const Shape<S>& sh) {
  if constexpr ((S & kCap) != 0 && (S & kWide) == 0) return sh.cap;
  return 0.f;
}

struct Seq {
  int q0, n, len, tiles, units;
};

// n / d for 0 <= n < 2^30 by the multiplier and shift of exact_divisor()
GPTQ_DEV int div_by(int n, uint32_t mul, uint32_t shift) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
}

// everything read from the caller's device arrays is clamped, so that no value
// in them makes an access leave its buffer
GPTQ_DEV Seq seq_info(const AttnParams& p, int i) {
  Seq s;
  const int total = static_cast<int>(p.n_tokens);
  const int a = min(max(p.starts[i], 0), total);
  const int b = min(max(p.starts[i + 1], a), total);
  s.q0 = a;
  s.n = b - a;
  s.len = min(max(p.lens[i], 0), p.max_len);
  s.tiles = (s.n * p.group + p.tile_rows - 1) >> p.tile_shift;
  s.units = max((s.len + kUnit - 1) / kUnit, 1);
  return s;
}

// inclusive sums over the wave, in DPP steps (row shifts by 1, 2, 4, 8, then the last lane of a row to
// the next one and of the first two rows to the others); lane 63 has the total
template <int CTRL, int ROWS>
GPTQ_DEV int dpp_or_zero(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
GPTQ_DEV int wave_scan(int v) {
  v += dpp_or_zero<0x111, 0xF>(v);
  v += dpp_or_zero<0x112, 0xF>(v);
  v += dpp_or_zero<0x114, 0xF>(v);
  v += dpp_or_zero<0x118, 0xF>(v);
  v += dpp_or_zero<0x142, 0xA>(v);
  v += dpp_or_zero<0x143, 0xC>(v);
  return v;
}
GPTQ_DEV float wave_scan(float v) {
  v += __int_as_float(dpp_or_zero<0x111, 0xF>(__float_as_int(v)));
  v += __int_as_float(dpp_or_zero<0x112, 0xF>(__float_as_int(v)));
  v += __int_as_float(dpp_or_zero<0x114, 0xF>(__float_as_int(v)));
  v += __int_as_float(dpp_or_zero<0x118, 0xF>(__float_as_int(v)));
  v += __int_as_float(dpp_or_zero<0x142, 0xA>(__float_as_int(v)));
  v += __int_as_float(dpp_or_zero<0x143, 0xC>(__float_as_int(v)));
  return v;
}
GPTQ_DEV float lane_value(float v, int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); }
GPTQ_DEV int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

struct Work {
  Seq s;
  int seq, tile, split, n_split;
  int slot;  // of the unit's first split (for this key head: times n_kv, plus h)
};

// Entry u of the list (SPLITS: of (tile, split) pairs; otherwise of the tiles
// whose keys are split).
// A sequence's keys are split into parts of at least `per` units, per = (all
// units) / target: a batch with enough tiles is not split, a long sequence among
// short ones is.  per is the same fp32 number in every workgroup; being off by
// rounding it only moves where the parts end.
template <bool SPLITS>
GPTQ_DEV bool find_work(const AttnParams& p, int u, Work& w) {
  const int lane = lane_id();
  Seq s{};
  float total = 0.f;
  for (int i0 = 0; i0 < p.n_seq; i0 += 64) {
    s = Seq{0, 0, 0, 0, 1};
    if (i0 + lane < p.n_seq) s = seq_info(p, i0 + lane);
    total += lane_value(wave_scan(static_cast<float>(s.tiles) * static_cast<float>(s.units)), 63);
  }
  const float inv_per = 1.f / fmaxf(total * p.inv_target, total <= p.few ? 2.f : p.min_units);
  int base = 0, slots = 0;
  for (int i0 = 0; i0 < p.n_seq; i0 += 64) {
    if (p.n_seq > 64) {
      s = Seq{0, 0, 0, 0, 1};
      if (i0 + lane < p.n_seq) s = seq_info(p, i0 + lane);
    }
    const int n_split = max(static_cast<int>(ceilf(static_cast<float>(s.units) * inv_per)), 1);
    const int pairs = s.tiles * n_split;
    const int cnt = SPLITS ? pairs : n_split > 1 ? s.tiles : 0;
    const int end = base + wave_scan(cnt);
    const int slot_end = slots + wave_scan(n_split > 1 ? pairs : 0);
    const uint64_t hit = __ballot(u < end);
    if (hit) {
      const int l = uniform(__builtin_ctzll(hit));
      w.seq = i0 + l;
      w.s.q0 = __builtin_amdgcn_readlane(s.q0, l);
      w.s.n = __builtin_amdgcn_readlane(s.n, l);
      w.s.len = __builtin_amdgcn_readlane(s.len, l);
      w.s.tiles = __builtin_amdgcn_readlane(s.tiles, l);
      w.n_split = __builtin_amdgcn_readlane(n_split, l);
      const int local = u - __builtin_amdgcn_readlane(end - cnt, l);
      w.slot = __builtin_amdgcn_readlane(n_split > 1 ? slot_end - pairs : 0, l);
      const int tile = SPLITS ? uniform(local / w.n_split) : local;
      w.split = SPLITS ? local - tile * w.n_split : 0;
      w.tile = SPLITS ? w.s.tiles - 1 - tile : tile;  // the ones that see most keys first
      w.slot += w.tile * w.n_split;
      return local >= 0 && w.tile >= 0;
    }
    base = __builtin_amdgcn_readlane(end, 63);
    slots = __builtin_amdgcn_readlane(slot_end, 63);
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
GPTQ_DEV uint32_t pack_f16(float lo, float hi) {  // v_cvt_pk_f16_f32, nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), f16x2_t));
}
GPTQ_DEV uint32_t pack_bf16(float lo, float hi) {  // v_cvt_pk_bf16_f32, nearest even
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t));
}
GPTQ_DEV float add_f16(uint32_t pair, float c) {  // c + both halves (v_dot2 with ones)
  return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2_t, pair), f16x2_t{1, 1}, c, false);
}

// The power of two that fp16 operands are taken relative to: 2^(e - 126) is
// above x, e its biased exponent (held in 24 .. 252, where the factors below are normal
// fp32 numbers), so x * down() < 2^15.
struct ProductUnit {
  int e;
  GPTQ_DEV float down() const { return __uint_as_float(static_cast<uint32_t>(253 + 15 - e) << 23); }
  GPTQ_DEV float up() const { return __uint_as_float(static_cast<uint32_t>(e + 1 - 15) << 23); }
  static constexpr int kLeast = 24, kMost = 252;
  GPTQ_DEV static int of(float x) {
    return min(max(static_cast<int>((__float_as_uint(x) >> 23) & 255u), kLeast), kMost);
  }
};
GPTQ_DEV float exp2_int(int d) {  // 2^d for d <= 127 (0 below -126; 2^127 above)
  return d < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + min(d, 127)) << 23);
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
// byte B of eight keys' words, in fp16 (exact)
template <int B>
GPTQ_DEV f16x8_t col8(const uint32_t (&w)[8]) {
  const u32x4_t v = {pack_f16(sbyte<B>(w[0]), sbyte<B>(w[1])), pack_f16(sbyte<B>(w[2]), sbyte<B>(w[3])),
                     pack_f16(sbyte<B>(w[4]), sbyte<B>(w[5])), pack_f16(sbyte<B>(w[6]), sbyte<B>(w[7]))};
  return __builtin_bit_cast(f16x8_t, v);
}
// both nibbles of byte B of eight keys' words, as 24 + code in fp16 (16 +
// nibble: 0x4C00 | nibble << 6, exact)
GPTQ_DEV uint32_t nib_pair(uint32_t w0, uint32_t w1, int byte) {
  return __builtin_amdgcn_perm(w1, w0, 0x0C000C00u | ((4u + byte) << 16) | byte);
}
template <int B>
GPTQ_DEV void col4(const uint32_t (&w)[8], f16x8_t& lo, f16x8_t& hi) {
  u32x4_t a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = nib_pair(w[2 * i], w[2 * i + 1], B);
    a[i] = ((t << 6) & 0x03C003C0u) | 0x4C004C00u;
    b[i] = ((t << 2) & 0x03C003C0u) | 0x4C004C00u;
  }
  lo = __builtin_bit_cast(f16x8_t, a);
  hi = __builtin_bit_cast(f16x8_t, b);
}

// ---------------------------------------------------- keys split over waves --
// A workgroup owns 16 MT rows of one (sequence, key head) and one key split;
// its four waves take turns of 32 keys, straight from global memory into the
// operands, and their results meet in LDS at the end.
//
// Scores are computed transposed, S^T = K Q^T (16x16x32): lane l holds key
// l % 16's codes at the HDP / 4 dims of its group g = l / 16, and its results
// are keys 4 g + r (r < 4) for query row l % 16.  Two such tiles (32 keys) are,
// without any exchange between lanes, the P^T operand of O^T = V^T P^T, when
// the sum over keys runs in that order; so lane l reads V at keys 4 g + r and
// 16 + 4 g + r, dims (l % 16) HDP / 16 + t, and byte t of its eight words
// makes the operand of output tile t.  Lane l then ends up with query row
// l % 16, dims g HDP / 4 ... in order.
//
// Bound: HBM, by the loads that fit in flight beside the operands' registers.
// 64 ragged sequences (292 MB of 8-bit keys and values) 56.5 us, 5.2 TB/s; four of
// 131000 keys at 4 bits (570 MB) 118 us, 4.8 TB/s; one of 1000 keys 6.6 us, four
// dependent trips to memory.  Four waves a workgroup and four workgroups a CU:
// eight waves and two took 83 us for the ragged batch.
constexpr int kSplitWaves = 4;

template <int HDP, int BITS, int MT, int S>
__global__ __launch_bounds__(64 * kSplitWaves, HDP <= 128 && MT == 1 ? 4 : 2) void attn_split_kernel(AttnParams p, Shape<S> sh) {
  using K = KeyLanes<HDP, BITS>;
  constexpr int kKW = K::kWords;               // words of K a lane holds per key: HDP / 4 dims
  constexpr int kVB = HDP * BITS / 128;        // bytes of V a lane holds per key: HDP / 16 dims
  constexpr int kVW = (kVB + 3) / 4;
  constexpr int kSteps = HDP / 32;             // products of a 16-key score tile
  constexpr int kTiles = HDP / 16;             // output tiles
  constexpr int kM = 16 * MT, NW = kSplitWaves;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int u = uniform(div_by(static_cast<int>(blockIdx.x), p.kv_mul, p.kv_shift));
  const int h = static_cast<int>(blockIdx.x) - u * p.n_kv;
  Work w;
  if (!find_work<true>(p, u, w)) return;
  const int rows = w.s.n * p.group;
  const int r0 = w.tile * kM;
  const int prefix = uniform(prefix_of<S>(sh, w.seq, w.s.len));
  // last key of the tile's first row, and the keys any of its rows sees
  const int first = max(w.s.len - w.s.n + uniform(div_by(r0, p.group_mul, p.group_shift)), prefix - 1);
  const int vis = max(w.s.len - w.s.n + uniform(div_by(min(r0 + kM, rows) - 1, p.group_mul, p.group_shift)) + 1, prefix);
  const int units = vis > 0 ? (vis - 1) / kUnit + 1 : 0;
  const int per = (units + w.n_split - 1) / w.n_split;
  const int key0 = w.split * per * kUnit, key1 = min(vis, (w.split + 1) * per * kUnit);

  // query operands, their sums (4 bits), and each row's last key
  bf16x8_t q[MT][kSteps];
  float bias[MT], slope[MT];
  int lim[MT], place[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = r0 + 16 * i + c;
    const bool live = r < rows;
    const int tok = live ? div_by(r, p.group_mul, p.group_shift) : 0;
    place[i] = w.s.len - w.s.n + tok;
    lim[i] = live ? max(place[i], prefix - 1) : -1;
    slope[i] = live ? slope_of<S>(sh, h * p.group + r - tok * p.group) : 0.f;
    const uint16_t* src = p.q + static_cast<int64_t>(w.s.q0 + tok) * p.ldq +
                          static_cast<int64_t>(h * p.group + (live ? r - tok * p.group : 0)) * p.hd;
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = K::q_dim(g, s, p.hd);
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (live && d >= 0) v = *reinterpret_cast<const u32x4_t*>(src + d);
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
  ProductUnit unit[MT];    // of acc and psum
  constexpr int kRoom = 6;  // when it is set, the largest product so far becomes 2^8 to 2^9 of it: 2^6 and more below what fits
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = kNoMax;
    l[i] = 0.f;
    psum[i] = 0.f;
    unit[i].e = ProductUnit::kLeast + kRoom;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  const int row_bytes = p.hd * BITS / 8;
  const int page_mask = (1 << p.page_shift) - 1;
  const int32_t* table = p.table + static_cast<int64_t>(w.seq) * p.ld_table;
  constexpr int kKL = K::kLoad;
  using k_vec_t = std::conditional_t<K::kAlign == 16, u32x4_t, u32x4_at8_t>;
  uint32_t koff[K::kLoads], voff;
#pragma unroll
  for (int e = 0; e < K::kLoads; ++e) koff[e] = static_cast<uint32_t>(c * row_bytes + K::begin(g, e, p.hd) * BITS / 8);
  // of V too a lane whose dims lie past head_dim reads the row's first ones: what it gives is not stored
  voff = static_cast<uint32_t>(4 * g * row_bytes + (c * (HDP / 16) < p.hd ? c * kVB : 0));
  // With a bias the keys are taken from the last one: scores fall with the distance, so the maximum is met
  // early, where the other order moves it at every turn.
  constexpr bool kDown = (S & kBias) != 0;
  for (int k0 = kDown ? key0 + ((key1 - 1 - key0) & ~31) - 32 * wave : key0 + 32 * wave; kDown ? k0 >= key0 : k0 < key1;
       k0 += kDown ? -32 * NW : 32 * NW) {
    uint32_t kw[2][kKW], vw[kVW][8];
    f32x4_t ks[2], vs[2];
    bool ok[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int k = k0 + 16 * b;
      const int page = table[min(k, key1 - 1) >> p.page_shift];
      ok[b] = k < key1 && page >= 0 && page < p.n_pages;
      const int64_t row = ((static_cast<int64_t>(ok[b] ? page : 0) * p.n_kv + h) << p.page_shift) + (k & page_mask);
      const uint8_t* kp = p.codes[0] + row * row_bytes;
#pragma unroll
      for (int e = 0; e < K::kLoads; ++e) {
        if (kKL == 4) {
          const u32x4_t v = *reinterpret_cast<const k_vec_t*>(kp + koff[e]);
#pragma unroll
          for (int j = 0; j < 4; ++j) kw[b][(4 * e + j) % kKW] = v[j];
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(kp + koff[e]);
          kw[b][0] = v.x;
          kw[b][1] = v.y;
        }
      }
      const uint8_t* vp = p.codes[1] + row * row_bytes;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint8_t* one = vp + static_cast<uint32_t>(r * row_bytes);
        if (kVB == 2) vw[0][4 * b + r] = *reinterpret_cast<const uint16_t*>(one + voff);
        if (kVB == 4) vw[0][4 * b + r] = *reinterpret_cast<const uint32_t*>(one + voff);
        if (kVB == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(one + voff);
          vw[0][4 * b + r] = v.x;
          vw[kVW - 1][4 * b + r] = v.y;
        }
        if (kVB == 16) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(one + voff);
#pragma unroll
          for (int e = 0; e < 4; ++e) vw[e % kVW][4 * b + r] = v[e];
        }
      }
      ks[b] = (reinterpret_cast<const f32x4_t*>(p.scales[0] + row))[g];
      vs[b] = (reinterpret_cast<const f32x4_t*>(p.scales[1] + row))[g];
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
        for (int r = 0; r < 4; ++r) {
          if constexpr (S == kAsIs) {
            s[i][4 * b + r] = a[r] * (ks[b][r] * p.scale_log2e);
          } else {
            const float away = static_cast<float>(place[i] - (k0 + 16 * b + 4 * g + r));
            const float rest = (S & kBias) ? fmaf(-slope[i], fabsf(away), cap_rest<S>(sh)) : cap_rest<S>(sh);
            s[i][4 * b + r] = capped<S>(sh, a[r], key_factor<S>(sh, ks[b][r], p.scale_log2e), rest);
          }
        }
      }
    }
    float vtop = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) vtop = fmaxf(vtop, fabsf(vs[j >> 2][j & 3]));
    f16x8_t pop[MT];
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
      // m and the unit move when a weight is far above m, or its product with the largest scale would not fit
      if (__any(mx - m[i] > 16.f || fast_exp2(mx - m[i]) * vtop * unit[i].down() > 32768.f)) {
        const float mn = fmaxf(m[i], max_over_groups(mx));
        const float alpha = fast_exp2(m[i] - mn);
        float top = alpha * __uint_as_float(static_cast<uint32_t>(unit[i].e - kRoom) << 23);  // the largest product before
#pragma unroll
        for (int j = 0; j < 8; ++j)  // (a select here costs registers that 8-bit heads of 128 do not have: 69 -> 109 us)
          if (!masked || see[j]) top = fmaxf(top, fabsf(fast_exp2(s[i][j] - mn) * vs[j >> 2][j & 3]));
        const int e = min(ProductUnit::of(max_over_groups(top)) + kRoom, ProductUnit::kMost);
        const float f = alpha * exp2_int(unit[i].e - e);
        m[i] = mn;
        unit[i].e = e;
        l[i] *= alpha;
        psum[i] *= f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][t][r] *= f;
      }
      const float down = unit[i].down();
      float pv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = fast_exp2(s[i][j] - m[i]);
        l[i] += e;
        pv[j] = e * vs[j >> 2][j & 3] * down;
        if (masked && !see[j]) pv[j] = 0.f;  // the scale of a hidden key may be anything
      }
      const u32x4_t pk = {pack_f16(pv[0], pv[1]), pack_f16(pv[2], pv[3]), pack_f16(pv[4], pv[5]), pack_f16(pv[6], pv[7])};
      if (BITS == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) psum[i] = add_f16(pk[e], psum[i]);
      }
      pop[i] = __builtin_bit_cast(f16x8_t, pk);
    }
#pragma unroll
    for (int e = 0; e < kVW; ++e) {
      f16x8_t vop[8];
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
          acc[i][e * kPer + t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vop[t], pop[i], acc[i][e * kPer + t], 0, 0, 0);
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
  const int64_t slot = static_cast<int64_t>(w.slot + w.split) * p.n_kv + h;
  const bool whole = w.n_split == 1;
  if (!whole && static_cast<uint64_t>(slot) >= static_cast<uint64_t>(p.max_slots)) return;  // the whole workgroup
  float* part = p.partial + slot * (kM * (HDP + 2));
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    float top = kNoMax;
#pragma unroll
    for (int v = 0; v < NW; ++v) top = fmaxf(top, wm[v][16 * i + c]);
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) sum += wl[v][16 * i + c] * fast_exp2(wm[v][16 * i + c] - top);
    // divided by the weights' sum before the unit comes off: a mean of values fits where their sum may not
    const float f = fast_exp2(m[i] - top) * (sum == 0.f ? 0.f : 1.f / sum), up = unit[i].up();
    // lane l: dims g HDP / 4 + r HDP / 16 + t
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int t = 0; t < kTiles; t += 4) {
        f32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = f * (acc[i][t + e][r] - (BITS == 4 ? 24.f * psum[i] : 0.f)) * up;
        *reinterpret_cast<f32x4_t*>(&wo[wave][c][g * (HDP / 4) + r * (HDP / 16) + t]) = v;
      }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * HDP / 4; e += 64 * NW) {
      const int row = e / (HDP / 4), d = (e % (HDP / 4)) * 4;
      const int r = r0 + 16 * i + row;
      if (r >= rows || d >= p.hd) continue;  // nor does the join read the others
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
          float t2 = kNoMax, all = 0.f;  // kNoMax: saw nothing
#pragma unroll
          for (int v = 0; v < NW; ++v) t2 = fmaxf(t2, wm[v][16 * i + row]);
#pragma unroll
          for (int v = 0; v < NW; ++v) all += wl[v][16 * i + row] * fast_exp2(wm[v][16 * i + row] - t2);
          part[kM * HDP + 16 * i + row] = t2;
          part[kM * HDP + kM + 16 * i + row] = all;
        }
      } else {
        const int tok = div_by(r, p.group_mul, p.group_shift);
        const uint2 b = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
        *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(w.s.q0 + tok) * p.ldo +
                                  static_cast<int64_t>(h * p.group + r - tok * p.group) * p.hd + d) = b;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------- rows split over waves --
// A workgroup owns 128 rows of one (sequence, key head) and one key split; each
// of its four waves has 32 of the rows, and all walk the keys in tiles of 64.
// (Eight waves of 32 rows, one workgroup a CU, convert half as often but wait
// for each other: 202 us against 205 for four 2048-token prompts of 32 heads, 476
// against 345 for the chunks of 300 to 700 tokens with 64-wide heads.)
//
// Per tile the codes are turned into operands once, into LDS: the key codes
// as bf16 integers, the values as fp16 code * (scale * 2^-range) (two roundings).
// That holds while the scales of the keys so far lie within 2^8 of each other: then
// values stay in fp16's normal range, and a weight is lost (below 2^-33 of the largest) only
// where it and its value are that small against the row's largest.  From the first tile
// that goes past it, values are bare codes (exact) and each weight carries its value's
// scale, in units of the row's own largest product (scaled_tile): a slower path for
// caches whose scales spread wider than those of activations do, or hold zeros (with
// zeros among them the four prompts below take 7% longer, the chunks 35%).
// 32x32x16 products: S^T = K Q^T leaves lane l (query row l % 32, half h = l / 32)
// with keys 8 a + 4 h + b of a 32-key block; 16 of them in that order are the
// P^T operand of O^T = V^T P^T, so V's operand holds keys 4 h + b and 8 + 4 h + b
// of its 16, and P never moves between lanes.  A key operand is 64 lanes of 16
// bytes, stored lane by lane (1040-byte stride: the writers of one operand then
// touch all banks), so its LDS reads are contiguous.
//
// Two tiles of LDS: while one is multiplied, the next one's codes, loaded to
// registers two tiles ahead, are converted into the other; one barrier a tile.
// Weights are taken relative to 2^-8 of the largest, and the row maximum is only moved
// when a lane's weights sum to more than 2^15, which fp16 holds; p keeps its relative
// precision: the usual tile then costs a multiply-add and an exp2 per score, half a
// conversion and half a sum.
//
// Bound: the products, the exponentials and the codes' conversion share the
// waves' issue slots.  Four prompts of 2048 tokens, 32 heads of 128: 205 us (0.67
// PFLOP/s of the causal half; the matrix cores are busy 28% of the cycles of a profiled run); one
// of 16384 tokens 0.86 PFLOP/s.
// A wave with rows past the sequence's last keeps to careful_tile: such rows have no
// maximum (11 sequences of 80 to 160 tokens over 3600 to 18000 keys, 3 heads of 96:
// 80 us; their bytes and products need 11).
constexpr int kFrag = 1040;  // bytes of an operand in LDS
constexpr float kGrow = 32768.f;
constexpr float kAbove = 8.f;    // log2 of the largest weight when the maximum moves
constexpr int kSpread = 8;       // powers of two between the value scales that the plain path takes
constexpr float kFar = 0x1p20f;  // maxima past this leave the plain tile: see careful_tile

// what a thread holds of a tile on its way: its dims of one key or of one value
template <int HDP, int BITS>
struct TileShare {
  static constexpr int kD = HDP / 4;             // dims
  static constexpr int kCD = kD < 16 ? kD : 16;  // dims of one load
  static constexpr int kW = kD * BITS / 32;      // words
  uint32_t w[kW];
};

template <int HDP, int BITS, int S>
__global__ __launch_bounds__(256, HDP <= 64 ? 3 : HDP <= 128 ? 2 : 1) void attn_tile_kernel(AttnParams p, Shape<S> sh) {
  using R = TileShare<HDP, BITS>;
  constexpr int kKeys = 64, kM = 128;
  constexpr int kSteps = HDP / 16, kDb = HDP / 32;
  constexpr int kKF = 2 * kSteps;  // key operands of a tile
  __shared__ __attribute__((aligned(16))) uint8_t lk[2][kKF * kFrag], lv[2][kKeys * HDP * 2];
  __shared__ __attribute__((aligned(16))) float lks[2][kKeys], lvs[2][kKeys];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int c = lane & 31, hf = lane >> 5;
  const int u = uniform(div_by(static_cast<int>(blockIdx.x), p.kv_mul, p.kv_shift));
  const int h = static_cast<int>(blockIdx.x) - u * p.n_kv;
  Work w;
  if (!find_work<true>(p, u, w)) return;
  const int rows = w.s.n * p.group;
  const int r0 = w.tile * kM;
  const int prefix = uniform(prefix_of<S>(sh, w.seq, w.s.len));
  const int vis = max(w.s.len - w.s.n + uniform(div_by(min(r0 + kM, rows) - 1, p.group_mul, p.group_shift)) + 1, prefix);
  const int units = vis > 0 ? (vis - 1) / kUnit + 1 : 0;
  const int per = (units + w.n_split - 1) / w.n_split;
  const int key0 = w.split * per * kUnit, key1 = min(vis, (w.split + 1) * per * kUnit);

  // this wave's rows: their last keys, and the query operand
  const int r = r0 + 32 * wave + c;
  const bool live = r < rows;
  const int tok = live ? div_by(r, p.group_mul, p.group_shift) : 0, qh = live ? r - tok * p.group : 0;
  const int place = w.s.len - w.s.n + tok;
  const int lim = live ? max(place, prefix - 1) : -1;
  const float slope = live ? slope_of<S>(sh, h * p.group + qh) : 0.f;
  const int wplace = w.s.len - w.s.n + uniform(div_by(r0 + 32 * wave, p.group_mul, p.group_shift));  // the wave's first row's
  const int wplast = w.s.len - w.s.n + uniform(div_by(min(r0 + 32 * wave + 32, rows) - 1, p.group_mul, p.group_shift));  // its last one's
  const int wfirst = max(wplace, prefix - 1);  // last key of the first row
  const int wlast = r0 + 32 * wave < rows ? max(wplast, prefix - 1) : -1;
  bf16x8_t q[kSteps];
  float bias = 0.f;
  {
    const uint16_t* src = p.q + static_cast<int64_t>(w.s.q0 + tok) * p.ldq + static_cast<int64_t>(h * p.group + qh) * p.hd;
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = 16 * s + 8 * hf;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (live && d < p.hd) v = *reinterpret_cast<const u32x4_t*>(src + d);
      if (BITS == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += __uint_as_float(v[e] << 16) + __uint_as_float(v[e] & 0xFFFF0000u);
        v = u32x4_t{(v[0] & 0xFFFFu) | (v[2] << 16), (v[0] >> 16) | (v[2] & 0xFFFF0000u),
                    (v[1] & 0xFFFFu) | (v[3] << 16), (v[1] >> 16) | (v[3] & 0xFFFF0000u)};
      }
      q[s] = __builtin_bit_cast(bf16x8_t, v);
    }
    if (BITS == 4) bias = -24.f * (sum + __shfl_xor(sum, 32));
  }

  f32x16_t acc[kDb];
#pragma unroll
  for (int t = 0; t < kDb; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[t][e] = 0.f;
  float m = kNoMax, l = 0.f;
  // largest and least exponents of the value scales so far, the next tile's among them, and whether they lie
  // too far apart; range: the largest that acc is relative to
  int range = ProductUnit::kLeast, top_next = ProductUnit::kLeast, low_next = ProductUnit::kMost;
  float top_bound = 0.f, low_bound = __builtin_inff();  // scales in [low_bound, top_bound) change neither
  bool spread = false;

  const int row_bytes = p.hd * BITS / 8;
  const int page_mask = (1 << p.page_shift) - 1;
  const int32_t* table = p.table + static_cast<int64_t>(w.seq) * p.ld_table;
  // conversion of a tile: wave sg has 16 of its keys, four threads a key, a quarter of
  // the dims of its key and of its value each.  A thread whose dims lie past
  // head_dim reads the row's first ones instead: q is zero there, and what the
  // values give there is not stored.
  const int sg = wave, kkey = lane / 4, kpart = lane % 4;
  const int own = 16 * sg + kkey;  // the thread's key of a tile
  uint32_t coff[R::kD / R::kCD];
#pragma unroll
  for (int i = 0; i < R::kD / R::kCD; ++i) {
    const int d = kpart * R::kD + R::kCD * i;
    coff[i] = static_cast<uint32_t>(kkey * row_bytes + (d < p.hd ? d * BITS / 8 : 0));
  }
  // Values lie in LDS as rows of fp16 (a key's dims side by side) and are read transposed:
  // ds_read_b64_tr_b16 gives each lane of 16 the column of its number of a block of
  // 4 rows x 16 columns, of which each lane names 4 columns of a row.  64-byte
  // block b of row r sits at block b ^ (r & 3) (rows of two blocks: b ^ bit 1 of
  // r) and 16-byte chunk j of it at j ^ (r & 1): four rows of a transposed read
  // and the eight threads of two keys that write at once each touch all banks once.
  auto value_at = [&](int r, int byte) {
    const int b = byte >> 6, j = (byte >> 4) & 3;
    const int bb = HDP == 64 ? b ^ ((r >> 1) & 1) : b ^ (r & 3);
    return r * (HDP * 2) + bb * 64 + ((j ^ (r & 1)) * 16) + (byte & 15);
  };

  // A tile's keys are loaded while the tile two before it is multiplied, its
  // values one tile before; no load is under a condition, so that the loads stay
  // between the products: past the last key the row's last page is read again,
  // and a page that is not there is read as page 0.
  R tk, tv;              // codes: of the next tile's keys until they are converted, then the one's after; of its values
  float ks, vall;        // scales of key `lane` of the keys' tile
  bool vlive;            // that key is there
  int page;              // its page entry, loaded a tile earlier
  uint64_t there;        // the keys of the tile whose page is there
  int64_t vrow = 0;      // the wave's 16 keys of that tile: their first row in the cache
  // Tiles are counted by `base` from key0 on; with a bias (scores fall with the distance) they are taken
  // from the last one, so that the first ones have the maximum.  Past the end the first keys are loaded again.
  const int turn = 2 * key0 + ((key1 - 1 - key0) & ~(kKeys - 1));
  auto keys_of = [&](int base) { return (S & kBias) ? max(turn - base, key0) : base; };
  auto load_page = [&](int base) { page = table[min(keys_of(base) + lane, key1 - 1) >> p.page_shift]; };
  auto load_codes = [&](const uint8_t* src, R& t) {
#pragma unroll
    for (int i = 0; i < R::kD / R::kCD; ++i) {
      constexpr int kWords = R::kCD * BITS / 32;
      if (kWords == 4) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(src + coff[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) t.w[(4 * i + e) % R::kW] = v[e];
      } else if (kWords == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(src + coff[i]);
        t.w[(2 * i) % R::kW] = v.x;
        t.w[(2 * i + 1) % R::kW] = v.y;
      } else {
        t.w[i % R::kW] = *reinterpret_cast<const uint32_t*>(src + coff[i]);
      }
    }
  };
  auto load_keys = [&](int count, R& t) {  // by `page`
    const int base = keys_of(count), key = base + lane;
    const bool ok = key < key1 && page >= 0 && page < p.n_pages;
    there = __ballot(ok);
    const int pg = ok ? page : 0;
    const int64_t all = ((static_cast<int64_t>(pg) * p.n_kv + h) << p.page_shift) + (key & page_mask);
    vlive = ok;
    vall = p.scales[1][all];
    ks = p.scales[0][all];
    const int pw = __builtin_amdgcn_readlane(pg, 16 * sg);
    vrow = ((static_cast<int64_t>(pw) * p.n_kv + h) << p.page_shift) + ((base + 16 * sg) & page_mask);
    load_codes(p.codes[0] + vrow * row_bytes, t);
  };
  auto load_values = [&](R& t) { load_codes(p.codes[1] + vrow * row_bytes, t); };
  // codes in registers -> operands in LDS, in pieces: the range of the tile's
  // value scales, the key scales, 8 dims of the thread's key, 8 of its value
  auto convert_range = [&](float v) {
    if (__any(fabsf(v) >= top_bound || fabsf(v) < low_bound)) {
      int top = v == v ? ProductUnit::of(fabsf(v)) : ProductUnit::kLeast;
      int low = v == v ? top : ProductUnit::kMost;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        top = max(top, __shfl_xor(top, d));
        low = min(low, __shfl_xor(low, d));
      }
      top_next = max(top_next, uniform(top));
      low_next = min(low_next, uniform(low));
      top_bound = __uint_as_float(static_cast<uint32_t>(top_next + 1) << 23);
      low_bound = low_next == ProductUnit::kLeast ? 0.f : __uint_as_float(static_cast<uint32_t>(low_next) << 23);
      spread = top_next - low_next > kSpread;
    }
  };
  // A value whose scale is not finite makes the key's scores NaN (and its operand 0), so that it
  // reaches only the rows that see the key.  Every wave writes the same 64 scales.  Returns the value
  // scale of key `lane`, NaN if there is no such key or scale.
  auto key_scales = [&](int buf) {
    const float nan = __uint_as_float(0x7FC00000u), v = fabsf(vall) < __builtin_inff() ? vall : nan;
    lks[buf][lane] = vlive && v != v ? nan : key_factor<S>(sh, ks, p.scale_log2e);
    return vlive ? v : nan;
  };
  auto convert_key = [&](const R& t, int buf, int i) {
    const int d = kpart * R::kD + 8 * i;
    const bf16x8_t v = BITS == 8 ? row8(t.w[2 * i % R::kW], t.w[(2 * i + 1) % R::kW]) : row4(t.w[i % R::kW]);
    *reinterpret_cast<bf16x8_t*>(&lk[buf][((own >> 5) * kSteps + (d >> 4)) * kFrag + ((own & 31) + 4 * (d & 8)) * 16]) = v;
  };
  // The factor of the thread's value, twice in fp16: under 2^7, so that values and weights of up to 2^8
  // are in ProductUnit's unit together.  Or 1, and the scales go to LDS.
  auto value_factor = [&](float v, int buf) {
    if (spread) {
      lvs[buf][lane] = v == v ? v : 0.f;
      return f16x2_t{1, 1};
    }
    const float f = __shfl(v == v ? v * __uint_as_float(static_cast<uint32_t>(253 + 7 - top_next) << 23) : 0.f, own);
    return __builtin_bit_cast(f16x2_t, pack_f16(f, f));
  };
  auto convert_value = [&](const R& t, f16x2_t f, int buf, int i) {
    u32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f16x2_t code;  // exact
      if (BITS == 8) {
        // 1024 + (code + 128) in fp16 is 0x6400 | (code ^ 0x80)
        const uint32_t w = t.w[(2 * i + (j >> 1)) % R::kW] ^ 0x80808080u;
        code = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, w, (j & 1) ? 0x04030402u : 0x04010400u)) -
               f16x2_t{1152, 1152};
      } else {
        const uint32_t w = t.w[i % R::kW] >> (8 * j);
        code = __builtin_bit_cast(f16x2_t, (w & 0x0Fu) | ((w & 0xF0u) << 12) | 0x64006400u) - f16x2_t{1032, 1032};
      }
      o[j] = __builtin_bit_cast(uint32_t, static_cast<f16x2_t>(code * f));
    }
    *reinterpret_cast<u32x4_t*>(&lv[buf][value_at(own, (kpart * R::kD + 8 * i) * 2)]) = o;
  };

  // products on operand x of a 32-key block b of the tile in `buf`
  auto key_operand = [&](int buf, int b, int x) {
    return *reinterpret_cast<const bf16x8_t*>(&lk[buf][(b * kSteps + x) * kFrag + lane * 16]);
  };
  // x = kDb a + i: keys 32 b + 16 a .., output block i; the lane's address names row 4 hf + s / 4 and
  // columns 16 (group & 1) + 4 (s % 4) of the block, s = lane % 16
  typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
  uint32_t voff[kDb];  // of the first such block; rows of other blocks differ by multiples of 8, which move no swizzle
#pragma unroll
  for (int i = 0; i < kDb; ++i)
    voff[i] = static_cast<uint32_t>(value_at(4 * hf + ((lane & 15) >> 2), 64 * i + ((lane >> 4) & 1) * 32 + 8 * (lane & 3)));
  auto value_operand = [&](int buf, int b, int x) {
    uint8_t* lo = &lv[buf][voff[x % kDb]] + (32 * b + 16 * (x / kDb)) * (HDP * 2);
    uint8_t* hi = lo + 8 * (HDP * 2);
    const s16x4_t u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)lo);
    const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)hi);
    typedef __attribute__((__vector_size__(8 * sizeof(short)))) short s16x8_t;
    return __builtin_bit_cast(f16x8_t, (s16x8_t{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]}));
  };
  constexpr int kPv = 2 * kDb;

  // A tile as it comes: masks, a maximum that moves, a range that grows.  Taken for
  // the first tile of a workgroup, the last ones of causal rows and wherever
  // the plain tile below finds that it does not fit.  half 1: its first 32
  // keys are done already.
  // The plain tile's s sk - m is one multiply-add, whose product is not rounded as
  // m was: off by 2^-24 |m|.  Rows whose maximum lies past +-2^20 (or that have none)
  // stay here, where equal scores give equal weights at any magnitude.
  bool far = true;
  // the scores of a tile's keys (from block `half`), -inf where hidden; returns their maximum
  auto tile_scores = [&](int base, int buf, uint64_t shown, int half, f32x16_t (&s)[2]) {
    const int rel = lim - base - 4 * hf;
    const float away = static_cast<float>(place - base - 4 * hf);
    auto seen = [&](int b, int e) {  // element e of block b: key 32 b + 8 (e / 4) + 4 hf + e % 4
      return 32 * b + 8 * (e >> 2) + (e & 3) <= rel && ((shown >> (32 * b + 16 * (e >> 3))) & 1u);  // 16 keys share a page
    };
    float mx = kNoMax;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (b < half) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e) s[b][e] = bias;
#pragma unroll
      for (int x = 0; x < kSteps; ++x)
        s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_operand(buf, b, x), q[x], s[b], 0, 0, 0);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (b < half) continue;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const f32x4_t ks = *reinterpret_cast<const f32x4_t*>(&lks[buf][32 * b + 8 * a + 4 * hf]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (S == kAsIs) {
            s[b][4 * a + e] *= ks[e];
          } else {
            const float gap = fabsf(away - static_cast<float>(32 * b + 8 * a + e));
            const float rest = (S & kBias) ? fmaf(-slope, gap, cap_rest<S>(sh)) : cap_rest<S>(sh);
            s[b][4 * a + e] = capped<S>(sh, s[b][4 * a + e], ks[e], rest);
          }
          if (!seen(b, 4 * a + e)) s[b][4 * a + e] = kNegInf;
          mx = fmaxf(mx, s[b][4 * a + e]);
        }
      }
    }
    return fmaxf(mx, __shfl_xor(mx, 32));
  };
  auto rescale = [&](float f) {
#pragma unroll
    for (int i = 0; i < kDb; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e] *= f;
  };
  auto careful_tile = [&](int base, int buf, uint64_t shown, int half, int tile_range) {
    f32x16_t s[2];
    const float mx = fmaxf(m, tile_scores(base, buf, shown, half, s) - kAbove);
    const float fm = fast_exp2(m - mx);
    m = mx;
    far = __any(fabsf(m) > kFar);
    l *= fm;
    rescale(fm * exp2_int(range - tile_range));
    range = tile_range;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (b < half) continue;
      u32x4_t pk[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        pk[e >> 2][e & 3] = pack_f16(fast_exp2(s[b][2 * e] - m), fast_exp2(s[b][2 * e + 1] - m));
        l = add_f16(pk[e >> 2][e & 3], l);
      }
#pragma unroll
      for (int x = 0; x < kPv; ++x)
        acc[x % kDb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(value_operand(buf, b, x), __builtin_bit_cast(f16x8_t, pk[x / kDb]),
                                                              acc[x % kDb], 0, 0, 0);
    }
  };
  // A tile whose values are bare codes.  most: the row's largest product of weight and value scale, which
  // gives acc's unit; m here is the maximum itself.
  float most = 0.f;
  auto scaled_tile = [&](int base, int buf, uint64_t shown) {
    f32x16_t s[2];
    const float mx = fmaxf(m, tile_scores(base, buf, shown, 0, s));
    const float fm = fast_exp2(m - mx);
    m = mx;
    l *= fm;
    float top = 0.f;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const f32x4_t vs = *reinterpret_cast<const f32x4_t*>(&lvs[buf][32 * b + 8 * a + 4 * hf]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = fast_exp2(s[b][4 * a + e] - m);
          l += p;
          s[b][4 * a + e] = p * vs[e];
          top = fmaxf(top, fabsf(s[b][4 * a + e]));
        }
      }
    const int before = ProductUnit::of(most);
    most = fmaxf(most * fm, fmaxf(top, __shfl_xor(top, 32)));
    const ProductUnit unit{ProductUnit::of(most)};
    rescale(fm * exp2_int(before - unit.e));
    const float down = unit.down();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      u32x4_t pk[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) pk[e >> 2][e & 3] = pack_f16(s[b][2 * e] * down, s[b][2 * e + 1] * down);
#pragma unroll
      for (int x = 0; x < kPv; ++x)
        acc[x % kDb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(value_operand(buf, b, x), __builtin_bit_cast(f16x8_t, pk[x / kDb]),
                                                              acc[x % kDb], 0, 0, 0);
    }
  };

  uint64_t shown = 0, shown_next = 0;  // `there` of the current tile, and the next one's
  int buf = 0, base = key0;
  float vs_next = 0.f;
  if (key0 < key1) {
    R k0;
    load_page(key0);
    load_keys(key0, k0);
    load_page(key0 + kKeys);
    load_values(tv);
    vs_next = key_scales(0);
    shown = there;
    load_keys(key0 + kKeys, tk);
    load_page(key0 + 2 * kKeys);
    convert_range(vs_next);
    const f16x2_t f = value_factor(vs_next, 0);
#pragma unroll
    for (int i = 0; i < R::kD / 8; ++i) convert_key(k0, 0, i);
#pragma unroll
    for (int i = 0; i < R::kD / 8; ++i) convert_value(tv, f, 0, i);
  }
  auto tile_barrier = [&] {  // a tile's operands are written, and the other buffer's have been read
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };
  // the next tile's keys, and the loads behind them
  auto next_keys = [&] {
    shown_next = there;
    load_values(tv);
    vs_next = key_scales(buf ^ 1);
#pragma unroll
    for (int i = 0; i < R::kD / 8; ++i) convert_key(tk, buf ^ 1, i);
    load_keys(base + 2 * kKeys, tk);
    load_page(base + 3 * kKeys);
  };
  // its values; then it is the current tile
  auto next_values = [&] {
    convert_range(vs_next);
    const f16x2_t f = value_factor(vs_next, buf ^ 1);
#pragma unroll
    for (int i = 0; i < R::kD / 8; ++i) convert_value(tv, f, buf ^ 1, i);
    shown = shown_next;
    base += kKeys;
    buf ^= 1;
  };
  // The next tile is converted past the last one too; nothing reads it then.
  while (base < key1) {
    int half = 0, tile_range = 0;
    bool fits = true, keys_done = false, tile_spread = false;
    while (base < key1) {
      tile_barrier();
      half = 0;
      keys_done = false;
      tile_range = top_next;  // the one this tile's values were written in (the next tile's may be wider)
      tile_spread = spread;
      const int keys = keys_of(base);
      const bool before = keys + kKeys - 1 <= wplace;
      fits = base > key0 && keys + kKeys - 1 <= wfirst && (!(S & kBias) || before || keys >= wplast) && shown == ~uint64_t{0} && tile_range == range && !far && !tile_spread;
      if (!fits) break;
      // The plain tile: every key seen, the maximum and the range as they were.
      // Four groups of products, each with arithmetic between them that does not
      // depend on it, so that the matrix cores run while the wave goes on:
      //   scores of keys 0..31   | next tile's key codes -> operands
      //   scores of keys 32..63  | weights of keys 0..31
      //   output of keys 0..31   | weights of keys 32..63
      //   output of keys 32..63  | next tile's value codes -> operands
      f32x16_t s0, s1;
      u32x4_t pk[4];
      f32x4_t ks[4];
      float l0 = 0.f, l1 = 0.f;
      // The bias of key keys + 4 hf + i for this row, away +- slope i: all keys of a plain tile lie before the
      // places of the wave's rows, or all behind them (kBias).
      const float toward = before ? slope : -slope;
      const float away = toward * static_cast<float>(keys + 4 * hf - place);
      float rest = 0.f;  // of a score, less the maximum
      // log2 of the weight of element e of block b
      auto power = [&](float score, int b, int e) {
        const float f = ks[e >> 2][e & 3];
        if constexpr (S == kAsIs) return fmaf(score, f, -m);
        return capped<S>(sh, score, f, (S & kBias) ? fmaf(toward, static_cast<float>(32 * b + 8 * (e >> 2) + (e & 3)), rest) : rest);
      };
      // n of the 16 weights 2^(s sk - m) of a block, rounded to fp16, and their sum
      auto weights = [&](const f32x16_t& s, int b, int from, int to, float& sum) {
        asm volatile("" : "+v"(m));  // not before this place between the products
        if constexpr (S != kAsIs) rest = cap_rest<S>(sh) + ((S & kBias) ? away : 0.f) - m;
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          if (e >= from && e < to) {
            const uint32_t two = pack_f16(fast_exp2(power(s[e], b, e)), fast_exp2(power(s[e + 1], b, e + 1)));
            pk[2 * b + (e >> 3)][(e >> 1) & 3] = two;
            sum = add_f16(two, sum);
          }
      };
      auto scales_of = [&](int b) {
#pragma unroll
        for (int a = 0; a < 4; ++a) ks[a] = *reinterpret_cast<const f32x4_t*>(&lks[buf][32 * b + 8 * a + 4 * hf]);
      };
      constexpr int kAhead = 2;  // operands read before they are needed
      bf16x8_t ko[kSteps];
      f16x8_t vo[kPv];
#pragma unroll
      for (int e = 0; e < 16; ++e) s0[e] = s1[e] = bias;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) ko[x] = key_operand(buf, 0, x);
      shown_next = there;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < kSteps; ++x) {
        if (x + kAhead < kSteps) ko[x + kAhead] = key_operand(buf, 0, x + kAhead);
        s0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ko[x], q[x], s0, 0, 0, 0);
        if (x == 0) load_values(tv);
        if (x == 1) vs_next = key_scales(buf ^ 1);
        constexpr int kEvery = kSteps / (R::kD / 8);
        if (x % kEvery == kEvery - 1) convert_key(tk, buf ^ 1, x / kEvery);
        __builtin_amdgcn_sched_barrier(0);
      }
      keys_done = true;
      scales_of(0);
#pragma unroll
      for (int x = 0; x < kAhead; ++x) ko[x] = key_operand(buf, 1, x);
#pragma unroll
      for (int x = 0; x < kSteps; ++x) {
        if (x + kAhead < kSteps) ko[x + kAhead] = key_operand(buf, 1, x + kAhead);
        s1 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ko[x], q[x], s1, 0, 0, 0);
        if (x == 0) load_keys(base + 2 * kKeys, tk);
        if (x == 1) load_page(base + 3 * kKeys);
        weights(s0, 0, 16 * x / kSteps, 16 * (x + 1) / kSteps, l0);
        __builtin_amdgcn_sched_barrier(0);
      }
      // a lane's 16 weights sum to more than 2^15: one may be
      fits = !__any(l0 > kGrow);
      if (!fits) break;
      l += l0;
      scales_of(1);
#pragma unroll
      for (int x = 0; x < kAhead; ++x) vo[x] = value_operand(buf, 0, x);
#pragma unroll
      for (int x = 0; x < kPv; ++x) {
        if (x + kAhead < kPv) vo[x + kAhead] = value_operand(buf, 0, x + kAhead);
        acc[x % kDb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vo[x], __builtin_bit_cast(f16x8_t, pk[x / kDb]), acc[x % kDb], 0, 0, 0);
        weights(s1, 1, 16 * x / kPv, 16 * (x + 1) / kPv, l1);
        __builtin_amdgcn_sched_barrier(0);
      }
      half = 1;
      fits = !__any(l1 > kGrow);
      if (!fits) break;
      l += l1;
      convert_range(vs_next);
      const f16x2_t f = value_factor(vs_next, buf ^ 1);
#pragma unroll
      for (int x = 0; x < kAhead; ++x) vo[x] = value_operand(buf, 1, x);
#pragma unroll
      for (int x = 0; x < kPv; ++x) {
        if (x + kAhead < kPv) vo[x + kAhead] = value_operand(buf, 1, x + kAhead);
        acc[x % kDb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vo[x], __builtin_bit_cast(f16x8_t, pk[2 + x / kDb]), acc[x % kDb], 0, 0, 0);
        constexpr int kEvery = kPv / (R::kD / 8);
        if (x % kEvery == kEvery - 1) convert_value(tv, f, buf ^ 1, x / kEvery);
        __builtin_amdgcn_sched_barrier(0);
      }
      shown = shown_next;
      base += kKeys;
      buf ^= 1;
    }
    if (fits || tile_spread) break;
    if (!keys_done) next_keys();
    if (keys_of(base) <= wlast) careful_tile(keys_of(base), buf, shown, half, tile_range);  // else a causal tile past the wave's rows
    next_values();
  }
  // Scaled tiles, from one whose barrier is behind (all waves see the same scales, and come here at the same
  // tile).  From here weights are relative to the largest itself.
  m += kAbove;
  l *= 0x1p-8f;
  most = __uint_as_float(static_cast<uint32_t>(range) << 23);
  while (base < key1) {
    next_keys();
    if (keys_of(base) <= wlast) scaled_tile(keys_of(base), buf, shown);
    next_values();
    if (base < key1) tile_barrier();
  }

  // lane l: query row c, dims 32 i + 8 a + 4 hf + e
  l += __shfl_xor(l, 32);
  const int64_t slot = static_cast<int64_t>(w.slot + w.split) * p.n_kv + h;
  const float up = ProductUnit{ProductUnit::of(most)}.up();
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (!live) return;  // the join does not read such rows either
  if (w.n_split > 1) {
    if (static_cast<uint64_t>(slot) >= static_cast<uint64_t>(p.max_slots)) return;
    float* part = p.partial + slot * (kM * (HDP + 2));
    const int row = 32 * wave + c;
    if (hf == 0) {
      part[kM * HDP + row] = m;
      part[kM * HDP + kM + row] = l;
    }
#pragma unroll
    for (int i = 0; i < kDb; ++i)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        f32x4_t o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = acc[i][4 * a + e] * inv * up;
        *reinterpret_cast<f32x4_t*>(part + row * HDP + 32 * i + 8 * a + 4 * hf) = o;
      }
    return;
  }
  uint16_t* dst = p.out + static_cast<int64_t>(w.s.q0 + tok) * p.ldo + static_cast<int64_t>(h * p.group + qh) * p.hd;
#pragma unroll
  for (int i = 0; i < kDb; ++i)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int d = 32 * i + 8 * a + 4 * hf;
      if (d < p.hd)
        *reinterpret_cast<uint2*>(dst + d) = make_uint2(pack_bf16(acc[i][4 * a] * inv * up, acc[i][4 * a + 1] * inv * up),
                                                        pack_bf16(acc[i][4 * a + 2] * inv * up, acc[i][4 * a + 3] * inv * up));
    }
}

// Joins the splits of a tile, in their order: means of values, by the sums of their
// weights.  One workgroup per (split tile, key head) and 32 rows; the other tiles
// were written by the kernels above.
// Latency of the parts' loads bounds it: eight parts are in flight at a time
// (32 tiles of 25 parts: 7.5 us; 16.4 us one at a time), and a tile of 128 rows
// goes to four workgroups (11 sequences of 80 to 160 rows over 3600 to 18000 keys, 3
// heads: 10.6 us, 32.9 in one; eight workgroups 7.7, but 2 us more where nothing is split).
constexpr int kJoinRows = 32;

template <int HDP>
__global__ __launch_bounds__(512) void attn_join_kernel(AttnParams p) {
  constexpr int kAt = 8;
  const int kM = p.tile_rows;
  const int u = uniform(div_by(static_cast<int>(blockIdx.x), p.kv_mul, p.kv_shift));
  const int h = static_cast<int>(blockIdx.x) - u * p.n_kv;
  Work w;
  if (!find_work<false>(p, u, w)) return;
  const int rows = w.s.n * p.group, r0 = w.tile * kM;
  const int64_t slot0 = static_cast<int64_t>(w.slot) * p.n_kv + h;
  if (slot0 < 0 || slot0 + static_cast<int64_t>(w.n_split - 1) * p.n_kv >= p.max_slots) return;
  const int64_t step = static_cast<int64_t>(p.n_kv) * (kM * (HDP + 2));
  const float* part = p.partial + slot0 * (kM * (HDP + 2));
  const int row0 = static_cast<int>(blockIdx.y) * kJoinRows;
  for (int e = threadIdx.x; e < min(kM, kJoinRows) * HDP / 4; e += 512) {
    const int row = row0 + e / (HDP / 4), d = (e % (HDP / 4)) * 4;
    const int r = r0 + row;
    if (r >= rows || d >= p.hd) continue;
    float top = kNoMax, sum = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < w.n_split; s0 += kAt) {
      float m[kAt], l[kAt], mx = top;
      f32x4_t v[kAt];
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const float* one = part + min(s0 + j, w.n_split - 1) * step;
        m[j] = one[kM * HDP + row];
        l[j] = one[kM * HDP + kM + row];
        v[j] = *reinterpret_cast<const f32x4_t*>(one + row * HDP + d);
      }
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        if (s0 + j >= w.n_split) m[j] = kNegInf;
        mx = fmaxf(mx, m[j]);
      }
      sum *= fast_exp2(top - mx);
      top = mx;
      float all = sum;
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        l[j] = s0 + j < w.n_split ? l[j] * fast_exp2(m[j] - top) : 0.f;  // 0 for a part that saw nothing
        all += l[j];
      }
      const float inv = all == 0.f ? 0.f : 1.f / all, f0 = sum * inv;
      sum = all;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= f0;
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const float f = l[j] * inv;
        if (s0 + j < w.n_split) {
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] += f * v[j][i];
        }
      }
    }
    const int tok = div_by(r, p.group_mul, p.group_shift);
    *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(w.s.q0 + tok) * p.ldo +
                              static_cast<int64_t>(h * p.group + r - tok * p.group) * p.hd + d) =
        make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
  }
}

// (n * mul) >> shift == n / d for 0 <= n < 2^30: mul = ceil(2^(30 + L) / d) with
// 2^L >= d exceeds 2^(30 + L) / d by less than 1, which adds less than
// n / 2^(30 + L) < 1 / d to the quotient
void exact_divisor(int32_t d, uint32_t* mul, uint32_t* shift) {
  uint32_t l = 0;
  while ((int64_t{1} << l) < d) ++l;
  *shift = 30 + l;
  *mul = static_cast<uint32_t>(((uint64_t{1} << (30 + l)) + d - 1) / d);
}

int head_pad(int hd) { return hd <= 64 ? 64 : hd <= 128 ? 128 : 256; }

template <int Q, int S>
Shape<Q> split_shape(const Shape<S>& s) {
  if constexpr (Q == kAsIs) return {};
  else return {s.slopes, s.prefixes, s.cap, s.twice};
}

template <int HDP, int BITS, int S>
void attn_go(const AttnParams& p, const Shape<S>& sh, unsigned blocks, unsigned joins, hipStream_t st) {
  constexpr int t = 64 * kSplitWaves;
  // Slopes of zero cost the split kernel, which waits for memory, no time; the tile kernel has a form of its own without.
  constexpr int Q = S == kAsIs ? kAsIs : (S & ~kPrefix) | kBias;
  const Shape<Q> split = split_shape<Q>(sh);
  if (p.tile_rows == 128) attn_tile_kernel<HDP, BITS, S><<<blocks, 256, 0, st>>>(p, sh);
  else if (HDP <= 128 && p.tile_rows == 32) attn_split_kernel<HDP, BITS, HDP <= 128 ? 2 : 1, Q><<<blocks, t, 0, st>>>(p, split);
  else attn_split_kernel<HDP, BITS, 1, Q><<<blocks, t, 0, st>>>(p, split);
  if (joins) attn_join_kernel<HDP><<<dim3(joins, (p.tile_rows + kJoinRows - 1) / kJoinRows), 512, 0, st>>>(p);
}

template <int S>
void attn_head(const AttnParams& p, const Shape<S>& sh, int bits, unsigned b, unsigned j, hipStream_t st) {
  const int hp = head_pad(p.hd);
  if (bits == 8) {
    if (hp == 64) attn_go<64, 8, S>(p, sh, b, j, st);
    else if (hp == 128) attn_go<128, 8, S>(p, sh, b, j, st);
    else attn_go<256, 8, S>(p, sh, b, j, st);
  } else {
    if (hp == 64) attn_go<64, 4, S>(p, sh, b, j, st);
    else if (hp == 128) attn_go<128, 4, S>(p, sh, b, j, st);
    else attn_go<256, 4, S>(p, sh, b, j, st);
  }
}

}  // namespace

AttnPlan attention_plan(const CacheShape& c, int64_t n_tokens, int32_t n_heads, int32_t n_seq, int64_t ld_table, int n_cu) {
  AttnPlan a{};
  const int64_t group = n_heads / c.n_kv;
  // Rows a sequence, on average: up to 16, one row block, for single tokens; up to
  // 64, two row blocks that share the conversion of the keys (in tiles of 16, 32 and
  // 128, 8 key heads: 32 sequences of 32 rows over 4096 keys 90, 72 and 84 us, of 64
  // rows 133, 103 and 101; but one sequence of 48 rows over 2000 keys 11.5, 15.6 and 19.9).
  // A batch that mixes the two goes by the average: 32 single tokens over 4096 keys
  // with a prompt of 1024 take 135 us, 52 and 40 in two calls; launching both kernels
  // for every batch would cost short prompts two launches that find nothing.
  // Heads wider than 128 have no registers for the second block (256 wide, 16 sequences
  // over 4096 keys: 32 rows 72 us in tiles of 16, 113 in tiles of 128; 64 rows 108 and 117).
  const int64_t per_seq = (n_tokens * group + n_seq - 1) / n_seq;
  a.tile_rows = per_seq > 64 ? 128 : per_seq > 16 && c.hd <= 128 ? 32 : 16;
  // split kernel: a little under the workgroups that fit (four a CU, two for wide
  // heads or two row blocks), so that few are left for a second round
  a.target = a.tile_rows == 16 && c.hd <= 128 ? 3 * n_cu : 2 * n_cu;
  // four units a split, one turn or two of a wave, so that there are few parts to
  // join; two where that gives no CU a second workgroup (one token, 1000 keys, 32
  // key heads: 10.4 us in fours, 9.0 in twos; 8000 keys, 8 key heads: 12.7 and 15.4)
  a.min_units = 4;
  a.few = a.tile_rows == 128 ? 0 : 2 * n_cu / c.n_kv;
  const int64_t tiles = (n_tokens * group) / a.tile_rows + std::min<int64_t>(n_seq, n_tokens);
  a.joins = tiles * c.n_kv;
  a.blocks = a.joins + a.target + 64;  // 64: the split is decided in fp32
  // no sequence can have more units than one split holds: nothing to join
  const int64_t most = (ld_table * c.page + kUnit - 1) / kUnit;
  if (most <= a.min_units) {
    a.joins = 0;
    a.few = 0;
    a.blocks = tiles * c.n_kv;
  } else {
    a.joins = std::min(a.joins, static_cast<int64_t>(a.target) + 64);  // tiles of two parts and more
    a.slots = 2 * static_cast<int64_t>(a.target) + 64;  // a split sequence has fewer than 2 units / per parts
    a.ws_bytes = static_cast<size_t>(a.slots) * a.tile_rows * (head_pad(c.hd) + 2) * 4;
  }
  return a;
}

hipError_t attention_launch(const AttnPlan& plan, const CacheShape& c, const void* q, int64_t ldq, int64_t n_tokens,
                            int32_t n_heads, const void* kc, const void* vc, const float* ks, const float* vs,
                            const int32_t* table, int64_t ld_table, const int32_t* starts, const int32_t* lens,
                            int32_t n_seq, float scale, const AttnShape& shape, void* out, int64_t ldo, void* ws, hipStream_t st) {
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
  p.tile_shift = __builtin_ctz(static_cast<unsigned>(plan.tile_rows));
  p.max_len = static_cast<int32_t>(ld_table * c.page);
  p.inv_target = static_cast<float>(c.n_kv) / static_cast<float>(plan.target);
  p.min_units = static_cast<float>(plan.min_units);
  p.few = static_cast<float>(plan.few);
  exact_divisor(p.group, &p.group_mul, &p.group_shift);
  exact_divisor(p.n_kv, &p.kv_mul, &p.kv_shift);
  p.scale_log2e = scale * 1.4426950408889634f;
  const unsigned b = static_cast<unsigned>(plan.blocks), j = static_cast<unsigned>(plan.joins);
  const double cap = shape.cap;
  auto go = [&](auto flags) {
    constexpr int S = decltype(flags)::value;
    attn_head<S>(p, Shape<S>{shape.slopes, shape.prefixes, static_cast<float>(cap * 1.4426950408889634),
                             static_cast<float>(cap > 0 ? 2.0 / cap : 0.0)}, c.bits, b, j, st);
  };
  if (shape.cap > kWideCap) go(std::integral_constant<int, kCap | kWide | kBias>{});
  else if (shape.cap > 0.f && shape.slopes) go(std::integral_constant<int, kCap | kBias>{});
  else if (shape.cap > 0.f) go(std::integral_constant<int, kCap>{});
  else if (shape.slopes) go(std::integral_constant<int, kBias>{});
  else if (shape.prefixes) go(std::integral_constant<int, kPrefix>{});
  else attn_head<kAsIs>(p, {}, c.bits, b, j, st);
  return hipGetLastError();
}

}  // namespace gptq
