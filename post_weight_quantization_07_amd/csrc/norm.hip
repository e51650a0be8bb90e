// Root-mean-square norm of tokens with the residual's addition, into 8-bit codes
// with a scale per token, into bf16 or into fp32.
//
//   h = x + r,  s = 1 / sqrt(mean h^2 + eps),  y = s (h w)
//   codes of y's row: those of the row u = h w, since s is common to it;
//   scale = s max |u| / 127
// h and u are one fp32 rounding each (h is stored rounded once more to r's type,
// y and the codes come from the fp32 h).  The squares are summed in fp64: fp32
// would lose rows past 2^64 and below 2^-75, and the sum's rounding is then no
// part of the error.  One reduction gives sum h^2 and max |u| together.
#include "gptq_common.h"
#include "gptq_internal.h"
#include "quant_row.h"

#include <algorithm>

namespace gptq {
namespace {

struct NormParams {
  const void* x;
  const void* res;      // null: h = x
  const void* weight;   // null: ones
  void* sum;            // null: h is not kept
  void* y;              // null: codes only
  int8_t* codes;        // null: y only
  float* scales;
  int32_t* sums;        // null: not wanted
  int64_t m, d, ldx, ldr, lds;
  double inv_d, eps;
  int32_t w_bf16, y_bf16;
};

// Eight values of a row, `left` elements before its end, as they lie in memory (16
// bytes of bf16, 32 of fp32; zeros past the end).  Accesses are whole vectors at any
// alignment, which the memory pipe takes; with TAIL (d is no multiple of 8) the
// last ones of a row go element by element (8192 rows of 4100: element by
// element throughout 200 us, so 82).
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef f32x4_t f32x4_any_t __attribute__((aligned(2)));
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2_t;
typedef u32x2_t u32x2_any_t __attribute__((aligned(1)));

template <bool BF16, bool TAIL>
GPTQ_DEV void raw_load(const char* at, int64_t left, u32x4_t (&r)[BF16 ? 1 : 2]) {
#pragma unroll
  for (int j = 0; j < (BF16 ? 1 : 2); ++j) r[j] = u32x4_t{0u, 0u, 0u, 0u};
  if (left >= 8) {
#pragma unroll
    for (int j = 0; j < (BF16 ? 1 : 2); ++j) r[j] = reinterpret_cast<const u32x4_any_t*>(at)[j];
  } else if (TAIL && left > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) {
        if constexpr (BF16) r[0][i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[i]) << (16 * (i & 1));
        else r[i >> 2][i & 3] = reinterpret_cast<const uint32_t*>(at)[i];
      }
  }
}
template <bool BF16>
GPTQ_DEV float raw_value(const u32x4_t (&r)[BF16 ? 1 : 2], int i) {
  if constexpr (BF16) return __uint_as_float((i & 1) ? r[0][i >> 1] & 0xFFFF0000u : r[0][i >> 1] << 16);
  else return __uint_as_float(r[i >> 2][i & 3]);
}
// h = x + r of eight values
template <bool XB, int RES>
GPTQ_DEV void raw_sum(const u32x4_t (&x)[XB ? 1 : 2], const u32x4_t (&r)[RES == 1 ? 1 : 2], float (&h)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = raw_value<XB>(x, i);
    if constexpr (RES != 0) h[i] += raw_value<RES == 1>(r, i);
  }
}
// rounded once for bf16
template <bool TAIL>
GPTQ_DEV void row_store(bool bf16, char* at, int64_t left, const float (&v)[8]) {
  if (left >= 8) {
    if (bf16) {
      const auto two = [&](int i) { return f32_to_bf16(v[i]) | (static_cast<uint32_t>(f32_to_bf16(v[i + 1])) << 16); };
      *reinterpret_cast<u32x4_any_t*>(at) = u32x4_t{two(0), two(2), two(4), two(6)};
    } else {
      reinterpret_cast<f32x4_any_t*>(at)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
      reinterpret_cast<f32x4_any_t*>(at)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    }
  } else if (TAIL && left > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) {
        if (bf16) reinterpret_cast<uint16_t*>(at)[i] = f32_to_bf16(v[i]);
        else reinterpret_cast<float*>(at)[i] = v[i];
      }
  }
}
// their codes; returns the codes' sum (those past the end are 0)
template <bool TAIL>
GPTQ_DEV int code_store(int8_t* at, int64_t left, const float (&v)[8], const RowScale& rs) {
  if (left <= 0) return 0;
  uint32_t w[2];
  row_codes<127, 0>(v, rs, w);
  if (!TAIL || left >= 8) {
    *reinterpret_cast<u32x2_any_t*>(at) = u32x2_t{w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) at[i] = static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
  return __builtin_amdgcn_sdot4(w[0], 0x01010101, __builtin_amdgcn_sdot4(w[1], 0x01010101, 0, false), false);
}
// eight weights (ones without any)
template <bool TAIL>
GPTQ_DEV void load_weight(const NormParams& p, int64_t e, float (&w)[8]) {
  const int64_t left = p.d - e;
  if (!p.weight) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  } else if (p.w_bf16) {
    u32x4_t r[1];
    raw_load<true, TAIL>(static_cast<const char*>(p.weight) + e * 2, left, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = raw_value<true>(r, i);
  } else {
    u32x4_t r[2];
    raw_load<false, TAIL>(static_cast<const char*>(p.weight) + e * 4, left, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = raw_value<false>(r, i);
  }
}

GPTQ_DEV double wave_sum(double v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
  return v;
}

// A row's factor s = 1 / sqrt(mean h^2 + eps), in two: below fp32's normal range (rows past 2^126) it would keep
// fewer bits, so that it is held times 2^64 there, and what it multiplies times 2^-64 first (exact, or of a product
// that vanishes).
struct RowFactor {
  float s, first;
};
GPTQ_DEV RowFactor row_factor(double mean_and_eps) {
  const double s = rsqrt(mean_and_eps);
  const bool small = s < 0x1p-126;
  return {static_cast<float>(small ? s * 0x1p64 : s), small ? 0x1p-64f : 1.0f};
}
GPTQ_DEV float row_times(const RowFactor& f, float u) { return u * f.first * f.s; }
// eight of them, the first factor only where it is one
GPTQ_DEV void row_times(const RowFactor& f, float (&u)[8]) {
  if (f.first != 1.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] *= f.first;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] *= f.s;
}

// T threads per row (T = 64: four rows a workgroup), up to 8 CH T values of it in
// registers between the sum and the store.  A workgroup walks over rows: the weight
// is loaded once, and with AHEAD the next row's loads go out before this row's
// reduction.  What a thread reads of a row it alone writes, so that h may be stored over
// x or the residual.  Bound: HBM: 16384 rows of 4096 (bf16, residual, codes) 93 us or 5.0 TB/s
// of a large copy's 5.2 (113 with a workgroup a row), 32768 of 512 23 us (41), 777 of 5120 in
// fp32 13.7 us; one row 4 us of kernel.
template <int T, int CH, bool XB, int RES, bool TAIL, bool AHEAD>  // RES: 0 none, 1 bf16, 2 fp32
__global__ __launch_bounds__(T == 64 ? 256 : T) void norm_kernel(NormParams p) {
  constexpr int kRows = (T == 64) ? 4 : 1;
  constexpr int kWaves = T / 64;
  constexpr bool kOne = kWaves == 1;
  constexpr int kX = XB ? 2 : 4, kR = RES == 1 ? 2 : 4;  // bytes of an element
  const int t = (T == 64) ? (threadIdx.x & 63) : threadIdx.x;
  const int wave = threadIdx.x >> 6;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows + ((T == 64) ? wave : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  __shared__ double red[2][kWaves];
  __shared__ uint32_t redmax[2][kWaves];
  __shared__ int redsum[2][kWaves];
  auto at = [&](int c) { return (static_cast<int64_t>(c) * T + t) * 8; };
  float w[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) load_weight<TAIL>(p, at(c), w[c]);
  u32x4_t xr[CH][XB ? 1 : 2], rr[CH][RES == 1 ? 1 : 2];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t left = row < p.m ? p.d - at(c) : 0;
      raw_load<XB, TAIL>(static_cast<const char*>(p.x) + (row * p.ldx + at(c)) * kX, left, xr[c]);
      if constexpr (RES != 0) raw_load<RES == 1, TAIL>(static_cast<const char*>(p.res) + (row * p.ldr + at(c)) * kR, left, rr[c]);
    }
  };
  if (AHEAD) fetch(first);
  int turn = 0;
  int64_t before = -1;  // the row whose code sum is not stored yet (several waves)
  // every wave of a workgroup makes the same turns: with one wave a row there is no barrier
  for (int64_t row = first; row < p.m; row += step, turn ^= 1) {
    float h[CH][8];
    if (!AHEAD) fetch(row);
#pragma unroll
    for (int c = 0; c < CH; ++c) raw_sum<XB, RES>(xr[c], rr[c], h[c]);
    if (AHEAD) fetch(row + step);
    double ss = 0.0;
    uint32_t am = 0u;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fma(static_cast<double>(h[c][i]), static_cast<double>(h[c][i]), ss);
        am = max(am, abs_bits(h[c][i] * w[c][i]));
      }
    ss = wave_sum(ss);
    am = group_max<64>(am);
    if (!kOne) {
      if ((threadIdx.x & 63) == 0) {
        red[turn][wave] = ss;
        redmax[turn][wave] = am;
      }
      __syncthreads();  // the last row's code sums are there too
      ss = 0.0;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        ss += red[turn][v];
        am = max(am, redmax[turn][v]);
      }
      if (p.sums && before >= 0 && threadIdx.x == 0) {
        int all = 0;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) all += redsum[turn ^ 1][v];
        p.sums[before] = all;
      }
    }
    const RowFactor factor = row_factor(fma(ss, p.inv_d, p.eps));
    RowScale rs = row_scale(am, 127.f);
    if (am < 0x7F800000u) rs.scale = __fdiv_rn(row_times(factor, __uint_as_float(am)), 127.f);
    int sum = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t e = at(c), left = p.d - e;
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = h[c][i] * w[c][i];
      if (RES && p.sum) row_store<TAIL>(RES == 1, static_cast<char*>(p.sum) + (row * p.lds + e) * kR, left, h[c]);
      if (p.codes) sum += code_store<TAIL>(p.codes + row * p.d + e, left, u, rs);
      if (p.y) {
        row_times(factor, u);
        row_store<TAIL>(p.y_bf16 != 0, static_cast<char*>(p.y) + (row * p.d + e) * (p.y_bf16 ? 2 : 4), left, u);
      }
    }
    if (!p.codes) continue;
    if (t == 0) p.scales[row] = rs.scale;
    if (p.sums) {
      sum = group_sum<64>(sum);
      if (kOne) {
        if (t == 0) p.sums[row] = sum;
      } else if ((threadIdx.x & 63) == 0) {
        redsum[turn][wave] = sum;
      }
      before = row;
    }
  }
  if (!kOne && p.codes && p.sums && before >= 0) {
    __syncthreads();
    if (threadIdx.x == 0) {
      int all = 0;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) all += redsum[turn ^ 1][v];
      p.sums[before] = all;
    }
  }
}

// Rows too long to hold, one a workgroup, read twice, the second time from the caches (2048 rows of
// 28672, bf16, residual, codes: 101 us, 4.1 TB/s).
constexpr int kLongT = 1024;
template <bool XB, int RES, bool TAIL>
__global__ __launch_bounds__(kLongT) void norm_long_kernel(NormParams p) {
  constexpr int kWaves = kLongT / 64;
  constexpr int kX = XB ? 2 : 4, kR = RES == 1 ? 2 : 4;
  __shared__ double red[kWaves];
  __shared__ uint32_t redmax[kWaves];
  __shared__ int redsum[kWaves];
  const int64_t row = blockIdx.x;
  const int wave = threadIdx.x >> 6;
  auto load = [&](int64_t e, float (&h)[8], float (&w)[8]) {
    u32x4_t x[XB ? 1 : 2], r[RES == 1 ? 1 : 2];
    raw_load<XB, TAIL>(static_cast<const char*>(p.x) + (row * p.ldx + e) * kX, p.d - e, x);
    if constexpr (RES != 0) raw_load<RES == 1, TAIL>(static_cast<const char*>(p.res) + (row * p.ldr + e) * kR, p.d - e, r);
    raw_sum<XB, RES>(x, r, h);
    load_weight<TAIL>(p, e, w);
  };
  float h[8], w[8];
  double ss = 0.0;
  uint32_t am = 0u;
  for (int64_t e = static_cast<int64_t>(threadIdx.x) * 8; e < p.d; e += kLongT * 8) {
    load(e, h, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss = fma(static_cast<double>(h[i]), static_cast<double>(h[i]), ss);
      am = max(am, abs_bits(h[i] * w[i]));
    }
  }
  ss = wave_sum(ss);
  am = group_max<64>(am);
  if ((threadIdx.x & 63) == 0) {
    red[wave] = ss;
    redmax[wave] = am;
  }
  __syncthreads();
  ss = 0.0;
  for (int v = 0; v < kWaves; ++v) {
    ss += red[v];
    am = max(am, redmax[v]);
  }
  const RowFactor factor = row_factor(fma(ss, p.inv_d, p.eps));
  RowScale rs = row_scale(am, 127.f);
  if (am < 0x7F800000u) rs.scale = __fdiv_rn(row_times(factor, __uint_as_float(am)), 127.f);
  int sum = 0;
  for (int64_t e = static_cast<int64_t>(threadIdx.x) * 8; e < p.d; e += kLongT * 8) {
    load(e, h, w);
    if (RES && p.sum) row_store<TAIL>(RES == 1, static_cast<char*>(p.sum) + (row * p.lds + e) * kR, p.d - e, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] *= w[i];
    if (p.codes) sum += code_store<TAIL>(p.codes + row * p.d + e, p.d - e, h, rs);
    if (p.y) {
      row_times(factor, h);
      row_store<TAIL>(p.y_bf16 != 0, static_cast<char*>(p.y) + (row * p.d + e) * (p.y_bf16 ? 2 : 4), p.d - e, h);
    }
  }
  if (!p.codes) return;
  sum = group_sum<64>(sum);
  if ((threadIdx.x & 63) == 0) redsum[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    p.scales[row] = rs.scale;
    sum = 0;
    for (int v = 0; v < kWaves; ++v) sum += redsum[v];
    if (p.sums) p.sums[row] = sum;
  }
}

template <bool XB, int RES>
void norm_size(const NormParams& p, int n_cu, hipStream_t st) {
  // up to eight workgroups a CU, as many as its wave slots hold at 256 threads, each over its share of the rows
  const int64_t room = 8ll * n_cu;
  const unsigned small = static_cast<unsigned>(std::min((p.m + 3) / 4, room)), wide = static_cast<unsigned>(std::min(p.m, room));
  if (p.d % 8 == 0) {
    if (p.d <= 512) norm_kernel<64, 1, XB, RES, false, true><<<small, 256, 0, st>>>(p);
    else if (p.d <= 1024) norm_kernel<64, 2, XB, RES, false, true><<<small, 256, 0, st>>>(p);
    else if (p.d <= 2048) norm_kernel<256, 1, XB, RES, false, true><<<wide, 256, 0, st>>>(p);
    else if (p.d <= 4096) norm_kernel<256, 2, XB, RES, false, true><<<wide, 256, 0, st>>>(p);
    else if (p.d <= 6144) norm_kernel<256, 3, XB, RES, false, true><<<wide, 256, 0, st>>>(p);
    else if (p.d <= 8192) norm_kernel<512, 2, XB, RES, false, true><<<wide, 512, 0, st>>>(p);
    else if (p.d <= 16384) norm_kernel<512, 4, XB, RES, false, false><<<wide, 512, 0, st>>>(p);
    else norm_long_kernel<XB, RES, false><<<static_cast<unsigned>(p.m), kLongT, 0, st>>>(p);
  } else {
    if (p.d <= 1024) norm_kernel<64, 2, XB, RES, true, true><<<small, 256, 0, st>>>(p);
    else if (p.d <= 4096) norm_kernel<256, 2, XB, RES, true, true><<<wide, 256, 0, st>>>(p);
    else if (p.d <= 8192) norm_kernel<512, 2, XB, RES, true, true><<<wide, 512, 0, st>>>(p);
    else if (p.d <= 16384) norm_kernel<512, 4, XB, RES, true, false><<<wide, 512, 0, st>>>(p);
    else norm_long_kernel<XB, RES, true><<<static_cast<unsigned>(p.m), kLongT, 0, st>>>(p);
  }
}

}  // namespace

hipError_t norm_launch(const NormCall& c, int n_cu, hipStream_t st) {
  NormParams p{};
  p.weight = c.weight;
  p.w_bf16 = c.w_bf16;
  p.y_bf16 = c.y_bf16;
  p.d = c.d;
  p.ldx = c.ldx;
  p.ldr = c.ldr;
  p.lds = c.lds;
  p.inv_d = 1.0 / static_cast<double>(c.d);
  p.eps = c.eps;
  const int res = !c.res ? 0 : c.res_bf16 ? 1 : 2;
  constexpr int64_t kMost = int64_t{1} << 21;  // rows of a launch, which has fewer than 2^32 threads
  for (int64_t r = 0; r < c.m; r += kMost) {
    p.m = std::min(c.m - r, kMost);
    p.x = static_cast<const char*>(c.x) + r * c.ldx * (c.x_bf16 ? 2 : 4);
    if (c.res) p.res = static_cast<const char*>(c.res) + r * c.ldr * (c.res_bf16 ? 2 : 4);
    if (c.sum) p.sum = static_cast<char*>(c.sum) + r * c.lds * (c.res_bf16 ? 2 : 4);
    if (c.y) p.y = static_cast<char*>(c.y) + r * c.d * (c.y_bf16 ? 2 : 4);
    if (c.codes) {
      p.codes = c.codes + r * c.d;
      p.scales = c.scales + r;
      if (c.sums) p.sums = c.sums + r;
    }
    if (c.x_bf16) {
      if (res == 0) norm_size<true, 0>(p, n_cu, st);
      else if (res == 1) norm_size<true, 1>(p, n_cu, st);
      else norm_size<true, 2>(p, n_cu, st);
    } else {
      if (res == 0) norm_size<false, 0>(p, n_cu, st);
      else if (res == 1) norm_size<false, 1>(p, n_cu, st);
      else norm_size<false, 2>(p, n_cu, st);
    }
  }
  return hipGetLastError();
}

}  // namespace gptq
