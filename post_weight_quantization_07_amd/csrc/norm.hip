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

template <bool VEC>
GPTQ_DEV void row_load(bool bf16, const void* base, int64_t row0, int64_t e, int64_t d, float (&v)[8]) {
  if (bf16) tok_load<true, VEC>(base, row0, e, d, v);
  else tok_load<false, VEC>(base, row0, e, d, v);
}

// eight values of a row, rounded once for bf16
template <bool VEC>
GPTQ_DEV void row_store(bool bf16, void* base, int64_t row0, int64_t e, int64_t d, const float (&v)[8]) {
  if (e >= d) return;
  if (bf16) {
    uint16_t* to = static_cast<uint16_t*>(base) + row0 + e;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
    if (VEC) {
      *reinterpret_cast<u32x4_t*>(to) = u32x4_t{w[0], w[1], w[2], w[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < d) to[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float* to = static_cast<float*>(base) + row0 + e;
    if (VEC) {
      reinterpret_cast<f32x4_t*>(to)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
      reinterpret_cast<f32x4_t*>(to)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < d) to[i] = v[i];
    }
  }
}

GPTQ_DEV double wave_sum(double v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
  return v;
}

// T threads per row (T = 64: four rows a workgroup); h of a row of up to 8 CH T
// values stays in registers between the sum and the store.  Longer rows are
// read again; what a thread reads then is what it alone writes, so that h may
// be stored over x or the residual.  Bound: HBM.
template <int T, int CH, bool XB, int RES, bool VEC>  // RES: 0 none, 1 bf16, 2 fp32
__global__ __launch_bounds__(T == 64 ? 256 : T) void norm_kernel(NormParams p) {
  constexpr int kRows = (T == 64) ? 4 : 1;
  constexpr int kWaves = T / 64;
  const int t = (T == 64) ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + ((T == 64) ? (threadIdx.x >> 6) : 0);
  if (row >= p.m) return;  // T == 64: whole waves, and there is no barrier below
  const bool held = p.d <= static_cast<int64_t>(T) * 8 * CH;
  auto load_h = [&](int64_t e, float (&h)[8]) {
    row_load<VEC>(XB, p.x, row * p.ldx, e, p.d, h);
    if (RES) {
      float r[8];
      row_load<VEC>(RES == 1, p.res, row * p.ldr, e, p.d, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] += r[i];
    }
  };
  auto load_w = [&](int64_t e, float (&w)[8]) {
    if (p.weight) {
      row_load<VEC>(p.w_bf16 != 0, p.weight, 0, e, p.d, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.f;
    }
  };
  double ss = 0.0;
  uint32_t am = 0u;
  auto gather = [&](const float (&h)[8], const float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss = fma(static_cast<double>(h[i]), static_cast<double>(h[i]), ss);
      am = max(am, abs_bits(h[i] * w[i]));
    }
  };
  float h[CH][8], w[CH][8];
  if (held) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t e = (static_cast<int64_t>(c) * T + t) * 8;
      load_h(e, h[c]);
      load_w(e, w[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) gather(h[c], w[c]);
  } else {
    for (int64_t e = static_cast<int64_t>(t) * 8; e < p.d; e += T * 8) {
      load_h(e, h[0]);
      load_w(e, w[0]);
      gather(h[0], w[0]);
    }
  }
  ss = wave_sum(ss);
  am = group_max<64>(am);
  __shared__ double red[kWaves];
  __shared__ uint32_t redmax[kWaves];
  __shared__ int redsum[kWaves];
  if (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) {
      red[threadIdx.x >> 6] = ss;
      redmax[threadIdx.x >> 6] = am;
    }
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      ss += red[v];
      am = max(am, redmax[v]);
    }
  }
  const float rstd = static_cast<float>(rsqrt(fma(ss, p.inv_d, p.eps)));
  RowScale rs = row_scale(am, 127.f);
  if (am < 0x7F800000u) rs.scale = __fdiv_rn(__uint_as_float(am) * rstd, 127.f);
  int sum = 0;
  auto put = [&](int64_t e, const float (&hv)[8], const float (&wv)[8]) {
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = hv[i] * wv[i];
    if (RES && p.sum) row_store<VEC>(RES == 1, p.sum, row * p.lds, e, p.d, hv);
    if (p.codes) sum += tok_store<VEC>(p.codes, row * p.d, e, p.d, u, rs);
    if (p.y) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] *= rstd;
      row_store<VEC>(p.y_bf16 != 0, p.y, row * p.d, e, p.d, u);
    }
  };
  if (held) {
#pragma unroll
    for (int c = 0; c < CH; ++c) put((static_cast<int64_t>(c) * T + t) * 8, h[c], w[c]);
  } else {
    for (int64_t e = static_cast<int64_t>(t) * 8; e < p.d; e += T * 8) {
      load_h(e, h[0]);
      load_w(e, w[0]);
      put(e, h[0], w[0]);
    }
  }
  if (!p.codes) return;
  if (p.sums) {
    sum = group_sum<64>(sum);
    if (kWaves > 1) {
      if ((threadIdx.x & 63) == 0) redsum[threadIdx.x >> 6] = sum;
      __syncthreads();
      sum = 0;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) sum += redsum[v];
    }
  }
  if (t == 0) {
    p.scales[row] = rs.scale;
    if (p.sums) p.sums[row] = sum;
  }
}

template <int T, int CH, bool XB, int RES>
void norm_vec(const NormParams& p, bool vec, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(T == 64 ? (p.m + 3) / 4 : p.m));
  constexpr int b = T == 64 ? 256 : T;
  if (vec) norm_kernel<T, CH, XB, RES, true><<<grid, b, 0, st>>>(p);
  else norm_kernel<T, CH, XB, RES, false><<<grid, b, 0, st>>>(p);
}

template <int T, int CH>
void norm_go(const NormParams& p, bool x_bf16, int res, bool vec, hipStream_t st) {
  if (x_bf16) {
    if (res == 0) norm_vec<T, CH, true, 0>(p, vec, st);
    else if (res == 1) norm_vec<T, CH, true, 1>(p, vec, st);
    else norm_vec<T, CH, true, 2>(p, vec, st);
  } else {
    if (res == 0) norm_vec<T, CH, false, 0>(p, vec, st);
    else if (res == 1) norm_vec<T, CH, false, 1>(p, vec, st);
    else norm_vec<T, CH, false, 2>(p, vec, st);
  }
}

bool whole(const void* p, int64_t ld, bool bf16) {  // rows begin 16-byte aligned
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % (bf16 ? 8 : 4) == 0;
}

}  // namespace

hipError_t norm_launch(const NormCall& c, hipStream_t st) {
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
  const bool vec = c.d % 8 == 0 && whole(c.x, c.ldx, c.x_bf16) && (!c.res || whole(c.res, c.ldr, c.res_bf16)) &&
                   (!c.sum || whole(c.sum, c.lds, c.res_bf16)) && whole(c.weight, 0, c.w_bf16) && whole(c.y, 0, c.y_bf16) &&
                   (reinterpret_cast<uintptr_t>(c.codes) & 7u) == 0;
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
    if (c.d <= 2048) norm_go<64, 4>(p, c.x_bf16, res, vec, st);
    else if (c.d <= 8192) norm_go<256, 4>(p, c.x_bf16, res, vec, st);
    else if (c.d <= 16384) norm_go<512, 4>(p, c.x_bf16, res, vec, st);
    else norm_go<1024, 4>(p, c.x_bf16, res, vec, st);
  }
  return hipGetLastError();
}

}  // namespace gptq
