// Product of a quantized layer in 8-bit integers: a scale per token for the
// activations and a scale per output channel for the weights.
//
//   y[t, n] = sx[t] sw[n] (sum_k cx[t, k] cw[n, k] - off[n] sum_k cx[t, k])
//
// cx are the codes of x's rows (quant_row.h), cw the layer's codes shifted
// into int8, off its zero points shifted the same way (absent: symmetric).
// Every sum is a 32-bit integer and exact: d_in <= 65536 keeps both below
// 2^30 in magnitude and their difference below 2^31.  The only roundings are the
// conversion of the sum to fp32, the two scales and the store.
#include "gptq_common.h"
#include "gptq_internal.h"
#include "quant_row.h"

#include <algorithm>
#include <cmath>

namespace gptq {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4_t;
typedef __attribute__((__vector_size__(16 * sizeof(int)))) int i32x16_t;
typedef __attribute__((address_space(3))) void lds_void_t;

// ------------------------------------------------------------ token codes --
// T threads per row (T = 64: four rows a workgroup), a row of up to 8 CH T
// values in registers between the maximum and the codes, so x is read once;
// longer rows are read a second time (from the caches).  VEC: rows are
// 16-byte aligned and d a multiple of 8.  Bound: HBM (x read, codes written):
// 2048 x 28672 bf16 in 42 us, 4.2 TB/s; 509 x 11008 fp32, all of it in flight at
// once, 7.9 us; 16 x 4096 4.2 us, a launch and one trip to HBM.
template <int T, int CH, bool BF16, bool VEC>
__global__ __launch_bounds__(T == 64 ? 256 : T) void token_codes_kernel(const void* __restrict__ x, int64_t m, int64_t d,
                                                                        int64_t ldx, int8_t* __restrict__ codes,
                                                                        float* __restrict__ scales,
                                                                        int32_t* __restrict__ sums) {
  constexpr int kRows = (T == 64) ? 4 : 1;
  constexpr int kWaves = T / 64;
  const int t = (T == 64) ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + ((T == 64) ? (threadIdx.x >> 6) : 0);
  if (row >= m) return;  // T == 64: whole waves, and there is no barrier below
  const int64_t x0 = row * ldx, c0 = row * d;
  const bool held = d <= static_cast<int64_t>(T) * 8 * CH;
  float v[CH][8];
  uint32_t am = 0u;
  if (held) {
#pragma unroll
    for (int c = 0; c < CH; ++c) tok_load<BF16, VEC>(x, x0, (static_cast<int64_t>(c) * T + t) * 8, d, v[c]);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) am = max(am, abs_bits(v[c][i]));
  } else {
    for (int64_t e = static_cast<int64_t>(t) * 8; e < d; e += T * 8) {
      tok_load<BF16, VEC>(x, x0, e, d, v[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) am = max(am, abs_bits(v[0][i]));
    }
  }
  am = group_max<64>(am);
  __shared__ uint32_t red[kWaves];
  __shared__ int redsum[kWaves];
  if (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = am;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) am = max(am, red[w]);
  }
  const RowScale rs = row_scale(am, 127.f);
  int sum = 0;
  if (held) {
#pragma unroll
    for (int c = 0; c < CH; ++c) sum += tok_store<VEC>(codes, c0, (static_cast<int64_t>(c) * T + t) * 8, d, v[c], rs);
  } else {
    for (int64_t e = static_cast<int64_t>(t) * 8; e < d; e += T * 8) {
      tok_load<BF16, VEC>(x, x0, e, d, v[0]);
      sum += tok_store<VEC>(codes, c0, e, d, v[0], rs);
    }
  }
  if (sums) {
    sum = group_sum<64>(sum);
    if (kWaves > 1) {
      if ((threadIdx.x & 63) == 0) redsum[threadIdx.x >> 6] = sum;
      __syncthreads();
      sum = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += redsum[w];
    }
  }
  if (t == 0) {
    scales[row] = rs.scale;
    if (sums) sums[row] = sum;
  }
}

template <int T, int CH>
void token_codes_go(const void* x, bool bf16, bool vec, int64_t m, int64_t d, int64_t ldx, int8_t* codes, float* scales,
                    int32_t* sums, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(T == 64 ? (m + 3) / 4 : m));
  const int b = T == 64 ? 256 : T;
  if (bf16 && vec) token_codes_kernel<T, CH, true, true><<<grid, b, 0, st>>>(x, m, d, ldx, codes, scales, sums);
  else if (bf16) token_codes_kernel<T, CH, true, false><<<grid, b, 0, st>>>(x, m, d, ldx, codes, scales, sums);
  else if (vec) token_codes_kernel<T, CH, false, true><<<grid, b, 0, st>>>(x, m, d, ldx, codes, scales, sums);
  else token_codes_kernel<T, CH, false, false><<<grid, b, 0, st>>>(x, m, d, ldx, codes, scales, sums);
}

// ---------------------------------------------------------- layer layout --
// qweight words (gptq_pack's code stream) of a layer with one group per output
// channel -> int8 rows.  One thread per (output row, 32 codes); a one-time step.
__global__ __launch_bounds__(256) void integer_weight_kernel(const int32_t* __restrict__ qweight,
                                                             const int32_t* __restrict__ zeros, int bits, int64_t d_in,
                                                             int64_t d_out, int8_t* __restrict__ w,
                                                             int32_t* __restrict__ offsets) {
  const int64_t n = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (n >= d_out) return;
  const int mid = 1 << (bits - 1);
  const uint32_t mask = (1u << bits) - 1u;
  for (int64_t run = blockIdx.y; run < d_in / 32; run += gridDim.y) {
    uint32_t in[8], out[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) in[k] = (k < bits) ? static_cast<uint32_t>(qweight[(run * bits + k) * d_out + n]) : 0u;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      out[q] = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int bit = bits * (4 * q + k), wi = bit >> 5, off = bit & 31;
        uint64_t two = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j == wi) two = in[j] | (static_cast<uint64_t>(j + 1 < 8 ? in[j + 1] : 0u) << 32);
        const int c = static_cast<int>(static_cast<uint32_t>(two >> off) & mask) - mid;
        out[q] |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * k);
      }
    }
    u32x4_t* dst = reinterpret_cast<u32x4_t*>(w + n * d_in + run * 32);
    dst[0] = u32x4_t{out[0], out[1], out[2], out[3]};
    dst[1] = u32x4_t{out[4], out[5], out[6], out[7]};
  }
  if (blockIdx.y == 0 && offsets) offsets[n] = zeros[n] - mid;
}

// ------------------------------------------------------------------ product --
struct IntParams {
  const int8_t* x;       // [m, ldx]
  const float* x_scales;
  const int32_t* x_sums;
  const int8_t* w;       // [d_out, d_in]
  const float* w_scales;
  const int32_t* w_offsets;
  void* y;               // [m, d_out]
  int64_t m, d_out, ldx;
  int32_t d_in;
  int32_t y_bf16;
  const void* xraw;      // x not yet quantized (the fused stream kernel), its row stride,
  int64_t ldxraw;
  int32_t xvec;          // and whether its rows are 16-byte aligned
  int32_t yvec;          // rows of y (and of a residual) take whole vectors of four
};

// What follows the scales (E: kPlain, kLinear, kGated).
//   kLinear  y = act(z + bias) + residual
//   kGated   y = act(z + bias) (z' + bias'), z' of a second layer over the same x
enum { kPlain = 0, kLinear = 1, kGated = 2 };
template <int E>
struct Epilogue {};
template <>
struct Epilogue<kLinear> {
  const float* bias;   // or null
  const void* res;     // [m, ldr], or null
  int64_t ldr;
  int32_t act, res_bf16;
};
template <>
struct Epilogue<kGated> {
  const int8_t* w;     // the second layer: as in IntParams
  const float* w_scales;
  const int32_t* w_offsets;
  const float* bias;   // of the first, or null
  const float* bias2;  // of the second
  int32_t act;
};

// Logistic forms go through 2^x and a reciprocal (an ulp each; the exponent's
// rounding adds |z| 2^-24 where the result is next to 0).  gelu takes z Phi(z), Phi(-a) = erfc(a / sqrt(2)) / 2, with erfc in
// the form t exp(P(t) - x^2), t = 1 / (1 + x / 2), of Press, Teukolsky, Vetterling and Flannery (Numerical Recipes,
// the chapter on special functions): here t 2^(P(t) - a^2 log2(e) / 2), t = 1 / (1 + a / sqrt(8)), P of degree 9 fitted anew to
// the exponent.  The fit is off by 2^-22 relative at any a, so that the result holds far below 0, where 1 + erf would
// cancel; the exponent is rounded in fp32 at its own size, which adds about a^2 2^-24: 2^-20 in all at
// a = 4, 2^-17 at 12, always under (a^2 + 18) 2^-23.  NaN passes through all of them.
GPTQ_DEV float logistic(float z, float t) {  // z / (1 + e^-t)
  return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * t));
}
GPTQ_DEV float gelu(float z) {
  const float a = fabsf(z), t = __builtin_amdgcn_rcpf(fmaf(0.35355339059327376f, a, 1.f));
  float q = 0.24347086250782013f;
  q = fmaf(q, t, -1.1733814477920532f);
  q = fmaf(q, t, 2.1254589557647705f);
  q = fmaf(q, t, -1.6174057722091675f);
  q = fmaf(q, t, 0.3914777338504791f);
  q = fmaf(q, t, -0.26540711522102356f);
  q = fmaf(q, t, 0.1390586793422699f);
  q = fmaf(q, t, 0.5397483110427856f);
  q = fmaf(q, t, 1.4427276849746704f);
  q = fmaf(q, t, -2.8257482051849365f);
  const float below = a * (t * __builtin_amdgcn_exp2f(fmaf(-0.7213475204444817f * a, a, q)));  // a Phi(-a)
  return z < 0.f ? -below : z - fminf(below, 1.f);  // (it is less than 0.18; at infinity inf 0, and infinity is kept)
}
GPTQ_DEV float activate(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;
    case kActGelu: return gelu(z);
    case kActGeluTanh: return logistic(z, 1.5957691216057308f * (z + 0.044715f * z * z * z));
    case kActSilu: return logistic(z, z);
    default: return z;
  }
}
// n values, the choice made once for all
template <int N>
GPTQ_DEV void activate(float (&z)[N], int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = activate(z[i], kActRelu);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = activate(z[i], kActGelu);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = activate(z[i], kActGeluTanh);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = activate(z[i], kActSilu);
      break;
    default: break;
  }
}

GPTQ_DEV void int_put(const IntParams& p, int64_t row, int64_t col, float v) {
  if (p.y_bf16)
    static_cast<uint16_t*>(p.y)[row * p.d_out + col] = f32_to_bf16(v);
  else
    static_cast<float*>(p.y)[row * p.d_out + col] = v;
}
GPTQ_DEV float linear_out(const Epilogue<kLinear>& e, float z, float bias, float res) {
  return activate(z + bias, e.act) + res;
}
// a value that has its scales, to y
GPTQ_DEV void int_finish(const IntParams& p, const Epilogue<kPlain>&, int64_t row, int64_t col, float z) {
  int_put(p, row, col, z);
}
GPTQ_DEV void int_finish(const IntParams& p, const Epilogue<kLinear>& e, int64_t row, int64_t col, float z) {
  float r = 0.f;
  if (e.res) r = e.res_bf16 ? load1<true>(e.res, row * e.ldr + col) : load1<false>(e.res, row * e.ldr + col);
  int_put(p, row, col, linear_out(e, z, e.bias ? e.bias[col] : 0.f, r));
}
// the two sums of a gated product, to y
GPTQ_DEV void gated_finish(const IntParams& p, const Epilogue<kGated>& e, int64_t row, int64_t col, int gate, int up,
                           float sx, int xsum) {
  if (p.w_offsets) gate -= p.w_offsets[col] * xsum;
  if (e.w_offsets) up -= e.w_offsets[col] * xsum;
  const float zg = (static_cast<float>(gate) * sx) * p.w_scales[col] + (e.bias ? e.bias[col] : 0.f);
  const float zu = (static_cast<float>(up) * sx) * e.w_scales[col] + (e.bias2 ? e.bias2[col] : 0.f);
  int_put(p, row, col, activate(zg, e.act) * zu);
}

// Few tokens: the weights are streamed once, bound by HBM.  A workgroup owns 16 R
// output channels; its eight waves take turns of 64 kU k, and each 16x16x64
// product takes its 16 weight rows straight from global memory (16 bytes a
// lane) and the tokens' codes from the caches or LDS.  The next turn's weights are
// loaded before the current one's products (loading its x early too measured no
// faster).  The waves' sums meet in LDS.
// R: the tokens' codes are as many bytes as 16 weight rows, so with R = 1 half of
// what the CUs load is x; R row blocks share each load of x where d_out gives
// every CU a workgroup all the same (16 tokens through 28672 x 8192: 67 us with
// R = 1, 63 with R = 4, 49 with x not read at all).
// 16 tokens: 11008 x 4096 15.1 us (a kernel that only reads those 45 MB takes
// 12 to 15), 8192 x 28672 57 us, 4.1 TB/s.
// FUSED (one to four tokens): x is quantized here, by every workgroup for
// itself and into LDS, while its first weights are on their way: one launch, and
// reading the tokens again from L2 costs less than a second one.  bf16 tokens are loaded
// before those weights, since loads come back in their order (11008 -> 4096, one token:
// 15.9 us against 17.3; two layers 8192 -> 28672, gated: 88 against 95; fp32 ones, twice
// the registers, 5% slower so).
// ONCE (FUSED, up to kOnceElems values): one turn has all of K, so no next weights are held, and
// three workgroups run on a CU instead of two (one token in a replayed graph, 4096 -> 4096 6.3 us, 7.1
// without; -> 11008 12.3 and 15.8, through two such layers, gated, 19.3 and 25.5).
constexpr int kSW = 8;                // waves
constexpr int kFusedElems = 16384;    // tokens * d_in at most
constexpr int kOnceElems = 4096;      // tokens * d_in of ONCE at most, a turn of R = 1

// kGated: a block of 16 weight rows is eight channels of the gate and the same eight
// of the second layer, so that both weights stream through one loop.
template <int E>
GPTQ_DEV const int8_t* block_row(const IntParams& p, const Epilogue<E>&, int64_t block, int c) {
  return p.w + min(block * 16 + c, p.d_out - 1) * p.d_in;
}
template <>
GPTQ_DEV const int8_t* block_row<kGated>(const IntParams& p, const Epilogue<kGated>& e, int64_t block, int c) {
  return (c < 8 ? p.w : e.w) + min(block * 8 + (c & 7), p.d_out - 1) * p.d_in;
}

template <int R, int MT, int FUSED, bool ONCE, int E>  // FUSED: 0 codes given, 1 bf16, 2 fp32, 3 bf16 after the weights
__global__ __launch_bounds__(64 * kSW, ONCE ? 6 : 2) void integer_stream_kernel(IntParams p, Epilogue<E> ep) {
  constexpr int kU = R == 1 && MT == 1 ? 8 : R == 4 || MT == 4 ? 2 : 4;
  constexpr int kTurn = kSW * 64 * kU;
  static_assert(!ONCE || kTurn >= kOnceElems, "one turn has all of K");
  constexpr int kElems = ONCE ? kOnceElems : kFusedElems;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int64_t block0 = static_cast<int64_t>(blockIdx.x) * R;
  // Block of tokens (64 of them where there are more).  Taken from the grid for fewer too: the compiler then waits
  // for the first weights before it asks for the others, which arrive earlier so (16 tokens' codes through
  // 11008 x 4096 16.3 us against 17.1, 8192 x 28672 51.2 against 52.4; where one round of loads is all, 4096 x
  // 4096, 0.2 us later).
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 16 * MT;
  const int8_t* wrow[R];
#pragma unroll
  for (int j = 0; j < R; ++j) wrow[j] = block_row<E>(p, ep, block0 + j, c) + 16 * g;
  const int8_t* xrow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xrow[i] = p.x + min(t0 + 16 * i + c, p.m - 1) * p.ldx + 16 * g;
  const i32x4_t zero = {0, 0, 0, 0};
  auto load_w = [&](int k0, i32x4_t (&b)[kU][R]) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = k0 + 64 * u;
#pragma unroll
      for (int j = 0; j < R; ++j) b[u][j] = k + 16 * g < p.d_in ? *reinterpret_cast<const i32x4_t*>(wrow[j] + k) : zero;
    }
  };
  i32x4_t b[kU][R];
  if (FUSED != 1) load_w(wave * 64 * kU, b);

  __shared__ __attribute__((aligned(16))) int8_t xl[FUSED ? kElems : 16];
  __shared__ float xs[4];
  __shared__ int xsum[4];
  if (FUSED) {
    // All tokens at once, eight values a thread and round: their maxima, then their code
    // sums, meet in LDS, those of a single token one a wave, of several by atomics
    // (integers: any order gives the same; four tokens of 4096 one behind the other 33 us
    // a call, at once 30; but one token by atomics 26 instead of 25).
    constexpr bool kBf16 = FUSED != 2;
    constexpr int kQ = kElems / 8 / (64 * kSW);
    __shared__ uint32_t most[4], wave_most[kSW];
    __shared__ int wave_sum[kSW];
    const bool one = p.m == 1;
    if (!one && threadIdx.x < 4) {
      most[threadIdx.x] = 0u;
      xsum[threadIdx.x] = 0;
    }
    const int chunks = p.d_in / 8, all = static_cast<int>(p.m) * chunks;
    float v[kQ][8];
    int tok[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int e = q * 64 * kSW + static_cast<int>(threadIdx.x);
      tok[q] = e < all ? (e >= chunks) + (e >= 2 * chunks) + (e >= 3 * chunks) : 0;
      const int64_t at = tok[q] * p.ldxraw + 8 * (e - tok[q] * chunks);
      if (e < all && p.xvec) {
        load8<kBf16>(p.xraw, at, v[q]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[q][i] = e < all ? load1<kBf16>(p.xraw, at + i) : 0.f;
      }
    }
    if (FUSED == 1) {
      load_w(wave * 64 * kU, b);
      asm volatile("" ::: "memory");  // (not before x's loads, which come back in their order)
    }
    uint32_t am1 = 0u;
    if (one) {
#pragma unroll
      for (int q = 0; q < kQ; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) am1 = max(am1, abs_bits(v[q][i]));
      am1 = group_max<64>(am1);
      if (lane == 0) wave_most[wave] = am1;
    }
    __syncthreads();
    if (one) {
#pragma unroll
      for (int w = 0; w < kSW; ++w) am1 = max(am1, wave_most[w]);
      const RowScale rs = row_scale(am1, 127.f);
      int sum = 0;
#pragma unroll
      for (int q = 0; q < kQ; ++q) sum += tok_store<true>(xl, 0, 8 * (q * 64 * kSW + static_cast<int>(threadIdx.x)), p.d_in, v[q], rs);
      sum = group_sum<64>(sum);
      if (lane == 0) wave_sum[wave] = sum;
      __syncthreads();
      if (threadIdx.x == 0) {
        sum = 0;
#pragma unroll
        for (int w = 0; w < kSW; ++w) sum += wave_sum[w];
        xs[0] = rs.scale;
        xsum[0] = sum;
      }
    } else {
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        if (q * 64 * kSW >= all) break;
        uint32_t am = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) am = max(am, abs_bits(v[q][i]));
        am = group_max<4>(am);  // d_in % 32 == 0: four lanes have one token
        if (__all(tok[q] == __builtin_amdgcn_readfirstlane(tok[q]))) {
          am = group_max<64>(am);
          if (lane == 0) atomicMax(&most[tok[q]], am);
        } else if ((lane & 3) == 0) {
          atomicMax(&most[tok[q]], am);
        }
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        if (q * 64 * kSW >= all) break;
        const int e = q * 64 * kSW + static_cast<int>(threadIdx.x);
        const RowScale rs = row_scale(most[tok[q]], 127.f);
        int sum = e < all ? tok_store<true>(xl, 0, 8 * e, 8 * all, v[q], rs) : 0;
        sum = group_sum<4>(sum);
        if (__all(tok[q] == __builtin_amdgcn_readfirstlane(tok[q]))) {
          sum = group_sum<64>((lane & 3) == 0 ? sum : 0);
          if (lane == 0) atomicAdd(&xsum[tok[q]], sum);
        } else if ((lane & 3) == 0) {
          atomicAdd(&xsum[tok[q]], sum);
        }
      }
      if (threadIdx.x < 4) xs[threadIdx.x] = row_scale(most[threadIdx.x], 127.f).scale;
      __syncthreads();
    }
  }

  i32x4_t acc[R][MT];
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = zero;
  for (int k0 = wave * 64 * kU; k0 < p.d_in; k0 += kTurn) {
    i32x4_t a[kU][MT], next[kU][R];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = k0 + 64 * u;
      const bool in = k + 16 * g < p.d_in;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (FUSED) a[u][i] = in ? *reinterpret_cast<const i32x4_t*>(xl + min(c, static_cast<int>(p.m) - 1) * p.d_in + k + 16 * g) : zero;
        else a[u][i] = in ? *reinterpret_cast<const i32x4_t*>(xrow[i] + k) : zero;
      }
    }
    if (!ONCE) load_w(k0 + kTurn, next);
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][i], b[u][j], acc[j][i], 0, 0, 0);
    if (ONCE) break;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < R; ++j) b[u][j] = next[u][j];
  }
  __shared__ int part[kSW][R][MT][16][17];
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][j][i][4 * g + r][c] = acc[j][i][r];
  __syncthreads();
  constexpr int kC = E == kGated ? 8 : 16;  // channels of a block
  for (int e = threadIdx.x; e < R * MT * 16 * kC; e += 64 * kSW) {
    const int tc = e % kC, j = (e / kC) % R, tr = (e / (kC * R)) & 15, i = e / (16 * kC * R);
    const int64_t col = (block0 + j) * kC + tc, row = t0 + 16 * i + tr;
    if (col >= p.d_out || row >= p.m) continue;
    const int off = p.w_offsets ? p.w_offsets[col] : 0;
    const float sx = FUSED ? xs[tr & 3] : p.x_scales[row], sw = p.w_scales[col];
    int s = 0;
#pragma unroll
    for (int w = 0; w < kSW; ++w) s += part[w][j][i][tr][tc];
    if constexpr (E == kGated) {
      int s2 = 0;
#pragma unroll
      for (int w = 0; w < kSW; ++w) s2 += part[w][j][i][tr][tc + 8];
      gated_finish(p, ep, row, col, s, s2, sx, FUSED ? xsum[tr & 3] : p.x_sums ? p.x_sums[row] : 0);
    } else {
      if (p.w_offsets) s -= off * (FUSED ? xsum[tr & 3] : p.x_sums[row]);
      int_finish(p, ep, row, col, (static_cast<float>(s) * sx) * sw);
    }
  }
}

// Some tokens (up to sixteen) and many channels: as above, but the codes lie in LDS, once for a
// workgroup that walks over the row blocks, so that only weights are loaded.
// Sixteen waves split K; the sums meet in LDS by integer atomics (any order
// gives the same), in one of two buffers by turns: a buffer is read and cleared
// between the barriers of its row block and of the next one.
constexpr int kRW = 16, kRU = 4;
constexpr int64_t kResidentBytes = 152 * 1024;  // codes, 16 bytes of padding a row (bank conflicts)

template <int E>
__global__ __launch_bounds__(64 * kRW, 4) void integer_resident_kernel(IntParams p, Epilogue<E> ep) {
  constexpr int kTurn = kRW * 64 * kRU;
  extern __shared__ __attribute__((aligned(16))) int8_t xr[];  // [m][d_in + 16]
  __shared__ int sum[2][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  constexpr int kC = E == kGated ? 8 : 16;  // channels of a row block
  const int blocks = static_cast<int>((p.d_out + kC - 1) / kC), m = static_cast<int>(p.m);
  const int k_first = wave * 64 * kRU + 16 * g;
  const i32x4_t zero = {0, 0, 0, 0};
  auto load_w = [&](int rb, int k0, i32x4_t (&b)[kRU]) {
    const int8_t* w = block_row<E>(p, ep, rb, c);
#pragma unroll
    for (int u = 0; u < kRU; ++u) {
      const int k = k0 + 64 * u;
      b[u] = (rb < blocks && k < p.d_in) ? *reinterpret_cast<const i32x4_t*>(w + k) : zero;
    }
  };
  i32x4_t b[kRU];
  int rb = blockIdx.x, k0 = k_first;
  load_w(rb, k0, b);
  const int pitch = p.d_in + 16, chunks = p.d_in / 16;
  for (int t = 0; t < m; ++t)
    for (int e = threadIdx.x; e < chunks; e += 64 * kRW)
      *reinterpret_cast<i32x4_t*>(xr + t * pitch + 16 * e) = *reinterpret_cast<const i32x4_t*>(p.x + t * p.ldx + 16 * e);
  for (int e = threadIdx.x; e < 2 * 16 * 17; e += 64 * kRW) (&sum[0][0][0])[e] = 0;
  __syncthreads();
  const int8_t* xrow = xr + min(c, m - 1) * pitch;
  i32x4_t acc = zero;
  int buf = 0;
  while (rb < blocks) {
    // k0 counts this wave's turns; every wave makes the same number a row block
    const bool last = k0 - k_first + kTurn >= p.d_in;
    const int nrb = last ? rb + static_cast<int>(gridDim.x) : rb, nk = last ? k_first : k0 + kTurn;
    i32x4_t next[kRU], a[kRU];
    load_w(nrb, nk, next);
#pragma unroll
    for (int u = 0; u < kRU; ++u) {
      const int k = k0 + 64 * u;
      a[u] = *reinterpret_cast<const i32x4_t*>(xrow + min(k, p.d_in - 16));  // past d_in the weights are zeros
    }
#pragma unroll
    for (int u = 0; u < kRU; ++u) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u], b[u], acc, 0, 0, 0);
    if (last) {
#pragma unroll
      for (int r = 0; r < 4; ++r) atomicAdd(&sum[buf][4 * g + r][c], acc[r]);
      acc = zero;
      __syncthreads();
      if (threadIdx.x < 256) {
        const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
        const int64_t col = static_cast<int64_t>(rb) * kC + tc % kC;
        int s = sum[buf][tr][tc];
        sum[buf][tr][tc] = 0;
        if constexpr (E == kGated) {
          const int s2 = __shfl_down(s, 8);  // all of a wave's lanes are here
          if (tc < 8 && col < p.d_out && tr < m)
            gated_finish(p, ep, tr, col, s, s2, p.x_scales[tr], p.x_sums ? p.x_sums[tr] : 0);
        } else if (col < p.d_out && tr < m) {
          const int off = p.w_offsets ? p.w_offsets[col] : 0;
          const float sx = p.x_scales[tr], sw = p.w_scales[col];
          if (p.w_offsets) s -= off * p.x_sums[tr];
          int_finish(p, ep, tr, col, (static_cast<float>(s) * sx) * sw);
        }
      }
      buf ^= 1;
    }
    rb = nrb;
    k0 = nk;
#pragma unroll
    for (int u = 0; u < kRU; ++u) b[u] = next[u];
  }
}

template <int R, int E>
void stream_go(const IntParams& p, const Epilogue<E>& ep, int fused, hipStream_t st) {
  constexpr int kC = E == kGated ? 8 : 16;
  const dim3 grid(static_cast<unsigned>((p.d_out + kC * R - 1) / (kC * R)), static_cast<unsigned>((p.m + 63) / 64));
  const int t = 64 * kSW;
  if constexpr (R == 1) {
    if (fused && p.m * p.d_in <= kOnceElems) {
      if (fused == 1) integer_stream_kernel<1, 1, 1, true, E><<<grid, t, 0, st>>>(p, ep);
      else integer_stream_kernel<1, 1, 2, true, E><<<grid, t, 0, st>>>(p, ep);
      return;
    }
  }
  if constexpr (R == 2) {
    // One token's blocks of two, past ONCE: the weights first (5120 -> 13824 19.2 us, 20.2 with the token first, 4128
    // -> 13824 16.8 and 19.1; but 8192 -> 13824 28.7 and 28.5, 14336 -> 13824 44.1 and 42.0, two tokens of 5120 21.0 and 20.0).
    if (fused == 1 && p.m == 1 && p.d_in < 8192) {
      integer_stream_kernel<2, 1, 3, false, E><<<grid, t, 0, st>>>(p, ep);
      return;
    }
  }
  if (fused == 1) integer_stream_kernel<R, 1, 1, false, E><<<grid, t, 0, st>>>(p, ep);
  else if (fused == 2) integer_stream_kernel<R, 1, 2, false, E><<<grid, t, 0, st>>>(p, ep);
  else if (p.m <= 16) integer_stream_kernel<R, 1, 0, false, E><<<grid, t, 0, st>>>(p, ep);
  else if (p.m <= 32) integer_stream_kernel<R, 2, 0, false, E><<<grid, t, 0, st>>>(p, ep);
  else if constexpr (R <= 2) integer_stream_kernel<R, 4, 0, false, E><<<grid, t, 0, st>>>(p, ep);
}

// Many tokens: 64 WM x 64 WN output tiles on v_mfma_i32_32x32x32_i8, four waves
// of 32 WM x 32 WN each.  Rows of both operands are k-contiguous, so a step of 128
// bytes of a tile's rows goes to LDS by buffer_load ... lds as it lies in memory,
// through a ring of steps, and the MFMA operands are 16-byte LDS reads.  Each
// quarter step's operands are read while the previous quarter's products run; one barrier
// a step publishes the next step's data and frees the slot that has just been read.
// LDS rows are 128 bytes; 16-byte chunk c of row r sits at c ^ ((r >> 1) & 7), so
// 16 lanes that read one chunk of 16 rows touch all 64 banks once.
// The way into LDS is what the tiles wait for beside the products: a KB of it takes a CU
// some 66 cycles in pieces of 64 bytes and 45 in whole lines of 128 (the kernel of 2048 x 28672 ->
// 8192 alone, without a residual: 405 us and 356; wider pieces of a row are no faster), whatever the depth of
// the ring; with nothing else to do 33, through registers too.  That kernel with a residual
// 370 us, 2.6 POP/s, the gated 2048 x 8192 -> 2 x 28672 770 us, 2.5 POP/s (an 8192-cubed library
// product 2.07), matrix cores busy two thirds of the cycles; 509 x 11008 -> 4096 36 us.
constexpr int kTStep = 128;

#define GPTQ_VMCNT(n) (((n) & 15) | (((n) >> 4) << 14) | 0x0F70)
#define GPTQ_VMCNT_LDS(n) (((n) & 15) | (((n) >> 4) << 14) | 0x0070)  // and no LDS read on its way

GPTQ_DEV __amdgpu_buffer_rsrc_t rows_rsrc(const int8_t* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  const int n = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo),
                                           static_cast<short>(0), n, 0x00020000);
}

// one piece (8 rows x 128 bytes) of a step to LDS, k0 bytes into the rows
GPTQ_DEV void tile_dma(__amdgpu_buffer_rsrc_t rs, uint8_t* piece, uint32_t voff, uint32_t k0) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)piece, 16, voff, k0, 0, 0);
}

template <int W>
GPTQ_DEV void tile_read(const uint8_t* op, uint32_t off, i32x4_t (&f)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) f[i] = *reinterpret_cast<const i32x4_t*>(op + off + i * 4096);
}

// after product K of N: its share of the LDS reads and of the loads to LDS
template <int K, int N, int READS, int LOADS>
GPTQ_DEV void tile_spread() {
  if constexpr (K < N) {
    constexpr int reads = (K + 1) * READS / N - K * READS / N, loads = (K + 1) * LOADS / N - K * LOADS / N;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
    if constexpr (loads > 0) __builtin_amdgcn_sched_group_barrier(0x020, loads, 0);
    tile_spread<K + 1, N, READS, LOADS>();
  }
}

// The products of a quarter step, with the next one's reads, and LOADS loads to LDS issued before, spread over them.
template <int WM, int WN, int LOADS>
GPTQ_DEV void tile_quarter(const i32x4_t (&a)[WM], const i32x4_t (&b)[WN], const uint8_t* nA, const uint8_t* nB,
                           uint32_t offA, uint32_t offB, i32x4_t (&na)[WM], i32x4_t (&nb)[WN], i32x16_t (&acc)[WM][WN]) {
  tile_read<WM>(nA, offA, na);
  tile_read<WN>(nB, offB, nb);
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
  tile_spread<0, WM * WN, WM + WN, LOADS>();
}

struct TileGrid {
  int32_t nm, nn;      // tiles along m and d_out
  int32_t slices, per; // K slices and steps of each
  int32_t* partial;    // [slice][m][d_out] when slices > 1
};

// Workgroups go round-robin over the 8 XCDs, each with its own L2: the tiles are
// cut into 8 runs, and a run walks up to eight tiles of m before the next one of
// d_out, so the workgroups of one XCD share rows of both operands.
GPTQ_DEV void tile_of(const TileGrid& g, int b, int& tm, int& tn, int& slice) {
  const int total = g.nm * g.nn * g.slices;
  const int x = b & 7, base = total >> 3, rem = total & 7;
  int q = x * base + min(x, rem) + (b >> 3);
  slice = q / (g.nm * g.nn);
  q -= slice * (g.nm * g.nn);
  const int strip = q / (8 * g.nn), rows = min(8, g.nm - 8 * strip);
  q -= strip * 8 * g.nn;
  tm = 8 * strip + q % rows;
  tn = q / rows;
}

enum { kOutF32 = 0, kOutBf16 = 1, kOutPart = 2 };

struct TileRow {  // of x
  float scale;
  int sum;
};

// What follows the sums of a tile.  A wave's sums, two blocks of 32 rows at a time,
// go through LDS that the operands have left (its own slots, so no barrier), and
// come back as four channels of a row: whole vectors of y and of the residual,
// which is loaded four rows ahead, and code for sixteen values instead of 256: with
// the choice of an activation unrolled over all of them the code left the
// instruction cache, 40 us of a call.  Rows lie bare in LDS, 32 WN words; row bit 2 flips word
// bit 5, so that the two halves of a wave write to different banks.
template <int WM, int WN, int OUT, int E>
GPTQ_DEV void tile_out(const IntParams& p, const Epilogue<E>& ep, const i32x16_t (&acc)[WM][WN], uint8_t* r0, uint8_t* r1,
                       const TileRow* rows, int64_t m0, int64_t n0, int wm, int wn, int mrows) {
  constexpr int kLayers = E == kGated ? 2 : 1;
  constexpr int kPitch = 32 * WN;               // words
  constexpr int kWide = kPitch / kLayers;       // channels of the wave
  constexpr int kAcross = kWide / 4;            // lanes of a row
  constexpr int kRows = 64 / kAcross, kB = 4;   // rows at a time, and times in flight
  const int lane = lane_id(), r = lane & 31, hi = lane >> 5;
  const int ch = 4 * (lane % kAcross), sub = lane / kAcross;
  const int at = E == kGated ? (ch >> 5) * 64 + (ch & 31) : ch;
  const int64_t col = n0 + wn * kWide + ch;
  const int live = static_cast<int>(max(min(p.d_out - col, int64_t{4}), int64_t{0}));
  float sw[kLayers][4], bias[kLayers][4];
  int off[kLayers][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t c = min(col + j, p.d_out - 1);
    sw[0][j] = p.w_scales[c];
    off[0][j] = p.w_offsets ? p.w_offsets[c] : 0;
    bias[0][j] = 0.f;
    if constexpr (E != kPlain) bias[0][j] = ep.bias ? ep.bias[c] : 0.f;
    if constexpr (E == kGated) {
      sw[1][j] = ep.w_scales[c];
      off[1][j] = ep.w_offsets ? ep.w_offsets[c] : 0;
      bias[1][j] = ep.bias2 ? ep.bias2[c] : 0.f;
    }
  }
  // y and the residual through buffer resources over the tile's rows: what lies past m, or past
  // d_out (offset 2^31), is dropped, or loaded as zeros
  constexpr int kSize = OUT == kOutBf16 ? 2 : 4;
  const int dout = static_cast<int>(p.d_out);
  const __amdgpu_buffer_rsrc_t ry =
      rows_rsrc(static_cast<const int8_t*>(p.y) + m0 * p.d_out * kSize, static_cast<int64_t>(mrows) * dout * kSize);
  __amdgpu_buffer_rsrc_t rres = ry;
  uint32_t lead = 0;
  if constexpr (E == kLinear) {
    const int size = ep.res_bf16 ? 2 : 4;
    lead = static_cast<uint32_t>(ep.ldr) * size;
    rres = rows_rsrc(static_cast<const int8_t*>(ep.res) + m0 * ep.ldr * size,
                     ep.res ? ((mrows - 1) * ep.ldr + p.d_out) * size : 0);
  }
  const uint32_t outside = 0x80000000u;
  // four values of the residual, as they lie there
  auto load_res = [&](int row, u32x4_t& raw) {
    raw = u32x4_t{0u, 0u, 0u, 0u};
    if constexpr (E == kLinear) {
      if (!ep.res) return;
      const uint32_t at = static_cast<uint32_t>(row) * lead;
      if (ep.res_bf16) {
        const uint32_t c = static_cast<uint32_t>(col) * 2;
        if (p.yvec) {
          const auto two = __builtin_amdgcn_raw_buffer_load_b64(rres, live ? at + c : outside, 0, 0);
          raw[0] = two[0];
          raw[1] = two[1];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            raw[j >> 1] |= static_cast<uint32_t>(static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(
                               rres, j < live ? at + c + 2 * j : outside, 0, 0))) << (16 * (j & 1));
        }
      } else {
        const uint32_t c = static_cast<uint32_t>(col) * 4;
        if (p.yvec) {
          raw = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rres, live ? at + c : outside, 0, 0));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) raw[j] = __builtin_amdgcn_raw_buffer_load_b32(rres, j < live ? at + c + 4 * j : outside, 0, 0);
        }
      }
    }
  };
  auto res_of = [&](const u32x4_t& raw, int j) {
    if constexpr (E == kLinear) {
      if (ep.res_bf16) return __uint_as_float((j & 1) ? raw[j >> 1] & 0xFFFF0000u : raw[j >> 1] << 16);
      return __uint_as_float(raw[j]);
    }
    return 0.f;
  };
  auto store = [&](int row, const float* v) {
    const uint32_t to = static_cast<uint32_t>(row) * static_cast<uint32_t>(dout * kSize) + static_cast<uint32_t>(col) * kSize;
    if (OUT == kOutBf16) {
      typedef float f32x2v_t __attribute__((ext_vector_type(2)));
      typedef __bf16 bf16x2v_t __attribute__((ext_vector_type(2)));
      typedef __attribute__((__vector_size__(8))) uint32_t u32x2_t;
      const u32x2_t two = {__builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2v_t{v[0], v[1]}), bf16x2v_t)),
                           __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2v_t{v[2], v[3]}), bf16x2v_t))};
      if (p.yvec) {
        __builtin_amdgcn_raw_buffer_store_b64(two, ry, live ? to : outside, 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          __builtin_amdgcn_raw_buffer_store_b16(static_cast<short>(two[j >> 1] >> (16 * (j & 1))), ry, j < live ? to + 2 * j : outside, 0, 0);
      }
    } else if (p.yvec) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, (f32x4_t{v[0], v[1], v[2], v[3]})), ry, live ? to : outside, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(v[j]), ry, j < live ? to + 4 * j : outside, 0, 0);
    }
  };
  // (row sums of codes and offsets fit 24 bits: 127 65536 < 2^23)
  auto scaled = [&](int sum, int l, int j, int rowsum, float rowscale) {
    return (static_cast<float>(sum - __mul24(off[l][j], rowsum)) * rowscale) * sw[l][j];
  };
  constexpr int kHalves = WM == 1 ? 1 : 2;
#pragma unroll
  for (int i = 0; i < WM; i += kHalves) {
    const int row0 = (wm * WM + i) * 32 + sub;
    u32x4_t ahead[kB];
#pragma unroll
    for (int b = 0; b < kB; ++b) load_res(row0 + b * kRows, ahead[b]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
#pragma unroll
    for (int half = 0; half < kHalves; ++half)
#pragma unroll
      for (int j = 0; j < WN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          reinterpret_cast<int*>(half ? r1 : r0)[(8 * (e >> 2) + 4 * hi + (e & 3)) * kPitch + ((32 * j + r) ^ (32 * hi))] = acc[i + half][j][e];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
    __builtin_amdgcn_wave_barrier();
    struct Held {
      i32x4_t sum[kLayers][kB];
      float sc[kB];
      int sm[kB];
    } next;
    auto read = [&](int q, Held& h) {
      const uint8_t* from = q < 32 ? r0 : r1;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const int rr = (q & 31) + b * kRows + sub;
        const int word = rr * kPitch + (at ^ (((rr >> 2) & 1) * 32));
        h.sum[0][b] = reinterpret_cast<const i32x4_t*>(from)[word >> 2];
        if constexpr (E == kGated) h.sum[1][b] = reinterpret_cast<const i32x4_t*>(from)[(word ^ 32) >> 2];
        h.sc[b] = rows[row0 + q + b * kRows].scale;
        h.sm[b] = rows[row0 + q + b * kRows].sum;
      }
    };
    read(0, next);
#pragma unroll 1
    for (int q = 0; q < 32 * kHalves; q += kRows * kB) {
      const Held now = next;
      u32x4_t res[kB];
#pragma unroll
      for (int b = 0; b < kB; ++b) res[b] = ahead[b];
      if (q + kRows * kB < 32 * kHalves) {
        read(q + kRows * kB, next);
#pragma unroll
        for (int b = 0; b < kB; ++b) load_res(row0 + q + (kB + b) * kRows, ahead[b]);
      }
      float v[4 * kB];
#pragma unroll
      for (int b = 0; b < kB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * b + j] = scaled(now.sum[0][b][j], 0, j, now.sm[b], now.sc[b]);
      if constexpr (E != kPlain) {
#pragma unroll
        for (int b = 0; b < kB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * b + j] += bias[0][j];
        activate(v, ep.act);
#pragma unroll
        for (int b = 0; b < kB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (E == kLinear) v[4 * b + j] += res_of(res[b], j);
            if constexpr (E == kGated) v[4 * b + j] *= scaled(now.sum[1][b][j], 1, j, now.sm[b], now.sc[b]) + bias[1][j];
          }
      }
#pragma unroll
      for (int b = 0; b < kB; ++b) store(row0 + q + b * kRows, v + 4 * b);
    }
  }
}

// kGated: the 64 WN weight rows of a tile are 32 WN channels of both layers, in
// blocks of 32 by turns: a wave's products 2 j and 2 j + 1 are the same channels of
// the gate and of the second layer, in the same lanes.  A wave's loads, 16 WN of
// the rows, never mix the layers inside a piece.
template <int WM, int WN, int OUT, int E>
__global__ __launch_bounds__(256) void integer_tile_kernel(IntParams p, TileGrid g, Epilogue<E> ep) {
  constexpr int kCols = E == kGated ? 32 * WN : 64 * WN;  // channels of a tile
  constexpr int kA = WM * 64 * kTStep, kB = WN * 64 * kTStep;
  // Tiles of 64 tokens have little to multiply: a deeper ring.
  constexpr int kSlots = WM == 1 ? 4 : 2;
  constexpr int kA2 = kSlots == 4 ? kA : 16, kB2 = kSlots == 4 ? kB : 16;
  // one array per slot: the compiler then sees that reads of one slot do not alias loads in flight into another
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[kA], sA1[kA], sA2[kA2], sA3[kA2];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[kB], sB1[kB], sB2[kB2], sB3[kB2];
  __shared__ TileRow rows[64 * WM];
  int tm, tn, slice;
  tile_of(g, static_cast<int>(blockIdx.x), tm, tn, slice);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = static_cast<int64_t>(tm) * (64 * WM), n0 = static_cast<int64_t>(tn) * kCols;
  const int mrows = static_cast<int>(min(p.m - m0, int64_t{64 * WM}));
  const int nrows = static_cast<int>(min(p.d_out - n0, int64_t{kCols}));
  const __amdgpu_buffer_rsrc_t ra = rows_rsrc(p.x + m0 * p.ldx, (mrows - 1) * p.ldx + p.d_in);
  // the layer of the wave's pieces: of all of them, or (kGated in wide tiles) of the first four and the last four
  const int8_t *w_lo = p.w, *w_hi = p.w;
  if constexpr (E == kGated) {
    w_lo = WN == 2 && (wave & 1) ? ep.w : p.w;
    w_hi = WN == 2 ? w_lo : ep.w;
  }
  const __amdgpu_buffer_rsrc_t rb = rows_rsrc(w_lo + n0 * p.d_in, static_cast<int64_t>(nrows) * p.d_in);
  const __amdgpu_buffer_rsrc_t rb_hi = rows_rsrc(w_hi + n0 * p.d_in, static_cast<int64_t>(nrows) * p.d_in);
  // A piece is 8 rows; lane l has row l / 8 of it and writes position l % 8 of that row.
  constexpr int kPA = 2 * WM, kPB = 2 * WN;  // pieces of a step, per wave
  const int prow = lane >> 3;
  uint32_t va[kPA], vb[kPB];
  const int kc = ((lane & 7) ^ ((prow >> 1) & 3)) * 16;  // pieces of even number; the others' rows are four pairs on
#pragma unroll
  for (int u = 0; u < kPA; ++u) {
    const int row = (wave * kPA + u) * 8 + prow;
    va[u] = row < mrows ? static_cast<uint32_t>(row * static_cast<int>(p.ldx) + (kc ^ ((u & 1) * 64))) : 0x80000000u;
  }
#pragma unroll
  for (int u = 0; u < kPB; ++u) {
    const int piece = wave * kPB + u;  // kGated: 4 pieces of the one layer, 4 of the other
    const int row = (E == kGated ? 4 * (piece >> 3) + (piece & 3) : piece) * 8 + prow;
    vb[u] = row < nrows ? static_cast<uint32_t>(row * p.d_in + (kc ^ ((u & 1) * 64))) : 0x80000000u;
  }
  const int s0 = slice * g.per;
  const int steps = min(g.per, (p.d_in + kTStep - 1) / kTStep - s0);
  auto slotA = [&](int u) -> uint8_t* {
    switch (u % kSlots) {
      case 0: return sA0; case 1: return sA1; case 2: return sA2; default: return sA3;
    }
  };
  auto slotB = [&](int u) -> uint8_t* {
    switch (u % kSlots) {
      case 0: return sB0; case 1: return sB1; case 2: return sB2; default: return sB3;
    }
  };
  // What lies past the row's end is loaded as zeros, and steps past the slice's end as nothing but them
  // (the lane's offset 2^31: out of range; k0, the scalar one, never passes the rows' bytes).
  auto issue_x = [&](int s, int slot) {
    const int k0 = s < steps ? (s0 + s) * kTStep : p.d_in, left = p.d_in - k0;
#pragma unroll
    for (int u = 0; u < kPA; ++u)
      tile_dma(ra, slotA(slot) + (wave * kPA + u) * 1024, (kc ^ ((u & 1) * 64)) < left ? va[u] : 0x80000000u, k0);
  };
  auto issue_w = [&](int s, int slot) {
    const int k0 = s < steps ? (s0 + s) * kTStep : p.d_in, left = p.d_in - k0;
#pragma unroll
    for (int u = 0; u < kPB; ++u)
      tile_dma(E == kGated && u >= 4 ? rb_hi : rb, slotB(slot) + (wave * kPB + u) * 1024,
               (kc ^ ((u & 1) * 64)) < left ? vb[u] : 0x80000000u, k0);
  };
  // operand reads: row l % 32 of a 32-row tile, chunk 2 quarter + l / 32
  const int r = lane & 31, hi = lane >> 5;
  uint32_t oa[4], ob[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t o = static_cast<uint32_t>(r * 128 + (((2 * h + hi) ^ ((r >> 1) & 7)) * 16));
    oa[h] = o + wm * WM * 4096;
    ob[h] = o + wn * WN * 4096;
  }
  i32x16_t acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  i32x4_t a0[WM], b0[WN], a1[WM], b1[WN];
  constexpr int kL = kPA + kPB;  // loads of one step, per wave
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    issue_w(u, u);
    if (u < kSlots - 1) issue_x(u, u);
  }
  __builtin_amdgcn_s_waitcnt(GPTQ_VMCNT((kSlots - 1) * kL - kPA));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  tile_read<WM>(sA0, oa[0], a0);
  tile_read<WN>(sB0, ob[0], b0);
  // steps in blocks of a ring's length; the ones past the end multiply zeros
  for (int s = 0; s < steps; s += kSlots) {
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      // half of a step's loads in each of two quarters: all in one keep the wave waiting at the address unit,
      // later ones arrive late (a call of 2048 x 28672 -> 8192 with a residual, codes' launch included, 419 us with all in
      // the first, 422 in three, 410 so)
      issue_x(s + u + kSlots - 1, u + kSlots - 1);
      tile_quarter<WM, WN, kPA>(a0, b0, slotA(u), slotB(u), oa[1], ob[1], a1, b1, acc);
      tile_quarter<WM, WN, 0>(a1, b1, slotA(u), slotB(u), oa[2], ob[2], a0, b0, acc);
      tile_quarter<WM, WN, 0>(a0, b0, slotA(u), slotB(u), oa[3], ob[3], a1, b1, acc);
      // the last quarter's operands are in registers, in every wave past the barrier, and the next step's data in LDS
      __builtin_amdgcn_s_waitcnt(GPTQ_VMCNT_LDS((kSlots - 2) * kL));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      issue_w(s + u + kSlots, u);
      tile_quarter<WM, WN, kPB>(a1, b1, slotA(u + 1), slotB(u + 1), oa[0], ob[0], a0, b0, acc);
    }
  }
  // Element e of lane l: row 8 (e / 4) + 4 (l / 32) + e % 4, column l % 32.  The K
  // slices' stores go through buffer resources over the tile's rows: rows past m
  // and columns past d_out (offset 2^31) are dropped in hardware.
  __builtin_amdgcn_s_waitcnt(GPTQ_VMCNT(0));  // the loads past the end still write LDS
  const int dout = static_cast<int>(p.d_out);
  constexpr int kLayers = E == kGated ? 2 : 1;
  auto col_of = [&](int j) {  // channel of the lane's products j
    return static_cast<int>(n0) + (E == kGated ? (wn * WN + j) >> 1 : wn * WN + j) * 32 + r;
  };
  const uint32_t row0 = static_cast<uint32_t>(wm * WM * 32 + 4 * hi);
  if (OUT == kOutPart) {
    const __amdgpu_buffer_rsrc_t rp =
        rows_rsrc(reinterpret_cast<int8_t*>(g.partial + (static_cast<int64_t>(slice) * p.m + m0) * (p.d_out * kLayers)),
                  static_cast<int64_t>(mrows) * dout * kLayers * 4);
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      const int col = col_of(j);
#pragma unroll
      for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t row = row0 + 32 * i + 8 * (e >> 2) + (e & 3);
          const uint32_t at = row * dout * kLayers + (E == kGated ? (j & 1) * dout : 0) + col;
          __builtin_amdgcn_raw_buffer_store_b32(acc[i][j][e], rp, col < dout ? at * 4 : 0x80000000u, 0, 0);
        }
    }
    return;
  }
  for (int e = threadIdx.x; e < mrows; e += 256) rows[e] = TileRow{p.x_scales[m0 + e], p.x_sums ? p.x_sums[m0 + e] : 0};
  __syncthreads();  // and every wave is done with the operands' LDS
  uint8_t* own = wave == 0 ? sA0 : wave == 1 ? sA1 : wave == 2 ? sB0 : sB1;
  tile_out<WM, WN, OUT, E>(p, ep, acc, own, own + 4096 * WN, rows, m0, n0, wm, wn, mrows);
}

// sums of the K slices (integers: any order gives the same), four columns a
// thread where rows are whole vectors.  Bound: the caches and HBM (four slices
// of 509 x 4096, 33 MB, in 10 us).
template <int V, int E>
__global__ __launch_bounds__(256) void integer_join_kernel(IntParams p, TileGrid g, Epilogue<E> ep) {
  typedef int ivec_t __attribute__((ext_vector_type(V)));
  const int64_t col = (blockIdx.x * 256ll + threadIdx.x) * V;
  if (col >= p.d_out) return;
  float sw[V];
  int off[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    sw[j] = p.w_scales[col + j];
    off[j] = p.w_offsets ? p.w_offsets[col + j] : 0;
  }
  constexpr int kLayers = E == kGated ? 2 : 1;
  for (int64_t row = blockIdx.y; row < p.m; row += gridDim.y) {
    ivec_t s[kLayers] = {};
    for (int k = 0; k < g.slices; ++k)
#pragma unroll
      for (int l = 0; l < kLayers; ++l)
        s[l] += *reinterpret_cast<const ivec_t*>(g.partial + ((k * p.m + row) * kLayers + l) * p.d_out + col);
    const float sx = p.x_scales[row];
    const int sum = p.x_sums ? p.x_sums[row] : 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (E == kGated) gated_finish(p, ep, row, col + j, s[0][j], s[1][j], sx, sum);
      else int_finish(p, ep, row, col + j, (static_cast<float>(s[0][j] - off[j] * sum) * sx) * sw[j]);
    }
  }
}

// few tokens of few values: quantized by every workgroup of the stream kernel itself
bool fuses(int64_t m, int64_t d_in) { return m <= 4 && m * d_in <= kFusedElems; }

// Row blocks a workgroup of the stream kernel takes: as many as leave every CU one, where the tokens are
// given in codes (us of one token's codes with 1, 2 and 4: 1024 -> 11008 5.9, 5.2, 5.3; 2048 -> 32000 19.3, 17.2,
// 17.7; but up to four tokens 4096 -> 11008 13.5, 14.7, 16.1, 5120 -> 13824 19.3, 19.8, 20.9; 7168 -> 14336 23.2,
// 22.1).
// Tokens quantized by each workgroup for itself (fused) are read and rounded once a block more in blocks of one,
// hardly longer than its first weights take, and those end more evenly.
//   one token  a round of the workgroups of ONCE, three a CU, has 48 blocks of rows a CU: up to there one block
//              (2048 -> 11008 8.1, 10.3, 10.5; 256 -> 8192 5.1, 5.7, 5.6).  Past it short rows are mostly their
//              quantization (512 -> 32000 11.0, 10.4, 7.1; 1024 -> 16384 8.6, 7.4, 7.8), longer ones as
//              long as two rounds do (1536 -> 24576 12.9, 12.7, 13.6; -> 64000 27.8, 26.1, 24.1), from 2560
//              values on one block again (3200 -> 24576 18.5, 22, 22.2; 14336 -> 20480 56, 63, 81), but for rows
//              past 4096 values that are not many (6144 -> 13824 23, 22, 24).  Gated, whose blocks end with two
//              products for one, from 2048 (2048 -> 2 x 16000 17.7, 19.0, 19.4; 1024 -> 2 x 16000 14.7, 13.8, 12.3)
//   two to four  that costs more than it gives (four tokens of 4096 -> 2 x 11008 36 and 30 with one and
//              four), unless they are a turn and the blocks few (two of 2048 -> 11008 7.8 and 10.0;
//              -> 32000 17.7 and 17.6; two of 512 -> 16384 7.7 and 6.2)
int stream_rows(int64_t m, int64_t d_in, int64_t d_out, bool fused, bool gated, int n_cu) {
  const int64_t a_cu = d_out / n_cu;  // rows of a CU
  const int r = a_cu >= 64 ? 4 : a_cu >= 32 ? 2 : 1;
  if (fused && m == 1) {
    if (d_out <= 48ll * n_cu) return 1;
    if (d_in <= (gated ? 512 : 1024) || (d_in < (gated ? 2048 : 2560) && d_out > 96ll * n_cu)) return 4;
    if (d_in <= kOnceElems || a_cu >= 64) return 1;
  } else if (fused) {
    if (m * d_in <= kOnceElems && d_out < (m * d_in <= 1024 ? 48ll : 96ll) * n_cu) return 1;
  } else if (m <= 4 && d_in >= 4096 && d_in < 6144 && a_cu < 64) {
    return 1;
  }
  return m > 32 ? std::min(r, 2) : r;
}

// The launch of a product: kernel, tile and K slices.
struct IntPlan {
  int kind;  // 0: stream, 1: 128 x 128 tiles, 2: 256 x 256, 3: 64 x 128
  int slices, per;
  size_t partial_bytes;
};

// Of the stream kernel (up to 1024 tokens) and the tiles, in 1 to 16 slices of K, the one that should take
// least, by what each costs (us), fitted to the times of all of them over 5 to 4096 tokens and twenty shapes of
// weights, 256 x 4096 to 28672 x 8192, codes given, in replayed graphs.  For k values a token, n rows of weights:
//   stream, up to 16 tokens   kStreamLaunch and the longer of the weights at 6.9 TB/s (some come from the caches)
//           and of the rounds' K
//   stream, more tokens       kBlockLaunch, the weights at 3.8 TB/s and for every begun round of workgroups
//           kBlockRound and 38 ps a token (up to 64) and k: a workgroup loads its tokens' codes beside the weights
//   tiles   kTileLaunch, then the longer of the rounds' steps and of the bytes at 6.6 TB/s; K slices cost a
//           second launch and their sums' way to memory and back
// The choice is 1.5% slower than the best of them in the mean.  (us, stream and 64-row, 128-row, 256-row tiles in
// their best slices: 17 x 4096 -> 4096 8.3, 10.9, 13.6, -; 64 x 4096 -> 11008 28.9, 17.3, 19.7, -;
// 64 x 28672 -> 8192 93, 48, 55, -; 128 x 1024 -> 1024 5.4, 6.6, 8.4, -; 512 x 4096 -> 4096 -, 17.4, 25.9, 29.8;
// 2048 x 4096 -> 1024 -, 13.5, 23.5, 28; 2048 x 4096 -> 4096 -, 63, 39.9, 53;
// 1024 x 8192 -> 8192 -, 115, 77, 81; 2048 x 8192 -> 8192 -, 222, 143, 114.)
constexpr double kStreamLaunch = 5.0, kStreamRate = 6.9e6, kStreamTurn = 0.7e-3;   // us, bytes a us, us a k
constexpr double kBlockLaunch = 1.0, kBlockRate = 3.8e6, kBlockRound = 1.4, kBlockToken = 38e-6;
constexpr double kTileLaunch = 4.5, kTileRate = 6.6e6, kJoinLaunch = 5.0, kJoinRate = 4.3e6;
IntPlan int_plan(int64_t m, int64_t d_in, int64_t d_out, int n_cu) {
  IntPlan a{0, 1, 0, 0};
  if (fuses(m, d_in)) return a;
  const double k = static_cast<double>(d_in), n = static_cast<double>(d_out), rows = static_cast<double>(m);
  double least = 1e300;
  if (m <= 1024) {
    const double blocks = std::ceil(n / (16.0 * stream_rows(m, d_in, d_out, false, false, n_cu))) * std::ceil(rows / 64.0);
    const double rounds = std::max(1.0, blocks / n_cu);
    if (m <= 16) least = kStreamLaunch + std::max(k * n / kStreamRate, kStreamTurn * k * rounds);
    else least = kBlockLaunch + k * n / kBlockRate + std::ceil(rounds) * (kBlockRound + kBlockToken * std::min(rows, 64.0) * k);
  }
  const int64_t steps = (d_in + kTStep - 1) / kTStep;
  const double sums = 8.0 * rows * n / kJoinRate;  // of a slice, there and back
  struct Tile {
    int kind, high, wide;
    double step, full;  // us a step: of a round with one workgroup a CU, with two
  };
  constexpr Tile tiles[3] = {{3, 64, 128, 0.44, 0.44}, {1, 128, 128, 0.84, 1.05}, {2, 256, 256, 1.34, 1.34}};
  for (const Tile& t : tiles) {
    // Many tokens of long rows leave the L2s between their strips of 64 (2048 x 11008 -> 2048: 77 us, 62 in slices
    // of 256-row tiles; 1500 x 8224 -> 1800: 67 and 50, though 1030 of them 39 and 42): outside the fitted terms.
    if (t.kind == 3 && m > 1024 && d_in > 8192) continue;
    const double count = static_cast<double>(((m + t.high - 1) / t.high) * ((d_out + t.wide - 1) / t.wide));
    const double room = t.kind == 1 ? 2.0 * n_cu : n_cu, bytes = k * (n + rows) / kTileRate;
    for (int sl = 0; sl <= 4 && (sl == 0 || steps >> sl >= 4); ++sl) {  // 2^sl slices
      const int64_t per = (steps + (int64_t{1} << sl) - 1) >> sl, slices = (steps + per - 1) / per;
      const double parts = count * static_cast<double>(slices), whole = std::floor(parts / room), rest = parts - whole * room;
      const double last = rest <= 0.0 ? 0.0 : rest <= n_cu ? t.step : t.full;
      double cost = kTileLaunch + std::max(static_cast<double>(per) * (whole * t.full + last), bytes);
      if (slices > 1) cost += kJoinLaunch + static_cast<double>(slices) * sums;
      if (cost < least) {
        least = cost;
        a.kind = t.kind;
        a.slices = static_cast<int>(slices);
        a.per = static_cast<int>(per);
      }
    }
  }
  a.partial_bytes = a.slices > 1 ? static_cast<size_t>(a.slices) * m * d_out * 4 : 0;
  return a;
}

}  // namespace

hipError_t token_codes_launch(const void* x, bool bf16, int64_t m, int64_t d, int64_t ldx, int8_t* codes, float* scales,
                              int32_t* sums, hipStream_t st) {
  const int64_t e = bf16 ? 8 : 4;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (reinterpret_cast<uintptr_t>(codes) & 7u) == 0 &&
                   ldx % e == 0 && d % 8 == 0;
  constexpr int64_t kMost = int64_t{1} << 21;  // rows of a launch, which has fewer than 2^32 threads
  for (int64_t r = 0; r < m; r += kMost) {
    const int64_t n = std::min(m - r, kMost);
    const void* xr = static_cast<const char*>(x) + r * ldx * (bf16 ? 2 : 4);
    int8_t* c = codes + r * d;
    float* sc = scales + r;
    int32_t* sm = sums ? sums + r : nullptr;
    if (d <= 2048) token_codes_go<64, 4>(xr, bf16, vec, n, d, ldx, c, sc, sm, st);
    else if (d <= 8192) token_codes_go<256, 4>(xr, bf16, vec, n, d, ldx, c, sc, sm, st);
    else if (d <= 16384) token_codes_go<256, 8>(xr, bf16, vec, n, d, ldx, c, sc, sm, st);
    else if (d <= 32768) token_codes_go<512, 8>(xr, bf16, vec, n, d, ldx, c, sc, sm, st);
    else token_codes_go<1024, 4>(xr, bf16, vec, n, d, ldx, c, sc, sm, st);
  }
  return hipGetLastError();
}

hipError_t integer_weight_launch(const int32_t* qweight, const int32_t* zeros, int bits, int64_t d_in, int64_t d_out,
                                 int8_t* w, int32_t* offsets, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((d_out + 255) / 256), static_cast<unsigned>(std::min<int64_t>(d_in / 32, 32768)));
  integer_weight_kernel<<<grid, 256, 0, st>>>(qweight, zeros, bits, d_in, d_out, w, offsets);
  return hipGetLastError();
}

namespace {
// kLinear's slices are kPlain's: what follows the sums is the join's
template <int WM, int WN, int E>
void tile_go(const IntParams& p, const TileGrid& g, const Epilogue<E>& ep, unsigned blocks, hipStream_t st) {
  if (g.slices > 1) {
    if constexpr (E == kGated) integer_tile_kernel<WM, WN, kOutPart, E><<<blocks, 256, 0, st>>>(p, g, ep);
    else integer_tile_kernel<WM, WN, kOutPart, kPlain><<<blocks, 256, 0, st>>>(p, g, {});
  } else if (p.y_bf16) {
    integer_tile_kernel<WM, WN, kOutBf16, E><<<blocks, 256, 0, st>>>(p, g, ep);
  } else {
    integer_tile_kernel<WM, WN, kOutF32, E><<<blocks, 256, 0, st>>>(p, g, ep);
  }
}
size_t up256(size_t v) { return (v + 255) & ~size_t{255}; }
}  // namespace

namespace {
size_t plan_workspace(const IntPlan& plan, int64_t m, int64_t d_in, bool codes_given) {
  const size_t part = up256(plan.partial_bytes);
  return codes_given || fuses(m, d_in) ? part : part + up256(static_cast<size_t>(m) * d_in) + 2 * up256(static_cast<size_t>(m) * 4);
}
}  // namespace

// workspace: the K slices' sums, then (x not given as codes) codes, scales and sums
size_t integer_matmul_workspace(int64_t m, int64_t d_in, int64_t d_out, bool codes_given, int n_cu) {
  return plan_workspace(int_plan(m, d_in, d_out, n_cu), m, d_in, codes_given);
}

bool integer_reads_x(int64_t m, int64_t d_in, bool codes_given) { return codes_given || fuses(m, d_in); }

namespace {
// The launches of a product whose x, layer and y stand in p (x in codes, or
// FUSED: raw); rows: of all weights that it reads.
template <int E>
hipError_t product_go(const IntParams& p, const IntPlan& plan, const Epilogue<E>& ep, int f, int64_t rows, int32_t* partial,
                      int n_cu, hipStream_t st) {
  if (plan.kind == 0) {
    // Sixteen tokens through 28672 x 8192: 53 us with the codes in LDS, 63 us with
    // four row blocks that share them.  With fewer row blocks than four a CU it
    // is no faster (11008 x 4096: 17.5 against 16.5 us): the codes are read once
    // a workgroup, and the CUs that have one row block more than the others end late.
    if (f == 0 && p.m <= 16 && p.m * (p.d_in + 16) <= kResidentBytes && rows >= 64ll * n_cu) {
      integer_resident_kernel<E><<<static_cast<unsigned>(n_cu), 64 * kRW,
                                   static_cast<size_t>(p.m * (p.d_in + 16)), st>>>(p, ep);
      return hipGetLastError();
    }
    const int r = stream_rows(p.m, p.d_in, rows, f != 0, E == kGated, n_cu);
    if (r == 4) stream_go<4, E>(p, ep, f, st);
    else if (r == 2) stream_go<2, E>(p, ep, f, st);
    else stream_go<1, E>(p, ep, f, st);
    return hipGetLastError();
  }
  const int64_t edge = plan.kind == 2 ? 256 : 128, high = plan.kind == 3 ? 64 : edge;
  TileGrid g{};
  g.nm = static_cast<int32_t>((p.m + high - 1) / high);
  g.nn = static_cast<int32_t>((rows + edge - 1) / edge);
  g.slices = plan.slices;
  g.per = plan.per;
  g.partial = partial;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(g.nm) * g.nn * g.slices);
  if (plan.kind == 2) tile_go<4, 4, E>(p, g, ep, blocks, st);
  else if (plan.kind == 3) tile_go<1, 2, E>(p, g, ep, blocks, st);
  else tile_go<2, 2, E>(p, g, ep, blocks, st);
  if (g.slices > 1) {
    const unsigned along = static_cast<unsigned>(std::min<int64_t>(p.m, 32768));
    if (p.d_out % 4 == 0)
      integer_join_kernel<4, E><<<dim3(static_cast<unsigned>((p.d_out / 4 + 255) / 256), along), 256, 0, st>>>(p, g, ep);
    else
      integer_join_kernel<1, E><<<dim3(static_cast<unsigned>((p.d_out + 255) / 256), along), 256, 0, st>>>(p, g, ep);
  }
  return hipGetLastError();
}
}  // namespace

hipError_t integer_launch(const IntCall& c, void* ws, size_t ws_bytes, int n_cu, hipStream_t st, bool* fits) {
  const bool gated = c.up.w != nullptr;
  const int64_t rows = gated ? 2 * c.d_out : c.d_out;
  const IntPlan plan = int_plan(c.m, c.d_in, rows, n_cu);
  const size_t need = plan_workspace(plan, c.m, c.d_in, c.xt == kXInt8);
  *fits = need == 0 || (ws && ws_bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0);
  if (!*fits) return hipSuccess;
  IntParams p{};
  p.x = static_cast<const int8_t*>(c.x);
  p.ldx = c.ldx;
  const bool offsets = c.layer.offsets || c.up.offsets;
  p.x_scales = c.x_scales;
  p.x_sums = offsets ? c.x_sums : nullptr;
  const int64_t vec = c.xt == kXBf16 ? 8 : 4;
  const bool fused = c.xt != kXInt8 && fuses(c.m, c.d_in);
  if (fused) {
    p.xraw = c.x;
    p.ldxraw = c.ldx;
    p.xvec = c.ldx % vec == 0 && (reinterpret_cast<uintptr_t>(c.x) & 15u) == 0;
  } else if (c.xt != kXInt8) {
    uint8_t* b = static_cast<uint8_t*>(ws) + up256(plan.partial_bytes);
    int8_t* codes = reinterpret_cast<int8_t*>(b);
    float* sc = reinterpret_cast<float*>(b + up256(static_cast<size_t>(c.m) * c.d_in));
    int32_t* sm = reinterpret_cast<int32_t*>(b + up256(static_cast<size_t>(c.m) * c.d_in) + up256(static_cast<size_t>(c.m) * 4));
    const hipError_t e = token_codes_launch(c.x, c.xt == kXBf16, c.m, c.d_in, c.ldx, codes, sc, offsets ? sm : nullptr, st);
    if (e != hipSuccess) return e;
    p.x = codes;
    p.ldx = c.d_in;
    p.x_scales = sc;
    p.x_sums = offsets ? sm : nullptr;
  }
  p.w = c.layer.w;
  p.w_scales = c.layer.scales;
  p.w_offsets = c.layer.offsets;
  p.y = c.y;
  p.m = c.m;
  p.d_out = c.d_out;
  p.d_in = static_cast<int32_t>(c.d_in);
  p.y_bf16 = c.y_bf16 ? 1 : 0;
  const auto whole = [](const void* at, bool bf16) { return (reinterpret_cast<uintptr_t>(at) & (bf16 ? 7u : 15u)) == 0; };
  p.yvec = c.d_out % 4 == 0 && whole(c.y, c.y_bf16) && (!c.res || (c.ldr % 4 == 0 && whole(c.res, c.res_bf16)));
  const int f = !fused ? 0 : c.xt == kXBf16 ? 1 : 2;
  int32_t* partial = static_cast<int32_t*>(ws);
  if (gated) {
    const Epilogue<kGated> ep{c.up.w, c.up.scales, c.up.offsets, c.layer.bias, c.up.bias, c.act};
    return product_go<kGated>(p, plan, ep, f, rows, partial, n_cu, st);
  }
  if (c.layer.bias || c.res || c.act != kActNone) {
    const Epilogue<kLinear> ep{c.layer.bias, c.res, c.ldr, c.act, c.res_bf16 ? 1 : 0};
    return product_go<kLinear>(p, plan, ep, f, rows, partial, n_cu, st);
  }
  return product_go<kPlain>(p, plan, {}, f, rows, partial, n_cu, st);
}

}  // namespace gptq
