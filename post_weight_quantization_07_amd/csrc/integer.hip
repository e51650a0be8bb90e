// Product of a quantized layer in 8-bit integers: a scale per token for the
// activations and a scale per output channel for the weights.
//
//   y[t, n] = sx[t] sw[n] (sum_k cx[t, k] cw[n, k] - off[n] sum_k cx[t, k])
//
// cx are the codes of x's rows (quant_row.h), cw the layer's codes shifted
// into int8, off its zero points shifted the same way (absent: symmetric).
// Every sum is a 32-bit integer and exact: d_in <= 65536 keeps both below
// 2^30 in magnitude and their difference below 2^31.  The only roundings are the conversion of the sum to
// fp32, the two scales and the store.
#include "gptq_common.h"
#include "gptq_internal.h"
#include "quant_row.h"

#include <algorithm>

namespace gptq {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4_t;
typedef __attribute__((__vector_size__(16 * sizeof(int)))) int i32x16_t;
typedef __attribute__((address_space(3))) void lds_void_t;

// ------------------------------------------------------------ token codes --
// T threads per row (T = 64: four rows a workgroup), a row of up to 32 T
// values in registers between the maximum and the codes, so x is read once;
// longer rows are read a second time (from the caches).  VEC: rows are
// 16-byte aligned and d a multiple of 8.  Bound: HBM (x read, codes written).
constexpr int kChunks = 4;

template <bool BF16, bool VEC>
GPTQ_DEV void tok_load(const void* x, int64_t row0, int64_t e, int64_t d, float (&v)[8]) {
  if (VEC) {
    if (e < d) {
      load8<BF16>(x, row0 + e, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (e + i < d) ? load1<BF16>(x, row0 + e + i) : 0.f;
  }
}

template <bool VEC>
GPTQ_DEV int tok_store(int8_t* codes, int64_t at, int64_t e, int64_t d, const float (&v)[8], const RowScale& rs) {
  uint32_t w[2] = {0u, 0u};
  int sum = 0;
  if (e >= d) return 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = static_cast<int>(row_code<127>(v[i], rs));
    sum += c;
    w[i >> 2] |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * (i & 3));
  }
  if (VEC) {
    *reinterpret_cast<uint2*>(codes + at + e) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < d) codes[at + e + i] = static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
  return sum;
}

template <int T, bool BF16, bool VEC>
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
  const bool held = d <= static_cast<int64_t>(T) * 8 * kChunks;
  float v[kChunks][8];
  uint32_t am = 0u;
  if (held) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) tok_load<BF16, VEC>(x, x0, (static_cast<int64_t>(c) * T + t) * 8, d, v[c]);
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
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
    for (int c = 0; c < kChunks; ++c) sum += tok_store<VEC>(codes, c0, (static_cast<int64_t>(c) * T + t) * 8, d, v[c], rs);
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

template <int T>
void token_codes_go(const void* x, bool bf16, bool vec, int64_t m, int64_t d, int64_t ldx, int8_t* codes, float* scales,
                    int32_t* sums, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(T == 64 ? (m + 3) / 4 : m));
  const int b = T == 64 ? 256 : T;
  if (bf16 && vec) token_codes_kernel<T, true, true><<<grid, b, 0, st>>>(x, m, d, ldx, codes, scales, sums);
  else if (bf16) token_codes_kernel<T, true, false><<<grid, b, 0, st>>>(x, m, d, ldx, codes, scales, sums);
  else if (vec) token_codes_kernel<T, false, true><<<grid, b, 0, st>>>(x, m, d, ldx, codes, scales, sums);
  else token_codes_kernel<T, false, false><<<grid, b, 0, st>>>(x, m, d, ldx, codes, scales, sums);
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
};

GPTQ_DEV void int_store(const IntParams& p, int64_t row, int64_t col, int acc, int off, float sw) {
  if (p.w_offsets) acc -= off * p.x_sums[row];
  const float v = (static_cast<float>(acc) * p.x_scales[row]) * sw;
  if (p.y_bf16)
    static_cast<uint16_t*>(p.y)[row * p.d_out + col] = f32_to_bf16(v);
  else
    static_cast<float*>(p.y)[row * p.d_out + col] = v;
}

// Few tokens: the weights are streamed once.  A workgroup owns 16 output
// channels, its four waves take turns of 256 k, and each 16x16x64 product
// takes its 16 weight rows straight from global memory (16 bytes a lane) and
// the tokens' codes from the caches.  The waves' sums meet in LDS.
template <int MT>
__global__ __launch_bounds__(256) void integer_stream_kernel(IntParams p) {
  constexpr int kNW = 4, kU = 4;  // waves; 64-byte steps per turn
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 16 * MT;
  const int8_t* wrow = p.w + min(n0 + c, p.d_out - 1) * p.d_in;
  const int8_t* xrow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xrow[i] = p.x + min(t0 + 16 * i + c, p.m - 1) * p.ldx;
  i32x4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = i32x4_t{0, 0, 0, 0};
  const i32x4_t zero = {0, 0, 0, 0};
  for (int k0 = wave * 64 * kU; k0 < p.d_in; k0 += kNW * 64 * kU) {
    i32x4_t b[kU], a[kU][MT];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = k0 + 64 * u + 16 * g;
      const bool in = k < p.d_in;
      b[u] = in ? *reinterpret_cast<const i32x4_t*>(wrow + k) : zero;
#pragma unroll
      for (int i = 0; i < MT; ++i) a[u][i] = in ? *reinterpret_cast<const i32x4_t*>(xrow[i] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][i], b[u], acc[i], 0, 0, 0);
  }
  __shared__ int part[kNW][MT][16][17];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][i][4 * g + r][c] = acc[i][r];
  __syncthreads();
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  const int64_t col = n0 + tc;
  if (col >= p.d_out) return;
  const float sw = p.w_scales[col];
  const int off = p.w_offsets ? p.w_offsets[col] : 0;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = t0 + 16 * i + tr;
    if (row >= p.m) break;
    int s = 0;
#pragma unroll
    for (int w = 0; w < kNW; ++w) s += part[w][i][tr][tc];
    int_store(p, row, col, s, off, sw);
  }
}

}  // namespace

hipError_t token_codes_launch(const void* x, bool bf16, int64_t m, int64_t d, int64_t ldx, int8_t* codes, float* scales,
                              int32_t* sums, hipStream_t st) {
  const int64_t e = bf16 ? 8 : 4;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (reinterpret_cast<uintptr_t>(codes) & 7u) == 0 &&
                   ldx % e == 0 && d % 8 == 0;
  if (d <= 64 * 8 * kChunks) token_codes_go<64>(x, bf16, vec, m, d, ldx, codes, scales, sums, st);
  else if (d <= 256 * 8 * kChunks) token_codes_go<256>(x, bf16, vec, m, d, ldx, codes, scales, sums, st);
  else token_codes_go<1024>(x, bf16, vec, m, d, ldx, codes, scales, sums, st);
  return hipGetLastError();
}

hipError_t integer_weight_launch(const int32_t* qweight, const int32_t* zeros, int bits, int64_t d_in, int64_t d_out,
                                 int8_t* w, int32_t* offsets, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((d_out + 255) / 256), static_cast<unsigned>(std::min<int64_t>(d_in / 32, 32768)));
  integer_weight_kernel<<<grid, 256, 0, st>>>(qweight, zeros, bits, d_in, d_out, w, offsets);
  return hipGetLastError();
}

size_t integer_matmul_workspace(int64_t m, int64_t d_in, int64_t d_out, bool codes_given, int n_cu) {
  if (codes_given) return 0;
  auto up = [](size_t v) { return (v + 255) & ~size_t{255}; };
  return up(static_cast<size_t>(m) * d_in) + 2 * up(static_cast<size_t>(m) * 4);
}

hipError_t integer_matmul_launch(const void* x, int xt, const float* x_scales, const int32_t* x_sums, int64_t m,
                                 int64_t d_in, int64_t ldx, const int8_t* w, const float* w_scales,
                                 const int32_t* w_offsets, int64_t d_out, void* y, bool y_bf16, void* ws, int n_cu,
                                 hipStream_t st) {
  IntParams p;
  p.x = static_cast<const int8_t*>(x);
  p.ldx = ldx;
  p.x_scales = x_scales;
  p.x_sums = x_sums;
  if (xt != kXInt8) {
    auto up = [](size_t v) { return (v + 255) & ~size_t{255}; };
    uint8_t* b = static_cast<uint8_t*>(ws);
    int8_t* codes = reinterpret_cast<int8_t*>(b);
    float* sc = reinterpret_cast<float*>(b + up(static_cast<size_t>(m) * d_in));
    int32_t* sm = reinterpret_cast<int32_t*>(b + up(static_cast<size_t>(m) * d_in) + up(static_cast<size_t>(m) * 4));
    const hipError_t e = token_codes_launch(x, xt == kXBf16, m, d_in, ldx, codes, sc, w_offsets ? sm : nullptr, st);
    if (e != hipSuccess) return e;
    p.x = codes;
    p.ldx = d_in;
    p.x_scales = sc;
    p.x_sums = sm;
  }
  p.w = w;
  p.w_scales = w_scales;
  p.w_offsets = w_offsets;
  p.y = y;
  p.m = m;
  p.d_out = d_out;
  p.d_in = static_cast<int32_t>(d_in);
  p.y_bf16 = y_bf16 ? 1 : 0;
  const unsigned gx = static_cast<unsigned>((d_out + 15) / 16);
  if (m <= 16) integer_stream_kernel<1><<<dim3(gx, 1), 256, 0, st>>>(p);
  else integer_stream_kernel<2><<<dim3(gx, static_cast<unsigned>((m + 31) / 32)), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace gptq
