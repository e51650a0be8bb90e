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
  if (e >= d) return 0;
  uint32_t w[2];
  row_codes<127, 0>(v, rs, w);
  const int sum = __builtin_amdgcn_sdot4(w[0], 0x01010101, __builtin_amdgcn_sdot4(w[1], 0x01010101, 0, false), false);
  if (VEC) {
    *reinterpret_cast<uint2*>(codes + at + e) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < d) codes[at + e + i] = static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
  return sum;
}

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
};

GPTQ_DEV void int_put(const IntParams& p, int64_t row, int64_t col, float v) {
  if (p.y_bf16)
    static_cast<uint16_t*>(p.y)[row * p.d_out + col] = f32_to_bf16(v);
  else
    static_cast<float*>(p.y)[row * p.d_out + col] = v;
}
GPTQ_DEV void int_store(const IntParams& p, int64_t row, int64_t col, int acc, int off, float sw) {
  if (p.w_offsets) acc -= off * p.x_sums[row];
  int_put(p, row, col, (static_cast<float>(acc) * p.x_scales[row]) * sw);
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
// 12 to 15), 8192 x 28672 57 us, 4.1 TB/s.  32 and 64 tokens of 11008 x 4096: 22 and 30 us.
// FUSED (one to four tokens): x is quantized here, by every workgroup for
// itself and into LDS, while its first weights are on their way: one launch, and
// reading the tokens again from L2 costs less than a second one (4096 x 4096: 7.2 us
// against 6.5 + 4.2).
constexpr int kSW = 8;                // waves
constexpr int kFusedElems = 16384;    // tokens * d_in at most

template <int R, int MT, int FUSED>  // FUSED: 0 codes given, 1 bf16, 2 fp32
__global__ __launch_bounds__(64 * kSW, 2) void integer_stream_kernel(IntParams p) {
  constexpr int kU = R == 1 && MT == 1 ? 8 : R == 4 || MT == 4 ? 2 : 4;
  constexpr int kTurn = kSW * 64 * kU;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16 * R;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 16 * MT;
  const int8_t* wrow[R];
#pragma unroll
  for (int j = 0; j < R; ++j) wrow[j] = p.w + min(n0 + 16 * j + c, p.d_out - 1) * p.d_in + 16 * g;
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
  load_w(wave * 64 * kU, b);

  __shared__ __attribute__((aligned(16))) int8_t xl[FUSED ? kFusedElems : 16];
  __shared__ float xs[4];
  __shared__ int xsum[4];
  if (FUSED) {
    constexpr bool kBf16 = FUSED == 1;
    __shared__ uint32_t red[kSW];
    __shared__ int redsum[kSW];
    const int chunks = p.d_in / 8;
    for (int t = 0; t < static_cast<int>(p.m); ++t) {
      constexpr int kQ = kFusedElems / 8 / (64 * kSW);  // chunks a thread, at most
      float v[kQ][8];
      uint32_t am = 0u;
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const int e = q * 64 * kSW + static_cast<int>(threadIdx.x);
        if (e < chunks && p.xvec) {
          load8<kBf16>(p.xraw, t * p.ldxraw + 8 * e, v[q]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[q][i] = e < chunks ? load1<kBf16>(p.xraw, t * p.ldxraw + 8 * e + i) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) am = max(am, abs_bits(v[q][i]));
      }
      am = group_max<64>(am);
      if (lane == 0) red[wave] = am;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kSW; ++w) am = max(am, red[w]);
      const RowScale rs = row_scale(am, 127.f);
      int sum = 0;
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const int e = q * 64 * kSW + static_cast<int>(threadIdx.x);
        if (e < chunks) sum += tok_store<true>(xl, static_cast<int64_t>(t) * p.d_in, 8 * e, p.d_in, v[q], rs);
      }
      sum = group_sum<64>(sum);
      if (lane == 0) redsum[wave] = sum;
      __syncthreads();
      if (threadIdx.x == 0) {
        int all = 0;
#pragma unroll
        for (int w = 0; w < kSW; ++w) all += redsum[w];
        xs[t] = rs.scale;
        xsum[t] = all;
      }
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
    load_w(k0 + kTurn, next);
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][i], b[u][j], acc[j][i], 0, 0, 0);
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
  for (int e = threadIdx.x; e < R * MT * 256; e += 64 * kSW) {
    const int tc = e & 15, j = (e >> 4) % R, tr = (e / (16 * R)) & 15, i = e / (256 * R);
    const int64_t col = n0 + 16 * j + tc, row = t0 + 16 * i + tr;
    if (col >= p.d_out || row >= p.m) continue;
    int s = 0;
#pragma unroll
    for (int w = 0; w < kSW; ++w) s += part[w][j][i][tr][tc];
    const int off = p.w_offsets ? p.w_offsets[col] : 0;
    const float sw = p.w_scales[col];
    if (FUSED) int_put(p, row, col, (static_cast<float>(s - off * xsum[tr & 3]) * xs[tr & 3]) * sw);
    else int_store(p, row, col, s, off, sw);
  }
}

// Some tokens (up to sixteen) and many channels: as above, but the codes lie in LDS, once for a
// workgroup that walks over the row blocks, so that only weights are loaded.
// Sixteen waves split K; the sums meet in LDS by integer atomics (any order
// gives the same), in one of two buffers by turns: a buffer is read and cleared
// between the barriers of its row block and of the next one.
constexpr int kRW = 16, kRU = 4;
constexpr int64_t kResidentBytes = 152 * 1024;  // codes, 16 bytes of padding a row (bank conflicts)

__global__ __launch_bounds__(64 * kRW, 4) void integer_resident_kernel(IntParams p) {
  constexpr int kTurn = kRW * 64 * kRU;
  extern __shared__ __attribute__((aligned(16))) int8_t xr[];  // [m][d_in + 16]
  __shared__ int sum[2][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int blocks = static_cast<int>((p.d_out + 15) / 16), m = static_cast<int>(p.m);
  const int k_first = wave * 64 * kRU + 16 * g;
  const i32x4_t zero = {0, 0, 0, 0};
  auto load_w = [&](int rb, int k0, i32x4_t (&b)[kRU]) {
    const int8_t* w = p.w + min(static_cast<int64_t>(rb) * 16 + c, p.d_out - 1) * p.d_in;
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
        const int64_t col = static_cast<int64_t>(rb) * 16 + tc;
        const int s = sum[buf][tr][tc];
        sum[buf][tr][tc] = 0;
        if (col < p.d_out && tr < m) int_store(p, tr, col, s, p.w_offsets ? p.w_offsets[col] : 0, p.w_scales[col]);
      }
      buf ^= 1;
    }
    rb = nrb;
    k0 = nk;
#pragma unroll
    for (int u = 0; u < kRU; ++u) b[u] = next[u];
  }
}

template <int R>
void stream_go(const IntParams& p, int fused, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((p.d_out + 16 * R - 1) / (16 * R)));
  const int t = 64 * kSW;
  if (fused == 1) integer_stream_kernel<R, 1, 1><<<grid, t, 0, st>>>(p);
  else if (fused == 2) integer_stream_kernel<R, 1, 2><<<grid, t, 0, st>>>(p);
  else if (p.m <= 16) integer_stream_kernel<R, 1, 0><<<grid, t, 0, st>>>(p);
  else if (p.m <= 32) integer_stream_kernel<R, 2, 0><<<grid, t, 0, st>>>(p);
  else if constexpr (R <= 2) integer_stream_kernel<R, 4, 0><<<dim3(grid.x, static_cast<unsigned>((p.m + 63) / 64)), t, 0, st>>>(p);
}

// Many tokens: 64 WM x 64 WN output tiles on v_mfma_i32_32x32x32_i8, four waves
// of 32 WM x 32 WN each.  Rows of both operands are k-contiguous, so a 64-byte
// step of a tile goes to LDS by buffer_load ... lds as it lies in memory, through
// a ring of four steps, and the MFMA operands are 16-byte LDS reads.  Each half
// step's operands are read while the previous half's products run; one barrier
// a step publishes the next step's data and frees the slot read two halves ago.
// LDS rows are 64 bytes; 16-byte chunk c of row r sits at c ^ ((r >> 2) & 3), so
// 16 lanes that read one chunk of 16 rows touch all 64 banks once.
// Bound: the matrix cores, and the clock that they leave.  2048 x 28672 -> 8192 on
// 256 x 256 tiles: 409 us, 2.35 POP/s, the matrix cores busy 62% of the cycles.  Four waves of 128 x 128 read half the LDS
// bytes a product of 64 x 64; 128 x 128 tiles are for grids too small for the others
// (509 x 11008 -> 4096: 36 us in four K slices, 1.28 POP/s; an eight-step ring, one
// workgroup a CU, 38 us).
constexpr int kTStep = 64, kSlots = 4;

#define GPTQ_VMCNT(n) (((n) & 15) | (((n) >> 4) << 14) | 0x0F70)

GPTQ_DEV __amdgpu_buffer_rsrc_t rows_rsrc(const int8_t* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  const int n = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo),
                                           static_cast<short>(0), n, 0x00020000);
}

// one piece (16 rows x 64 bytes) of a step to LDS
GPTQ_DEV void tile_dma(__amdgpu_buffer_rsrc_t rs, uint8_t* piece, uint32_t voff, int kc, int k0, int d_in) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)piece, 16, (k0 + kc < d_in) ? voff + k0 : 0x80000000u, 0, 0,
                                           0);
}

template <int W>
GPTQ_DEV void tile_read(const uint8_t* op, uint32_t off, i32x4_t (&f)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) f[i] = *reinterpret_cast<const i32x4_t*>(op + off + i * 2048);
}

template <int WM, int WN>
GPTQ_DEV void tile_half(const i32x4_t (&a)[WM], const i32x4_t (&b)[WN], const uint8_t* nA, const uint8_t* nB,
                        uint32_t offA, uint32_t offB, i32x4_t (&na)[WM], i32x4_t (&nb)[WN], i32x16_t (&acc)[WM][WN]) {
  tile_read<WM>(nA, offA, na);
  tile_read<WN>(nB, offB, nb);
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
  // the next half's reads and this half's loads spread over the products
  constexpr int kProd = WM * WN / (WM + WN);
#pragma unroll
  for (int k = 0; k < WM + WN; ++k) {
    __builtin_amdgcn_sched_group_barrier(0x008, kProd, 0);                // products
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                    // one LDS read
    if ((k & 1) == 0) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // one load to LDS
  }
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

template <int WM, int WN, int OUT>
__global__ __launch_bounds__(256) void integer_tile_kernel(IntParams p, TileGrid g) {
  constexpr int kA = WM * 64 * kTStep, kB = WN * 64 * kTStep;
  // one array per slot: the compiler then sees that reads of one slot do not alias loads in flight into another
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[kA], sA1[kA], sA2[kA], sA3[kA];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[kB], sB1[kB], sB2[kB], sB3[kB];
  int tm, tn, slice;
  tile_of(g, static_cast<int>(blockIdx.x), tm, tn, slice);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = static_cast<int64_t>(tm) * (64 * WM), n0 = static_cast<int64_t>(tn) * (64 * WN);
  const int mrows = static_cast<int>(min(p.m - m0, int64_t{64 * WM}));
  const int nrows = static_cast<int>(min(p.d_out - n0, int64_t{64 * WN}));
  const __amdgpu_buffer_rsrc_t ra = rows_rsrc(p.x + m0 * p.ldx, (mrows - 1) * p.ldx + p.d_in);
  const __amdgpu_buffer_rsrc_t rb = rows_rsrc(p.w + n0 * p.d_in, static_cast<int64_t>(nrows) * p.d_in);
  const int kc = (((lane & 3) ^ ((lane >> 4) & 3)) * 16);
  uint32_t va[WM], vb[WN];
#pragma unroll
  for (int u = 0; u < WM; ++u) {
    const int row = (wave * WM + u) * 16 + (lane >> 2);
    va[u] = row < mrows ? static_cast<uint32_t>(row * static_cast<int>(p.ldx) + kc) : 0x80000000u;
  }
#pragma unroll
  for (int u = 0; u < WN; ++u) {
    const int row = (wave * WN + u) * 16 + (lane >> 2);
    vb[u] = row < nrows ? static_cast<uint32_t>(row * p.d_in + kc) : 0x80000000u;
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
  // steps past the slice's end load nothing (every lane out of range: zeros)
  auto issue_a = [&](int s, int slot) {
    const int k0 = s < steps ? (s0 + s) * kTStep : p.d_in;
#pragma unroll
    for (int u = 0; u < WM; ++u) tile_dma(ra, slotA(slot) + (wave * WM + u) * 1024, va[u], kc, k0, p.d_in);
  };
  auto issue_b = [&](int s, int slot) {
    const int k0 = s < steps ? (s0 + s) * kTStep : p.d_in;
#pragma unroll
    for (int u = 0; u < WN; ++u) tile_dma(rb, slotB(slot) + (wave * WN + u) * 1024, vb[u], kc, k0, p.d_in);
  };
  // operand reads: row l % 32 of a 32-row tile, chunk 2 half + l / 32
  const int r = lane & 31, hi = lane >> 5;
  uint32_t oa[2], ob[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t o = static_cast<uint32_t>(r * 64 + (((2 * h + hi) ^ ((r >> 2) & 3)) * 16));
    oa[h] = o + wm * WM * 2048;
    ob[h] = o + wn * WN * 2048;
  }
  i32x16_t acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  i32x4_t a0[WM], b0[WN], a1[WM], b1[WN];
  constexpr int kL = WM + WN;  // loads of one step, per wave
#pragma unroll
  for (int u = 0; u < kSlots - 1; ++u) {
    issue_a(u, u);
    issue_b(u, u);
  }
  __builtin_amdgcn_s_waitcnt(GPTQ_VMCNT((kSlots - 2) * kL));
  __builtin_amdgcn_s_barrier();
  tile_read<WM>(sA0, oa[0], a0);
  tile_read<WN>(sB0, ob[0], b0);
  // steps in blocks of a ring's length; the ones past the end multiply zeros
  for (int s = 0; s < steps; s += kSlots) {
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      __builtin_amdgcn_s_waitcnt(GPTQ_VMCNT((kSlots - 3) * kL));
      __builtin_amdgcn_s_barrier();
      issue_a(s + u + kSlots - 1, u + kSlots - 1);
      tile_half<WM, WN>(a0, b0, slotA(u), slotB(u), oa[1], ob[1], a1, b1, acc);
      issue_b(s + u + kSlots - 1, u + kSlots - 1);
      tile_half<WM, WN>(a1, b1, slotA(u + 1), slotB(u + 1), oa[0], ob[0], a0, b0, acc);
    }
  }
  // Element e of lane l: row 8 (e / 4) + 4 (l / 32) + e % 4, column l % 32.
  // Stores go through buffer resources over the tile's rows: rows past m and
  // columns past d_out (offset 2^31) are dropped in hardware.
  __builtin_amdgcn_s_waitcnt(GPTQ_VMCNT(0));  // the loads past the end still write LDS
  const int dout = static_cast<int>(p.d_out);
  const uint32_t row0 = static_cast<uint32_t>(wm * WM * 32 + 4 * hi);
  if (OUT == kOutPart) {
    const __amdgpu_buffer_rsrc_t rp =
        rows_rsrc(reinterpret_cast<int8_t*>(g.partial + (static_cast<int64_t>(slice) * p.m + m0) * p.d_out),
                  static_cast<int64_t>(mrows) * dout * 4);
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      const int col = static_cast<int>(n0) + (wn * WN + j) * 32 + r;
#pragma unroll
      for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t row = row0 + 32 * i + 8 * (e >> 2) + (e & 3);
          __builtin_amdgcn_raw_buffer_store_b32(acc[i][j][e], rp, col < dout ? (row * dout + col) * 4 : 0x80000000u, 0, 0);
        }
    }
    return;
  }
  __syncthreads();  // the operands' LDS now holds the tile's row scales and code sums
  float* lsc = reinterpret_cast<float*>(sA0);
  int* lsm = reinterpret_cast<int*>(sB0);
  for (int e = threadIdx.x; e < mrows; e += 256) {
    lsc[e] = p.x_scales[m0 + e];
    lsm[e] = p.w_offsets ? p.x_sums[m0 + e] : 0;
  }
  __syncthreads();
  constexpr int size = OUT == kOutBf16 ? 2 : 4;
  const __amdgpu_buffer_rsrc_t ry =
      rows_rsrc(static_cast<const int8_t*>(p.y) + m0 * p.d_out * size, static_cast<int64_t>(mrows) * dout * size);
#pragma unroll
  for (int j = 0; j < WN; ++j) {
    const int col = static_cast<int>(n0) + (wn * WN + j) * 32 + r;
    const float sw = col < dout ? p.w_scales[col] : 0.f;
    const int off = (col < dout && p.w_offsets) ? p.w_offsets[col] : 0;
    const uint32_t at = col < dout ? static_cast<uint32_t>(col * size) : 0x80000000u;
#pragma unroll
    for (int i = 0; i < WM; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t row = row0 + 32 * i + 8 * q;
        const f32x4_t sc = *reinterpret_cast<const f32x4_t*>(lsc + row);
        const i32x4_t sm = *reinterpret_cast<const i32x4_t*>(lsm + row);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = (static_cast<float>(acc[i][j][4 * q + e] - off * sm[e]) * sc[e]) * sw;
          const uint32_t to = at + (row + e) * static_cast<uint32_t>(dout * size);
          if (OUT == kOutBf16)
            __builtin_amdgcn_raw_buffer_store_b16(static_cast<short>(f32_to_bf16(v)), ry, to, 0, 0);
          else
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(v), ry, to, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// sums of the K slices (integers: any order gives the same), four columns a
// thread where rows are whole vectors.  Bound: the caches and HBM (four slices
// of 509 x 4096, 33 MB, in 10 us).
template <int V>
__global__ __launch_bounds__(256) void integer_join_kernel(IntParams p, TileGrid g) {
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
  for (int64_t row = blockIdx.y; row < p.m; row += gridDim.y) {
    ivec_t s = {};
    for (int k = 0; k < g.slices; ++k) s += *reinterpret_cast<const ivec_t*>(g.partial + (k * p.m + row) * p.d_out + col);
    const float sx = p.x_scales[row];
    const int sum = p.w_offsets ? p.x_sums[row] : 0;
#pragma unroll
    for (int j = 0; j < V; ++j) int_put(p, row, col + j, (static_cast<float>(s[j] - off[j] * sum) * sx) * sw[j]);
  }
}

// few tokens of few values: quantized by every workgroup of the stream kernel itself
bool fuses(int64_t m, int64_t d_in) { return m <= 4 && m * d_in <= kFusedElems; }

// row blocks a workgroup of the stream kernel takes: as many as leave every CU one
int stream_rows(int64_t m, int64_t d_out, int n_cu) {
  const int r = d_out >= 64ll * n_cu ? 4 : d_out >= 32ll * n_cu ? 2 : 1;
  return m > 32 ? std::min(r, 2) : r;
}

// The stream kernel reads the weights with less ado than the tiles do, but a
// workgroup's turns also load its tokens' codes.  What that costs, fitted to
// both kernels' times over 2 to 512 tokens and weights of 512 x 512 to
// 28672 x 8192: 1 us and 31 ps a token (of its padded block) and k, for each
// round of workgroups; against it the tiles' prologue, slices and join, 9.1 us and
// 65 ns per MB of weights.  (us, stream and tiles: 64 x 4096 -> 4096 14.0, 14.8;
// 100 of them 20.6, 15.8; 64 x 11008 -> 4096 30.7, 25.2; 24 of them 17.4, 22.9;
// 64 x 28672 -> 1024 71, 22; 256 x 2048 -> 2048 12.4, 13.5; 512 x 512 -> 512 4.4, 7.6.)
bool streams(int64_t m, int64_t d_in, int64_t d_out, int n_cu) {
  if (fuses(m, d_in)) return true;
  const int64_t rows = 16 * stream_rows(m, d_out, n_cu), pad = m <= 16 ? 16 : m <= 32 ? 32 : 64;
  const double blocks = static_cast<double>((d_out + rows - 1) / rows) * static_cast<double>((m + 63) / 64);
  const double extra = std::max(1.0, blocks / n_cu) * (1.0 + 31e-6 * static_cast<double>(pad * d_in));
  return extra <= 9.1 + 6.5e-8 * static_cast<double>(d_in) * static_cast<double>(d_out);
}

// The launch of a product: kernel, tile and K slices.
struct IntPlan {
  int kind;  // 0: stream, 1: 128 x 128 tiles, 2: 256 x 256
  int slices, per;
  size_t partial_bytes;
};

IntPlan int_plan(int64_t m, int64_t d_in, int64_t d_out, int n_cu) {
  IntPlan a{0, 1, 0, 0};
  if (streams(m, d_in, d_out, n_cu)) return a;
  // 256 x 256 tiles where they give more than half the CUs one, or where K is
  // long enough for slices of 2048 that do (1024 x 11008 -> 4096 in four slices: 70 us, 88
  // in 128 x 128 tiles; 2048 x 28672 -> 1024 in eight: 82 and 105; but 1024 x 1024 -> 4096: 23
  // and 11; 509 x 11008 -> 4096 with its codes and join, in eight slices of 1376: 53.2 and 52.0)
  const int64_t t256 = ((m + 255) / 256) * ((d_out + 255) / 256), t128 = ((m + 127) / 128) * ((d_out + 127) / 128);
  a.kind = t256 > n_cu / 2 || (d_in >= 8192 && m > 128 && t256 * 8 >= n_cu && t256 * d_in >= 2048ll * n_cu) ? 2 : 1;
  const int64_t tiles = a.kind == 2 ? t256 : t128;
  const int steps = static_cast<int>((d_in + kTStep - 1) / kTStep);
  const int64_t room = a.kind == 2 ? n_cu : 2 * n_cu;
  int64_t sl = std::max<int64_t>(1, room / tiles);
  sl = std::min<int64_t>(sl, std::max(1, steps / 16));
  a.per = static_cast<int>((steps + sl - 1) / sl);
  a.slices = (steps + a.per - 1) / a.per;
  if (a.slices > 1) a.partial_bytes = static_cast<size_t>(a.slices) * m * d_out * 4;
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
template <int WM, int WN>
void tile_go(const IntParams& p, const TileGrid& g, unsigned blocks, hipStream_t st) {
  if (g.slices > 1) integer_tile_kernel<WM, WN, kOutPart><<<blocks, 256, 0, st>>>(p, g);
  else if (p.y_bf16) integer_tile_kernel<WM, WN, kOutBf16><<<blocks, 256, 0, st>>>(p, g);
  else integer_tile_kernel<WM, WN, kOutF32><<<blocks, 256, 0, st>>>(p, g);
}
size_t up256(size_t v) { return (v + 255) & ~size_t{255}; }
}  // namespace

// workspace: the K slices' sums, then (x not given as codes) codes, scales and sums
size_t integer_matmul_workspace(int64_t m, int64_t d_in, int64_t d_out, bool codes_given, int n_cu) {
  const size_t part = up256(int_plan(m, d_in, d_out, n_cu).partial_bytes);
  return codes_given || fuses(m, d_in) ? part : part + up256(static_cast<size_t>(m) * d_in) + 2 * up256(static_cast<size_t>(m) * 4);
}

hipError_t integer_matmul_launch(const void* x, int xt, const float* x_scales, const int32_t* x_sums, int64_t m,
                                 int64_t d_in, int64_t ldx, const int8_t* w, const float* w_scales,
                                 const int32_t* w_offsets, int64_t d_out, void* y, bool y_bf16, void* ws, int n_cu,
                                 hipStream_t st) {
  const IntPlan plan = int_plan(m, d_in, d_out, n_cu);
  IntParams p{};
  p.x = static_cast<const int8_t*>(x);
  p.ldx = ldx;
  p.x_scales = x_scales;
  p.x_sums = x_sums;
  const int64_t vec = xt == kXBf16 ? 8 : 4;
  const bool fused = xt != kXInt8 && fuses(m, d_in);
  if (fused) {
    p.xraw = x;
    p.ldxraw = ldx;
    p.xvec = ldx % vec == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
  } else if (xt != kXInt8) {
    uint8_t* b = static_cast<uint8_t*>(ws) + up256(plan.partial_bytes);
    int8_t* codes = reinterpret_cast<int8_t*>(b);
    float* sc = reinterpret_cast<float*>(b + up256(static_cast<size_t>(m) * d_in));
    int32_t* sm = reinterpret_cast<int32_t*>(b + up256(static_cast<size_t>(m) * d_in) + up256(static_cast<size_t>(m) * 4));
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
  if (plan.kind == 0) {
    const int f = !fused ? 0 : xt == kXBf16 ? 1 : 2;
    // Sixteen tokens through 28672 x 8192: 53 us with the codes in LDS, 63 us with
    // four row blocks that share them.  With fewer row blocks than four a CU it
    // is no faster (11008 x 4096: 17.5 against 16.5 us): the codes are read once
    // a workgroup, and the CUs that have one row block more than the others end late.
    if (f == 0 && m <= 16 && m * (d_in + 16) <= kResidentBytes && d_out >= 64ll * n_cu) {
      integer_resident_kernel<<<static_cast<unsigned>(n_cu), 64 * kRW,
                                static_cast<size_t>(m * (d_in + 16)), st>>>(p);
      return hipGetLastError();
    }
    const int r = stream_rows(m, d_out, n_cu);
    if (r == 4) stream_go<4>(p, f, st);
    else if (r == 2) stream_go<2>(p, f, st);
    else stream_go<1>(p, f, st);
    return hipGetLastError();
  }
  const int64_t edge = plan.kind == 2 ? 256 : 128;
  TileGrid g{};
  g.nm = static_cast<int32_t>((m + edge - 1) / edge);
  g.nn = static_cast<int32_t>((d_out + edge - 1) / edge);
  g.slices = plan.slices;
  g.per = plan.per;
  g.partial = static_cast<int32_t*>(ws);
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(g.nm) * g.nn * g.slices);
  if (plan.kind == 2) tile_go<4, 4>(p, g, blocks, st);
  else tile_go<2, 2>(p, g, blocks, st);
  if (g.slices > 1) {
    const unsigned rows = static_cast<unsigned>(std::min<int64_t>(m, 32768));
    if (d_out % 4 == 0)
      integer_join_kernel<4><<<dim3(static_cast<unsigned>((d_out / 4 + 255) / 256), rows), 256, 0, st>>>(p, g);
    else
      integer_join_kernel<1><<<dim3(static_cast<unsigned>((d_out + 255) / 256), rows), 256, 0, st>>>(p, g);
  }
  return hipGetLastError();
}

}  // namespace gptq
