// Residual add + RMS norm, written out or quantized on the way (the operand of the projection that
// follows it in a transformer block).
//
//   r = bf16(x + res)                      the residual stream, held in 16 bits
//   y = bf16(r * (1 / sqrt(mean(r^2) + eps)) * w)
//
// The sum of squares and both products are binary32; y is rounded once, and what is quantized is y,
// so the codes are those of osc_quant_act_multi on osc_rmsnorm's output, bit for bit.
//
// HBM-bound: x and res are read once and r, the codes and scales written once; the row stays in
// registers between the sum and the quantization, so nothing is read twice.  A lane holds 8 channels at a
// time, neighbours side by side, so that every load and store instruction covers whole contiguous lines.
// A row takes the four wavefronts of a workgroup, which meet in LDS once for its sum.  (A row a wavefront,
// without the barrier, leaves a lane eight times the arithmetic of a 4096-wide row one after the other and
// fewer wavefronts to overlap it: 4096 rows of 4096 into E4M3 take 33.3 us that way, 23.2 to 25.3 this way at 4.7
// to 5.1 TB/s, 16 rows into E2M1 8.6 and 3.7; 1537 rows of 8192 take 17.1 to 18.)  All streams are read or written once and go past the caches' residents.
#include "osc_quant_blk.h"

namespace osc {
namespace {

constexpr int kPlainOut = -1;  // FMT: y itself, row-major bf16

__device__ __forceinline__ float bf_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const bf2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// NC chunks of 8 channels a lane (H <= 2048 * NC)
template <int G, int FMT, int MODE, int M, int NC>
__global__ __launch_bounds__(256) void k_rmsnorm(const u4* __restrict__ X, const u4* RES, const u4* __restrict__ W,
                                                 int rows, int H, float eps, TableArg tab, u4* ROUT,
                                                 uint8_t* __restrict__ Q, uint8_t* __restrict__ SC,
                                                 uint16_t* __restrict__ side) {
  __shared__ float part[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = blockIdx.x;
  const int c0 = threadIdx.x;
  constexpr int STEP = 256;
  const int chunks = H >> 3;
  const long row = (long)r * chunks;
  u4 x[NC], w[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    x[i] = u4{0, 0, 0, 0};
    if (c0 + i * STEP < chunks) x[i] = __builtin_nontemporal_load(X + row + c0 + i * STEP);
  }
  if (RES) {
    u4 t[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (c0 + i * STEP < chunks) t[i] = __builtin_nontemporal_load(RES + row + c0 + i * STEP);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (c0 + i * STEP < chunks) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = pack_bf(bf_lo(x[i][j]) + bf_lo(t[i][j]), bf_hi(x[i][j]) + bf_hi(t[i][j]));
        __builtin_nontemporal_store(x[i], ROUT + row + c0 + i * STEP);  // read by this lane: ROUT may be RES
      }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (c0 + i * STEP < chunks) w[i] = W[c0 + i * STEP];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = bf_lo(x[i][j]), hi = bf_hi(x[i][j]);
      sum = __builtin_fmaf(lo, lo, sum);
      sum = __builtin_fmaf(hi, hi, sum);
    }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  sum = part[0] + part[1] + part[2] + part[3];
  const float rstd = 1.0f / __builtin_sqrtf(sum / (float)H + eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * STEP;
    if (c < chunks) {
      u4 y;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = pack_bf(bf_lo(x[i][j]) * rstd * bf_lo(w[i][j]), bf_hi(x[i][j]) * rstd * bf_hi(w[i][j]));
      if constexpr (FMT == kPlainOut) reinterpret_cast<u4*>(Q)[row + c] = y;
      else quant_chunk<G, FMT, MODE, M>(y, r, c * 8, rows, tab, Q, SC, side);
    }
  }
}

struct NormCall {
  const u4 *x, *res, *w;
  int rows, H;
  float eps;
  const TableArg* tab;
  u4* rout;
  uint8_t *q, *sc;
  uint16_t* side;
  hipStream_t st;
};

template <int G, int FMT, int MODE, int M>
hipError_t launch_shape(const NormCall& c) {
#define OSC_NORM(NC)                                                                                             \
  hipLaunchKernelGGL((k_rmsnorm<G, FMT, MODE, M, NC>), dim3(c.rows), dim3(256), 0, c.st, c.x, c.res, c.w, c.rows, \
                     c.H, c.eps, *c.tab, c.rout, c.q, c.sc, c.side)
  // the registers of a lane follow the row's width: 24 dwords up to 4096 channels, 48 up to 8192
  if (c.H <= 4096) OSC_NORM(2);
  else if (c.H <= 8192) OSC_NORM(4);
  else if (c.H <= 16384) OSC_NORM(8);
  else OSC_NORM(32);
#undef OSC_NORM
  return hipGetLastError();
}

template <int G, int FMT>
hipError_t launch_table(const NormCall& c, bool table, int m) {
  if constexpr (FMT == OSC_MXFP4 || FMT == OSC_FP6P) {
    if (table) switch (m) {
        case 1: return launch_shape<G, FMT, kExtractZero, 1>(c);
        case 2: return launch_shape<G, FMT, kExtractZero, 2>(c);
        default: return launch_shape<G, FMT, kExtractZero, 3>(c);
      }
  }
  if (table) return hipErrorInvalidValue;
  return launch_shape<G, FMT, kNoTable, 1>(c);
}

template <int G>
hipError_t launch_fmt(const NormCall& c, bool table, int m, osc_fmt fmt) {
  if (fmt == OSC_FP6P) {
    if constexpr (G == 16) return launch_table<16, OSC_FP6P>(c, table, m);
    return hipErrorInvalidValue;  // E3M2 pairs exist for G = 16 only
  }
  return fmt == OSC_MXFP4 ? launch_table<G, OSC_MXFP4>(c, table, m) : launch_table<G, OSC_MXFP8>(c, table, m);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st) {
  static const TableArg empty = {};
  const NormCall c{static_cast<const u4*>(a.X), static_cast<const u4*>(a.RES), static_cast<const u4*>(a.W), a.S, a.H,
                   a.eps, a.tab ? a.tab : &empty, static_cast<u4*>(a.RES_OUT), static_cast<uint8_t*>(a.QX), a.SX,
                   static_cast<uint16_t*>(a.B), st};
  if (!a.SX) return launch_shape<32, kPlainOut, kNoTable, 1>(c);  // y written out (QX is its buffer)
  switch (a.G) {
    case 16: return launch_fmt<16>(c, a.tab != nullptr, a.m, a.afmt);
    case 32: return launch_fmt<32>(c, a.tab != nullptr, a.m, a.afmt);
    default: return launch_fmt<64>(c, a.tab != nullptr, a.m, a.afmt);
  }
}

}  // namespace osc
