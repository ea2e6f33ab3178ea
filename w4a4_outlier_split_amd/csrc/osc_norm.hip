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
// registers between the sum and the quantization (16 to 64 registers a lane), so nothing is read
// twice.  A lane holds 32-channel blocks, as the block encoder wants them (a quad of lanes is one
// row's 128-channel panel); the row's sum crosses the lanes of a wavefront and then the four
// wavefronts of the workgroup through LDS.
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

// ROWS rows a workgroup of four wavefronts: a wavefront instruction covers ROWS rows x 16 / ROWS
// panels, a sweep of the workgroup 64 / ROWS panels; NS sweeps cover the row (H <= NS * 8192 / ROWS).
template <int G, int FMT, int MODE, int M, int ROWS, int NS>
__global__ __launch_bounds__(256) void k_rmsnorm(const u4* __restrict__ X, const u4* RES, const u4* __restrict__ W,
                                                 int rows, int H, float eps, TableArg tab, u4* ROUT,
                                                 uint8_t* __restrict__ Q, uint8_t* __restrict__ SC,
                                                 uint16_t* __restrict__ side) {
  constexpr int PW = 16 / ROWS;  // panels of a wavefront
  __shared__ float part[4][ROWS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b = lane & 3;
  const int lr = (lane >> 2) & (ROWS - 1);
  const int r = blockIdx.x * ROWS + lr;
  const int p0 = wave * PW + (lane >> 2) / ROWS;
  const int npan = H >> 7;
  uint32_t x[NS][16], w[NS][16];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int p = p0 + s * 4 * PW;
    if (r < rows && p < npan) {
      const long at = ((long)r * H + p * 128 + b * 32) >> 3;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const u4 t = X[at + c];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[s][4 * c + i] = t[i];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[s][j] = 0;
    }
  }
  if (RES) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int p = p0 + s * 4 * PW;
      if (r < rows && p < npan) {
        const long at = ((long)r * H + p * 128 + b * 32) >> 3;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const u4 t = RES[at + c];
          u4 o;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = x[s][4 * c + i] =
                pack_bf(bf_lo(x[s][4 * c + i]) + bf_lo(t[i]), bf_hi(x[s][4 * c + i]) + bf_hi(t[i]));
          ROUT[at + c] = o;  // the lane that read the place writes it: ROUT may be RES
        }
      }
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float lo = bf_lo(x[s][j]), hi = bf_hi(x[s][j]);
      sum = __builtin_fmaf(lo, lo, sum);
      sum = __builtin_fmaf(hi, hi, sum);
    }
  // lanes of one row: bits 0-1 (the quad) and the bits above the row's
  sum += __shfl_xor(sum, 1);
  sum += __shfl_xor(sum, 2);
#pragma unroll
  for (int d = 4 * ROWS; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if (b == 0 && (lane >> 2) < ROWS) part[wave][lr] = sum;
  __syncthreads();
  const float rstd =
      1.0f / __builtin_sqrtf((part[0][lr] + part[1][lr] + part[2][lr] + part[3][lr]) / (float)H + eps);
  if (r >= rows) return;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int p = p0 + s * 4 * PW;
    if (p < npan) {
      const long wat = (p * 128 + b * 32) >> 3;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const u4 t = W[wat + c];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[s][4 * c + i] = t[i];
      }
    }
  }
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int p = p0 + s * 4 * PW;
    if (p < npan) {
      uint32_t y[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        y[j] = pack_bf(bf_lo(x[s][j]) * rstd * bf_lo(w[s][j]), bf_hi(x[s][j]) * rstd * bf_hi(w[s][j]));
      if constexpr (FMT == kPlainOut) {
        u4* out = reinterpret_cast<u4*>(Q) + (((long)r * H + p * 128 + b * 32) >> 3);
#pragma unroll
        for (int c = 0; c < 4; ++c) out[c] = u4{y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]};
      } else {
        quant_block<G, FMT, MODE, M>(y, r, p, b, rows, tab, Q, SC, side);
      }
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
#define OSC_NORM(ROWS, NS)                                                                                       \
  hipLaunchKernelGGL((k_rmsnorm<G, FMT, MODE, M, ROWS, NS>), dim3((c.rows + ROWS - 1) / ROWS), dim3(256), 0, c.st, \
                     c.x, c.res, c.w, c.rows, c.H, c.eps, *c.tab, c.rout, c.q, c.sc, c.side)
  if (c.H <= 8192 && c.rows >= 2048) {
    if (c.H <= 4096) OSC_NORM(4, 2);
    else OSC_NORM(4, 4);
  } else if (c.H <= 8192) {
    OSC_NORM(1, 1);
  } else {
    OSC_NORM(1, 8);
  }
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
