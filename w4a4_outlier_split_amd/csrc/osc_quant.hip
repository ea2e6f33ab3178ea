// Group quantization with outlier extraction (OSC page "W4A4量化技术：OSC框架如何实现高效LLM部署",
// §3.2: copy the table-indexed channel into B, zero it, scale the zeroed group, microscaling-
// quantize) and the offline weight preparation of §3.3 (same kernel, the indexed channel is
// copied into the contiguous W_L block without zeroing); E4M3 for the down-projection's input
// (§4), and the G = 16 pairs carried as E3M2 under one scale per 32 elements.
//
// Data flow: HBM-bound (VALU-bound with the MLP glue).  Outputs go to the tiled layout the GEMMs
// stream: codes in panels of 128 channels (R rows x 64 bytes of E2M1, 128 of E4M3, or 64 + 32
// of E3M2 pairs), scales in panels of 4 groups (8 when G = 16; one per 32 channels for pairs),
// B / W_L in panels of 32 groups.  Each lane holds one 32-channel block of one row: a wavefront
// covers 16 rows of one 128-channel panel (lane l: row l / 4, block b = l % 4), loading each
// row's 256 bytes as four 16-byte pieces per lane, and every code store instruction writes whole
// contiguous kilobytes of the panel.  The group amax is an integer max over the bf16 magnitude
// bits (|x| ordering == bit ordering for finite values).  The E8M0 code is read straight off the
// amax exponent field: floor(log2 amax) - emax + 127 = E - 2 (E2M1) or E - 8 (E4M3), floored at
// 0 (an amax of zero or below 2^-125 gives the minimum scale 2^-127).  Element encoding uses
// gfx950's scaled conversion instructions, which divide by the scale's power of two and round to
// nearest-even; E2M1 saturates in hardware, E4M3 does not, so E4M3 magnitudes are first clamped
// to 448 * 2^e (exactly representable in bf16).
#include "osc_quant_blk.h"

namespace osc {
namespace {

// ------------------------------------------------------------------ MLP glue
// In a Qwen3-shaped MLP block the down-projection reads h = silu(gate) * up, the two halves of
// the up-projection's bf16 output (not an OSC step; the quantization of W2's input then follows
// §3.2 / §4 as for any activation).  h is fixed as a sequence of binary32 operations so that it
// is reproducible bit for bit: e = exp(-g), s = g / (1 + e) (correctly rounded division),
// h = bf16 round-to-nearest-even of s * u.  exp by Cody and Waite's method: n = rint(x log2 e)
// (one binary32 product), r = x - n ln2 with ln2 split into a 16-significant-bit head and a
// binary32 tail (two fused multiply-adds), e^r by its degree-6 Taylor polynomial in Horner form
// (fused multiply-adds), then the exact scaling by 2^n; x > 88 gives +inf and x < -86 gives 0,
// so every finite intermediate is a normal number.
__device__ __forceinline__ float glu_exp(float x) {
#pragma clang fp contract(off)
  if (x > 88.0f) return __builtin_inff();
  if (x < -86.0f) return 0.0f;
  const float n = __builtin_rintf(x * 1.44269504088896341f);
  float r = __builtin_fmaf(-n, 0.693145751953125f, x);  // head: 45426 / 2^16, exact
  r = __builtin_fmaf(-n, 1.42860682030941723e-6f, r);   // tail: ln 2 - head
  float p = 1.0f / 720.0f;
  p = __builtin_fmaf(p, r, 1.0f / 120.0f);
  p = __builtin_fmaf(p, r, 1.0f / 24.0f);
  p = __builtin_fmaf(p, r, 1.0f / 6.0f);
  p = __builtin_fmaf(p, r, 0.5f);
  p = __builtin_fmaf(p, r, 1.0f);
  p = __builtin_fmaf(p, r, 1.0f);
  return __builtin_ldexpf(p, (int)n);
}

__device__ __forceinline__ uint32_t glu_one(uint32_t gbits, uint32_t ubits) {
#pragma clang fp contract(off)
  const float g = __builtin_bit_cast(float, gbits << 16);
  const float u = __builtin_bit_cast(float, ubits << 16);
  const float e = glu_exp(-g);
  const float sv = g / (1.0f + e);
  const uint32_t t = __builtin_bit_cast(uint32_t, sv * u);
  return (t + 0x7FFFu + ((t >> 16) & 1u)) >> 16;  // round to nearest even (finite values)
}

// 8 bf16 of gate and the 8 of up at the same columns -> 8 bf16 of h
__device__ __forceinline__ u4 glu_chunk(u4 g, u4 u) {
  u4 h;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = glu_one(g[i] & 0xFFFFu, u[i] & 0xFFFFu) | (glu_one(g[i] >> 16, u[i] >> 16) << 16);
  return h;
}

// h written out (bf16, row-major S x F): the glue on its own, for calibrating the W2 table.
__global__ __launch_bounds__(256) void k_swiglu(const u4* __restrict__ GU, int rows, int F, u4* __restrict__ Hout) {
  const long chunks = (long)rows * (F >> 3);
  for (long c = blockIdx.x * 256L + threadIdx.x; c < chunks; c += (long)gridDim.x * 256) {
    const long r = c / (F >> 3);
    const long q = c - r * (F >> 3);
    const u4* row = GU + r * (F >> 2);
    Hout[c] = glu_chunk(__builtin_nontemporal_load(row + q), __builtin_nontemporal_load(row + (F >> 3) + q));
  }
}

// The quantization kernel (activations and weights without the MLP glue).  The block a lane holds
// is two 16-groups (G = 16 and the pairs), one group (G = 32), or half of one (G = 64: the halves
// sit in neighbouring lanes of the same row and meet in one DPP lane swap for the amax).  Pairs
// re-encode to E3M2 with the conversion instructions: each group's E2M1 codes back to bf16 at the
// relative scale, then all 32 values to E3M2 in one instruction.
constexpr int kBlkRows = 16;

template <int G, int FMT, int MODE, int M>
__global__ __launch_bounds__(256) void k_quant_blk(const u4* __restrict__ X, int rows, int H, TableArg tab,
                                                   uint8_t* __restrict__ Q, uint8_t* __restrict__ SC,
                                                   uint16_t* __restrict__ side) {
  const int npan = H >> 7;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 6);  // wave -> (row block, panel), panel fastest
  const int rb = w / npan;
  const int p = w - rb * npan;
  const int lane = threadIdx.x & 63;
  const int b = lane & 3;  // block of the panel
  const int r = rb * kBlkRows + (lane >> 2);
  if (r >= rows) return;  // a row's four lanes leave together: the G = 64 swap stays inside a row
  const int col0 = p * 128 + b * 32;
  uint32_t x[16];  // dword j: channels col0 + 2j (low half), 2j + 1
  const u4* src = X + (long)r * (H >> 3) + (col0 >> 3);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const u4 t = src[c];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * c + i] = t[i];
  }
  quant_block<G, FMT, MODE, M>(x, r, p, b, rows, tab, Q, SC, side);
}

template <int G, int FMT, int MODE>
hipError_t launch_blk_m(const u4* x, int rows, int H, int m, const TableArg& t, uint8_t* q, uint8_t* SC,
                        uint16_t* sd, unsigned grid, hipStream_t st) {
  switch (m) {
    case 1: hipLaunchKernelGGL((k_quant_blk<G, FMT, MODE, 1>), dim3(grid), dim3(256), 0, st, x, rows, H, t, q, SC, sd); break;
    case 2: hipLaunchKernelGGL((k_quant_blk<G, FMT, MODE, 2>), dim3(grid), dim3(256), 0, st, x, rows, H, t, q, SC, sd); break;
    default: hipLaunchKernelGGL((k_quant_blk<G, FMT, MODE, 3>), dim3(grid), dim3(256), 0, st, x, rows, H, t, q, SC, sd); break;
  }
  return hipGetLastError();
}

// The quantization of h = glu(gate, up) for a gated MLP's down-projection: X holds rows of 2H bf16
// (gate | up).  The glue is long vector arithmetic, so this kernel keeps 8 channels per lane (few
// registers, many resident wavefronts): a wavefront owns 8 rows x one 128-channel panel, 16 lanes
// covering a row's 256 bytes of h per load instruction and 4 rows at once; groups are G/8 adjacent
// lanes, their amax reduced across lanes with DPP swaps (quant_chunk).
constexpr int kRowsPerWave = 8;

template <int G, int FMT, int MODE, int M>
__global__ __launch_bounds__(256) void k_quant_glu(const u4* __restrict__ X, int rows, int H, TableArg tab,
                                                   uint8_t* __restrict__ Q, uint8_t* __restrict__ SC,
                                                   uint16_t* __restrict__ side) {
  const int npan = H >> 7;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 6);  // wave -> (row block, panel), panel fastest
  const int rb = w / npan;
  const int p = w - rb * npan;
  if (rb * kRowsPerWave >= rows) return;  // whole wavefront past the last row
  const int lane = threadIdx.x & 63;
  const int cc = lane & 15;  // chunk of the panel row
  const int col0 = p * 128 + cc * 8;
  const int r0 = rb * kRowsPerWave + (lane >> 4);
  // rows past the end are skipped by whole 16-lane row segments, so a group's lanes agree
  constexpr int U = kRowsPerWave / 4;
  u4 vg[U], vu[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 4 * u;
    if (r < rows) {
      const u4* row = X + (long)r * (H >> 2);
      vg[u] = __builtin_nontemporal_load(row + (col0 >> 3));
      vu[u] = __builtin_nontemporal_load(row + ((H + col0) >> 3));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 4 * u;
    if (r < rows) quant_chunk<G, FMT, MODE, M>(glu_chunk(vg[u], vu[u]), r, col0, rows, tab, Q, SC, side);
  }
}

template <int G, int FMT, int MODE>
hipError_t launch_glu_m(const u4* x, int rows, int H, int m, const TableArg& t, uint8_t* q, uint8_t* SC,
                        uint16_t* sd, unsigned grid, hipStream_t st) {
  switch (m) {
    case 1: hipLaunchKernelGGL((k_quant_glu<G, FMT, MODE, 1>), dim3(grid), dim3(256), 0, st, x, rows, H, t, q, SC, sd); break;
    case 2: hipLaunchKernelGGL((k_quant_glu<G, FMT, MODE, 2>), dim3(grid), dim3(256), 0, st, x, rows, H, t, q, SC, sd); break;
    default: hipLaunchKernelGGL((k_quant_glu<G, FMT, MODE, 3>), dim3(grid), dim3(256), 0, st, x, rows, H, t, q, SC, sd); break;
  }
  return hipGetLastError();
}

template <int G, int FMT>
hipError_t dispatch_glu(const void* X, int rows, int H, int m, const TableArg* tab, int mode, void* Q, uint8_t* SC,
                        void* side, hipStream_t st) {
  const long waves = (long)((rows + kRowsPerWave - 1) / kRowsPerWave) * (H >> 7);
  const unsigned grid = (unsigned)((waves + 3) / 4);
  const u4* x = static_cast<const u4*>(X);
  uint8_t* q = static_cast<uint8_t*>(Q);
  uint16_t* sd = static_cast<uint16_t*>(side);
  static const TableArg empty = {};
  const TableArg& t = tab ? *tab : empty;
  if constexpr (FMT != OSC_MXFP8)
    if (mode == kExtractZero) return launch_glu_m<G, FMT, kExtractZero>(x, rows, H, m, t, q, SC, sd, grid, st);
  if (mode != kNoTable) return hipErrorInvalidValue;  // the glue feeds activations only (no copy mode)
  hipLaunchKernelGGL((k_quant_glu<G, FMT, kNoTable, 1>), dim3(grid), dim3(256), 0, st, x, rows, H, t, q, SC, sd);
  return hipGetLastError();
}

// mode: the table mode (kNoTable for E4M3)
template <int G, int FMT>
hipError_t dispatch_blk(const void* X, int rows, int H, int m, const TableArg* tab, int mode, void* Q, uint8_t* SC,
                        void* side, hipStream_t st) {
  const long waves = (long)((rows + kBlkRows - 1) / kBlkRows) * (H >> 7);
  const unsigned grid = (unsigned)((waves + 3) / 4);
  const u4* x = static_cast<const u4*>(X);
  uint8_t* q = static_cast<uint8_t*>(Q);
  uint16_t* sd = static_cast<uint16_t*>(side);
  static const TableArg empty = {};
  const TableArg& t = tab ? *tab : empty;
  if constexpr (FMT != OSC_MXFP8) {
    if (mode == kExtractZero) return launch_blk_m<G, FMT, kExtractZero>(x, rows, H, m, t, q, SC, sd, grid, st);
    if (mode == kCopyOnly) return launch_blk_m<G, FMT, kCopyOnly>(x, rows, H, m, t, q, SC, sd, grid, st);
  }
  if (mode != kNoTable) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_quant_blk<G, FMT, kNoTable, 1>), dim3(grid), dim3(256), 0, st, x, rows, H, t, q, SC, sd);
  return hipGetLastError();
}

template <int G, bool GLU>
hipError_t dispatch_fmt(const void* X, int rows, int H, int m, const TableArg* tab, int mode, osc_fmt fmt, void* Q,
                        uint8_t* SC, void* side, hipStream_t st) {
  if (fmt == OSC_FP6P) {
    if constexpr (G == 16) {
      if constexpr (GLU) return dispatch_glu<16, OSC_FP6P>(X, rows, H, m, tab, mode, Q, SC, side, st);
      return dispatch_blk<16, OSC_FP6P>(X, rows, H, m, tab, mode, Q, SC, side, st);
    }
    return hipErrorInvalidValue;  // E3M2 pairs exist for G = 16 only
  }
  if constexpr (GLU) {
    if (fmt == OSC_MXFP4) return dispatch_glu<G, OSC_MXFP4>(X, rows, H, m, tab, mode, Q, SC, side, st);
    return dispatch_glu<G, OSC_MXFP8>(X, rows, H, m, tab, mode, Q, SC, side, st);
  }
  if (fmt == OSC_MXFP4) return dispatch_blk<G, OSC_MXFP4>(X, rows, H, m, tab, mode, Q, SC, side, st);
  return dispatch_blk<G, OSC_MXFP8>(X, rows, H, m, tab, mode, Q, SC, side, st);
}

// ------------------------------------------------------------------ table builder
// §3.1 Algorithm 1 for one (position, layer), with up to m entries per group (m = 1 is the page's
// single channel; m = 2, 3 the §6 direction).  One workgroup per group k; threads stride over
// calibration rows.  In each row, each of the m largest |x| (lower channel first among equal
// magnitudes) that exceeds alpha times the group's mean |x| is an event of its channel, decided
// in fp64 (the sum of G bf16 magnitudes is formed in channel order); channel histograms are
// accumulated in LDS.  Entry e is the e-th most frequent event channel (lower channel first on
// ties) while its count reaches rho * R.
template <int G>
__global__ __launch_bounds__(256) void k_build_table(const uint16_t* __restrict__ X, int R, int H, int m, double alpha,
                                                     double rho, int32_t* __restrict__ L, int32_t* __restrict__ hits,
                                                     int32_t* __restrict__ events) {
  __shared__ int hist[G];
  __shared__ int nev;
  const int k = blockIdx.x;
  for (int j = threadIdx.x; j < G; j += 256) hist[j] = 0;
  if (threadIdx.x == 0) nev = 0;
  __syncthreads();
  int my_events = 0;
  for (int r = threadIdx.x; r < R; r += 256) {
    const uint16_t* row = X + (long)r * H + (long)k * G;
    float a[G];
    double sum = 0.0;
    for (int j = 0; j < G; ++j) {
      a[j] = fabsf(__builtin_bit_cast(float, (uint32_t)row[j] << 16));
      sum += (double)a[j];
    }
    const double thr = alpha * (sum / G);
    // the m largest magnitudes, lower channel first on ties
    int top[kMaxChannels] = {-1, -1, -1};
    for (int j = 0; j < G; ++j) {
      int pos = m;
      for (int e = m - 1; e >= 0; --e)
        if (top[e] < 0 || a[j] > a[top[e]]) pos = e;
      if (pos < m) {
        for (int e = m - 1; e > pos; --e) top[e] = top[e - 1];
        top[pos] = j;
      }
    }
    bool any = false;
    for (int e = 0; e < m; ++e)
      if ((double)a[top[e]] > thr) {
        atomicAdd(&hist[top[e]], 1);
        any = true;
      }
    my_events += any ? 1 : 0;
  }
  atomicAdd(&nev, my_events);
  __syncthreads();
  if (threadIdx.x == 0) {
    bool taken[G];
    for (int j = 0; j < G; ++j) taken[j] = false;
    bool stop = false;
    for (int e = 0; e < m; ++e) {
      int js = -1;
      for (int j = 0; j < G; ++j)
        if (!taken[j] && (js < 0 || hist[j] > hist[js])) js = j;
      taken[js] = true;
      hits[k * m + e] = hist[js];
      if (!stop && hist[js] > 0 && (double)hist[js] >= rho * (double)R) {
        L[k * m + e] = js;
      } else {
        stop = true;
        L[k * m + e] = -1;
      }
    }
    events[k] = nev;
  }
}

}  // namespace

hipError_t launch_quant(const void* X, int rows, int H, int G, int m, const TableArg* tab, int mode, osc_fmt fmt,
                        void* Q, uint8_t* SC, void* side, hipStream_t st, bool glu) {
  if ((long)rows * H == 0) return hipSuccess;
  if (glu && mode == kCopyOnly) return hipErrorInvalidValue;  // the glue feeds activations only
  switch (G) {
    case 16:
      return glu ? dispatch_fmt<16, true>(X, rows, H, m, tab, mode, fmt, Q, SC, side, st)
                 : dispatch_fmt<16, false>(X, rows, H, m, tab, mode, fmt, Q, SC, side, st);
    case 32:
      return glu ? dispatch_fmt<32, true>(X, rows, H, m, tab, mode, fmt, Q, SC, side, st)
                 : dispatch_fmt<32, false>(X, rows, H, m, tab, mode, fmt, Q, SC, side, st);
    default:
      return glu ? dispatch_fmt<64, true>(X, rows, H, m, tab, mode, fmt, Q, SC, side, st)
                 : dispatch_fmt<64, false>(X, rows, H, m, tab, mode, fmt, Q, SC, side, st);
  }
}

hipError_t launch_swiglu(const void* GU, int rows, int F, void* Hout, hipStream_t st) {
  const long chunks = (long)rows * (F >> 3);
  if (chunks == 0) return hipSuccess;
  const long blocks = (chunks + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 8192 ? blocks : 8192);
  hipLaunchKernelGGL(k_swiglu, dim3(grid), dim3(256), 0, st, static_cast<const u4*>(GU), rows, F,
                     static_cast<u4*>(Hout));
  return hipGetLastError();
}

hipError_t launch_build_table(const void* Xcal, int R, int H, int G, int m, double alpha, double rho, int32_t* L,
                              int32_t* hits, int32_t* events, hipStream_t st) {
  const uint16_t* x = static_cast<const uint16_t*>(Xcal);
  const int K = H / G;
  switch (G) {
    case 16:
      hipLaunchKernelGGL(k_build_table<16>, dim3(K), dim3(256), 0, st, x, R, H, m, alpha, rho, L, hits, events);
      break;
    case 32:
      hipLaunchKernelGGL(k_build_table<32>, dim3(K), dim3(256), 0, st, x, R, H, m, alpha, rho, L, hits, events);
      break;
    default:
      hipLaunchKernelGGL(k_build_table<64>, dim3(K), dim3(256), 0, st, x, R, H, m, alpha, rho, L, hits, events);
      break;
  }
  return hipGetLastError();
}

}  // namespace osc
