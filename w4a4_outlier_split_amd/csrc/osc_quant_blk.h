// The block encoder shared by the quantization kernels of libosc: one lane's 32 channels of one row
// (bf16 bits in registers) -> extraction, E8M0 scale, element codes, stores in the tiled layout.
#pragma once

#include "osc_internal.h"

namespace osc {
namespace {

typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef short s2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned u2 __attribute__((ext_vector_type(2)));
typedef unsigned u6 __attribute__((ext_vector_type(6)));
typedef __bf16 bf32 __attribute__((ext_vector_type(32)));

__device__ __forceinline__ us2 as_us2(uint32_t w) { return __builtin_bit_cast(us2, w); }
__device__ __forceinline__ uint32_t as_u32(us2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ bf2 as_bf2(uint32_t w) { return __builtin_bit_cast(bf2, w); }

// dword d (lane-varying, 0 <= d < N) of the N words w[0..N), by a binary tree of selects on d's bits
template <int N>
__device__ __forceinline__ uint32_t pick(const uint32_t* w, int d) {
  uint32_t t[N];
#pragma unroll
  for (int j = 0; j < N; ++j) t[j] = w[j];
#pragma unroll
  for (int n = N, bit = 1; n > 1; n >>= 1, bit <<= 1) {
    const bool hi = (d & bit) != 0;
#pragma unroll
    for (int j = 0; j < n / 2; ++j) t[j] = hi ? t[2 * j + 1] : t[2 * j];
  }
  return t[0];
}

// One lane's block: channels [128p + 32b, +32) of row r, dword j of x holding channels 2j (low half)
// and 2j + 1.  The row's four lanes b = 0..3 of the panel are a quad and call this together.
template <int G, int FMT, int MODE, int M>
__device__ __forceinline__ void quant_block(const uint32_t (&x)[16], int r, int p, int b, int rows, const TableArg& tab,
                                            uint8_t* __restrict__ Q, uint8_t* __restrict__ SC,
                                            uint16_t* __restrict__ side) {
  static_assert(FMT != OSC_FP6P || G == 16, "E3M2 pairs of 16-groups");
  static_assert(FMT != OSC_MXFP8 || MODE == kNoTable, "no extraction on the E4M3 path");
  constexpr int NG = G == 16 ? 2 : 1;  // groups (G = 64: group halves) in the block
  constexpr int GW = 16 / NG;           // dwords of each
  const int col0 = p * 128 + b * 32;
  uint32_t v[16];  // x with the listed slots zeroed
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = x[j];
  if (MODE != kNoTable) {
    // entry e of group k goes to compensation column k*m + e (+0 for -1), written by the lane that
    // holds the channel (G = 64, entry -1: the lane of the group's first half)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int k = G == 64 ? col0 >> 6 : G == 32 ? col0 >> 5 : (col0 >> 4) + g;
      const int base = G == 64 ? (b & 1) * 32 : 0;  // the group's channel at this lane's dword 0
#pragma unroll
      for (int e = 0; e < M; ++e) {
        const int ent = tab.v[k * M + e];
        const int loc = ent - base;
        const bool own = ent >= 0 && loc < 2 * GW && (G != 64 || loc >= 0);
        const int d = loc >> 1;
        const uint32_t word = pick<GW>(x + GW * g, d & (GW - 1));
        const uint32_t val = own ? ((ent & 1) ? (word >> 16) : (word & 0xFFFFu)) : 0u;
        if (MODE == kExtractZero) {
          // masked in the running copy: two entries may share a dword
          const uint32_t keep = (ent & 1) ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
          for (int j = 0; j < GW; ++j) v[GW * g + j] = own && d == j ? (v[GW * g + j] & keep) : v[GW * g + j];
        }
        const int col = k * M + e;
        if (G != 64 || own || (ent < 0 && (b & 1) == 0))
          side[((long)(col >> 5) * rows + r) * 32 + (col & 31)] = (uint16_t)val;
      }
    }
  }
  int sx[NG];
  uint32_t codes[8];  // E2M1: 4 dwords of 8 codes; E4M3: 8 dwords of 4 codes
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    us2 mx = as_us2(v[GW * g] & 0x7FFF7FFFu);
#pragma unroll
    for (int j = 1; j < GW; ++j) mx = __builtin_elementwise_max(mx, as_us2(v[GW * g + j] & 0x7FFF7FFFu));
    int amax = mx.x > mx.y ? mx.x : mx.y;
    if constexpr (G == 64) amax = max(amax, __builtin_amdgcn_update_dpp(0, amax, 0xB1, 0xF, 0xF, false));
    const int E = amax >> 7;
    sx[g] = FMT == OSC_MXFP8 ? (E > 8 ? E - 8 : 0) : (E > 2 ? E - 2 : 0);
    const float scale = __builtin_bit_cast(float, (uint32_t)sx[g] << 23);  // only the exponent field is used
    if constexpr (FMT == OSC_MXFP8) {
      // saturate: |x| <= 448 * 2^e, i.e. exponent field sx + 8 with mantissa 0b1100000
      const uint32_t lim = (((uint32_t)sx[g] + 8u) << 7) | 0x60u;
      const us2 lim2 = {(unsigned short)lim, (unsigned short)lim};
#pragma unroll
      for (int hh = 0; hh < GW / 2; ++hh) {
        uint32_t c2[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t w0 = v[GW * g + 2 * hh + q];
          c2[q] = (w0 & 0x80008000u) | as_u32(__builtin_elementwise_min(as_us2(w0 & 0x7FFF7FFFu), lim2));
        }
        s2 o = {0, 0};
        o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, as_bf2(c2[0]), scale, false);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, as_bf2(c2[1]), scale, true);
        codes[(GW / 2) * g + hh] = __builtin_bit_cast(uint32_t, o);
      }
    } else {
#pragma unroll
      for (int hh = 0; hh < GW / 4; ++hh) {
        const uint32_t* s4 = v + GW * g + 4 * hh;
        uint32_t out = 0;
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(s4[0]), scale, 0);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(s4[1]), scale, 1);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(s4[2]), scale, 2);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(s4[3]), scale, 3);
        codes[(GW / 4) * g + hh] = out;
      }
    }
  }
  if constexpr (FMT != OSC_FP6P) {
    // codes: the block's 16 (E2M1) or 32 (E4M3) bytes of the row's 64 / 128 in the panel; scales
    // at G = 16 in panels of 8 groups (this block's two adjacent), else of 4
    if constexpr (FMT == OSC_MXFP8) {
      // the row's 128 bytes are the four lanes' 32 in lane order: each store writes one contiguous
      // half row, lane b its bytes [16b, 16b + 16) of the half (from lane 2*half + b/2 of the row's
      // quad, that lane's first or second 16 bytes by b's parity)
      u4 lo, hi;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int a0 = __builtin_amdgcn_mov_dpp((int)codes[i], 0x50, 0xF, 0xF, false);      // quad lanes 0,0,1,1
        const int a1 = __builtin_amdgcn_mov_dpp((int)codes[4 + i], 0x50, 0xF, 0xF, false);
        const int c0 = __builtin_amdgcn_mov_dpp((int)codes[i], 0xFA, 0xF, 0xF, false);      // quad lanes 2,2,3,3
        const int c1 = __builtin_amdgcn_mov_dpp((int)codes[4 + i], 0xFA, 0xF, 0xF, false);
        lo[i] = (uint32_t)((b & 1) ? a1 : a0);
        hi[i] = (uint32_t)((b & 1) ? c1 : c0);
      }
      u4* dst = reinterpret_cast<u4*>(Q + ((long)p * rows + r) * 128 + b * 16);
      __builtin_nontemporal_store(lo, dst);
      __builtin_nontemporal_store(hi, dst + 4);
    } else {
      __builtin_nontemporal_store(u4{codes[0], codes[1], codes[2], codes[3]},
                                  reinterpret_cast<u4*>(Q + ((long)p * rows + r) * 64 + b * 16));
    }
    if constexpr (G == 16) {
      *reinterpret_cast<uint16_t*>(SC + ((long)p * rows + r) * 8 + 2 * b) = (uint16_t)(sx[0] | (sx[1] << 8));
    } else if constexpr (G == 32) {
      SC[((long)p * rows + r) * 4 + b] = (uint8_t)sx[0];
    } else {
      const int k = col0 >> 6;
      if ((b & 1) == 0) SC[((long)(k >> 2) * rows + r) * 4 + (k & 3)] = (uint8_t)sx[0];
    }
  } else {
    const int hi = sx[0] > sx[1] ? sx[0] : sx[1];
    const int Ep = hi > 2 ? hi - 2 : 0;
    // Each group's E2M1 values back as bf16, times 2^t with t = s_group - E_pair <= 2 (exact: at
    // most 24 in magnitude), then one conversion of all 32 values to E3M2 at unit scale: exact
    // where the value is an E3M2 number, else rounded to nearest, ties to the even code.  Below
    // t = -10 every magnitude is under 1/32 and becomes a signed zero either way, so t is floored.
    bf32 y;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int t = sx[g] - Ep > -10 ? sx[g] - Ep : -10;
      const float rel = __builtin_bit_cast(float, (uint32_t)(127 + t) << 23);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t c = codes[2 * g + hh];
        const int o = 16 * g + 8 * hh;
        const bf2 a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, rel, 0);
        const bf2 a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, rel, 1);
        const bf2 a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, rel, 2);
        const bf2 a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, rel, 3);
        y[o + 0] = a0[0], y[o + 1] = a0[1], y[o + 2] = a1[0], y[o + 3] = a1[1];
        y[o + 4] = a2[0], y[o + 5] = a2[1], y[o + 6] = a3[0], y[o + 7] = a3[1];
      }
    }
    const u6 f = __builtin_amdgcn_cvt_scalef32_pk32_bf6_bf16(y, 1.0f);
    // the 24-byte fragment (code i at bits [6i, 6i + 6)): 16 bytes to the first region, 8 to the
    // second, whose 8-byte pieces sit at position b ^ (((r >> 1) ^ (r >> 3)) & 3) in the row
    const u4 first = {f[0], f[1], f[2], f[3]};
    const u2 second = {f[4], f[5]};
    const long stage = (long)p * rows * 96;
    __builtin_nontemporal_store(first, reinterpret_cast<u4*>(Q + stage + (long)r * 64 + b * 16));
    __builtin_nontemporal_store(
        second, reinterpret_cast<u2*>(Q + stage + (long)rows * 64 + (long)r * 32 + 8 * (b ^ (((r >> 1) ^ (r >> 3)) & 3))));
    SC[((long)p * rows + r) * 4 + b] = (uint8_t)Ep;
  }
}

}  // namespace
}  // namespace osc
