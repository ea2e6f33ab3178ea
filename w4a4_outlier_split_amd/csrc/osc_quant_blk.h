// The encoders shared by the quantization kernels of libosc: bf16 bits in registers -> extraction, E8M0
// scale, element codes, stores in the tiled layout.  quant_chunk takes 8 channels of a row a lane (a group
// is 2, 4 or 8 lanes), quant_block 32.
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

// ---- E3M2 pairs (G = 16 pairs carried by one scale per 32 elements)
// E2M1 code c (at its 16-group's scale code) -> E3M2 code of the same value at the pair's scale
// code, t = s_group - E_pair <= 2: the value 1.m * 2^p (p = -1 for 0.5) lands at exponent q = p + t;
// q >= -2 is a normal E3M2 number, below that it is a multiple of 1/16 rounded to nearest, ties to
// the even code (only when the pair's scale codes differ by more than 5).
__device__ __forceinline__ uint32_t e2m1_to_e3m2(uint32_t c, int t) {
  // selects only (no early return): the compiler keeps it branch-free
  const uint32_t sign = (c & 8u) << 2;
  const int mu = c & 7;
  const int p = mu == 1 ? -1 : (mu >> 1) - 1;
  const int m = mu == 1 ? 0 : (mu & 1);
  const int q = p + t;
  const uint32_t normal = (uint32_t)(((q + 3) << 2) | (m << 1));
  const int units = q == -3 ? 2 + m : q == -4 ? (m ? 2 : 1) : q == -5 ? m : 0;  // of 1/16
  const uint32_t mag = mu == 0 ? 0u : q >= -2 ? normal : (uint32_t)units;
  return sign | mag;
}

// 8 E2M1 codes (one dword, code i in nibble i) at shift t = s_group - E_pair <= 2 -> their E3M2
// codes, 48 bits: code i at bits [6i, 6i+6) of lo (bits 0..31) | hi16 << 32.
__device__ __forceinline__ void e3m2_8(uint32_t codes4, int t, uint32_t& lo, uint32_t& hi16) {
  lo = 0, hi16 = 0;
  if (t >= -1) {
    // groups within 3 scale codes of each other: every nonzero magnitude lands on a normal E3M2
    // number, code = base(mu) + 4t with base = 8 for 0.5 and 2 mu + 8 above -- four codes per
    // dword, one byte each (a byte permute looks up the base)
    auto bytes = [](uint32_t n) {  // 4 nibbles -> 4 bytes
      return (n & 0xFu) | ((n & 0xF0u) << 4) | ((n & 0xF00u) << 8) | ((n & 0xF000u) << 12);
    };
    auto conv = [&](uint32_t e) {
      const uint32_t mu = e & 0x07070707u;
      const uint32_t base = __builtin_amdgcn_perm(0x16141210u, 0x0E0C0800u, mu);
      const uint32_t nz = __builtin_amdgcn_perm(0x01010101u, 0x01010100u, mu);
      const uint32_t c = t >= 0 ? base + nz * (uint32_t)(4 * t) : base - nz * 4u;
      const uint32_t x = c | ((e & 0x08080808u) << 2);  // sign bit 3 -> 5
      return (x & 0x3Fu) | ((x >> 2) & 0xFC0u) | ((x >> 4) & 0x3F000u) | ((x >> 6) & 0xFC0000u);  // 4 x 6 bits
    };
    const uint32_t a = conv(bytes(codes4 & 0xFFFFu)), b = conv(bytes(codes4 >> 16));
    lo = a | (b << 24);
    hi16 = b >> 8;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c6 = e2m1_to_e3m2((codes4 >> (4 * i)) & 15u, t);
      const int bit = 6 * i;
      if (bit + 6 <= 32) {
        lo |= c6 << bit;
      } else if (bit >= 32) {
        hi16 |= c6 << (bit - 32);
      } else {
        lo |= c6 << bit;
        hi16 |= c6 >> (32 - bit);
      }
    }
  }
}

// E3M2 pairs at 8 channels per lane: the lane's 8 E2M1 codes (one dword, channel 2i
// in the low nibble of byte i) -> the pair's E3M2 codes and its stores.  The four lanes of a quad hold one 32-element block (lanes 0-1: 16-group
// 2b, lanes 2-3: 2b+1); lane q's 8 codes are bits [48q, 48q+48) of the block's 24-byte fragment.
__device__ __forceinline__ void pair_store(uint32_t codes4, int sx, int r, int col0, int rows,
                                           uint8_t* __restrict__ Q, uint8_t* __restrict__ SC) {
  const int sx_other = __builtin_amdgcn_update_dpp(0, sx, 0x4E, 0xF, 0xF, false);  // the other 16-group
  const int hi = sx > sx_other ? sx : sx_other;
  const int E = hi > 2 ? hi - 2 : 0;
  const int t = sx - E;
  uint32_t lo, hi16;  // 48 bits: lo = bits 0..31, hi16 = bits 32..47
  e3m2_8(codes4, t, lo, hi16);
  // every lane of the quad learns the four 48-bit pieces
  const uint32_t lo0 = __builtin_amdgcn_update_dpp(0, lo, 0x00, 0xF, 0xF, false);
  const uint32_t lo1 = __builtin_amdgcn_update_dpp(0, lo, 0x55, 0xF, 0xF, false);
  const uint32_t lo2 = __builtin_amdgcn_update_dpp(0, lo, 0xAA, 0xF, 0xF, false);
  const uint32_t lo3 = __builtin_amdgcn_update_dpp(0, lo, 0xFF, 0xF, 0xF, false);
  const uint32_t h0 = __builtin_amdgcn_update_dpp(0, hi16, 0x00, 0xF, 0xF, false);
  const uint32_t h1 = __builtin_amdgcn_update_dpp(0, hi16, 0x55, 0xF, 0xF, false);
  const uint32_t h2 = __builtin_amdgcn_update_dpp(0, hi16, 0xAA, 0xF, 0xF, false);
  const uint32_t h3 = __builtin_amdgcn_update_dpp(0, hi16, 0xFF, 0xF, 0xF, false);
  const int q = (col0 >> 3) & 3;     // lane in the quad
  const int b = (col0 & 127) >> 5;   // block in the stage
  const long stage = (long)(col0 >> 7) * rows * 96;
  // fragment dwords 0..3 (one per lane) -> the first R x 64 bytes of the stage
  const uint32_t d = q == 0 ? lo0 : q == 1 ? (h0 | (lo1 << 16)) : q == 2 ? ((lo1 >> 16) | (h1 << 16)) : lo2;
  __builtin_nontemporal_store(d, reinterpret_cast<uint32_t*>(Q + stage + (long)r * 64 + b * 16 + q * 4));
  // dwords 4, 5 (lanes 0, 1) -> the R x 32 bytes after them, block position XOR-permuted by row
  if (q < 2) {
    const uint32_t e = q == 0 ? (h2 | (lo3 << 16)) : ((lo3 >> 16) | (h3 << 16));
    __builtin_nontemporal_store(
        e, reinterpret_cast<uint32_t*>(Q + stage + (long)rows * 64 + (long)r * 32 + 8 * (b ^ (((r >> 1) ^ (r >> 3)) & 3)) + q * 4));
  }
  // one scale byte per block, at the G = 32 scale layout
  if (q == 0) {
    const int k32 = col0 >> 5;
    SC[((long)(k32 >> 2) * rows + r) * 4 + (k32 & 3)] = (uint8_t)E;
  }
}

// One 16-byte chunk c (8 bf16 of one row): extraction, group scale, encoding, tiled stores.
template <int G, int FMT, int MODE, int M>
__device__ __forceinline__ void quant_chunk(u4 v, int r, int col0, int rows, const TableArg& tab,
                                            uint8_t* __restrict__ Q, uint8_t* __restrict__ SC,
                                            uint16_t* __restrict__ side) {
  constexpr int LPG = G / 8;  // lanes per group
  const int k = col0 / G;
  const int q = (col0 % G) >> 3;
  constexpr int SPG = G == 16 ? 8 : 4;  // groups per scale panel
  const long code_at = ((long)(col0 >> 7) * rows + r) * 16 + ((col0 & 127) >> 3);  // in 4 / 8-byte units
  const long scale_at = ((long)(k / SPG) * rows + r) * SPG + k % SPG;
  const uint32_t x0 = v[0], x1 = v[1], x2 = v[2], x3 = v[3];  // as loaded
  uint32_t w0 = x0, w1 = x1, w2 = x2, w3 = x3;                  // with the listed slots zeroed

  if (MODE != kNoTable) {
    // entries k*m .. k*m+m-1 of the table list distinct channels of group k (or -1); entry e goes
    // to compensation column k*m + e, written by the lane holding the channel (or lane 0 of the
    // group, as +0, for -1)
#pragma unroll
    for (int e = 0; e < M; ++e) {
      {
        const int ent = tab.v[k * M + e];
        const bool own = ent >= 0 && (ent >> 3) == q;
        uint32_t val = 0;
        if (own) {
          const int c = ent & 7;
          const uint32_t word = (c >> 1) == 0 ? x0 : (c >> 1) == 1 ? x1 : (c >> 1) == 2 ? x2 : x3;
          val = (c & 1) ? (word >> 16) : (word & 0xFFFFu);
          if (MODE == kExtractZero) {
            const uint32_t keep = (c & 1) ? 0x0000FFFFu : 0xFFFF0000u;
            w0 = (c >> 1) == 0 ? (w0 & keep) : w0;
            w1 = (c >> 1) == 1 ? (w1 & keep) : w1;
            w2 = (c >> 1) == 2 ? (w2 & keep) : w2;
            w3 = (c >> 1) == 3 ? (w3 & keep) : w3;
          }
        }
        const int col = k * M + e;
        if (own || (ent < 0 && q == 0)) side[((long)(col >> 5) * rows + r) * 32 + (col & 31)] = (uint16_t)val;
      }
    }
  }

  // group amax over the magnitude bits
  us2 mx = __builtin_elementwise_max(as_us2(w0 & 0x7FFF7FFFu), as_us2(w1 & 0x7FFF7FFFu));
  mx = __builtin_elementwise_max(mx, as_us2(w2 & 0x7FFF7FFFu));
  mx = __builtin_elementwise_max(mx, as_us2(w3 & 0x7FFF7FFFu));
  int amax = mx.x > mx.y ? mx.x : mx.y;
  // group max across the LPG adjacent lanes with DPP lane swaps: neighbours (quad_perm 1,0,3,2),
  // pairs (quad_perm 2,3,0,1), then the two quads of an 8-lane row half (half-row mirror)
  amax = max(amax, __builtin_amdgcn_update_dpp(0, amax, 0xB1, 0xF, 0xF, false));
  if constexpr (LPG >= 4) amax = max(amax, __builtin_amdgcn_update_dpp(0, amax, 0x4E, 0xF, 0xF, false));
  if constexpr (LPG >= 8) amax = max(amax, __builtin_amdgcn_update_dpp(0, amax, 0x141, 0xF, 0xF, false));
  const int E = amax >> 7;
  const int sx = FMT != OSC_MXFP8 ? (E > 2 ? E - 2 : 0) : (E > 8 ? E - 8 : 0);
  if (FMT != OSC_FP6P && q == 0) SC[scale_at] = (uint8_t)sx;
  const float scale = __builtin_bit_cast(float, (uint32_t)sx << 23);  // only the exponent field is used

  if constexpr (FMT == OSC_FP6P) {
    static_assert(G == 16, "E3M2 pairs carry two 16-groups");
    uint32_t out = 0;
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(w0), scale, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(w1), scale, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(w2), scale, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(w3), scale, 3);
    pair_store(out, sx, r, col0, rows, Q, SC);
  } else if (FMT == OSC_MXFP4) {
    uint32_t out = 0;
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(w0), scale, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(w1), scale, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(w2), scale, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, as_bf2(w3), scale, 3);
    __builtin_nontemporal_store(out, reinterpret_cast<uint32_t*>(Q) + code_at);
  } else {
    // saturate: |x| <= 448 * 2^e, i.e. exponent field sx + 8 with mantissa 0b1100000
    const uint32_t lim = (((uint32_t)sx + 8u) << 7) | 0x60u;
    const us2 lim2 = {(unsigned short)lim, (unsigned short)lim};
    w0 = (w0 & 0x80008000u) | as_u32(__builtin_elementwise_min(as_us2(w0 & 0x7FFF7FFFu), lim2));
    w1 = (w1 & 0x80008000u) | as_u32(__builtin_elementwise_min(as_us2(w1 & 0x7FFF7FFFu), lim2));
    w2 = (w2 & 0x80008000u) | as_u32(__builtin_elementwise_min(as_us2(w2 & 0x7FFF7FFFu), lim2));
    w3 = (w3 & 0x80008000u) | as_u32(__builtin_elementwise_min(as_us2(w3 & 0x7FFF7FFFu), lim2));
    s2 o0 = {0, 0}, o1 = {0, 0};
    o0 = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o0, as_bf2(w0), scale, false);
    o0 = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o0, as_bf2(w1), scale, true);
    o1 = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o1, as_bf2(w2), scale, false);
    o1 = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o1, as_bf2(w3), scale, true);
    const u2 o = {__builtin_bit_cast(uint32_t, o0), __builtin_bit_cast(uint32_t, o1)};
    __builtin_nontemporal_store(o, reinterpret_cast<u2*>(Q) + code_at);
  }
}

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
