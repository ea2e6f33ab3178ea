// What the attention kernels over the paged cache share: where keys and values lie, the small tile (16 rows, keys from memory into
// registers) and the large one (256 rows on a ring of keys in LDS), and whole-number helpers for dealing out the work.
#pragma once

#include "osc_device.h"
#include "osc_internal.h"
#include "osc_lanes.h"

namespace osc {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

constexpr int kSmallRows = 16;
constexpr int kLargeRows = 256;
constexpr int kRing = 4;        // tiles of 64 keys in LDS
constexpr int kCUs = 256;
// The running maximum is left as it is while no score exceeds it by more than kSlack (in the exponent
// of 2): P is then at most 2^kSlack, and binary32 holds sums over 2^30 keys of them times values below 2^80;
// neither format loses precision by the factor.
constexpr float kSlack = 16.0f;

// branches that the loops seldom take: the registers are laid out for the other side
__device__ __forceinline__ bool rare(bool c) { return __builtin_expect(c, 0); }

struct Tile {
  int row0, rows;  // the tile's rows (token, head of the group): first and end, inside the request
  int tok0;        // the request's first token
  int first;       // position of that token: token i sees the keys up to first + i
  int kv;          // keys of the request that may be read
  const int32_t* pages;
  int lo, hi;      // the steps of keys to take (64 keys each)
  long part;       // first row of the workspace for a part of a tile, -1: the whole tile
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// the page of key `key`, -1 behind the request's keys or off the pool
__device__ __forceinline__ int page_of(const AttnArgs& a, const Tile& t, int key) {
  const int id = (unsigned)key < (unsigned)t.kv ? t.pages[key >> a.sh] : -1;
  return id >= 0 && id < a.NP ? id : -1;
}

// element offset of (page, key head): K and V blocks have the same size
template <int D>
__device__ __forceinline__ long block_at(const AttnArgs& a, int id, int h) {
  return (((long)id * a.HKV + h) << a.sh) * D;
}

// ------------------------------------------------------------------ dealing out the work
__device__ __forceinline__ long lane_of(long v, int src) {
  const unsigned lo = __builtin_amdgcn_readlane((int)v, src), hi = __builtin_amdgcn_readlane((int)(v >> 32), src);
  return (long)((unsigned long)hi << 32 | lo);
}

__device__ __forceinline__ long uniform(long v) {  // a value that all lanes share, into scalar registers
  const unsigned lo = __builtin_amdgcn_readfirstlane((int)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (long)((unsigned long)hi << 32 | lo);
}

// the next request with tokens behind r, of which the caller knows
__device__ __forceinline__ int next_request(const AttnArgs& a, int r) {
  for (int from = r + 1; from < a.R; from += 64) {
    const int x = from + (int)(threadIdx.x & 63);
    const unsigned long long has = __ballot(x < a.R && clampi(a.CU[x + 1], 0, a.S) > clampi(a.CU[x], 0, a.S));
    if (has) return from + __ffsll(has) - 1;
  }
  return r;
}

// a / b for 0 <= a, 0 < b, a / b < 2^50, by way of 64-bit floating point (a division of integers takes five times as long)
__device__ __forceinline__ long divide(long a, long b) {
  long q = (long)((double)a / (double)b);
  while (q * b > a) --q;
  while ((q + 1) * b <= a) ++q;
  return q;
}

// A row's mask among the new keys, and bits j0 .. j0 + 63 of what it sees: all of the context ahead of them, nothing behind.
// The words are read with the row's query: a load in the midst of the keys' would be waited for behind all that are under way.
constexpr int kWords = OSC_MAX_TREE / 64;
struct Words {
  unsigned long long w[kWords];
  template <typename Args>
  __device__ __forceinline__ void load(const Args& a, long row) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = i < a.W ? a.MASK[row * a.W + i] : 0;
  }
  __device__ __forceinline__ unsigned long long word(int i) const {
    unsigned long long x = i < 0 ? ~0ull : 0;
#pragma unroll
    for (int j = 0; j < kWords; ++j) x = i == j ? w[j] : x;
    return x;
  }
  __device__ __forceinline__ unsigned long long window(int j0) const {
    const int i = j0 >> 6, s = j0 & 63;
    const unsigned long long lo = word(i), hi = word(i + 1);
    return s ? lo >> s | hi << (64 - s) : lo;
  }
};

// which of 8 values are not finite
__device__ __forceinline__ int not_finite(v4i w) {
  int f = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) f |= ((w[i] & 0x7F80) == 0x7F80 ? 1 << 2 * i : 0) | ((w[i] & 0x7F800000) == 0x7F800000 ? 2 << 2 * i : 0);
  return f;
}
// values whose bits are set in f become 0
__device__ __forceinline__ v4i without(v4i w, int f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] &= ((f >> 2 * i) & 1 ? 0 : 0xFFFF) | ((f >> 2 * i) & 2 ? 0 : (int)0xFFFF0000);
  return w;
}

// A bit pattern over the 16 lanes of a row
__device__ __forceinline__ int or_row(int v) {
  v |= __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false);
  v |= __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false);
  v |= __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false);
  v |= __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false);
  return v;
}

// ------------------------------------------------------------------ small tiles
// Rows are the query heads of a token (and the next tokens'), so a decode with 4 heads to a key head uses 4 of 16:
// the products are idle anyway where every key is read once.  No LDS on the way: a key's row and a channel's run of
// keys are 16-byte pieces in the very lanes that the products want, and four wavefronts with a step each in flight
// and 512 workgroups cover the latency.  (64 decodes: 284 us with pages looked up in the step, 191 so, 5.6 TB/s.)
// TREE: behind the context, whose keys all rows see, a row's mask says which of the new keys it sees (so few rows have nodes of one word).
template <int D, bool TREE, typename Args>
__device__ __forceinline__ void small_tile(const Args& a, const Tile& t, int h, float* lds) {
  constexpr int DK = D / 32, DB = D / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, grp = lane >> 4;
  const int g = a.g;
  const __bf16* Kc = static_cast<const __bf16*>(a.KC);
  const __bf16* Vc = static_cast<const __bf16*>(a.VC);
  const int row = t.row0 + col;
  const bool live = row < t.rows;
  const int tok = row / g;
  const long out_row = (long)(t.tok0 + tok) * a.HQ + h * g + (row - tok * g);
  v8bf q[DK];
#pragma unroll
  for (int s = 0; s < DK; ++s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[s][i] = (__bf16)0.0f;
    if (live) q[s] = *reinterpret_cast<const v8bf*>(static_cast<const __bf16*>(a.Q) + out_row * D + s * 32 + grp * 8);
  }
  unsigned long long word = 0;
  if constexpr (TREE) word = live ? a.MASK[(long)(t.tok0 + tok) * a.W] : 0;
  const int last = live ? t.first + tok : -1;  // the last key of the lane's row
  const int tok_end = ((t.row0 + 16 < t.rows ? t.row0 + 16 : t.rows) - 1) / g;
  const int kend = TREE ? t.kv : clampi(t.first + tok_end + 1, 0, t.kv);
  const int lo = 2 * t.lo, hi = clampi((kend + 31) >> 5, lo, 2 * t.hi);  // steps of 32 keys

  v4f o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = v4f{0, 0, 0, 0};
  float m = neg_inf(), mc = 0.0f, l = 0.0f;
  const float c = a.scale_log2;
  // the pages of the wavefront's next 32 steps, a run of 16 keys a lane (a page holds at least one)
  int ids = 0;
  for (int st = lo + wave, n = 0; st < hi; st += 4, ++n) {
    const int k0 = st * 32;
    if ((n & 31) == 0) ids = page_of(a, t, k0 + (lane >> 1) * 128 + (lane & 1) * 16);
    const int id0 = __builtin_amdgcn_readlane(ids, 2 * (n & 31)), id1 = __builtin_amdgcn_readlane(ids, 2 * (n & 31) + 1);
    const bool whole = k0 + 32 <= t.kv && id0 >= 0 && id1 >= 0;
    const int idl = (grp & 2) ? id1 : id0;  // V's keys 8 * grp ..
    const int u = k0 + (grp & 2) * 8;
    const __bf16* vp = Vc + block_at<D>(a, idl < 0 ? 0 : idl, h) + ((long)col << a.sh) + (u & a.mask) + (grp & 1) * 8;
    v8bf kf[2][DK], vf[DB];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int kr = 8 * (col >> 2) + 4 * x + (col & 3);  // the key (of 32) in row col of score tile x
      const int id = kr < 16 ? id0 : id1;
      const int uk = k0 + (kr & 16);
      const __bf16* kp = Kc + block_at<D>(a, id < 0 ? 0 : id, h) + (long)((uk & a.mask) + (kr & 15)) * D + grp * 8;
#pragma unroll
      for (int s = 0; s < DK; ++s) kf[x][s] = *reinterpret_cast<const v8bf*>(kp + s * 32);
    }
#pragma unroll
    for (int d = 0; d < DB; ++d) vf[d] = *reinterpret_cast<const v8bf*>(vp + ((long)(16 * d) << a.sh));
    v4f sc[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      sc[x] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < DK; ++s) sc[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[x][s], q[s], sc[x], 0, 0, 0);
    }
    // scores of keys k0 + 8 grp + 4 x + i; the masked ones are selected away, whatever they hold
    const int limit = idl < 0 ? -1 : last;
    float mx = neg_inf();
    if constexpr (TREE) {
      if (!whole || k0 + 32 > t.first) {
        const int nv = idl < 0 ? 0 : clampi(t.kv - (k0 + 8 * grp), 0, 8), there = (1 << nv) - 1;  // which of the lane's keys exist
        int bad = 0;
#pragma unroll
        for (int d = 0; d < DB; ++d) {  // 0 * NaN is not 0: such values go, and rows that see the key become NaN by its score
          const v4i w = __builtin_bit_cast(v4i, vf[d]);
          const int f = not_finite(w);
          bad |= f & there;
          vf[d] = __builtin_bit_cast(v8bf, without(w, f | (there ^ 255)));
        }
        bad = or_row(bad);
        const int j0 = k0 + 8 * grp - t.first;  // of the lane's first key among the new ones
        const int see = (int)(j0 >= 64 ? 0 : j0 >= 0 ? word >> j0 : j0 <= -8 ? 255 : word << -j0 | ((1 << -j0) - 1)) & there;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (((see & bad) >> (4 * x + i)) & 1) sc[x][i] = __builtin_nanf("");
            if (!((see >> (4 * x + i)) & 1)) sc[x][i] = neg_inf();
          }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, sc[x][i]);
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (k0 + 8 * grp + 4 * x + i > limit) sc[x][i] = neg_inf();
          mx = fmaxf(mx, sc[x][i]);
        }
      if (!whole) {  // V of keys that do not exist may hold anything, and 0 * NaN is not 0
        const int nv = idl < 0 ? 0 : t.kv - (k0 + 8 * grp);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 8; ++i) vf[d][i] = i < nv ? vf[d][i] : (__bf16)0.0f;
      }
    }
    if (__any(mx * c > mc + kSlack || (m == neg_inf() && mx > neg_inf()))) {
      const float mn = fmaxf(m, max_groups(mx));
      const float ms = mn == neg_inf() ? 0.0f : mn;
      const float f = __builtin_amdgcn_exp2f(m * c - ms * c);
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= f;
      m = mn;
      mc = ms * c;
    }
    v8bf p, rest;  // the weights, and what their rounding leaves out
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x][i], c, -mc));
        l += e;
        p[4 * x + i] = (__bf16)e;
        rest[4 * x + i] = (__bf16)(e - (float)p[4 * x + i]);
      }
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[d], p, o[d], 0, 0, 0);
      o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[d], rest, o[d], 0, 0, 0);
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  // merge the wavefronts: m, l and O^T of each through LDS
  float* ml = lds;                   // [4][2][16]
  float* ob = lds + 128;             // [4][16][D + 4]
  __syncthreads();  // the tile before is merged
  if (grp == 0) ml[wave * 32 + col] = m, ml[wave * 32 + 16 + col] = l;
#pragma unroll
  for (int d = 0; d < DB; ++d) *reinterpret_cast<v4f*>(ob + (wave * 16 + col) * (D + 4) + 16 * d + 4 * grp) = o[d];
  __syncthreads();
  constexpr int PT = 16 * D / 256;  // values a thread joins
  const int orow = threadIdx.x / (D / PT), d0 = (threadIdx.x % (D / PT)) * PT;
  float mm = neg_inf();
#pragma unroll
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ml[w * 32 + orow]);
  const float ms = mm == neg_inf() ? 0.0f : mm;
  float ll = 0.0f, acc[PT];
#pragma unroll
  for (int i = 0; i < PT; ++i) acc[i] = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = __builtin_amdgcn_exp2f((ml[w * 32 + orow] - ms) * c);
    ll += f * ml[w * 32 + 16 + orow];
#pragma unroll
    for (int i = 0; i < PT; ++i) acc[i] += f * ob[(w * 16 + orow) * (D + 4) + d0 + i];
  }
  const int r = t.row0 + orow;
  if (r >= t.rows) return;
  if (t.part < 0) {
    const int tk = r / g;
    const long at = (long)(t.tok0 + tk) * a.HQ + h * g + (r - tk * g);
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;  // no key: zeros
#pragma unroll
    for (int i = 0; i < PT; i += 4) {
      v4bf b;
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = (__bf16)(acc[i + j] * inv);
      *reinterpret_cast<v4bf*>(static_cast<__bf16*>(a.O) + at * D + d0 + i) = b;
    }
  } else {
    const long at = t.part + orow;
#pragma unroll
    for (int i = 0; i < PT; i += 4)
      *reinterpret_cast<v4f*>(a.PO + at * D + d0 + i) = v4f{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
    if (d0 == 0) *reinterpret_cast<float2*>(a.PM + at * 2) = float2{ms * c, ll};
  }
}

// ------------------------------------------------------------------ large tiles
// LDS: a ring of tiles of K [64 keys][D] and V^T [4 runs of 16 keys][D][16].  K rows hold their
// 16-byte pieces at position piece ^ (row & (D/8 - 1)), V^T rows their two halves at half ^ (d >> 3 & 1):
// the 16 lanes that LDS serves together then read 16 different 16-byte columns of its 256.
// LDS-DMA of half of one run of 16 keys, which lie in one page (block: its byte offset for the key head, K's and
// V's alike; from slot `at`): the keys 8 part .. of K, the rows D/2 part .. of V^T.  off: the lane's place in the
// first 1024 bytes.
template <int D>
__device__ __forceinline__ int k_place(int lane) {
  constexpr int CH = D / 8;  // 16-byte pieces of a K row
  return lane / CH * D * 2 + (((lane % CH) ^ (lane / CH)) << 4);
}
template <int D>
__device__ __forceinline__ void load_k(const AttnArgs& a, long block, int at, int part, int off, lds_u8* buf) {
  const auto r = panel_rsrc(static_cast<const uint8_t*>(a.KC) + block, (2l * D) << a.sh);
  // D = 128: the row's number is 8 part + 4 i + lane / 16, and its pieces stand at position piece ^ row number
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    dma16s(r, off ^ (D == 128 ? part * 128 + i * 64 : 0), (at + 8 * part) * D * 2 + i * 1024, buf + i * 1024);
}
__device__ __forceinline__ int v_place(int lane, int sh) {  // row d = lane / 2, its halves in turn
  return ((lane >> 1) << (sh + 1)) + (((lane & 1) ^ ((lane >> 4) & 1)) << 4);
}
template <int D>
__device__ __forceinline__ void load_v(const AttnArgs& a, long block, int at, int part, int off, lds_u8* buf) {
  const auto r = panel_rsrc(static_cast<const uint8_t*>(a.VC) + block, (2l * D) << a.sh);
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    dma16s(r, off, at * 2 + ((part * (D / 64) + i) << (a.sh + 6)), buf + i * 1024);
}

// Eight wavefronts, a ring of kRing tiles of 64 keys in LDS filled three tiles ahead; one barrier a tile, behind
// which the tile before is free.  A wavefront holds 32 rows' queries (64 registers' worth with a tile's keys in
// flight) and output (64): 64 rows would halve the LDS reads a product but need the accumulation registers, whose copies
// cost more; four wavefronts, two workgroups a CU, read each key twice from LDS (587 us for the prompt of 8192, 495 to 535
// so).  A step has 32 products of 32 cycles for each wavefront, 2048 cycles a SIMD, and takes about 3500: one wavefront's
// exponentials run beside the other's products, the rest is LDS and the barrier.
// The weights enter the second product as one bf16 each (2^-8 at most), and their sum is that of the rounded ones, so it stays an average of the
// values: the products bound the step, and two bf16 each, as small tiles have them, are half as many again (trees of 64 nodes in 32 requests 126 us, 159
// so, 256 nodes over 32700 keys 148 and 199; the error of an output 2.2e-3 of its size, 1.7e-3 so, which is its own rounding).
// TREE: behind the context, whose keys all rows see, a row's mask says which of the new keys it sees.
template <int D, bool TREE, typename Args>
__device__ __forceinline__ void large_tile(const Args& a, const Tile& t, int h, uint8_t* lds) {
  constexpr int DK = D / 16, DB = D / 32, CH = D / 8, HALF = 64 * D * 2, TILE = 2 * HALF;
  unsigned* const flags = reinterpret_cast<unsigned*>(lds + kRing * TILE);  // TREE: keys of a tile with a value that is not finite, two in turn
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // worked out again for each tile: nothing of the lane's places is kept from one to the next
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int g = a.g;
  const int row0 = t.row0 + wave * 32, row = row0 + col;
  const bool live = row < t.rows;
  const int tok = row / g;
  const long out_row = (long)(t.tok0 + tok) * a.HQ + h * g + (row - tok * g);
  v8bf q[DK];
#pragma unroll
  for (int s = 0; s < DK; ++s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[s][i] = (__bf16)0.0f;
    if (live) q[s] = *reinterpret_cast<const v8bf*>(static_cast<const __bf16*>(a.Q) + out_row * D + s * 16 + half * 8);
  }
  Words words;
  if constexpr (TREE) words.load(a, live ? t.tok0 + tok : t.tok0);
  const int base = t.first;
  const int last = live ? base + tok - 8 * half : -1;  // the last key the row sees, from the lane's first
  // the first row of the wavefront sees the fewest keys: tiles up to it need no mask
  const int wfirst = TREE ? base - 1 : base + row0 / g;
  const int lo = t.lo, hi = t.hi;
  v16f o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = v16f{};
  float m = neg_inf(), l = 0.0f;  // the running maximum (times c; -inf: no key yet) and sum of the lane's row
  const float c = a.scale_log2;

  if (lo < hi) {
    // The pages of 16 tiles, a run of 16 keys a lane, and those of the next 16: a page that is looked up
    // when it is needed would be waited for behind the DMA that is under way.
    int ids = page_of(a, t, (lo * 4 + lane) * 16), next_ids = page_of(a, t, (lo * 4 + 64 + lane) * 16);
    auto bad_of = [&](int n, int k0) {  // runs of 16 keys without a page; 16: the request ends in this tile
      return ((int)(__ballot(ids < 0) >> ((n & 15) * 4)) & 15) | (k0 + 64 > t.kv ? 16 : 0);
    };
    // A wavefront loads half a run: 8 keys of K, half the rows of V^T.
    const int run = wave >> 1, part = wave & 1;
    const int koff = k_place<D>(lane), voff = v_place(lane, a.sh);
    lds_u8* const lk = (lds_u8*)lds + (run * 16 + part * 8) * D * 2;
    lds_u8* const lv = (lds_u8*)lds + HALF + run * D * 32 + part * D * 16;
    auto load = [&](int n) {
      const int id = __builtin_amdgcn_readlane(ids, (n & 15) * 4 + run);
      const long block = 2 * block_at<D>(a, id < 0 ? 0 : id, h);
      const int at = ((lo + n) * 64 + run * 16) & a.mask, slot = (n & (kRing - 1)) * TILE;
      load_k<D>(a, block, at, part, koff, lk + slot);
      load_v<D>(a, block, at, part, voff, lv + slot);
    };
    constexpr int LOADS = D / 32;  // of a wavefront for a tile
    lds_barrier();  // the tile before is done with the ring
    if (TREE && tid < 4) flags[tid] = 0;
    int bads = 0;  // eight bits a tile: st, st + 1, st + 2 (the lowest first)
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) {
      if (lo + i < hi) load(i);
      bads |= bad_of(i, (lo + i) * 64) << (8 * i);
    }
    // row `col` of a score block holds its key 16 (b / 2) + 8 hh + 4 (b % 2) + j, col = 8 b + 4 hh + j; piece
    // 2 k + half of a row stands at position (2 k + half) ^ row number, where 2 k changes the higher bits only
    const int kr = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);
    const int ka = kr * D * 2 + ((half ^ (kr & (CH - 1))) << 4), va = HALF + col * 32 + ((half ^ ((col >> 3) & 1)) << 4);
    int slot = 0;  // of tile st
    int turn = 0;  // of the flags
    // The part of a step that loads and waits; the runs of keys missing in the tile, and 16 where the request ends.
    auto begin = [&](int st) {
      const int k0 = st * 64, n = st - lo;
      if (st + 2 < hi) wait_vm<2 * LOADS>();
      else wait_vm<0>();
      lds_barrier();  // tile st has landed, tile st - 1 is no longer read
      if (rare(((n + 3) & 15) == 0)) {
        ids = next_ids;
        next_ids = page_of(a, t, (st * 4 + 76 + lane) * 16);
      }
      if (st + 3 < hi) load(n + 3);
      bads |= bad_of(n + 3, k0 + 192) << 24;
      const int bad = bads & 31;
      bads = (int)((unsigned)bads >> 8);
      // V of keys that do not exist may hold anything, and 0 * NaN is not 0
      if constexpr (TREE) {
        // Nor may what a new key's holds reach the rows that do not see it: such values go, and rows that see the key
        // become NaN by its score.
        if (rare(bad != 0 || k0 + 63 > wfirst)) {
          // (the flags of the tile looked through before were last read ahead of this tile's barrier, and are set behind a later one's)
          turn ^= 1;
          int x = tid;
          asm volatile("" : "+v"(x));  // rarely run: nothing of it is kept in registers over the loop
          if (x < 2) flags[2 * (turn ^ 1) + x] = 0;
#pragma unroll
          for (int i = 0; i < D / 64; ++i, x += 512) {  // 8 keys of one channel
            const int u = x / (2 * D), key = u * 16 + (((x ^ (x >> 4)) & 1) << 3);
            const int left = (bad >> u) & 1 ? 0 : clampi(t.kv - (k0 + key), 0, 8), there = (1 << left) - 1;
            v4i* const v = reinterpret_cast<v4i*>(lds + slot + HALF) + x;
            const v4i w = *v;
            const int f = not_finite(w);
            if (f & there) atomicOr(&flags[2 * turn + (key >> 5)], (unsigned)(f & there) << (key & 31));
            if (f | (there ^ 255)) *v = without(w, f | (there ^ 255));
          }
          lds_barrier();
        }
      } else if (rare(bad != 0)) {
        uint16_t* v = reinterpret_cast<uint16_t*>(lds + slot + HALF);
        int first = tid;
        asm volatile("" : "+v"(first));  // rarely run: nothing of it is kept in registers over the loop
        for (int i = first; i < 64 * D; i += 512) {
          const int u = i / (16 * D), d = (i / 16) % D, e = i & 15;
          const int key = u * 16 + ((((e >> 3) ^ (d >> 3)) & 1) << 3) + (e & 7);
          if (k0 + key >= t.kv || ((bad >> u) & 1)) v[i] = 0;
        }
        lds_barrier();
      }
      return bad;
    };
    if (row0 >= t.rows) {  // a wavefront without a row loads its share, and leaves the rest to the others
      for (int st = lo; st < hi; ++st) {
        begin(st);
        slot = (slot + TILE) & (kRing * TILE - 1);
      }
      return;
    }
    for (int st = lo; st < hi; ++st) {
      const int k0 = st * 64, bad = begin(st);
      // Scores: element i of block x is key 32 x + 16 (i / 8) + 8 half + i % 8.  All operands are read ahead of the
      // first product (left to itself the compiler reads each when it is due, and every product waits for LDS),
      // and the two blocks take turns, so that no product waits for the one before.
      v16f s[2];
      v8bf kf[2][DK];
#pragma unroll
      for (int k = 0; k < DK; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) kf[x][k] = *reinterpret_cast<const v8bf*>(lds + x * (HALF / 2) + ((slot + ka) ^ (k * 32)));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < DK; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) s[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[x][k], q[k], k == 0 ? v16f{} : s[x], 0, 0, 0);
      auto value = [&](int y, int d) { return *reinterpret_cast<const v8bf*>(lds + slot + va + (y * DB + d) * 1024); };
      v8bf vf[2][DB];
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int d = 0; d < DB; ++d) vf[y][d] = value(y, d);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (TREE) {
        if (k0 + 63 > wfirst || bad) {
          unsigned long long see = words.window(k0 - base);
          if (k0 + 64 > t.kv) see &= k0 < t.kv ? ~0ull >> (64 - (t.kv - k0)) : 0;
          see &= ~(((bad & 1 ? 0xFFFFull : 0) | (bad & 2 ? 0xFFFFull << 16 : 0)) | ((bad & 4 ? 0xFFFFull << 32 : 0) | (bad & 8 ? 0xFFFFull << 48 : 0)));
          const unsigned long long odd = see & ((unsigned long long)flags[2 * turn + 1] << 32 | flags[2 * turn]);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const unsigned seen = (unsigned)(see >> (16 * y + 8 * half)) & 255, nan = (unsigned)(odd >> (16 * y + 8 * half)) & 255;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x = s[y >> 1][8 * (y & 1) + i];
              s[y >> 1][8 * (y & 1) + i] = (nan >> i) & 1 ? __builtin_nanf("") : (seen >> i) & 1 ? x : neg_inf();
            }
          }
        }
      } else if (k0 + 63 > wfirst || bad) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int end = (bad >> y) & 1 ? -1 : last - k0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (16 * y + i > end) s[y >> 1][8 * (y & 1) + i] = neg_inf();
        }
      }
      float mx = neg_inf();
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[x][i]);
      mx *= c;
      if (__any(mx > m + kSlack)) {
        const float mn = fmaxf(m, max_halves(mx));
        const float f = __builtin_amdgcn_exp2f(m - (mn == neg_inf() ? 0.0f : mn));
        l *= f;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] *= f;
        m = mn;
      }
      const float mc = m == neg_inf() ? 0.0f : m;
      const v2bf one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        v8bf p;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const v2bf e = {(__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[y >> 1][8 * (y & 1) + i], c, -mc)),
                          (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[y >> 1][8 * (y & 1) + i + 1], c, -mc))};
          p[i] = e[0], p[i + 1] = e[1];
          l = __builtin_amdgcn_fdot2_f32_bf16(e, one, l, false);
        }
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[y & 1][d], p, o[d], 0, 0, 0);
        if (y < 2) {
#pragma unroll
          for (int d = 0; d < DB; ++d) vf[y][d] = value(y + 2, d);
        }
      }
      slot = (slot + TILE) & (kRing * TILE - 1);
    }
  }
  l += __shfl_xor(l, 32);
  if (!live) return;
  if (t.part < 0) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no key: zeros
    __bf16* out = static_cast<__bf16*>(a.O) + out_row * D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v4bf b;
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = (__bf16)(o[d][4 * i + j] * inv);
        *reinterpret_cast<v4bf*>(out + d * 32 + 8 * i + 4 * half) = b;
      }
  } else {
    const long at = t.part + wave * 32 + col;
    if constexpr (TREE) {  // as the lanes hold them: 16 bytes a lane, 1024 a store
      v4f* out = reinterpret_cast<v4f*>(a.PO + (t.part + wave * 32) * D) + lane;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(4 * d + i) * 64] = v4f{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
      if (half == 0) *reinterpret_cast<float2*>(a.PM + at * 2) = float2{m, l};
      return;
    }
    float* out = a.PO + at * D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<v4f*>(out + d * 32 + 8 * i + 4 * half) =
            v4f{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    if (half == 0) *reinterpret_cast<float2*>(a.PM + at * 2) = float2{m, l};
  }
}

}  // namespace
}  // namespace osc
