// Attention of new tokens over the paged cache.
//
//   O[t][hq] = sum_j softmax_j(scale * q . k_j) v_j      over the keys j <= kv - n + i
//
// for token i of the n new tokens of a request whose cache holds kv keys (its new ones included), in
// one pass over the keys: with m the running maximum of a row's scores and l the running sum of
// exp(s - m), a tile of keys adds P = exp(S - m) to l and P V to the unnormalised output, and where
// m grows both are scaled by exp(m_old - m_new).  Scores, m, l and the output are binary32.  The matrix instruction
// takes no operand wider than bf16 beside bf16 values.  The small kernel, whose products wait for memory, takes a weight as two
// bf16, itself and what its rounding leaves out (2^-16 of it is lost; 64 decodes take 191 us as before, one 0.2 us more).  The
// large one, bound by its products, takes it rounded (each weight off by at most 2^-8 of itself, in either direction), and
// sums it into l as rounded, two weights a dot product.
//
// The HQ / HKV query heads that read one key head are rows of one tile, token by token, so a tile's
// keys serve all of them.  Both products run transposed, S^T = K Q^T and O^T = V^T P^T: a lane then
// holds scores of one query only (its maximum and sum are in-lane), and since the keys' order inside
// a tile is free, K's rows are read in the order that leaves each lane's scores as the very operand
// of the second product, with no exchange between lanes.  V^T's rows are contiguous keys in the
// cache's V layout [page][head][D][slot].
//
// Two kernels, by the call's tokens and requests:
//   small (single tokens): tiles of 16 rows, the cache read from memory straight into registers, every byte once;
//     the four wavefronts take 32 keys each in turn and are merged at the end.  HBM-bound: 64 decodes over 136
//     thousand keys (1.07 GB of cache) take 191 us, 5.6 TB/s.  A single decode over 4000 keys takes 10 us and 4 for the
//     join, bound by the chain of page table, keys, scores and two launches (its 16 MB are worth 3.5 us).
//   large: tiles of 256 rows, eight wavefronts of 32 rows each, one workgroup a CU; 64 keys of K and V^T at a
//     time in a ring in LDS, loaded by LDS-DMA three tiles ahead, so that a key is fetched once for 256 rows.  Bound
//     by what the matrix unit and the rest draw together: the card lowers its clock under this load, so
//     what counts is work per product.  A prompt of 8192 (32 query and 8 key heads of 128): 493 to 535 us with the
//     clock of the card, 1.03 to 1.11 PFLOP/s of the 1.35 to 1.55 that large matrix products reach; without loads,
//     barriers and exponentials it would be 458 us.  33 tokens over 32700 keys take 45 us and 10 for the join: a
//     tile of 132 rows on eight wavefronts, whose rate the chain through a step's two products sets.
// The work is cut evenly, whatever the lengths: all tiles of a key head stand in a row, each as long as the keys
// that it sees, and the row is cut into as many equal parts as workgroups run at once.  A workgroup takes
// its part, tile by tile.  A tile that a cut goes through has its unnormalised outputs left in the workspace, at
// most two tiles for a workgroup, and a second launch joins them in a fixed order.  The lengths are on the
// device, so each wavefront works the cuts out for itself.  (Chunks of 1024 and 765 tokens behind 1320 and 7946 keys, beside two
// idle requests, 135 GFLOP: 168 to 175 us, 20 of them for the join of 58 MB.)  Large tiles are left whole instead where that is
// quicker (whole_pays), which each wavefront finds from the lengths as well: one launch serves both.  (A choice by the host could
// go by the call's rows only, tokens or not: one token over 32000 keys in a call with room for 8192 then took 480 us, 39 so.  Two
// launches of which one has nothing to do take 2 to 3 us more.)
#include "osc_device.h"
#include "osc_internal.h"

namespace osc {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

constexpr int kSmallRows = 16;
constexpr int kLargeRows = 256;
constexpr int kRing = 4;        // tiles of 64 keys in LDS
constexpr int kCUs = 256;
constexpr int kMaxCuts = 61;    // of one tile: its parts, two more at most, are the lanes of the join
// Keys that a workgroup's part has at least.  (A prompt of 300 cut at 64, 128, 256: 24, 30, 38 us; 200 tokens on one key
// head behind 800: 35, 31, 34.)
constexpr int kMinKeys = 128;
// The running maximum is left as it is while no score exceeds it by more than kSlack (in the exponent
// of 2): P is then at most 2^kSlack, and binary32 holds sums over 2^30 keys of them times values below 2^80;
// neither format loses precision by the factor.
constexpr float kSlack = 16.0f;

// branches that the loops seldom take: the registers are laid out for the other side
__device__ __forceinline__ bool rare(bool c) { return __builtin_expect(c, 0); }

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

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

// max of a value over the lanes that differ in bit 5, and in bits 4 and 5: the swap instructions
// exchange half-wavefronts (16-lane rows) of two registers, so of two copies of v they leave each
// lane its own and its partner's.  (The results are read as integers first: a bit cast straight from a
// vector's element reads element 0 whichever is named.)
__device__ __forceinline__ float max_halves(float v) {
  const unsigned a = __builtin_bit_cast(unsigned, v);
  const auto x = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const unsigned x0 = x[0], x1 = x[1];
  return fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1));
}
__device__ __forceinline__ float max_groups(float v) {
  const unsigned a = __builtin_bit_cast(unsigned, v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const unsigned x0 = x[0], x1 = x[1];
  return max_halves(fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1)));
}

// The same and the sum over all lanes.  A row of 16 lanes first: neighbours, pairs, then the two mirrors.
template <int CTRL>
__device__ __forceinline__ float lane_swap(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float max_wave(float v) {
  v = fmaxf(v, lane_swap<0xB1>(v));
  v = fmaxf(v, lane_swap<0x4E>(v));
  v = fmaxf(v, lane_swap<0x141>(v));
  v = fmaxf(v, lane_swap<0x140>(v));
  return max_groups(v);
}
__device__ __forceinline__ float sum_wave(float v) {
  v += lane_swap<0xB1>(v);
  v += lane_swap<0x4E>(v);
  v += lane_swap<0x141>(v);
  v += lane_swap<0x140>(v);
  const unsigned a = __builtin_bit_cast(unsigned, v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const unsigned x0 = x[0], x1 = x[1];
  const unsigned b = __builtin_bit_cast(unsigned, __builtin_bit_cast(float, x0) + __builtin_bit_cast(float, x1));
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const unsigned y0 = y[0], y1 = y[1];
  return __builtin_bit_cast(float, y0) + __builtin_bit_cast(float, y1);
}

// ------------------------------------------------------------------ small tiles
// Rows are the query heads of a token (and the next tokens'), so a decode with 4 heads to a key head uses 4 of 16:
// the products are idle anyway where every key is read once.  No LDS on the way: a key's row and a channel's run of
// keys are 16-byte pieces in the very lanes that the products want, and four wavefronts with a step each in flight
// and 512 workgroups cover the latency.  (64 decodes: 284 us with pages looked up in the step, 191 so, 5.6 TB/s.)
template <int D>
__device__ __forceinline__ void small_tile(const AttnArgs& a, const Tile& t, int h, float* lds) {
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
  const int last = live ? t.first + tok : -1;  // the last key of the lane's row
  const int tok_end = ((t.row0 + 16 < t.rows ? t.row0 + 16 : t.rows) - 1) / g;
  const int kend = clampi(t.first + tok_end + 1, 0, t.kv);
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
template <int D>
__device__ __forceinline__ void large_tile(const AttnArgs& a, const Tile& t, int h, uint8_t* lds) {
  constexpr int DK = D / 16, DB = D / 32, CH = D / 8, HALF = 64 * D * 2, TILE = 2 * HALF;
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
  const int base = t.first;
  const int last = live ? base + tok - 8 * half : -1;  // the last key the row sees, from the lane's first
  // the first row of the wavefront sees the fewest keys: tiles up to it need no mask
  const int wfirst = base + row0 / g;
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
      if (rare(bad != 0)) {  // V of keys that do not exist may hold anything, and 0 * NaN is not 0
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
      if (k0 + 63 > wfirst || bad) {
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

// ------------------------------------------------------------------ the cuts
// The tiles of ROWS rows of a request and their lengths: tile i sees the keys up to its last token, base + (i +
// 1) tau with tau tokens a tile, and the i tiles ahead of it together (exactly, in whole numbers) before(i).
// whole: every tile has the length 1.  Tokens behind the call's S rows count for the others' positions, and keys
// behind the table's pages for the tokens', but neither is looked at.
template <int ROWS>
struct Request {
  int c0, n, first, kv, tiles;
  long base, tau;
  __device__ __forceinline__ Request(const AttnArgs& a, int r, bool whole) {
    c0 = clampi(a.CU[r], 0, a.S);
    const int c1 = clampi(a.CU[r + 1], 0, a.S);
    n = c1 > c0 ? c1 - c0 : 0;
    const int held = a.KV[r] > 0 ? a.KV[r] : 0, beyond = a.CU[r + 1] > a.S ? a.CU[r + 1] - a.S : 0;
    const long at = (long)held - n - beyond;
    constexpr long most = 1l << 30;  // as many positions as a table can hold: 32 bits do from here on
    first = (int)(at < -most ? -most : at < most ? at : most);
    kv = clampi(first + n, 0, (int)((long)a.MB << a.sh));
    tiles = (n * a.g + ROWS - 1) / ROWS;
    base = whole ? 1 : kv > n ? kv - n : 0;
    tau = whole ? 0 : (ROWS + a.g - 1) / a.g;
  }
  __device__ __forceinline__ long before(long i) const { return i * base + tau * (i * (i + 1) / 2); }
  __device__ __forceinline__ long all() const { return before(tiles); }
};

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

// Whole tiles or cut ones?  A key head has s CUs to itself.  Whole, its tiles take as long as the CU that has most of
// them; cut, a CU's even share, a quarter more for partial outputs and keys that are no longer read in step, and `once` keys' time
// for pieces of tiles and the join: 1000, and 500 more where whole tiles would save the join's launch.  With three tiles a CU
// and more, the share is what counts as long as no tile is longer; with fewer, a CU has the longest tile beside its share at
// worst.  (Of 551 calls with both sides measured, 2 to 6000 tokens of 1 to 40 requests on 1 to 32 key heads, this takes the slower
// side's time by more than a twentieth in 28, by more than an eighth in 14; with 1500 keys in 76 and 53.)
constexpr int kOnce = 1000, kOnceAndLaunch = 1500;
__host__ __device__ inline long slots_of(int HKV) { return HKV < kCUs ? kCUs / HKV : 1; }
__host__ __device__ inline bool whole_pays(long s, long tiles, long most, long all, long once) {
  return 4 * most * s <= all + 4 * once * s || (tiles >= 3 * s && most * s <= all);
}
// One request with tiles of base + tau, base + 2 tau, ... keys, the longest first: a CU has one, or two of which the
// longest pair is the s-th and the next.
__host__ __device__ inline bool whole_pays_alone(long s, long tiles, long base, long tau, long once) {
  if (tiles > 2 * s) return true;
  const long one = base + tau * tiles, two = tiles > s ? 2 * base + tau * (2 * tiles + 1 - 2 * s) : 0;
  const long all = tiles * base + tau * (tiles * (tiles + 1) / 2);
  return 4 * (one > two ? one : two) * s <= 5 * all + 4 * once * s;
}

// All tiles of a key head in a row, cut into `parts` equal parts, or each tile a part: as the caller says, or as the
// lengths are (whole_pays).  A wavefront's lanes hold a share of the requests each.
enum How { kCut, kWhole, kEither };
template <int ROWS, How HOW>
struct Cuts {
  typedef Request<ROWS> Req;
  long all, upto;  // the row's length; the lane's requests end there
  long mine;       // length of the lane's requests
  long each;       // all / parts
  int over;        // all % parts
  int r0, r1, parts;
  bool whole;

  __device__ __forceinline__ Cuts(const AttnArgs& a) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // as in large_tile
    const int per = (a.R + 63) >> 6;
    r0 = lane * per < a.R ? lane * per : a.R;
    r1 = r0 + per < a.R ? r0 + per : a.R;
    long most = 0;  // the longest tile
    long count = 0, counted;  // tiles of the lane's requests, and up to their end
    mine = 0;
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      const Req q(a, r, HOW == kWhole);
      mine += q.all();
      const long last = q.tiles > 0 ? q.base + q.tiles * q.tau : 0;
      most = last > most ? last : most;
      count += q.tiles;
    }
    upto = mine, counted = count;
    const int lanes = (a.R + per - 1) / per;
    for (int d = 1; d < lanes; d <<= 1) {  // up to each lane
      const long up = __shfl_up(upto, d), other = __shfl_up(most, d);
      const long tiles = HOW == kEither ? __shfl_up(counted, d) : 0;
      if (lane >= d) {
        upto += up, counted += tiles;
        most = other > most ? other : most;
      }
    }
    all = lane_of(upto, lanes - 1);
    most = lane_of(most, lanes - 1);
    whole = HOW == kWhole;
    if (HOW == kEither) {
      const long s = slots_of(a.HKV);
      whole = whole_pays(s, lane_of(counted, lanes - 1), most, all, kOnce);
      if (a.R == 1) {
        const Req q(a, 0, false);
        whole = whole || whole_pays_alone(s, q.tiles, q.base, q.tau, kOnce);
      }
    }
    if (whole) {  // a workgroup takes several only where there are more tiles than workgroups
      if (HOW == kEither) {
        mine = count, upto = counted;
        all = lane_of(upto, lanes - 1);
      }
      const long p = HOW == kEither ? gridDim.x / a.HKV : all;
      parts = (int)(p < all ? p : all > 0 ? all : 1);
    } else {
      long p = a.target;
      if (p > all / kMinKeys) p = all / kMinKeys;
      if (most > 0 && p > kMaxCuts && p > kMaxCuts * divide(all, most)) p = kMaxCuts * divide(all, most);
      parts = p < 1 ? 1 : (int)p;
    }
    each = HOW == kWhole ? 1 : divide(all, parts);
    over = HOW == kWhole ? 0 : (int)(all - each * parts);
  }
  // where part w begins
  __device__ __forceinline__ long cut(int w) const {
    return each * w + (HOW == kCut ? over * w / parts : divide((long)over * w, parts));
  }

  // The tile at `at` of the row (0 <= at < all): its request, its number there, and where it begins.
  __device__ __forceinline__ void find(const AttnArgs& a, long at, int& r, int& tile, long& begin) const {
    const int src = __ffsll(__ballot(at < upto)) - 1;
    long from = upto - mine;
    int hit = r0, i = 0;
    for (int x = r0; x < r1; ++x) {
      const Req q(a, x, whole);
      const long len = q.all();
      if (at - from < len) {
        if (whole) {
          i = (int)(at - from);
        } else if (q.tiles > 1) {
          // the largest i with before(i) <= at - from: the root of the parabola, put right by whole numbers
          const double b = (double)q.base + 0.5 * (double)q.tau, y = (double)(at - from);
          i = (int)((sqrt(b * b + 2.0 * (double)q.tau * y) - b) / (double)q.tau);
          i = i < 0 ? 0 : i < q.tiles ? i : q.tiles - 1;
          while (i + 1 < q.tiles && q.before(i + 1) <= at - from) ++i;
          while (i > 0 && q.before(i) > at - from) --i;
        }
        from += q.before(i);
        hit = x;
        break;
      }
      from += len;
    }
    r = __builtin_amdgcn_readlane(hit, src);
    tile = __builtin_amdgcn_readlane(i, src);
    begin = lane_of(from, src);
  }
};

// Workgroup: key head h = blockIdx % HKV (an XCD takes every eighth workgroup, so with eight key heads each XCD's
// L2 holds one head's cache), part w = blockIdx / HKV of the head's row; body(t, h) for each tile of the part in
// turn.  Whole tiles, one for a part or a few neighbours, take a request's later tiles first, which see the most keys, and all
// from their first key, so that the tiles that run together stream the same keys.  Otherwise the workgroup notes a tile that begins in its part
// and goes on behind it, for the join.
// What outlives a tile is held in scalar registers and no more than needed: the body needs all vector registers
// that there are.
template <int ROWS, How HOW, typename Body>
__device__ __forceinline__ void each_tile(const AttnArgs& a, Body body) {
  const int h = blockIdx.x % a.HKV, w = blockIdx.x / a.HKV;
  auto noted = [&](const int4& note) {
    if (threadIdx.x == 0 && w < a.target) a.NOTE[h * a.target + w] = note;
  };
  bool any, whole;
  int r = 0, i = 0, parts, over;
  long begin = 0, first = 0, end = 0, each;
  {
    const Cuts<ROWS, HOW> cuts(a);
    any = w < cuts.parts && cuts.all > 0;
    if (any) {
      first = uniform(cuts.cut(w)), end = uniform(cuts.cut(w + 1));
      cuts.find(a, first, r, i, begin);
    }
    parts = __builtin_amdgcn_readfirstlane(cuts.parts), over = __builtin_amdgcn_readfirstlane(cuts.over);
    each = uniform(cuts.each);
    whole = HOW == kEither ? __builtin_amdgcn_readfirstlane(cuts.whole) : HOW == kWhole;
  }
  if (!any || whole) noted(int4{0, 0, 0, 0});
  if (!any) return;
  for (;;) {
    const Request<ROWS> q(a, r, whole);
    const long len = uniform(whole ? 1 : q.before(i + 1) - q.before(i));
    const int tiles = __builtin_amdgcn_readfirstlane(q.tiles);
    Tile t;
    t.tok0 = __builtin_amdgcn_readfirstlane(q.c0);
    t.first = __builtin_amdgcn_readfirstlane(q.first);
    t.kv = __builtin_amdgcn_readfirstlane(q.kv);
    t.pages = a.TABLE + (long)r * a.MB;
    t.rows = __builtin_amdgcn_readfirstlane(q.n) * a.g;
    t.row0 = (whole ? tiles - 1 - i : i) * ROWS;
    const int tile_end = t.row0 + ROWS < t.rows ? t.row0 + ROWS : t.rows;
    const int steps = (clampi(t.first + (tile_end - 1) / a.g + 1, 0, t.kv) + 63) >> 6;
    t.lo = 0, t.hi = __builtin_amdgcn_readfirstlane(steps), t.part = -1;
    const bool last = HOW == kWhole || begin + len >= end;
    if (!whole) {
      if (begin < first) t.lo = (int)uniform(divide((first - begin) * steps, len));
      if (begin + len > end) t.hi = (int)uniform(divide((end - begin) * steps, len));
      // a tile of several parts: in the workgroup's second place where it begins there, in the first behind a cut
      if (begin < first || begin + len > end)
        t.part = (((long)h * a.target + w) * 2 + (begin < first ? 0 : 1)) * ROWS;
      if (last) {
        int ns = 0;
        if (begin >= first && begin + len > end) {  // the parts that begin in the tile: kMaxCuts and two at most
          const int p = w + 1 + (int)(threadIdx.x & 63);
          ns = 1 + __popcll(__ballot(p < parts && each * p + over * p / parts < begin + len));
        }
        noted(int4{ns, t.row0, t.rows, t.tok0});
      }
    }
    if (!last) {
      begin += len;
      if (++i == tiles) i = 0, r = next_request(a, r);
    }
    body(t, h);
    if (last) return;
  }
}

template <int D>
__global__ __launch_bounds__(256, 2) void k_attn_small(AttnArgs a) {
  __shared__ __align__(16) float lds[128 + 4 * 16 * (D + 4)];
  each_tile<kSmallRows, kCut>(a, [&](const Tile& t, int h) { small_tile<D>(a, t, h, lds); });
}

// Heads of 64 need half the LDS and may have two workgroups a CU, if 128 registers do.  (8192 tokens in a table of 40960 keys:
// 315 us, 350 with the 140 registers that the cuts would take; 33 tokens over 32700 keys 39 and 38.)
template <int D, How HOW>
__global__ __launch_bounds__(512, D == 64 ? 4 : 2) void k_attn_large(AttnArgs a) {
  extern __shared__ __align__(16) uint8_t dlds[];
  each_tile<kLargeRows, HOW>(a, [&](const Tile& t, int h) { large_tile<D>(a, t, h, dlds); });
}

// The weighted sum of a row's parts 0 .. ns - 1 in their order, FLY of them in flight: part k at src + place(k) * D,
// its weight in lane k (0 in lane 63).
template <int FLY, int D, typename vE, typename Place>
__device__ __forceinline__ vE weigh(const float* src, Place place, int ns, float f) {
  vE acc = {};
  for (int k = 0; k < ns; k += FLY) {
    vE v[FLY];
#pragma unroll
    for (int i = 0; i < FLY; ++i) v[i] = *reinterpret_cast<const vE*>(src + place(k + i < ns ? k + i : ns - 1) * D);
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int bits = __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), k + i < ns ? k + i : 63);
      const float wt = __builtin_bit_cast(float, bits);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) acc[e] += wt != 0.0f ? v[i][e] * wt : 0.0f;
    }
  }
  return acc;
}

// Joins the parts of the tile that part w noted: o = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k with m the largest
// m_k, in the order of the parts.  A row a wavefront: lane k holds the maximum and sum of part w + k, and the lanes
// D / 64 values of the row each.  HBM-bound where the parts are many (58 MB in 20 us, launch and all); a few rows
// (4 us) are bound by the launch and two loads one after the other, so the values' loads all start at once.
// (A workgroup a tile took 9 us for one decode and 24 for 33 tokens over 32700 keys, whose 132 rows have 31 parts each: 4 and 10 now.)
template <int D, int ROWS>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int E = D / 64;
  typedef float vE __attribute__((ext_vector_type(E)));
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.x % a.HKV, w = blockIdx.x / a.HKV;
  const int4 note = a.NOTE[h * a.target + w];
  const int ns = __builtin_amdgcn_readfirstlane(note.x);
  const int x = blockIdx.y * 4 + wave, row = note.y + x;
  if (ns == 0 || row >= note.z) return;
  // row x of the tile in part w + k: in that workgroup's second place for k = 0, in its first for the others
  auto place = [&](int k) { return (((long)h * a.target + w + k) * 2 + (k == 0 ? 1 : 0)) * ROWS + x; };
  float2 ml = {0.0f, 0.0f};
  if (lane < ns) ml = *reinterpret_cast<const float2*>(a.PM + place(lane) * 2);
  const bool any = ml.y != 0.0f;  // a part of no keys has a sum of 0, and its output does not count
  const float m = max_wave(any ? ml.x : neg_inf());
  const float f = any ? __builtin_amdgcn_exp2f(ml.x - m) : 0.0f;
  const float l = sum_wave(f * ml.y);
  const float* src = a.PO + lane * E;
  const vE acc = ns <= 4 ? weigh<4, D, vE>(src, place, ns, f) : weigh<16, D, vE>(src, place, ns, f);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = row / a.g;
  __bf16* out = static_cast<__bf16*>(a.O) + ((long)(note.w + tok) * a.HQ + h * a.g + (row - tok * a.g)) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = (__bf16)(acc[e] * inv);
}

}  // namespace

// Small tiles where there are at most as many tokens as requests: single tokens, in all likelihood.  (Of 2125 keys, 64
// of them: 105 us, 122 in large tiles; 256 of 500: 104 and 138; 16 of 8000: 100 either way.)  A chunk among as many idle
// requests is right there but slow (512 tokens behind 8000 among 511 idle ones: 440 us, 114 in large tiles).
// Large tiles are left whole by the host, without a workspace and a join, where the table is too short for a cut to pay, or where it
// holds no more than one request's tokens and a tile, if they fill the call's rows: a call of fewer tokens takes no longer
// than that.  Else the device chooses, which costs whole tiles 6 to 8 us for the lengths and the join that has nothing to do
// (a prompt of 300 in a table of 40960 keys 22 us, 16 in its own; 2000: 65 and 58; 8192: 501 and 493).
AttnPlan attn_plan(int S, int R, int HQ, int HKV, int D, long keys) {
  AttnPlan p;
  p.small = S <= R;
  const int g = HQ / HKV;
  const long rows = (long)S * g, tiles = (rows + kLargeRows - 1) / kLargeRows;  // were all of the tokens one request's
  const long s = slots_of(HKV), tau = (kLargeRows + g - 1) / g;
  const bool whole = whole_pays(s, 0, keys, 0, kOnceAndLaunch) ||
                     (R == 1 && keys - S <= kLargeRows && whole_pays_alone(s, tiles, 0, tau, kOnceAndLaunch) &&
                      whole_pays_alone(s, tiles, keys > S ? keys - S : 0, tau, kOnceAndLaunch));
  p.target = whole && !p.small ? 0 : ((p.small ? 2 : 1) * kCUs + HKV - 1) / HKV;  // workgroups that run at once
  p.grid = p.small ? 0 : (int)(rows / kLargeRows + (R < S ? R : S));  // whole tiles of a key head, at most
  // Where requests may have no token or few, several tiles for a workgroup are cheaper than workgroups without any, each of
  // which looks for its part through all requests.  (512 tokens behind 8000 keys among 511 idle requests, 513 rows: 114 us, 190 with a
  // workgroup for every tile that there could be; 512 requests of 2 tokens: 214, 325.)
  if (p.target > 0 && p.grid > 2 * rows / kLargeRows + p.target) p.grid = (int)(2 * rows / kLargeRows) + p.target;
  if (p.grid < p.target) p.grid = p.target;
  const long kept = (long)HKV * p.target * 2 * (p.small ? kSmallRows : kLargeRows);
  p.ws_bytes = kept * (D + 2) * 4 + (long)HKV * p.target * (long)sizeof(int4);
  return p;
}

// At most S HQ / 256 + R HKV < 2^20 + 2^22 workgroups of 512 threads: under a launch's 2^32.
template <int D, How HOW>
static hipError_t launch_large(const AttnArgs& a, unsigned grid, hipStream_t st) {
  constexpr int bytes = kRing * 64 * D * 4;
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(k_attn_large<D, HOW>), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attn_large<D, HOW>), dim3(grid), dim3(512), bytes, st, a);
  return hipGetLastError();
}

template <int D>
static hipError_t launch_d(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  const unsigned grid = (unsigned)p.grid * (unsigned)a.HKV, joins = (unsigned)(p.target * a.HKV);
  const long rows = (long)a.S * a.g;  // of a tile at most, too
  if (p.small) {
    hipLaunchKernelGGL(k_attn_small<D>, dim3(grid), dim3(256), 0, st, a);
    const unsigned jy = (unsigned)(((rows < kSmallRows ? rows : kSmallRows) + 3) / 4);
    hipLaunchKernelGGL((k_attn_join<D, kSmallRows>), dim3(joins, jy), dim3(256), 0, st, a);
    return hipGetLastError();
  }
  const hipError_t e = joins == 0 ? launch_large<D, kWhole>(a, grid, st) : launch_large<D, kEither>(a, grid, st);
  if (e != hipSuccess || joins == 0) return e;
  const unsigned jy = (unsigned)(((rows < kLargeRows ? rows : kLargeRows) + 3) / 4);
  hipLaunchKernelGGL((k_attn_join<D, kLargeRows>), dim3(joins, jy), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_attn(const AttnArgs& a, int D, const AttnPlan& p, hipStream_t st) {
  return D == 128 ? launch_d<128>(a, p, st) : launch_d<64>(a, p, st);
}

}  // namespace osc
