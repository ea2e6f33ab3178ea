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
#include "osc_attn_dev.h"

namespace osc {
namespace {

constexpr int kMaxCuts = 61;    // of one tile: its parts, two more at most, are the lanes of the join
// Keys that a workgroup's part has at least.  (A prompt of 300 cut at 64, 128, 256: 24, 30, 38 us; 200 tokens on one key
// head behind 800: 35, 31, 34.)
constexpr int kMinKeys = 128;

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
  each_tile<kSmallRows, kCut>(a, [&](const Tile& t, int h) { small_tile<D, false>(a, t, h, lds); });
}

// Heads of 64 need half the LDS and may have two workgroups a CU, if 128 registers do.  (8192 tokens in a table of 40960 keys:
// 315 us, 350 with the 140 registers that the cuts would take; 33 tokens over 32700 keys 39 and 38.)
template <int D, How HOW>
__global__ __launch_bounds__(512, D == 64 ? 4 : 2) void k_attn_large(AttnArgs a) {
  extern __shared__ __align__(16) uint8_t dlds[];
  each_tile<kLargeRows, HOW>(a, [&](const Tile& t, int h) { large_tile<D, false>(a, t, h, dlds); });
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
