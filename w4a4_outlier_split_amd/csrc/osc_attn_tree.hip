// Attention of trees of drafted tokens over the paged cache.
//
//   O[t][hq] = sum_j softmax_j(scale * q . k_j) v_j      over the context j < kv - n, and the new keys that the
//                                                        bits of MASK[t] name
//
// with the running maximum and sum, the transposed products and the layouts of osc_attn.hip.  A tree's rows all see the
// context, which is nearly all of the keys: a tile's length is that of its request, and a mask is needed in the last steps only.
//
// Two kernels: tiles of 16 rows from registers where a tree's rows (nodes times the query heads of a key head) fit into one, tiles of 256
// on the ring of keys in LDS otherwise, so that a request's keys are read from memory once.  Every row of tiles is cut evenly among as
// many workgroups as run at once, since a step's few trees have no tiles to fill the card with; a second launch joins the cut ones.
// Measured with 32 query and 8 key heads of 128, both launches: 8 nodes in each of 32 requests, 109 thousand keys, 96 us, bound by HBM
// (441 MB in the first kernel's 92 us, 4.8 TB/s); 64 nodes there 123 to 129, where the tiles' steps of 2 us run beside the same bytes and 35 MB of
// partial outputs are written and read again; 256 nodes over 32700 keys 144 to 151, bound by the steps (2 us, of which the matrix unit works 0.85
// to 1); 16 nodes over 4000 keys 15.6, a chain of latencies: lengths and cuts 1.4, the request 0.8, pages, queries and masks 1.3, first keys 2.1, steps
// 2 to 4, stores 0.5, and two launches.
#include "osc_attn_dev.h"

namespace osc {
namespace {

typedef unsigned long long u64;

// ------------------------------------------------------------------ the cuts
// A request's tiles of ROWS rows, each as long as its keys (in steps of 64; 1 at least, so that rows without a key get their zeros).
template <int ROWS>
struct TreeRequest {
  int c0 = 0, n = 0, first = 0, kv = 0, tiles = 0, steps = 1;
  __device__ __forceinline__ TreeRequest() {}
  __device__ __forceinline__ TreeRequest(const AttnArgs& a, int r) {
    c0 = clampi(a.CU[r], 0, a.S);
    const int c1 = clampi(a.CU[r + 1], 0, a.S);
    n = c1 > c0 ? c1 - c0 : 0;
    const int held = a.KV[r] > 0 ? a.KV[r] : 0, beyond = a.CU[r + 1] > a.S ? a.CU[r + 1] - a.S : 0;
    const long at = (long)held - n - beyond;
    constexpr long most = 1l << 30;  // as many positions as a table can hold: 32 bits do from here on
    first = (int)(at < -most ? -most : at < most ? at : most);
    kv = clampi(first + n, 0, (int)((long)a.MB << a.sh));
    tiles = (int)(((long)n * a.g + ROWS - 1) / ROWS);
    steps = kv > 0 ? (kv + 63) >> 6 : 1;
  }
  __device__ __forceinline__ long all() const { return (long)tiles * steps; }
  // a lane's, in scalar registers
  __device__ __forceinline__ TreeRequest of(int lane) const {
    TreeRequest q;
    q.c0 = __builtin_amdgcn_readlane(c0, lane), q.n = __builtin_amdgcn_readlane(n, lane);
    q.first = __builtin_amdgcn_readlane(first, lane), q.kv = __builtin_amdgcn_readlane(kv, lane);
    q.tiles = __builtin_amdgcn_readlane(tiles, lane), q.steps = __builtin_amdgcn_readlane(steps, lane);
    return q;
  }
};

// Workgroup: key head h = blockIdx % HKV, part w = blockIdx / HKV of the row in which all tiles of the head stand, cut into equal
// parts, as many as workgroups run at once; body(t, h) for each tile of the part in turn.  A tile that a cut goes through has
// its unnormalised outputs left in the workspace: in the workgroup's second place where it begins there, in the first behind a cut.
// The workgroup in whose part such a tile begins notes it, for the join.
template <int ROWS, typename Body>
__device__ __forceinline__ void each_tree_tile(const TreeArgs& a, Body body) {
  typedef TreeRequest<ROWS> Req;
  const int h = blockIdx.x % a.HKV, w = blockIdx.x / a.HKV;
  const int lane = threadIdx.x & 63;
  const int per = (a.R + 63) >> 6;
  int r = 0, i = 0, parts = 1, over = 0;  // over < parts <= 512: their products fit into 32 bits
  long begin = 0, first = 0, end = 0, each = 0, all;
  // A lane has `per` requests; where that is one, it keeps it, and nobody reads the lengths again.
  const int r0 = lane * per < a.R ? lane * per : a.R, r1 = r0 + per < a.R ? r0 + per : a.R;
  Req own = r0 < r1 ? Req(a, r0) : Req();
  {
    long mine = own.all();
#pragma unroll 4
    for (int x = r0 + 1; x < r1; ++x) mine += Req(a, x).all();
    long upto = mine;
    const int lanes = (a.R + per - 1) / per;
    for (int d = 1; d < lanes; d <<= 1) {
      const long up = __shfl_up(upto, d);
      if (lane >= d) upto += up;
    }
    all = lane_of(upto, lanes - 1);
    long p = a.target;
    if (p > all) p = all;  // (two steps a part at least: 16 nodes over 500 keys 11.8 us, 8.9 so; 64 over 1000 16.1 and 12.7; the join is the same)
    parts = p < 1 ? 1 : (int)p;
    each = uniform(divide(all, parts));
    over = (int)(all - each * parts);
    if (w < parts && all > 0) {
      first = each * w + over * w / parts, end = each * (w + 1) + over * (w + 1) / parts;
      // the tile at `first`: its request, its number there, and where it begins
      const int src = __ffsll(__ballot(first < upto)) - 1;
      long from = upto - mine;
      int hit = r0;
      Req q = own;
      while (hit + 1 < r1 && first - from >= q.all()) {  // (what the lanes but src find is not used)
        from += q.all();
        q = Req(a, ++hit);
      }
      const int num = (int)divide(first > from ? first - from : 0, q.steps);
      r = __builtin_amdgcn_readlane(hit, src);
      i = __builtin_amdgcn_readlane(num, src);
      begin = lane_of(from + (long)num * q.steps, src);
    }
  }
  if (w >= parts || all == 0) {
    if (threadIdx.x == 0 && w < a.target) a.NOTE[h * a.target + w] = int4{0, 0, 0, 0};
    return;
  }
  const unsigned long long has = __ballot(own.n > 0);
  for (;;) {
    const Req q = per == 1 ? own.of(r) : Req(a, r).of(0);
    Tile t;
    t.tok0 = q.c0, t.first = q.first, t.kv = q.kv;
    t.pages = a.TABLE + (long)r * a.MB;
    t.rows = q.n * a.g;
    t.row0 = i * ROWS;
    const int len = q.steps;
    t.lo = begin < first ? (int)(first - begin) : 0;
    t.hi = begin + len > end ? (int)(end - begin) : len;
    const bool last = begin + len >= end;
    t.part = -1;
    if (begin < first || begin + len > end) t.part = (((long)h * a.target + w) * 2 + (begin < first ? 0 : 1)) * ROWS;
    if (last) {
      int ns = 0;
      if (begin >= first && begin + len > end) {  // the parts that begin in the tile
        ns = 1;
        for (int p0 = w + 1;; p0 += 64) {
          const int p = p0 + lane;
          const int more = __popcll(__ballot(p < parts && each * p + over * p / parts < begin + len));
          ns += more;
          if (more < 64) break;
        }
      }
      if (threadIdx.x == 0) a.NOTE[h * a.target + w] = int4{ns, t.row0, t.rows, t.tok0};
    } else {
      begin += len;
      if (++i == q.tiles) i = 0, r = per > 1 ? next_request(a, r) : r + __ffsll(has >> r >> 1);
    }
    body(t, h);
    if (last) return;
  }
}

template <int D>
__global__ __launch_bounds__(256, 2) void k_attn_tree_small(TreeArgs a) {
  __shared__ __align__(16) float lds[128 + 4 * 16 * (D + 4)];
  each_tree_tile<kSmallRows>(a, [&](const Tile& t, int h) { small_tile<D, true>(a, t, h, lds); });
}

template <int D>
__global__ __launch_bounds__(512, 2) void k_attn_tree_large(TreeArgs a) {
  extern __shared__ __align__(16) uint8_t dlds[];
  each_tree_tile<kLargeRows>(a, [&](const Tile& t, int h) { large_tile<D, true>(a, t, h, dlds); });
}

// Joins the parts of the tile that part w noted: o = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k with m the largest
// m_k, in a fixed order.  A lane has a piece of 16 bytes of a row's outputs, and reads its parts and their maxima and sums
// FLY at once: the parts lie far apart, and a load that waits for another takes 2 to 3 us.
// FIND, where there are fewer tiles than parts: workgroup j of a head looks for its j-th noted tile.  (A workgroup for each part, most of them
// with nothing to do: 256 nodes over 32700 keys 13.7 us, 9.3 so; 16 over 4000 19 and 4.)
// SHARE > 1, for few tiles of many parts each: that many wavefronts take parts of the same pieces in turn and join theirs through LDS
// (else a wavefront's chain is long and the card empty).
template <int D, int ROWS, int SHARE, bool FIND>
__global__ __launch_bounds__(512) void k_attn_tree_join(TreeArgs a) {
  constexpr int FLY = 4, P = D / 4;  // pieces of a row
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.x % a.HKV;
  int w = blockIdx.x / a.HKV;
  int4 note;
  if constexpr (FIND) {
    constexpr int MOST = 2 * kCUs / 64;  // a lane's notes
    int4 noted[MOST];
    int left = w;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      noted[i] = int4{0, 0, 0, 0};
      if (i * 64 < a.target && i * 64 + lane < a.target) noted[i] = a.NOTE[h * a.target + i * 64 + lane];
    }
    w = -1;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      u64 has = __ballot(noted[i].x > 0);
      const int n = __popcll(has);
      if (w < 0 && left < n) {
        for (; left > 0; --left) has &= has - 1;
        const int src = __ffsll(has) - 1;
        w = i * 64 + src;
        note = int4{__builtin_amdgcn_readlane(noted[i].x, src), __builtin_amdgcn_readlane(noted[i].y, src),
                    __builtin_amdgcn_readlane(noted[i].z, src), __builtin_amdgcn_readlane(noted[i].w, src)};
      }
      left -= n;
    }
    if (w < 0) return;
  } else {
    note = a.NOTE[h * a.target + w];
  }
  const int ns = __builtin_amdgcn_readfirstlane(note.x < a.target - w ? note.x : a.target - w);
  if (ns <= 0) return;
  // Which row of the tile, and which of its channels, the lane's piece holds: in order, or (tiles of 256 rows) 4 channels from 32 d + 8 i +
  // 4 half of row `col` of a wavefront's 32, where d, i come from the piece's store and half, col from its lane.
  const int piece = (SHARE > 1 ? blockIdx.y : blockIdx.y * 8 + wave) * 64 + lane;
  const int x = ROWS == kLargeRows ? piece / (32 * P) * 32 + (lane & 31) : piece / P;
  const int c = ROWS == kLargeRows ? (piece / 64 % (P / 2)) * 8 + 4 * (lane >> 5) : piece % P * 4;
  const int row = note.y + x, tok = row / a.g;
  // (a workspace that another call is writing as well may note anything: no row but the call's own)
  const bool mine = x < ROWS && row >= 0 && row < note.z && note.w >= 0 && note.w < a.S && tok < a.S - note.w;
  if (SHARE == 1 && !mine) return;
  // part w + k: in that workgroup's second place for k = 0, in its first for the others
  auto place = [&](int k) { return (((long)h * a.target + w + k) * 2 + (k == 0 ? 1 : 0)) * ROWS; };
  float m = neg_inf(), l = 0.0f;
  v4f acc = {};
  if (mine)
    for (int k0 = SHARE > 1 ? wave : 0; k0 < ns; k0 += SHARE * FLY) {
      float2 v[FLY];
      v4f o[FLY];
#pragma unroll
      for (int i = 0; i < FLY; ++i) {
        v[i] = float2{0.0f, 0.0f}, o[i] = v4f{};
        if (k0 + i * SHARE < ns) {
          const long at = place(k0 + i * SHARE);
          v[i] = *reinterpret_cast<const float2*>(a.PM + (at + x) * 2);
          o[i] = reinterpret_cast<const v4f*>(a.PO + at * D)[piece];
        }
      }
      float mn = m;
#pragma unroll
      for (int i = 0; i < FLY; ++i) mn = v[i].y != 0.0f ? fmaxf(mn, v[i].x) : mn;  // a part of no keys has a sum of 0, and its output does not count
      const float z = mn == neg_inf() ? 0.0f : mn, fm = __builtin_amdgcn_exp2f(m - z);
      l *= fm, acc *= fm;
      m = mn;
#pragma unroll
      for (int i = 0; i < FLY; ++i) {
        const bool counts = v[i].y != 0.0f;
        const float f = counts ? __builtin_amdgcn_exp2f(v[i].x - z) : 0.0f;
        l += counts ? f * v[i].y : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += counts ? o[i][e] * f : 0.0f;
      }
    }
  if constexpr (SHARE > 1) {
    __shared__ float2 ml[SHARE][64];
    __shared__ v4f out[SHARE][64];
    ml[wave][lane] = float2{m, l}, out[wave][lane] = acc;
    __syncthreads();
    if (wave != 0 || !mine) return;
#pragma unroll
    for (int k = 1; k < SHARE; ++k) m = fmaxf(m, ml[k][lane].x);
    const float z = m == neg_inf() ? 0.0f : m;
    l = 0.0f, acc = v4f{};
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
      const float f = __builtin_amdgcn_exp2f(ml[k][lane].x - z);
      l += f * ml[k][lane].y, acc += f * out[k][lane];
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  v4bf out4;
#pragma unroll
  for (int e = 0; e < 4; ++e) out4[e] = (__bf16)(acc[e] * inv);
  *reinterpret_cast<v4bf*>(static_cast<__bf16*>(a.O) + ((long)(note.w + tok) * a.HQ + h * a.g + (row - tok * a.g)) * D + c) = out4;
}

}  // namespace

// Small tiles where a tree's rows fit into one.  (4 query heads to a key head, 64 trees over 2000 keys each: of 4 nodes 95 us, 102 in large tiles;
// of 8 nodes, which would be two small tiles, 102 in large ones.  A third kernel, with tiles of 32 rows from registers, took 99 there, and 96 where large
// tiles take 91, 32 trees of 8 nodes over 109 thousand keys: not kept.)
TreePlan attn_tree_plan(int HQ, int HKV, int D, int N) {
  TreePlan p;
  p.N = N;
  const bool small = N * (HQ / HKV) <= kSmallRows;
  p.rows = small ? kSmallRows : kLargeRows;
  p.target = ((small ? 2 : 1) * kCUs + HKV - 1) / HKV;  // workgroups that run at once
  const long kept = (long)HKV * p.target * 2 * p.rows;
  p.ws_bytes = kept * (D + 2) * 4 + (long)HKV * p.target * (long)sizeof(int4);
  return p;
}

template <int D, int ROWS>
static hipError_t launch_rows(const TreeArgs& a, int N, hipStream_t st) {
  const unsigned grid = (unsigned)a.target * (unsigned)a.HKV;
  if constexpr (ROWS == kLargeRows) {
    constexpr int bytes = kRing * 64 * D * 4 + 16;
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(k_attn_tree_large<D>), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_attn_tree_large<D>, dim3(grid), dim3(512), bytes, st, a);
  } else {
    hipLaunchKernelGGL(k_attn_tree_small<D>, dim3(grid), dim3(256), 0, st, a);
  }
  // the 64 pieces of a tile that a wavefront joins; no more rows than the call has tokens
  const long most = ((long)a.S * a.g + 31) / 32 * 32, pieces = (most < ROWS ? most : ROWS) * (D / 4) / 64;
  const long all = (long)a.S * a.g / ROWS + (a.R < a.S ? a.R : a.S);  // tiles that there can be, whatever the lengths
  const unsigned found = (unsigned)((all < a.target ? all : a.target) * a.HKV), eights = (unsigned)((pieces + 7) / 8);
  // Tiles of 24 parts and more, were all requests alike, are joined by 8 wavefronts each.  The search pays where at most half of the parts can
  // begin a tile (8 trees of 64 nodes, 32 parts a head: 8.9 us with it, 14.8 without; 15 trees 15.6 and 13.0, 32 of 8 nodes 11.4 and 4.9).
  if (24 * (long)a.R * ((N * a.g + ROWS - 1) / ROWS) <= a.target) {
    hipLaunchKernelGGL((k_attn_tree_join<D, ROWS, 8, true>), dim3(found, (unsigned)pieces), dim3(512), 0, st, a);
  } else if (2 * all <= a.target) {
    hipLaunchKernelGGL((k_attn_tree_join<D, ROWS, 1, true>), dim3(found, eights), dim3(512), 0, st, a);
  } else {
    hipLaunchKernelGGL((k_attn_tree_join<D, ROWS, 1, false>), dim3(grid, eights), dim3(512), 0, st, a);
  }
  return hipGetLastError();
}

template <int D>
static hipError_t launch_d(const TreeArgs& a, const TreePlan& p, hipStream_t st) {
  return p.rows == kSmallRows ? launch_rows<D, kSmallRows>(a, p.N, st) : launch_rows<D, kLargeRows>(a, p.N, st);
}

hipError_t launch_attn_tree(const TreeArgs& a, int D, const TreePlan& p, hipStream_t st) {
  return D == 128 ? launch_d<128>(a, p, st) : launch_d<64>(a, p, st);
}

}  // namespace osc
