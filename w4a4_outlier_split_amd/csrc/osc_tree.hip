// Trees of drafted tokens: positions and masks from parents, the walk along the chosen tokens, and the move of the
// accepted nodes' keys and values.
#include "osc_internal.h"

namespace osc {
namespace {

typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// a request's rows: the first, and how many nodes of its tree count
struct Nodes {
  int c0, n, nodes;
  __device__ __forceinline__ Nodes(const int32_t* CU, int r, int T, int N) {
    c0 = clampi(CU[r], 0, T);
    const int c1 = clampi(CU[r + 1], 0, T);
    n = c1 > c0 ? c1 - c0 : 0;
    nodes = n < N ? n : N;
  }
};

// ------------------------------------------------------------------ positions and masks
// anc(i) = {i} u anc(parent(i)), depth(i) = |anc(i)| - 1.  A node a thread, a request a workgroup: in round k a node adds the
// set of the ancestor 2^k steps above to its own and takes that one's as its next, so chains of 256 nodes are done in 8
// rounds.  Latency-bound: two loads one behind the other, the rounds in LDS, one store (16 trees of 16 nodes 2.6 us, 512 of
// 200 with 4 words of mask each 6.3).  One more workgroup for each 256 rows that the call's padding may have fills those (up to
// 64; the loop takes the rest).
template <int W>
__global__ __launch_bounds__(64 * W) void k_tree_plan(TreeMaskArgs a) {
  constexpr int M = 64 * W;
  const int i = threadIdx.x;
  if ((int)blockIdx.x >= a.R) {  // rows of no request
    const int before = clampi(a.CU[0], 0, a.T), behind = clampi(a.CU[a.R], 0, a.T);
    const long none = before + (a.T - behind);
    const long stride = (long)(gridDim.x - a.R) * M;
    for (long x = (long)(blockIdx.x - a.R) * M + i; x < none; x += stride) {
      const long t = x < before ? x : behind + (x - before);
      a.POS[t] = -1;
#pragma unroll
      for (int w = 0; w < W; ++w) a.MASK[t * W + w] = 0;
    }
    return;
  }
  __shared__ u64 mask[W][M];
  __shared__ short up[M];
  const Nodes q(a.CU, blockIdx.x, a.T, a.N);
  const int ctx = a.CTX[blockIdx.x];
  const bool live = i < q.nodes;
  int p = live ? a.PARENT[q.c0 + i] : -1;
  if (p < 0 || p >= i) p = -1;
  u64 m[W];
#pragma unroll
  for (int w = 0; w < W; ++w) m[w] = i >> 6 == w ? 1ull << (i & 63) : 0, mask[w][i] = m[w];
  up[i] = (short)p;
  for (int far = 1; far < M; far *= 2) {
    if (!__syncthreads_or(p >= 0)) break;
    if (p >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) m[w] |= mask[w][p];
      p = up[p];
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) mask[w][i] = m[w];
    up[i] = (short)p;
  }
  if (live) {
    int depth = -1;
#pragma unroll
    for (int w = 0; w < W; ++w) depth += __popcll(m[w]), a.MASK[(long)(q.c0 + i) * W + w] = m[w];
    const long pos = (long)(ctx > 0 ? ctx : 0) + depth;
    a.POS[q.c0 + i] = (int)(pos < 0x7FFFFFFF ? pos : 0x7FFFFFFF);
  }
  for (int x = q.nodes + i; x < q.n; x += M) {
    a.POS[q.c0 + x] = -1;
#pragma unroll
    for (int w = 0; w < W; ++w) a.MASK[(long)(q.c0 + x) * W + w] = 0;
  }
}

// ------------------------------------------------------------------ the accepted path
// A wavefront a request, W nodes a lane.  Each step asks all nodes at once whether they are a child of the path's last node with
// the chosen token, so it costs W comparisons and a ballot, whatever the tree's size.  Latency-bound: offsets, then
// all of the nodes' words in one go, then the steps in registers (one tree of 16 nodes 1.7 us, 32 of 64 nodes 3.4 to 4.7).
template <int W>
__global__ __launch_bounds__(64) void k_tree_accept(AcceptArgs a) {
  const int r = blockIdx.x, lane = threadIdx.x;
  const Nodes q(a.CU, r, a.T, a.N);
  int parent[W], token[W], choice[W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int i = 64 * w + lane;
    parent[w] = -1, token[w] = choice[w] = -1;
    if (i < q.nodes) {
      const long t = q.c0 + i;
      const int p = a.PARENT[t], slot = a.SLOT[t], pos = a.P > 0 ? a.POS[t] : 0;
      token[w] = a.TOKEN[t];
      choice[w] = a.CHOICE[t * a.ldc];
      const bool written = slot >= 0 && (a.P == 0 || (pos >= 0 && pos < a.P));
      // a node that can follow: its parent's number; -2 for one that can be the first
      parent[w] = !written ? -1 : i == 0 ? -2 : p >= 0 && p < i ? p : -1;
    }
  }
  int acc = 0, cur = -1, next = -1;
  if (__builtin_amdgcn_readlane(parent[0], 0) == -2) cur = 0;
  while (cur >= 0) {  // at most `nodes` steps: each node is behind the one before
    if (lane == 0) a.PATH[(long)r * a.N + acc] = cur;
    ++acc;
    next = -1;
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (cur >> 6 == w) next = __builtin_amdgcn_readlane(choice[w], cur & 63);
    int child = -1;
#pragma unroll
    for (int w = W - 1; w >= 0; --w) {
      const u64 hit = __ballot(parent[w] == cur && token[w] == next && next >= 0);
      if (hit) child = 64 * w + __ffsll(hit) - 1;
    }
    cur = child;
  }
  for (int k = acc + lane; k < a.N; k += 64) a.PATH[(long)r * a.N + k] = -1;
  if (lane == 0) a.ACC[r] = acc, a.NEXT[r] = next;
}

// ------------------------------------------------------------------ the move in the caches
// Node PATH[k] goes to the slot of node k <= PATH[k].  Threads own a piece of a slot's keys (16 bytes), four of a wavefront a channel of the values,
// and take the moves in turn, four in flight: a slot that is written was read before, since a later move reads from behind it.
// Values stand 2 bytes a slot and channel, so each is a line of its own, and the lines bound it: 28 moves of 32 trees in 36 layers
// with 8 heads of 128, 8 MB by what moves, touch 73 MB of lines and take 26 to 28 us.  Moves in flight by lanes, rather than one behind the other in a
// thread (37 to 43): a load of 64 channels waits for 64 lines.  (Two lanes a channel 29 to 30, eight 34 to 35; two layers a
// workgroup 25 to 28, four 30 to 32.)
__global__ __launch_bounds__(256) void k_tree_commit(CommitArgs a, int blocks) {
  __shared__ int from[OSC_MAX_TREE], to[OSC_MAX_TREE];
  __shared__ int moves;
  const int part = blockIdx.x % blocks, r = blockIdx.x / blocks, layer = blockIdx.y;
  const Nodes q(a.CU, r, a.T, a.N);
  const int acc = clampi(a.ACC[r], 0, q.nodes);
  if (acc < 2) return;
  // the moves in order, without those that stay
  const int k = threadIdx.x, lane = k & 63;
  int src = -1, dst = -1;
  if (k > 0 && k < acc) {
    const int p = a.PATH[(long)r * a.N + k];
    if (p > k && p < q.nodes) src = a.SLOT[q.c0 + p], dst = a.SLOT[q.c0 + k];
  }
  const long slots = (long)a.NP << a.sh;
  const bool move = src >= 0 && dst >= 0 && src < slots && dst < slots;
  const u64 all = __ballot(move);
  __shared__ int ahead[4];
  if (lane == 0) ahead[k >> 6] = __popcll(all);
  __syncthreads();
  int at = __popcll(all & ((1ull << lane) - 1));
  for (int w = 0; w < k >> 6; ++w) at += ahead[w];
  if (move) from[at] = src, to[at] = dst;
  if (k == 255) moves = at + (move ? 1 : 0);
  __syncthreads();
  const int n = moves, mask = (1 << a.sh) - 1;
  const int pieces = a.HKV * a.D / 8, x = part * 256 + k;  // 16-byte pieces of a token's keys (8 at least); then its values' channels, four threads each
  if (x < pieces) {
    uint8_t* kc = static_cast<uint8_t*>(a.KC[layer]);
    const int row = a.D / 8, h = x / row, c = x - h * row;
    auto place = [&](int s) { return kc + ((((((long)(s >> a.sh) * a.HKV + h) << a.sh) + (s & mask)) * a.D + 8 * c) << 1); };
    for (int i = 0; i < n; i += 4) {
      u4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const u4*>(place(from[i + j < n ? i + j : n - 1]));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) *reinterpret_cast<u4*>(place(to[i + j])) = v[j];
    }
  } else if (x < pieces + 4 * a.HKV * a.D) {
    uint16_t* vc = static_cast<uint16_t*>(a.VC[layer]);
    const int y = (x - pieces) / 4, turn = (x - pieces) % 4, h = y / a.D, d = y - h * a.D;
    auto place = [&](int s) { return vc + (((((long)(s >> a.sh) * a.HKV + h) * a.D + d) << a.sh) + (s & mask)); };
    for (int i = turn; i - turn < n; i += 4) {
      uint16_t v = 0;
      if (i < n) v = *place(from[i]);
      __builtin_amdgcn_wave_barrier();  // the four have read, then they write
      if (i < n) *place(to[i]) = v;
    }
  }
}

}  // namespace

hipError_t launch_tree_plan(const TreeMaskArgs& a, hipStream_t st) {
  const long pad = ((long)a.T + 255) / 256;
  const dim3 grid((unsigned)(a.R + (pad > 64 ? 64 : pad)));
  switch (a.W) {
    case 1: hipLaunchKernelGGL(k_tree_plan<1>, grid, dim3(64), 0, st, a); break;
    case 2: hipLaunchKernelGGL(k_tree_plan<2>, grid, dim3(128), 0, st, a); break;
    case 3: hipLaunchKernelGGL(k_tree_plan<3>, grid, dim3(192), 0, st, a); break;
    default: hipLaunchKernelGGL(k_tree_plan<4>, grid, dim3(256), 0, st, a); break;
  }
  return hipGetLastError();
}

hipError_t launch_tree_accept(const AcceptArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.R);
  switch ((a.N + 63) / 64) {
    case 1: hipLaunchKernelGGL(k_tree_accept<1>, grid, dim3(64), 0, st, a); break;
    case 2: hipLaunchKernelGGL(k_tree_accept<2>, grid, dim3(64), 0, st, a); break;
    case 3: hipLaunchKernelGGL(k_tree_accept<3>, grid, dim3(64), 0, st, a); break;
    default: hipLaunchKernelGGL(k_tree_accept<4>, grid, dim3(64), 0, st, a); break;
  }
  return hipGetLastError();
}

// At most 4096 requests times 2112 parts (1024 heads of 128) by 128 layers.
hipError_t launch_tree_commit(const CommitArgs& a, hipStream_t st) {
  const int blocks = (a.HKV * a.D / 8 + 4 * a.HKV * a.D + 255) / 256;
  hipLaunchKernelGGL(k_tree_commit, dim3((unsigned)(a.R * blocks), (unsigned)a.layers), dim3(256), 0, st, a, blocks);
  return hipGetLastError();
}

}  // namespace osc
