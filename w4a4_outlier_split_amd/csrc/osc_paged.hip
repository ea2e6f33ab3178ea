// The page plan of a serving step and the write of its keys and values into the paged cache.
#include "osc_internal.h"

namespace osc {
namespace {

typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

constexpr long kMaxInt = 0x7FFFFFFF;

// ------------------------------------------------------------------ page plan
// Latency-bound (a few kilobytes): one launch, and as short a chain of dependent loads as there is.  Every
// workgroup takes the prefix sums over the requests itself (R <= OSC_MAX_REQUESTS lengths from L2, kept in
// LDS) instead of waiting for another launch, and then a token and a new table entry a thread, each
// found by a binary search in those sums.  A token behind the pages that a request had reads its page from
// the free list, not from the table that other workgroups are writing, so no order between them matters.
// 64 decodes take 3.9 us, 512 requests with 20 thousand tokens 5.4 (8.7 with four tokens a thread and the lengths
// read again for each).
__device__ __forceinline__ int upper(const int* v, int n, int t) {  // first index with v[i] > t
  int lo = 0;
  while (n > 0) {
    const int h = n >> 1;
    if (v[lo + h] > t) n = h;
    else lo += h + 1, n -= h + 1;
  }
  return lo;
}

__global__ __launch_bounds__(256) void k_page_plan(PlanArgs a) {
  extern __shared__ int lds[];
  int* cu = lds;                 // [R + 1] tokens before request r
  int* pg = lds + a.R + 1;       // [R + 1] new pages before request r
  int* ctx = lds + 2 * (a.R + 1);  // [R] tokens in the cache
  __shared__ long wsum[2][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = a.HEAD ? a.HEAD[0] : 0;
  const long head = h > 0 ? h : 0;
  const long cap = (long)a.MB << a.sh;  // positions that a table row holds
  const long m = (1l << a.sh) - 1;
  const int per = (a.R + 255) / 256;
  const int r0 = tid * per, r1 = r0 + per < a.R ? r0 + per : a.R;
  auto had = [&](long c) { return ((c < cap ? c : cap) + m) >> a.sh; };  // pages of c tokens
  auto len = [&](int r) { return (long)(a.NEW[r] > 0 ? a.NEW[r] : 0); };
  long sn = 0, sp = 0;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const long c = a.CTX[r] > 0 ? a.CTX[r] : 0, n = len(r);
    ctx[r] = (int)c;
    sn += n, sp += had(c + n) - had(c);
  }
  long in = sn, ip = sp;  // inclusive over the wavefront's threads
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long un = __shfl_up(in, d), up = __shfl_up(ip, d);
    if (lane >= d) in += un, ip += up;
  }
  if (lane == 63) wsum[0][wave] = in, wsum[1][wave] = ip;
  __syncthreads();
  long bn = in - sn, bp = ip - sp;
  for (int w = 0; w < wave; ++w) bn += wsum[0][w], bp += wsum[1][w];
  for (int r = r0; r < r1; ++r) {
    const long c = ctx[r], n = len(r);
    cu[r] = (int)(bn < kMaxInt ? bn : kMaxInt);
    pg[r] = (int)(bp < kMaxInt ? bp : kMaxInt);
    if (blockIdx.x == 0) {
      a.CU[r] = cu[r];
      a.KV[r] = (int)(c + n < kMaxInt ? c + n : kMaxInt);
    }
    bn += n, bp += had(c + n) - had(c);
  }
  if (tid == 255) {  // the last thread's sums are the totals, with or without requests of its own
    const long tn = wsum[0][0] + wsum[0][1] + wsum[0][2] + wsum[0][3];
    const long tp = wsum[1][0] + wsum[1][1] + wsum[1][2] + wsum[1][3];
    cu[a.R] = (int)(tn < kMaxInt ? tn : kMaxInt);
    pg[a.R] = (int)(tp < kMaxInt ? tp : kMaxInt);
    if (blockIdx.x == 0) a.CU[a.R] = cu[a.R], a.USED[0] = pg[a.R];
  }
  __syncthreads();
  auto from_pool = [&](long j) {  // the j-th page of this step, -1 behind the list or off the pool
    const int id = head + j < a.F ? a.FREE[head + j] : -1;
    return id >= 0 && id < a.NP ? id : -1;
  };
  const long stride = (long)gridDim.x * 256, first = (long)blockIdx.x * 256 + tid;
  for (long t = first; t < a.T; t += stride) {
    int slot = -1, pos = -1;
    if (t < cu[a.R]) {
      const int r = upper(cu, a.R + 1, (int)t) - 1;
      const long at = (long)ctx[r] + (t - cu[r]);
      pos = (int)(at < kMaxInt ? at : kMaxInt);
      if (at < cap) {
        const long q = at >> a.sh, have = had(ctx[r]);
        int id;
        if (q < have) {
          id = a.TABLE[(long)r * a.MB + q];
          if (id < 0 || id >= a.NP) id = -1;
        } else {
          id = from_pool(pg[r] + (q - have));
        }
        if (id >= 0) slot = (id << a.sh) + (int)(at & m);
      }
    }
    a.POS[t] = pos;
    a.SLOT[t] = slot;
  }
  for (long j = first; j < pg[a.R]; j += stride) {
    const int r = upper(pg, a.R + 1, (int)j) - 1;
    a.TABLE[(long)r * a.MB + had(ctx[r]) + (j - pg[r])] = from_pool(j);
  }
}

// ------------------------------------------------------------------ heads -> queries and cache
// Per head of a token: q and k are normed over the head (binary32 sum of D squares, if asked),
// rotated (the halves x1, x2 of the head by the position's angles: x1 cos - x2 sin, x2 cos + x1 sin)
// and rounded once; v is copied.  HBM-bound: every element is read and written once (4097 tokens of 32 + 8 + 8 heads
// of 128, 103 MB: 22.5 us, 4.6 TB/s, as a copy; 16 tokens 3 us, the latency of slot, row and store).
// One launch for both parts, so that small steps pay one; neither part waits for the other:
//   blocks of the first part: 256 threads take 2048 / D heads of q and k, D/16 lanes a head, each
//     with 8 channels of both halves, so the rotation stays in a lane and the norm crosses D/16.
//   blocks of the second part: V's cache is [D][page], so 64 tokens of one head turn round in LDS
//     and each store instruction writes one channel of 64 tokens, neighbours in the page (written
//     token by token, 2 bytes at a time would each touch a line of their own).
template <int D>
__global__ __launch_bounds__(256) void k_qkv_append(AppendArgs a, int qk_blocks) {
  constexpr int LH = D / 16;           // lanes a head
  constexpr int HB = 256 / LH;         // heads a block
  const int tid = threadIdx.x;
  const long ntok = (long)a.NP << a.sh;
  const int W = a.HQ + 2 * a.HKV;
  auto usable = [&](int slot, int pos) { return slot >= 0 && slot < ntok && (!a.CS || (pos >= 0 && pos < a.P)); };
  if ((int)blockIdx.x < qk_blocks) {
    const long item = (long)blockIdx.x * HB + tid / LH;
    const int heads = a.HQ + a.HKV;
    if (item >= (long)a.S * heads) return;  // a head's lanes leave together
    const int t = (int)(item / heads), hd = (int)(item - (long)t * heads);
    const int c = (tid % LH) * 8;
    const int slot = a.SLOT[t], pos = a.CS ? a.POS[t] : 0;
    const __bf16* src = static_cast<const __bf16*>(a.QKV) + ((long)t * W + hd) * D + c;
    const bf8 r1 = *reinterpret_cast<const bf8*>(src), r2 = *reinterpret_cast<const bf8*>(src + D / 2);
    float x1[8], x2[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x1[i] = (float)r1[i], x2[i] = (float)r2[i];
    const __bf16* w = static_cast<const __bf16*>(hd < a.HQ ? a.WQ : a.WK);
    if (w) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x1[i], x1[i], __builtin_fmaf(x2[i], x2[i], s));
#pragma unroll
      for (int d = 1; d < LH; d <<= 1) s += __shfl_xor(s, d);
      const float rstd = 1.0f / __builtin_sqrtf(s / (float)D + a.eps);
      const bf8 w1 = *reinterpret_cast<const bf8*>(w + c), w2 = *reinterpret_cast<const bf8*>(w + c + D / 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) x1[i] *= rstd * (float)w1[i], x2[i] *= rstd * (float)w2[i];
    }
    if (!usable(slot, pos)) return;
    if (a.CS) {
      const float* cs = a.CS + (long)pos * D + c;
      float co[8], si[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) co[i] = cs[i], si[i] = cs[i + D / 2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = x1[i], v = x2[i];
        x1[i] = u * co[i] - v * si[i];
        x2[i] = v * co[i] + u * si[i];
      }
    }
    __bf16* dst;
    if (hd < a.HQ) {
      dst = static_cast<__bf16*>(a.Q) + ((long)t * a.HQ + hd) * D + c;
    } else {
      const long page = slot >> a.sh;
      dst = static_cast<__bf16*>(a.KC) + (((page * a.HKV + (hd - a.HQ)) << a.sh) + (slot & ((1 << a.sh) - 1))) * D + c;
    }
    bf8 o1, o2;
#pragma unroll
    for (int i = 0; i < 8; ++i) o1[i] = (__bf16)x1[i], o2[i] = (__bf16)x2[i];
    *reinterpret_cast<bf8*>(dst) = o1;
    *reinterpret_cast<bf8*>(dst + D / 2) = o2;
    return;
  }
  // V: row stride of D/2 + 1 dwords, odd, so that 64 tokens' dwords of one channel pair fall on 64 banks
  __shared__ uint32_t tile[64 * (D / 2 + 1)];
  const int vb = blockIdx.x - qk_blocks;
  const int h = vb % a.HKV, t0 = (vb / a.HKV) * 64;
  constexpr int CH = D / 8;  // 16-byte pieces of a head
  for (int i = tid; i < 64 * CH; i += 256) {
    const int t = i / CH, c = i % CH;
    if (t0 + t < a.S) {
      const u4 v = *reinterpret_cast<const u4*>(static_cast<const uint16_t*>(a.QKV) +
                                                ((long)(t0 + t) * W + a.HQ + a.HKV + h) * D + c * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[t * (D / 2 + 1) + c * 4 + j] = v[j];
    }
  }
  __syncthreads();
  const int lane = tid & 63, wave = tid >> 6;
  if (t0 + lane >= a.S) return;
  const int slot = a.SLOT[t0 + lane];
  if (!usable(slot, a.CS ? a.POS[t0 + lane] : 0)) return;
  uint16_t* dst = static_cast<uint16_t*>(a.VC) + ((((long)(slot >> a.sh) * a.HKV + h) * D) << a.sh) +
                  (slot & ((1 << a.sh) - 1));
#pragma unroll 8
  for (int i = 0; i < D / 8; ++i) {
    const int c2 = wave * (D / 8) + i;  // channel pair
    const uint32_t v = tile[lane * (D / 2 + 1) + c2];
    dst[(long)(2 * c2) << a.sh] = (uint16_t)v;
    dst[(long)(2 * c2 + 1) << a.sh] = (uint16_t)(v >> 16);
  }
}

}  // namespace

hipError_t launch_page_plan(const PlanArgs& a, hipStream_t st) {
  // a token a thread, at least one workgroup (the sums), at most two for each of the 256 CUs
  const long want = ((long)a.T + 255) / 256;
  const unsigned grid = (unsigned)(want < 1 ? 1 : want > 512 ? 512 : want);
  hipLaunchKernelGGL(k_page_plan, dim3(grid), dim3(256), (size_t)(3 * a.R + 2) * sizeof(int), st, a);
  return hipGetLastError();
}

hipError_t launch_qkv_append(const AppendArgs& a, hipStream_t st) {
  const int hb = a.D == 128 ? 32 : 64;
  const long qk = ((long)a.S * (a.HQ + a.HKV) + hb - 1) / hb;
  const long v = (long)((a.S + 63) / 64) * a.HKV;
  if (a.D == 128) hipLaunchKernelGGL(k_qkv_append<128>, dim3((unsigned)(qk + v)), dim3(256), 0, st, a, (int)qk);
  else hipLaunchKernelGGL(k_qkv_append<64>, dim3((unsigned)(qk + v)), dim3(256), 0, st, a, (int)qk);
  return hipGetLastError();
}

}  // namespace osc
