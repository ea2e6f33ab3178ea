// Attention of new tokens over the paged cache.
//
//   O[t][hq] = sum_j softmax_j(scale * q . k_j) v_j      over the keys j <= kv - n + i
//
// for token i of the n new tokens of a request whose cache holds kv keys (its new ones included), in
// one pass over the keys: with m the running maximum of a row's scores and l the running sum of
// exp(s - m), a tile of keys adds P = exp(S - m) to l and P V to the unnormalised output, and where
// m grows both are scaled by exp(m_old - m_new).  Scores, m, l and the output are binary32; P is
// rounded to bf16 for the matrix instruction (each weight off by at most 2^-9 of itself, as V's own
// rounding is), l sums the unrounded P.
//
// The HQ / HKV query heads that read one key head are rows of one tile, token by token, so a tile's
// keys serve all of them.  Both products run transposed, S^T = K Q^T and O^T = V^T P^T: a lane then
// holds scores of one query only (its maximum and sum are in-lane), and since the keys' order inside
// a tile is free, K's rows are read in the order that leaves each lane's scores as the very operand
// of the second product, with no exchange between lanes.  V^T's rows are contiguous keys in the
// cache's V layout [page][head][D][slot].
//
// Two tile shapes, one launch, chosen per request by its row count n * HQ/HKV:
//   small (at most kSmallRows): 16 rows, the cache read from memory straight into registers; the
//     four wavefronts take 32 keys each in turn and are merged at the end.  HBM-bound.
//   large: 128 rows, four wavefronts of 32 rows each; 64 keys of K and V^T at a time in LDS, loaded
//     by LDS-DMA while the previous 64 are worked on.  Bound by the matrix and vector units.
// With few tiles the keys are cut into ranges whose unnormalised outputs go to the workspace and are
// joined by a second launch in a fixed order.  The lengths are on the device, so the cut is made there:
// every workgroup adds up the step's work, from which follow the steps of 64 keys that one unit of
// work takes, each request's number of ranges, and the unit that is the workgroup's own.
#include "osc_device.h"
#include "osc_internal.h"

namespace osc {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

constexpr int kSmallRows = 32;
constexpr int kLargeRows = 128;
constexpr int kSlots = 512;     // workgroups that run at once: two on each of 256 CUs
constexpr int kMaxSplit = 64;   // ranges of a request's keys (the join's lanes)
constexpr int kMinSteps = 4;    // 64-key steps that a range has at least
// the running maximum is left as it is while no score exceeds it by more than 2^kSlack (in the
// exponent of 2): P is then at most 2^kSlack, which binary32 sums and bf16's exponent take as well
constexpr float kSlack = 8.0f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

struct Tile {
  int row0, rows;  // the tile's rows (token, head of the group): first and end, inside the request
  int split, ns;   // which of the request's ranges of keys
  int tok0, n;     // the request's first token and token count
  int kv;          // keys of the request
  const int32_t* pages;
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

__device__ __forceinline__ void request(const AttnArgs& a, int r, Tile& t) {
  const int c0 = clampi(a.CU[r], 0, a.S), c1 = clampi(a.CU[r + 1], 0, a.S);
  t.tok0 = c0;
  t.n = c1 > c0 ? c1 - c0 : 0;
  t.kv = clampi(a.KV[r], 0, (int)((long)a.MB << a.sh));
  t.pages = a.TABLE + (long)r * a.MB;
}

// the page of key `key`, -1 behind the request's keys or off the pool
__device__ __forceinline__ int page_of(const AttnArgs& a, const Tile& t, int key) {
  const int id = key < t.kv ? t.pages[key >> a.sh] : -1;
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

// ------------------------------------------------------------------ small tiles
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
  const int last = live ? t.kv - t.n + tok : -1;  // the last key of the lane's row
  const int tok_end = ((t.row0 + 16 < t.rows ? t.row0 + 16 : t.rows) - 1) / g;
  const int kend = clampi(t.kv - t.n + tok_end + 1, 0, t.kv);
  const int steps = (kend + 31) >> 5;
  const int lo = (int)((long)steps * t.split / t.ns), hi = (int)((long)steps * (t.split + 1) / t.ns);

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
    v8bf p;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x][i], c, -mc));
        l += e;
        p[4 * x + i] = (__bf16)e;
      }
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[d], p, o[d], 0, 0, 0);
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  // merge the wavefronts: m, l and O^T of each through LDS
  float* ml = lds;                   // [4][2][16]
  float* ob = lds + 128;             // [4][16][D + 4]
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
  const int tk = r / g;
  const long at = (long)(t.tok0 + tk) * a.HQ + h * g + (r - tk * g);
  if (a.CNT && t.split == 0 && d0 == 0) a.CNT[at] = t.ns;
  if (t.ns == 1) {
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;  // no key: zeros
#pragma unroll
    for (int i = 0; i < PT; i += 4) {
      v4bf b;
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = (__bf16)(acc[i + j] * inv);
      *reinterpret_cast<v4bf*>(static_cast<__bf16*>(a.O) + at * D + d0 + i) = b;
    }
  } else {
    const long rows = (long)a.S * a.HQ;
#pragma unroll
    for (int i = 0; i < PT; i += 4)
      *reinterpret_cast<v4f*>(a.PO + (t.split * rows + at) * D + d0 + i) = v4f{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
    if (d0 == 0) *reinterpret_cast<float2*>(a.PM + (t.split * rows + at) * 2) = float2{ms * c, ll};
  }
}

// ------------------------------------------------------------------ large tiles
// LDS: two buffers of K [64 keys][D] and V^T [4 runs of 16 keys][D][16].  K rows hold their 16-byte
// pieces at position piece ^ (row & (D/8 - 1)), V^T rows their two halves at half ^ (d >> 3 & 1): the
// 16 lanes that LDS serves together then read 16 different 16-byte columns of its 256.
template <int D>
__device__ __forceinline__ void load_kv(const AttnArgs& a, int id, int h, int k0, lds_u8* buf) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int key = k0 + wave * 16;  // this wavefront's run of keys: inside page id
  const long base = block_at<D>(a, id < 0 ? 0 : id, h);
  const int at = key & a.mask;
  constexpr int CH = D / 8;                 // 16-byte pieces of a K row
  const __bf16* kb = static_cast<const __bf16*>(a.KC) + base + (long)at * D;
  const __bf16* vb = static_cast<const __bf16*>(a.VC) + base + at;
  lds_u8* kl = buf + wave * 16 * D * 2;
  lds_u8* vl = buf + 64 * D * 2 + wave * D * 32;
#pragma unroll
  for (int i = 0; i < 16 * CH / 64; ++i) {
    const int row = i * (64 / CH) + lane / CH;
    const int piece = (lane % CH) ^ (row & (CH - 1));
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(kb + row * D + piece * 8),
                                     (__attribute__((address_space(3))) void*)(kl + i * 1024), 16, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int d = i * 32 + lane / 2;
    const int half = (lane & 1) ^ ((d >> 3) & 1);
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(vb + ((long)d << a.sh) + half * 8),
                                     (__attribute__((address_space(3))) void*)(vl + i * 1024), 16, 0, 0);
  }
}

template <int D>
__device__ __forceinline__ void large_tile(const AttnArgs& a, const Tile& t, int h, uint8_t* lds) {
  constexpr int DK = D / 16, DB = D / 32, CH = D / 8;
  constexpr int BUF = 64 * D * 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int g = a.g;
  const int row = t.row0 + wave * 32 + col;
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
  const int base = t.kv - t.n;
  const int last = live ? base + tok : -1;
  const int tile_end = t.row0 + kLargeRows < t.rows ? t.row0 + kLargeRows : t.rows;
  const int kend = clampi(base + (tile_end - 1) / g + 1, 0, t.kv);
  // the first row of the wavefront sees the fewest keys: tiles up to it need no mask
  const int wfirst = base + (t.row0 + wave * 32) / g;
  const int steps = (kend + 63) >> 6;
  const int lo = (int)((long)steps * t.split / t.ns), hi = (int)((long)steps * (t.split + 1) / t.ns);

  v16f o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = neg_inf(), mc = 0.0f, l = 0.0f;
  const float c = a.scale_log2;
  lds_u8* lb = (lds_u8*)lds;
  // row `col` of score block x holds key 32 x + 16 (a / 2) + 8 hh + 4 (a % 2) + j, col = 8 a + 4 hh + j
  const int perm = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);

  // The pages of 16 steps, a run of 16 keys a lane.  They are fetched a block of steps ahead: a load
  // waited for here would be waited for behind the DMA that the step has just begun.
  int ids = page_of(a, t, (lo * 4 + lane) * 16), next_ids = page_of(a, t, (lo * 4 + 64 + lane) * 16);
  if (lo < hi) load_kv<D>(a, __builtin_amdgcn_readlane(ids, wave), h, lo * 64, lb);
  for (int st = lo; st < hi; ++st) {
    const int k0 = st * 64;
    const int n = (st - lo) & 15;
    uint8_t* buf = lds + ((st - lo) & 1) * BUF;
    int bad = (int)(__ballot(ids < 0) >> (n * 4)) & 15;  // runs of 16 keys without a page
    if (k0 + 64 > t.kv) bad |= 16;
    wait_vm<0>();
    lds_barrier();  // this buffer has landed, and the other one is no longer read
    if (n == 15) {
      ids = next_ids;
      next_ids = page_of(a, t, ((st + 1) * 4 + 64 + lane) * 16);
    }
    if (st + 1 < hi)
      load_kv<D>(a, __builtin_amdgcn_readlane(ids, ((n + 1) & 15) * 4 + wave), h, k0 + 64, lb + ((st - lo + 1) & 1) * BUF);
    if (bad) {  // V of keys that do not exist may hold anything, and 0 * NaN is not 0
      uint16_t* v = reinterpret_cast<uint16_t*>(buf + 64 * D * 2);
      for (int i = threadIdx.x; i < 64 * D; i += 256) {
        const int u = i / (16 * D), d = (i / 16) % D, e = i & 15;
        const int key = u * 16 + ((((e >> 3) ^ (d >> 3)) & 1) << 3) + (e & 7);
        if (k0 + key >= t.kv || ((bad >> u) & 1)) v[i] = 0;
      }
      lds_barrier();
    }
    v16f s[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[x][i] = 0.0f;
      const int kr = 32 * x + perm;
#pragma unroll
      for (int k = 0; k < DK; ++k) {
        const v8bf kf = *reinterpret_cast<const v8bf*>(buf + kr * D * 2 + (((2 * k + half) ^ (kr & (CH - 1))) << 4));
        s[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[k], s[x], 0, 0, 0);
      }
    }
    if (k0 + 63 > wfirst || bad) {
      // element i of block x is key 32 x + 16 (i / 8) + 8 half + i % 8
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = 32 * x + 16 * (i >> 3) + 8 * half + (i & 7);
          if (k0 + key > last || ((bad >> (2 * x + (i >> 3))) & 1)) s[x][i] = neg_inf();
        }
    }
    float mx = neg_inf();
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[x][i]);
    if (__any(mx * c > mc + kSlack || (m == neg_inf() && mx > neg_inf()))) {
      const float mn = fmaxf(m, max_halves(mx));
      const float ms = mn == neg_inf() ? 0.0f : mn;
      const float f = __builtin_amdgcn_exp2f(m * c - ms * c);
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= f;
      m = mn;
      mc = ms * c;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        v8bf p;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][8 * y + i], c, -mc));
          l += e;
          p[i] = (__bf16)e;
        }
        const uint8_t* vt = buf + 64 * D * 2 + (2 * x + y) * D * 32;
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          const int dr = d * 32 + col;
          const v8bf vf = *reinterpret_cast<const v8bf*>(vt + dr * 32 + ((half ^ ((dr >> 3) & 1)) << 4));
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, p, o[d], 0, 0, 0);
        }
      }
  }
  l += __shfl_xor(l, 32);
  if (!live) return;
  if (a.CNT && t.split == 0 && half == 0) a.CNT[out_row] = t.ns;
  if (t.ns == 1) {
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
    const long at = (long)t.split * a.S * a.HQ + out_row;
    float* out = a.PO + at * D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<v4f*>(out + d * 32 + 8 * i + 4 * half) =
            v4f{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    if (half == 0) *reinterpret_cast<float2*>(a.PM + at * 2) = float2{mc, l};
  }
}

// A request's tiles, and the 64-key steps that each takes (a step's cost is about the same for both
// shapes: the small one waits for memory, the large one works).
__device__ __forceinline__ void shape(const AttnArgs& a, int r, int& tiles, int& steps) {
  const int c0 = clampi(a.CU[r], 0, a.S), c1 = clampi(a.CU[r + 1], 0, a.S);
  const int rows = (c1 > c0 ? c1 - c0 : 0) * a.g;
  tiles = rows > kSmallRows ? (rows + kLargeRows - 1) / kLargeRows : (rows + 15) >> 4;
  steps = (clampi(a.KV[r], 0, (int)((long)a.MB << a.sh)) + 63) >> 6;
}

// Workgroups: key heads fastest (an XCD takes every eighth workgroup, so with eight key heads each XCD's
// L2 holds one head's cache), then units of work: requests in order, a request's later tiles first (they
// see the most keys), a tile's ranges of keys in order.  Every wavefront finds the unit by itself, its
// lanes a share of the requests each.
template <int D>
__global__ __launch_bounds__(256, 2) void k_attn(AttnArgs a) {
  __shared__ __align__(16) uint8_t lds[64 * D * 8 > 128 * 4 + 4 * 16 * (D + 4) * 4 ? 64 * D * 8 : 128 * 4 + 4 * 16 * (D + 4) * 4];
  const int h = blockIdx.x % a.HKV;
  const int unit = blockIdx.x / a.HKV;
  const int lane = threadIdx.x & 63;
  const int per = (a.R + 63) >> 6;
  const int r0 = lane * per, r1 = r0 + per < a.R ? r0 + per : a.R;
  int tiles, steps;
  int chunk = 0x7FFFFFFF;  // steps of a unit
  if (a.cap > 1) {
    long sum = 0;
    for (int r = r0; r < r1; ++r) {
      shape(a, r, tiles, steps);
      sum += (long)tiles * steps;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    const long want = (sum + a.target - 1) / a.target;
    chunk = want < kMinSteps ? kMinSteps : want < chunk ? (int)want : chunk;
  }
  auto ranges = [&](int st) {  // of a request of st steps
    const int n = a.cap > 1 ? (int)(((long)st + chunk - 1) / chunk) : 1;
    return n < 1 ? 1 : n < a.cap ? n : a.cap;
  };
  int units = 0;
  for (int r = r0; r < r1; ++r) {
    shape(a, r, tiles, steps);
    units += tiles * ranges(steps);
  }
  int upto = units;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(upto, d);
    if (lane >= d) upto += up;
  }
  const unsigned long long mine = __ballot(unit >= upto - units && unit < upto);
  if (mine == 0) return;  // no such unit: the grid is an upper bound
  int in = unit - (upto - units), hit = r0, ns = 1, nt = 0;
  for (int r = r0; r < r1; ++r) {
    shape(a, r, tiles, steps);
    const int n = ranges(steps);
    hit = r, ns = n, nt = tiles;
    if (in < tiles * n) break;
    in -= tiles * n;
  }
  const int src = __ffsll(mine) - 1;
  hit = __builtin_amdgcn_readlane(hit, src);
  in = __builtin_amdgcn_readlane(in, src);
  ns = __builtin_amdgcn_readlane(ns, src);
  nt = __builtin_amdgcn_readlane(nt, src);
  Tile t;
  request(a, hit, t);
  t.rows = t.n * a.g;
  t.ns = ns;
  t.split = in % ns;
  const int tile = nt - 1 - in / ns;
  if (t.rows <= kSmallRows) {
    t.row0 = tile * 16;
    small_tile<D>(a, t, h, reinterpret_cast<float*>(lds));
  } else {
    t.row0 = tile * kLargeRows;
    large_tile<D>(a, t, h, lds);
  }
}

// Joins the ranges of each row that was cut: WPR wavefronts a row, D / 64 values a lane, lane s holding
// range s's maximum and sum; the ranges are added in an order that their number alone fixes.
// HBM-bound on the partial outputs; with few rows four wavefronts share one, to have its loads in flight at once.
template <int D, int WPR>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int E = D / 64;
  typedef float vE __attribute__((ext_vector_type(E)));
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long row = (long)blockIdx.x * (4 / WPR) + wave / WPR;
  const int part = wave % WPR;
  const long first = (long)clampi(a.CU[0], 0, a.S) * a.HQ, end = (long)clampi(a.CU[a.R], 0, a.S) * a.HQ;
  if (row < first || row >= end) return;
  const int ns = __builtin_amdgcn_readfirstlane(clampi(a.CNT[row], 1, a.cap));
  if (ns == 1) return;  // written by its tile
  const long rows = (long)a.S * a.HQ;
  float2 ml = {0.0f, 0.0f};
  if (lane < ns) ml = *reinterpret_cast<const float2*>(a.PM + (lane * rows + row) * 2);
  const bool any = ml.y != 0.0f;  // a range of no keys has a sum of 0 and no output
  float m = any ? ml.x : neg_inf();
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float f = any ? __builtin_amdgcn_exp2f(ml.x - m) : 0.0f;
  float l = f * ml.y;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
  const int s0 = ns * part / WPR, s1 = ns * (part + 1) / WPR;
  const float* src = a.PO + row * D + lane * E;
  vE acc = {};
  for (int s = s0; s < s1; s += 8) {
    vE v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = s + i < s1 ? s + i : s1 - 1;
      v[i] = *reinterpret_cast<const vE*>(src + x * rows * D);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = s + i < s1 ? __shfl(f, s + i) : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += w != 0.0f ? v[i][e] * w : 0.0f;
    }
  }
  if constexpr (WPR > 1) {
    __shared__ vE half[WPR][64];
    half[part][lane] = acc;
    __syncthreads();  // the wavefronts of a workgroup share the row: all are here or none
    if (part != 0) return;
#pragma unroll
    for (int p = 1; p < WPR; ++p) acc += half[p][lane];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  __bf16* out = static_cast<__bf16*>(a.O) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = (__bf16)(acc[e] * inv);
}

}  // namespace

// Units and ranges of a call.  A request of more than kSmallRows rows has rows / 128 large tiles rounded
// up, any other two small ones at most; the units are at most one more for each tile than the work
// divided by a unit's (osc_attn.hip's kernel takes at least work / target steps for a unit).
AttnPlan attn_plan(int S, int R, int HQ, int HKV, int D, int page, int MB) {
  const long rows = (long)S * (HQ / HKV);
  const long big = rows / (kSmallRows + 1);
  const long large = big > 0 ? rows / kLargeRows + (big < R ? big : R) : 0;
  const long few = rows / 16 + R < 2l * R ? rows / 16 + R : 2l * R;
  const long tiles = large + few;
  // tiles that are expected to work: all rows in 128-row tiles, or one small tile a request
  const long busy = (rows / R > kSmallRows ? (rows + kLargeRows - 1) / kLargeRows : R) * HKV;
  AttnPlan p;
  const long steps = ((long)MB * page + 63) / 64;
  long cap = steps / kMinSteps;  // were a request's table full
  if (cap > kMaxSplit) cap = kMaxSplit;
  if (busy >= 4 * kSlots || cap < 1) cap = 1;
  p.cap = (int)cap;
  p.target = (kSlots + HKV - 1) / HKV;
  p.units = cap == 1 ? tiles : tiles * cap < p.target + tiles ? tiles * cap : p.target + tiles;
  p.ws_bytes = cap > 1 ? cap * S * HQ * (long)(D + 2) * 4 + (long)S * HQ * 4 : 0;
  return p;
}

hipError_t launch_attn(const AttnArgs& a, int D, long units, hipStream_t st) {
  const long grid = units * a.HKV;
  if (grid > 0x7FFFFFFFL) return hipErrorInvalidValue;
  if (D == 128) hipLaunchKernelGGL(k_attn<128>, dim3((unsigned)grid), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_attn<64>, dim3((unsigned)grid), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.cap == 1) return e;
  const long rows = (long)a.S * a.HQ;
  if (rows <= 4096) {
    if (D == 128) hipLaunchKernelGGL((k_attn_join<128, 4>), dim3((unsigned)rows), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_attn_join<64, 4>), dim3((unsigned)rows), dim3(256), 0, st, a);
  } else {
    const unsigned jg = (unsigned)((rows + 3) / 4);
    if (D == 128) hipLaunchKernelGGL((k_attn_join<128, 1>), dim3(jg), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_attn_join<64, 1>), dim3(jg), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace osc
