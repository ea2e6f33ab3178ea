// Log probabilities, entropy and the most likely tokens from rows of logits, in one pass over them.
//
// With u = scale log2(e) x, a reference R near the row's largest u, l = sum 2^(u - R) and t = sum 2^(u - R) (u - R):
//   log2 p(v) = u_v - R - log2 l,   entropy = log2 l - t / l  (in bits),
// and parts with references R_a, R_b join as l = l_a 2^(R_a - R) + ..., t = 2^(R_a - R) (t_a + (R_a - R) l_a) + ...
// Threads keep R, l and t of their own and move R where a value exceeds it by more than kSlack.
//
// The K largest come along.  They stand in the K vectors (of 16 bytes) whose largest values are the best, so vectors are noted, not
// values: a comparison a vector, where it holds a list entry.  The first 8 vectors of each thread (one, where a part is short) give 256
// maxima, whose K-th largest is a bound that at least K vectors reach.  From then on a vector that reaches the bound
// is noted by its wavefront, in a list of its own in LDS, so that none waits for another: a few times K of a row in usual orders.
// A list that is nearly full is cut to the vectors that reach a better bound.  At the end the best K vectors of all lists, and
// seldom a few more, are read once more and their values put in order.  (Noting the values: 2048 rows of 151936, K = 5 and 64, 154 and
// 250 us, see below.)
#include "osc_internal.h"

namespace osc {
namespace {

typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kRound = 8;        // vectors of 16 bytes a thread and round
constexpr int kList = 256;       // vectors that a wavefront notes
constexpr int kCut = kList - 64; // from here on a vector of each lane may not find room
constexpr int kVectors = 4 * kList, kValues = 8 * kThreads;
constexpr int kParts = 64 * OSC_MAX_TOP;  // values of a row's parts
constexpr float kSlack = 4.0f;
constexpr int kNone = 0x007FFFFF;  // the key of -inf

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// values in the order of unsigned numbers (no NaN; both zeros alike), and back
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned b = __builtin_bit_cast(unsigned, x == 0.0f ? 0.0f : x);
  return b ^ ((int)b < 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned k) {
  return __builtin_bit_cast(float, k ^ ((int)k < 0 ? 0x80000000u : 0xFFFFFFFFu));
}

struct Sum {  // R (-inf: nothing yet), l, t
  float r, l, t;
};
__device__ __forceinline__ float base_of(float r) { return r == neg_inf() ? 0.0f : r; }
__device__ __forceinline__ Sum join(Sum a, Sum b) {
  const float r = fmaxf(a.r, b.r), z = base_of(r);
  // a part that has seen no value above -inf weighs nothing; its sums are 0, or NaN, which stays
  const float da = base_of(a.r) - z, db = base_of(b.r) - z;
  const float fa = a.r == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(da), fb = b.r == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(db);
  // 0 times the distance of parts so far away that nothing of them is left
  return {r, fa * a.l + fb * b.l, fa * (a.t + (fa == 0.0f ? 0.0f : da) * a.l) + fb * (b.t + (fb == 0.0f ? 0.0f : db) * b.l)};
}

template <int CAP>
struct Lds {  // CAP: values, or vectors, noted
  unsigned key[CAP];
  int idx[CAP];
  Sum sums[4];
  unsigned top[kThreads];
  int votes[2][4];
  unsigned worst;
};

// how many threads' flags are set, over the workgroup; `turn` alternates from call to call
template <int CAP>
__device__ __forceinline__ int vote(Lds<CAP>& s, int mine, int& turn) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mine += __shfl_xor(mine, d);
  if ((threadIdx.x & 63) == 0) s.votes[turn][threadIdx.x >> 6] = mine;
  __syncthreads();
  const int all = s.votes[turn][0] + s.votes[turn][1] + s.votes[turn][2] + s.votes[turn][3];
  turn ^= 1;
  return all;
}

// Cuts the n noted values to the K best (n >= K).  All threads, behind a barrier.
template <int CAP>
__device__ __attribute__((noinline)) void prune(Lds<CAP>& s, int n, int K) {
  constexpr int PER = CAP / kThreads;
  unsigned k[PER];
  int ix[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = threadIdx.x + i * kThreads;
    k[i] = j < n ? s.key[j] : 0, ix[i] = j < n ? s.idx[j] : 0x7FFFFFFF;
  }
  __syncthreads();
  int turn = 0;
  unsigned low = 0;  // the largest key that K values reach
  for (int bit = 31; bit >= 0; --bit) {
    const unsigned trial = low | 1u << bit;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += k[i] >= trial;
    if (vote(s, mine, turn) >= K) low = trial;
  }
  int above = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) above += k[i] > low;
  const int need = K - vote(s, above, turn);
  int last = 0;  // the smallest index up to which `need` values have that key: one below it has not
  for (int bit = 23; bit >= 0; --bit) {
    const int trial = last | 1 << bit;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += k[i] == low && ix[i] < trial;
    if (vote(s, mine, turn) < need) last = trial;
  }
  if (threadIdx.x == 0) s.votes[turn][0] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (k[i] > low || (k[i] == low && ix[i] <= last)) {
      const int at = atomicAdd(&s.votes[turn][0], 1);
      s.key[at] = k[i], s.idx[at] = ix[i];
    }
  __syncthreads();
}

// A key that at least K of the workgroup's values reach: the K-th largest of the threads' largest keys (0 if there are fewer).
// BITS: how many of a key's upper bits count.  Every wavefront takes all 256 keys, four a lane, and settles a bit at a time.
template <int BITS, int CAP>
__device__ __forceinline__ unsigned reached(Lds<CAP>& s, unsigned mine, int K) {
  s.top[threadIdx.x] = mine;
  __syncthreads();
  unsigned k[4], low = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = s.top[64 * j + (threadIdx.x & 63)];
  for (int bit = 31; bit >= 32 - BITS; --bit) {
    const unsigned trial = low | 1u << bit;
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) n += __popcll(__ballot(k[j] >= trial));
    if (n >= K) low = trial;
  }
  return low;
}

// The best of the entries k[], ix[] that the threads hold (0: none) into the list, from its start: those that reach a bound that K of
// them do, K at least if there are as many, and seldom more than 256.  Returns their number.  All threads.
template <int BITS, int PER, int CAP>
__device__ __forceinline__ int gather(Lds<CAP>& s, const unsigned (&k)[PER], const int (&ix)[PER], int K) {
  unsigned most = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) most = most > k[i] ? most : k[i];
  if (threadIdx.x == 0) s.votes[0][0] = 0;
  const unsigned bound = reached<BITS>(s, most, K);
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (k[i] >= bound && k[i] > 0) {
      const int at = atomicAdd(&s.votes[0][0], 1);
      s.key[at] = k[i], s.idx[at] = ix[i];
    }
  __syncthreads();
  const int n = s.votes[0][0];
  __syncthreads();
  return n;
}

// Cuts a wavefront's list of n vectors, kCut < n <= kList, to those that reach a better bound: the K-th largest of
// the lanes' largest, or where that leaves more than half a list, the K-th best of all.
struct Kept {
  int n;        // how many are left
  float bound;  // all that is as large as that, and
  int last;     // where it is that large, up to this index
};
__device__ __attribute__((noinline)) Kept cut(unsigned* key, int* idx, int n, int K, Kept old) {
  constexpr int PER = kList / 64;
  const int lane = threadIdx.x & 63;
  unsigned k[PER], most = 0;
  int ix[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + 64 * i;
    k[i] = j < n ? key[j] : 0, ix[i] = j < n ? idx[j] : 0x7FFFFFFF;
    most = most > k[i] ? most : k[i];
  }
  auto count = [&](auto&& holds) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += __popcll(__ballot(holds(i)));
    return c;
  };
  unsigned low = 0;
  for (int bit = 31; bit >= 0; --bit)
    if (__popcll(__ballot(most >= (low | 1u << bit))) >= K) low |= 1u << bit;
  int last = 0x7FFFFFFF;
  if (count([&](int i) { return k[i] >= low; }) > kList / 2) {
    low = 0;
    for (int bit = 31; bit >= 0; --bit)
      if (count([&](int i) { return k[i] >= (low | 1u << bit); }) >= K) low |= 1u << bit;
    const int need = K - count([&](int i) { return k[i] > low; });
    last = 0;  // the smallest index up to which `need` values have that key
    for (int bit = 23; bit >= 0; --bit)
      if (count([&](int i) { return k[i] == low && ix[i] < (last | 1 << bit); }) < need) last |= 1 << bit;
  }
  int have = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool keep = k[i] > low || (k[i] == low && ix[i] <= last && k[i] > 0);
    const u64 who = __ballot(keep);
    const int at = have + __popcll(who & ((1ull << lane) - 1));
    if (keep) key[at] = k[i], idx[at] = ix[i];
    have += __popcll(who);
  }
  const float bound = value_of(low);
  return {have, bound, bound > old.bound || last < old.last ? last : old.last};
}

// The K best of the n noted values in order: write(place, key, index) for each, then none(place) for places without one.
template <int CAP, typename Write, typename None>
__device__ __forceinline__ void in_order(Lds<CAP>& s, int n, int K, Write write, None none) {
  if (n > kThreads) {  // as many are alike
    prune(s, n, K);
    n = K;
  }
  const int i = threadIdx.x;
  if (i < n) {
    const u64 mine = (u64)s.key[i] << 32 | (unsigned)~s.idx[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += ((u64)s.key[j] << 32 | (unsigned)~s.idx[j]) > mine;
    if (place < K) write(place, s.key[i], s.idx[i]);
  }
  if (i >= n && i < K) none(i);
}

__device__ __forceinline__ bool is_none(const Sum& s) { return !(s.l > 0.0f) || !(s.r < __builtin_inff()); }

__device__ __forceinline__ float logp(const Sum& s, float log2l, float x, float c) {
  return (__builtin_fmaf(x, c, -base_of(s.r)) - log2l) * 0.6931471805599453f;
}

template <bool F32>
__device__ __forceinline__ float logit(const LogprobsArgs& a, long at) {
  return F32 ? static_cast<const float*>(a.X)[at] : (float)static_cast<const __bf16*>(a.X)[at];
}

// A row's outputs, from its sums and the n noted values.
template <bool F32, int CAP>
__device__ __forceinline__ void finish(const LogprobsArgs& a, int row, const Sum& s, Lds<CAP>& lds, int n) {
  const bool none = is_none(s);
  const float c = a.scale_log2, nan = __builtin_nanf(""), log2l = none ? nan : log2f(s.l);
  for (int i = threadIdx.x; i < a.M; i += kThreads) {
    const long at = (long)row * a.M + i;
    const int id = a.ID[at];
    a.LP[at] = none ? nan : id < 0 || id >= a.V ? neg_inf() : logp(s, log2l, logit<F32>(a, (long)row * a.ld + id), c);
  }
  if (a.ENT && threadIdx.x == 0) a.ENT[row] = none ? nan : (log2l - s.t / s.l) * 0.6931471805599453f;
  if (a.K == 0) return;
  const long out = (long)row * a.K;
  in_order(
      lds, n, a.K,
      [&](int at, unsigned key, int idx) {
        a.TOPV[out + at] = none ? nan : logp(s, log2l, value_of(key), c);
        a.TOPI[out + at] = none ? -1 : idx;
      },
      [&](int at) { a.TOPV[out + at] = none ? nan : neg_inf(), a.TOPI[out + at] = -1; });
}

template <int CAP>
__device__ __forceinline__ Sum join_all(Sum s, Lds<CAP>& lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const Sum o = {__shfl_xor(s.r, d), __shfl_xor(s.l, d), __shfl_xor(s.t, d)};
    s = (threadIdx.x & d) ? join(o, s) : join(s, o);  // the same on both sides
  }
  if ((threadIdx.x & 63) == 0) lds.sums[threadIdx.x >> 6] = s;
  __syncthreads();
  return join(join(lds.sums[0], lds.sums[1]), join(lds.sums[2], lds.sums[3]));
}

// A part's record in the workspace: its sums, the number of its best values, and them.
struct Record {
  Sum s;
  int n;
};
__host__ __device__ inline long record_bytes(int K) { return (long)sizeof(Record) + 8l * K; }

template <bool F32>
__global__ __launch_bounds__(kThreads, 4) void k_logprobs(LogprobsArgs a) {
  constexpr int E = F32 ? 4 : 8;  // values of a vector
  __shared__ Lds<(kValues > kVectors ? kValues : kVectors)> lds;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks;
  const int tid = threadIdx.x;
  const uint8_t* x0 = static_cast<const uint8_t*>(a.X) + (long)row * a.ld * (F32 ? 4 : 2);
  const int skew = (int)(reinterpret_cast<uintptr_t>(x0) & 15) / (F32 ? 4 : 2);  // values ahead of the row in its first vector
  const u4* xv = reinterpret_cast<const u4*>(x0 - skew * (F32 ? 4 : 2));
  const int vectors = (a.V + skew + E - 1) / E;
  const int v0 = (int)((long)vectors * chunk / a.chunks), v1 = (int)((long)vectors * (chunk + 1) / a.chunks);
  const int whole0 = skew > 0 ? 1 : 0, whole1 = (a.V + skew) / E;  // vectors that are the row's throughout
  const float c = a.scale_log2;
  const unsigned ninf = F32 ? 0xFF800000u : 0xFF80FF80u;

  // vector v of the row; what is not the row's as -inf, and nothing behind the row's end is read
  auto load = [&](int v) {
    u4 q = {ninf, ninf, ninf, ninf};
    if (v >= v1) return q;
    if (v >= whole0 && v < whole1) return xv[v];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = v * E - skew + i;
      const bool in = e >= 0 && e < a.V;
      if (F32) {
        q[i & 3] = in ? static_cast<const unsigned*>(a.X)[(long)row * a.ld + e] : ninf;
      } else {
        const unsigned w = in ? static_cast<const uint16_t*>(a.X)[(long)row * a.ld + e] : 0xFF80u;
        q[(i >> 1) & 3] = i & 1 ? (q[(i >> 1) & 3] & 0xFFFF) | w << 16 : (q[(i >> 1) & 3] & 0xFFFF0000u) | w;
      }
    }
    return q;
  };
  auto value = [&](const u4& q, int i) {
    const unsigned w = q[F32 ? i & 3 : (i >> 1) & 3];  // (a bit cast straight from a vector's element reads element 0)
    return __builtin_bit_cast(float, F32 ? w : i & 1 ? w & 0xFFFF0000u : w << 16);
  };

  Sum s = {neg_inf(), 0.0f, 0.0f};
  float z = 0.0f;              // - R, or 0
  float limit = neg_inf();     // the largest logit that R need not move for
  const float slack = kSlack / c;
  // values up to `most` into the sums: R moves where they exceed it
  auto room = [&](float most) {
    if (most > limit) {
      s = join(s, Sum{most * c, 0.0f, 0.0f});
      z = -base_of(s.r), limit = most + slack;
    }
  };
  // a vector into the sums; its largest value
  auto add = [&](const u4& q) {
    float most = fmaxf(value(q, 0), value(q, 1));
#pragma unroll
    for (int i = 2; i < E; i += 2) most = fmaxf(fmaxf(most, value(q, i)), value(q, i + 1));
    room(most);
    float d = __builtin_fmaf(value(q, 0), c, z), l = __builtin_amdgcn_exp2f(d), t = l * d;
#pragma unroll
    for (int i = 1; i < E; ++i) {
      d = __builtin_fmaf(value(q, i), c, z);
      const float e = __builtin_amdgcn_exp2f(d);
      l += e, t = __builtin_fmaf(e, d, t);
    }
    if (t != t) {  // 0 * -inf, of tokens that are masked out (or a NaN, which stays)
      t = 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        d = __builtin_fmaf(value(q, i), c, z);
        t = __builtin_fmaf(__builtin_amdgcn_exp2f(d), fmaxf(d, -1000.0f), t);
      }
    }
    s.l += l, s.t += t;
    return most;
  };
  // the wavefront's list, its bound (no more than the K-th best of its values and the workgroup's first ones), and how many there are
  unsigned* const keys = lds.key + (tid >> 6) * kList;
  int* const idxs = lds.idx + (tid >> 6) * kList;
  float bound = a.K > 0 ? neg_inf() : __builtin_nanf("");
  int bound_idx = 0x7FFFFFFF, have = 0;
  auto note = [&](float most, int v) {
    const bool takes = most >= bound && most > neg_inf() && (most > bound || v <= bound_idx);
    const u64 who = __ballot(takes);
    if (who == 0) return;
    const int at = have + __popcll(who & ((1ull << (tid & 63)) - 1));
    if (takes) keys[at] = key_of(most), idxs[at] = v;
    have += __popcll(who);
    if (have > kCut) {
      const Kept kept = cut(keys, idxs, have, a.K, Kept{have, bound, bound_idx});
      have = __builtin_amdgcn_readfirstlane(kept.n), bound = kept.bound, bound_idx = kept.last;
    }
  };
  // Rounds of vectors that are the row's throughout, the next one's asked for as this one's are done with; then what is left of such
  // vectors.  The row's first and last vector, if they are not, go to the threads 0 .. E - 1 and E .. 2 E - 1, a value each.
  constexpr int STEP = kRound * kThreads, BITS = F32 ? 32 : 16;  // BITS: of a key, that differ
  const int w0 = v0 > whole0 ? v0 : whole0, w1 = v1 < whole1 ? v1 : whole1;
  const int rounds = w1 > w0 ? (w1 - w0) / STEP : 0;
  const bool edges = v0 < w0 || v1 > w1;
  const int edge = tid < E && v0 < w0 ? v0 : tid >= E && v1 > w1 && v1 > w0 ? v1 - 1 : v1;
  float edge_value = neg_inf();
  if (edges && tid < 2 * E && edge < v1) {
    const int e = edge * E - skew + (tid & (E - 1));
    if (e >= 0 && e < a.V) edge_value = logit<F32>(a, (long)row * a.ld + e);
  }
  int v = w0 + tid;
  if (rounds > 0) {
    u4 q[kRound];
    float most[kRound], all = neg_inf();
#pragma unroll
    for (int u = 0; u < kRound; ++u) q[u] = xv[v + u * kThreads];
#pragma unroll
    for (int u = 0; u < kRound; ++u) most[u] = add(q[u]), all = fmaxf(all, most[u]);
    if (a.K > 0) {
      const unsigned low = reached<BITS>(lds, key_of(all), a.K);
      bound = low <= (unsigned)kNone ? neg_inf() : value_of(low);
    }
    const int more = rounds > 1 ? STEP : 0;
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      note(most[u], v + u * kThreads);
      q[u] = xv[v + more + u * kThreads];
    }
    for (int r = 1; r < rounds; ++r) {
      v += STEP;
      const int next = r + 1 < rounds ? STEP : 0;
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        note(add(q[u]), v + u * kThreads);
        q[u] = xv[v + next + u * kThreads];
      }
    }
    v += STEP;
  }
  float edge_most = neg_inf();  // in the first of a vector's threads
  if (edges) {
    room(edge_value);
    const float d = __builtin_fmaf(edge_value, c, z), e = __builtin_amdgcn_exp2f(d);
    s.l += e, s.t = __builtin_fmaf(e, fmaxf(d, -1000.0f), s.t);
    float m = edge_value;
#pragma unroll
    for (int x = 1; x < E; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    if (tid < 2 * E && (tid & (E - 1)) == 0) edge_most = m;
    if (rounds > 0) note(edge_most, edge);
  }
  float most[kRound];
  {
    u4 q[kRound];
    const u4 none = {ninf, ninf, ninf, ninf};
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      const int x = v + u * kThreads;
      q[u] = none;
      if (x < w1) q[u] = xv[x];
    }
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      most[u] = neg_inf();
      if (w0 + rounds * STEP + u * kThreads < w1) most[u] = add(q[u]);  // (the same for all)
    }
  }
  int n = 0;
  if (a.K > 0) {
    if (rounds == 0) {  // what the threads hold is all
      unsigned k[kRound + 1];
      int ix[kRound + 1];
#pragma unroll
      for (int u = 0; u < kRound; ++u) k[u] = most[u] > neg_inf() ? key_of(most[u]) : 0, ix[u] = v + u * kThreads;
      k[kRound] = edge_most > neg_inf() ? key_of(edge_most) : 0, ix[kRound] = edge;
      n = gather<BITS>(lds, k, ix, a.K);
    } else {
#pragma unroll
      for (int u = 0; u < kRound; ++u) note(most[u], v + u * kThreads);
      constexpr int PER = kList / 64;
      unsigned k[PER];
      int ix[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int j = (tid & 63) + 64 * i;
        k[i] = j < have ? keys[j] : 0, ix[i] = j < have ? idxs[j] : 0;
      }
      n = gather<BITS>(lds, k, ix, a.K);
    }
    if (n > kThreads) {  // as many are alike
      prune(lds, n, a.K);
      n = a.K;
    }
    // the vectors' values that reach the worst of their largest, if there are K of them
    const unsigned mine = tid < n ? lds.key[tid] : 0xFFFFFFFFu;
    const u4 best = load(tid < n ? lds.idx[tid] : v1);
    const int e0 = tid < n ? lds.idx[tid] * E - skew : 0;
    if (tid == 0) lds.worst = 0xFFFFFFFFu, lds.votes[0][0] = 0;
    __syncthreads();
    atomicMin(&lds.worst, mine);
    __syncthreads();
    const float worst = n < a.K ? neg_inf() : value_of(lds.worst);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float x = value(best, i);
      if (x > neg_inf() && x >= worst) {
        const int at = atomicAdd(&lds.votes[0][0], 1);
        lds.key[at] = key_of(x), lds.idx[at] = e0 + i;
      }
    }
    __syncthreads();
    n = lds.votes[0][0];
  }
  s = join_all(s, lds);
  if (a.chunks == 1) {
    finish<F32>(a, row, s, lds, n);
    return;
  }
  uint8_t* rec = static_cast<uint8_t*>(a.WS) + blockIdx.x * record_bytes(a.K);
  if (tid == 0) *reinterpret_cast<Record*>(rec) = Record{s, n < a.K ? n : a.K};
  if (a.K == 0) return;
  uint2* best = reinterpret_cast<uint2*>(rec + sizeof(Record));
  in_order(lds, n, a.K, [&](int at, unsigned key, int idx) { best[at] = uint2{key, (unsigned)idx}; }, [&](int at) { best[at] = uint2{0, 0}; });
}

// A row's parts in their order, from one batch of loads: the sums, and the parts' best values, of which those that reach the
// K-th largest of the threads' largest are noted.
template <bool F32>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(LogprobsArgs a) {
  constexpr int PER = kParts / kThreads;
  __shared__ Lds<kParts> lds;
  const int row = blockIdx.x, tid = threadIdx.x, K = a.K;
  const uint8_t* rec = static_cast<const uint8_t*>(a.WS) + (long)row * a.chunks * record_bytes(K);
  auto at = [&](int c) { return rec + c * record_bytes(K); };
  Sum s = {neg_inf(), 0.0f, 0.0f};
  if (tid < a.chunks) s = reinterpret_cast<const Record*>(at(tid))->s;  // at most as many as a wavefront's lanes
  unsigned k[PER];
  int ix[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = tid + i * kThreads, ch = K > 0 ? j / K : 0;
    k[i] = 0, ix[i] = 0;
    if (i * kThreads < a.chunks * K && ch < a.chunks) {
      const uint2 v = reinterpret_cast<const uint2*>(at(ch) + sizeof(Record))[j - ch * K];
      k[i] = v.x, ix[i] = (int)v.y;
    }
  }
  s = join_all(s, lds);
  finish<F32>(a, row, s, lds, K > 0 ? gather<F32 ? 32 : 16>(lds, k, ix, K) : 0);
}

}  // namespace

// Rows are cut where there are fewer than workgroups that the card needs (4 a CU), into parts of 2048 values at least.
LogprobsPlan logprobs_plan(int S, int V, int K) {
  LogprobsPlan p;
  long want = S > 0 ? (1024 + S - 1) / S : 1;
  const long most = V / 2048;
  if (want > most) want = most;
  if (want > 64) want = 64;  // 64 parts of at most OSC_MAX_TOP values are what the join holds
  p.chunks = want < 1 ? 1 : (int)want;
  p.ws_bytes = p.chunks > 1 ? (long)S * p.chunks * record_bytes(K) : 0;
  return p;
}

template <bool F32>
static hipError_t launch(const LogprobsArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(k_logprobs<F32>, dim3((unsigned)a.S * (unsigned)a.chunks), dim3(kThreads), 0, st, a);
  if (a.chunks > 1) hipLaunchKernelGGL(k_logprobs_join<F32>, dim3((unsigned)a.S), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_logprobs(const LogprobsArgs& a, hipStream_t st) {
  return a.xt == OSC_Y_F32 ? launch<true>(a, st) : launch<false>(a, st);
}

}  // namespace osc
