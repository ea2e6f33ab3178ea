// Log probabilities, entropy and the most likely tokens from rows of logits, in one pass over them.
//
// With u = scale log2(e) x, a reference R near the row's largest u, l = sum 2^(u - R) and t = sum 2^(u - R) (u - R):
//   log2 p(v) = u_v - R - log2 l,   entropy = log2 l - t / l  (in bits),
// and parts with references R_a, R_b join as l = l_a 2^(R_a - R) + ..., t = 2^(R_a - R) (t_a + (R_a - R) l_a) + ...
// Threads keep R, l and t of their own and move R where a value exceeds it by more than kSlack.
//
// The K largest come along.  They stand in the K vectors (of 16 bytes) whose largest values are the best, so vectors are noted, not
// values: a comparison a vector, where it holds a list entry.  The first 8 vectors of each thread give 256 maxima, whose K-th largest
// is a bound that at least K vectors reach.  From then on a vector that reaches the bound is noted by its wavefront, in a list of its
// own in LDS, so that none waits for another: a few times K of a row in usual orders.  A list that is nearly full is cut to the
// vectors that reach a better bound.  A part of fewer than 8 vectors a thread stays in registers, and is chosen from there.  At the
// end the best K vectors, and seldom a few more, are read once more and their values put in order.  (Noting the values instead:
// 2048 rows of 151936, K = 5 and 64, 154 and 250 us; vectors 117 and 125.)
//
// Many rows are bound by HBM: 2048 bf16 rows of 151936 with 5 alternatives take 117 us, 5.3 TB/s, 512 take 37, and a round's loads
// are under way while the round before is summed up.  One row is bound by latency: 13.2 us, 7 for a part's loads, maxima and choice, one
// behind the other, and 6.3 for the parts' join.  Equal logits, which reach every bound, are the slow order: 2048 rows of zeros 120 us, one 23 to 30.
#include "osc_internal.h"
#include "osc_lanes.h"

namespace osc {
namespace {

typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kRound = 8;        // vectors of 16 bytes a thread and round
constexpr int kList = 256;       // vectors that a wavefront notes
constexpr int kCut = kList - 64; // from here on a vector of each lane may not find room
constexpr int kHeld = (kRound + 1) * kThreads;  // vectors of a part that stays in registers, with the row's first and last; 8 values of 256 vectors
static_assert(kHeld >= 4 * kList && kHeld >= 8 * kThreads, "the wavefronts' lists and the best vectors' values have room");
constexpr int kParts = 64 * OSC_MAX_TOP;  // values of a row's parts
constexpr float kSlack = 4.0f;  // (terms up to 2^4: the sums lose nothing by the factor)
constexpr int kNone = 0x007FFFFF;  // the key of -inf

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

// A noted value or vector: its key, and the lower index first.  0 is none.
__device__ __forceinline__ u64 entry(unsigned key, int idx) { return (u64)key << 32 | (unsigned)~idx; }
__device__ __forceinline__ unsigned key_in(u64 e) { return (unsigned)(e >> 32); }
__device__ __forceinline__ int index_in(u64 e) { return (int)~(unsigned)e; }

constexpr int kAhead = 8;  // entries that in_order reads at once
template <int CAP>
struct Lds {
  u64 list[CAP + kAhead];
  Sum sums[4];
  unsigned top[2][kThreads];  // for two bounds: none is written while the other may be read
  int votes[2][4];
  u64 differ[4];
};

// Those of the threads' entries that reach `low` (> 0) behind the s.votes[0][0] that the list has, which count on.  (An atomic
// addition for each lane: the compiler takes the lanes one by one, and one row with 64 alternatives 18.5 us, 15.2 so.)
template <int PER, int CAP>
__device__ __forceinline__ void append(Lds<CAP>& s, const u64 (&e)[PER], u64 low) {
  const int lane = threadIdx.x & 63;
  u64 who[PER];
  int n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) who[i] = __ballot(e[i] >= low), n += __popcll(who[i]);
  if (n == 0) return;
  int at = 0;
  if (lane == 0) at = atomicAdd(&s.votes[0][0], n);
  at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (e[i] >= low) s.list[at + __popcll(who[i] & ((1ull << lane) - 1))] = e[i];
    at += __popcll(who[i]);
  }
}

// Cuts the n entries of the list to the K best (n >= K); the worst of those.  All threads, behind a barrier.  Run where values are
// alike, rows of zeros in a padded step for instance, so the bits that all entries share are left out.
template <int CAP>
__device__ __attribute__((noinline)) u64 prune(Lds<CAP>& s, int n, int K) {
  constexpr int PER = CAP / kThreads;
  const int wave = threadIdx.x >> 6;
  const u64 first = s.list[0];
  u64 e[PER], differ = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = threadIdx.x + i * kThreads;
    e[i] = j < n ? s.list[j] : 0;
    differ |= j < n ? e[i] ^ first : 0;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) differ |= __shfl_xor(differ, d);
  if ((threadIdx.x & 63) == 0) s.differ[wave] = differ;
  __syncthreads();
  differ = s.differ[0] | s.differ[1] | s.differ[2] | s.differ[3];
  u64 low = first & ~differ;  // the largest entry that K reach, bit by bit
  int turn = 0;
  while (differ != 0) {
    const u64 bit = 1ull << (63 - __clzll(differ)), trial = low | bit;
    differ ^= bit;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += __popcll(__ballot(e[i] >= trial));
    if ((threadIdx.x & 63) == 0) s.votes[turn][wave] = mine;
    __syncthreads();
    if (s.votes[turn][0] + s.votes[turn][1] + s.votes[turn][2] + s.votes[turn][3] >= K) low = trial;
    turn ^= 1;  // (read ahead of the next barrier, written behind it)
  }
  __syncthreads();  // (the votes are read)
  if (threadIdx.x == 0) s.votes[0][0] = 0;
  __syncthreads();
  append(s, e, low > 0 ? low : 1);
  __syncthreads();
  return low;
}

// A key that at least K of the workgroup's values reach: the K-th largest of the threads' largest keys (0 if there are fewer), of
// which the upper 16 bits count.  Every wavefront takes all 256 keys, four a lane, and settles a bit at a time.
template <int CAP>
__device__ __forceinline__ unsigned reached(Lds<CAP>& s, int which, unsigned mine, int K) {
  s.top[which][threadIdx.x] = mine;
  __syncthreads();
  unsigned k[4], low = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = s.top[which][64 * j + (threadIdx.x & 63)];
  for (int bit = 31; bit >= 16; --bit) {
    const unsigned trial = low | 1u << bit;
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) n += __popcll(__ballot(k[j] >= trial));
    if (n >= K) low = trial;
  }
  return low;
}

// The best of the entries that the threads hold into the list, from its start: those whose key reaches a bound that K of
// them do, K at least if there are as many, and seldom more than 256.  Returns their number, and the bound.  All threads.
template <int PER, int CAP>
__device__ __forceinline__ int gather(Lds<CAP>& s, const u64 (&e)[PER], int K, unsigned& bound) {
  u64 most = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) most = most > e[i] ? most : e[i];
  if (threadIdx.x == 0) s.votes[0][0] = 0;
  bound = reached(s, 1, key_in(most), K);
  append(s, e, bound > 0 ? (u64)bound << 32 : 1);
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
__device__ __attribute__((noinline)) Kept cut(u64* list, int n, int K, Kept old) {
  constexpr int PER = kList / 64;
  const int lane = threadIdx.x & 63;
  u64 e[PER], most = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + 64 * i;
    e[i] = j < n ? list[j] : 0;
    most = most > e[i] ? most : e[i];
  }
  auto count = [&](u64 least) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += __popcll(__ballot(e[i] >= least));
    return c;
  };
  u64 low = 0;
  for (int bit = 63; bit >= 32; --bit)
    if (__popcll(__ballot(most >= (low | 1ull << bit))) >= K) low |= 1ull << bit;
  int last = 0x7FFFFFFF;
  if (count(low) > kList / 2) {
    low = 0;
    for (int bit = 63; bit >= 0; --bit)
      if (count(low | 1ull << bit) >= K) low |= 1ull << bit;
    last = index_in(low);
  }
  int have = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool keep = e[i] >= low && e[i] > 0;
    const u64 who = __ballot(keep);
    if (keep) list[have + __popcll(who & ((1ull << lane) - 1))] = e[i];
    have += __popcll(who);
  }
  const float bound = value_of(key_in(low));
  return {have, bound, bound > old.bound || last < old.last ? last : old.last};
}

// The K best of the list's n entries in order: write(place, entry) for each, then none(place) for places without one.  All
// threads, behind a barrier.
template <int CAP, typename Write, typename None>
__device__ __forceinline__ void in_order(Lds<CAP>& s, int n, int K, Write write, None none) {
  if (n > kThreads) {  // as many are alike
    prune(s, n, K);
    n = K;
  }
  const int i = threadIdx.x;
  if (i < kAhead) s.list[n + i] = 0;
  __syncthreads();
  if (i < n) {
    const u64 mine = s.list[i];
    int place = 0;
    for (int j = 0; j < n; j += kAhead) {
      u64 e[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) e[x] = s.list[j + x];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) place += e[x] > mine;
    }
    if (place < K) write(place, mine);
  }
  if (i >= n && i < K) none(i);
}

// No value above -inf, a NaN, or +inf: that shows in R, or in the sum alone, where no finite value moves R any more (kSlack over
// the smallest scales is +inf).
__device__ __forceinline__ bool is_none(const Sum& s) { return !(s.l > 0.0f && s.l < __builtin_inff()) || !(s.r < __builtin_inff()); }

// (no probability is over 1, nor an entropy below 0, by rounding)
__device__ __forceinline__ float logp(const Sum& s, float log2l, float x, float c) {
  const float p = (__builtin_fmaf(x, c, -base_of(s.r)) - log2l) * 0.6931471805599453f;
  return p > 0.0f ? 0.0f : p;
}

template <bool F32>
__device__ __forceinline__ float logit(const LogprobsArgs& a, long at) {
  return F32 ? static_cast<const float*>(a.X)[at] : (float)static_cast<const __bf16*>(a.X)[at];
}

// The first of a row's given tokens that the thread has, asked for ahead of the row's sums.
template <bool F32>
struct Given {
  int id = -1;
  float x = 0.0f;
  __device__ __forceinline__ Given(const LogprobsArgs& a, int row, int i) {
    if (i >= a.M) return;
    id = a.ID[(long)row * a.M + i];
    if (id >= a.V) id = -1;
    if (id >= 0) x = logit<F32>(a, (long)row * a.ld + id);
  }
};

// A row's outputs, from its sums and the n noted values.
template <bool F32, int CAP>
__device__ __forceinline__ void finish(const LogprobsArgs& a, int row, const Sum& s, Given<F32> given, Lds<CAP>& lds, int n) {
  const bool none = is_none(s);
  const float c = a.scale_log2, nan = __builtin_nanf(""), log2l = none ? nan : log2f(s.l);
  for (int i = threadIdx.x; i < a.M; i += kThreads) {
    if (i >= kThreads) given = Given<F32>(a, row, i);
    a.LP[(long)row * a.M + i] = none ? nan : given.id < 0 ? neg_inf() : logp(s, log2l, given.x, c);
  }
  if (a.ENT && threadIdx.x == 0) a.ENT[row] = none ? nan : fmaxf((log2l - s.t / s.l) * 0.6931471805599453f, 0.0f);
  if (a.K == 0) return;
  const long out = (long)row * a.K;
  in_order(
      lds, n, a.K,
      [&](int at, u64 e) {
        a.TOPV[out + at] = none ? nan : logp(s, log2l, value_of(key_in(e)), c);
        a.TOPI[out + at] = none ? -1 : index_in(e);
      },
      [&](int at) { a.TOPV[out + at] = none ? nan : neg_inf(), a.TOPI[out + at] = -1; });
}

// The threads' sums joined, the same in all: around the largest R, lanes by a tree, then the wavefronts.
template <int CAP>
__device__ __forceinline__ Sum join_all(Sum s, Lds<CAP>& lds) {
  const Sum at = join(Sum{max_wave(s.r), 0.0f, 0.0f}, s);  // (what lies at 0 adds nothing)
  s = Sum{at.r, sum_wave(at.l), sum_wave(at.t)};
  if ((threadIdx.x & 63) == 0) lds.sums[threadIdx.x >> 6] = s;
  __syncthreads();
  return join(join(lds.sums[0], lds.sums[1]), join(lds.sums[2], lds.sums[3]));
}

// A part's record in the workspace: its sums, and its K best values (0: fewer).
struct Record {
  Sum s;
  int unused;
};
__host__ __device__ inline long record_bytes(int K) { return (long)sizeof(Record) + 8l * K; }

template <bool F32>
__global__ __launch_bounds__(kThreads, 4) void k_logprobs(LogprobsArgs a) {
  constexpr int E = F32 ? 4 : 8;  // values of a vector
  __shared__ Lds<kHeld> lds;
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

  const Given<F32> given(a, row, a.chunks == 1 ? tid : a.M);
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
  u64* const list = lds.list + (tid >> 6) * kList;
  float bound = a.K > 0 ? neg_inf() : __builtin_nanf("");
  int bound_idx = 0x7FFFFFFF, have = 0;
  auto note = [&](float most, int v) {
    const bool takes = most >= bound && most > neg_inf() && (most > bound || v <= bound_idx);
    const u64 who = __ballot(takes);
    if (who == 0) return;
    const int at = have + __popcll(who & ((1ull << (tid & 63)) - 1));
    if (takes) list[at] = entry(key_of(most), v);
    have += __popcll(who);
    if (have > kCut) {
      const Kept kept = cut(list, have, a.K, Kept{have, bound, bound_idx});
      have = __builtin_amdgcn_readfirstlane(kept.n), bound = kept.bound, bound_idx = kept.last;
    }
  };
  // Rounds of vectors that are the row's throughout, the next one's asked for as this one's are done with; then what is left of such
  // vectors.  The row's first and last vector, if they are not, go to the threads 0 .. E - 1 and E .. 2 E - 1, a value each.
  constexpr int STEP = kRound * kThreads;
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
  u4 q[kRound];
  auto ask = [&](bool rest) {  // the vectors from v on; what lies behind the last of the rest is not used
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      const int x = v + u * kThreads;
      q[u] = xv[rest && x >= w1 ? w1 - 1 : x];
    }
  };
  if (rounds > 0) {
    float most[kRound], all = neg_inf();
    ask(false);
#pragma unroll
    for (int u = 0; u < kRound; ++u) most[u] = add(q[u]), all = fmaxf(all, most[u]);
    v += STEP;
    if (rounds > 1) ask(false);
    else ask(true);
    if (a.K > 0) {
      const unsigned low = reached(lds, 0, key_of(all), a.K);
      bound = low <= (unsigned)kNone ? neg_inf() : value_of(low);
    }
#pragma unroll
    for (int u = 0; u < kRound; ++u) note(most[u], v - STEP + u * kThreads);
    for (int r = 2; r < rounds; ++r) {
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        note(add(q[u]), v + u * kThreads);
        q[u] = xv[v + STEP + u * kThreads];
      }
      v += STEP;
    }
    if (rounds > 1) {
#pragma unroll
      for (int u = 0; u < kRound; ++u) {
        note(add(q[u]), v + u * kThreads);
        const int x = v + STEP + u * kThreads;
        q[u] = xv[x < w1 ? x : w1 - 1];
      }
      v += STEP;
    }
  } else if (w1 > w0) {
    ask(true);
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
#pragma unroll
  for (int u = 0; u < kRound; ++u) {
    most[u] = neg_inf();
    if (w0 + rounds * STEP + u * kThreads < w1) {  // (the same for all)
#pragma unroll
      for (int i = 0; i < 4; ++i) q[u][i] = v + u * kThreads < w1 ? q[u][i] : ninf;
      most[u] = add(q[u]);
    }
  }
  int n = 0;
  if (a.K > 0) {
    auto noted = [&](float most, int v) { return most > neg_inf() ? entry(key_of(most), v) : 0; };
    unsigned worst;  // of the vectors' largest values
    if (rounds == 0) {  // what the threads hold is all
      u64 e[kRound + 1];
#pragma unroll
      for (int u = 0; u < kRound; ++u) e[u] = noted(most[u], v + u * kThreads);
      e[kRound] = noted(edge_most, edge);
      n = gather(lds, e, a.K, worst);
    } else {
#pragma unroll
      for (int u = 0; u < kRound; ++u) note(most[u], v + u * kThreads);
      constexpr int PER = kList / 64;
      u64 e[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int j = (tid & 63) + 64 * i;
        e[i] = j < have ? list[j] : 0;
      }
      n = gather(lds, e, a.K, worst);
    }
    if (n > kThreads) {  // as many are alike
      worst = key_in(prune(lds, n, a.K));
      n = a.K;
    }
    // the vectors' values that reach as much, of which there are K unless there are not as many at all
    const int at = tid < n ? index_in(lds.list[tid]) : v1;
    const u4 best = load(at);
    if (tid == 0) lds.votes[0][0] = 0;
    u64 e[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float x = value(best, i);
      e[i] = x > neg_inf() && key_of(x) >= worst ? entry(key_of(x), at * E - skew + i) : 0;
    }
    __syncthreads();
    append(lds, e, 1);
    __syncthreads();
    n = lds.votes[0][0];
  }
  s = join_all(s, lds);
  if (a.chunks == 1) {
    finish<F32>(a, row, s, given, lds, n);
    return;
  }
  uint8_t* rec = static_cast<uint8_t*>(a.WS) + blockIdx.x * record_bytes(a.K);
  if (tid == 0) *reinterpret_cast<Record*>(rec) = Record{s, 0};
  if (a.K == 0) return;
  u64* kept = reinterpret_cast<u64*>(rec + sizeof(Record));
  in_order(lds, n, a.K, [&](int at, u64 e) { kept[at] = e; }, [&](int at) { kept[at] = 0; });
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
  u64 e[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = tid + i * kThreads, ch = K > 0 ? j / K : 0;
    e[i] = 0;
    // (the parts' best go to different threads, or few threads' largest would be much larger than the others')
    if (i * kThreads < a.chunks * K && ch < a.chunks) e[i] = reinterpret_cast<const u64*>(at(ch) + sizeof(Record))[(j - ch * K + ch) % K];
  }
  const Given<F32> given(a, row, tid);
  s = join_all(s, lds);
  unsigned bound;
  finish<F32>(a, row, s, given, lds, K > 0 ? gather(lds, e, K, bound) : 0);
}

}  // namespace

// Rows are cut where there are fewer than CUs, for two workgroups a CU, in parts of 2048 values at least.  (Rows of 151936, 8 alternatives, both
// launches: 128 rows 22 us in four parts each, 25 in two, 24 in eight; 256 rows 29 in two, 29 whole; 384 rows 37 and 35; 512 rows 46 and 37.)
LogprobsPlan logprobs_plan(int S, int V, int K) {
  LogprobsPlan p;
  long want = S >= 256 || S == 0 ? 1 : (512 + S - 1) / S;
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
