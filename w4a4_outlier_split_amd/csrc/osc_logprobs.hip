// Log probabilities, entropy and the most likely tokens from rows of logits, in one pass over them.
//
// With u = scale log2(e) x, a reference R near the row's largest u, l = sum 2^(u - R) and t = sum 2^(u - R) (u - R):
//   log2 p(v) = u_v - R - log2 l,   entropy = log2 l - t / l  (in bits),
// and parts with references R_a, R_b join as l = l_a 2^(R_a - R) + ..., t = 2^(R_a - R) (t_a + (R_a - R) l_a) + ...
// Threads keep R, l and t of their own and move R where a value exceeds it by more than kSlack.
//
// The K largest come along: the first 64 values of each thread give 256 maxima, whose K-th largest is a bound that at
// least K values reach.  From then on a value that reaches the bound is noted, with its index, in LDS: a few times K
// of a row in usual orders.  Should the list run over, the round is taken again in small steps, and the list is cut to its K best between them,
// whose last is the new bound.  What is noted depends on the order of the wavefronts, the K best of it do not.
#include "osc_internal.h"

namespace osc {
namespace {

typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kRound = 8;        // vectors of 16 bytes a thread and round
constexpr int kCap = 4096;       // noted values
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

struct Lds {
  unsigned key[kCap];
  int idx[kCap];
  Sum sums[4];
  unsigned top[kThreads];
  int count[3];
  int votes[2][4];
};

// how many threads' flags are set, over the workgroup; `turn` alternates from call to call
__device__ __forceinline__ int vote(Lds& s, int mine, int& turn) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mine += __shfl_xor(mine, d);
  if ((threadIdx.x & 63) == 0) s.votes[turn][threadIdx.x >> 6] = mine;
  __syncthreads();
  const int all = s.votes[turn][0] + s.votes[turn][1] + s.votes[turn][2] + s.votes[turn][3];
  turn ^= 1;
  return all;
}

// Cuts the n noted values to the K best (n >= K); the bound becomes the last of them.  All threads, behind a barrier.
__device__ __forceinline__ void prune(Lds& s, int n, int K, unsigned& bound, int& bound_idx) {
  constexpr int PER = kCap / kThreads;
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
  bound = low, bound_idx = last;
}

// The K best of the n noted values in order: write(place, key, index) for each, then none(place) for places without one.
template <typename Write, typename None>
__device__ __forceinline__ void in_order(Lds& s, int n, int K, Write write, None none) {
  if (n > kThreads) {
    unsigned b;
    int bi;
    prune(s, n, K, b, bi);
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
template <bool F32>
__device__ __forceinline__ void finish(const LogprobsArgs& a, int row, const Sum& s, Lds& lds, int n) {
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

__device__ __forceinline__ Sum join_all(Sum s, Lds& lds) {
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
__global__ __launch_bounds__(kThreads) void k_logprobs(LogprobsArgs a) {
  constexpr int E = F32 ? 4 : 8;  // values of a vector
  __shared__ Lds lds;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks;
  const int tid = threadIdx.x;
  const uint8_t* x0 = static_cast<const uint8_t*>(a.X) + (long)row * a.ld * (F32 ? 4 : 2);
  const int skew = (int)(reinterpret_cast<uintptr_t>(x0) & 15) / (F32 ? 4 : 2);  // values ahead of the row in its first vector
  const u4* xv = reinterpret_cast<const u4*>(x0 - skew * (F32 ? 4 : 2));
  const int vectors = (a.V + skew + E - 1) / E;
  const int v0 = (int)((long)vectors * chunk / a.chunks), v1 = (int)((long)vectors * (chunk + 1) / a.chunks);
  const float c = a.scale_log2;
  const unsigned ninf = F32 ? 0xFF800000u : 0xFF80FF80u;

  // vector v of the row; what is not the row's as -inf, and nothing behind the row's end is read
  auto load = [&](int v) {
    u4 q = {ninf, ninf, ninf, ninf};
    if (v >= v1) return q;
    const int e0 = v * E - skew;
    if (e0 + E <= a.V) {
      q = xv[v];
      if (e0 >= 0) return q;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const bool in = e0 + i >= 0 && e0 + i < a.V;
      if (F32) {
        const unsigned w = in ? static_cast<const unsigned*>(a.X)[(long)row * a.ld + e0 + i] : ninf;
        q[i & 3] = w;
      } else {
        const unsigned w = in ? static_cast<const uint16_t*>(a.X)[(long)row * a.ld + e0 + i] : 0xFF80u;
        q[(i >> 1) & 3] = i & 1 ? (q[(i >> 1) & 3] & 0xFFFF) | w << 16 : (q[(i >> 1) & 3] & 0xFFFF0000u) | w;
      }
    }
    return q;
  };
  auto value = [&](const u4& q, int i) {
    const unsigned w = q[F32 ? i & 3 : (i >> 1) & 3];  // (a bit cast straight from a vector's element reads element 0)
    return __builtin_bit_cast(float, F32 ? w : i & 1 ? w & 0xFFFF0000u : w << 16);
  };
  auto largest = [&](const u4& q) {
    float m = value(q, 0);
#pragma unroll
    for (int i = 1; i < E; ++i) m = fmaxf(m, value(q, i));
    return m;
  };

  if (tid < 3) lds.count[tid] = 0;
  Sum s = {neg_inf(), 0.0f, 0.0f};
  float bound = neg_inf();
  int bound_idx = 0x7FFFFFFF, have = 0;
  bool first = true;
  int turn = 0;
  for (int v = v0; v < v1; v += kRound * kThreads) {
    u4 q[kRound];
#pragma unroll
    for (int u = 0; u < kRound; ++u) q[u] = load(v + u * kThreads + tid);
    float round_max = neg_inf();
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      const float m = largest(q[u]);
      round_max = fmaxf(round_max, m);
      const float mu = m * c;
      if (mu > base_of(s.r) + kSlack || (s.r == neg_inf() && mu > neg_inf())) s = join(s, Sum{mu, 0.0f, 0.0f});
      const float z = -base_of(s.r);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float d = __builtin_fmaf(value(q[u], i), c, z), e = __builtin_amdgcn_exp2f(d);
        s.l += e;
        s.t = __builtin_fmaf(e, fmaxf(d, -1000.0f), s.t);
      }
    }
    if (a.K == 0) continue;
    if (first) {
      first = false;
      lds.top[tid] = key_of(round_max);
      __syncthreads();
      unsigned k[4], low = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = lds.top[64 * j + (tid & 63)];
      for (int bit = 31; bit >= (F32 ? 0 : 16); --bit) {
        const unsigned trial = low | 1u << bit;
        int n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) n += __popcll(__ballot(k[j] >= trial));
        if (n >= a.K) low = trial;
      }
      bound = low <= (unsigned)kNone ? neg_inf() : value_of(low);
    }
    auto note = [&](int u, int* count) {
      if (!(largest(q[u]) >= bound)) return;
      const int e0 = (v + u * kThreads + tid) * E - skew;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float x = value(q[u], i);
        if (x > neg_inf() && (x > bound || (x == bound && e0 + i <= bound_idx))) {
          const int at = have + atomicAdd(count, 1);
          if (at < kCap) lds.key[at] = key_of(x), lds.idx[at] = e0 + i;
        }
      }
    };
#pragma unroll
    for (int u = 0; u < kRound; ++u) note(u, &lds.count[turn]);
    // the counter of the next round but one: it was last read ahead of the barrier before
    if (tid == 0) lds.count[turn == 2 ? 0 : turn + 1] = 0;
    __syncthreads();
    const int total = have + lds.count[turn];
    turn = turn == 2 ? 0 : turn + 1;
    if (total <= kCap) {
      have = total;
      continue;
    }
    // too many: once more, a vector a thread at a time
#pragma unroll 1
    for (int u = 0; u < kRound; ++u) {
      __syncthreads();
      if (have + kThreads * E > kCap) {
        unsigned b;
        prune(lds, have, a.K, b, bound_idx);
        have = a.K;
        bound = value_of(b);
      }
      if (tid == 0) lds.count[turn] = 0;
      __syncthreads();
      // q[u] by selection: a register cannot be indexed
      u4 w = q[0];
#pragma unroll
      for (int y = 1; y < kRound; ++y)
        if (y == u) w = q[y];
      const u4 keep = q[0];
      q[0] = w;
      const int e0 = (v + u * kThreads + tid) * E - skew;
      if (largest(w) >= bound) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float x = value(w, i);
          if (x > neg_inf() && (x > bound || (x == bound && e0 + i <= bound_idx))) {
            const int at = have + atomicAdd(&lds.count[turn], 1);
            lds.key[at] = key_of(x), lds.idx[at] = e0 + i;
          }
        }
      }
      q[0] = keep;
      __syncthreads();
      have += lds.count[turn];
    }
    __syncthreads();
    if (tid < 3) lds.count[tid] = 0;
    __syncthreads();
  }
  s = join_all(s, lds);
  if (a.chunks == 1) {
    finish<F32>(a, row, s, lds, have);
    return;
  }
  uint8_t* rec = static_cast<uint8_t*>(a.WS) + blockIdx.x * record_bytes(a.K);
  if (tid == 0) *reinterpret_cast<Record*>(rec) = Record{s, have < a.K ? have : a.K};
  if (a.K == 0) return;
  unsigned* keys = reinterpret_cast<unsigned*>(rec + sizeof(Record));
  in_order(lds, have, a.K, [&](int at, unsigned key, int idx) { keys[at] = key, keys[a.K + at] = (unsigned)idx; }, [](int) {});
}

// A row's parts in their order.
template <bool F32>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(LogprobsArgs a) {
  __shared__ Lds lds;
  const int row = blockIdx.x, tid = threadIdx.x;
  const uint8_t* rec = static_cast<const uint8_t*>(a.WS) + (long)row * a.chunks * record_bytes(a.K);
  auto at = [&](int c) { return rec + c * record_bytes(a.K); };
  Sum s = {neg_inf(), 0.0f, 0.0f};
  int mine = 0;
  if (tid < a.chunks) {  // at most as many as a wavefront's lanes
    const Record& r = *reinterpret_cast<const Record*>(at(tid));
    s = r.s, mine = r.n;
  }
  if (tid == 0) lds.count[0] = 0;
  s = join_all(s, lds);
  if (a.K > 0) {
    for (int i = tid; i < a.chunks * a.K; i += kThreads) {
      const int c = i / a.K, k = i - c * a.K;
      const Record& r = *reinterpret_cast<const Record*>(at(c));
      if (k < r.n) {
        const unsigned* keys = reinterpret_cast<const unsigned*>(at(c) + sizeof(Record));
        const int to = atomicAdd(&lds.count[0], 1);
        lds.key[to] = keys[k], lds.idx[to] = (int)keys[a.K + k];
      }
    }
  }
  (void)mine;
  __syncthreads();
  finish<F32>(a, row, s, lds, lds.count[0]);
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
