// topk.hip -- the K largest logits of each row with their columns, and the
// row's log-sum-exp at a temperature.
//
// Order: larger logits first, equal ones (the zeros of both signs too) by
// ascending column, NaN before everything. With a logit's bits made into a
// whole number o in its order, that is the order of the 64-bit keys
// (o, ~column), and keys are distinct.
//
// A work-group each row. The K-th largest of the first stretch's group maxima
// (a group: some of one thread's logits) is a bound that at least K logits
// reach; only logits that reach it become keys in LDS: of logits in no order,
// with G of them a group and n groups, about K / (n G) of the row. The first
// stretch is read once more for its keys (from the caches), the rest once. When
// there are many keys, or they do not fit, the K largest are kept and the bound
// rises to the last of them. The sum of exponentials is carried along per
// thread. Logits of -inf never become keys that way; where fewer than K others
// are there, the first of them fill up.
//
// Few rows are cut into segments, whose sorted lists a second kernel merges.
//
// 4096 rows of 128256 bf16, K = 64: 255 us, 4.1 TB/s; vector instructions take 57%
// of the cycles (ten a logit: conversion, comparison, one multiply-add, the
// exponential, its sum, and what the keys cost), the rest is waits at barriers and
// for loads. One row of 151936 fp32, K = 20: 23 us in two launches.
//
// Rows in ascending order cost most: every logit reaches the bound so far, no
// tile's keys fit, and each piece is sorted. The same 4096 rows 17.8 ms instead of
// 0.26 (K = 1024: 22.7 instead of 1.37), the one row 49 us.
#include "group_launch.hpp"
#include "losses_launch.hpp"
#include "mma256.hpp"

namespace lmhead {

namespace {

constexpr int TK_THREADS = 256;
constexpr int TK_CAP = 4096;   // keys in LDS
constexpr int TK_TILE = 4;     // 16-byte pieces a thread in flight
constexpr int TK_FIRST = 8;    // ... in the first stretch
constexpr int TK_COUNT = 512;  // keys up to which places are counted, not sorted
// Up to this ref / temperature (in powers of 2) x c - ref c is one multiply-add: what the
// product's rounding adds to the exponent, 2^-5, is no more than lse's own rounding. Past
// 2^31 it would be 128: every term 0, or infinite.
constexpr float TK_PRODUCT = 1048576.0f;
constexpr float TK_NEG_INF = -__builtin_inff();
constexpr float TK_LOWEST = -__FLT_MAX__;

__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);  // -0 to 0
  return x != x ? 0xFFFFFFFFu : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t o) {
  return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// The elements of a 16-byte piece.
template <typename T>
struct Piece {
  static constexpr int N = 16 / sizeof(T), PER_WORD = 4 / sizeof(T);
  static constexpr uint32_t NEG_INF = sizeof(T) == 4 ? 0xFF800000u : std::is_same_v<T, _Float16> ? 0xFC00u : 0xFF80u;
  static __device__ __forceinline__ float at(const u32x4 &v, int i) {
    // (a bit cast of a vector's element itself would take the first one)
    const uint32_t word = v[i / PER_WORD];
    if constexpr (sizeof(T) == 4)
      return __builtin_bit_cast(float, word);
    else if constexpr (std::is_same_v<T, _Float16>)
      return (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? word >> 16 : word));
    else
      return __builtin_bit_cast(float, i & 1 ? word & 0xFFFF0000u : word << 16);
  }
  // -inf in the places of a piece that begins at element `first` of `V` that are not there
  static __device__ __forceinline__ u32x4 cut(const u32x4 &v, int first, int V) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t word = v[j];
#pragma unroll
      for (int h = 0; h < PER_WORD; ++h) {
        const uint32_t mask = sizeof(T) == 4 ? 0xFFFFFFFFu : 0xFFFFu << (16 * h), inf = NEG_INF << (16 * h);
        word = (uint32_t)(first + j * PER_WORD + h) < (uint32_t)V ? word : (word & ~mask) | inf;
      }
      r[j] = word;
    }
    return r;
  }
};

// Sorts n keys (a power of two, at least 128) in descending order. Pairs that
// one wave works on stay within 128 keys for distances up to 64, so only
// longer ones meet at a barrier.
__device__ __forceinline__ void sort_step(uint64_t *key, int n, int k, int j) {
  for (int p = threadIdx.x; p < n / 2; p += TK_THREADS) {
    const int i = ((p & ~(j - 1)) << 1) | (p & (j - 1));
    const uint64_t a = key[i], b = key[i | j];
    if ((a < b) == ((i & k) == 0)) {
      key[i] = b;
      key[i | j] = a;
    }
  }
}
__device__ __forceinline__ void sort_keys(uint64_t *key, int n) {
  __syncthreads();
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      sort_step(key, n, k, j);
      if (j > 64 || (j == 1 && k >= 128)) __syncthreads();
      else sched_fence();
    }
}
// The K largest of n keys (at most TK_COUNT) to their places: keys are distinct
// (but for those of nothing, 0), and a key's place is the number of larger ones.
// For that few a third of a sort's steps: each of those is a round trip to LDS.
__device__ __forceinline__ void count_places(uint64_t *key, int n, int K) {
  constexpr int Q = TK_COUNT / TK_THREADS;
  const int tid = threadIdx.x;
  __syncthreads();
  uint64_t mine[Q];
  int place[Q] = {};
#pragma unroll
  for (int q = 0; q < Q; ++q) mine[q] = q * TK_THREADS + tid < n ? key[q * TK_THREADS + tid] : 0;
  if (n <= TK_THREADS) {
#pragma unroll 8
    for (int i = 0; i < n; ++i) place[0] += key[i] > mine[0] ? 1 : 0;
  } else {
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const uint64_t other = key[i];
#pragma unroll
      for (int q = 0; q < Q; ++q) place[q] += other > mine[q] ? 1 : 0;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (mine[q] != 0 && place[q] < K) key[place[q]] = mine[q];
}
// The largest v that at least K of the wave's 64 R values reach (0 when there
// are not as many but of 0), bit by bit.
template <int R>
__device__ __forceinline__ uint32_t kth_value(const uint32_t (&x)[R], int K) {
  uint32_t v = 0;
#pragma unroll 1
  for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
    int n = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) n += __popcll(__ballot(x[r] >= (v | bit)));
    if (n >= K) v |= bit;
  }
  return v;
}
__device__ __forceinline__ int power_of_two(int n, int least) {
  while (least < n) least <<= 1;
  return least;
}

struct TopkPart {
  const uint8_t *logits;
  int64_t M, V, row_bytes;
  int K;
  int segments;
  float c;             // log2(e) / temperature
  float temperature;
  void *values;        // [M, K], segments == 1
  int32_t *ids;
  float *lse;
  uint64_t *lists;     // [M, segments, K]
  float2 *sums;        // [M, segments] {largest, sum of exp((x - largest) / temperature)}
};

__device__ __forceinline__ void fold_sum(float &m, float &s, float om, float os, float c) {
  const float n = fmaxf(m, om);
  const float a = s == 0.0f ? 0.0f : __fmul_rn(s, __builtin_amdgcn_exp2f(__fmul_rn(c, __fsub_rn(m, n))));
  const float b = os == 0.0f ? 0.0f : __fmul_rn(os, __builtin_amdgcn_exp2f(__fmul_rn(c, __fsub_rn(om, n))));
  s = __fadd_rn(a, b);
  m = n;
}
__device__ __forceinline__ float lse_of(float m, float s, float temperature) {
  return s == 0.0f ? TK_NEG_INF : __fadd_rn(__fdiv_rn(m, temperature), logf(s));
}

// One of a row's results. The K logits that reach the bounds exist (V >= K); an
// address is made from a column of the row only, all the same.
template <typename T>
__device__ __forceinline__ void put(const TopkPart &p, int64_t row, int k, uint64_t key) {
  const uint32_t col = ~(uint32_t)key;
  p.ids[row * p.K + k] = (int32_t)col;
  if (col < (uint64_t)p.V)
    static_cast<T *>(p.values)[row * p.K + k] = reinterpret_cast<const T *>(p.logits + row * p.row_bytes)[col];
}

template <typename T>
__global__ __launch_bounds__(TK_THREADS, 4) void topk_part_kernel(TopkPart p) {
  constexpr int N = Piece<T>::N;
  __shared__ uint64_t key[TK_CAP];
  __shared__ int count;
  __shared__ uint32_t kth;  // the group maximum of that place
  __shared__ float2 wave_sums[TK_THREADS / 64];
  const int64_t g = group_number(), row = g / p.segments;
  if (row >= p.M) return;
  const int seg = (int)(g - row * p.segments), tid = threadIdx.x, K = p.K;
  // 16-byte pieces from the aligned address at or before the row's start
  const uint8_t *const start = p.logits + row * p.row_bytes;
  const int off = (int)(reinterpret_cast<uint64_t>(start) & 15), shift = off / (int)sizeof(T);
  const u32x4 *const base = reinterpret_cast<const u32x4 *>(start - off);
  const int V = (int)p.V, pieces = (V + shift + N - 1) / N;
  const int per = (pieces + p.segments - 1) / p.segments;
  const int lo = seg * per < pieces ? seg * per : pieces, hi = lo + per < pieces ? lo + per : pieces;

  float ref = TK_NEG_INF, sum = 0.0f;  // this thread's sum of exp((x - ref) / temperature)
  float bound = TK_LOWEST;             // no logit below it is wanted; never -inf
  float most = TK_NEG_INF;             // the largest logit that became an entry lately
  int keys = 0;                        // entries that are keys; behind them {column, logit}

  // Tiles of TK_TILE pieces a thread from piece `from` to `to`, the next in
  // flight; -inf where there is nothing, which adds nothing and is not wanted.
  auto tiles = [&](int from, int to, auto &&f) {
    u32x4 w[TK_TILE], next[TK_TILE];
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < TK_TILE; ++k) {
        const int i = i0 + k * TK_THREADS + tid;
        next[k] = base[i < to ? i : from];
      }
    };
    if (from < to) load(from);
#pragma unroll 1
    for (int i0 = from; i0 < to; i0 += TK_TILE * TK_THREADS) {
#pragma unroll
      for (int k = 0; k < TK_TILE; ++k) w[k] = next[k];
      if (i0 + TK_TILE * TK_THREADS < to) load(i0 + TK_TILE * TK_THREADS);
      // nearly every tile lies whole inside the row
      if (i0 * N < shift || (i0 + TK_TILE * TK_THREADS) * N - shift > V || i0 + TK_TILE * TK_THREADS > to)
#pragma unroll
        for (int k = 0; k < TK_TILE; ++k) {
          const int i = i0 + k * TK_THREADS + tid;
          w[k] = Piece<T>::cut(w[k], i < to ? i * N - shift : V, V);
        }
      f(w, i0 + tid);
    }
  };
  auto raise = [&](float x) {
    if (x > ref) {
      sum = sum == 0.0f ? 0.0f : __fmul_rn(sum, __builtin_amdgcn_exp2f(__fmul_rn(p.c, __fsub_rn(ref, x))));
      ref = x;
    }
  };
  // {column, logit} of the logits of P pieces that reach the bound. A wave
  // counts its own and reserves their places at once (none where they do not
  // fit: then the tile is taken again); the writes need no answer. The ballots
  // are kept as scalar numbers, or each test of one would cost vector operations.
  auto take = [&](auto pc, const u32x4 *w, int i) {
    constexpr int P = decltype(pc)::value;
    uint64_t set[P * N];
    int n = 0;
#pragma unroll
    for (int k = 0; k < P * N; ++k) {
      set[k] = __ballot(!(Piece<T>::at(w[k / N], k % N) < bound));
      asm("" : "+s"(set[k]));
      n += __popcll(set[k]);
    }
    if (n == 0) return;
    int at = 0;
    if ((tid & 63) == 0) at = atomicAdd(&count, n);
    at = __builtin_amdgcn_readfirstlane(at);
    if (at + n > TK_CAP) return;
#pragma unroll
    for (int k4 = 0; k4 < P * N; k4 += 4) {
      if ((set[k4] | set[k4 + 1] | set[k4 + 2] | set[k4 + 3]) == 0) continue;
#pragma unroll
      for (int k = k4; k < k4 + 4; ++k)
        if (set[k] != 0) {
          const float x = Piece<T>::at(w[k / N], k % N);
          const int place = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(set[k] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)set[k], 0));
          if (__builtin_amdgcn_inverse_ballot_w64(set[k])) {
            key[place] = (uint64_t)__builtin_bit_cast(uint32_t, x) << 32 | (uint32_t)((i + k / N * TK_THREADS) * N - shift + k % N);
            most = x > most ? x : most;
          }
          at += __popcll(set[k]);
        }
    }
  };
  // adds a tile to the thread's sum: none of its logits is above ref
  auto add = [&](const u32x4 (&w)[TK_TILE]) {
    const float rc = -__fmul_rn(ref, p.c);
    if (fabsf(rc) < TK_PRODUCT) {
#pragma unroll
      for (int k = 0; k < TK_TILE; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e)
          sum = __fadd_rn(sum, __builtin_amdgcn_exp2f(__fmaf_rn(Piece<T>::at(w[k], e), p.c, rc)));
    } else {  // the difference first
#pragma unroll
      for (int k = 0; k < TK_TILE; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e)
          sum = __fadd_rn(sum, __builtin_amdgcn_exp2f(__fmul_rn(p.c, __fsub_rn(Piece<T>::at(w[k], e), ref))));
    }
  };
  // Of the first n keys those that are among the K largest logits (with all that
  // equal the last of them); all threads, after a barrier. What comes later has
  // larger columns, so a logit equal to the last is not wanted any more.
  auto prune = [&](int n) {
    constexpr int Q = TK_COUNT / TK_THREADS;
    for (int i = keys + tid; i < n; i += TK_THREADS) {
      const uint64_t raw = key[i];
      key[i] = (uint64_t)order_of(__builtin_bit_cast(float, (uint32_t)(raw >> 32))) << 32 | ~(uint32_t)raw;
    }
    keys = n;
    if (n > TK_COUNT) {
      const int all = power_of_two(n, 128);
      for (int i = n + tid; i < all; i += TK_THREADS) key[i] = 0;
      sort_keys(key, all);
      keys = n < K ? n : K;
      if (tid == 0) {
        count = keys;
        kth = (uint32_t)(key[K - 1] >> 32);
      }
    } else if (n >= K) {
      __syncthreads();
      uint64_t mine[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) mine[q] = q * TK_THREADS + tid < n ? key[q * TK_THREADS + tid] : 0;
      if (tid < 64) {
        uint32_t x[TK_COUNT / 64];
#pragma unroll
        for (int r = 0; r < TK_COUNT / 64; ++r) x[r] = r * 64 + tid < n ? (uint32_t)(key[r * 64 + tid] >> 32) : 0;
        const uint32_t v = kth_value(x, K);
        if (tid == 0) {
          kth = v;
          count = 0;
        }
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const uint64_t all = __ballot(mine[q] != 0 && (uint32_t)(mine[q] >> 32) >= kth);
        if (all == 0) continue;
        int at = 0;
        if ((tid & 63) == 0) at = atomicAdd(&count, __popcll(all));
        at = __builtin_amdgcn_readfirstlane(at) + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
        if (all >> (tid & 63) & 1) key[at] = mine[q];
      }
      __syncthreads();
      keys = count;
    } else if (tid == 0) {
      count = n;  // not what a tile that did not fit has made of it
    }
    __syncthreads();
    if (n >= K) {
      const uint32_t last = kth, infinite = order_of(__builtin_inff());
      bound = fmaxf(last < infinite ? of_order(last + 1) : __builtin_inff(), TK_LOWEST);
      // (not the bound, which may lie above the row's largest logit: where a step of
      // fp32 there is an exponent of 128 or more, no term would be left)
      raise(of_order(last));
    }
  };

  if (tid == 0) {
    count = 0;
    kth = 0;
  }
  // the bound from the first stretch's group maxima: of all of a thread's
  // pieces, half of them, or each
  const int mid = lo + TK_FIRST * TK_THREADS < hi ? lo + TK_FIRST * TK_THREADS : hi;
  const int group = K <= TK_THREADS / 4 ? TK_FIRST : K <= TK_THREADS ? TK_FIRST / 2 : 1;
  uint32_t *const maxima = reinterpret_cast<uint32_t *>(key);  // [TK_FIRST / group][TK_THREADS]
  {
    float gm = TK_NEG_INF;
    int done = 0;
#pragma unroll
    for (int k = 0; k < TK_FIRST; ++k) maxima[k * TK_THREADS + tid] = 0;
    tiles(lo, mid, [&](const u32x4 (&w)[TK_TILE], int) {
#pragma unroll
      for (int k = 0; k < TK_TILE; ++k) {
#pragma unroll
        for (int e = 0; e < N; ++e) gm = fmaxf(gm, Piece<T>::at(w[k], e));
        ++done;
        if (done % group == 0) {
          maxima[(done / group - 1) * TK_THREADS + tid] = order_of(gm);
          gm = TK_NEG_INF;
        }
      }
    });
    if (done % group != 0) maxima[done / group * TK_THREADS + tid] = order_of(gm);
  }
  __syncthreads();
  if (tid < 64) {
    constexpr int R = TK_THREADS / 64;
    auto find = [&](auto rc) {
      uint32_t x[decltype(rc)::value];
#pragma unroll
      for (int r = 0; r < decltype(rc)::value; ++r) x[r] = maxima[r * 64 + tid];
      return kth_value(x, K);
    };
    const uint32_t v = group == TK_FIRST ? find(std::integral_constant<int, R>{})
                       : group > 1       ? find(std::integral_constant<int, 2 * R>{})
                                         : find(std::integral_constant<int, TK_FIRST * R>{});
    if (tid == 0) kth = v;
  }
  __syncthreads();
  // (a group of no logits is one of -inf: any other reaches that)
  if (kth != 0) bound = fmaxf(of_order(kth), TK_LOWEST);
  raise(bound);
  __syncthreads();
  int total = 0;  // entries so far
  tiles(lo, hi, [&](const u32x4 (&w)[TK_TILE], int i) {
    constexpr int P = 16 / N;  // the ballots of 16 logits at a time stay in scalar registers
#pragma unroll
    for (int k = 0; k < TK_TILE; k += P) take(std::integral_constant<int, P>{}, w + k, i + k * TK_THREADS);
    __syncthreads();
    int n = count;
    const bool fits = n <= TK_CAP;
    // of a tile that did not fit, which waves found room is chance: as if none had
    if (fits) raise(most);
    most = TK_NEG_INF;
    if (n > keys + K + 64) {
      // pruned; where the tile's keys did not fit, piece by piece
      if (!fits) n = total;
#pragma unroll 1
      for (int k = 0;; ++k) {
        __syncthreads();
        prune(n);
        if (fits || k == TK_TILE) break;
        const u32x4 one = k == 0 ? w[0] : k == 1 ? w[1] : k == 2 ? w[2] : w[3];
        take(std::integral_constant<int, 1>{}, &one, i + k * TK_THREADS);
        raise(most);
        most = TK_NEG_INF;
        __syncthreads();
        n = count;
      }
      n = keys;
    }
    total = n;
    add(w);
    __syncthreads();
  });
  {
    prune(total);
    int n = keys;
    if (n <= TK_COUNT) count_places(key, n, K);  // more are sorted already, and K
    __syncthreads();
    if (n > K) n = K;
    // the first logits of -inf, where there are not enough others
    for (int64_t c0 = (int64_t)lo * N - shift; n < K && c0 < (int64_t)hi * N - shift; c0 += TK_THREADS) {
      const int64_t col = c0 + tid;
      const bool mine = col >= 0 && col < V && col < (int64_t)hi * N - shift &&
                        (float)reinterpret_cast<const T *>(start)[col] == TK_NEG_INF;
      const uint64_t all = __ballot(mine);
      if ((tid & 63) == 0) reinterpret_cast<int *>(wave_sums)[tid >> 6] = __popcll(all);
      __syncthreads();
      int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
#pragma unroll
      for (int w = 0; w < TK_THREADS / 64; ++w) {
        const int c = reinterpret_cast<int *>(wave_sums)[w];
        if (w < (tid >> 6)) at += c;
        n += c;
      }
      if (mine && at < K) key[at] = (uint64_t)order_of(TK_NEG_INF) << 32 | ~(uint32_t)col;
      __syncthreads();
    }
    if (tid == 0) count = n < K ? n : K;
    __syncthreads();
  }

  // the sums: lanes by exchanges, then the waves
#pragma unroll
  for (int d = 32; d; d >>= 1) fold_sum(ref, sum, __shfl_xor(ref, d), __shfl_xor(sum, d), p.c);
  if ((tid & 63) == 0) wave_sums[tid >> 6] = float2{ref, sum};
  __syncthreads();
  if (tid == 0)
#pragma unroll
    for (int k = 1; k < TK_THREADS / 64; ++k) fold_sum(ref, sum, wave_sums[k].x, wave_sums[k].y, p.c);
  if (p.segments == 1) {
    for (int k = tid; k < K; k += TK_THREADS) put<T>(p, row, k, key[k]);
    if (tid == 0) p.lse[row] = lse_of(ref, sum, p.temperature);
  } else {
    for (int k = tid; k < K; k += TK_THREADS) p.lists[g * K + k] = k < count ? key[k] : 0;
    if (tid == 0) p.sums[g] = float2{ref, sum};
  }
}

// Merges a row's lists. With S lists, the smallest of their q-th largest keys,
// q = ceil(K / S), is a bound that K keys reach; those that do are sorted out: some
// 300 of 1280 for K = 20 of 64 lists (q = 1: the least of 64 maxima), some 140 of
// 1050 for K = 50 of 21.
template <typename T>
__global__ __launch_bounds__(TK_THREADS) void topk_merge_kernel(TopkPart p) {
  __shared__ uint64_t out[TK_CAP];
  __shared__ uint64_t bound;
  __shared__ int count;
  const int64_t row = group_number();
  if (row >= p.M) return;
  const int tid = threadIdx.x, K = p.K, S = p.segments, all = S * K;
  const uint64_t *const in = p.lists + row * all;
  if (tid < 64) {  // at most 64 segments
    uint64_t least = tid < S ? in[tid * K + (K + S - 1) / S - 1] : ~0ull;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const uint64_t other = __shfl_xor(least, d);
      least = other < least ? other : least;
    }
    if (tid == 0) {
      bound = least;
      count = 0;
    }
  }
  __syncthreads();
  const uint64_t least = bound;
  for (int i = tid; i < all; i += TK_THREADS) {
    const uint64_t k = in[i];
    if (k >= least && k != 0) out[atomicAdd(&count, 1)] = k;  // keys are distinct: their order does not matter
  }
  __syncthreads();
  const int n = count;
  if (n <= TK_COUNT) {
    count_places(out, n, K);
  } else {
    const int pow2 = power_of_two(n, 128);
    for (int i = n + tid; i < pow2; i += TK_THREADS) out[i] = 0;
    sort_keys(out, pow2);
  }
  __syncthreads();
  for (int k = tid; k < K; k += TK_THREADS) put<T>(p, row, k, out[k]);
  if (tid < 64) {  // at most 64 segments
    const float2 e = tid < p.segments ? p.sums[row * p.segments + tid] : float2{TK_NEG_INF, 0.0f};
    float m = e.x, s = e.y;
#pragma unroll
    for (int d = 32; d; d >>= 1) fold_sum(m, s, __shfl_xor(m, d), __shfl_xor(s, d), p.c);
    if (tid == 0) p.lse[row] = lse_of(m, s, p.temperature);
  }
}

// Segments of a row: enough for four work-groups a CU, of at least two pieces
// a thread (a segment has a bound to find however short it is), and no more
// than the merge holds.
struct TopkPlan {
  int segments;
  int64_t lists, sums, bytes;
};
TopkPlan topk_plan(int64_t M, int64_t V, int64_t K, int size) {
  TopkPlan p;
  int64_t s = M > 0 ? 1024 / M : 1;
  const int64_t most = V * size / 16 / (2 * TK_THREADS);
  if (s > most) s = most;
  if (s > TK_CAP / K) s = TK_CAP / K;
  if (s > 64) s = 64;
  p.segments = (int)(s > 1 ? s : 1);
  p.lists = 0;
  p.sums = p.segments > 1 ? 8 * M * p.segments * K : 0;
  p.bytes = p.sums + (p.segments > 1 ? 8 * M * p.segments : 0);
  return p;
}

template <typename T>
hipError_t topk(const TopkArgs &c, hipStream_t s) {
  const TopkPlan pl = topk_plan(c.M, c.V, c.K, sizeof(T));
  uint8_t *const ws = static_cast<uint8_t *>(c.workspace);
  // (a temperature below fp32's normal numbers: a difference of 0 stays one)
  const double factor = 1.4426950408889634 / (double)c.temperature;
  const TopkPart p{static_cast<const uint8_t *>(c.logits), c.M, c.V, c.ld * (int64_t)sizeof(T), (int)c.K, pl.segments,
                   (float)(factor < __FLT_MAX__ ? factor : __FLT_MAX__), c.temperature, c.values, c.ids, c.lse,
                   reinterpret_cast<uint64_t *>(ws + pl.lists), reinterpret_cast<float2 *>(ws + pl.sums)};
  hipError_t e = launch_kernel(topk_part_kernel<T>, numbered_grid(c.M * pl.segments), dim3(TK_THREADS), s, p);
  if (e == hipSuccess && pl.segments > 1)
    e = launch_kernel(topk_merge_kernel<T>, numbered_grid(c.M), dim3(TK_THREADS), s, p);
  return e;
}

}  // namespace

// Whatever the logits' type.
int64_t topk_bytes(int64_t M, int64_t V, int64_t K) {
  const int64_t a = topk_plan(M, V, K, 4).bytes, b = topk_plan(M, V, K, 2).bytes;
  return a > b ? a : b;
}

hipError_t launch_topk(const TopkArgs &c, hipStream_t s) {
  return c.logits_type == OUT_F32    ? topk<float>(c, s)
         : c.logits_type == OUT_BF16 ? topk<__bf16>(c, s)
                                     : topk<_Float16>(c, s);
}

}  // namespace lmhead
