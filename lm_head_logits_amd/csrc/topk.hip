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
// reach, and only logits that reach it become keys in LDS: of logits in no order,
// with G of them a group and n groups, about K / (n G) of the row. The first
// stretch is read once more for its keys (from the caches), the rest once. The
// keys are sorted (bitonic, in LDS) when there are many or they do not fit, and
// at the end; the K largest are kept, the bound rises to the last of them. The
// sum of exponentials is carried along per thread.
//
// Few rows are cut into segments, whose sorted lists a second kernel merges two
// and two: the larger of a[i] and b[K - 1 - i] are the K largest of both.
#include "group_launch.hpp"
#include "losses_launch.hpp"
#include "mma256.hpp"

namespace lmhead {

namespace {

constexpr int TK_THREADS = 256, TK_CAP = 4096, TK_FIRST = 8, TK_TILE = 4, TK_SOFT = 512;
constexpr float TK_NEG_INF = -__builtin_inff();

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
  static constexpr int N = 16 / sizeof(T);
  static __device__ __forceinline__ float at(const u32x4 &v, int i) {
    // (a bit cast of a vector's element itself would take the first one)
    const uint32_t word = v[i / (N / 4)];
    if constexpr (sizeof(T) == 4)
      return __builtin_bit_cast(float, word);
    else if constexpr (std::is_same_v<T, _Float16>)
      return (float)__builtin_bit_cast(f16x2, word)[i & 1];
    else
      return __builtin_bit_cast(float, i & 1 ? word & 0xFFFF0000u : word << 16);
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
__device__ __forceinline__ int power_of_two(int n, int least) {
  while (least < n) least <<= 1;
  return least;
}

struct TopkPart {
  const uint8_t *logits;
  int64_t M, V, row_bytes;
  int K, lists_K;      // lists_K: K as a power of two
  int segments;
  float c;             // log2(e) / temperature
  float temperature;
  void *values;        // [M, K], segments == 1
  int32_t *ids;
  float *lse;
  uint64_t *lists;     // [M, segments, lists_K]
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
  const int lo = seg * per, hi = lo + per < pieces ? lo + per : pieces;

  float top = TK_NEG_INF, sum = 0.0f;  // this thread's largest logit, and its sum
  uint64_t bound = 0;                  // keys above it are wanted
  float bound_x = TK_NEG_INF;          // no logit below it has one

  // a piece's logits; EDGE: what lies outside the row or the segment is -inf,
  // which adds nothing
  auto unpack = [&](auto edge, const u32x4 &v, int i, float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      x[e] = Piece<T>::at(v, e);
      if constexpr (decltype(edge)::value) x[e] = (uint32_t)(i * N - shift + e) < (uint32_t)V && i < hi ? x[e] : TK_NEG_INF;
    }
  };
  // Tiles of TK_TILE pieces a thread from piece `from` to `to`, the next in flight.
  auto tiles = [&](int from, int to, auto &&f) {
    u32x4 w[TK_TILE], next[TK_TILE];
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < TK_TILE; ++k) {
        const int i = i0 + k * TK_THREADS + tid;
        next[k] = i < to ? base[i] : u32x4{0, 0, 0, 0};
      }
    };
    load(from);
#pragma unroll 1
    for (int i0 = from; i0 < to; i0 += TK_TILE * TK_THREADS) {
#pragma unroll
      for (int k = 0; k < TK_TILE; ++k) w[k] = next[k];
      load(i0 + TK_TILE * TK_THREADS);
      // nearly every tile lies whole inside the row
      if (i0 * N >= shift && (i0 + TK_TILE * TK_THREADS) * N - shift <= V && i0 + TK_TILE * TK_THREADS <= hi)
        f(std::false_type{}, w, i0 + tid);
      else
        f(std::true_type{}, w, i0 + tid);
    }
  };
  // adds a tile to the thread's sum, with its maxima by piece
  auto add = [&](auto edge, const u32x4 (&w)[TK_TILE], int i, float (&most)[TK_TILE]) {
    float x[TK_TILE][N], m = TK_NEG_INF;
#pragma unroll
    for (int k = 0; k < TK_TILE; ++k) {
      unpack(edge, w[k], i + k * TK_THREADS, x[k]);
      most[k] = x[k][0];
#pragma unroll
      for (int e = 1; e < N; ++e) most[k] = fmaxf(most[k], x[k][e]);
      m = fmaxf(m, most[k]);
    }
    if (m > top) {
      sum = sum == 0.0f ? 0.0f : __fmul_rn(sum, __builtin_amdgcn_exp2f(__fmul_rn(p.c, __fsub_rn(top, m))));
      top = m;
    }
    const float ref = top == TK_NEG_INF ? 0.0f : top;
#pragma unroll
    for (int k = 0; k < TK_TILE; ++k)
#pragma unroll
      for (int e = 0; e < N; ++e)
        sum = __fadd_rn(sum, __builtin_amdgcn_exp2f(__fmul_rn(p.c, __fsub_rn(x[k][e], ref))));
  };
  // the keys of a piece that are above the bound
  auto take = [&](auto edge, const u32x4 &v, int i) {
    float x[N];
    unpack(edge, v, i, x);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!(x[e] < bound_x)) {
        const uint32_t col = (uint32_t)(i * N - shift + e);
        const uint64_t k = (uint64_t)order_of(x[e]) << 32 | (uint32_t)~col;
        if (k > bound && (!decltype(edge)::value || (col < (uint32_t)V && i < hi))) {
          const int at = atomicAdd(&count, 1);
          if (at < TK_CAP) key[at] = k;
        }
      }
  };
  // the K largest of the keys so far; all threads
  auto compact = [&]() {
    __syncthreads();
    const int c = count, n = power_of_two(c, 128);
    for (int i = c + tid; i < n; i += TK_THREADS) key[i] = 0;
    sort_keys(key, n);
    if (c >= K) {
      bound = key[K - 1];
      bound_x = of_order((uint32_t)(bound >> 32));
    }
    __syncthreads();
    if (tid == 0) count = c < K ? c : K;
    __syncthreads();
  };
  // a tile's keys: all at once, or, where they do not fit, piece by piece
  auto take_tile = [&](auto edge, const u32x4 (&w)[TK_TILE], int i) {
    const int before = count;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK_TILE; ++k) take(edge, w[k], i + k * TK_THREADS);
    __syncthreads();
    if (count > TK_CAP) {
      __syncthreads();
      if (tid == 0) count = before;
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < TK_TILE; ++k) {
        if (count > TK_CAP - TK_THREADS * N) compact();
        __syncthreads();
        take(edge, k == 0 ? w[0] : k == 1 ? w[1] : k == 2 ? w[2] : w[3], i + k * TK_THREADS);
        __syncthreads();
      }
    } else if (count > TK_SOFT && count > 4 * K) {
      compact();
    }
  };

  if (tid == 0) count = 0;
  // the first stretch's sum, and the bound from its groups' maxima
  const int mid = lo + TK_FIRST * TK_THREADS < hi ? lo + TK_FIRST * TK_THREADS : hi;
  const int group = K <= TK_THREADS / 4 ? TK_FIRST : K <= TK_THREADS ? TK_FIRST / 4 : 1;  // pieces of one thread
  for (int k = tid; k < TK_FIRST / group * TK_THREADS; k += TK_THREADS) key[k] = 0;
  {
    float gm = TK_NEG_INF;
    int done = 0;
    tiles(lo, mid, [&](auto edge, const u32x4 (&w)[TK_TILE], int i) {
      float most[TK_TILE];
      add(edge, w, i, most);
#pragma unroll
      for (int k = 0; k < TK_TILE; ++k) {
        gm = fmaxf(gm, most[k]);
        ++done;
        // a group of no logits is one of -inf: any logit reaches that
        if (done % group == 0) {
          key[(done / group - 1) * TK_THREADS + tid] = (uint64_t)order_of(gm) << 32;
          gm = TK_NEG_INF;
        }
      }
    });
    if (done % group != 0) key[done / group * TK_THREADS + tid] = (uint64_t)order_of(gm) << 32;
  }
  sort_keys(key, TK_FIRST / group * TK_THREADS);
  if (key[K - 1] != 0) {
    bound = key[K - 1] - 1;
    bound_x = of_order((uint32_t)(key[K - 1] >> 32));
  }
  __syncthreads();
  tiles(lo, mid, take_tile);
  tiles(mid, hi, [&](auto edge, const u32x4 (&w)[TK_TILE], int i) {
    float most[TK_TILE];
    add(edge, w, i, most);
    take_tile(edge, w, i);
  });
  compact();

  // the sums: lanes by exchanges, then the waves
#pragma unroll
  for (int d = 32; d; d >>= 1) fold_sum(top, sum, __shfl_xor(top, d), __shfl_xor(sum, d), p.c);
  if ((tid & 63) == 0) wave_sums[tid >> 6] = float2{top, sum};
  __syncthreads();
  if (tid == 0)
#pragma unroll
    for (int k = 1; k < TK_THREADS / 64; ++k) fold_sum(top, sum, wave_sums[k].x, wave_sums[k].y, p.c);
  if (p.segments == 1) {
    for (int k = tid; k < K; k += TK_THREADS) put<T>(p, row, k, key[k]);
    if (tid == 0) p.lse[row] = lse_of(top, sum, p.temperature);
  } else {
    for (int k = tid; k < p.lists_K; k += TK_THREADS) p.lists[g * p.lists_K + k] = k < count ? key[k] : 0;
    if (tid == 0) p.sums[g] = float2{top, sum};
  }
}

// Merges a row's lists.
template <typename T>
__global__ __launch_bounds__(TK_THREADS) void topk_merge_kernel(TopkPart p) {
  __shared__ uint64_t key[TK_CAP];
  const int64_t row = group_number();
  if (row >= p.M) return;
  const int tid = threadIdx.x, L = p.lists_K;
  int lists = power_of_two(p.segments, 2);
  for (int i = tid; i < lists * L; i += TK_THREADS)
    key[i] = i < p.segments * L ? p.lists[row * p.segments * L + i] : 0;
  __syncthreads();
  for (; lists > 1; lists >>= 1) {
    // list l of the next round from lists l and l + lists / 2
    const int n = lists / 2 * L;
    for (int i = tid; i < n; i += TK_THREADS) {
      const uint64_t a = key[i], b = key[n + (i | (L - 1)) - (i & (L - 1))];
      if (a < b) key[i] = b;
    }
    __syncthreads();
    for (int j = L >> 1; j; j >>= 1) {
      for (int q = tid; q < n / 2; q += TK_THREADS) {
        const int i = ((q & ~(j - 1)) << 1) | (q & (j - 1));
        const uint64_t a = key[i], b = key[i | j];
        if (a < b) {
          key[i] = b;
          key[i | j] = a;
        }
      }
      __syncthreads();
    }
  }
  for (int k = tid; k < p.K; k += TK_THREADS) put<T>(p, row, k, key[k]);
  if (tid == 0) {
    float m = TK_NEG_INF, s = 0.0f;
    for (int k = 0; k < p.segments; ++k) {
      const float2 e = p.sums[row * p.segments + k];
      fold_sum(m, s, e.x, e.y, p.c);
    }
    p.lse[row] = lse_of(m, s, p.temperature);
  }
}

// Segments of a row: enough for four work-groups a CU, of at least two pieces
// a thread (a segment costs a sort however short it is), and no more lists than
// the merge holds.
struct TopkPlan {
  int segments, lists_K;
  int64_t lists, sums, bytes;
};
TopkPlan topk_plan(int64_t M, int64_t V, int64_t K, int size) {
  TopkPlan p;
  p.lists_K = 1;
  while (p.lists_K < K) p.lists_K *= 2;
  int64_t s = M > 0 ? 1024 / M : 1;
  const int64_t most = V * size / 16 / (2 * TK_THREADS), fit = TK_CAP / p.lists_K;
  if (s > most) s = most;
  if (s > fit) s = fit;
  if (s > 64) s = 64;
  p.segments = (int)(s > 1 ? s : 1);
  p.lists = 0;
  p.sums = p.segments > 1 ? 8 * M * p.segments * p.lists_K : 0;
  p.bytes = p.sums + (p.segments > 1 ? 8 * M * p.segments : 0);
  return p;
}

template <typename T>
hipError_t topk(const TopkArgs &c, hipStream_t s) {
  const TopkPlan pl = topk_plan(c.M, c.V, c.K, sizeof(T));
  uint8_t *const ws = static_cast<uint8_t *>(c.workspace);
  const TopkPart p{static_cast<const uint8_t *>(c.logits), c.M, c.V, c.ld * (int64_t)sizeof(T), (int)c.K, pl.lists_K,
                   pl.segments, (float)(1.4426950408889634 / (double)c.temperature), c.temperature, c.values, c.ids, c.lse,
                   reinterpret_cast<uint64_t *>(ws + pl.lists), reinterpret_cast<float2 *>(ws + pl.sums)};
  hipError_t e = launch_kernel(topk_part_kernel<T>, numbered_grid(c.M * pl.segments), dim3(TK_THREADS), s, p);
  if (e == hipSuccess && pl.segments > 1)
    e = launch_kernel(topk_merge_kernel<T>, numbered_grid(c.M), dim3(TK_THREADS), s, p);
  return e;
}

}  // namespace

// Whatever the logits' type: fp32 rows are cut into the most segments.
int64_t topk_bytes(int64_t M, int64_t V, int64_t K) { return topk_plan(M, V, K, 4).bytes; }

hipError_t launch_topk(const TopkArgs &c, hipStream_t s) {
  return c.logits_type == OUT_F32    ? topk<float>(c, s)
         : c.logits_type == OUT_BF16 ? topk<__bf16>(c, s)
                                     : topk<_Float16>(c, s);
}

}  // namespace lmhead
