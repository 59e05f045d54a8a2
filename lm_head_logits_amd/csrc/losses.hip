// losses.hip -- losses of the head's logits beyond the cross entropy against
// tokens (xent.hip): the divergence from a teacher's top logits, the clipped
// policy loss with a KL term, the logistic loss of preferred pairs; and their
// gradients.
//
//   t[m, v] = (alpha (hidden[m, :] . W[v, :]) + bias[v]) / T
//   lse[m] = log sum_v e^t[m, v],  q = e^(t - lse)
//   distill      p_k = e^(s_k / T - n) over the teacher's entries present, n their
//                log-sum-exp or the teacher's own
//                loss[m] = sum_k p_k (log p_k - log q[id_k])
//                G[m, v] = g_m (P q[v] - sum_k p_k [v = id_k]),  P = sum_k p_k
//   token losses logp[m] = t[m, y_m] - lse[m], c[m] = d loss / d logp[m],
//                G[m, v] = g c_m ([v = y_m] - q[v])
//   policy       r = e^(logp - old), d = ref - logp
//                loss[m] = -min(r A, clip(r) A) + kl (e^d - d - 1)
//                c = -r A [r A <= clip(r) A] + kl (1 - e^d)
//   preference   S = sum or mean of logp over a sequence,
//                z = beta ((S_w - ref_w) - (S_l - ref_l)) - margin
//                loss = -(1 - e) log sigma(z) - e log sigma(-z)
//   grad_hidden = alpha / T G W,  grad_W = alpha / T G^T hidden,  grad_bias = 1 / T sum_m G
//
// Forward: one matrix product whose epilogue keeps, per row and 256-column
// tile, the largest t and the sum of exponentials, and the t that the loss
// asks for (the target's, or the teacher's entries'); a second kernel folds a
// row's tiles and makes its loss and c. Backward: the pieces of xent.hip; G of a
// piece either by the product again or, where the forward pass kept t (fp32),
// from memory.
//
// 1 / T: alpha / T and a copy of the bias divided by T go into the products.
//
// Bound by the matrix pipes (mma256.hpp) but for few rows, where the weight's
// bytes bind, and short products (H = 2048, some hundred rows), whose tiles'
// epilogues show. 4096 rows, H = 4096, V = 128256, 64 teacher's logits a row: forward
// 3.17-3.24 ms (0.13-0.28 of it t's stores), per piece of 32256 columns G from t 0.144 ms
// (800 MB at 5.5 TB/s), G W 0.68-0.73 ms (1.46-1.57 PFLOP/s), G^T hidden 0.77-0.81
// (1.31-1.38); 9.7-9.95 ms in all, 12.5 with t made again.
//
// Roundings: t, the statistics, probabilities, coefficients and grad_bias are
// fp32, sums over a sequence and pairs' margins fp64. G is rounded to the inputs'
// 16-bit type, scaled (loss_coef_kernel), but for the targets' entries in bf16
// (targets_apart), with which grad_W's rows of those tokens are rounded a second time.
#include "losses_launch.hpp"
#include "xent_core.hpp"

namespace lmhead {

namespace {

constexpr int32_t NO_ID = 0x7FFFFFFF;

// Rows that are not trained on are left out of the work. With more than
// LR_DIRECT rows, one row tile, the others' hidden rows are copied one behind
// the other and their number stays on the device, where every kernel reads it;
// with fewer nothing would be saved by it. (Their rows are then copied for the
// backward pass by the kernel that makes the rows' losses, with zeros in those
// left out: what stands there does not reach grad_W as 0 times infinity.)
// (4096 rows, H = 4096, two fifths left out: the step 12.0 -> 8.4 ms, of which the
// copies are 0.02.)
constexpr int64_t LR_DIRECT = MM_T;

// What the forward pass leaves for the backward pass, in one buffer.
struct StateLayout {
  int64_t count, rows, inv, hidden, y, lse, coef, own, up, bias, ids, p, tk, t, bytes;
};
int64_t padded(int64_t V) { return ceil_div(V, MM_T) * MM_T; }
StateLayout state_layout(int64_t M, int64_t H, int64_t V, int64_t K, bool keep) {
  StateLayout s;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t b = at;
    at += align256(bytes);
    return b;
  };
  const bool packed = M > LR_DIRECT;
  s.count = take(4);
  s.rows = take(packed ? 4 * M : 0);
  s.inv = take(packed ? 4 * M : 0);
  s.hidden = take(2 * M * H);
  s.y = take(4 * M);
  s.lse = take(4 * M);
  s.coef = take(4 * M);
  s.own = take(4 * M);
  s.up = take(4 * M);
  s.bias = take(4 * V);
  s.ids = take(4 * M * K);
  s.p = take(4 * M * K);
  s.tk = take(4 * M * K);
  s.t = take(keep ? 4 * M * padded(V) : 0);
  s.bytes = at;
  return s;
}
// Rows of the work ("packed") are numbered 0 .. n - 1; without packing they are the call's.
struct State {
  int32_t *count;  // n; nullptr without packing
  int32_t *rows;   // [n] the call's row; nullptr
  int32_t *inv;    // [M] the packed row, -1 where left out; nullptr
  uint16_t *hidden;  // [n, H]; without packing zeros in the rows left out
  int32_t *y;      // [n] target column or -1
  float *lse;      // [n]; +inf in rows left out
  float *coef;     // [n] d loss / d logp; distill: P
  float *own;      // [n] G's entry of the row that weighs most, of an upstream gradient of 1: the
                   // target's, coef (1 - q), or of the teacher's the largest, P q - p
  int32_t *up;     // [n] which element of the upstream gradient is the row's
  float *bias;     // [V] bias / T, where T != 1
  int32_t *ids;    // [M, K] the teacher's tokens in ascending order, NO_ID behind the last
  float *p, *tk;   // [M, K] their probabilities and the head's t
  float *t;        // [n, V in whole tiles] every t (-inf behind the last), where they are kept
};
State state_at(void *base, const StateLayout &l, int64_t M) {
  uint8_t *const b = static_cast<uint8_t *>(base);
  const bool packed = M > LR_DIRECT;
  auto ints = [&](int64_t at) { return packed ? reinterpret_cast<int32_t *>(b + at) : nullptr; };
  return State{ints(l.count), ints(l.rows), ints(l.inv), reinterpret_cast<uint16_t *>(b + l.hidden),
               reinterpret_cast<int32_t *>(b + l.y),    reinterpret_cast<float *>(b + l.lse),
               reinterpret_cast<float *>(b + l.coef),   reinterpret_cast<float *>(b + l.own),
               reinterpret_cast<int32_t *>(b + l.up),
               reinterpret_cast<float *>(b + l.bias),   reinterpret_cast<int32_t *>(b + l.ids),
               reinterpret_cast<float *>(b + l.p),      reinterpret_cast<float *>(b + l.tk),
               reinterpret_cast<float *>(b + l.t)};
}

constexpr int64_t LR_CHUNK = 4096;  // rows counted at a time
struct ForwardLayout {
  int64_t part, tlogit, rowlogp, ent, P, ptr, chunks, state, bytes;
};
ForwardLayout forward_layout(int64_t M, int64_t H, int64_t V, int64_t K, bool with_state) {
  ForwardLayout f;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t b = at;
    at += align256(bytes);
    return b;
  };
  const int64_t nvt = ceil_div(V, MM_T);
  f.part = take(8 * M * nvt);
  f.tlogit = take(4 * M);
  f.rowlogp = take(4 * M);
  f.ent = take(K ? 4 * M : 0);
  f.P = take(K ? 4 * M : 0);
  f.chunks = take(4 * ceil_div(M, LR_CHUNK));
  f.ptr = take(K ? 2 * M * (nvt + 1) : 0);
  f.state = take(with_state ? 0 : state_layout(M, H, V, K, false).bytes);
  f.bytes = at;
  return f;
}

// ---------------------------------------------------------------------------
// Before the product
// ---------------------------------------------------------------------------

__global__ __launch_bounds__(256) void loss_bias_scale_kernel(const float *__restrict__ bias, int64_t V, float T,
                                                              float *__restrict__ out) {
  const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (v < V) out[v] = __fdiv_rn(bias[v], T);
}

// A row of the teacher's entries, one wave each: their probabilities, and the
// entries in the order of their tokens (by counting for each the smaller pairs
// (token, place)), with the first entry of every 256-column tile. An entry
// whose token is no column of the call, or whose logit is -inf, is absent.
constexpr int DP_WAVES = 4;
struct DistillPrep {
  const void *ids;
  int ids64;
  int64_t M, V, K;
  const void *logits;
  OutType type;
  const float *teacher_lse;
  float T;
  int32_t *sid;    // [M, K]
  float *sp;       // [M, K]
  uint16_t *ptr;   // [M, nvt + 1] entries before each tile; nullptr where t is kept
  float *ent;      // [M] sum p log p
  float *P;        // [M] sum p
};
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = __fadd_rn(x, __shfl_xor(x, d));
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const float o = __shfl_xor(x, d);
    x = x != x || o != o ? __builtin_nanf("") : fmaxf(x, o);
  }
  return x;
}
// E: entries a lane, at least K / 64
template <int E>
__global__ __launch_bounds__(64 * DP_WAVES) void distill_prep_kernel(DistillPrep c) {
  __shared__ int32_t id_sh[DP_WAVES][64 * E], sorted_sh[DP_WAVES][64 * E];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = group_number() * DP_WAVES + wave;
  if (m >= c.M) return;  // waves work alone
  int32_t *const id_w = id_sh[wave], *const sorted = sorted_sh[wave];
  const int K = (int)c.K;
  int32_t id[E];
  float v[E];
  float mx = NEG_INF;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int k = lane + 64 * e;
    id[e] = NO_ID;
    v[e] = NEG_INF;
    if (k < K) {
      const int64_t at = m * c.K + k;
      const int64_t i = c.ids64 ? static_cast<const int64_t *>(c.ids)[at] : (int64_t)static_cast<const int32_t *>(c.ids)[at];
      const float s = c.type == OUT_F32    ? static_cast<const float *>(c.logits)[at]
                      : c.type == OUT_BF16 ? (float)static_cast<const __bf16 *>(c.logits)[at]
                                           : (float)static_cast<const _Float16 *>(c.logits)[at];
      if (i >= 0 && i < c.V && s != NEG_INF) {
        id[e] = (int32_t)i;
        v[e] = s;
        mx = mx != mx || v[e] != v[e] ? __builtin_nanf("") : fmaxf(mx, v[e]);
      }
      id_w[k] = id[e];
    }
  }
  mx = wave_max(mx);
  // From here on (s - largest) / T: s / T itself may be past fp32's range (the type's
  // lowest value at T < 1). Where the teacher's lse is given, s / T.
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = __fdiv_rn(c.teacher_lse != nullptr ? v[e] : __fsub_rn(v[e], mx), c.T);
  float s = 0.0f;
  const float lse_t = c.teacher_lse != nullptr ? c.teacher_lse[m] : 0.0f;
  if (c.teacher_lse == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (id[e] != NO_ID) s = __fadd_rn(s, expf(v[e]));
    s = wave_sum(s);
  }
  const float ls = logf(s);
  float p[E], ent = 0.0f, P = 0.0f;
  int count = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    p[e] = 0.0f;
    if (id[e] != NO_ID) {
      const float lp = c.teacher_lse != nullptr ? __fsub_rn(v[e], lse_t) : __fsub_rn(v[e], ls);
      p[e] = expf(lp);
      if (p[e] != 0.0f) ent = __fadd_rn(ent, __fmul_rn(p[e], lp));
      P = __fadd_rn(P, p[e]);
      ++count;
    }
  }
  ent = wave_sum(ent);
  P = wave_sum(P);
#pragma unroll
  for (int d = 32; d; d >>= 1) count += __shfl_xor(count, d);
  sched_fence();  // other lanes' values: LDS keeps a wave's order
  int rank[E];
#pragma unroll
  for (int e = 0; e < E; ++e) rank[e] = 0;
  for (int j = 0; j < K; ++j) {
    const int32_t other = id_w[j];
#pragma unroll
    for (int e = 0; e < E; ++e) rank[e] += other < id[e] || (other == id[e] && j < lane + 64 * e) ? 1 : 0;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (lane + 64 * e < K) {
      sorted[rank[e]] = id[e];
      c.sid[m * c.K + rank[e]] = id[e];
      c.sp[m * c.K + rank[e]] = p[e];
    }
  sched_fence();
  const int64_t nvt = (c.V + MM_T - 1) / MM_T;
  for (int64_t t = lane; c.ptr != nullptr && t <= nvt; t += 64) {
    int lo = 0, hi = count;  // the first of the present entries at or past the tile's first column
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (sorted[mid] < t * MM_T) lo = mid + 1;
      else hi = mid;
    }
    c.ptr[m * (nvt + 1) + t] = (uint16_t)lo;
  }
  if (lane == 0) {
    c.ent[m] = ent;
    c.P[m] = c.teacher_lse == nullptr && count > 0 ? (P != P ? P : 1.0f) : P;
  }
}

// Which rows are worked on: those of a teacher with entries; those with a
// target, within the sequences where there are any.
struct Select {
  const float *P;      // distill: [M] mass of the entries
  const void *target;  // else
  int target64;
  int64_t ignore, M, V;
  const void *starts;  // preference: [bounds]
  int starts64;
  int64_t last;        // the last bound's place
  __device__ __forceinline__ int64_t bound(int64_t i) const {
    return starts64 ? static_cast<const int64_t *>(starts)[i] : (int64_t)static_cast<const int32_t *>(starts)[i];
  }
  // (column of the target, or 0 where a row has none of its own; -1: left out)
  __device__ __forceinline__ int64_t column(int64_t m, int64_t lo, int64_t hi) const {
    if (P != nullptr) return P[m] == 0.0f ? -1 : 0;
    return m >= lo && m < hi ? target_of(target, target64, m, ignore, V) : -1;
  }
};
constexpr int LR_THREADS = 256, LR_ROWS = 4;
__device__ __forceinline__ int block_sum(int x, int (&sh)[LR_THREADS / 64]) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
  __syncthreads();
  x = sh[0] + sh[1] + sh[2] + sh[3];
  __syncthreads();
  return x;
}
// Rows worked on in each chunk of LR_CHUNK (only where there are several).
__global__ __launch_bounds__(LR_THREADS) void loss_count_kernel(Select c, int32_t *chunks) {
  __shared__ int sh[LR_THREADS / 64];
  const int64_t lo = c.starts != nullptr ? c.bound(0) : 0, hi = c.starts != nullptr ? c.bound(c.last) : c.M;
  const int64_t m0 = (int64_t)blockIdx.x * LR_CHUNK;
  int n = 0;
#pragma unroll 8
  for (int64_t m = m0 + threadIdx.x; m < m0 + LR_CHUNK && m < c.M; m += LR_THREADS) n += c.column(m, lo, hi) >= 0 ? 1 : 0;
  n = block_sum(n, sh);
  if (threadIdx.x == 0) chunks[blockIdx.x] = n;
}
// Four rows a work-group, which counts the rows before them by itself; copies
// the hidden rows that are worked on, clears the outputs of the others. (4096 rows,
// H = 4096: 17.6 us; sixteen a work-group, whose copies then follow each other: 21.)
struct Gather {
  Select sel;
  const int32_t *chunks;
  const uint16_t *hidden;
  int64_t H;
  State st;
  float *zero0, *zero1;  // [M] outputs of rows left out, or nullptr
};
__global__ __launch_bounds__(LR_THREADS) void loss_gather_kernel(Gather c) {
  __shared__ int sh[LR_THREADS / 64];
  __shared__ int32_t list[LR_ROWS];
  const Select &s = c.sel;
  const int tid = threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.x * LR_ROWS, chunk = r0 / LR_CHUNK;
  const int64_t lo = s.starts != nullptr ? s.bound(0) : 0, hi = s.starts != nullptr ? s.bound(s.last) : s.M;
  int n = 0;
  for (int64_t k = tid; k < chunk; k += LR_THREADS) n += c.chunks[k];
#pragma unroll 8
  for (int64_t m = chunk * LR_CHUNK + tid; m < r0; m += LR_THREADS) n += s.column(m, lo, hi) >= 0 ? 1 : 0;
  const int before = block_sum(n, sh);
  if (tid < 64) {  // one wave: the ballot is its own
    const int64_t m = r0 + tid;
    const bool mine = tid < LR_ROWS && m < s.M;
    const int64_t y = mine ? s.column(m, lo, hi) : -1;
    const uint64_t set = __ballot(y >= 0);
    const int place = __popcll(set & ((1ull << tid) - 1)), kept = __popcll(set);
    if (mine) {
      c.st.inv[m] = y >= 0 ? before + place : -1;
      if (y >= 0) {
        list[place] = (int32_t)m;
        c.st.rows[before + place] = (int32_t)m;
        c.st.y[before + place] = s.P != nullptr ? -1 : (int32_t)y;
      } else {
        if (c.zero0 != nullptr) c.zero0[m] = 0.0f;
        if (c.zero1 != nullptr) c.zero1[m] = 0.0f;
      }
    }
    if (tid == 0) {
      sh[0] = kept;
      if (r0 + LR_ROWS >= s.M) *c.st.count = before + kept;
    }
  }
  __syncthreads();
  const uint32_t per = (uint32_t)(c.H / 8), total = (uint32_t)sh[0] * per;  // 16-byte pieces
  const u32x4 *const from = reinterpret_cast<const u32x4 *>(c.hidden);
  u32x4 *const to = reinterpret_cast<u32x4 *>(c.st.hidden) + (int64_t)before * per;
  for (uint32_t e0 = tid; e0 < total; e0 += 4 * LR_THREADS) {
    u32x4 v[4];
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t e = e0 + k * LR_THREADS < total ? e0 + k * LR_THREADS : e0, r = e / per;
      v[k] = from[(int64_t)list[r] * per + (e - r * per)];
    }
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      if (e0 + k * LR_THREADS < total) to[e0 + k * LR_THREADS] = v[k];
  }
}

// ---------------------------------------------------------------------------
// The product's epilogue
// ---------------------------------------------------------------------------

struct LossFwdArgs {
  const uint8_t *hidden, *W;
  int64_t M, H, V;
  float alpha;
  const float *bias;
  const int32_t *count;  // packed rows (State): their number, in the place of M
  const int32_t *rows;
  const int32_t *y;      // ... and their targets
  const void *target;    // else
  int target64;
  int64_t ignore;
  float2 *part;        // [vocabulary tile][M] {largest t, sum of exp(t - largest)}
  float *tlogit;       // neither: [M] t at the target (rows with one)
  const int32_t *sid;  // PICK: the teacher's entries (distill_prep_kernel)
  const uint16_t *ptr;
  float *tk;           // ... [M, K] t at them
  int64_t K;
  float *t;            // KEEP: [M, padded V]
  __device__ __forceinline__ void set_rows() {
    if (count != nullptr) M = mm_uni(*count);
  }
  __device__ __forceinline__ int64_t row(int64_t m) const { return rows != nullptr ? rows[m] : m; }
  __device__ __forceinline__ int32_t column(int64_t m) const {
    return y != nullptr ? y[m] : (int32_t)target_of(target, target64, m, ignore, V);
  }
};

// PICK: t at the rows' entries in the tile instead of at one target. Through
// LDS, 32 rows at a time: all 256 columns of the rows are written, then 16
// threads a row take that row's entries from it. Groups of rows without an
// entry are left out. (4096 rows with 64 entries, H = 4096, V = 128256: 0.16 ms of
// 3.08.)
//
// KEEP: t of the whole tile to memory, for the backward pass (0.13-0.28 ms). The
// kernels that make the rows' losses read from it what else is picked here: with
// those entries picked here all the same a forward pass took 0.27 ms longer than
// one with a target a row, so 0.03 ms.
template <int ET, bool PICK, bool KEEP>
struct LossStats {
  LossFwdArgs p;
  u32x4 *epi;
  int64_t nmt, nvt;

  __device__ __forceinline__ int64_t tiles() const { return nmt * nvt; }
  __device__ __forceinline__ MmJob job(int32_t t) const {
    int64_t mt, vt;
    mm_tile_at(t, nmt, nvt, mt, vt);
    return logits_job(p.hidden, p.W, p.M, p.H, p.V, mt * MM_T, vt * MM_T);
  }
  __device__ __forceinline__ void epilogue(MmTile<ET> &tile, int32_t t) const {
    int64_t mt, vt;
    mm_tile_at(t, nmt, nvt, mt, vt);
    const int64_t m0 = mt * MM_T, n0 = vt * MM_T;
    const LanePlace at;
    float bias[2][2][4];
    column_bias<ET>(p.bias, p.V, n0, at, 0, bias[0]);
    column_bias<ET>(p.bias, p.V, n0, at, 1, bias[1]);
    float2 *const stat = reinterpret_cast<float2 *>(epi);  // [4][256]
    uint32_t *const groups = reinterpret_cast<uint32_t *>(epi) + 4 * MM_T * 2;
    if (PICK && threadIdx.x == 0) *groups = 0;
    const int rows = (int)(p.M - m0 < MM_T ? p.M - m0 : MM_T);
    const uint32_t ldt = (uint32_t)(nvt * MM_T);
    rsrc_t rs;
    if constexpr (KEEP) rs = make_rsrc(p.t + m0 * ldt + n0, ((rows - 1) * ldt + MM_T) * 4);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = MmTile<ET>::row(at.wm, at.li, x, i);
        const int64_t m = m0 + row;
        float mx = NEG_INF;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float v = __fmaf_rn(p.alpha, tile.c[x][y][i][j][q], bias[y][j][q]);
              tile.c[x][y][i][j][q] = v;
              mx = fmaxf(mx, v);
            }
        if constexpr (KEEP) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              __builtin_amdgcn_raw_buffer_store_b128(
                  __builtin_bit_cast(u32x4, tile.c[x][y][i][j]), rs,
                  row < rows ? (uint32_t)((row * ldt + MmTile<ET>::col(at.wn, at.lg, y, j)) * 4) : OFF_NONE, 0, LOAD_DEFAULT);
        }
        if constexpr (!PICK && !KEEP) {
          const int32_t yt = m < p.M ? p.column(m) - (int32_t)n0 : -1;
          if (has_column<ET>(at, 0, yt) || has_column<ET>(at, 1, yt)) {
            float v = 0.0f;
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  if (yt == MmTile<ET>::col(at.wn, at.lg, y, j) + q) v = tile.c[x][y][i][j][q];
            p.tlogit[m] = v;
          }
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        // a tile of only -inf sums nothing: its terms are taken against 0
        const float mz = mx == NEG_INF ? 0.0f : mx;
        float s = 0.0f;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) s = __fadd_rn(s, exp_diff(tile.c[x][y][i][j][q], mz));
        s = __fadd_rn(s, __shfl_xor(s, 16));
        s = __fadd_rn(s, __shfl_xor(s, 32));
        if (at.lg == 0) stat[at.wn * MM_T + row] = float2{mx, s};
      }
    lds_barrier();
    const int tid = mm_tid();
    if (tid < MM_T && m0 + tid < p.M) {
      float mx = NEG_INF, s = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, stat[w * MM_T + tid].x);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 e = stat[w * MM_T + tid];
        if (e.y != 0.0f) s = __fadd_rn(s, __fmul_rn(e.y, exp_diff(e.x, mx)));
      }
      p.part[vt * p.M + m0 + tid] = float2{mx, s};
    }
    if constexpr (PICK) {
      // thread (row tid / 16 of a group, entry tid % 16): the entries of the
      // row of each of the eight groups
      const int pr = tid >> 4, pe = tid & 15;
      // (every load for all eight groups before the first is used)
      uint32_t range[8], some = 0;
      int32_t at_row[8], id[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t m = m0 + 128 * (k >> 2) + 64 * (pr >> 4) + 16 * (k & 3) + (pr & 15);
        at_row[k] = m < p.M ? (int32_t)p.row(m) : -1;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint16_t *const r = p.ptr + (at_row[k] < 0 ? 0 : at_row[k]) * (nvt + 1) + vt;
        range[k] = at_row[k] < 0 ? 0u : r[0] | (uint32_t)r[1] << 16;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t e = (range[k] & 0xFFFF) + pe, end = range[k] >> 16;
        id[k] = e < end ? p.sid[at_row[k] * p.K + e] : 0;
        if ((range[k] & 0xFFFF) < end) some |= 1u << k;
      }
      if (some != 0 && pe == 0) atomicOr(groups, some);
      lds_barrier();
      const uint32_t mask = mm_uni(*groups);
      lds_barrier();  // the flags are read: their place may be written
      float *const box = reinterpret_cast<float *>(epi);  // [32][256], 16-byte pieces xor-ed with the row
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = x * 4 + i;
          if ((mask >> k & 1) == 0) continue;
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int piece = MmTile<ET>::col(at.wn, at.lg, y, j) >> 2;
              *reinterpret_cast<f32x4 *>(box + (at.wm * 16 + at.li) * MM_T + 4 * (piece ^ at.li)) = tile.c[x][y][i][j];
            }
          lds_barrier();
          int32_t col = id[k];
          for (uint32_t e = (range[k] & 0xFFFF) + pe; e < range[k] >> 16;) {
            const uint32_t c = (uint32_t)(col - (int32_t)n0) & (MM_T - 1);
            p.tk[at_row[k] * p.K + e] = box[pr * MM_T + 4 * ((c >> 2) ^ (pr & 15)) + (c & 3)];
            e += 16;
            if (e < range[k] >> 16) col = p.sid[at_row[k] * p.K + e];
          }
          lds_barrier();
        }
    }
    // the next tile's epilogue is barriers away
  }
};

template <int ET, bool PICK, bool KEEP>
__global__ __launch_bounds__(MM_THREADS, 1) void loss_stats_kernel(LossFwdArgs p) {
  MM_SHARED();
  MM_EPI_SHARED();
  p.set_rows();
  const LossStats<ET, PICK, KEEP> prob{p, mm_epi, (p.M + MM_T - 1) / MM_T, (p.V + MM_T - 1) / MM_T};
  mm_run<ET, false, false>(prob, mm_buf);
}

// ---------------------------------------------------------------------------
// The rows' losses
// ---------------------------------------------------------------------------

// Folds the tiles of row m, as xent.hip does: 16 rows per work-group, 64
// threads per row, each thread tiles s, s + 64, ... in ascending order, then the
// 64 in eights and the eights, in order. Every thread of the row returns with
// the result: the largest t and the log of the sum of exp(t - largest).
__device__ __forceinline__ float2 fold_row(const float2 *part, int64_t M, int64_t nvt, int64_t m, bool ok,
                                           float2 (&sh)[XC_SLICES][XC_ROWS]) {
  const int r = threadIdx.x % XC_ROWS, sl = threadIdx.x / XC_ROWS;
  float mx = NEG_INF, s = 0.0f;
  if (ok) {
    for (int64_t t0 = sl; t0 < nvt; t0 += 8 * XC_SLICES) {
      float2 e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t t = t0 + k * XC_SLICES;
        e[k] = t < nvt ? part[t * M + m] : float2{NEG_INF, 0.0f};
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) fold_stat(mx, s, e[k]);
    }
  }
  sh[sl][r] = float2{mx, s};
  __syncthreads();
  if (sl < 8) {
    mx = NEG_INF;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) fold_stat(mx, s, sh[8 * sl + k][r]);
  }
  __syncthreads();
  if (sl < 8) sh[sl][r] = float2{mx, s};
  __syncthreads();
  mx = NEG_INF;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) fold_stat(mx, s, sh[k][r]);
  __syncthreads();
  return float2{mx, s};
}
// every logit -inf: log-sum-exp -inf
__device__ __forceinline__ float row_lse(float2 f, float ls) { return f.y == 0.0f ? NEG_INF : __fadd_rn(f.x, ls); }
// log q of a column from the largest logit, not from lse as rounded: that of a
// token that is nearly certain is far below half a step of its lse
__device__ __forceinline__ float log_q(float t, float2 f, float ls) {
  return t == NEG_INF ? NEG_INF : __fsub_rn(__fsub_rn(t, f.x), ls);
}

// What the kernels that make the rows' losses share.
struct RowsArgs {
  const float2 *part;
  int64_t M, nvt;
  State st;
  Select sel;               // without packing
  const uint16_t *hidden;   // ... and [M, H] to be copied, or nullptr
  int64_t H;
  __device__ __forceinline__ int64_t column(int64_t m) const {
    return sel.column(m, sel.starts != nullptr ? sel.bound(0) : 0, sel.starts != nullptr ? sel.bound(sel.last) : M);
  }
  // the work-group's 16 rows, a wave each
  __device__ __forceinline__ void copy(int64_t m0) const {
    static_assert(XC_SLICES * XC_ROWS == 64 * XC_ROWS);
    const int64_t m = m0 + threadIdx.x / 64, per = H / 8;
    if (hidden == nullptr || m >= M) return;
    const bool worked_on = column(m) >= 0;
    const u32x4 *const from = reinterpret_cast<const u32x4 *>(hidden) + m * per;
    u32x4 *const to = reinterpret_cast<u32x4 *>(st.hidden) + m * per;
#pragma unroll 4
    for (int64_t i = threadIdx.x % 64; i < per; i += 64) to[i] = worked_on ? from[i] : u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ int64_t rows() const { return st.count != nullptr ? *st.count : M; }
  __device__ __forceinline__ int64_t row(int64_t m) const { return st.rows != nullptr ? st.rows[m] : m; }
  int64_t ldt;              // of the kept t; 0 where it is not
};
struct DistillRows {
  RowsArgs r;
  int64_t K;
  const float *ent, *P;
  float *loss;
};
__global__ __launch_bounds__(XC_ROWS * XC_SLICES) void distill_rows_kernel(DistillRows c) {
  __shared__ float2 sh[XC_SLICES][XC_ROWS];
  const int r = threadIdx.x % XC_ROWS, sl = threadIdx.x / XC_ROWS;
  const int64_t m = (int64_t)blockIdx.x * XC_ROWS + r, n = c.r.rows();
  if (m - r >= n) return;  // the whole work-group
  c.r.copy(m - r);
  const int64_t row = m < n ? c.r.row(m) : 0;
  const float P = m < n ? c.P[row] : 0.0f;
  if (c.r.ldt != 0 && m < n) {
#pragma unroll 1
    for (int64_t k = sl; k < c.K; k += XC_SLICES) {  // the thread's own, below
      const int32_t id = c.r.st.ids[row * c.K + k];
      if (id != NO_ID) c.r.st.tk[row * c.K + k] = c.r.st.t[m * c.r.ldt + id];
    }
  }
  const float2 f = fold_row(c.r.part, n, c.r.nvt, m, m < n, sh);
  const float ls = logf(f.y);
  float sum = 0.0f, own = 0.0f;
  if (m < n)
    for (int64_t k = sl; k < c.K; k += XC_SLICES) {
      const float p = c.r.st.p[row * c.K + k];
      if (p != 0.0f) {
        const float lq = log_q(c.r.st.tk[row * c.K + k], f, ls), e = __fsub_rn(__fmul_rn(P, expf(lq)), p);
        sum = __fadd_rn(sum, __fmul_rn(p, lq));
        own = fabsf(e) > fabsf(own) ? e : own;
      }
    }
  sh[sl][r] = float2{sum, own};
  __syncthreads();
  if (sl != 0 || m >= n) return;
  const int slices = c.K < XC_SLICES ? (int)c.K : XC_SLICES;  // the others have no entry
#pragma unroll 8
  for (int k = 1; k < slices; ++k) {
    const float2 e = sh[k][r];
    sum = __fadd_rn(sum, e.x);
    own = fabsf(e.y) > fabsf(own) ? e.y : own;
  }
  c.r.st.lse[m] = P == 0.0f ? __builtin_inff() : row_lse(f, ls);
  c.r.st.y[m] = -1;
  c.r.st.up[m] = (int32_t)row;
  c.r.st.coef[m] = P;
  c.r.st.own[m] = own;
  c.loss[row] = P == 0.0f ? 0.0f : __fsub_rn(c.ent[row], sum);
}

// coef (1 - q) of a target with that log q
__device__ __forceinline__ float own_share(float coef, float logp) {
  return coef == 0.0f ? 0.0f : __fmul_rn(coef, -expm1f(logp));
}

struct TokenRows {
  RowsArgs r;
  const float *tlogit;
  float *logp;     // [M]
  // policy
  const float *advantage, *old_logp, *ref_logp;
  float low, high, kl;
  float *loss;
};
// The clipped loss and the KL term of one token, and their derivative.
__device__ __forceinline__ void policy_token(const TokenRows &c, int64_t m, float logp, float &loss, float &coef) {
  const float A = c.advantage[m];
  const float r = c.old_logp != nullptr ? expf(__fsub_rn(logp, c.old_logp[m])) : 1.0f;
  const float held = fminf(fmaxf(r, __fsub_rn(1.0f, c.low)), __fadd_rn(1.0f, c.high));
  const float ra = __fmul_rn(r, A), ca = __fmul_rn(held, A);
  loss = coef = 0.0f;
  if (A != 0.0f) {  // else 0, also where the ratio has overflowed
    const bool free = ra <= ca;
    loss = free ? -ra : ra != ra ? ra : -ca;  // NaN of any origin
    coef = free ? -ra : loss != loss ? loss : 0.0f;
  }
  if (c.ref_logp != nullptr && c.kl != 0.0f) {
    const float d = __fsub_rn(c.ref_logp[m], logp), e = expm1f(d);
    loss = __fadd_rn(loss, __fmul_rn(c.kl, d == __builtin_inff() ? d : __fsub_rn(e, d)));
    coef = __fsub_rn(coef, __fmul_rn(c.kl, e));
  }
}
template <bool POLICY>
__global__ __launch_bounds__(XC_ROWS * XC_SLICES) void token_rows_kernel(TokenRows c) {
  __shared__ float2 sh[XC_SLICES][XC_ROWS];
  const int r = threadIdx.x % XC_ROWS, sl = threadIdx.x / XC_ROWS;
  const int64_t m = (int64_t)blockIdx.x * XC_ROWS + r, n = c.r.rows();
  if (m - r >= n) return;  // the whole work-group
  c.r.copy(m - r);
  const bool packed = c.r.st.rows != nullptr;
  int64_t y = -1;
  float t = 0.0f;
  if (sl == 0 && m < n) {
    y = packed ? c.r.st.y[m] : c.r.column(m);
    if (y >= 0) t = c.r.ldt != 0 ? c.r.st.t[m * c.r.ldt + y] : c.tlogit[m];
  }
  const float2 f = fold_row(c.r.part, n, c.r.nvt, m, m < n, sh);
  if (sl != 0 || m >= n) return;
  const float ls = logf(f.y);
  const int64_t row = c.r.row(m);
  const float logp = y >= 0 ? log_q(t, f, ls) : 0.0f;
  c.r.st.lse[m] = y >= 0 ? row_lse(f, ls) : __builtin_inff();
  if (!packed) c.r.st.y[m] = (int32_t)y;
  c.logp[row] = logp;
  float loss = 0.0f, coef = 0.0f;
  if constexpr (POLICY) {
    if (y >= 0) policy_token(c, row, logp, loss, coef);
    c.loss[row] = loss;
    c.r.st.up[m] = (int32_t)row;
  } else {
    c.r.st.up[m] = 0;  // preference_pairs_kernel knows the rows' pairs
  }
  c.r.st.coef[m] = coef;
  c.r.st.own[m] = own_share(coef, logp);
}

// One pair of sequences, one work-group: their sums in 64 bits in a fixed
// order (differences of sums over thousands of tokens are wanted), the loss,
// and the derivative for every row of theirs.
constexpr int PP_THREADS = 256;
struct Pairs {
  const void *starts;
  int starts64;
  int64_t pairs, M, V;
  const void *target;
  int target64;
  int64_t ignore;
  const float *rowlogp, *ref;
  float beta, margin, smoothing;
  int average;
  float *loss, *logp, *coef, *own;
  int32_t *up;
  const int32_t *inv;  // State
};
__global__ __launch_bounds__(PP_THREADS) void preference_pairs_kernel(Pairs c) {
  __shared__ double sh[2][PP_THREADS];
  __shared__ float der[2];
  const int tid = threadIdx.x;
  const int64_t pair = blockIdx.x;
  auto bound = [&](int64_t i) {
    const int64_t b = c.starts64 ? static_cast<const int64_t *>(c.starts)[i] : (int64_t)static_cast<const int32_t *>(c.starts)[i];
    return b < 0 ? (int64_t)0 : b > c.M ? c.M : b;
  };
  double total[2], size[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int64_t q = pair + w * c.pairs, lo = bound(q), hi = bound(q + 1);
    double s = 0.0, n = 0.0;
    for (int64_t m = lo + tid; m < hi; m += PP_THREADS)
      if (target_of(c.target, c.target64, m, c.ignore, c.V) >= 0) {
        s += c.rowlogp[m];
        n += 1.0;
      }
    sh[0][tid] = s;
    sh[1][tid] = n;
    __syncthreads();
    for (int d = PP_THREADS / 2; d; d >>= 1) {
      if (tid < d) {
        sh[0][tid] += sh[0][tid + d];
        sh[1][tid] += sh[1][tid + d];
      }
      __syncthreads();
    }
    total[w] = sh[0][0];
    size[w] = c.average && sh[1][0] > 0.0 ? sh[1][0] : 1.0;
    __syncthreads();
  }
  if (tid == 0) {
    double lead[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      total[w] /= size[w];
      c.logp[pair + w * c.pairs] = (float)total[w];
      lead[w] = total[w] - (c.ref != nullptr ? (double)c.ref[pair + w * c.pairs] : 0.0);
    }
    const double z = (double)c.beta * (lead[0] - lead[1]) - (double)c.margin, e = c.smoothing;
    // -log sigma(z) = max(-z, 0) + log(1 + e^-|z|)
    const double soft = log1p(exp(-fabs(z)));
    // infinite on one side only, where that side has weight
    const double neg = fmax(-z, 0.0) + soft, pos = fmax(z, 0.0) + soft;
    c.loss[pair] = (float)(z != z ? z : (e != 1.0 ? (1.0 - e) * neg : 0.0) + (e != 0.0 ? e * pos : 0.0));
    const double dz = (e - 1.0 / (1.0 + exp(z))) * (double)c.beta;
    der[0] = (float)(dz / size[0]);
    der[1] = (float)(-dz / size[1]);
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int64_t q = pair + w * c.pairs, lo = bound(q), hi = bound(q + 1);
    for (int64_t m = lo + tid; m < hi; m += PP_THREADS)
      if (target_of(c.target, c.target64, m, c.ignore, c.V) >= 0) {
        const int64_t at = c.inv != nullptr ? c.inv[m] : m;
        if (at < 0) continue;  // bounds that do not ascend
        c.coef[at] = der[w];
        c.own[at] = own_share(der[w], c.rowlogp[m]);
        c.up[at] = (int32_t)pair;
      }
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// The rows' coefficients of G, scaled as in xent.hip: by f, at most top / the
// largest finite one. Target losses: a = b = -g c. Distill: a = g P, b = g (the
// factor of the entries), no target. Every work-group finds the scale by itself up to
// LC_ONE rows; with more, one work-group finds it in a launch of its own.
//
// Which f: a row's gradients hang on a few entries of G and on how those happen to
// round. Of LC_TRIES factors over an octave that with the smallest error of the
// entries that weigh most is taken: one a row, its target's (where G has it) or its
// teacher's largest, of LC_SAMPLES rows spread over those worked on. Error of the
// gradients over that of a correctly rounded result, over 130 drawn batches of 50 to
// 4000 rows: 1.01 to 1.42.
// (Distillation's grad_hidden over forty: without the choice 1.09 to 1.51, the worst
// factor 1.36 to 2.2, chosen by all entries of the first 1024 / K rows 1.06 to 1.69, so of
// few rows worse than none, by the largest of each row 1.05 to 1.38, the best factor
// 1.05 to 1.37.)
//
// The splits of G W's K (the piece's columns) that fill the last round of
// work-groups best, at least 256 columns each; chosen much as bwd_plan does, from
// the rows worked on, by one wave. More splits have to fill 10% more: every one is
// a sum of grad_hidden to write and to read again (764 rows, H = 2048, ten splits
// against 32 that fill 6% more: the product 200 us against 247, the sums joined in
// 12 against 42).
// `cap`: row tiles times splits that the sums have room for.
struct SplitPlan {
  int32_t splits;
};
// The columns of a split of a piece of np: those of the shorter, last piece are shorter.
__host__ __device__ __forceinline__ int64_t split_of(int64_t np, int64_t splits) {
  return ((np + splits - 1) / splits + 63) / 64 * 64;
}
// A split more is looked at where there are fewer tiles without it.
constexpr int32_t SPLIT_TILES = 4 * 256;
__device__ __forceinline__ void plan_splits(int32_t n, int32_t H, int32_t vp, int32_t cap, SplitPlan *out) {
  const uint32_t nmt = (n + MM_T - 1) / MM_T, tiles = nmt * ((H + MM_T - 1) / MM_T), cus = 256;
  const uint32_t s = threadIdx.x + 1;
  const bool ok = s == 1 || (s * 256 <= (uint32_t)vp && s * nmt <= (uint32_t)cap && tiles * (s - 1) < SPLIT_TILES);
  const float use = ok && tiles > 0 ? (float)(tiles * s) / (float)((tiles * s + cus - 1) / cus * cus) : 0.0f;
  float best = 0.0f;
  int32_t splits = 1;
#pragma unroll
  for (int k = 0; k < 64; ++k) {
    const float u = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, use), k));
    if (u > best * 1.1f) {
      best = u;
      splits = k + 1;
    }
  }
  if (threadIdx.x == 0) {
    const int32_t k = (int32_t)split_of(vp, splits);
    out->splits = (vp + k - 1) / k;
  }
}

// The targets' entries of G, g c (1 - q), are the largest by far, and their rounding to
// bf16 would be most of the gradients' error (1.2 to 1.4 times that of a correctly rounded
// result; in a frequent token's row of grad_W, a sum of rows of either sign, up to half of
// grad_W's root mean square). They are kept apart: 0 stands there in G, and
// loss_out_kernel adds them in fp32, which leaves 1.00 times, and 2^-7 of an element or of
// the root mean square. (A step of 4096 rows on the decode head, 2367 of them worked on:
// 6265 us against 6240; 126 rows on a small head 50.9 against 51.1, since no scale is
// chosen.) Not for fp16, whose G has three bits more: grad_W's row of a token is rounded
// before they are added to it, and among fp16's least numbers that shows. Nor for a
// teacher's largest entries (error 1.00 to 1.09 times, for 0.6% more time of a large step):
// they are less of their token's row, and that row's two roundings then pass, once in a
// million elements, what one and G's would be.
template <int ET>
constexpr bool targets_apart = ET == ET_BF16;

constexpr int LC_THREADS = 256;
constexpr int64_t LC_ONE = 32768;
constexpr float LC_STEP = 0.95760328f;  // 2^(-1 / 16)
constexpr int LC_TRIES = 16, LC_SAMPLES = 4 * LC_THREADS;
constexpr int F16_TOP = 14;  // fp16 G is scaled to 2^14 at most, bf16 G to 1
struct LossCoef {
  const float *g;
  int64_t M;
  const float *lse, *coef;
  const int32_t *y, *up, *count;
  int distill;
  float top;
  float *scale;                   // {the scale f, 1 / f, find_scale's exponent}
  RowCoef *rows;
  int have_scale, write_rows;
  SplitPlan *plan;
  int64_t H, vp, cap;
  const float *own;
  const float *p, *tk;            // teacher's entries
  const int32_t *sid;
  int64_t K;
  // c = 0: nothing, whatever g is (rows of no sequence have no upstream gradient)
  __device__ __forceinline__ void of(float c, float g, float &a, float &b) const {
    a = c == 0.0f ? 0.0f : __fmul_rn(distill ? c : -c, g);
    b = distill && c != 0.0f ? g : a;
  }
  __device__ __forceinline__ RowCoef row(int64_t m, float f) const {
    float a, b;
    const float c = coef[m];
    of(c, c == 0.0f ? 0.0f : g[up[m]], a, b);
    return RowCoef{__fmul_rn(a, f), __fmul_rn(b, f), lse[m], distill ? -1 : y[m]};
  }
};
// The scale: all threads of a work-group, all rows. exponent: no finite coefficient times
// the scale is above 2^exponent.
template <int ET>
__device__ __forceinline__ float find_scale(const LossCoef &p, int &exponent) {
  float f = 1.0f;
  __shared__ float sh[LC_THREADS / 64];
  // The samples, unscaled entries of G: their loads go out before the rows'.
  constexpr int S = LC_SAMPLES / LC_THREADS;
  float entry[S];
  const bool apart = targets_apart<ET> && !p.distill;  // then G has no entry that weighs so much
  const int samples = apart ? 0 : (int)(p.M < LC_SAMPLES ? p.M : LC_SAMPLES);
  float o[S];
  int32_t o_up[S];
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int j = threadIdx.x + k * LC_THREADS, m = p.M <= LC_SAMPLES ? j : (int)(j * p.M / LC_SAMPLES);
    o[k] = j < samples ? p.own[m] : 0.0f;
    o_up[k] = j < samples ? p.up[m] : 0;
  }
#pragma unroll
  for (int k = 0; k < S; ++k) entry[k] = o[k] == 0.0f ? 0.0f : __fmul_rn(o[k], p.g[o_up[k]]);
  float mx = 0.0f;
  for (int64_t m0 = threadIdx.x; m0 < p.M; m0 += 8 * LC_THREADS) {
    float c[8], g[8];
    int32_t u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // past the last: the last again
      const int64_t m = m0 + k * LC_THREADS < p.M ? m0 + k * LC_THREADS : p.M - 1;
      c[k] = p.coef[m];
      u[k] = p.up[m];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = c[k] == 0.0f ? 0.0f : p.g[u[k]];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a, b;
      p.of(c[k], g[k], a, b);
      a = fabsf(a);
      b = fabsf(b);
      mx = fmaxf(mx, fmaxf(a < __builtin_inff() ? a : 0.0f, b < __builtin_inff() ? b : 0.0f));
    }
  }
  for (int d = 32; d; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < LC_THREADS / 64; ++w) mx = fmaxf(mx, sh[w]);
  exponent = ilogbf(mx > 0.0f ? mx : 1.0f) + 1;
  // f and 1 / f both well inside the normal range, else no scale
  if (mx > 1e-30f && mx < 1e30f) {
    exponent = ET == ET_F16 ? F16_TOP : 0;
    f = __fdiv_rn(p.top, mx);
    if (apart) return f;
    __shared__ float err[LC_TRIES][LC_THREADS + 1];
    float e2[LC_TRIES] = {};
    auto sample = [&](float g) {  // an entry of G, unscaled
      float x = __fmul_rn(g, f);
      if (!(fabsf(x) <= 2.0f * p.top)) x = 0.0f;
      float back = 1.0f;  // 1 / the factor tried
#pragma unroll
      for (int j = 0; j < LC_TRIES; ++j) {
        const uint32_t r = mm_pack2<ET>(x, 0.0f);
        float d;
        if constexpr (ET == ET_F16)
          d = (float)__builtin_bit_cast(_Float16, (uint16_t)r);
        else
          d = __builtin_bit_cast(float, r << 16);
        d = __fmul_rn(__fsub_rn(d, x), back);
        e2[j] = __fmaf_rn(d, d, e2[j]);
        x = __fmul_rn(x, LC_STEP);
        back = __fmul_rn(back, 1.0f / LC_STEP);
      }
    };
#pragma unroll
    for (int k = 0; k < S; ++k)
      if (k * LC_THREADS < samples) sample(entry[k]);
#pragma unroll
    for (int j = 0; j < LC_TRIES; ++j) err[j][threadIdx.x] = e2[j];
    __syncthreads();
    {
      const int j = threadIdx.x / 16, part = threadIdx.x % 16;
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < LC_THREADS; k += 16) s = __fadd_rn(s, err[j][k + part]);
#pragma unroll
      for (int d = 1; d < 16; d *= 2) s = __fadd_rn(s, __shfl_xor(s, d));
      __syncthreads();
      if (part == 0) err[0][j] = s;
    }
    __syncthreads();
    float least = err[0][0], factor = 1.0f, best = 1.0f;
#pragma unroll
    for (int j = 1; j < LC_TRIES; ++j) {
      factor = __fmul_rn(factor, LC_STEP);
      if (err[0][j] < least) {
        least = err[0][j];
        best = factor;
      }
    }
    f = __fmul_rn(f, best);
  }
  return f;
}
template <int ET>
__global__ __launch_bounds__(LC_THREADS) void loss_coef_kernel(LossCoef p) {
  if (p.count != nullptr) {
    p.M = *p.count;
    if (blockIdx.x == 0 && threadIdx.x < 64 && !p.have_scale)
      plan_splits((int32_t)p.M, (int32_t)p.H, (int32_t)p.vp, (int32_t)p.cap, p.plan);
  }
  int exponent = 0;
  const float f = p.have_scale ? p.scale[0] : find_scale<ET>(p, exponent);
  if (!p.have_scale && blockIdx.x == 0 && threadIdx.x == 0) {
    p.scale[0] = f;
    p.scale[1] = __fdiv_rn(1.0f, f);
    p.scale[2] = (float)exponent;
  }
  const int64_t m = (int64_t)blockIdx.x * LC_THREADS + threadIdx.x;
  if (p.write_rows && m < p.M) p.rows[m] = p.row(m, f);
}

// Packed rows: their number is known on the device.
struct OnDevice {
  const int32_t *count;   // nullptr: not packed, and the splits are known
  const SplitPlan *plan;
  __device__ __forceinline__ void apply(XentBwdArgs &p) const {
    if (count == nullptr) return;
    p.M = mm_uni(*count);
    p.ksplit = split_of(p.np, (int64_t)mm_uni((uint32_t)plan->splits));
  }
};

template <int ET, bool DB>
__global__ __launch_bounds__(MM_THREADS, 1) void loss_grad_kernel(XentBwdArgs p, OnDevice dev) {
  MM_SHARED();
  MM_EPI_SHARED();
  dev.apply(p);
  const XentGrad<ET, DB, targets_apart<ET>> prob{p, mm_epi, (p.M + MM_T - 1) / MM_T, p.np / MM_T};
  mm_run<ET, false, false>(prob, mm_buf);
}

// G at entry k of a row's teacher, over what the product's epilogue or the kept t
// left there: a q - b p from the entry's t, the dense value's own fp32 operations,
// rounded once. An id that a row has more than once is written by each of them
// with the sum of their p.
template <int ET>
__device__ __forceinline__ uint16_t entry_of_G(const RowCoef &r, const int32_t *sid, const float *p, const float *tk, int64_t row,
                                               int64_t K, int64_t k) {
  const int64_t at = row * K;
  const int32_t id = sid[at + k];
  int64_t first = k;
  while (first > 0 && sid[at + first - 1] == id) --first;
  float sum = 0.0f;
  for (int64_t j = first; j < K && sid[at + j] == id; ++j) sum = __fadd_rn(sum, p[at + j]);
  const float q = r.a == 0.0f ? 0.0f : exp_diff(tk[at + k], r.lse == NEG_INF ? 0.0f : r.lse);
  return (uint16_t)mm_pack2<ET>(__fsub_rn(__fmul_rn(r.a, q), __fmul_rn(r.b, sum)), 0.0f);
}

// G of a piece from the kept t: the same operations on the same values as the
// product's epilogue, so the same bits. 2048 columns and R rows a work-group,
// eight columns a thread; four rows' loads in flight: 5.5 TB/s of reads and writes (as with R = 8 or 16).
// grad_bias: the column sums of R rows.
//
// FEW (a small G of rows that are not packed): the rows' coefficients and their
// scale are found here, by every work-group, and the teacher's entries are
// written here where grad_bias does not want their sums; both are launches of
// their own otherwise (a step of 37 rows, H = 256, V = 4096: 53.8 -> 50.0 us, and
// 48.1 with the scale's loads at once).
constexpr int KEPT_FEW = 4, KEPT_MANY = 32;  // rows a work-group: few where there are few, for the sake of work-groups
constexpr int64_t KEPT_GROUPS = 1024;        // work-groups up to which each finds the scale: one round of them
int kept_rows(int64_t M) { return M <= LR_DIRECT ? KEPT_FEW : KEPT_MANY; }
bool kept_few(int64_t M, int64_t V) {
  return M <= LR_DIRECT && ceil_div(M, KEPT_FEW) * ceil_div(V, 2048) <= KEPT_GROUPS;
}
template <int ET, bool DB, int R, bool FEW>
__global__ __launch_bounds__(256) void loss_kept_kernel(XentBwdArgs p, OnDevice dev, const float *t, int64_t ldt, LossCoef few,
                                                        int entries) {
  if (!FEW) dev.apply(p);
  const int64_t chunks = (p.np + 2047) / 2048, g = group_number(), rt = g / chunks, c0 = (g - rt * chunks) * 2048;
  const int64_t m0 = rt * R, c = c0 + 8 * threadIdx.x;
  if (m0 >= p.M) return;
  float f = 1.0f;
  if constexpr (FEW) {
    int exponent;  // loss_coef_kernel leaves it, where the entries' sums want it
    f = find_scale<ET>(few, exponent);
    if (g == 0 && threadIdx.x == 0) {
      few.scale[0] = f;
      few.scale[1] = __fdiv_rn(1.0f, f);
    }
  }
  const int rows = (int)(p.M - m0 < R ? p.M - m0 : R);
  if (c < p.np) {  // np is a multiple of 256
    float sum[8] = {};
    const float *at = t + m0 * ldt + p.v0 + c;
    uint16_t *out = reinterpret_cast<uint16_t *>(p.G) + m0 * p.ldg + c;
    for (int r0 = 0; r0 < rows; r0 += 4) {
      f32x4 v[4][2];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[k][h] = __builtin_nontemporal_load(
              reinterpret_cast<const f32x4 *>(at + (r0 + k < rows ? r0 + k : rows - 1) * ldt + 4 * h));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (r0 + k >= rows) break;
        RowCoef r;
        if constexpr (FEW) r = few.row(m0 + r0 + k, f);
        else r = p.rows[m0 + r0 + k];
        if (r.lse == NEG_INF) r.lse = 0.0f;
        float g8[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) g8[q] = r.a == 0.0f ? 0.0f : __fmul_rn(r.a, exp_diff(v[k][q >> 2][q & 3], r.lse));
        const int64_t y = r.y - p.v0 - c;
        if (y >= 0 && y < 8)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (y == q) {
              g8[q] = __fsub_rn(g8[q], r.b);
              if constexpr (targets_apart<ET>) {  // in the sums only
                if constexpr (DB) sum[q] = __fadd_rn(sum[q], g8[q]);
                g8[q] = 0.0f;
              }
            }
        if constexpr (DB)
#pragma unroll
          for (int q = 0; q < 8; ++q) sum[q] = __fadd_rn(sum[q], g8[q]);
        *reinterpret_cast<u32x4 *>(out + (r0 + k) * p.ldg) = u32x4{
            mm_pack2<ET>(g8[0], g8[1]), mm_pack2<ET>(g8[2], g8[3]), mm_pack2<ET>(g8[4], g8[5]), mm_pack2<ET>(g8[6], g8[7])};
      }
    }
    if constexpr (DB) {
      const float back = FEW ? __fdiv_rn(1.0f, f) : p.scale[1];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<f32x4 *>(p.colpart + rt * p.ldg + c + 4 * h) = f32x4{
            __fmul_rn(back, sum[4 * h]), __fmul_rn(back, sum[4 * h + 1]), __fmul_rn(back, sum[4 * h + 2]), __fmul_rn(back, sum[4 * h + 3])};
    }
  }
  if constexpr (FEW && !DB) {
    if (entries) {
      dma_barrier();  // what the entries lie over has been written
      for (int64_t e = threadIdx.x; e < rows * few.K; e += 256) {
        const int64_t m = m0 + e / few.K, k = m * few.K + e % few.K;
        const int32_t id = few.sid[k];
        const int64_t col = id - p.v0;
        if (id == NO_ID || col < c0 || col >= c0 + 2048 || col >= p.np) continue;
        reinterpret_cast<uint16_t *>(p.G)[m * p.ldg + col] = entry_of_G<ET>(few.row(m, f), few.sid, few.p, few.tk, m, few.K, e % few.K);
      }
    }
  }
}
template <int ET, bool DB>
hipError_t kept_grad(const XentBwdArgs &p, const OnDevice &dev, const float *t, int64_t ldt, const LossCoef &few, bool entries,
                     hipStream_t s) {
  const int R = kept_rows(p.M);
  return launch_kernel(kept_few(p.M, p.V)  ? loss_kept_kernel<ET, DB, KEPT_FEW, true>
                       : R == KEPT_FEW ? loss_kept_kernel<ET, DB, KEPT_FEW, false>
                                       : loss_kept_kernel<ET, DB, KEPT_MANY, false>,
                       numbered_grid(ceil_div(p.M, R) * ceil_div(p.np, 2048)), dim3(256), s, p, dev, t, ldt, few, entries ? 1 : 0);
}

// The entries of a piece.
//
// grad_bias: what the entries add to it, as whole numbers of 2^-shift of the
// largest coefficient, so that the order of the additions does not matter. (Of the
// power of two above it, scaled or, outside the scale's range, as it is.)
__device__ __forceinline__ double entry_unit(const float *scale, int shift) {
  return ldexp(1.0, shift - (int)scale[2]);
}
struct DistillEntries {
  XentBwdArgs b;
  int64_t K;
  const int32_t *sid, *inv;
  const float *p, *tk;
  unsigned long long *bias;  // [V] or nullptr
  int shift;
};
template <int ET>
__global__ __launch_bounds__(256) void distill_entries_kernel(DistillEntries c) {
  const int64_t e = group_number() * 256 + threadIdx.x;
  if (e >= c.b.M * c.K) return;
  const int32_t id = c.sid[e];
  if (id == NO_ID || id < c.b.v0 || id >= c.b.v0 + c.b.np) return;
  const int64_t row = e / c.K, k = e - row * c.K, m = c.inv != nullptr ? c.inv[row] : row;
  if (m < 0) return;
  const RowCoef r = c.b.rows[m];
  reinterpret_cast<uint16_t *>(c.b.G)[m * c.b.ldg + (id - c.b.v0)] = entry_of_G<ET>(r, c.sid, c.p, c.tk, row, c.K, k);
  if (c.bias != nullptr) {
    const double x = -(double)r.b * (double)c.p[e] * entry_unit(c.b.scale, c.shift);
    // (below 2^(shift + 1) but for what is not finite, which makes the whole row of G so,
    // and with it every sum)
    if (fabs(x) < 0x1p62) atomicAdd(c.bias + id, (unsigned long long)llrint(x));
  }
}

__global__ __launch_bounds__(256) void loss_zero_kernel(uint32_t *__restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}
hipError_t zero_words(void *p, int64_t n, hipStream_t s) {
  const int64_t blocks = ceil_div(n, 256);
  return launch_kernel(loss_zero_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), s,
                       static_cast<uint32_t *>(p), n);
}

// grad_bias of one piece: the column sums of the row tiles (of `tile` rows) in
// ascending order, the entries' share, and 1 / T.
__global__ __launch_bounds__(256) void loss_bias_kernel(const float *__restrict__ colpart, int64_t M,
                                                        const int32_t *__restrict__ count, int tile, int64_t vp, int64_t n, const long long *__restrict__ entries,
                                                        const float *__restrict__ scale, int shift, float T,
                                                        float *__restrict__ db) {
  const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (v >= n) return;
  float s = 0.0f;
  const int64_t nmt = ((count != nullptr ? *count : M) + tile - 1) / tile;
#pragma unroll 8
  for (int64_t t = 0; t < nmt; ++t) s = __fadd_rn(s, colpart[t * vp + v]);
  if (entries != nullptr) s = (float)((double)s + (double)entries[v] / entry_unit(scale, shift) * (double)scale[1]);
  db[v] = __fdiv_rn(s, T);
}

template <int ET>
__global__ __launch_bounds__(MM_THREADS, 1) void loss_dhidden_kernel(XentBwdArgs p, OnDevice dev) {
  MM_SHARED();
  dev.apply(p);
  const XentDHidden<ET> prob{p, (p.M + MM_T - 1) / MM_T, (p.H + MM_T - 1) / MM_T,
                             (p.np + p.ksplit - 1) / p.ksplit};
  mm_run<ET, false, true>(prob, mm_buf);
}
template <int ET>
__global__ __launch_bounds__(MM_THREADS, 1) void loss_dweight_kernel(XentBwdArgs p, OnDevice dev) {
  MM_SHARED();
  MM_EPI_SHARED();
  dev.apply(p);
  const XentDWeight<ET> prob{p, mm_epi, p.np / MM_T, (p.H + MM_T - 1) / MM_T};
  mm_run<ET, true, true>(prob, mm_buf);
}

// Both products of a small piece in one launch, as in xent.hip.
template <int ET>
__global__ __launch_bounds__(MM_THREADS, 1) void loss_products_kernel(XentBwdArgs p, OnDevice dev, uint32_t ga) {
  MM_SHARED();
  MM_EPI_SHARED();
  dev.apply(p);
  const int64_t nht = (p.H + MM_T - 1) / MM_T;
  if (blockIdx.x < ga) {
    const XentDHidden<ET> prob{p, (p.M + MM_T - 1) / MM_T, nht, (p.np + p.ksplit - 1) / p.ksplit};
    mm_run<ET, false, true>(prob, mm_buf, blockIdx.x, ga);
  } else {
    const XentDWeight<ET> prob{p, mm_epi, p.np / MM_T, nht};
    mm_run<ET, true, true>(prob, mm_buf, blockIdx.x - ga, gridDim.x - ga);
  }
}
// At most 64 rows: G^T hidden without the core (xent_core.hpp).
template <int ET>
__global__ __launch_bounds__(64 * XO_WAVES, 3) void loss_outer_kernel(XentBwdArgs p, int64_t per_slab) {
  XO_SHARED();
  xent_outer<ET>(p, per_slab, xo_g0, xo_g1, xo_stage);
}

// The rows of each target, where there are more than OUT_CHUNK rows. notes and used from zeros.
struct TokenLists {
  int2 *notes;      // [V] {M - a token's first row, its rows}
  int4 *used;       // {tokens of up to OUT_SHORT rows, places of order, other tokens}
  int32_t *tokens;  // [M] the tokens, the others from the end on, ...
  int2 *lists;      // [M] ... and {place in order, rows}
  int32_t *order;   // [n] the rows, token by token
};
// What the products leave to do: grad_hidden from its sums, and the targets' entries of G
// (targets_apart).
struct LossOut {
  const float *dh;  // [splits][n, H]
  int64_t M, H;
  const int32_t *count, *inv;
  const SplitPlan *plan;
  int splits;       // not packed
  float alpha;
  const float *scale;
  uint16_t *out;          // grad_hidden or nullptr
  // targets kept apart (else W is nullptr)
  const uint16_t *W, *hidden;  // hidden: State's
  const int32_t *y, *up;
  const float *own, *g;
  uint16_t *dw;           // grad_W
  int64_t tokens;         // work-groups of its rows, the first ones
  TokenLists lists;       // more than OUT_CHUNK rows
  __device__ __forceinline__ float entry(int64_t m) const {
    const float o = own[m];
    return o == 0.0f ? 0.0f : __fmul_rn(o, g[up[m]]);
  }
};
template <int ET>
__device__ __forceinline__ void unpack8(const u32x4 &v, float (&x)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t word = v[q / 2];
    if constexpr (ET == ET_F16)
      x[q] = (float)__builtin_bit_cast(_Float16, (uint16_t)(q & 1 ? word >> 16 : word));
    else
      x[q] = __builtin_bit_cast(float, q & 1 ? word & 0xFFFF0000u : word << 16);
  }
}
template <int ET>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  return u32x4{mm_pack2<ET>(x[0], x[1]), mm_pack2<ET>(x[2], x[3]), mm_pack2<ET>(x[4], x[5]), mm_pack2<ET>(x[6], x[7])};
}

// grad_W's row of a token: what the product left there (rounded), and the entries of the
// rows whose target it is, in those rows' order. With up to OUT_CHUNK rows there is a
// work-group a row and slab of columns, which looks at all targets and ends at once where the
// row is not the token's first. With more, three kernels before make lists (of each token's
// first row and number of rows, of the lists' places, of the rows), and the work-groups take
// token after token. With short rows several threads have the same columns: they take a row each.
// (Backward pass with and without, H = 4096, targets distributed as 1 / rank: 4096 rows,
// V = 128256, 6633 against 6595 us, all of one target 7078 against 6595; 16384 rows 27.19
// ms against 27.00; 65536 rows, V = 32000, 28.24 against 27.54, of which the lists 0.3.)
constexpr int OUT_CHUNK = 4096, OUT_BATCH = 1024, OUT_SLAB_FEW = 2048, OUT_SLAB_MANY = 512, OUT_SHORT = 16;
// The rows of base .. base + OUT_CHUNK - 1 before n whose target is the token, in order, to
// LDS as numbers from base on, by 256 threads; how many, or -1 where one lies before `first`.
__device__ __forceinline__ int find_rows(const int32_t *y, int64_t base, int64_t n, int32_t token, int64_t first,
                                         uint16_t (&found)[OUT_CHUNK], int (&sh)[4]) {
  static_assert(OUT_CHUNK == 256 * 16);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r = base + threadIdx.x * 16;
  uint32_t mask = 0;
#pragma unroll
  for (int h = 0; h < 4; ++h)
    if (r + 4 * h < n) {  // (y's room is whole 256 bytes)
      const int4 v = *reinterpret_cast<const int4 *>(y + r + 4 * h);
      mask |= ((v.x == token ? 1u : 0u) | (v.y == token ? 2u : 0u) | (v.z == token ? 4u : 0u) | (v.w == token ? 8u : 0u)) << (4 * h);
    }
  if (r + 16 > n) mask &= r < n ? (1u << (n - r)) - 1 : 0u;
  if (__syncthreads_or(mask != 0 && r + __builtin_ctz(mask | 0x10000u) < first)) return -1;
  const int mine = __popc(mask);
  int at = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int other = __shfl_up(at, d);
    at += lane >= d ? other : 0;
  }
  if (lane == 63) sh[wave] = at;
  __syncthreads();
  at -= mine;
  for (int w = 0; w < wave; ++w) at += sh[w];
  for (; mask != 0; mask &= mask - 1) found[at++] = (uint16_t)(threadIdx.x * 16 + __builtin_ctz(mask));
  const int all = sh[0] + sh[1] + sh[2] + sh[3];
  __syncthreads();
  return all;
}

struct TokenRowsOf {
  const int32_t *y, *count;
  int64_t M;
  TokenLists to;
};
__global__ __launch_bounds__(256) void loss_tokens_kernel(TokenRowsOf c) {
  const int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int32_t token = m < *c.count ? c.y[m] : -1;
  // a frequent token's additions follow each other: one for all of a wave's
  for (uint64_t todo = __ballot(token >= 0); todo != 0;) {
    const int lane = __builtin_ctzll(todo);
    const int32_t one = __builtin_amdgcn_readlane(token, lane);
    const uint64_t same = __ballot(token == one);
    if ((int)(threadIdx.x & 63) == lane) {
      atomicMax(&c.to.notes[one].x, (int32_t)(c.M - m));
      atomicAdd(&c.to.notes[one].y, __popcll(same));
    }
    todo &= ~same;
  }
}
// The tokens' lists and their places, which are chance (what is in a list is not), a wave 64
// rows: one addition to `used` each, one a token would take 0.3 ms for 20000 tokens.
__global__ __launch_bounds__(256) void loss_places_kernel(TokenRowsOf c) {
  const int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int lane = threadIdx.x & 63;
  const int32_t token = m < *c.count ? c.y[m] : -1;
  int2 note = token >= 0 ? c.to.notes[token] : int2{0, 0};
  if (note.x != (int32_t)(c.M - m)) note.y = 0;  // not the first
  int place = note.y;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int other = __shfl_up(place, d);
    place += lane >= d ? other : 0;
  }
  const uint64_t few = __ballot(note.y > 0 && note.y <= OUT_SHORT), many = __ballot(note.y > OUT_SHORT), below = (1ull << lane) - 1;
  const int all = __shfl(place, 63);
  unsigned long long at = 0;
  int back = 0;
  if (lane == 0 && all > 0) {
    at = atomicAdd(reinterpret_cast<unsigned long long *>(&c.to.used->x), (unsigned long long)all << 32 | __popcll(few));
    if (many != 0) back = atomicAdd(&c.to.used->z, __popcll(many));
  }
  const int first = __shfl((int)(uint32_t)at, 0), base = __shfl((int)(at >> 32), 0);
  back = __shfl(back, 0);
  if (note.y == 0) return;
  place += base - note.y;
  const int64_t i = note.y <= OUT_SHORT ? first + __popcll(few & below) : c.M - 1 - back - __popcll(many & below);
  c.to.tokens[i] = token;
  c.to.lists[i] = int2{place, note.y};
  if (note.y == 1) c.to.order[place] = (int32_t)m;
}
// ... and the rows of those with more than one, the longest first.
__global__ __launch_bounds__(256) void loss_lists_kernel(TokenRowsOf c) {
  __shared__ uint16_t found[OUT_CHUNK];
  __shared__ int sh[4];
  const int64_t n = *c.count;
  const int4 used = *c.to.used;
  for (int64_t i = blockIdx.x; i < used.x + used.z; i += gridDim.x) {
    const int64_t t = i < used.z ? c.M - 1 - i : i - used.z;
    const int2 list = c.to.lists[t];
    if (list.y == 1) continue;
    const int32_t token = c.to.tokens[t];
    int done = 0;
    for (int64_t base = (c.M - c.to.notes[token].x) / OUT_CHUNK * OUT_CHUNK; done < list.y && base < n; base += OUT_CHUNK) {
      const int more = find_rows(c.y, base, n, token, 0, found, sh);
      for (int k = threadIdx.x; k < more; k += 256) c.to.order[list.x + done + k] = (int32_t)(base + found[k]);
      done += more;
      __syncthreads();
    }
  }
}

struct TokenShared {
  int32_t rows[OUT_BATCH];
  float entries[OUT_BATCH];
  float sums[256][8];
};
template <int ET>
__device__ __forceinline__ void put_token(const LossOut &c, u32x4 *to, const u32x4 &main, const float (&sum)[8]) {
  float x[8];
  unpack8<ET>(main, x);
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = __fmaf_rn(c.alpha, sum[q], x[q]);
  *to = pack8<ET>(x);
}
// row_at(i): the token's rows
template <int ET, int SLAB, typename F>
__device__ __forceinline__ void add_token(const LossOut &c, TokenShared &sh, int32_t token, int64_t slab, int count, F &&row_at) {
  const int tid = threadIdx.x;
  const int per = c.H < SLAB ? (int)c.H / 8 : SLAB / 8;  // threads a row
  const int parts = 256 / per, part = tid / per;
  const int64_t col = slab * SLAB + tid % per * 8;
  const bool works = part < parts && col < c.H;
  float sum[8] = {};
  auto add = [&](auto nc, int e0) {  // that many rows' loads in flight
    constexpr int N = decltype(nc)::value;
    u32x4 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = *reinterpret_cast<const u32x4 *>(c.hidden + sh.rows[e0 + k * parts] * c.H + col);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float h[8];
      unpack8<ET>(v[k], h);
      const float x = sh.entries[e0 + k * parts];
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] = __fmaf_rn(x, h[q], sum[q]);
    }
  };
  for (int b = 0; b < count; b += OUT_BATCH) {
    const int listed = count - b < OUT_BATCH ? count - b : OUT_BATCH;
    for (int i = tid; i < listed; i += 256) {
      const int32_t r = row_at(b + i);
      sh.rows[i] = r;
      sh.entries[i] = c.entry(r);
    }
    __syncthreads();
    if (works) {
      int e0 = part;
      for (; e0 + 7 * parts < listed; e0 += 8 * parts) add(std::integral_constant<int, 8>{}, e0);
      for (; e0 + parts < listed; e0 += 2 * parts) add(std::integral_constant<int, 2>{}, e0);
      if (e0 < listed) add(std::integral_constant<int, 1>{}, e0);
    }
    __syncthreads();
  }
  if (parts > 1) {
#pragma unroll
    for (int q = 0; q < 8; ++q) sh.sums[tid][q] = sum[q];
    __syncthreads();
  }
  if (part != 0 || !works) return;
  for (int k = 1; k < parts; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] = __fadd_rn(sum[q], sh.sums[k * per + tid][q]);
  u32x4 *const to = reinterpret_cast<u32x4 *>(c.dw + token * c.H + col);
  put_token<ET>(c, to, *to, sum);
}
template <int ET, bool MANY>
__device__ __forceinline__ void out_tokens(const LossOut &c, int64_t group) {
  __shared__ TokenShared sh;
  if constexpr (MANY) {
    const int64_t slabs = (c.H + OUT_SLAB_MANY - 1) / OUT_SLAB_MANY;
    const int4 used = *c.lists.used;
    for (int64_t i = group; i < used.z * slabs; i += c.tokens) {
      const int64_t t = c.M - 1 - i / slabs;
      const int2 list = c.lists.lists[t];
      const int32_t *const order = c.lists.order + list.x;
      add_token<ET, OUT_SLAB_MANY>(c, sh, c.lists.tokens[t], i % slabs, list.y, [&](int k) { return order[k]; });
    }
    // most tokens have a row or two: a wave each
    for (int64_t i = group * 4 + threadIdx.x / 64; i < used.x * slabs; i += 4 * c.tokens) {
      const int64_t t = i / slabs, col = (i - t * slabs) * OUT_SLAB_MANY + (threadIdx.x & 63) * 8;
      if (col >= c.H) continue;
      const int2 list = c.lists.lists[t];
      u32x4 *const to = reinterpret_cast<u32x4 *>(c.dw + c.lists.tokens[t] * c.H + col);
      const u32x4 main = *to;
      float sum[8] = {};
      for (int k = 0; k < list.y; k += 2) {
        const int32_t r0 = c.lists.order[list.x + k], r1 = c.lists.order[list.x + (k + 1 < list.y ? k + 1 : k)];
        const u32x4 v0 = *reinterpret_cast<const u32x4 *>(c.hidden + r0 * c.H + col);
        const u32x4 v1 = *reinterpret_cast<const u32x4 *>(c.hidden + r1 * c.H + col);
        const float e0 = c.entry(r0), e1 = k + 1 < list.y ? c.entry(r1) : 0.0f;
        float h[8];
        unpack8<ET>(v0, h);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] = __fmaf_rn(e0, h[q], sum[q]);
        if (k + 1 == list.y) break;
        unpack8<ET>(v1, h);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] = __fmaf_rn(e1, h[q], sum[q]);
      }
      put_token<ET>(c, to, main, sum);
    }
  } else {
    __shared__ uint16_t found[OUT_CHUNK];
    __shared__ int counts[4];
    const int64_t slabs = (c.H + OUT_SLAB_FEW - 1) / OUT_SLAB_FEW, n = c.count != nullptr ? *c.count : c.M, m = group / slabs;
    if (m >= n) return;
    const int32_t token = c.y[m];
    if (token < 0) return;
    const int count = find_rows(c.y, 0, n, token, m, found, counts);
    if (count > 0) add_token<ET, OUT_SLAB_FEW>(c, sh, token, group % slabs, count, [&](int k) { return (int32_t)found[k]; });
  }
}

// grad_hidden: the splits' sums in ascending order, scaled, with the target's entry,
// rounded once; 0 in the rows left out.
template <int ET, bool MANY>
__global__ __launch_bounds__(256, 5) void loss_out_kernel(LossOut c) {
  const int64_t group = group_number();
  if (targets_apart<ET> && group < c.tokens) {
    out_tokens<ET, MANY>(c, group);
    return;
  }
  const int64_t e = ((group - c.tokens) * 256 + threadIdx.x) * 8;
  if (c.out == nullptr || e >= c.M * c.H) return;
  const int64_t row = e / c.H, m = c.inv != nullptr ? c.inv[row] : row;
  if (m < 0) {
    *reinterpret_cast<u32x4 *>(c.out + e) = u32x4{0, 0, 0, 0};
    return;
  }
  const int64_t n = (c.count != nullptr ? *c.count : c.M) * c.H, at = m * c.H + (e - row * c.H);
  const int splits = c.count != nullptr ? c.plan->splits : c.splits;
  f32x4 s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) s[h] = *reinterpret_cast<const f32x4 *>(c.dh + at + 4 * h);
  auto more = [&](auto nc, int k0) {  // that many splits' loads in flight
    constexpr int N = decltype(nc)::value;
    f32x4 v[N][2];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) v[k][h] = *reinterpret_cast<const f32x4 *>(c.dh + (k0 + k) * n + at + 4 * h);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[h][q] = __fadd_rn(s[h][q], v[k][h][q]);
  };
  int k0 = 1;
  for (; k0 + 8 <= splits; k0 += 8) more(std::integral_constant<int, 8>{}, k0);
  for (; k0 + 2 <= splits; k0 += 2) more(std::integral_constant<int, 2>{}, k0);
  if (k0 < splits) more(std::integral_constant<int, 1>{}, k0);
  const float f = __fmul_rn(c.alpha, c.scale[1]);
  float x[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = __fmul_rn(f, s[q / 4][q % 4]);
  const int32_t token = targets_apart<ET> && c.W != nullptr ? c.y[m] : -1;
  if (token >= 0) {
    float w[8];
    unpack8<ET>(*reinterpret_cast<const u32x4 *>(c.W + token * c.H + (e - row * c.H)), w);
    const float entry = __fmul_rn(c.alpha, c.entry(m));
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = __fmaf_rn(entry, w[q], x[q]);
  }
  *reinterpret_cast<u32x4 *>(c.out + e) = pack8<ET>(x);
}

// Pieces of up to an eighth more columns, where G^T hidden then takes fewer
// rounds of work-groups in all: 594 tiles of columns by 8 of H (V = 151936, H = 2048)
// in two pieces of 297 are twice ten rounds for 256 CUs, in 320 and 274 ten and nine.
// Not past bwd_plan's 256 MiB of G. Backward passes, ms, H, V, rows: 2048, 151936, 1000
// 1.273 -> 1.257, 4096 rows 4.45 -> 4.38; 4096, 151936, 4096 8.05 -> 7.95; 4096, 200000,
// 2048 5.48 -> 5.39; 8192, 50257, 8192 10.50 -> 10.23; 8192, 128256, 2048 (a round of 64
// less) 6.60 -> 6.58; 1024, 262144, 1337 1.688 -> 1.704. With G of 261 and 272 MiB, 1337
// rows, V = 200000: H = 4096 3.97 -> 4.13, H = 2048 2.15 -> 2.20.
int64_t whole_rounds(int64_t vp, int64_t M, int64_t H, int64_t V) {
  const int64_t nht = ceil_div(H, MM_T), all = ceil_div(V, MM_T), n = vp / MM_T, unit = ceil_div(256, nht);
  auto rounds = [&](int64_t per) { return all / per * ceil_div(per * nht, 256) + ceil_div(all % per * nht, 256); };
  const int64_t more = ceil_div(n, unit) * unit;
  const bool fits = 2 * M * more * MM_T <= (int64_t)256 << 20 || more * MM_T <= 8192;
  return n < all && more < all && more <= n + n / 8 && fits && rounds(more) < rounds(n) ? more * MM_T : vp;
}

// Row tiles times splits of the plans (plan_splits) for up to nmt row tiles. (65536 rows,
// H = 4096: one sum of all rows, 1 GB, where three had been kept.)
int64_t most_parts(int64_t nmt, int64_t nht, int64_t vp) {
  int64_t most = nmt;
  for (int64_t k = 1; k <= nmt && k * nht < SPLIT_TILES; ++k) {
    int64_t s = (SPLIT_TILES - 1) / (k * nht) + 1;
    if (s > vp / 256) s = vp / 256;
    if (s > 64) s = 64;
    if (s * k > most) most = s * k;
  }
  return most;
}

// bwd_plan's pieces, with room for the sums of grad_hidden of whatever rows are
// worked on: `cap` row tiles times splits.
struct BackwardLayout {
  int64_t vp, cap;
  int splits;
  int64_t scale, plan, rows, col, dh, G, entries, lists, bytes;
};
BackwardLayout backward_layout(int64_t M, int64_t H, int64_t V, int64_t K, bool keep, bool bias) {
  BackwardLayout b;
  const BwdPlan pl = bwd_plan(M, H, V, bias);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += align256(bytes);
    return o;
  };
  const int64_t nmt = ceil_div(M, MM_T);
  b.vp = whole_rounds(pl.vp, M, H, V);
  b.splits = (int)ceil_div(b.vp, split_of(b.vp, pl.splits));
  // fewer rows than the call's take more splits: with three fifths of 4096 rows
  // (H = 4096) 160 tiles would leave 96 of 256 CUs without one; three splits of
  // them fill 94%
  b.cap = pl.splits > 3 || M <= LR_DIRECT ? pl.splits * nmt : 3 * nmt;
  if (M > LR_DIRECT) {
    const int64_t most = most_parts(nmt, ceil_div(H, MM_T), b.vp);
    if (most < b.cap) b.cap = most;
  }
  b.scale = take(12);
  b.plan = take(sizeof(SplitPlan));
  b.rows = take(16 * M);
  b.col = take(bias ? 4 * (keep ? ceil_div(M, kept_rows(M)) : nmt) * b.vp : 0);
  b.dh = take(4 * H * b.cap * (M > LR_DIRECT ? MM_T : M));  // not packed: one row tile
  b.G = take(2 * M * b.vp);
  b.entries = take(bias && K ? 8 * V : 0);
  b.lists = take(K == 0 && M > OUT_CHUNK ? 16 + 8 * (V + M) + 8 * M : 0);
  b.bytes = at;
  return b;
}

// What the three forward passes begin with: the memory's places, the bias.
struct Setup {
  State st;
  ForwardLayout lay;
  uint8_t *ws;
  LossFwdArgs a;
};
hipError_t set_up(const LossHead &h, const LossMemory &mem, int64_t K, hipStream_t s, Setup &u) {
  u.lay = forward_layout(h.M, h.H, h.V, K, mem.state != nullptr);
  u.ws = static_cast<uint8_t *>(mem.workspace);
  u.st = state_at(mem.state != nullptr ? mem.state : u.ws + u.lay.state, state_layout(h.M, h.H, h.V, K, mem.keep != 0),
                  h.M);
  u.a = LossFwdArgs{};
  u.a.hidden = static_cast<const uint8_t *>(u.st.rows != nullptr ? u.st.hidden : h.hidden);
  u.a.W = static_cast<const uint8_t *>(h.W);
  u.a.M = h.M;
  u.a.H = h.H;
  u.a.V = h.V;
  u.a.alpha = (float)((double)h.alpha / (double)h.temperature);
  u.a.bias = h.bias;
  u.a.count = u.st.count;
  u.a.rows = u.st.rows;
  u.a.y = u.st.rows != nullptr ? u.st.y : nullptr;
  u.a.part = reinterpret_cast<float2 *>(u.ws + u.lay.part);
  u.a.tlogit = reinterpret_cast<float *>(u.ws + u.lay.tlogit);
  u.a.K = K;
  u.a.t = u.st.t;
  if (h.M == 0 || h.bias == nullptr || h.temperature == 1.0f) return hipSuccess;
  u.a.bias = u.st.bias;
  return launch_kernel(loss_bias_scale_kernel, dim3((unsigned)ceil_div(h.V, 256)), dim3(256), s, h.bias, h.V,
                       h.temperature, u.st.bias);
}
// The rows worked on, one behind the other.
hipError_t gather(const LossHead &h, const Setup &u, const Select &sel, float *zero0, float *zero1, hipStream_t s) {
  if (u.st.rows == nullptr) return hipSuccess;
  int32_t *const chunks = reinterpret_cast<int32_t *>(u.ws + u.lay.chunks);
  hipError_t e = hipSuccess;
  if (h.M > LR_CHUNK)
    e = launch_kernel(loss_count_kernel, dim3((unsigned)ceil_div(h.M, LR_CHUNK)), dim3(LR_THREADS), s, sel, chunks);
  if (e == hipSuccess)
    e = launch_kernel(loss_gather_kernel, dim3((unsigned)ceil_div(h.M, LR_ROWS)), dim3(LR_THREADS), s,
                      Gather{sel, chunks, static_cast<const uint16_t *>(h.hidden), h.H, u.st, zero0, zero1});
  return e;
}
template <bool PICK, bool KEEP>
hipError_t stats(const LossHead &h, const LossFwdArgs &a, hipStream_t s) {
  const int64_t tiles = ceil_div(h.M, MM_T) * ceil_div(h.V, MM_T);
  return launch_kernel(h.in_f16 ? loss_stats_kernel<ET_F16, PICK, KEEP> : loss_stats_kernel<ET_BF16, PICK, KEEP>,
                       mm_grid(tiles), dim3(MM_THREADS), s, a);
}
template <bool PICK>
hipError_t stats(const LossHead &h, const LossFwdArgs &a, bool keep, hipStream_t s) {
  return keep ? stats<false, true>(h, a, s) : stats<PICK, false>(h, a, s);
}
void set_targets(LossFwdArgs &a, const LossTargets &y) {
  a.target = y.target;
  a.target64 = y.wide;
  a.ignore = y.ignore;
}
RowsArgs rows_args(const LossHead &h, const LossMemory &mem, const Setup &u, const Select &sel) {
  return RowsArgs{u.a.part, h.M, ceil_div(h.V, MM_T), u.st, sel,
                  mem.state != nullptr && u.st.rows == nullptr ? static_cast<const uint16_t *>(h.hidden) : nullptr, h.H,
                  mem.keep != 0 ? padded(h.V) : 0};
}
dim3 rows_grid(int64_t M) { return dim3((unsigned)ceil_div(M, XC_ROWS)); }

template <int ET>
hipError_t backward(const LossBackward &c, hipStream_t s) {
  const LossHead &h = c.head;
  const BackwardLayout lay = backward_layout(h.M, h.H, h.V, c.K, c.mem.keep != 0, c.grad_bias != nullptr);
  uint8_t *const ws = static_cast<uint8_t *>(c.mem.workspace);
  const State st = state_at(c.mem.state, state_layout(h.M, h.H, h.V, c.K, c.mem.keep != 0), h.M);
  float *const scale = reinterpret_cast<float *>(ws + lay.scale);
  SplitPlan *const plan = reinterpret_cast<SplitPlan *>(ws + lay.plan);
  RowCoef *const rows = reinterpret_cast<RowCoef *>(ws + lay.rows);
  const float top = ET == ET_F16 ? (float)(1 << F16_TOP) : 1.0f;
  LossCoef r{c.grad_loss, h.M, st.lse, st.coef, st.y, st.up, st.count, c.K > 0, top, scale, rows, 0, 1,
             plan, h.H, lay.vp, lay.cap, st.own, st.p, st.tk, st.ids, c.K};
  hipError_t e = hipSuccess;
  if (h.M > LC_ONE) {
    r.write_rows = 0;
    e = launch_kernel(loss_coef_kernel<ET>, dim3(1), dim3(LC_THREADS), s, r);
    r.write_rows = r.have_scale = 1;
  }
  const bool few = c.mem.keep != 0 && kept_few(h.M, h.V);  // loss_kept_kernel finds them itself
  if (e == hipSuccess && (!few || (c.K > 0 && c.grad_bias != nullptr)))
    e = launch_kernel(loss_coef_kernel<ET>, dim3((unsigned)ceil_div(h.M, LC_THREADS)), dim3(LC_THREADS), s, r);
  XentBwdArgs p{};
  p.hidden = reinterpret_cast<const uint8_t *>(st.hidden);
  p.W = static_cast<const uint8_t *>(h.W);
  p.M = h.M;
  p.H = h.H;
  p.V = h.V;
  p.alpha = (float)((double)h.alpha / (double)h.temperature);
  p.bias = h.bias == nullptr || h.temperature == 1.0f ? h.bias : st.bias;
  p.rows = rows;
  p.scale = scale;
  p.ldg = lay.vp;
  p.G = ws + lay.G;
  p.colpart = c.grad_bias != nullptr ? reinterpret_cast<float *>(ws + lay.col) : nullptr;
  p.dh = reinterpret_cast<float *>(ws + lay.dh);
  p.dw = static_cast<uint16_t *>(c.grad_W);
  const OnDevice dev{st.count, plan};
  const int64_t nmt = ceil_div(h.M, MM_T), nht = ceil_div(h.H, MM_T);
  // whole numbers of 2^-shift: their sum over all rows stays below 2^62
  int shift = 61;
  for (int64_t k = h.M * (c.K > 0 ? c.K : 1); k > 0; k >>= 1) --shift;
  if (shift > 44) shift = 44;
  const bool sums = c.grad_bias != nullptr && c.K > 0;
  unsigned long long *const entries = sums ? reinterpret_cast<unsigned long long *>(ws + lay.entries) : nullptr;
  if (e == hipSuccess && sums) e = zero_words(entries, 2 * h.V, s);
  for (int64_t v0 = 0; v0 < h.V && e == hipSuccess; v0 += lay.vp) {
    p.v0 = v0;
    p.first = v0 == 0;
    const int64_t nv = h.V - v0 < lay.vp ? h.V - v0 : lay.vp;
    p.np = ceil_div(nv, MM_T) * MM_T;
    p.ksplit = split_of(p.np, lay.splits);
    if (c.mem.keep)
      e = c.grad_bias != nullptr ? kept_grad<ET, true>(p, dev, st.t, padded(h.V), r, false, s)
                                 : kept_grad<ET, false>(p, dev, st.t, padded(h.V), r, c.K > 0, s);
    else
      e = launch_kernel(c.grad_bias != nullptr ? loss_grad_kernel<ET, true> : loss_grad_kernel<ET, false>,
                        mm_grid(nmt * (p.np / MM_T)), dim3(MM_THREADS), s, p, dev);
    if (e == hipSuccess && c.K > 0 && (!few || c.grad_bias != nullptr))
      e = launch_kernel(distill_entries_kernel<ET>, numbered_grid(ceil_div(h.M * c.K, 256)), dim3(256), s,
                        DistillEntries{p, c.K, st.ids, st.inv, st.p, st.tk, entries, shift});
    if (e == hipSuccess && c.grad_bias != nullptr)
      e = launch_kernel(loss_bias_kernel, dim3((unsigned)ceil_div(nv, 256)), dim3(256), s,
                        static_cast<const float *>(p.colpart), h.M, static_cast<const int32_t *>(st.count),
                        c.mem.keep ? kept_rows(h.M) : (int)MM_T, lay.vp, nv,
                        sums ? reinterpret_cast<const long long *>(entries) + v0 : nullptr, static_cast<const float *>(scale),
                        shift, h.temperature, c.grad_bias + v0);
    const int64_t ta = nht * lay.cap, tb = nht * (p.np / MM_T);  // ta: the most there are
    if (e == hipSuccess && c.grad_hidden != nullptr && c.grad_W != nullptr && ta + tb <= device_cus()) {
      e = launch_kernel(loss_products_kernel<ET>, dim3((unsigned)(ta + tb)), dim3(MM_THREADS), s, p, dev, (uint32_t)ta);
      continue;
    }
    if (e == hipSuccess && c.grad_hidden != nullptr)
      e = launch_kernel(loss_dhidden_kernel<ET>, mm_grid(ta), dim3(MM_THREADS), s, p, dev);
    if (e == hipSuccess && c.grad_W != nullptr) {
      if (h.M <= XO_ROWS) {
        // three work-groups per CU, spread over the slabs of hidden's columns
        const int64_t slots = ceil_div(3 * (int64_t)device_cus(), nht), n = ceil_div(nv, 128);
        const int64_t per_slab = n < slots ? n : slots;
        e = launch_kernel(loss_outer_kernel<ET>, dim3((unsigned)(nht * per_slab)), dim3(64 * XO_WAVES), s, p, per_slab);
      } else {
        e = launch_kernel(loss_dweight_kernel<ET>, mm_grid(tb), dim3(MM_THREADS), s, p, dev);
      }
    }
  }
  const bool apart = targets_apart<ET> && c.K == 0;
  LossOut out{p.dh, h.M, h.H, st.count, st.inv, plan, lay.splits, p.alpha, scale, static_cast<uint16_t *>(c.grad_hidden),
              apart ? static_cast<const uint16_t *>(h.W) : nullptr, st.hidden, st.y, st.up, st.own, c.grad_loss,
              static_cast<uint16_t *>(c.grad_W), 0, {}};
  const bool many = apart && c.grad_W != nullptr && h.M > OUT_CHUNK;
  if (many) {
    uint8_t *const lists = ws + lay.lists;
    int4 *const used = reinterpret_cast<int4 *>(lists);
    int2 *const notes = reinterpret_cast<int2 *>(used + 1);
    int32_t *const words = reinterpret_cast<int32_t *>(notes + h.V + h.M);
    out.lists = TokenLists{notes, used, words, notes + h.V, words + h.M};
    const TokenRowsOf of{st.y, st.count, h.M, out.lists};
    if (e == hipSuccess) e = zero_words(lists, 4 + 2 * h.V, s);
    if (e == hipSuccess) e = launch_kernel(loss_tokens_kernel, dim3((unsigned)ceil_div(h.M, 256)), dim3(256), s, of);
    if (e == hipSuccess) e = launch_kernel(loss_places_kernel, dim3((unsigned)ceil_div(h.M, 256)), dim3(256), s, of);
    if (e == hipSuccess) e = launch_kernel(loss_lists_kernel, dim3((unsigned)(8 * device_cus())), dim3(256), s, of);
    out.tokens = 4 * (int64_t)device_cus();  // as many as there is room for
  } else if (apart && c.grad_W != nullptr) {
    out.tokens = h.M * ceil_div(h.H, OUT_SLAB_FEW);
  }
  const int64_t groups = out.tokens + (out.out != nullptr ? ceil_div(h.M * h.H, 2048) : 0);
  if (e == hipSuccess && groups > 0)
    e = launch_kernel(many ? loss_out_kernel<ET, true> : loss_out_kernel<ET, false>, numbered_grid(groups), dim3(256), s, out);
  return e;
}

}  // namespace

int64_t loss_state_bytes(int64_t M, int64_t H, int64_t V, int64_t K, bool keep) {
  return state_layout(M, H, V, K, keep).bytes;
}
int64_t loss_forward_bytes(int64_t M, int64_t H, int64_t V, int64_t K, bool with_state) {
  return forward_layout(M, H, V, K, with_state).bytes;
}
int64_t loss_backward_bytes(int64_t M, int64_t H, int64_t V, int64_t K, bool keep, bool bias) {
  return backward_layout(M, H, V, K, keep, bias).bytes;
}

hipError_t launch_distill_forward(const DistillForward &c, hipStream_t s) {
  const LossHead &h = c.head;
  Setup u;
  hipError_t e = set_up(h, c.mem, c.K, s, u);
  if (e != hipSuccess) return e;
  uint16_t *const ptr = reinterpret_cast<uint16_t *>(u.ws + u.lay.ptr);
  float *const ent = reinterpret_cast<float *>(u.ws + u.lay.ent), *const P = reinterpret_cast<float *>(u.ws + u.lay.P);
  const DistillPrep d{c.ids, c.ids64, h.M, h.V, c.K, c.logits, c.logits_type, c.teacher_lse, h.temperature,
                      u.st.ids, u.st.p, c.mem.keep != 0 ? nullptr : ptr, ent, P};
  e = launch_kernel(c.K <= 64 ? distill_prep_kernel<1> : c.K <= 256 ? distill_prep_kernel<4> : distill_prep_kernel<16>,
                    numbered_grid(ceil_div(h.M, DP_WAVES)), dim3(64 * DP_WAVES), s, d);
  Select sel{};
  sel.P = P;
  sel.M = h.M;
  if (e == hipSuccess) e = gather(h, u, sel, c.loss, nullptr, s);
  u.a.sid = u.st.ids;
  u.a.ptr = ptr;
  u.a.tk = u.st.tk;
  if (e == hipSuccess) e = stats<true>(h, u.a, c.mem.keep != 0, s);
  if (e == hipSuccess)
    e = launch_kernel(distill_rows_kernel, rows_grid(h.M), dim3(XC_ROWS * XC_SLICES), s,
                      DistillRows{rows_args(h, c.mem, u, sel), c.K, ent, P, c.loss});
  return e;
}

hipError_t launch_policy_forward(const PolicyForward &c, hipStream_t s) {
  Setup u;
  hipError_t e = set_up(c.head, c.mem, 0, s, u);
  if (e != hipSuccess) return e;
  set_targets(u.a, c.y);
  Select sel{nullptr, c.y.target, c.y.wide, c.y.ignore, c.head.M, c.head.V, nullptr, 0, 0};
  e = gather(c.head, u, sel, c.loss, c.logp, s);
  if (e == hipSuccess) e = stats<false>(c.head, u.a, c.mem.keep != 0, s);
  TokenRows r{};
  r.r = rows_args(c.head, c.mem, u, sel);
  r.tlogit = u.a.tlogit;
  r.logp = c.logp;
  r.advantage = c.advantage;
  r.old_logp = c.old_logp;
  r.ref_logp = c.ref_logp;
  r.low = c.clip_low;
  r.high = c.clip_high;
  r.kl = c.kl_coef;
  r.loss = c.loss;
  if (e == hipSuccess)
    e = launch_kernel(token_rows_kernel<true>, rows_grid(c.head.M), dim3(XC_ROWS * XC_SLICES), s, r);
  return e;
}

hipError_t launch_preference_forward(const PreferenceForward &c, hipStream_t s) {
  Setup u;
  hipError_t e = set_up(c.head, c.mem, 0, s, u);
  if (e != hipSuccess) return e;
  set_targets(u.a, c.y);
  float *const rowlogp = reinterpret_cast<float *>(u.ws + u.lay.rowlogp);
  if (c.head.M > 0) {
    // without pairs there are no bounds, and no row is worked on
    Select sel{nullptr, c.y.target, c.y.wide, c.y.ignore, c.head.M, c.pairs > 0 ? c.head.V : 0, c.pairs > 0 ? c.starts : nullptr,
               c.starts64, 2 * c.pairs};
    e = gather(c.head, u, sel, nullptr, nullptr, s);
    if (e == hipSuccess) e = stats<false>(c.head, u.a, c.mem.keep != 0, s);
    TokenRows r{};
    r.r = rows_args(c.head, c.mem, u, sel);
    r.tlogit = u.a.tlogit;
    r.logp = rowlogp;
    if (e == hipSuccess)
      e = launch_kernel(token_rows_kernel<false>, rows_grid(c.head.M), dim3(XC_ROWS * XC_SLICES), s, r);
  }
  if (e == hipSuccess && c.pairs > 0)
    e = launch_kernel(preference_pairs_kernel, dim3((unsigned)c.pairs), dim3(PP_THREADS), s,
                      Pairs{c.starts, c.starts64, c.pairs, c.head.M, c.head.V, c.y.target, c.y.wide, c.y.ignore,
                            rowlogp, c.ref_logp, c.beta, c.margin, c.smoothing, c.average, c.loss, c.logp, u.st.coef,
                            u.st.own, u.st.up, u.st.inv});
  return e;
}

hipError_t launch_loss_backward(const LossBackward &c, hipStream_t s) {
  if (c.head.M == 0 || c.grad_loss == nullptr) {  // sums over no rows, or of zeros
    hipError_t e = hipSuccess;
    if (c.grad_hidden != nullptr && c.head.M > 0) e = zero_words(c.grad_hidden, c.head.M * c.head.H / 2, s);
    if (e == hipSuccess && c.grad_W != nullptr) e = zero_words(c.grad_W, c.head.V * c.head.H / 2, s);
    if (e == hipSuccess && c.grad_bias != nullptr) e = zero_words(c.grad_bias, c.head.V, s);
    return e;
  }
  return c.head.in_f16 ? backward<ET_F16>(c, s) : backward<ET_BF16>(c, s);
}

}  // namespace lmhead
