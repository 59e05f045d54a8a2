// embed.hip -- the embedding lookup out[m, :] = scale W[ids[m], :] and its
// gradient by sorted tokens, grad_W[v, :] = scale sum over {m : ids[m] = v}
// of grad_out[m, :].
//
// Ids outside [0, V) (and, in the gradient, the padding id) have a row of
// zeros and no gradient, so a vocabulary shard can be handed ids - v0.
//
// Both are bound by bytes. The gradient's fixed cost is finding each token's
// positions: the positions are put in the order of (id, position), so that
// the rows of one id follow each other and are summed at fp32 in ascending
// position, the same bits every run; no float atomics. A dense gradient is
// first filled with zeros by work-groups that ride along in the sorting
// kernels' launches: the sort needs few CUs and the fill is what takes long.
//
// Measured: the lookup of 8192 rows of H = 4096 23 µs (134 MB, 5.8 TB/s; a
// device copy reaches 4.7-5.0). Its gradient, V = 128256: 195 µs dense (1.12 GB,
// 5.7 TB/s; the fill alone is 154), 59 µs added to a gradient that is there.
#include "kstep.hpp"
#include "ops_launch.hpp"

namespace lmhead {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

__device__ __forceinline__ int64_t id_at(const void *ids, int ids64, int64_t m) {
  return ids64 ? static_cast<const int64_t *>(ids)[m] : (int64_t)static_cast<const int32_t *>(ids)[m];
}

template <bool F16>
__device__ __forceinline__ float from16(uint32_t bits) {
  if constexpr (F16)
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  else
    return __builtin_bit_cast(float, bits << 16);
}
template <bool F16>
__device__ __forceinline__ uint32_t to16(float f) {
  if constexpr (F16)
    return out_bits16<_Float16>(f);
  else
    return bf16_rne(f);
}

// ---------------------------------------------------------------------------
// Lookup: 16 bytes (8 elements) per thread and step, EL_STEPS rows' pieces in
// flight per thread. The product is taken at fp32 and rounded once.
// ---------------------------------------------------------------------------
constexpr int EL_THREADS = 256, EL_STEPS = 4;

template <bool F16, typename Index>
__global__ __launch_bounds__(EL_THREADS) void embed_kernel(const void *ids, int ids64, Index pieces,
                                                           Index ppr, const uint16_t *__restrict__ W,
                                                           int64_t V, float scale,
                                                           uint16_t *__restrict__ out) {
  const Index p0 = (Index)group_number() * (EL_THREADS * EL_STEPS) + threadIdx.x;
  u32x4 v[EL_STEPS];
#pragma unroll
  for (int s = 0; s < EL_STEPS; ++s) {
    const Index p = p0 + s * EL_THREADS;
    v[s] = u32x4{0, 0, 0, 0};
    if (p < pieces) {
      const Index m = p / ppr, c = p - m * ppr;
      const int64_t id = id_at(ids, ids64, m);
      if (id >= 0 && id < V)
        v[s] = *reinterpret_cast<const u32x4 *>(W + ((int64_t)id * ppr + c) * 8);
    }
  }
#pragma unroll
  for (int s = 0; s < EL_STEPS; ++s) {
    const Index p = p0 + s * EL_THREADS;
    if (p >= pieces) break;
    if (scale != 1.0f) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[s][k] = to16<F16>(__fmul_rn(scale, from16<F16>(v[s][k] & 0xFFFFu))) |
                  (to16<F16>(__fmul_rn(scale, from16<F16>(v[s][k] >> 16))) << 16);
    }
    *reinterpret_cast<u32x4 *>(out + (int64_t)p * 8) = v[s];
  }
}

// ---------------------------------------------------------------------------
// Sorting the positions by (id, position).
// ---------------------------------------------------------------------------

// The key of position m: its id, or V where it has no gradient.
__device__ __forceinline__ uint32_t key_of(const void *ids, int ids64, int64_t m, int64_t V,
                                           int64_t padding) {
  const int64_t id = id_at(ids, ids64, m);
  return id >= 0 && id < V && id != padding ? (uint32_t)id : (uint32_t)V;
}

// A slice of the zero fill, done by the work-groups behind the sorting ones.
struct Fill {
  u32x4 *p;        // 16-byte words [from, to)
  int64_t from, to;
  int sort_blocks; // work-groups of the launch that sort
};
// A thread writes one piece: small work-groups in order fill fastest (1.05 GB
// alone: 256 threads of one piece 155 µs, of four 176, 1024 of sixteen 171).
// The stores are not kept in the caches: nothing reads the zeros, and what does
// not displace the rows to be summed leaves them there. In the sorting launches
// the work-groups have 1024 threads all the same (30011 positions, V = 151936, H
// = 2048, the whole call: one piece a thread 145 µs, four 160, sixteen 152; V =
// 262144, H = 8192 1030, 1186, 1124; V = 32000, H = 2048 77, 78, 76).
__device__ __forceinline__ void do_fill(const Fill &f) {
  const int64_t p = f.from + (group_number() - f.sort_blocks) * blockDim.x + threadIdx.x;
  if (p < f.to) __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, f.p + p);
}
int64_t fill_blocks(const Fill &f, int threads) { return f.to > f.from ? ceil_div(f.to - f.from, threads) : 0; }

// Few positions: a position's place is the number of smaller (id, position)
// pairs, counted against every other. A work-group ranks 64 positions, its
// waves splitting the others; M^2 comparisons are spread over the chip in one
// launch. Sixteen waves where the ranking is all there is to wait for; four
// under a dense gradient's fill, which takes longer than either and is faster
// from small work-groups. How few: see ranks().
template <int WAVES, int CHUNK>
__global__ __launch_bounds__(64 * WAVES) void embed_rank_kernel(const void *ids, int ids64, int M, int64_t V,
                                                                int64_t padding, uint32_t *__restrict__ keys,
                                                                uint32_t *__restrict__ order, Fill f) {
  if (group_number() >= f.sort_blocks) return do_fill(f);
  __shared__ alignas(16) uint32_t sk[CHUNK];
  __shared__ uint32_t cnt[WAVES][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + lane;
  const uint32_t ki = i < M ? key_of(ids, ids64, i, V, padding) : 0u;
  uint32_t n = 0;
  for (int c0 = 0; c0 < M; c0 += CHUNK) {
    const int cn = M - c0 < CHUNK ? M - c0 : CHUNK;
    __syncthreads();
    for (int j = threadIdx.x; j < CHUNK; j += 64 * WAVES)
      sk[j] = j < cn ? key_of(ids, ids64, c0 + j, V, padding) : 0xFFFFFFFFu;
    __syncthreads();
    // this wave's positions of the chunk, four at a time; positions before i
    // count with an equal id, later ones do not
    constexpr int PER = CHUNK / WAVES;
    const int j0 = wave * PER;
    const int jn = cn - j0 < PER ? (cn - j0 + 3) & ~3 : PER;
    const int i0 = blockIdx.x * 64;
    for (int j = 0; j < jn; j += 4) {
      const u32x4 k = *reinterpret_cast<const u32x4 *>(&sk[j0 + j]);
      const int p = c0 + j0 + j;
      if (p + 3 < i0 || p >= i0 + 64) {  // all four before, or all after, the 64
        const uint32_t lim = ki + (p < i0 ? 1u : 0u);
#pragma unroll
        for (int e = 0; e < 4; ++e) n += k[e] < lim ? 1u : 0u;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) n += k[e] < ki + (p + e < i ? 1u : 0u) ? 1u : 0u;
      }
    }
  }
  cnt[wave][lane] = n;
  __syncthreads();
  if (wave == 0 && i < M) {
    uint32_t r = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) r += cnt[w][lane];
    keys[r] = ki;
    order[r] = (uint32_t)i;
  }
}

// Else a stable radix sort, least digit first. A work-group owns a
// contiguous tile of positions, each of its 16 waves a contiguous part of it.
// embed_count_kernel counts the tile's digits; embed_scatter_kernel finds the
// tile's and its waves' first place for each digit from all tiles' counts, and
// places the positions in order (lanes of a wave with equal digits find each
// other by ballots).
constexpr int RX_THREADS = 1024, RX_WAVES = 16, RX_BITS = 9, RX_BINS = 1 << RX_BITS, RX_TILES = 256;

struct RadixArgs {
  const void *ids;           // first pass: keys come from here
  int ids64;
  int64_t V, padding;
  const uint32_t *keys_in, *order_in;  // later passes
  uint32_t *keys_out, *order_out;
  uint32_t *counts;          // [tiles][RX_BINS]
  int64_t M, tile;
  int tiles, shift, first;
};
__device__ __forceinline__ uint32_t radix_key(const RadixArgs &a, int64_t m) {
  return a.first ? key_of(a.ids, a.ids64, m, a.V, a.padding) : a.keys_in[m];
}

__global__ __launch_bounds__(RX_THREADS) void embed_count_kernel(RadixArgs a, Fill f) {
  if (group_number() >= f.sort_blocks) return do_fill(f);
  __shared__ uint32_t h[RX_BINS];
  for (int d = threadIdx.x; d < RX_BINS; d += RX_THREADS) h[d] = 0;
  __syncthreads();
  const int64_t m0 = blockIdx.x * a.tile, m1 = m0 + a.tile < a.M ? m0 + a.tile : a.M;
  for (int64_t m = m0 + threadIdx.x; m < m1; m += RX_THREADS)
    atomicAdd(&h[(radix_key(a, m) >> a.shift) & (RX_BINS - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < RX_BINS; d += RX_THREADS) a.counts[(int64_t)blockIdx.x * RX_BINS + d] = h[d];
}

__global__ __launch_bounds__(RX_THREADS) void embed_scatter_kernel(RadixArgs a, Fill f) {
  if (group_number() >= f.sort_blocks) return do_fill(f);
  __shared__ uint32_t at[RX_WAVES][RX_BINS];  // next place of (wave, digit)
  __shared__ uint32_t part[2][RX_BINS], sum[RX_BINS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // per digit: positions of earlier tiles, and of all tiles (two threads per
  // digit, the even and the odd tiles)
  {
    const int d = tid % RX_BINS, half = tid / RX_BINS;
    uint32_t before = 0, all = 0;
    for (int t = half; t < a.tiles; t += 2) {
      const uint32_t c = a.counts[(int64_t)t * RX_BINS + d];
      all += c;
      if (t < (int)blockIdx.x) before += c;
    }
    part[half][d] = all;
    __syncthreads();
    if (half == 0) sum[d] = part[0][d] + part[1][d];
    __syncthreads();
    // exclusive prefix of the totals over the digits
    for (int s = 1; s < RX_BINS; s <<= 1) {
      const uint32_t v = half == 0 && d >= s ? sum[d - s] : 0u;
      __syncthreads();
      if (half == 0) sum[d] += v;
      __syncthreads();
    }
    const uint32_t first = d > 0 ? sum[d - 1] : 0u;
    __syncthreads();
    part[half][d] = before;
    __syncthreads();
    if (half == 0) sum[d] = first + part[0][d] + part[1][d];
    for (int e = tid; e < RX_WAVES * RX_BINS; e += RX_THREADS) at[e / RX_BINS][e % RX_BINS] = 0;
    __syncthreads();
  }
  const int64_t m0 = blockIdx.x * a.tile, m1 = m0 + a.tile < a.M ? m0 + a.tile : a.M;
  const int64_t per = (a.tile + RX_WAVES * 64 - 1) / (RX_WAVES * 64) * 64;
  const int64_t w0 = m0 + wave * per, w1 = w0 + per < m1 ? w0 + per : m1;
  for (int64_t m = w0 + lane; m < w1; m += 64)
    atomicAdd(&at[wave][(radix_key(a, m) >> a.shift) & (RX_BINS - 1)], 1u);
  __syncthreads();
  if (tid < RX_BINS) {  // counts -> first places, wave by wave
    uint32_t p = sum[tid];
#pragma unroll
    for (int w = 0; w < RX_WAVES; ++w) {
      const uint32_t c = at[w][tid];
      at[w][tid] = p;
      p += c;
    }
  }
  __syncthreads();
  for (int64_t b = w0; b < w1; b += 64) {
    const int64_t m = b + lane;
    const bool ok = m < w1;
    const uint32_t key = ok ? radix_key(a, m) : 0u;
    const uint32_t d = (key >> a.shift) & (RX_BINS - 1);
    uint64_t same = __ballot(ok);
#pragma unroll
    for (int bit = 0; bit < RX_BITS; ++bit) {
      const uint64_t has = __ballot((d >> bit) & 1u);
      same &= ((d >> bit) & 1u) ? has : ~has;
    }
    if (ok) {
      const int r = __popcll(same & ((1ull << lane) - 1));
      const uint32_t place = at[wave][d] + r;
      __builtin_amdgcn_wave_barrier();
      if (r == 0) at[wave][d] += (uint32_t)__popcll(same);
      a.keys_out[place] = key;
      a.order_out[place] = a.first ? (uint32_t)m : a.order_in[m];
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------------------
// Summing. The sorted positions are cut into tiles; a work-group sums a tile's
// rows over 1024 columns, 8 per thread. An id whose positions all lie in the
// tile is written at once; the sums of an id that began in an earlier tile
// (slot 0) or goes on in the next (slot 1) go to the workspace, and
// embed_join_kernel adds those of an id in tile order.
// ---------------------------------------------------------------------------
constexpr int ES_THREADS = 128, ES_COLS = ES_THREADS * 8, ES_AHEAD = 8, ES_LIST = 256;

struct SumArgs {
  const uint32_t *keys, *order;
  int64_t M, H, V;
  int tile;                 // positions per tile
  const uint16_t *grad_out; // [M, H]
  float scale;
  int accumulate;
  uint16_t *grad_W;         // [V, H]
  float *part;              // [tiles][2][H]
};

template <bool F16, bool ACC>
__device__ __forceinline__ void write_row(const SumArgs &a, int64_t v, int64_t c, const float (&s)[8]) {
  u32x4 *const dst = reinterpret_cast<u32x4 *>(a.grad_W + v * a.H + c);
  u32x4 o = u32x4{0, 0, 0, 0};
  if constexpr (ACC) o = *dst;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo = __fmul_rn(a.scale, s[2 * k]), hi = __fmul_rn(a.scale, s[2 * k + 1]);
    if constexpr (ACC) {
      lo = __fadd_rn(from16<F16>(o[k] & 0xFFFFu), lo);
      hi = __fadd_rn(from16<F16>(o[k] >> 16), hi);
    }
    o[k] = to16<F16>(lo) | (to16<F16>(hi) << 16);
  }
  *dst = o;
}

template <bool F16, bool ACC>
__global__ __launch_bounds__(ES_THREADS) void embed_sum_kernel(SumArgs a) {
  // the tile's keys and positions, one load each for all of them, with the
  // keys before the first and after the last (ES_LIST positions at a time)
  __shared__ uint32_t sk[ES_LIST + 2], so[ES_LIST];
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int64_t t1 = t0 + a.tile < a.M ? t0 + a.tile : a.M;
  const int64_t c = (int64_t)blockIdx.y * ES_COLS + 8 * threadIdx.x;
  const bool on = c < a.H;
  const uint16_t *const src = a.grad_out + (on ? c : 0);
  const uint32_t none = (uint32_t)a.V;
  float s[8] = {};
  bool head = false;
  for (int64_t e0 = t0; e0 < t1; e0 += ES_LIST) {
    const int n = (int)(t1 - e0 < ES_LIST ? t1 - e0 : ES_LIST);
    __syncthreads();
    for (int i = threadIdx.x; i < ES_LIST + 2; i += ES_THREADS) {
      const int64_t e = e0 + i - 1;
      sk[i] = e >= 0 && e < a.M ? a.keys[e] : none + 1;
      if (i >= 1 && i <= ES_LIST) so[i - 1] = i <= n ? a.order[e] : 0u;
    }
    __syncthreads();
    if (e0 == t0) head = sk[0] == sk[1];  // the first id began in an earlier tile
    if (sk[1] == none) return;            // the ids without a gradient come last
    for (int i0 = 0; i0 < n; i0 += ES_AHEAD) {
      // loads and additions without conditions (past the tile: position 0,
      // masked to zeros): a load that only a branch uses is moved into it, and
      // a register that a load may or may not have written is waited for,
      // either of which puts the loads one behind the other
      u32x4 v[ES_AHEAD];
#pragma unroll
      for (int k = 0; k < ES_AHEAD; ++k)
        v[k] = *reinterpret_cast<const u32x4 *>(src + (int64_t)__builtin_amdgcn_readfirstlane(so[i0 + k]) * a.H);
#pragma unroll
      for (int k = 0; k < ES_AHEAD; ++k) {
        const int i = i0 + k;
        const uint32_t key = __builtin_amdgcn_readfirstlane(sk[i + 1]);
        const bool valid = i < n && key < none;
        const uint32_t mask = valid ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t w = v[k][q] & mask;
          s[2 * q] = __fadd_rn(s[2 * q], from16<F16>(w & 0xFFFFu));
          s[2 * q + 1] = __fadd_rn(s[2 * q + 1], from16<F16>(w >> 16));
        }
        const bool ends = __builtin_amdgcn_readfirstlane(sk[i + 2]) != key;
        if (valid && (ends || e0 + i + 1 >= t1)) {  // the id's last position, or the tile's
          if (on) {
            if (head || !ends) {
              float *const p = a.part + ((int64_t)blockIdx.x * 2 + (head ? 0 : 1)) * a.H + c;
              *reinterpret_cast<f32x4 *>(p) = f32x4{s[0], s[1], s[2], s[3]};
              *reinterpret_cast<f32x4 *>(p + 4) = f32x4{s[4], s[5], s[6], s[7]};
            } else {
              write_row<F16, ACC>(a, key, c, s);
            }
          }
          head = false;
#pragma unroll
          for (int q = 0; q < 8; ++q) s[q] = 0.0f;
        }
      }
    }
  }
}

// One work-group per tile in which an id begins that goes on: EJ_GROUPS groups
// of 64 lanes sum contiguous runs of the id's tiles (4 columns per lane),
// joined in order. Most tiles have none, so what a work-group costs that
// finds nothing to do counts: three loads in flight together.
constexpr int EJ_GROUPS = 8, EJ_LANES = 64, EJ_COLS = 4 * EJ_LANES;
template <bool F16>
__global__ __launch_bounds__(EJ_GROUPS * EJ_LANES) void embed_join_kernel(SumArgs a, int tiles) {
  const int t0 = blockIdx.x;
  const int64_t e0 = (int64_t)t0 * a.tile, last = e0 + a.tile;  // last: the next tile's first position (< M)
  const uint32_t key = a.keys[last - 1], next = a.keys[last], prev = a.keys[e0 > 0 ? e0 - 1 : 0];
  // an id that began in an earlier tile belongs to that one
  if (key == (uint32_t)a.V || next != key || (e0 > 0 && prev == key)) return;
  // the id's last tile: the largest t whose first position has this key
  int lo = t0 + 1, hi = tiles - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.keys[(int64_t)mid * a.tile] == key)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int n = lo - t0 + 1;  // partial sums: slot 1 of t0 (it does not begin earlier), slot 0 of the rest
  const int lane = threadIdx.x % EJ_LANES, g = threadIdx.x / EJ_LANES;
  const int64_t c = (int64_t)blockIdx.y * EJ_COLS + 4 * lane;
  const int per = (n + EJ_GROUPS - 1) / EJ_GROUPS;
  const int k0 = g * per, k1 = k0 + per < n ? k0 + per : n;
  f32x4 s = zero4();
  if (c < a.H) {
    constexpr int AH = 8;
    for (int k = k0; k < k1; k += AH) {
      f32x4 v[AH];
#pragma unroll
      for (int q = 0; q < AH; ++q) {
        const int kk = k + q < k1 ? k + q : k1 - 1;  // (a load without a condition, as above)
        v[q] = *reinterpret_cast<const f32x4 *>(a.part + ((int64_t)(t0 + kk) * 2 + (kk == 0 ? 1 : 0)) * a.H + c);
        if (k + q >= k1) v[q] = zero4();
      }
#pragma unroll
      for (int q = 0; q < AH; ++q)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] = __fadd_rn(s[x], v[q][x]);
    }
  }
  __shared__ f32x4 sh[EJ_GROUPS][EJ_LANES];
  sh[g][lane] = s;
  __syncthreads();
  if (g != 0 || c >= a.H) return;
#pragma unroll
  for (int w = 1; w < EJ_GROUPS; ++w)
#pragma unroll
    for (int x = 0; x < 4; ++x) s[x] = __fadd_rn(s[x], sh[w][lane][x]);
  uint16_t *const dst = a.grad_W + (int64_t)key * a.H + c;
  u32x2 o = u32x2{0, 0};
  if (a.accumulate) o = *reinterpret_cast<const u32x2 *>(dst);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float x = __fmul_rn(a.scale, s[2 * k]), y = __fmul_rn(a.scale, s[2 * k + 1]);
    if (a.accumulate) {
      x = __fadd_rn(from16<F16>(o[k] & 0xFFFFu), x);
      y = __fadd_rn(from16<F16>(o[k] >> 16), y);
    }
    o[k] = to16<F16>(x) | (to16<F16>(y) << 16);
  }
  *reinterpret_cast<u32x2 *>(dst) = o;
}

// Positions per tile: enough tiles to fill the chip, at most 512 (their partial
// sums are read back), at least 16 positions.
int sum_tile(int64_t M) {
  const int64_t t = ceil_div(M, 512);
  return (int)(t < 16 ? 16 : t);
}

// Which sort. Ranking is one launch against two per nine bits of the ids, and
// 8 ns per position while each work-group has a place of its own on the chip.
// Added to a gradient (µs, ranked / radix): H = 4096, V = 128256 4500 positions
// 46 / 47, 6144 53.5 / 51.9, 8192 63 / 59; H = 2048, V = 64000 37.4 / 38.3, 42.8 /
// 41.3, 49.9 / 46.5. Dense, it is hidden as long as the fill takes longer, about
// M ranks in the time of 30000 M elements (the whole call, V x H): 64000 x 2048
// 3500 positions 58 / 62, 4500 71 / 63; 128256 x 2048 8192 105 / 114, 10240 121 /
// 117; 128256 x 4096 16384 209 / 235, 32768 336 / 258; 32000 x 2048 2048 36 / 41,
// 8192 87 / 52; and up to 2048 positions whatever the table: 4096 x 256 29.5 / 31,
// at 4096 positions 43 / 32.
constexpr int64_t RANK_ALWAYS = 2048, RANK_ADDED = 5120, RANK_DENSE = 16384, RANK_FILL = 30000;
bool ranks(int64_t M, int64_t H, int64_t V, bool accumulate) {
  if (accumulate) return M <= RANK_ADDED;
  return M <= RANK_ALWAYS || (M <= RANK_DENSE && M * RANK_FILL <= V * H);
}

struct Plan {
  int64_t keys, order, keys2, order2, counts, part, bytes;
};
Plan plan(int64_t M, int64_t H) {
  Plan p;
  const int64_t list = align256(4 * M);
  p.keys = 0;
  p.order = list;
  const bool radix = M > RANK_ALWAYS;  // for some table, or added
  p.keys2 = 2 * list;
  p.order2 = p.keys2 + (radix ? list : 0);
  p.counts = p.order2 + (radix ? list : 0);
  p.part = p.counts + (radix ? (int64_t)RX_TILES * RX_BINS * 4 : 0);
  p.bytes = p.part + align256(ceil_div(M, sum_tile(M)) * 2 * H * 4);
  return p;
}

}  // namespace

int64_t embed_backward_bytes(int64_t M, int64_t H) { return M > 0 ? plan(M, H).bytes : 0; }

hipError_t launch_embed(const EmbedForward &c, hipStream_t s) {
  const int64_t ppr = c.H / 8, pieces = c.M * ppr;
  const dim3 grid = numbered_grid(ceil_div(pieces, EL_THREADS * EL_STEPS));
  const uint16_t *W = static_cast<const uint16_t *>(c.W);
  uint16_t *out = static_cast<uint16_t *>(c.out);
  // 32-bit piece numbers where they fit (a 64-bit division per piece costs
  // more than the piece's load)
  if (pieces < ((int64_t)1 << 32) - EL_THREADS * EL_STEPS) {
    auto k = c.in_f16 ? embed_kernel<true, uint32_t> : embed_kernel<false, uint32_t>;
    return launch_kernel(k, grid, dim3(EL_THREADS), s, c.ids, c.ids64, (uint32_t)pieces, (uint32_t)ppr, W, c.V,
                         c.scale, out);
  }
  auto k = c.in_f16 ? embed_kernel<true, uint64_t> : embed_kernel<false, uint64_t>;
  return launch_kernel(k, grid, dim3(EL_THREADS), s, c.ids, c.ids64, (uint64_t)pieces, (uint64_t)ppr, W, c.V,
                       c.scale, out);
}

namespace {
hipError_t launch_rank(const EmbedBackward &c, uint32_t *keys, uint32_t *order, const Fill &f, hipStream_t s) {
  const int waves = c.accumulate ? 16 : 4;
  auto k = c.accumulate ? embed_rank_kernel<16, 8192> : embed_rank_kernel<4, 2048>;
  return launch_kernel(k, numbered_grid(f.sort_blocks + fill_blocks(f, 64 * waves)), dim3(64 * waves), s,
                       c.ids, c.ids64, (int)c.M, c.V, c.padding, keys, order, f);
}
}  // namespace

hipError_t launch_embed_backward(const EmbedBackward &c, hipStream_t s) {
  const int64_t words = c.V * c.H / 8;  // 16-byte words of grad_W
  Fill f{static_cast<u32x4 *>(c.grad_W), 0, c.accumulate ? 0 : words, 0};
  if (c.M == 0) {
    if (c.accumulate) return hipSuccess;
    return launch_rank(c, nullptr, nullptr, f, s);
  }
  const Plan pl = plan(c.M, c.H);
  uint8_t *const ws = static_cast<uint8_t *>(c.workspace);
  uint32_t *keys = reinterpret_cast<uint32_t *>(ws + pl.keys);
  uint32_t *order = reinterpret_cast<uint32_t *>(ws + pl.order);
  hipError_t e = hipSuccess;
  if (ranks(c.M, c.H, c.V, c.accumulate)) {
    f.sort_blocks = (int)ceil_div(c.M, 64);
    e = launch_rank(c, keys, order, f, s);
  } else {
    RadixArgs a;
    a.ids = c.ids;
    a.ids64 = c.ids64;
    a.V = c.V;
    a.padding = c.padding;
    a.counts = reinterpret_cast<uint32_t *>(ws + pl.counts);
    a.M = c.M;
    a.tile = ceil_div(c.M, RX_TILES) < RX_THREADS ? RX_THREADS : ceil_div(c.M, RX_TILES);
    a.tiles = (int)ceil_div(c.M, a.tile);
    int bits = 1;
    while (((int64_t)1 << bits) <= c.V) ++bits;  // keys 0 .. V
    const int passes = (bits + RX_BITS - 1) / RX_BITS;
    uint32_t *ko[2] = {keys, reinterpret_cast<uint32_t *>(ws + pl.keys2)};
    uint32_t *oo[2] = {order, reinterpret_cast<uint32_t *>(ws + pl.order2)};
    const int64_t all = f.to;
    for (int p = 0; p < passes && e == hipSuccess; ++p) {
      const int to = (passes - 1 - p) & 1;  // the last pass writes (keys, order)
      a.first = p == 0;
      a.shift = p * RX_BITS;
      a.keys_in = ko[1 - to];
      a.order_in = oo[1 - to];
      a.keys_out = ko[to];
      a.order_out = oo[to];
      for (int half = 0; half < 2 && e == hipSuccess; ++half) {
        const int part = 2 * p + half;
        f.from = all * part / (2 * passes);
        f.to = all * (part + 1) / (2 * passes);
        f.sort_blocks = a.tiles;
        e = launch_kernel(half == 0 ? embed_count_kernel : embed_scatter_kernel,
                          numbered_grid(a.tiles + fill_blocks(f, RX_THREADS)), dim3(RX_THREADS), s, a, f);
      }
    }
  }
  if (e != hipSuccess) return e;
  SumArgs a;
  a.keys = keys;
  a.order = order;
  a.M = c.M;
  a.H = c.H;
  a.V = c.V;
  a.tile = sum_tile(c.M);
  a.grad_out = static_cast<const uint16_t *>(c.grad_out);
  a.scale = c.scale;
  a.accumulate = c.accumulate;
  a.grad_W = static_cast<uint16_t *>(c.grad_W);
  a.part = reinterpret_cast<float *>(ws + pl.part);
  const int tiles = (int)ceil_div(c.M, a.tile);
  auto sum = c.in_f16 ? (c.accumulate ? embed_sum_kernel<true, true> : embed_sum_kernel<true, false>)
                      : (c.accumulate ? embed_sum_kernel<false, true> : embed_sum_kernel<false, false>);
  e = launch_kernel(sum,
                    dim3((unsigned)tiles, (unsigned)ceil_div(c.H, ES_COLS)), dim3(ES_THREADS), s, a);
  if (e != hipSuccess || tiles < 2) return e;
  return launch_kernel(c.in_f16 ? embed_join_kernel<true> : embed_join_kernel<false>,
                       dim3((unsigned)(tiles - 1), (unsigned)ceil_div(c.H, EJ_COLS)), dim3(EJ_GROUPS * EJ_LANES), s, a,
                       tiles);
}

}  // namespace lmhead
