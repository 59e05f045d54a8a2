// xent_core.hpp -- what the kernels of the head's losses share (xent.hip,
// losses.hip; internal): the logits' products over mma256.hpp, the folds of
// softmax statistics, G = dL/dt of a piece of the vocabulary, and the two
// products made of G.
#pragma once

#include "mma256.hpp"
#include "ops_launch.hpp"

namespace lmhead {

namespace {

constexpr float NEG_INF = -__builtin_inff();
constexpr float LOG2E = 1.44269504088896340736f;  // log2 e

// e^(t - ref) by the hardware's 2^x (below 2^-126: 0). The factor log2 e is
// applied to the difference, not to t and ref: a finite t stays finite (a mask
// of the type's lowest value times log2 e would be -inf), and the rounding of
// the product is one of the difference. It costs a multiplication per logit.
__device__ __forceinline__ float exp_diff(float t, float ref) {
  return __builtin_amdgcn_exp2f(__fmul_rn(LOG2E, __fsub_rn(t, ref)));
}

// The row's target column, or -1.
__device__ __forceinline__ int64_t target_of(const void *target, int target64, int64_t m,
                                             int64_t ignore, int64_t V) {
  const int64_t y = target64 ? static_cast<const int64_t *>(target)[m]
                             : (int64_t)static_cast<const int32_t *>(target)[m];
  return y != ignore && y >= 0 && y < V ? y : -1;
}

// hidden W^T of tile (m0, n0): both operands K-inner, the K order of korder.hpp.
__device__ __forceinline__ MmJob logits_job(const uint8_t *hidden, const uint8_t *W, int64_t M, int64_t H,
                                            int64_t V, int64_t m0, int64_t n0) {
  const int64_t rb = H * 2, rows = M - m0, cols = V - n0;
  return MmJob{{hidden + m0 * rb, (uint32_t)rb, (int32_t)(rows < MM_T ? rows : MM_T), (uint32_t)rb},
               {W + n0 * rb, (uint32_t)rb, (int32_t)(cols < MM_T ? cols : MM_T), (uint32_t)rb},
               (int32_t)((rb + MM_STAGE_BYTES - 1) / MM_STAGE_BYTES),
               (int32_t)(korder_start(n0, H) / 64)};
}

// A lane's place in its wave's output.
struct LanePlace {
  int li, lg, wm, wn;
  __device__ __forceinline__ LanePlace() {
    const int tid = mm_tid(), lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    li = lane & 15;
    lg = lane >> 4;
    wm = wave >> 2;
    wn = wave & 3;
  }
};

// The biases of the lane's eight columns in half y; columns that are not there
// get -inf, so that their probability is 0.
template <int ET>
__device__ __forceinline__ void column_bias(const float *bias, int64_t V, int64_t n0, const LanePlace &at, int y,
                                            float (&b)[2][4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) b[j][q] = 0.0f;
  // 32-bit columns of the tile: 64-bit ones cost registers that the epilogues lack
  const int32_t cols = (int32_t)(V - n0 < MM_T ? V - n0 : MM_T);
  if (bias != nullptr || cols < MM_T) {
    const float *const first = bias != nullptr ? bias + n0 : nullptr;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t c = MmTile<ET>::col(at.wn, at.lg, y, j) + q;
        b[j][q] = (int32_t)c < cols ? (first != nullptr ? first[c] : 0.0f) : NEG_INF;
      }
  }
}

// Whether column c of the tile is one of the lane's in half y (columns y 128 +
// wn 32 + j 16 + 4 lg + q). Few are, so what is done for a row's target is
// skipped by nearly every wave instead of being a comparison per logit.
template <int ET>
__device__ __forceinline__ bool has_column(const LanePlace &at, int y, int32_t c) {
  return (c >> 5) == y * 4 + at.wn && ((c >> 2) & 3) == at.lg;
}

// Adds e = {largest t, sum of exp(t - largest)} of some columns to a row's {m, s}.
constexpr int XC_ROWS = 16, XC_SLICES = 64;  // rows per work-group of the fold, threads per row
__device__ __forceinline__ void fold_stat(float &m, float &s, float2 e) {
  const float n = fmaxf(m, e.x);
  const float a = s == 0.0f ? 0.0f : __fmul_rn(s, exp_diff(m, n));
  const float b = e.y == 0.0f ? 0.0f : __fmul_rn(e.y, exp_diff(e.x, n));
  s = __fadd_rn(a, b);
  m = n;
}

// What the epilogue needs of a row: G = a e^(t - lse) - b [v = y].
struct alignas(16) RowCoef {
  float a, b, lse;
  int32_t y;        // target column, or -1
};

struct XentBwdArgs {
  const uint8_t *hidden, *W;
  int64_t M, H, V;
  float alpha;
  const float *bias;
  const RowCoef *rows;
  const float *scale;  // {f, 1 / f}
  int64_t v0, np;      // this piece's first column and its columns (a multiple of 256)
  int64_t ldg;         // columns of a row of G in memory
  uint8_t *G;          // [M, ldg], 16 bits
  float *colpart;      // [row tile][ldg] column sums of G, or nullptr
  float *dh;           // [splits][M, H] fp32 sums
  int64_t ksplit;      // columns per split of G W
  int first;           // first piece: dh is written, not added to
  uint16_t *dw;        // [V, H]
};

// G of one piece; DB: and its column sums. APART: 0 in the place of a row's target, whose
// entry is in the column sums only.
template <int ET, bool DB, bool APART = false>
struct XentGrad {
  XentBwdArgs p;
  u32x4 *epi;
  int64_t nmt, ngt;

  __device__ __forceinline__ int64_t tiles() const { return nmt * ngt; }
  __device__ __forceinline__ MmJob job(int32_t t) const {
    int64_t mt, gt;
    mm_tile_at(t, nmt, ngt, mt, gt);
    return logits_job(p.hidden, p.W, p.M, p.H, p.V, mt * MM_T, p.v0 + gt * MM_T);
  }
  __device__ __forceinline__ void epilogue(MmTile<ET> &tile, int32_t t) const {
    int64_t mt, gt;
    mm_tile_at(t, nmt, ngt, mt, gt);
    const int64_t m0 = mt * MM_T, g0 = gt * MM_T, n0 = p.v0 + g0;
    const LanePlace at;
    const int64_t rows = p.M - m0 < MM_T ? p.M - m0 : MM_T;
    RowCoef rc[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + MmTile<ET>::row(at.wm, at.li, x, i);
        // e^-inf = 0 in rows past the end, and where the whole row is -inf
        rc[x][i] = m < p.M ? p.rows[m] : RowCoef{0.0f, 0.0f, __builtin_inff(), -1};
        if (rc[x][i].lse == NEG_INF) rc[x][i].lse = 0.0f;
        rc[x][i].y = rc[x][i].y < 0 ? -1 : rc[x][i].y - (int32_t)n0;
      }
    MmParts parts{epi, 0};
    const rsrc_t rs = mm_out_rsrc(p.G + (m0 * p.ldg + g0) * 2, p.ldg * 2, rows, 512);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float bias[2][4], colsum[2][4] = {};
      column_bias<ET>(p.bias, p.V, n0, at, y, bias);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int ip = 0; ip < 2; ++ip) {
#pragma unroll
          for (int i = 2 * ip; i < 2 * ip + 2; ++i) {
            const RowCoef &r = rc[x][i];
            f32x4 g[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                g[j][q] = __fmul_rn(
                    r.a, exp_diff(__fmaf_rn(p.alpha, tile.c[x][y][i][j][q], bias[j][q]), r.lse));
            if (has_column<ET>(at, y, r.y))
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  if (r.y == MmTile<ET>::col(at.wn, at.lg, y, j) + q) {
                    g[j][q] = __fsub_rn(g[j][q], r.b);
                    if constexpr (APART) {
                      if constexpr (DB) colsum[j][q] = __fadd_rn(colsum[j][q], g[j][q]);
                      g[j][q] = 0.0f;
                    }
                  }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if constexpr (DB)
#pragma unroll
                for (int q = 0; q < 4; ++q) colsum[j][q] = __fadd_rn(colsum[j][q], g[j][q]);
              parts.put<ET>(at.wm, at.wn, at.li, at.lg, i, j, g[j]);
            }
          }
          parts.flush<LOAD_DEFAULT>(rs, y, x, ip, (uint32_t)p.ldg * 2, (int)rows, 512);
        }
      if constexpr (DB) {
        // column sums: 16 rows of a block by lane exchanges, then the two wave
        // rows, through the buffer whose turn it is
        float *const cs = reinterpret_cast<float *>(parts.buf());  // [2][128]
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float s = colsum[j][q];
            s = __fadd_rn(s, dpp<DPP_QUAD_SWAP1>(s));
            s = __fadd_rn(s, dpp<DPP_QUAD_SWAP2>(s));
            s = __fadd_rn(s, dpp<DPP_ROW_HALF_MIRROR>(s));
            s = __fadd_rn(s, dpp<DPP_ROW_MIRROR>(s));
            if (at.li == 0) cs[at.wm * 128 + MmTile<ET>::col(at.wn, at.lg, 0, j) + q] = s;
          }
        lds_barrier();
        ++parts.n;
        const int c = mm_tid();
        if (c < 128)
          p.colpart[mt * p.ldg + g0 + y * 128 + c] = __fmul_rn(p.scale[1], __fadd_rn(cs[c], cs[128 + c]));
      }
    }
  }
};

// G W of one piece, one split of its columns, into that split's fp32 sums.
template <int ET>
struct XentDHidden {
  XentBwdArgs p;
  int64_t nmt, nht, splits;

  __device__ __forceinline__ int64_t tiles() const { return nmt * nht * splits; }
  __device__ __forceinline__ void place(int32_t t, int64_t &m0, int64_t &h0, int64_t &sp) const {
    int64_t mt, ht;
    const uint32_t per = (uint32_t)(nmt * nht);
    sp = mm_uni((uint32_t)t / per);
    mm_tile_at((uint32_t)t - (uint32_t)sp * per, nmt, nht, mt, ht);
    m0 = mt * MM_T;
    h0 = ht * MM_T;
  }
  __device__ __forceinline__ MmJob job(int32_t t) const {
    int64_t m0, h0, sp;
    place(t, m0, h0, sp);
    const int64_t k0 = sp * p.ksplit, kn = p.np - k0 < p.ksplit ? p.np - k0 : p.ksplit;
    const int64_t rows = p.M - m0 < MM_T ? p.M - m0 : MM_T;
    // the weight rows present (G is 0 in columns past them)
    int64_t wrows = p.V - p.v0 - k0 < kn ? p.V - p.v0 - k0 : kn;
    if (wrows < 0) wrows = 0;
    const int64_t rb = p.H * 2;
    return MmJob{{p.G + (m0 * p.ldg + k0) * 2, (uint32_t)(p.ldg * 2), (int32_t)rows, (uint32_t)(kn * 2)},
                 {p.W + (wrows > 0 ? (p.v0 + k0) * rb : 0) + h0 * 2, (uint32_t)rb, (int32_t)wrows,
                  (uint32_t)((p.H - h0) * 2)},
                 (int32_t)(kn / 64), 0};
  }
  __device__ __forceinline__ void epilogue(MmTile<ET> &tile, int32_t t) const {
    int64_t m0, h0, sp;
    place(t, m0, h0, sp);
    const LanePlace at;
    const int64_t rows = p.M - m0 < MM_T ? p.M - m0 : MM_T;
    float *const out = p.dh + (sp * p.M + m0) * p.H + h0;
    const rsrc_t rs = make_rsrc(out, (uint32_t)(((rows - 1) * p.H + (p.H - h0 < MM_T ? p.H - h0 : MM_T)) * 4));
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = MmTile<ET>::row(at.wm, at.li, x, i);
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = MmTile<ET>::col(at.wn, at.lg, y, j);
            const bool ok = r < rows && h0 + c < p.H;
            const uint32_t off = ok ? (uint32_t)((r * p.H + c) * 4) : OFF_NONE;
            f32x4 v = tile.c[x][y][i][j];
            if (!p.first) {
              const f32x4 o = __builtin_bit_cast(f32x4, load16(rs, off, 0));
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = __fadd_rn(o[q], v[q]);
            }
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, off, 0, LOAD_DEFAULT);
          }
      }
  }
};

// G^T hidden of one piece: its rows of grad_W.
template <int ET>
struct XentDWeight {
  XentBwdArgs p;
  u32x4 *epi;
  int64_t ngt, nht;

  __device__ __forceinline__ int64_t tiles() const { return ngt * nht; }
  __device__ __forceinline__ MmJob job(int32_t t) const {
    int64_t gt, ht;
    mm_tile_at(t, ngt, nht, gt, ht);
    const int64_t g0 = gt * MM_T, h0 = ht * MM_T;
    return MmJob{{p.G + g0 * 2, (uint32_t)(p.ldg * 2), (int32_t)p.M, (uint32_t)((p.ldg - g0) * 2)},
                 {p.hidden + h0 * 2, (uint32_t)(p.H * 2), (int32_t)p.M, (uint32_t)((p.H - h0) * 2)},
                 (int32_t)(p.M > 0 ? (p.M + 63) / 64 : 1), 0};
  }
  __device__ __forceinline__ void epilogue(MmTile<ET> &tile, int32_t t) const {
    int64_t gt, ht;
    mm_tile_at(t, ngt, nht, gt, ht);
    const int64_t g0 = gt * MM_T, h0 = ht * MM_T, nv = p.V - p.v0 - g0;
    const LanePlace at;
    const float f = __fmul_rn(p.alpha, p.scale[1]);
    const int64_t rows = nv < MM_T ? nv : MM_T, bytes = (p.H - h0) * 2;
    const rsrc_t rs = mm_out_rsrc(p.dw + (p.v0 + g0) * p.H + h0, p.H * 2, rows, bytes);
    MmParts parts{epi, 0};
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int ip = 0; ip < 2; ++ip) {
#pragma unroll
          for (int i = 2 * ip; i < 2 * ip + 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              f32x4 v = tile.c[x][y][i][j];
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = __fmul_rn(f, v[q]);
              parts.put<ET>(at.wm, at.wn, at.li, at.lg, i, j, v);
            }
          parts.flush<STORE_POLICY>(rs, y, x, ip, (uint32_t)p.H * 2, (int)rows, bytes);
        }
  }
};

// G^T hidden for at most 64 rows: one K stage, so what counts is the stream of
// grad_W's rows out, and the core's tiles, with one work-group per CU, spend
// most of their time between the loads and the stores. Here a work-group of four
// waves (three per CU) keeps 256 columns of hidden (a slab) in registers, 64 per
// wave, and walks down the vocabulary 128 columns of G at a time: the next ones
// load while these are multiplied and stored. Each 16 rows leave through 2 KB of
// the wave's own LDS as whole 128-byte lines, past the caches.
// H = 4096, V = 128256: one row 191 µs against the core's 266, 64 rows 193
// against 249 (1.05 GB at 5.5 TB/s). Neighbouring work-groups take neighbouring
// slabs, so that whole rows of grad_W are written at a time (each slab's in a
// range of its own: 30 µs more); with ordinary stores 45 to 55 µs more.
constexpr int XO_WAVES = 4, XO_ROWS = 64;
template <int ET>
__device__ __forceinline__ void xent_outer(const XentBwdArgs &p, int64_t per_slab, u32x4 *g0s, u32x4 *g1s, u32x4 *stage) {
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nslab = (p.H + MM_T - 1) / MM_T, first = blockIdx.x / nslab, slab = blockIdx.x - first * nslab;
  const int64_t h0 = slab * MM_T;
  const int64_t nv = p.V - p.v0 < p.np ? p.V - p.v0 : p.np, tiles = (nv + 127) / 128;
  // the core's loads are those of eight waves: this one does two waves' share
  MmSide<ET, true> sh[2], sg[2];
  auto load = [&](MmSide<ET, true>(&s)[2], const MmOperand &op, int h, u32x4 *dst) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      s[k].begin(op, 0);
      s[k].load(h, dst);
    }
  };
  const MmOperand oh{p.hidden + h0 * 2, (uint32_t)(p.H * 2), (int32_t)p.M, (uint32_t)((p.H - h0) * 2)};
  auto og = [&](int64_t t) {
    return MmOperand{p.G + t * 256, (uint32_t)(p.ldg * 2), (int32_t)p.M, (uint32_t)((p.ldg - t * 128) * 2)};
  };
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    sh[k].init(oh.ld, wave + 4 * k, lane, (wave & 1) * 64);
    sg[k].init((uint32_t)(p.ldg * 2), wave + 4 * k, lane, 0);
  }
  load(sh, oh, 0, g0s);
  load(sh, oh, 1, g1s);
  dma_barrier();
  u32x4 fb[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int s = 0; s < 2; ++s) fb[j][s] = sh[0].read(wave < 2 ? g0s : g1s, j, s);
  lds_barrier();  // hidden is read: G may come
  load(sg, og(first), 0, g0s);  // first < per_slab <= tiles
  dma_barrier();
  uint8_t *const stg = reinterpret_cast<uint8_t *>(stage + wave * 128);
  const float f = __fmul_rn(p.alpha, p.scale[1]);
  const int64_t cols = p.H - h0 - wave * 64;  // this wave's columns present (may be none)

  auto tile = [&](int64_t t, const u32x4 *cur, u32x4 *nxt) {
    // the other buffer was read before the barrier that ended the last tile
    const int64_t tn = t + per_slab;
    if (tn < tiles) load(sg, og(tn), 0, nxt);
    sched_fence();  // the loads stay ahead of the stores: the wait below counts on it
    const int64_t rows = nv - t * 128 < 128 ? nv - t * 128 : 128;
    uint16_t *const out = p.dw + (p.v0 + t * 128) * p.H + h0 + wave * 64;
    const rsrc_t rs = make_rsrc(cols > 0 ? out : p.dw,
                                cols > 0 ? (uint32_t)(((rows - 1) * p.H + (cols < 64 ? cols : 64)) * 2) : 0u);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      u32x4 fa[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) fa[s] = sg[0].read(cur, b, s);
      f32x4 acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j] = zero4();
#pragma unroll
        for (int s = 0; s < 2; ++s) acc[j] = mm_step<ET>(acc[j], fa[s], fb[j][s]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<u32x2 *>(stg + li * 128 + ((j ^ ((li >> 1) & 3)) * 32) + 8 * lg) =
            u32x2{mm_pack2<ET>(__fmul_rn(f, acc[j][0]), __fmul_rn(f, acc[j][1])),
                  mm_pack2<ET>(__fmul_rn(f, acc[j][2]), __fmul_rn(f, acc[j][3]))};
      __builtin_amdgcn_wave_barrier();  // other lanes' values: LDS keeps a wave's order
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int r = it * 8 + lane / 8, c = lane % 8;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(stg + r * 128 + (((c >> 1) ^ ((r >> 1) & 3)) * 32) + 16 * (c & 1));
        const bool ok = 16 * b + r < rows && 8 * c < cols;
        __builtin_amdgcn_raw_buffer_store_b128(v, rs, ok ? (uint32_t)(((16 * b + r) * p.H + 8 * c) * 2) : OFF_NONE, 0,
                                               STORE_POLICY);
      }
      __builtin_amdgcn_wave_barrier();  // these reads before the next block's writes
    }
    // the next tile's loads were issued before this one's 16 stores: all but
    // the last 16 operations have completed, so they have landed, and the
    // stores need not have
    wait_vm<16>();
    lds_barrier();
  };
  for (int64_t t = first; t < tiles; t += 2 * per_slab) {
    tile(t, g0s, g1s);
    if (t + per_slab < tiles) tile(t + per_slab, g1s, g0s);
  }
}
#define XO_SHARED()                                                        \
  __shared__ u32x4 xo_g0[MM_HALF], xo_g1[MM_HALF]; /* hidden, then G, two tiles */ \
  __shared__ u32x4 xo_stage[XO_WAVES * 128]

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

// The backward pass's plan: pieces of the vocabulary and splits of G W.
struct BwdPlan {
  int64_t vp, pieces, ksplit, splits;
  int64_t off_scale, off_rows, off_col, off_dh, off_g, bytes;
};
inline BwdPlan bwd_plan(int64_t M, int64_t H, int64_t V, bool bias) {
  BwdPlan p;
  const int64_t vall = ceil_div(V, MM_T) * MM_T;
  // G of a piece: 256 MiB (it then stays in the memory-side cache between the
  // three products), but at least 8192 columns, which give the products a
  // work-group per CU
  int64_t most = ((int64_t)256 << 20) / (2 * M) / MM_T * MM_T;
  if (most < 8192) most = 8192;
  p.pieces = ceil_div(vall, most);
  p.vp = ceil_div(ceil_div(vall, p.pieces), MM_T) * MM_T;
  p.pieces = ceil_div(V, p.vp);
  // G W has a tile per 256 rows and 256 of H, too few to fill the chip when M
  // is small: K (the piece's columns) is split, at least 256 columns each,
  // into as many splits as fill the last round of work-groups best
  const int64_t tiles = ceil_div(M, MM_T) * ceil_div(H, MM_T), cus = 256;
  double best = 0.0;
  p.splits = 1;
  for (int64_t s = 1; s <= 64 && s * 256 <= p.vp; ++s) {
    const double use = (double)(tiles * s) / (double)(ceil_div(tiles * s, cus) * cus);
    if (use > best * 1.05) {
      best = use;
      p.splits = s;
    }
    if (tiles * s >= cus * 4) break;
  }
  p.ksplit = ceil_div(ceil_div(p.vp, p.splits), 64) * 64;
  p.splits = ceil_div(p.vp, p.ksplit);
  p.off_scale = 0;
  p.off_rows = 256;
  p.off_col = p.off_rows + align256(16 * M);
  p.off_dh = p.off_col + (bias ? align256(4 * ceil_div(M, MM_T) * p.vp) : 0);
  p.off_g = p.off_dh + align256(4 * p.splits * M * H);
  p.bytes = p.off_g + align256(2 * M * p.vp);
  return p;
}

}  // namespace

}  // namespace lmhead
