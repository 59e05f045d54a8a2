// xent.hip -- softmax cross entropy of the head's logits against target
// tokens, and its gradients, in pieces of the vocabulary: the logits are
// never in memory.
//
//   t[m, v] = alpha (hidden[m, :] . W[v, :]) + bias[v]
//   lse[m]  = log sum_v exp t[m, v],   loss[m] = lse[m] - t[m, y_m]
//   G[m, v] = (g_m + l_m) exp(t[m, v] - lse[m]) - g_m [v = y_m]
//   grad_hidden = alpha G W,  grad_W = alpha G^T hidden,  grad_bias = sum_m G
//
// with g, l the gradients of loss and lse. A token is left out (loss 0, g
// taken as 0) when its target is ignore_index or no column of the call.
//
// Forward: one matrix product (mma256.hpp) whose epilogue keeps, per row and
// 256-column tile, the tile's largest t and its sum of exponentials, and the
// target's t; a second kernel folds the tiles of a row in a fixed order.
// Backward, per piece of the vocabulary: the product again, with the epilogue
// making G of the piece (16 bits, in the workspace), then G W added to fp32
// sums of grad_hidden, and G^T hidden, the piece's rows of grad_W. Three
// products of 2 M H V flops: making t again costs one product and saves
// keeping M V values from the forward pass.
//
// Everything is bound by the matrix pipes (mma256.hpp) except for few rows,
// where the weight's bytes bind, and for the smallest heads, where six short
// kernels follow each other. 4096 rows, H = 4096, V = 128256, from card to card:
// forward 2.9-3.1 ms (1.4-1.5 PFLOP/s, its epilogue included), per piece of 32256
// columns G 0.73-0.77 ms (1.40-1.48), G W 0.68-0.72 ms (1.50-1.59), G^T hidden
// 0.79-0.85 ms (1.28-1.37); 12.0-12.7 ms in all, of which the fourth product, t
// made again, is 2.9-3.1.
//
// Roundings: t, the statistics, p and grad_bias are fp32. G is rounded to the
// inputs' 16-bit type, which the matrix pipes take: at most 2^-8 (bf16) or
// 2^-11 (fp16) of each term of sums of M or V terms, the size of the 16-bit
// gradients' own rounding. It is kept scaled (xent_rows_kernel).
#include "xent_core.hpp"

namespace lmhead {

namespace {

struct XentFwdArgs {
  const uint8_t *hidden, *W;
  int64_t M, H, V;
  float alpha;
  const float *bias;
  const void *target;
  int target64;
  int64_t ignore;
  float2 *part;   // [vocabulary tile][M] {largest t, sum of exp(t - largest)}
  float *tlogit;  // [M] t at the target (rows with one)
};

template <int ET>
struct XentStats {
  XentFwdArgs p;
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
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = MmTile<ET>::row(at.wm, at.li, x, i);
        const int64_t m = m0 + row;
        const int32_t yt = m < p.M ? (int32_t)target_of(p.target, p.target64, m, p.ignore, p.V) - (int32_t)n0 : -1;
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
            for (int q = 0; q < 4; ++q)
              s = __fadd_rn(s, exp_diff(tile.c[x][y][i][j][q], mz));
        s = __fadd_rn(s, __shfl_xor(s, 16));
        s = __fadd_rn(s, __shfl_xor(s, 32));
        if (at.lg == 0) stat[at.wn * MM_T + row] = float2{mx, s};
      }
    lds_barrier();
    const int row = threadIdx.x;
    if (row < MM_T && m0 + row < p.M) {
      float mx = NEG_INF, s = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, stat[w * MM_T + row].x);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 e = stat[w * MM_T + row];
        if (e.y != 0.0f) s = __fadd_rn(s, __fmul_rn(e.y, exp_diff(e.x, mx)));
      }
      p.part[vt * p.M + m0 + row] = float2{mx, s};
    }
    // the next tile's epilogue is barriers away
  }
};

template <int ET>
__global__ __launch_bounds__(MM_THREADS, 1) void xent_stats_kernel(XentFwdArgs p) {
  MM_SHARED();
  MM_EPI_SHARED();
  const XentStats<ET> prob{p, mm_epi, (p.M + MM_T - 1) / MM_T, (p.V + MM_T - 1) / MM_T};
  mm_run<ET, false, false>(prob, mm_buf);
}

// Folds the tiles of a row: 16 rows per work-group, 64 threads per row, each
// thread tiles s, s + 64, ... in ascending order, then the 64 in eights and the
// eights, in order.
__global__ __launch_bounds__(XC_ROWS * XC_SLICES) void xent_combine_kernel(
    XentFwdArgs p, int64_t nvt, float *__restrict__ loss, float *__restrict__ lse) {
  __shared__ float2 sh[XC_SLICES][XC_ROWS];
  const int r = threadIdx.x % XC_ROWS, sl = threadIdx.x / XC_ROWS;
  const int64_t m = (int64_t)blockIdx.x * XC_ROWS + r;
  float mx = NEG_INF, s = 0.0f;
  if (m < p.M) {
    for (int64_t t0 = sl; t0 < nvt; t0 += 8 * XC_SLICES) {
      float2 e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t t = t0 + k * XC_SLICES;
        e[k] = t < nvt ? p.part[t * p.M + m] : float2{NEG_INF, 0.0f};
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
  if (sl != 0 || m >= p.M) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) fold_stat(mx, s, sh[k][r]);
  // every logit -inf: log-sum-exp -inf, and a target's probability 0
  const float ls = logf(s);
  lse[m] = s == 0.0f ? NEG_INF : __fadd_rn(mx, ls);
  // the loss from the largest logit, not from lse as rounded: a token that is
  // nearly certain has a loss far below half a step of its lse
  float out = 0.0f;
  if (target_of(p.target, p.target64, m, p.ignore, p.V) >= 0) {
    const float t = p.tlogit[m];
    out = t == NEG_INF ? __builtin_inff() : __fadd_rn(__fsub_rn(mx, t), ls);
  }
  loss[m] = out;
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// G is kept scaled by f = top / mx, mx the largest finite |a| or |b| of the rows and
// `top` a power of two, so that a row of that size has its largest entry, -b
// (1 - p) at the target, just below a power of two, where the 16-bit
// type's rounding is relatively finest: a batch's rows mostly share one size
// (the mean's 1 / n), and this halves the worst error of the entries that
// weigh most. top is 2^14 for fp16 (entries down to 2^-28 mx stay normal
// numbers; |G| <= 2 top) and 1 for bf16. scale[0] = f, scale[1] = 1 / f.
//
// One launch: every work-group finds the maximum over all rows by itself and
// writes its 256 rows' coefficients; M^2 / 256 reads of L2, negligible up to
// XR_ONE rows. With more rows one work-group finds the scale in a launch of
// its own (have_scale).
constexpr int XR_THREADS = 256;
constexpr int64_t XR_ONE = 32768;
struct XentRowsArgs {
  const float *g, *l, *lse;  // l may be nullptr
  const void *target;
  int target64;
  int64_t ignore, M, V;
  float top;
  float *scale;
  RowCoef *rows;
  int have_scale, write_rows;
};
__global__ __launch_bounds__(XR_THREADS) void xent_rows_kernel(XentRowsArgs p) {
  auto coef = [&](int64_t m, float &a, float &b) -> int64_t {
    const int64_t y = target_of(p.target, p.target64, m, p.ignore, p.V);
    b = y >= 0 ? p.g[m] : 0.0f;
    a = p.l != nullptr ? __fadd_rn(b, p.l[m]) : b;
    return y;
  };
  float f = 1.0f;
  if (p.have_scale) {
    f = p.scale[0];
  } else {
    __shared__ float sh[XR_THREADS / 64];
    float mx = 0.0f;
    for (int64_t m = threadIdx.x; m < p.M; m += XR_THREADS) {
      float a, b;
      coef(m, a, b);
      // of the finite ones: a row of inf or NaN is lost, the others are not
      a = fabsf(a);
      b = fabsf(b);
      mx = fmaxf(mx, fmaxf(a < __builtin_inff() ? a : 0.0f, b < __builtin_inff() ? b : 0.0f));
    }
    for (int d = 32; d; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < XR_THREADS / 64; ++w) mx = fmaxf(mx, sh[w]);
    // f and 1 / f both well inside the normal range, else no scale
    if (mx > 1e-30f && mx < 1e30f) f = __fdiv_rn(p.top, mx);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.scale[0] = f;
      p.scale[1] = __fdiv_rn(1.0f, f);
    }
  }
  const int64_t m = (int64_t)blockIdx.x * XR_THREADS + threadIdx.x;
  if (!p.write_rows || m >= p.M) return;
  float a, b;
  const int64_t y = coef(m, a, b);
  p.rows[m] = RowCoef{__fmul_rn(a, f), __fmul_rn(b, f), p.lse[m], (int32_t)y};
}

template <int ET, bool DB>
__global__ __launch_bounds__(MM_THREADS, 1) void xent_grad_kernel(XentBwdArgs p) {
  MM_SHARED();
  MM_EPI_SHARED();
  const XentGrad<ET, DB> prob{p, mm_epi, (p.M + MM_T - 1) / MM_T, p.np / MM_T};
  mm_run<ET, false, false>(prob, mm_buf);
}

// grad_bias of one piece: the row tiles' column sums in ascending order.
__global__ __launch_bounds__(256) void xent_bias_kernel(const float *__restrict__ colpart, int64_t nmt,
                                                        int64_t vp, int64_t n, float *__restrict__ db) {
  const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (v >= n) return;
  float s = 0.0f;
  for (int64_t t = 0; t < nmt; ++t) s = __fadd_rn(s, colpart[t * vp + v]);
  db[v] = s;
}

template <int ET>
__global__ __launch_bounds__(MM_THREADS, 1) void xent_dhidden_kernel(XentBwdArgs p) {
  MM_SHARED();
  const XentDHidden<ET> prob{p, (p.M + MM_T - 1) / MM_T, (p.H + MM_T - 1) / MM_T,
                             (p.np + p.ksplit - 1) / p.ksplit};
  mm_run<ET, false, true>(prob, mm_buf);
}

// grad_hidden: the splits' sums in ascending order, scaled, rounded once.
template <int ET>
__global__ __launch_bounds__(256) void xent_dhidden_out_kernel(const float *__restrict__ dh, int64_t n,
                                                               int splits, float alpha,
                                                               const float *__restrict__ scale,
                                                               uint16_t *__restrict__ out) {
  const int64_t e = (group_number() * 256 + threadIdx.x) * 8;
  if (e >= n) return;
  f32x4 s[2] = {zero4(), zero4()};
  if (splits == 1) {  // many rows: the loop would load the one sum eight times
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h] = *reinterpret_cast<const f32x4 *>(dh + e + 4 * h);
    splits = 0;
  }
  for (int k0 = 0; k0 < splits; k0 += 8) {
    f32x4 v[8][2];  // eight splits' loads in flight (past the last: the last again, not added)
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[k][h] = *reinterpret_cast<const f32x4 *>(dh + (k0 + k < splits ? k0 + k : splits - 1) * n + e + 4 * h);
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          s[h][q] = k0 + k < splits ? __fadd_rn(s[h][q], v[k][h][q]) : s[h][q];
  }
  const float f = __fmul_rn(alpha, scale[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 4; ++q) s[h][q] = __fmul_rn(f, s[h][q]);
  *reinterpret_cast<u32x4 *>(out + e) = u32x4{mm_pack2<ET>(s[0][0], s[0][1]), mm_pack2<ET>(s[0][2], s[0][3]),
                                              mm_pack2<ET>(s[1][0], s[1][1]), mm_pack2<ET>(s[1][2], s[1][3])};
}

template <int ET>
__global__ __launch_bounds__(MM_THREADS, 1) void xent_dweight_kernel(XentBwdArgs p) {
  MM_SHARED();
  MM_EPI_SHARED();
  const XentDWeight<ET> prob{p, mm_epi, p.np / MM_T, (p.H + MM_T - 1) / MM_T};
  mm_run<ET, true, true>(prob, mm_buf);
}

template <int ET>
__global__ __launch_bounds__(64 * XO_WAVES, 3) void xent_outer_kernel(XentBwdArgs p, int64_t per_slab) {
  XO_SHARED();
  xent_outer<ET>(p, per_slab, xo_g0, xo_g1, xo_stage);
}

// Both products of a small piece in one launch, side by side: work-groups up to
// `ga` make G W, the others G^T hidden (neither needs the other). 37 rows,
// H = 256, V = 4096: two launches of 11 and 9 µs become one of 11.
template <int ET>
__global__ __launch_bounds__(MM_THREADS, 1) void xent_products_kernel(XentBwdArgs p, uint32_t ga) {
  MM_SHARED();
  MM_EPI_SHARED();
  const int64_t nht = (p.H + MM_T - 1) / MM_T;
  if (blockIdx.x < ga) {
    const XentDHidden<ET> prob{p, (p.M + MM_T - 1) / MM_T, nht, (p.np + p.ksplit - 1) / p.ksplit};
    mm_run<ET, false, true>(prob, mm_buf, blockIdx.x, ga);
  } else {
    const XentDWeight<ET> prob{p, mm_epi, p.np / MM_T, nht};
    mm_run<ET, true, true>(prob, mm_buf, blockIdx.x - ga, gridDim.x - ga);
  }
}

__global__ __launch_bounds__(256) void zero_kernel(uint32_t *__restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}
hipError_t zero_words(void *p, int64_t n, hipStream_t s) {
  const int64_t blocks = ceil_div(n, 256);
  return launch_kernel(zero_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), s,
                       static_cast<uint32_t *>(p), n);
}

template <int ET>
hipError_t forward(const XentFwdArgs &p, float *loss, float *lse, hipStream_t s) {
  const int64_t nmt = ceil_div(p.M, MM_T), nvt = ceil_div(p.V, MM_T);
  hipError_t e = launch_kernel(xent_stats_kernel<ET>, mm_grid(nmt * nvt), dim3(MM_THREADS), s, p);
  if (e != hipSuccess) return e;
  return launch_kernel(xent_combine_kernel, dim3((unsigned)ceil_div(p.M, XC_ROWS)),
                       dim3(XC_ROWS * XC_SLICES), s, p, nvt, loss, lse);
}

template <int ET>
hipError_t backward(const XentBackward &c, uint8_t *ws, hipStream_t s) {
  const BwdPlan pl = bwd_plan(c.M, c.H, c.V, c.grad_bias != nullptr);
  float *const scale = reinterpret_cast<float *>(ws + pl.off_scale);
  RowCoef *const rows = reinterpret_cast<RowCoef *>(ws + pl.off_rows);
  XentRowsArgs r{c.grad_loss, c.grad_lse, c.lse, c.target, c.target64, c.ignore, c.M, c.V,
                 ET == ET_F16 ? 16384.0f : 1.0f, scale, rows, 0, 1};
  hipError_t e = hipSuccess;
  if (c.M > XR_ONE) {
    r.write_rows = 0;
    e = launch_kernel(xent_rows_kernel, dim3(1), dim3(XR_THREADS), s, r);
    r.write_rows = r.have_scale = 1;
  }
  if (e == hipSuccess)
    e = launch_kernel(xent_rows_kernel, dim3((unsigned)ceil_div(c.M, XR_THREADS)), dim3(XR_THREADS), s, r);
  XentBwdArgs p;
  p.hidden = static_cast<const uint8_t *>(c.hidden);
  p.W = static_cast<const uint8_t *>(c.W);
  p.M = c.M;
  p.H = c.H;
  p.V = c.V;
  p.alpha = c.alpha;
  p.bias = c.bias;
  p.rows = rows;
  p.scale = scale;
  p.ldg = pl.vp;
  p.G = ws + pl.off_g;
  p.colpart = c.grad_bias != nullptr ? reinterpret_cast<float *>(ws + pl.off_col) : nullptr;
  p.dh = reinterpret_cast<float *>(ws + pl.off_dh);
  p.ksplit = pl.ksplit;
  p.dw = static_cast<uint16_t *>(c.grad_W);
  const int64_t nmt = ceil_div(c.M, MM_T), nht = ceil_div(c.H, MM_T);
  for (int64_t v0 = 0; v0 < c.V && e == hipSuccess; v0 += pl.vp) {
    p.v0 = v0;
    p.first = v0 == 0;
    const int64_t nv = c.V - v0 < pl.vp ? c.V - v0 : pl.vp;
    p.np = ceil_div(nv, MM_T) * MM_T;
    e = launch_kernel(c.grad_bias != nullptr ? xent_grad_kernel<ET, true> : xent_grad_kernel<ET, false>, mm_grid(nmt * (p.np / MM_T)), dim3(MM_THREADS), s, p);
    if (e == hipSuccess && c.grad_bias != nullptr)
      e = launch_kernel(xent_bias_kernel, dim3((unsigned)ceil_div(nv, 256)), dim3(256), s,
                        static_cast<const float *>(p.colpart), nmt, pl.vp, nv, c.grad_bias + v0);
    const int64_t ta = nmt * nht * ceil_div(p.np, pl.ksplit), tb = nht * (p.np / MM_T);
    if (e == hipSuccess && c.grad_hidden != nullptr && c.grad_W != nullptr && ta + tb <= device_cus()) {
      e = launch_kernel(xent_products_kernel<ET>, dim3((unsigned)(ta + tb)), dim3(MM_THREADS), s, p, (uint32_t)ta);
      continue;
    }
    if (e == hipSuccess && c.grad_hidden != nullptr)
      e = launch_kernel(xent_dhidden_kernel<ET>, mm_grid(ta), dim3(MM_THREADS), s, p);
    if (e == hipSuccess && c.grad_W != nullptr) {
      if (c.M <= XO_ROWS) {
        // three work-groups per CU, spread over the slabs of hidden's columns
        const int64_t slots = ceil_div(3 * (int64_t)device_cus(), nht), n = ceil_div(nv, 128);
        const int64_t per_slab = n < slots ? n : slots;
        e = launch_kernel(xent_outer_kernel<ET>, dim3((unsigned)(nht * per_slab)), dim3(64 * XO_WAVES), s, p, per_slab);
      } else {
        e = launch_kernel(xent_dweight_kernel<ET>, mm_grid(tb), dim3(MM_THREADS), s, p);
      }
    }
  }
  if (e == hipSuccess && c.grad_hidden != nullptr)
    e = launch_kernel(xent_dhidden_out_kernel<ET>, numbered_grid(ceil_div(c.M * c.H, 2048)), dim3(256), s,
                      static_cast<const float *>(p.dh), c.M * c.H, (int)pl.splits, c.alpha,
                      static_cast<const float *>(scale), static_cast<uint16_t *>(c.grad_hidden));
  return e;
}

}  // namespace

int64_t xent_forward_bytes(int64_t M, int64_t V) { return align256(4 * M) + 8 * M * ceil_div(V, MM_T); }
int64_t xent_backward_bytes(int64_t M, int64_t H, int64_t V, bool bias) { return bwd_plan(M, H, V, bias).bytes; }

hipError_t launch_xent_forward(const XentForward &c, hipStream_t s) {
  XentFwdArgs p;
  p.hidden = static_cast<const uint8_t *>(c.hidden);
  p.W = static_cast<const uint8_t *>(c.W);
  p.M = c.M;
  p.H = c.H;
  p.V = c.V;
  p.alpha = c.alpha;
  p.bias = c.bias;
  p.target = c.target;
  p.target64 = c.target64;
  p.ignore = c.ignore;
  p.tlogit = static_cast<float *>(c.workspace);
  p.part = reinterpret_cast<float2 *>(static_cast<uint8_t *>(c.workspace) + align256(4 * c.M));
  return c.in_f16 ? forward<ET_F16>(p, c.loss, c.lse, s) : forward<ET_BF16>(p, c.loss, c.lse, s);
}

hipError_t launch_xent_backward(const XentBackward &c, hipStream_t s) {
  if (c.M == 0) {  // sums over no rows
    hipError_t e = hipSuccess;
    if (c.grad_W != nullptr) e = zero_words(c.grad_W, c.V * c.H / 2, s);
    if (e == hipSuccess && c.grad_bias != nullptr) e = zero_words(c.grad_bias, c.V, s);
    return e;
  }
  uint8_t *const ws = static_cast<uint8_t *>(c.workspace);
  return c.in_f16 ? backward<ET_F16>(c, ws, s) : backward<ET_BF16>(c, ws, s);
}

}  // namespace lmhead
