// int8.hip -- the 8-bit integer head: rows quantised to int8 with one scale
// each (tokens and vocabulary rows alike), and their product
//
//   logits[m, v] = alpha ((sum_k hq[m, k] wq[v, k]) hs[m]) ws[v] + bias[v]
//
// The sum is an exact int32 (H 2^14 <= 2^30), so its order does not matter and
// a row's logits do not depend on the call's other rows; the epilogue is fp32,
// each operation rounded in the order written.
//
// Up to 64 rows the call is one stream of the weight: int8_stream_kernel, the
// structure of the bf16 weight-streaming kernel (skinny.hip; its rings and
// waits are those of ring.hpp) at one byte per element. Above, the 256 x 256
// product of mma256.hpp.
//
// Measured with the quantisation of the hidden rows, H = 4096, V = 128256: one
// row 83 µs (526 MB, 6.3 TB/s), 48 rows with fp32 logits 91 µs (550 MB); 2048
// rows, V = 151936: 0.97-1.08 ms by card (2.4-2.6 POP/s). 130 rows, H = 2048, V =
// 151936: 91-105 µs by card (351 MB, 3.3-3.9 TB/s): 594 tiles are 2.3 rounds of
// the 256 work-groups, and half of what a stage loads is the hidden rows again;
// tiles of the last round cut in two took 90 µs where whole ones took 91, K
// starts spread over the weight's rows the same. The quantiser: 2048 rows of H =
// 4096 12 µs, a head of V = 128256 310-430 µs (1.58 GB read and written, up to 5.0
// TB/s; a device copy reaches 4.7-5.0).
#include "mma256.hpp"
#include "ops_launch.hpp"

namespace lmhead {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// Quantisation of rows: scale = max |x| / 127 (1 where that is 0), code =
// x / scale rounded to the nearest integer, ties to even. A work-group per
// row; rows of up to Q_KEEP pieces per thread stay in registers between the
// maximum and the codes, longer ones are read again.
// ---------------------------------------------------------------------------
constexpr int Q_THREADS = 256, Q_KEEP = 4;

template <bool F16>
__device__ __forceinline__ float elem(u32x4 v, int k) {
  const uint32_t b = (v[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
  if constexpr (F16)
    return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
  else
    return __builtin_bit_cast(float, b << 16);
}

template <bool F16>
__global__ __launch_bounds__(Q_THREADS) void quantize_int8_kernel(const uint16_t *__restrict__ x, int64_t rows,
                                                                  int64_t H, int8_t *__restrict__ q,
                                                                  float *__restrict__ scale) {
  const int64_t row = group_number();
  if (row >= rows) return;
  const u32x4 *const src = reinterpret_cast<const u32x4 *>(x + row * H);
  const int pieces = (int)(H / 8);
  u32x4 keep[Q_KEEP];
  uint32_t mx = 0;  // magnitude bits: their order is the values'
#pragma unroll
  for (int s = 0; s < Q_KEEP; ++s) {
    const int p = s * Q_THREADS + threadIdx.x;
    keep[s] = p < pieces ? src[p] : u32x4{0, 0, 0, 0};
  }
  auto fold = [&](u32x4 v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mx = max(mx, v[k] & 0x7FFFu);
      mx = max(mx, (v[k] >> 16) & 0x7FFFu);
    }
  };
#pragma unroll
  for (int s = 0; s < Q_KEEP; ++s) fold(keep[s]);
  for (int p = Q_KEEP * Q_THREADS + threadIdx.x; p < pieces; p += Q_THREADS) fold(src[p]);
  for (int d = 32; d; d >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d));
  __shared__ uint32_t sh[Q_THREADS / 64];
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < Q_THREADS / 64; ++w) mx = max(mx, sh[w]);
  float sc = __fdiv_rn(elem<F16>(u32x4{mx, 0, 0, 0}, 0), 127.0f);
  if (sc == 0.0f) sc = 1.0f;
  if (threadIdx.x == 0) scale[row] = sc;
  auto code = [&](u32x4 v, int k) -> uint32_t {
    const float r = rintf(__fdiv_rn(elem<F16>(v, k), sc));
    return (uint32_t)(int)fminf(fmaxf(r, -127.0f), 127.0f) & 0xFFu;
  };
  u32x2 *const dst = reinterpret_cast<u32x2 *>(q + row * H);
  auto put = [&](int p, u32x4 v) {
    u32x2 o = u32x2{0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k >> 2] |= code(v, k) << (8 * (k & 3));
    dst[p] = o;
  };
#pragma unroll
  for (int s = 0; s < Q_KEEP; ++s) {
    const int p = s * Q_THREADS + threadIdx.x;
    if (p < pieces) put(p, keep[s]);
  }
  for (int p = Q_KEEP * Q_THREADS + threadIdx.x; p < pieces; p += Q_THREADS) put(p, src[p]);
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------
struct I8Args {
  const uint8_t *hq;  // [M, H]
  const float *hs;    // [M]
  int64_t M, H;
  const uint8_t *wq;  // [V, H]
  const float *ws;    // [V]
  int64_t V;
  float alpha;
  const float *bias;  // [V] or nullptr
  void *out;          // [M, V]
};

__device__ __forceinline__ float i8_logit(int32_t acc, float hs, float ws, float alpha, bool has_bias, float b) {
  return epilogue_v(__fmul_rn(__fmul_rn((float)acc, hs), ws), alpha, has_bias, b);
}

// Stores `n` (of four) consecutive columns of one row; `vec`: the row's pieces
// of four are aligned for one store.
template <typename OutT>
__device__ __forceinline__ void store4(OutT *p, const float (&t)[4], int n, bool vec) {
  if constexpr (sizeof(OutT) == 4) {
    if (vec && n == 4) {
      *reinterpret_cast<f32x4 *>(p) = f32x4{t[0], t[1], t[2], t[3]};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < n) p[q] = t[q];
    }
  } else {
    uint16_t b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = out_bits16<OutT>(t[q]);
    if (vec && n == 4) {
      *reinterpret_cast<u32x2 *>(p) =
          u32x2{(uint32_t)b[0] | ((uint32_t)b[1] << 16), (uint32_t)b[2] | ((uint32_t)b[3] << 16)};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < n) reinterpret_cast<uint16_t *>(p)[q] = b[q];
    }
  }
}

// Up to 64 rows. Stage: 16 vocabulary rows x 128 bytes (two MFMA steps of 64);
// everything as in skinny.hip, in bytes: a wave's NB blocks stream through a
// ring of NSL LDS slots by direct-to-LDS loads, the hidden rows through two
// 128-byte chunks shared by the work-group. The weight is the first MFMA
// operand, so a lane ends with four consecutive columns of one row.
// A row's last chunk may be partial (H % 128 != 0): the hidden bytes past the
// row's end are zeros, so whatever the weight's are adds nothing.
constexpr int I8_CPR = 8;       // 16-byte pieces per hidden row per chunk
constexpr int I8_WSLOT = 128;   // 16-byte LDS slots of a block-stage
template <int R>
constexpr int i8_nb_max() { return R >= 4 ? 3 : 4; }

__device__ __forceinline__ int i8_hslot(int row, int ch) { return row * I8_CPR + (ch ^ (row & 7)); }
__device__ __forceinline__ int i8_wslot(int row, int p) { return row * 8 + (p ^ ((row >> 1) & 7)); }

template <int R, int NB, typename OutT, int NW, int NSL>
__global__ __launch_bounds__(64 * NW, NW >= 8 ? 1 : 2) void int8_stream_kernel(I8Args p, int64_t gblocks,
                                                                               int64_t kwg) {
  constexpr int THREADS = 64 * NW;
  constexpr int HPC = 16 * R * I8_CPR;
  constexpr int HL = (HPC + THREADS - 1) / THREADS;
  using S = Schedule<NB, NSL, HL, 2>;
  constexpr int NHR = S::NHR;
  constexpr int PERIOD = S::PERIOD;
  static_assert(NSL >= 2 && NSL <= 8, "a ring of 2 to 8 slots");
  constexpr int WLDS = NW * I8_WSLOT;
  __shared__ u32x4 hs[2][HPC];
  __shared__ u32x4 Wl0[WLDS], Wl1[WLDS], Wl2[NSL > 2 ? WLDS : 1], Wl3[NSL > 3 ? WLDS : 1],
      Wl4[NSL > 4 ? WLDS : 1], Wl5[NSL > 5 ? WLDS : 1], Wl6[NSL > 6 ? WLDS : 1], Wl7[NSL > 7 ? WLDS : 1];

  const int64_t M = p.M, H = p.H, V = p.V;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t ncb = (V + 15) / 16;
  const WaveCols wc = split_cols(blockIdx.x, gridDim.x, wave, NW, ncb, gblocks, kwg, H);
  const int64_t cb0 = wc.cb0, cb1 = wc.cb1;
  const bool active = cb1 > cb0;
  const int nbw = (int)(cb1 - cb0);
  const int64_t cend = cb1 * 16 < V ? cb1 * 16 : V;

  const rsrc_t wr = make_rsrc(p.wq + (active ? cb0 * 16 : 0) * H, active ? (uint32_t)((cend - cb0 * 16) * H) : 0u);
  const uint32_t wjstride = (uint32_t)(16 * H);
  uint32_t lvoff[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    lvoff[h] = (uint32_t)((lane / 8) * H + 16 * ((lane % 8) ^ ((4 * h + lane / 16) & 7)));

  const rsrc_t hr = make_rsrc(p.hq, (uint32_t)(M * H));
  uint32_t hvoff[HL];
  int hsl[HL], hch[HL];
#pragma unroll
  for (int i = 0; i < HL; ++i) {
    const int idx = i * THREADS + tid < HPC ? i * THREADS + tid : HPC - 1;
    const int row = idx / I8_CPR, ch = idx % I8_CPR;
    hvoff[i] = (uint32_t)(row * H + 16 * ch);
    hsl[i] = i8_hslot(row, ch);
    hch[i] = ch;
  }

  const int64_t hpieces = H / 16;
  const int64_t nchunks = (H + 127) / 128;
  const int64_t nunits = nchunks * NB;
  const int64_t krot = wc.kstart / 128;
  auto rowchunk = [&](int64_t c) { return c + krot < nchunks ? c + krot : c + krot - nchunks; };

  u32x4 hring[NHR][HL];
  auto load_hidden = [&](u32x4(&dst)[HL], int64_t c) {
    const int64_t pc = c < nchunks ? rowchunk(c) : c;
    const uint32_t soff = c < nchunks ? (uint32_t)(pc * 128) : OFF_NONE;
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      const uint32_t v = (c >= nchunks || pc * I8_CPR + hch[i] < hpieces) ? hvoff[i] : OFF_NONE;
      dst[i] = load16(hr, v, soff);
    }
  };
  auto store_hidden = [&](const u32x4(&src)[HL], int buf) {
#pragma unroll
    for (int i = 0; i < HL; ++i) hs[buf][hsl[i]] = src[i];
  };
  auto wbuf = [&](auto jc) -> u32x4 * {
    constexpr int J = decltype(jc)::value;
    if constexpr (J == 0) return Wl0;
    else if constexpr (J == 1) return Wl1;
    else if constexpr (J == 2) return Wl2;
    else if constexpr (J == 3) return Wl3;
    else if constexpr (J == 4) return Wl4;
    else if constexpr (J == 5) return Wl5;
    else if constexpr (J == 6) return Wl6;
    else return Wl7;
  };
  auto issue_unit = [&](int64_t u, u32x4 *wl, int j) {
    const uint32_t soff = u < nunits ? (uint32_t)(rowchunk(u / NB) * 128 + j * wjstride) : OFF_NONE;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      dma16_lds(wr, &wl[wave * I8_WSLOT + 64 * h], lvoff[h], u < nunits ? soff + (uint32_t)(h * 8 * H) : OFF_NONE);
  };

  i32x4 acc[NB][R];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[j][r] = i32x4{0, 0, 0, 0};
  u32x4 a0[R], a1[R];

  auto unit = [&](auto pc, int64_t ub) {
    constexpr int P = decltype(pc)::value;
    constexpr int J = P % NB;
    constexpr int BUF = (P / NB) & 1;
    const int64_t u = ub + P;
    u32x4 *wl = wbuf(std::integral_constant<int, P % NSL>{});
    wait_vm<S::wait_unit(P)>();
    if constexpr (J == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        a0[r] = hs[BUF][i8_hslot(16 * r + li, lg)];
        a1[r] = hs[BUF][i8_hslot(16 * r + li, 4 + lg)];
      }
    }
    if (J < nbw) {  // wave-uniform
      const u32x4 b0 = wl[wave * I8_WSLOT + i8_wslot(li, lg)];
      const u32x4 b1 = wl[wave * I8_WSLOT + i8_wslot(li, 4 + lg)];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[J][r] = mm_step<ET_I8>(acc[J][r], a0[r], b0);
#pragma unroll
      for (int r = 0; r < R; ++r) acc[J][r] = mm_step<ET_I8>(acc[J][r], a1[r], b1);
    }
    wait_lds();
    issue_unit(u + NSL, wl, (P + NSL) % NB);
    if constexpr ((P + NSL) % NB == 0) {
      sched_fence();  // the hidden loads after the unit's, as the wait counts assume
      load_hidden(hring[((P + NSL) / NB) % NHR], (u + NSL) / NB);
    }
    if constexpr (J == NB - 1) {
      wait_vm<S::wait_hidden(P)>();
      store_hidden(hring[(P / NB + 1) % NHR], BUF ^ 1);
      lds_barrier();
    }
  };

  static_for<NSL>([&](auto wcn) {
    constexpr int W_ = decltype(wcn)::value;
    issue_unit(W_, wbuf(wcn), W_ % NB);
    if constexpr (W_ % NB == 0) {
      sched_fence();
      load_hidden(hring[(W_ / NB) % NHR], W_ / NB);
    }
    sched_fence();
  });
  wait_vm<S::wait_hidden(-1)>();
  store_hidden(hring[0], 0);
  lds_barrier();
  int64_t ub = 0;
  for (; ub + PERIOD <= nunits; ub += PERIOD) static_for<PERIOD>([&](auto pc) { unit(pc, ub); });
  static_for<PERIOD>([&](auto pc) {
    if (ub + decltype(pc)::value < nunits) unit(pc, ub);  // work-group-uniform
  });
  if (!active) return;
  OutT *const out = static_cast<OutT *>(p.out);
  const bool has_bias = p.bias != nullptr, vec = V % 4 == 0;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int64_t c = (cb0 + j) * 16 + 4 * lg;
    const int n = c >= cend ? 0 : (cend - c < 4 ? (int)(cend - c) : 4);
    float ws[4], b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      ws[q] = q < n ? p.ws[c + q] : 0.0f;
      b[q] = q < n && has_bias ? p.bias[c + q] : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t m = 16 * r + li;
      if (m >= M || n == 0) continue;
      const float sc = p.hs[m];
      float t[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) t[q] = i8_logit(acc[j][r][q], sc, ws[q], p.alpha, has_bias, b[q]);
      store4<OutT>(out + m * V + c, t, n, vec);
    }
  }
}

template <int R, int NB, typename OutT, int NW, int NSL>
hipError_t stream_nb(const I8Args &a, const VSplit &sp, hipStream_t s) {
  return launch_kernel(int8_stream_kernel<R, NB, OutT, NW, NSL>, dim3((unsigned)sp.nvs), dim3(64 * NW), s, a,
                       sp.gblocks, sp.kwg);
}
template <int R, int NBM, typename OutT>
hipError_t stream_split(const I8Args &a, const VSplit &sp, hipStream_t s) {
  if constexpr (NBM > 1) {
    if (sp.nb < NBM) return stream_split<R, NBM - 1, OutT>(a, sp, s);
  }
  return stream_nb<R, NBM, OutT, 16, 4>(a, sp, s);
}
// The launch shapes of skinny.hip: few column blocks per CU take fewer waves
// and a deeper ring.
template <int R, typename OutT>
hipError_t stream_r(const I8Args &a, hipStream_t s) {
  const int64_t ncb = (a.V + 15) / 16, cus = device_cus();
  if (ncb <= 4 * cus) return stream_nb<R, 1, OutT, 4, 8>(a, vsplit(ncb, a.H, 4, 1), s);
  if (ncb <= 8 * cus) return stream_nb<R, 1, OutT, 8, 8>(a, vsplit(ncb, a.H, 8, 1), s);
  constexpr int NBM = i8_nb_max<R>();
  return stream_split<R, NBM, OutT>(a, vsplit(ncb, a.H, 16, NBM), s);
}

// More rows: 256 x 256 tiles. 16-bit logits leave through LDS as whole rows in
// 16-byte stores; rows not so aligned, and fp32 ones (whose four columns per
// lane are 64 contiguous bytes per row already), straight from the registers.
template <typename OutT>
struct Int8Tiles {
  I8Args p;
  u32x4 *epi;
  int64_t nmt, nvt;

  __device__ __forceinline__ int64_t tiles() const { return nmt * nvt; }
  __device__ __forceinline__ MmJob job(int32_t t) const {
    int64_t mt, vt;
    mm_tile_at(t, nmt, nvt, mt, vt);
    const int64_t m0 = mt * MM_T, n0 = vt * MM_T, rows = p.M - m0, cols = p.V - n0;
    const uint32_t rb = (uint32_t)p.H;
    return MmJob{{p.hq + m0 * p.H, rb, (int32_t)(rows < MM_T ? rows : MM_T), rb},
                 {p.wq + n0 * p.H, rb, (int32_t)(cols < MM_T ? cols : MM_T), rb},
                 (int32_t)((p.H + MM_STAGE_BYTES - 1) / MM_STAGE_BYTES), 0};
  }
  __device__ __forceinline__ void epilogue(MmTile<ET_I8> &tile, int32_t t) const {
    int64_t mt, vt;
    mm_tile_at(t, nmt, nvt, mt, vt);
    const int64_t m0 = mt * MM_T, n0 = vt * MM_T;
    const int64_t rows = p.M - m0 < MM_T ? p.M - m0 : MM_T, cols = p.V - n0 < MM_T ? p.V - n0 : MM_T;
    const int tid = mm_tid(), lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 2, wn = wave & 3;
    const bool has_bias = p.bias != nullptr;
    OutT *const out = static_cast<OutT *>(p.out) + m0 * p.V + n0;
    const bool vec = p.V % 4 == 0;
    const bool staged = sizeof(OutT) == 2 && p.V % 8 == 0;
    float sc[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = MmTile<ET_I8>::row(wm, li, x, i);
        sc[x][i] = r < rows ? p.hs[m0 + r] : 0.0f;
      }
    MmParts parts{epi, 0};
    const rsrc_t rs = mm_out_rsrc(out, p.V * 2, rows, cols * 2);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float ws[2][4], bv[2][4];
      int n[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = MmTile<ET_I8>::col(wn, lg, y, j);
        n[j] = c >= cols ? 0 : (cols - c < 4 ? (int)(cols - c) : 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          ws[j][q] = q < n[j] ? p.ws[n0 + c + q] : 0.0f;
          bv[j][q] = q < n[j] && has_bias ? p.bias[n0 + c + q] : 0.0f;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int ip = 0; ip < 2; ++ip) {
#pragma unroll
          for (int i = 2 * ip; i < 2 * ip + 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = MmTile<ET_I8>::row(wm, li, x, i);
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                v[q] = i8_logit(tile.c[x][y][i][j][q], sc[x][i], ws[j][q], p.alpha, has_bias, bv[j][q]);
              if (staged)
                parts.put<std::is_same_v<OutT, _Float16> ? ET_F16 : ET_BF16>(wm, wn, li, lg, i, j,
                                                                             f32x4{v[0], v[1], v[2], v[3]});
              else if (r < rows)
                store4<OutT>(out + r * p.V + MmTile<ET_I8>::col(wn, lg, y, j), v, n[j], vec);
            }
          if (staged) parts.flush<STORE_POLICY>(rs, y, x, ip, (uint32_t)p.V * 2, (int)rows, cols * 2);
        }
    }
  }
};

template <typename OutT>
__global__ __launch_bounds__(MM_THREADS, 1) void int8_tiled_kernel(I8Args p) {
  MM_SHARED();
  MM_EPI_SHARED();
  const Int8Tiles<OutT> prob{p, mm_epi, (p.M + MM_T - 1) / MM_T, (p.V + MM_T - 1) / MM_T};
  mm_run<ET_I8, false, false>(prob, mm_buf);
}

template <typename OutT>
hipError_t launch_t(const I8Args &a, hipStream_t s) {
  if (a.M <= 64) {
    switch ((a.M + 15) / 16) {
      case 1: return stream_r<1, OutT>(a, s);
      case 2: return stream_r<2, OutT>(a, s);
      case 3: return stream_r<3, OutT>(a, s);
      default: return stream_r<4, OutT>(a, s);
    }
  }
  return launch_kernel(int8_tiled_kernel<OutT>, mm_grid(ceil_div(a.M, MM_T) * ceil_div(a.V, MM_T)),
                       dim3(MM_THREADS), s, a);
}

}  // namespace

hipError_t launch_quantize_int8(const void *x, int64_t rows, int64_t H, int in_f16, int8_t *q, float *scale,
                                hipStream_t s) {
  return launch_kernel(in_f16 ? quantize_int8_kernel<true> : quantize_int8_kernel<false>, numbered_grid(rows),
                       dim3(Q_THREADS), s, static_cast<const uint16_t *>(x), rows, H, q, scale);
}

hipError_t launch_int8(const Int8Args &c, hipStream_t s) {
  const I8Args a{reinterpret_cast<const uint8_t *>(c.hq), c.hs, c.M, c.H, reinterpret_cast<const uint8_t *>(c.wq),
                 c.ws, c.V, c.alpha, c.bias, c.out};
  return c.out_type == OUT_F32    ? launch_t<float>(a, s)
         : c.out_type == OUT_BF16 ? launch_t<uint16_t>(a, s)
                                  : launch_t<_Float16>(a, s);
}

}  // namespace lmhead
