// mma256.hpp -- the 256 x 256 matrix-product core of the training and int8
// operators (internal).
//
//   C[m, n] = sum over k of A(m, k) B(n, k)
//
// A work-group of eight waves builds one 256 x 256 tile of C, its fp32 (int8:
// int32) accumulators in registers. Each operand is read in the layout it
// lies in memory, by one of two ways through LDS:
//   K-inner  a row of the tile is contiguous along K (hidden and W in
//            hidden W^T). A stage holds 128 bytes of every row; an MFMA
//            operand is one ds_read_b128.
//   K-outer  K runs over memory rows and the tile's rows lie along them (W in
//            G W, both operands of G^T hidden). A stage holds 64 memory rows;
//            the operand is read by two transposing LDS reads
//            (ds_read_b64_tr_b16: a 16-lane group reads 4 memory rows of 16
//            elements, lane i receives column i), so no transposed copy of
//            anything is made.
// Both leave lane 16 g + i with K elements 8 g .. 8 g + 7 of row i, the
// operand map of kstep.hpp.
//
// The MFMA takes B as its first operand, so accumulator register q of lane
// 16 g + i is C(row i, column 4 g + q) of its 16 x 16 block: a lane holds
// four consecutive columns of one row, which the epilogues want (row
// statistics need two lane exchanges, stores pack four columns).
//
// Schedule. A stage (64 K elements of 16 bits, 128 of int8) comes in four
// half-tiles A0, A1, B0, B1 of 128 rows (16 KB), two LDS stages (128 KB).
// Wave (wm, wn) of 2 x 4 owns rows wm 64 .. + 63 of both A halves and rows
// wn 32 .. + 31 of both B halves: four quadrants of 64 x 32. A stage is
// worked off in two phases of 32 MFMAs:
//   phase  reads into registers   MFMA            direct-to-LDS loads issued
//   X      A0(t), B1(t)           A0 B0, A0 B1    A1(t + 1), B0(t + 2)
//   Y      A1(t), B0(t + 1)       A1 B1, A1 B0    A0(t + 2), B1(t + 2)
// Each load refills an LDS region that the phase before has read. A phase is
// a read part, ended by waits and a barrier, and an MFMA part, ended by a
// barrier; waves 4-7 run one barrier behind waves 0-3, so while one of a
// SIMD's two waves reads and loads, the other feeds the matrix pipe.
//
// Why the waits suffice. (1) A region is refilled in the read part of the
// phase after the one that read it, when every wave's reads have returned:
// each wave waits for its own LDS reads (lgkmcnt 0) before the barrier that
// ends its read part, and the later group's read part ends with the barrier
// that starts the earlier group's next one. (2) What the next phase reads has
// landed: each wave retires its own share of those loads before the barrier
// that ends its read part. Loads complete in issue order and exactly four
// half-tiles (two loads per wave each) were issued after the ones in
// question, so vmcnt(8) retires them. Stages past the last load nothing
// (out-of-range offsets, which leave zeros), to keep the counts exact.
//
// Measured (4096 x 32768 x 4096, bf16 random data, alone): K-inner operands
// 865 µs (1.27 PFLOP/s), B K-outer 832 µs (4096 x 4096 x 32768, 1.32), both
// K-outer 935 µs (1.18); int8 467 µs (2.35 POP/s). Four phases of 16 MFMAs
// took 890 µs, the waves of a SIMD in step (no barrier of offset) 969 µs.
// Loads that all hit L2: 772 µs; no loads at all: 685 µs. So what is left is
// the loads' latency behind L2 and the tiles' starts and ends, during which
// a CU's one work-group leaves the matrix pipes idle.
#pragma once

#include "kstep.hpp"
#include "launch.hpp"
#include "ring.hpp"

namespace lmhead {

enum ElemType { ET_BF16 = 0, ET_F16 = 1, ET_I8 = 2 };

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int MM_T = 256;        // tile rows and columns
constexpr int MM_THREADS = 512;  // eight waves
constexpr int MM_HALF = 1024;    // 16-byte slots of a half-tile
constexpr int MM_STAGE_BYTES = 128;  // of a K-inner row per stage

// One operand of a tile, wave-uniform.
struct MmOperand {
  const uint8_t *base;  // K-inner: the tile's first row; K-outer: memory row 0, at the tile's first column
  int64_t ld;           // bytes between rows in memory
  int64_t rows;         // K-inner: tile rows present (1 .. 256); K-outer: memory rows (K) present
  int64_t cut;          // K-outer: bytes from `base` to the memory row's end (K-inner: unused)
  int64_t kbytes;       // K-inner: bytes of a row that belong to the product (K-outer: unused)
};

template <int ET>
struct MmAcc {
  using type = std::conditional_t<ET == ET_I8, i32x4, f32x4>;
};

template <int ET>
__device__ __forceinline__ typename MmAcc<ET>::type mm_step(typename MmAcc<ET>::type acc, u32x4 a,
                                                           u32x4 b) {
  if constexpr (ET == ET_I8)
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b),
                                                 __builtin_bit_cast(i32x4, a), acc, 0, 0, 0);
  else
    return kstep<ET == ET_F16>(acc, b, a);
}

// The accumulators of a wave: quadrant (A half, B half), 4 x 2 blocks.
template <int ET>
struct MmTile {
  typename MmAcc<ET>::type c[2][2][4][2];
  // C position of block (ah, bh, i, j) relative to the tile: this lane's row
  // and its first of four columns.
  static __device__ __forceinline__ int row(int wm, int li, int ah, int i) {
    return ah * 128 + wm * 64 + 16 * i + li;
  }
  static __device__ __forceinline__ int col(int wn, int lg, int bh, int j) {
    return bh * 128 + wn * 32 + 16 * j + 4 * lg;
  }
};

typedef __attribute__((address_space(3))) void mm_lds_void;
typedef __attribute__((address_space(3))) s16x4 mm_lds_s16x4;

// The stage buffers of a tile, declared in the kernel: half-tile h of stage s
// is its own array, so the compiler can tell a region being loaded from one
// being read.
struct MmBufs {
  u32x4 *p0, *p1, *p2, *p3, *p4, *p5, *p6, *p7;
  // array i (a constant after unrolling): stage i / 4, operand i / 2 % 2, half i % 2
  __device__ __forceinline__ u32x4 *at(int i) const {
    return i == 0 ? p0 : i == 1 ? p1 : i == 2 ? p2 : i == 3 ? p3 : i == 4 ? p4 : i == 5 ? p5 : i == 6 ? p6 : p7;
  }
  __device__ __forceinline__ u32x4 *a(int s, int h) const { return at(4 * s + h); }
  __device__ __forceinline__ u32x4 *b(int s, int h) const { return at(4 * s + 2 + h); }
};
#define MM_SHARED()                                                                \
  __shared__ u32x4 mmA00[MM_HALF], mmA10[MM_HALF], mmB00[MM_HALF], mmB10[MM_HALF]; \
  __shared__ u32x4 mmA01[MM_HALF], mmA11[MM_HALF], mmB01[MM_HALF], mmB11[MM_HALF]; \
  const MmBufs mm_buf{mmA00, mmA10, mmB00, mmB10, mmA01, mmA11, mmB01, mmB11}

// How one wave loads and reads one operand.
template <int ET, bool OUTER>
struct MmSide {
  MmOperand op;
  rsrc_t r;           // K-inner: the tile's rows
  uint32_t voff;      // this lane's offset of load 0 of a half-tile
  uint32_t voff1;     // ... of load 1 (K-inner: another swizzle)
  int wave, lane, li, lg;
  int w0;             // first row of this wave in a half: wm 64 or wn 32

  __device__ __forceinline__ void init(const MmOperand &o, int wave_, int lane_, int w0_) {
    op = o;
    wave = wave_;
    lane = lane_;
    li = lane_ & 15;
    lg = lane_ >> 4;
    w0 = w0_;
    if constexpr (OUTER) {
      // load u (= 2 wave, 2 wave + 1) of a half: memory rows 4 u .. 4 u + 3,
      // 16 pieces each; lane l fills slot l % 16 of row l / 16 with the piece
      // whose place there is its own (see slot_outer)
      const int piece = (lane % 16) ^ (((lane / 16) | ((wave & 1) << 2)) << 1);
      voff = (uint32_t)((lane / 16) * op.ld + 16 * piece);
      voff1 = voff;
    } else {
      // load u of a half: rows 8 u .. 8 u + 7, 8 pieces each; the swizzle of
      // row 8 u + l / 8 is (4 u + l / 16) & 7
      r = make_rsrc(op.base, (uint32_t)((op.rows - 1) * op.ld + op.kbytes));
      voff = (uint32_t)((lane / 8) * op.ld + 16 * ((lane % 8) ^ (lane / 16)));
      voff1 = (uint32_t)((lane / 8) * op.ld + 16 * ((lane % 8) ^ (4 + lane / 16)));
    }
  }

  // Half-tile h of memory stage `st` (< 0: none) into `dst`.
  __device__ __forceinline__ void load(int h, int64_t st, u32x4 *dst) const {
    const int u = 2 * wave;
    if constexpr (OUTER) {
      // the resource starts at the stage's first memory row (64-bit base: a
      // long K passes 32 bits) and ends with the last one present; rows past
      // it read as zero
      const int64_t k0 = st * 64;
      const int64_t left = st < 0 ? 0 : (op.rows - k0 < 64 ? op.rows - k0 : 64);
      const bool any = left > 0 && op.cut > 256 * h;
      const rsrc_t rs = make_rsrc(any ? op.base + k0 * op.ld : op.base,
                                  any ? (uint32_t)((left - 1) * op.ld + op.cut) : 0u);
      // columns past the row's end: a half wholly past it loads nothing; one
      // partly past it reads the next row's start there, into columns that
      // are never stored
      const uint32_t s0 = any ? (uint32_t)(4 * u * op.ld + 256 * h) : OFF_NONE;
      const uint32_t s1 = any ? (uint32_t)(4 * (u + 1) * op.ld + 256 * h) : OFF_NONE;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (mm_lds_void *)&dst[64 * u], 16, voff, s0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (mm_lds_void *)&dst[64 * (u + 1)], 16, voff1, s1, 0, 0);
    } else {
      const int64_t kb = st * MM_STAGE_BYTES;
      uint32_t v0 = voff, v1 = voff1;
      if (st >= 0 && kb + MM_STAGE_BYTES > op.kbytes) {  // uniform: the row's last, partial stage
        const int64_t p0 = (lane % 8) ^ (lane / 16), p1 = (lane % 8) ^ (4 + lane / 16);
        if (kb + 16 * p0 >= op.kbytes) v0 = OFF_NONE;
        if (kb + 16 * p1 >= op.kbytes) v1 = OFF_NONE;
      }
      const uint32_t s0 = st >= 0 ? (uint32_t)((h * 128 + 8 * u) * op.ld + kb) : OFF_NONE;
      const uint32_t s1 = st >= 0 ? (uint32_t)((h * 128 + 8 * (u + 1)) * op.ld + kb) : OFF_NONE;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mm_lds_void *)&dst[64 * u], 16, v0, s0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mm_lds_void *)&dst[64 * (u + 1)], 16, v1, s1, 0, 0);
    }
  }

  // The MFMA operand of rows w0 + 16 b .. of a half-tile, K-step s (0, 1).
  __device__ __forceinline__ u32x4 read(const u32x4 *src, int b, int s) const {
    if constexpr (OUTER) {
      // 16-lane group lg reads memory rows k = 32 s + 8 lg + 4 r + li / 4
      // (r = 0, 1), 16 elements = two pieces of each. Piece p of row k sits in
      // slot p ^ 2 ((k & 3) | (k >> 3 & 1) << 2): the eight rows that 32
      // lanes touch lie in eight distinct 32-byte pieces of the banks.
      u32x2 v[2];
#pragma unroll
      for (int r4 = 0; r4 < 2; ++r4) {
        const int k = 32 * s + 8 * lg + 4 * r4 + (li >> 2);
        const int p = (w0 + 16 * b) / 8 + ((li & 3) >> 1);
        const int slot = k * 16 + (p ^ (((k & 3) | (((k >> 3) & 1) << 2)) << 1));
        const uint8_t *at = reinterpret_cast<const uint8_t *>(src + slot) + 8 * (li & 1);
        v[r4] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                              (mm_lds_s16x4 *)(at)));
      }
      return u32x4{v[0][0], v[0][1], v[1][0], v[1][1]};
    } else {
      const int row = w0 + 16 * b + li;
      return src[row * 8 + ((4 * s + lg) ^ ((row >> 1) & 7))];
    }
  }
};

__device__ __forceinline__ void mm_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The main loop: `stages` K stages; `memstage(t)` is the memory stage that
// stage t of the order reads. On return every wave has met a barrier after
// its last LDS access and every direct load has landed, so the stage buffers
// are free.
template <int ET, bool AOUT, bool BOUT, typename F>
__device__ __forceinline__ void mm_main(MmTile<ET> &tile, const MmOperand &a, const MmOperand &b,
                                        int64_t stages, F &&memstage,
                                        const MmBufs &buf) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MmSide<ET, AOUT> sa;
  MmSide<ET, BOUT> sb;
  sa.init(a, wave, lane, (wave >> 2) * 64);
  sb.init(b, wave, lane, (wave & 3) * 32);
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) tile.c[x][y][i][j] = typename MmAcc<ET>::type{0, 0, 0, 0};

  // a tile of at most 128 rows of A leaves the second half out: half the
  // matrix work (uniform; its loads are out of range, the counts stay). Only
  // with both operands K-inner: with B K-outer the branch makes the compiler
  // spill.
  const bool tall = AOUT || BOUT || a.rows > 128;
  u32x4 fa[4][2], fb[3][2][2];  // A half in use; B halves in use (set, block, K-step)
  auto ms = [&](int64_t t) -> int64_t { return t < stages ? memstage(t) : -1; };
  auto readA = [&](const u32x4 *src) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) fa[i][s] = sa.read(src, i, s);
  };
  auto readB = [&](auto setc, const u32x4 *src) {
    constexpr int SET = decltype(setc)::value;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s) fb[SET][j][s] = sb.read(src, j, s);
  };
  auto mfma = [&](auto xc, auto yc, auto setc) {
    constexpr int X = decltype(xc)::value, Y = decltype(yc)::value, SET = decltype(setc)::value;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          tile.c[X][Y][i][j] = mm_step<ET>(tile.c[X][Y][i][j], fa[i][s], fb[SET][j][s]);
    __builtin_amdgcn_s_setprio(0);
  };
  using std::integral_constant;
  using I0 = integral_constant<int, 0>;
  using I1 = integral_constant<int, 1>;
  auto end_read = [&]() {
    wait_vm<8>();
    wait_lds();
    mm_barrier();
  };
  using I2 = integral_constant<int, 2>;
  auto stage = [&](auto sc, int64_t t) {
    constexpr int S = decltype(sc)::value;
    using SET = integral_constant<int, S>;
    using SETN = integral_constant<int, 1 - S>;
    readA(buf.a(S, 0));
    readB(I2{}, buf.b(S, 1));
    sa.load(1, ms(t + 1), buf.a(1 - S, 1));
    sb.load(0, ms(t + 2), buf.b(S, 0));
    end_read();
    mfma(I0{}, I0{}, SET{});
    mfma(I0{}, I1{}, I2{});
    mm_barrier();
    if (tall) readA(buf.a(S, 1));
    readB(SETN{}, buf.b(1 - S, 0));
    const int64_t m2 = ms(t + 2);
    sa.load(0, m2, buf.a(S, 0));
    sb.load(1, m2, buf.b(S, 1));
    end_read();
    if (tall) {
      mfma(I1{}, I1{}, I2{});
      mfma(I1{}, I0{}, SET{});
    }
    mm_barrier();
  };
  {
    const int64_t m = ms(0), n = ms(1);
    sb.load(0, m, buf.b(0, 0));
    sa.load(0, m, buf.a(0, 0));
    sb.load(1, m, buf.b(0, 1));
    sa.load(1, m, buf.a(0, 1));
    sb.load(0, n, buf.b(1, 0));
    sa.load(0, n, buf.a(1, 0));
    sb.load(1, n, buf.b(1, 1));
  }
  wait_vm<8>();
  mm_barrier();
  readB(I0{}, buf.b(0, 0));
  wait_lds();
  mm_barrier();
  if (wave >= 4) mm_barrier();
  for (int64_t t = 0; t < stages; t += 2) {
    stage(I0{}, t);
    stage(I1{}, t + 1);
  }
  if (wave < 4) mm_barrier();
  wait_vm<0>();
  wait_lds();
  mm_barrier();
}

// Position of a work-group among `n`: work-groups go to the eight XCDs
// round-robin, so that consecutive positions run on one XCD and share its L2.
__device__ __forceinline__ int64_t mm_position(int64_t n) {
  const int64_t b = blockIdx.x, q = n / 8, r = n % 8;
  const int64_t xcd = b % 8, pos = b / 8;
  return xcd < r ? xcd * (q + 1) + pos : r * (q + 1) + (xcd - r) * q + pos;
}

// Tile (a, b) of position t among na x nb: panels of four tiles of A, walked
// along B, so that the 32 work-groups of an XCD read 4 + 8 distinct operand
// tiles and not 32 + 1 (4096 x 32768 x 4096: 935 -> 891 µs against one panel
// of all of A; panels of 8: 906 µs).
__device__ __forceinline__ void mm_tile_at(int64_t t, int64_t na, int64_t nb, int64_t &a, int64_t &b) {
  constexpr int64_t PANEL = 4;
  const int64_t g = t / (PANEL * nb), h = na - g * PANEL < PANEL ? na - g * PANEL : PANEL;
  const int64_t r = t - g * PANEL * nb;
  a = g * PANEL + r % h;
  b = r / h;
}

// The LDS rows (512 bytes) of a 256 x 256 tile of 16-bit values: row r in
// stage array r / 32, its 32-byte pieces xor-ed with r so that the 16 rows one
// store touches fall in distinct banks.
__device__ __forceinline__ uint8_t *mm_tile_row(const MmBufs &buf, int hi, int r) {
  return reinterpret_cast<uint8_t *>(buf.at(hi)) + (r & 31) * 512;
}

// Two fp32 values to the 16-bit type, nearest even, low half first.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
template <int ET>
__device__ __forceinline__ uint32_t mm_pack2(float a, float b) {
  if constexpr (ET == ET_F16)
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Four columns of one row of the tile, as 16-bit values, into LDS.
template <int ET>
__device__ __forceinline__ void mm_stage4(const MmBufs &buf, int wm, int wn, int li, int lg,
                                       int x, int y, int i, int j, f32x4 v) {
  const int r = MmTile<ET>::row(wm, li, x, i);
  uint8_t *row = wm == 0 ? mm_tile_row(buf, x * 4 + (i >> 1), r) : mm_tile_row(buf, x * 4 + 2 + (i >> 1), r);
  const int piece = (y * 128 + wn * 32 + 16 * j) / 16;
  *reinterpret_cast<u32x2 *>(row + ((piece ^ (r & 15)) * 32) + 8 * lg) =
      u32x2{mm_pack2<ET>(v[0], v[1]), mm_pack2<ET>(v[2], v[3])};
}

// The staged tile to rows of `ld` bytes at `out`, `rows` rows of `bytes`
// bytes (a multiple of 16) present.
template <int POLICY>
__device__ __forceinline__ void mm_store_tile16(const MmBufs &buf, uint8_t *out, int64_t ld,
                                             int64_t rows, int64_t bytes) {
  const rsrc_t rs = make_rsrc(out, (uint32_t)((rows - 1) * ld + (bytes < 512 ? bytes : 512)));
  const int c = threadIdx.x % 32, r0 = threadIdx.x / 32;
#pragma unroll
  for (int it = 0; it < 16; ++it) {
    const int r = it * 16 + r0;
    const uint8_t *row = mm_tile_row(buf, it >> 1, r);
    const u32x4 v = *reinterpret_cast<const u32x4 *>(row + (((c >> 1) ^ (r & 15)) * 32) + 16 * (c & 1));
    const bool ok = r < rows && 16 * c < bytes;
    __builtin_amdgcn_raw_buffer_store_b128(v, rs, ok ? (uint32_t)(r * ld + 16 * c) : OFF_NONE, 0, POLICY);
  }
}

}  // namespace lmhead
