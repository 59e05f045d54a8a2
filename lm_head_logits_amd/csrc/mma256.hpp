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
// Tiles follow each other without a pause in the loads: a work-group stays on
// its CU and takes tile after tile (mm_run), and the last two stages of one
// already load the first two of the next, so a tile's epilogue runs while the
// next one's operands arrive. The epilogue therefore has LDS of its own (32 KB,
// MM_EPI) and leaves the stage buffers alone.
//
// Measured, with the epilogues of the kernels built on it (from card to card;
// rows of A x rows of B x K): K-inner operands 4096 x 32256 x 4096 730-770 µs
// (1.40-1.48 PFLOP/s), B K-outer 4096 x 4096 x 32256 680-720 µs (1.50-1.59), both
// K-outer 32256 x 4096 x 4096 790-850 µs (1.28-1.37), int8 2048 x 151936 x 4096 0.96-1.04
// ms (2.5-2.65 POP/s). Steps on the way, on a bench of the core alone with 32768
// columns, whose K-inner product then took 803 µs: four phases of 16 MFMAs 890,
// two of 32 865; the waves of a SIMD in step, without the barrier of offset, 969;
// a work-group per tile instead of tile after tile 865 (both K-outer 935 against
// 788); the 32x32x16 MFMA 907, in fewer cycles but at a lower clock. That is what
// bounds it now: the matrix pipes are busy 74-79% of the cycles (65% with both
// operands K-outer) and the card lowers its clock to 1.7-1.95 GHz under them; a
// copy whose loads all hit L2 ran 11% faster, one that loaded nothing 20%.
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
  uint32_t ld;          // bytes between rows in memory
  int32_t rows;         // K-inner: tile rows present (1 .. 256); K-outer: memory rows (K) present
  uint32_t bytes;       // K-inner: bytes of a row that belong to the product;
                        // K-outer: bytes from `base` to the memory row's end
};

// One tile: its operands and K stages, stage i of the order being memory stage
// (i + rot) mod stages (rot != 0 with both operands K-inner only, and rows of
// whole stages).
struct MmJob {
  MmOperand a, b;
  int32_t stages, rot;
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
constexpr int MM_EPI = 2048;  // 16-byte slots of the epilogue's LDS (32 KB)
#define MM_EPI_SHARED() __shared__ u32x4 mm_epi[MM_EPI]
#define MM_SHARED()                                                                \
  __shared__ u32x4 mmA00[MM_HALF], mmA10[MM_HALF], mmB00[MM_HALF], mmB10[MM_HALF]; \
  __shared__ u32x4 mmA01[MM_HALF], mmA11[MM_HALF], mmB01[MM_HALF], mmB11[MM_HALF]; \
  const MmBufs mm_buf{mmA00, mmA10, mmB00, mmB10, mmA01, mmA11, mmB01, mmB11}

// A wave-uniform value, in scalar registers whatever computed it.
__device__ __forceinline__ uint32_t mm_uni(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// How one wave loads and reads one operand. The loads follow the stages of the
// launch's tiles one after the other (MmStream moves both operands along).
template <int ET, bool OUTER>
struct MmSide {
  uint32_t voff[2];  // this lane's offsets of the two loads of a half-tile
  uint32_t cur[2];   // ... in the stage being loaded (K-inner: without what is past the row)
  uint32_t ld;
  rsrc_t rs;
  uint32_t lo, hi;   // K-outer: the stage's first memory row (64 bits: a long K passes 32)
  uint32_t bytes;    // MmOperand::bytes
  int32_t left;      // K-outer: memory rows from there on
  uint32_t kb;       // K-inner: the stage's offset in a row, OFF_NONE when there is none
  int wave, lane, li, lg;
  int w0;            // first row of this wave in a half: wm 64 or wn 32

  __device__ __forceinline__ int piece(int u) const {
    // K-outer, load u (= 0, 1; memory rows 8 wave + 4 u ..): 16 pieces a row;
    // lane l fills slot l % 16 of row l / 16 with the piece whose place there is
    // its own (see read). K-inner (rows 16 wave + 8 u ..): 8 pieces a row; the
    // swizzle of row 8 u + l / 8 is (4 u + l / 16) & 7.
    return OUTER ? (lane % 16) ^ (((lane / 16) | ((wave & 1) << 2)) << 1)
                 : (lane % 8) ^ (4 * u + lane / 16);
  }
  __device__ __forceinline__ void init(uint32_t ld_, int wave_, int lane_, int w0_) {
    ld = mm_uni(ld_);
    wave = wave_;
    lane = lane_;
    li = lane_ & 15;
    lg = lane_ >> 4;
    w0 = w0_;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      voff[u] = (uint32_t)(lane / (OUTER ? 16 : 8)) * ld + 16 * piece(u);
      cur[u] = voff[u];
    }
  }
  // To the first stage of a tile (in memory: stage rot).
  __device__ __forceinline__ void begin(const MmOperand &op, int32_t rot) {
    const uint64_t b = reinterpret_cast<uint64_t>(op.base);
    lo = mm_uni((uint32_t)b);
    hi = mm_uni((uint32_t)(b >> 32));
    bytes = mm_uni(op.bytes);
    if constexpr (OUTER) {
      left = (int32_t)mm_uni((uint32_t)op.rows);
      window();
    } else {
      rs = make_rsrc(op.base, (uint32_t)(op.rows - 1) * ld + op.bytes);
      kb = mm_uni((uint32_t)rot * MM_STAGE_BYTES);
    }
  }
  // K-outer: the resource starts at the stage's first memory row and ends with
  // the last one present; rows past it read as zero. Columns past the row's end
  // read the next row's start, into columns that are never stored.
  __device__ __forceinline__ void window() {
    const int32_t n = left < 64 ? left : 64;
    const uint64_t b = ((uint64_t)hi << 32) | lo;
    rs = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(b), (short)0,
                                           n > 0 ? (int)((uint32_t)(n - 1) * ld + bytes) : 0, RSRC_WORD3);
  }
  // To the next stage of the tile.
  __device__ __forceinline__ void step() {
    if constexpr (OUTER) {
      const uint64_t b = (((uint64_t)hi << 32) | lo) + 64ull * ld;
      lo = (uint32_t)b;
      hi = (uint32_t)(b >> 32);
      left -= 64;
      window();
    } else {
      kb += MM_STAGE_BYTES;
      if (kb >= bytes) kb = 0;  // rot != 0: round to the row's start
    }
  }
  // No stage: loads nothing.
  __device__ __forceinline__ void none() {
    if constexpr (OUTER) {
      left = 0;
      window();
    } else {
      kb = OFF_NONE;
    }
  }
  // K-inner: a row's last stage may be partial; what lies past the row is not
  // loaded. A branch around both (the empty asm keeps it one), so that rows of
  // whole stages pay no vector operations in a read part: 4% of the product.
  __device__ __forceinline__ void trim(bool last) {
    if constexpr (!OUTER) {
      if (bytes % MM_STAGE_BYTES != 0) {
        asm volatile("");
#pragma unroll
        for (int u = 0; u < 2; ++u)
          cur[u] = last && kb + 16 * piece(u) >= bytes ? OFF_NONE : voff[u];
      }
    }
  }

  // Half-tile h of the stage into `dst`.
  __device__ __forceinline__ void load(int h, u32x4 *dst) const {
    const uint32_t s = OUTER ? 8 * wave * ld + 256 * h : (h * 128 + 16 * wave) * ld + kb;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (mm_lds_void *)&dst[128 * wave], 16, cur[0], s, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (mm_lds_void *)&dst[128 * wave + 64], 16, cur[1],
                                             s + (OUTER ? 4 : 8) * ld, 0, 0);
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

// Where the work-groups' tiles lie. Work-groups go to the XCDs round-robin, so
// each XCD is given a contiguous range of the tiles, worked off in rounds of one
// tile per work-group: neighbours run at the same time and share the XCD's L2.
// Within a round the tiles rotate over the work-groups, so that none is always
// given the taller tiles of a pair.
struct MmWalk {
  uint32_t lo, hi, nw, wi, round;
  // Work-group b of g that share the tiles.
  __device__ __forceinline__ MmWalk(uint32_t tiles, uint32_t b, uint32_t g) {
    const uint32_t nx = g < 8 ? g : 8;
    const uint32_t x = b % nx, q = tiles / nx, r = tiles % nx;
    lo = x * q + (x < r ? x : r);
    hi = lo + q + (x < r ? 1 : 0);
    nw = (g - x + nx - 1) / nx;
    wi = b / nx;
    round = 0;
  }
  // The work-group's next tile, or -1.
  __device__ __forceinline__ int32_t next() {
    const uint32_t t = lo + round * nw + (wi + round) % nw;
    ++round;
    return t < hi ? (int32_t)mm_uni(t) : -1;
  }
};

// Tile (a, b) of position t among na x nb: panels of four tiles of A, walked
// along B, so that the 32 work-groups of an XCD read 4 + 8 distinct operand
// tiles and not 32 + 1 (4096 x 32768 x 4096: 935 -> 891 µs against one panel
// of all of A; panels of 8: 906 µs).
__device__ __forceinline__ void mm_tile_at(uint32_t t, uint32_t na, uint32_t nb, int64_t &a, int64_t &b) {
  constexpr uint32_t PANEL = 4;
  const uint32_t g = t / (PANEL * nb), h = na - g * PANEL < PANEL ? na - g * PANEL : PANEL;
  const uint32_t r = t - g * PANEL * nb, rb = r / h;
  a = mm_uni(g * PANEL + r - rb * h);
  b = mm_uni(rb);
}

// Runs the work-group's tiles of `p`:
//   p.tiles()           their number
//   p.job(t)            tile t (called by every wave, wave-uniform)
//   p.epilogue(tile, t) called by all waves at the same point of their barriers,
//                       which it may use; it has the accumulators and MM_EPI
//                       slots of LDS of its own. Vector memory operations that
//                       it leaves in flight only make later waits longer.
// Every job of a launch has the same row lengths (ld). `b` of `g`: this
// work-group among those that share the tiles.
template <int ET, bool AOUT, bool BOUT, typename P>
__device__ __forceinline__ void mm_run(const P &p, const MmBufs &buf, uint32_t b = blockIdx.x,
                                       uint32_t g = gridDim.x) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MmWalk walk((uint32_t)p.tiles(), b, g);
  int32_t tile_no = walk.next();
  if (tile_no < 0) return;
  MmSide<ET, AOUT> sa;
  MmSide<ET, BOUT> sb;

  using std::integral_constant;
  using I0 = integral_constant<int, 0>;
  using I1 = integral_constant<int, 1>;
  using I2 = integral_constant<int, 2>;
  // The stage being loaded: stage `l` of a tile's `lstages`, in pairs of stages
  // (an odd count ends with one of zeros). load_no: the tile it belongs to.
  int32_t l = 0, lstages, load_no = tile_no, rows_load;
  auto begin = [&](const MmJob &j) {
    lstages = (int32_t)mm_uni((uint32_t)j.stages);
    rows_load = (int32_t)mm_uni((uint32_t)j.a.rows);
    sa.begin(j.a, j.rot);
    sb.begin(j.b, j.rot);
  };
  auto trim = [&]() {
    sa.trim(l == lstages - 1);
    sb.trim(l == lstages - 1);
  };
  // To the next stage: an odd one (ODD) of the same tile, or an even one, which
  // may be the next tile's first.
  auto advance = [&](auto oddc) {
    constexpr bool ODD = decltype(oddc)::value != 0;
    ++l;
    if (l < lstages) {
      sa.step();
      sb.step();
    } else {
      if constexpr (!ODD) {
        l = 0;
        lstages = 0;
        if (load_no >= 0) load_no = walk.next();
      }
      if (!ODD && load_no >= 0) {
        begin(p.job(load_no));
      } else {
        sa.none();
        sb.none();
      }
    }
    trim();
  };
  {
    const MmJob j = p.job(tile_no);
    sa.init(j.a.ld, wave, lane, (wave >> 2) * 64);
    sb.init(j.b.ld, wave, lane, (wave & 3) * 32);
    begin(j);
    trim();
  }

  MmTile<ET> tile;
  u32x4 fa[4][2], fb[3][2][2];  // the A half in use; B0 of stages 0 and 1, B1 (block, K-step)
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
  // ends a read part: what the next phase reads has landed, this wave's own
  // reads have returned
  auto end_read = [&]() {
    wait_vm<8>();
    wait_lds();
    mm_barrier();
  };

  int32_t stages = lstages, rows = rows_load;  // of the tile being computed
  sb.load(0, buf.b(0, 0));
  sa.load(0, buf.a(0, 0));
  sb.load(1, buf.b(0, 1));
  sa.load(1, buf.a(0, 1));
  advance(I1{});
  sb.load(0, buf.b(1, 0));
  sa.load(0, buf.a(1, 0));
  sb.load(1, buf.b(1, 1));
  wait_vm<8>();  // stage 0's B0, A0, B1 (and A1 and B0 of what follows in flight)
  mm_barrier();
  readB(I0{}, buf.b(0, 0));
  wait_lds();
  mm_barrier();

  for (;;) {
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
    const bool tall = AOUT || BOUT || rows > 128;
    if (wave >= 4) mm_barrier();  // the second group runs one barrier behind
    for (int32_t t = 0; t < stages; t += 2) {
      auto stage = [&](auto sc) {
        constexpr int S = decltype(sc)::value;
        using SET = integral_constant<int, S>;
        using SETN = integral_constant<int, 1 - S>;
        readA(buf.a(S, 0));
        readB(I2{}, buf.b(S, 1));
        sa.load(1, buf.a(1 - S, 1));
        advance(sc);
        sb.load(0, buf.b(S, 0));
        end_read();
        mfma(I0{}, I0{}, SET{});
        mfma(I0{}, I1{}, I2{});
        mm_barrier();
        if (tall) readA(buf.a(S, 1));
        readB(SETN{}, buf.b(1 - S, 0));
        sa.load(0, buf.a(S, 0));
        sb.load(1, buf.b(S, 1));
        end_read();
        if (tall) {
          mfma(I1{}, I1{}, I2{});
          mfma(I1{}, I0{}, SET{});
        }
        mm_barrier();
      };
      stage(I0{});
      stage(I1{});
    }
    if (wave < 4) mm_barrier();
    p.epilogue(tile, tile_no);
    if (load_no < 0) break;
    tile_no = load_no;  // the loads are in the next tile by now
    stages = lstages;
    rows = rows_load;
  }
  wait_vm<0>();  // the loads of nothing write LDS too
}

// Work-groups of a launch of `tiles` tiles: one per CU, or per tile.
inline dim3 mm_grid(int64_t tiles) {
  const int64_t cus = device_cus();
  return dim3((unsigned)(tiles < cus ? tiles : cus));
}

// threadIdx.x, newly read: what an epilogue derives from it is worked out there
// and not, for all tiles, ahead of their loop, where it would take registers
// from the accumulators (50 spilled, reloaded behind every load in flight).
__device__ __forceinline__ int mm_tid() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
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

// 16-bit results leave through MM_EPI in eight parts: part (y, x, ip) holds the
// 64 rows 128 x + 64 wm + 32 ip + (0 .. 31) of the tile's columns y 128 .. + 127,
// row by row (256 bytes; its 32-byte pieces xor-ed with the row, for the
// banks), and is written to memory as whole rows in 16-byte stores. Two buffers
// take turns, so each part costs one barrier: a wave that writes a buffer has
// met, since it was last read, the barrier that its readers met after reading.
struct MmParts {
  u32x4 *epi;
  int n;  // parts so far

  __device__ __forceinline__ uint8_t *buf() const { return reinterpret_cast<uint8_t *>(epi) + (n & 1) * 16384; }
  // Four columns of one row: block (i, j) of quadrant (x, y).
  template <int ET>
  __device__ __forceinline__ void put(int wm, int wn, int li, int lg, int i, int j, f32x4 v) const {
    const int r = wm * 32 + (i & 1) * 16 + li;
    uint8_t *const at = buf() + r * 256 + (((wn * 2 + j) ^ (li & 7)) * 32) + 8 * lg;
    *reinterpret_cast<u32x2 *>(at) = u32x2{mm_pack2<ET>(v[0], v[1]), mm_pack2<ET>(v[2], v[3])};
  }
  // Writes part (y, x, ip): `rs` covers the tile from its first element, `ld`
  // bytes between rows, `rows` rows of `bytes` bytes (a multiple of 16) present.
  template <int POLICY>
  __device__ __forceinline__ void flush(rsrc_t rs, int y, int x, int ip, uint32_t ld, int rows, int64_t bytes) {
    lds_barrier();
    const int tid = mm_tid(), c = tid % 16, r0 = tid / 16;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int r = 128 * x + 64 * it + 32 * ip + r0;
      const u32x4 v = *reinterpret_cast<const u32x4 *>(buf() + (it * 32 + r0) * 256 +
                                                       (((c >> 1) ^ (r0 & 7)) * 32) + 16 * (c & 1));
      const uint32_t at = 256 * y + 16 * c;
      __builtin_amdgcn_raw_buffer_store_b128(v, rs, r < rows && at < bytes ? r * ld + at : OFF_NONE, 0, POLICY);
    }
    ++n;
  }
};
// The resource of flush(): `rows` rows of `bytes` bytes at `out`.
__device__ __forceinline__ rsrc_t mm_out_rsrc(void *out, int64_t ld, int64_t rows, int64_t bytes) {
  return make_rsrc(out, (uint32_t)((rows - 1) * ld + (bytes < 512 ? bytes : 512)));
}

}  // namespace lmhead
