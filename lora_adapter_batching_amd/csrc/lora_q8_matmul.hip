// lora_q8_matmul.hip -- the frozen projection's product on 8-bit rows and
// weights: y[t][j] (+)= sum_b sx[t][b] sw[j/128][b] sum_{k in b} x[t][k] w[j][k]
// over the 128-column blocks b, in fp32, rounded once to bf16.
//
// Both scales are powers of two, so the scaled matrix instruction
// (v_mfma_scale_f32_*_f8f6f4) takes their exponent bytes as they are stored
// and every product is summed at its true size: no separate scaling pass over
// the accumulators.
//
// Precision. The accumulators are fp32. Inside the instruction, eight
// neighbouring products are first added on a grid of 2^-13 of the largest
// one's power of two (measured; the unscaled fp8 instruction does the same),
// which leaves about 2e-5 of the result on normal inputs. The e4m3 rounding of
// the inputs is 2^-4 a value and the bf16 result's 2^-8, so it is kept: bf16
// products of the same bytes would be exact in fp32 at half the matrix rate
// and an expansion of every fragment.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lora_inspect.h"
#include "lora_internal.h"
#include "lora_q8.h"

namespace lora {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct MatArgs {
  const uint8_t* x;
  int64_t ldx;
  const uint8_t* xe;
  int64_t ldxe;
  const uint8_t* w;
  int64_t ldw;
  const uint8_t* we;
  int64_t ldwe;
  uint16_t* y;
  int64_t ldy;
  int32_t T, N;
  int32_t nkb;      // 128-column blocks of the sum
  int32_t tiles_t, tiles_n;
};

__device__ __forceinline__ i32x8 frag(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}
// D = A(32x64) B(64x32) + C on e4m3, each operand's rows scaled by 2^(e - 127)
// with e the low byte of its scale register (lane l: row l % 32). Lane l
// supplies 32 bytes of row l % 32; which of the 64 columns they are does not
// matter as long as both operands agree, since a 128-column block has one
// scale. Lane l holds D[8(i/4) + 4(l/32) + i%4][l%32].
__device__ __forceinline__ f32x16 mfma8_32(i32x8 a, i32x8 b, f32x16 c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, ea, 0, eb);
}
// The same with 16x16x128: lane l row l % 16, D[4(l/16) + i][l%16].
__device__ __forceinline__ f32x4 mfma8_16(i32x8 a, i32x8 b, f32x4 c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, ea, 0, eb);
}

// LDS-destination loads whose k position is a scalar offset. The descriptor
// ends with the last valid row; rows behind it have vector offsets past its
// end (with or without the scalar offset counted) and write zeros.
// M0 gets its wait state here (load_lds16 has the rule); the descriptor and the
// offset come from scalar instructions in the steps (all five waits: 374 instead
// of 371 us for 8192 tokens 4096 -> 14336), which the instruction-level tests check.
__device__ __forceinline__ void load_lds16_at(i32x4 rsrc, uint32_t lds_addr, uint32_t voff, uint32_t soff) {
  int m0_out;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds"
               : "={m0}"(m0_out)
               : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory");
  (void)m0_out;
}
// (Dwords are the exponents'. Their row may end inside a load, so the whole
// position is in the vector offset, which the descriptor checks. Their
// descriptors are made just ahead: all five waits.)
__device__ __forceinline__ void load_lds4_at(i32x4 rsrc, uint32_t lds_addr, uint32_t voff) {
  int m0_out;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tbuffer_load_dword %2, %3, %4 offen lds"
               : "={m0}"(m0_out)
               : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(0)
               : "memory");
  (void)m0_out;
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// Where the waves that share a ring meet: a ring of one wave needs no barrier.
template <int WAVES>
__device__ __forceinline__ void ring_barrier() {
  if constexpr (WAVES > 1) __builtin_amdgcn_s_barrier();
}

// Tile of workgroup b: each XCD (b % 8) takes a contiguous run of the tiles,
// ordered in groups of kGroupT token tiles, so that the tiles an XCD's CUs
// hold at one time share their x and w rows in its L2.
constexpr int kGroupT = 4;
__device__ __forceinline__ void tile_of(const MatArgs& a, int b, int grid, int& tt, int& tn) {
  const int q = grid >> 3, r = grid & 7, xcd = b & 7;
  const int id = xcd * q + min(xcd, r) + (b >> 3);
  const int per = kGroupT * a.tiles_n, g = id / per, in = id - g * per;
  const int size = min(kGroupT, a.tiles_t - g * kGroupT);
  tn = in / size;
  tt = g * kGroupT + (in - tn * size);
}

// ---------------------------------------------------------------------------
// Tiled product: BT tokens x BN columns per workgroup, the sum in steps of one
// 128-column block through a ring of S LDS stages. A stage holds the tile's w
// rows and x rows, 128 bytes each; the 16-byte piece c of row r sits at position
// c ^ swizzle(r), which spreads the rows of a fragment over the LDS banks (no
// conflicts counted). The loads write LDS directly, so the permutation is
// applied to the address each lane reads from.
//
// Small products cut the sum into KS parts: KS groups of waves with a ring each
// walk their own blocks side by side and their sums are added in group order,
// because one step's chain (barrier, LDS reads, matrix instructions) takes 0.3
// us however small the tile.
//
// What bounds the 256 x 256 tile: the matrix unit takes 2048 clocks a step, the
// CU's load path 1024 for its 64 KB (measured alone: 1370 with every CU
// loading). So
//  - the loads of step i + S are issued one by one between the matrix
//    instructions (in one piece, behind the barrier, they hold the wave until
//    the load path has taken the stage: 428 us instead of 413 for 8192 tokens
//    4096 -> 14336),
//  - rows are loaded in whole 128-byte lines: steps of 64 columns with twice
//    the stages took 1.5 times as long to load (439 us),
//  - the fragments of the next half step are read from LDS into a second set of
//    registers under the matrix instructions of the current half,
//  - the tile's exponents are fetched once, in the same way and ahead of the
//    first stage (through registers, row after row: 407 us instead of 390).
//  - its y leaves by non-temporal stores: all CUs end their tiles at about the
//    same time, and 4 MB of y an XCD would push the rows of the next tiles out of
//    its L2 (395 us without). Smaller tiles keep plain stores: their y
//    is small and the next operator reads it.
// Now 350-371 us by card, 2.6-2.75 PFLOP/s; where it takes 350-353, the library's fp8
// product without block scales, called in turn in the same process on inputs of the
// same distribution, takes 311-313 (8191 tokens 4096 -> 4096: 106-109 and 93-99). The
// steps run at 3.0 PFLOP/s; the rest is each tile's start and end (6 us of 52).
// ---------------------------------------------------------------------------
template <int BT_, int BN_, int WT_, int WN_, int S_, int KS_ = 1, bool STREAM_ = false>
struct Tile {
  static constexpr int BT = BT_, BN = BN_, WT = WT_, WN = WN_, S = S_, KS = KS_;
  static constexpr bool STREAM = STREAM_;               // y goes past the caches
  static constexpr int waves = WT * WN;                 // of one group; KS groups share the sum
  static constexpr int TT = BT / WT, TN = BN / WN;      // a wave's tokens and columns
  static constexpr int FT = TT / 32, FN = TN / 32;      // its fragments
  static constexpr int stage = (BN + BT) * 128;
  static constexpr int loads = stage / 1024 / waves;    // 1 KB (8 rows) each, per wave and step
  static constexpr int per = FT * FN >= FT + FN ? 1 : 2;  // fragments read per multiplication
  // Blocks of w a wave's columns lie in: one, or (tile widths that do not divide
  // into 128) each fragment's own.
  static constexpr int EW = (BN % 128 == 0 && 128 % TN == 0) || 128 % BN == 0 ? 1 : FN;
  static constexpr int erows = BT + (EW == 1 ? (BN + 127) / 128 : (BN + 254) / 128);  // exponent rows: tokens, w blocks
  static constexpr int ring = S * stage;                // one group's stages
  static constexpr int eoff = KS * ring;
  static constexpr int eloads = (erows + 4 * waves - 1) / (4 * waves);  // 256 bytes (4 rows) each, per wave
  static constexpr int egrp = eloads * waves * 256;     // one group's exponents
  static constexpr int eprow = TN * 4 + 16;             // epilogue row of one token (fp32, padded)
  static constexpr int parts = (KS - 1) * BT * BN * 4;  // the other groups' sums
  static constexpr int epi = parts + waves * 32 * eprow;
  static constexpr int used = eoff + KS * egrp;
  static constexpr int lds = used > epi ? used : epi;
  // the first wloads (xrows) loads of every wave are w rows (token exponents)
  static constexpr int wloads = BN / 8 / waves, xrows = BT / 4 / waves;
  static_assert(BN % (8 * waves) == 0 && BT % (4 * waves) == 0, "no load mixes the two operands");
  static_assert(stage % (1024 * waves) == 0 && TT % 32 == 0 && TN % 32 == 0, "whole loads and fragments");
  static_assert(FT + FN <= per * FT * FN, "every fragment of the next half is read");
  static_assert(S >= 2 && lds <= 160 * 1024, "fits the LDS");
};

// Exponents in LDS: rows of 16 dwords of four blocks each, dword d of row r at
// position d ^ (r / 4) % 16 (the bank of a wave's 32 rows then differs), refilled
// every kExpBlocks blocks (the first dword may begin up to three blocks earlier).
constexpr int kExpBlocks = 60;

__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }

template <class C, bool ADD>
__global__ __launch_bounds__(64 * C::waves * C::KS) void q8_tile_kernel(MatArgs a) {
  __shared__ alignas(1024) uint8_t smem[C::lds];
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)smem);
  const int lane = threadIdx.x & 63;
  const int wave0 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = C::KS > 1 ? wave0 / C::waves : 0, wave = wave0 - grp * C::waves;
  const int tid = threadIdx.x - grp * 64 * C::waves;
  // blocks [k0, k1) of the sum are this group's; all groups make `steps` steps
  const int steps = C::KS > 1 ? (a.nkb + C::KS - 1) / C::KS : a.nkb;
  const int k0 = grp * steps, k1 = min(a.nkb, k0 + steps);
  int tt, tn;
  tile_of(a, blockIdx.x, gridDim.x, tt, tn);
  const int t0 = tt * C::BT, n0 = tn * C::BN;
  const int vt = min(C::BT, a.T - t0), vn = min(C::BN, a.N - n0);  // valid rows of the tile
  const int64_t kbytes = (int64_t)a.nkb * 128;
  const i32x4 wr = mk_rsrc_words(a.w + (int64_t)n0 * a.ldw, (int64_t)(vn - 1) * a.ldw + kbytes);
  const i32x4 xr = mk_rsrc_words(a.x + (int64_t)t0 * a.ldx, (int64_t)(vt - 1) * a.ldx + kbytes);

  // Piece p of the wave: rows 8 (p * waves + wave) .. + 7 of the stage (w rows, then x rows).
  uint32_t voff[C::loads];
#pragma unroll
  for (int p = 0; p < C::loads; ++p) {
    const int r = 8 * (p * C::waves + wave) + (lane >> 3);
    const int c = (lane & 7) ^ swizzle(r);
    const bool isx = p >= C::wloads;
    voff[p] = (uint32_t)(isx ? (int64_t)(r - C::BN) * a.ldx : (int64_t)r * a.ldw) + 16u * c;
  }
  uint8_t* const ring = smem + grp * C::ring;
  const uint32_t ring0 = lds0 + (uint32_t)(grp * C::ring);
  // Load p of block kb; behind the group's last one the descriptors are empty and the
  // loads write zeros, so that every step issues (and waits for) the same
  // number without a branch between them. An empty descriptor needs a scalar offset of
  // 0: the range of a load ends at its bytes less that offset, which must not pass
  // below 0.
  auto load = [&](int kb, int slot, int p) {
    const int piece = p * C::waves + wave;
    i32x4 r = p >= C::wloads ? xr : wr;
    r[2] = kb < k1 ? r[2] : 0;
    load_lds16_at(r, ring0 + (uint32_t)(slot * C::stage + piece * 1024), voff[p], kb < k1 ? (uint32_t)kb * 128u : 0u);
  };

  const int eb0 = n0 >> 7, vb = ((n0 + vn - 1) >> 7) - eb0 + 1;
  const uint32_t* const es = reinterpret_cast<const uint32_t*>(smem + C::eoff + grp * C::egrp);
  const uint32_t es0 = lds0 + (uint32_t)(C::eoff + grp * C::egrp);
  // Loads the dwords with blocks kb0 .. of the group. What lies behind a row's
  // last block is never used (shift_exps).
  auto load_exps = [&](int kb0) {
    const int dwords = (a.nkb + 3) >> 2;
    const i32x4 xer = mk_rsrc_words(a.xe + (int64_t)t0 * a.ldxe, (int64_t)(vt - 1) * a.ldxe + 4 * dwords);
    const i32x4 wer = mk_rsrc_words(a.we + (int64_t)eb0 * a.ldwe, (int64_t)(vb - 1) * a.ldwe + 4 * dwords);
#pragma unroll
    for (int p = 0; p < C::eloads; ++p) {
      const int r0 = 4 * (p * C::waves + wave), r = r0 + (lane >> 4);
      const bool isx = p < C::xrows;
      const uint32_t row = (uint32_t)(isx ? (int64_t)r * a.ldxe : (int64_t)(r - C::BT) * a.ldwe);
      load_lds4_at(isx ? xer : wer, es0 + r0 * 64, row + 4u * ((lane & 15) ^ ((r >> 2) & 15)) + (uint32_t)(kb0 & ~3));
    }
  };

  const int wt = wave / C::WN, wn = wave % C::WN;
  const int m = lane & 31, h = lane >> 5;
  const int wrow = wn * C::TN + m, xrow = wt * C::TT + m;
  const int ncol0 = n0 + wn * C::TN;
  f32x16 acc[C::FT][C::FN];
#pragma unroll
  for (int i = 0; i < C::FT; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = zero_acc16();

  struct Exps {
    int w[C::EW], x[C::FT];
  };
  // Lane (m, h) reads pieces 4s + 2h and 4s + 2h + 1 of row m for half s.
  const int p0 = ((2 * h) ^ swizzle(m)) * 16, p1 = ((2 * h + 1) ^ swizzle(m)) * 16;
  auto read_frag = [&](int slot, int s, int row) {
    const uint8_t* p = ring + slot * C::stage + row * 128;
    return frag(*reinterpret_cast<const u32x4*>(p + (p0 ^ (64 * s))), *reinterpret_cast<const u32x4*>(p + (p1 ^ (64 * s))));
  };
  // The dwords that hold a step's exponents (those in LDS begin with kb0's);
  // shifted to the step's byte apart from the read, which takes its time.
  auto read_exps = [&](int kb, int kb0, Exps& e) {
    const int d = (kb >> 2) - (kb0 >> 2);
    auto at = [&](int r) { return (int)es[r * 16 + ((d ^ (r >> 2)) & 15)]; };
#pragma unroll
    for (int j = 0; j < C::EW; ++j) e.w[j] = at(C::BT + ((ncol0 + 32 * j) >> 7) - eb0);
#pragma unroll
    for (int i = 0; i < C::FT; ++i) e.x[i] = at(xrow + 32 * i);
  };
  // Behind the group's last block the exponent is 0 (2^-127), not the byte that
  // happens to follow: 255 there would make the empty stage's zeros NaN.
  auto shift_exps = [&](int kb, const Exps& e) {
    Exps o;
    const int sh = 8 * (kb & 3), width = kb < k1 ? 8 : 0;
#pragma unroll
    for (int j = 0; j < C::EW; ++j) o.w[j] = (int)__builtin_amdgcn_ubfe((uint32_t)e.w[j], sh, width);
#pragma unroll
    for (int i = 0; i < C::FT; ++i) o.x[i] = (int)__builtin_amdgcn_ubfe((uint32_t)e.x[i], sh, width);
    return o;
  };
  i32x8 fw[2][C::FN], fx[2][C::FT];
  // Half s of the group's step i: multiplies fragment set s and reads set s ^ 1 (the next
  // half). Half 1 issues the loads of step i + S into the stage of step i,
  // which every wave has read by then.
  auto half = [&](auto sc, const Exps& e, int i, int kb0, Exps& raw) {
    constexpr int s = decltype(sc)::value;
    constexpr int M = C::FT * C::FN;
    const int slot = (i + s) % C::S;
#pragma unroll
    for (int n = 0; n < M; ++n) {
      const int t = n / C::FN, j = n % C::FN;
      acc[t][j] = mfma8_32(fw[s][j], fx[s][t], acc[t][j], e.w[C::EW == 1 ? 0 : j], e.x[t]);
#pragma unroll
      for (int f = n * C::per; f < (n + 1) * C::per && f < C::FN + C::FT; ++f) {
        if (f < C::FN) fw[s ^ 1][f] = read_frag(slot, s ^ 1, wrow + 32 * f);
        else fx[s ^ 1][f - C::FN] = read_frag(slot, s ^ 1, C::BN + xrow + 32 * (f - C::FN));
      }
      if constexpr (s == 1) {
        // (behind the last block this reads a row that nothing uses)
        if (n == M / 2) read_exps(k0 + i + 1, kb0, raw);
#pragma unroll
        for (int p = n * C::loads / M; p < (n + 1) * C::loads / M; ++p) load(k0 + i + C::S, i % C::S, p);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  load_exps(k0);
#pragma unroll
  for (int s = 0; s < C::S; ++s)
#pragma unroll
    for (int p = 0; p < C::loads; ++p) load(k0 + s, s, p);
  wait_vm<(C::S - 1) * C::loads>();
  wait_lds();
  ring_barrier<C::waves>();
#pragma unroll
  for (int j = 0; j < C::FN; ++j) fw[0][j] = read_frag(0, 0, wrow + 32 * j);
#pragma unroll
  for (int i = 0; i < C::FT; ++i) fx[0][i] = read_frag(0, 0, C::BN + xrow + 32 * i);
  for (int i0 = 0; i0 < steps; i0 += kExpBlocks) {
    const int kb0 = k0 + i0;
    if (i0) {
      load_exps(kb0);
      wait_vm<0>();
      ring_barrier<C::waves>();
    }
    Exps raw;
    read_exps(kb0, kb0, raw);
    Exps e = shift_exps(kb0, raw);
    const int i1 = min(steps, i0 + kExpBlocks);
    for (int i = i0; i < i1; ++i) {
      half(std::integral_constant<int, 0>{}, e, i, kb0, raw);
      // step i is in registers; step i + 1 has landed (the later ones may still
      // be in flight); the barrier makes both true for every wave
      wait_vm<(C::S - 2) * C::loads>();
      wait_lds();
      ring_barrier<C::waves>();
      __builtin_amdgcn_sched_barrier(0);
      half(std::integral_constant<int, 1>{}, e, i, kb0, raw);
      e = shift_exps(k0 + i + 1, raw);
    }
    // the exponents are refilled only when every wave has read its last ones
    wait_lds();
    ring_barrier<C::waves>();
  }
  // The last steps' empty loads write LDS too: they end, in every wave, before
  // it is used for anything else.
  wait_vm<0>();
  wait_lds();
  __builtin_amdgcn_s_barrier();
  if constexpr (C::KS > 1) {
    // the groups' sums, added in group order
    f32x4* const part = reinterpret_cast<f32x4*>(smem);
    auto place = [&](int g, int i, int j, int q) {
      return ((((g - 1) * C::waves + wave) * C::FT + i) * C::FN + j) * 256 + q * 64 + lane;
    };
    if (grp) {
#pragma unroll
      for (int i = 0; i < C::FT; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            part[place(grp, i, j, q)] =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    }
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int g = 1; g < C::KS; ++g)
#pragma unroll
      for (int i = 0; i < C::FT; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 v = part[place(g, i, j, q)];
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][j][4 * q + c] += v[c];
          }
  }
  // Epilogue through LDS, so that a row's columns leave in whole lines:
  // 32 tokens at a time in fp32, 8 columns per lane back. What is added to is
  // read before the first store, into the registers that the fragments leave
  // free: loads and stores of the same matrix are kept in program order, and a
  // load behind a store would wait its whole latency.
  uint8_t* ep = smem + C::parts + wave * 32 * C::eprow;
  constexpr int LPR = C::TN / 8;        // lanes per row
  constexpr int NP = LPR / 2;           // passes over 32 LPR pieces of 8 columns
  auto place = [&](int i, int p, int& r, int& c, uint16_t*& yp) -> bool {
    r = (64 * p + lane) / LPR;
    c = (64 * p + lane) % LPR;
    const int t = t0 + wt * C::TT + 32 * i + r, ncol = ncol0 + 8 * c;
    yp = a.y + (int64_t)t * a.ldy + ncol;
    return t < a.T && ncol < a.N;
  };
  u32x4 old[C::FT][ADD ? NP : 1];
  if constexpr (ADD) {
#pragma unroll
    for (int i = 0; i < C::FT; ++i)
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        int r, c;
        uint16_t* yp;
        old[i][p] = zero16();
        if (place(i, p, r, c, yp)) old[i][p] = ld16(yp);
      }
  }
#pragma unroll
  for (int i = 0; i < C::FT; ++i) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        *reinterpret_cast<f32x4*>(ep + m * C::eprow + (32 * j + 8 * q + 4 * h) * 4) = v;
      }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      int r, c;
      uint16_t* yp;
      const bool in = place(i, p, r, c, yp);
      const f32x4 v0 = *reinterpret_cast<const f32x4*>(ep + r * C::eprow + c * 32);
      const f32x4 v1 = *reinterpret_cast<const f32x4*>(ep + r * C::eprow + c * 32 + 16);
      float f[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
      if constexpr (ADD) {
        float o[8];
        unpack8(old[i][p], o);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += o[e];
      }
      if (in) {
        if constexpr (C::STREAM) __builtin_nontemporal_store(pack8(f), reinterpret_cast<u32x4*>(yp));
        else st16(yp, pack8(f));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Few tokens: the weights are read once and that is the floor. A workgroup
// owns 16 columns and up to 16 tokens; its 8 waves take every eighth block of
// the sum straight from memory into fragments (no LDS on the way, each w row in
// whole 128-byte lines) and their parts are added in wave order. A CU holds four
// such workgroups. Wide projections have that many to hide the latency: one token
// 2560 -> 19456 10.4 us (4.8 TB/s), 16 tokens 14.7. 2560 columns are 160
// workgroups, less than one a CU, and then a wave's blocks follow each other, one
// load's latency each: one token 2560 -> 2560 4.0-4.6 us (three blocks a wave at
// most), 9728 -> 2560 8.2 (ten; its bytes take 4.8), 16 tokens 11.3. Two to four
// blocks in flight per wave, or 16 waves, were no faster; the sum is not divided
// over workgroups, which would need a workspace or a second launch.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;
constexpr int kFewTokens = 16;

template <bool ADD>
__global__ __launch_bounds__(64 * kFewWaves) void q8_few_kernel(MatArgs a) {
  __shared__ alignas(16) float part[kFewWaves][kFewTokens][16 + 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int vn = min(16, a.N - n0), vt = a.T;
  const int64_t kbytes = (int64_t)a.nkb * 128;
  const __amdgpu_buffer_rsrc_t wr = mk_rsrc(a.w + (int64_t)n0 * a.ldw, (int64_t)(vn - 1) * a.ldw + kbytes);
  const __amdgpu_buffer_rsrc_t xr = mk_rsrc(a.x, (int64_t)(vt - 1) * a.ldx + kbytes);
  const __amdgpu_buffer_rsrc_t xer = mk_rsrc(a.xe, (int64_t)(vt - 1) * a.ldxe + a.nkb);
  const __amdgpu_buffer_rsrc_t wer = mk_rsrc(a.we + (int64_t)(n0 >> 7) * a.ldwe, a.nkb);
  const bool row = r < vt;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < a.nkb; kb += kFewWaves) {
    const uint32_t k = (uint32_t)kb * 128u + 32u * g;
    const uint32_t wo = (uint32_t)((int64_t)r * a.ldw) + k;
    const uint32_t xo = row ? (uint32_t)((int64_t)r * a.ldx) + k : kOff;
    const u32x4 w0 = bld16(wr, wo), w1 = bld16(wr, wo + 16);
    const u32x4 x0 = bld16(xr, xo), x1 = bld16(xr, xo + 16);
    const int ew = __builtin_amdgcn_raw_buffer_load_b8(wer, kb, 0, 0);
    const int ex = __builtin_amdgcn_raw_buffer_load_b8(xer, row ? (int)((int64_t)r * a.ldxe) + kb : (int)kOff, 0, 0);
    acc = mfma8_16(frag(w0, w1), frag(x0, x1), acc, ew, ex);
  }
  *reinterpret_cast<f32x4*>(&part[wave][r][4 * g]) = acc;
  __syncthreads();
  const int t = threadIdx.x >> 1, c = (threadIdx.x & 1) * 8;
  if (t < vt && n0 + c < a.N) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
#pragma unroll
    for (int wv = 0; wv < kFewWaves; ++wv)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += part[wv][t][c + e];
    uint16_t* yp = a.y + (int64_t)t * a.ldy + n0 + c;
    if constexpr (ADD) {
      float o[8];
      unpack8(ld16(yp), o);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += o[e];
    }
    st16(yp, pack8(f));
  }
}

template <class C>
void launch_tile(MatArgs a, bool add, hipStream_t s) {
  a.tiles_t = (a.T + C::BT - 1) / C::BT;
  a.tiles_n = (a.N + C::BN - 1) / C::BN;
  const dim3 grid((unsigned)a.tiles_t * (unsigned)a.tiles_n), blk(64 * C::waves * C::KS);
  if (add) hipLaunchKernelGGL((q8_tile_kernel<C, true>), grid, blk, 0, s, a);
  else hipLaunchKernelGGL((q8_tile_kernel<C, false>), grid, blk, 0, s, a);
}

void launch_few(const MatArgs& a, bool add, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 15) / 16)), blk(64 * kFewWaves);
  if (add) hipLaunchKernelGGL(q8_few_kernel<true>, grid, blk, 0, s, a);
  else hipLaunchKernelGGL(q8_few_kernel<false>, grid, blk, 0, s, a);
}

// Tiles to choose from. A workgroup of a tile takes about fixed + step * (its
// blocks of the sum) microseconds while `slots` of them run, so a product takes
// that times the rounds its tiles need. Measured on 256 CUs (us; the sum is n
// blocks long): the largest tile has the best rate and needs the most of
// them, the small ones fill the GPU where there are few tokens.
//   tokens, k, n        256x256  128x128  128x128*  128x160  128x96  128x64  32x64  32x32
//   8192, 4096, 14336       367      451
//   8191, 4096, 4096        109      131       160      159     181     220
//   2048, 4096, 4096         45       35        40
//   1024, 4096, 4096                  27        21       22      31      30
//   256, 2560, 19456         35       23        27       19      24      30     69    107
//   128, 2560, 19456                  20        15       16      14      21     35     58
//   512, 2560, 2560                   19        14       15      12      11     22     31
//   128, 2560, 2560                   17        13       14      12      10      8     12
//   100, 9728, 2560                   51        32       38      30      25     15     21
//   37, 9728, 2560                    48        31       37      30      25     15     12
// (* with three stages, one workgroup per CU; the other holds two)
// The costs are a fit, and read low where a three-stage tile needs several rounds
// (128x128* at 8191 tokens 137 for 160, at 2048 34 for 40) and high for one round
// of 256x256 (55 for 45), and nothing in them stands for the weights' bytes. Where
// two tiles are near each other the choice can then be the slower one: of the
// sizes above, 2048 tokens 4096 -> 4096 takes 128x128* (40) over 128x128 (35).
struct TileChoice {
  int bt, bn, ks, stages, slots;
  float fixed, step;
  void (*launch)(MatArgs, bool, hipStream_t);
};
template <class C>
constexpr TileChoice choice(int slots, float fixed, float step) {
  return TileChoice{C::BT, C::BN, C::KS, C::S, slots, fixed, step, launch_tile<C>};
}
const TileChoice kTiles[] = {
    choice<Tile<256, 256, 2, 2, 2, 1, true>>(256, 10.6f, 1.40f),
    choice<Tile<128, 128, 2, 2, 2>>(512, 2.4f, 1.00f),
    choice<Tile<128, 128, 2, 2, 3>>(256, 6.2f, 0.34f),
    choice<Tile<128, 160, 4, 1, 3>>(256, 7.6f, 0.37f),
    choice<Tile<128, 96, 4, 1, 3>>(256, 6.3f, 0.26f),
    choice<Tile<128, 64, 2, 2, 3>>(256, 4.9f, 0.26f),
    choice<Tile<32, 64, 1, 2, 3, 4>>(256, 3.4f, 0.56f),
    choice<Tile<32, 32, 1, 1, 4, 4>>(256, 3.1f, 0.39f),
};

constexpr int64_t kMaxTiles = 0xffffffffll / 512;

// The tile for T tokens, N columns and a sum of nkb blocks; null: the few-token kernel.
const TileChoice* choose(int32_t T, int32_t N, int32_t nkb) {
  // One matrix fragment of tokens: the weights' bytes are all that counts (one
  // token 2560 -> 2560: 4.0 us against 6.2 with 32 x 32 tiles, 2560 -> 19456: 11
  // against 13 with 128 x 96; 16 tokens 2560 -> 2560 4.9 against 6.2, 9728 -> 2560
  // 12 either way). The one measured size that it loses is 16 tokens 2560 -> 19456,
  // 15 against 13: the border stays at the fragment's rows.
  // (A launch holds fewer than 2^32 threads, 512 of them per workgroup.)
  if (T <= kFewTokens && N <= 1 << 26) return nullptr;
  const TileChoice* best = &kTiles[0];  // (its grid is checked by the caller)
  double least = 0.;
  for (const TileChoice& c : kTiles) {
    const int64_t tiles = ((int64_t)T + c.bt - 1) / c.bt * (((int64_t)N + c.bn - 1) / c.bn);
    const double t = (double)((tiles + c.slots - 1) / c.slots) * (c.fixed + (double)c.step * ((nkb + c.ks - 1) / c.ks));
    if (&c == &kTiles[0] || (t < least && tiles <= kMaxTiles)) best = &c, least = t;
  }
  return best;
}

void launch_matmul(const MatArgs& a, bool add, hipStream_t s) {
  if (const TileChoice* c = choose(a.T, a.N, a.nkb)) c->launch(a, add, s);
  else launch_few(a, add, s);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_q8_matmul(const lora_q8_t* x, const lora_q8_t* w, void* y, int64_t ldy, uint32_t flags, void* stream) {
  clear_error();
  int st;
  if ((st = check_q8(x, "x", 1))) return st;
  if ((st = check_q8(w, "w", kQ8Block))) return st;
  if (flags & ~LORA_MATMUL_ACCUMULATE) return set_error(LORA_INVALID_ARGUMENT, "unknown flags 0x%x", flags);
  if (x->width != w->width)
    return set_error(LORA_INVALID_ARGUMENT, "x is %d wide and w %d: the sum runs over both", x->width, w->width);
  if (w->rows & 7) return set_error(LORA_INVALID_ARGUMENT, "w has %d rows (the width of y): a multiple of 8 is needed", w->rows);
  if (x->rows == 0 || w->rows == 0) return LORA_OK;
  if ((st = check_bf16_rows(y, ldy, w->rows, "y"))) return st;
  if (y == x->values || y == w->values) return set_error(LORA_INVALID_ARGUMENT, "y starts at an operand");
  // a tile's rows are addressed with 32-bit offsets from the tile's first row
  const int64_t most = 0x7fffff00 / 256;
  if (x->ld > most || w->ld > most || x->ld_exps > most || w->ld_exps > most)
    return set_error(LORA_UNSUPPORTED, "row strides above %lld bytes are not supported", (long long)most);
  if (((int64_t)x->rows + 255) / 256 * (((int64_t)w->rows + 255) / 256) > kMaxTiles || x->rows > 0x7fffff00 || w->rows > 0x7fffff00)
    return set_error(LORA_UNSUPPORTED, "y of %d x %d is too large for one call", x->rows, w->rows);
  MatArgs a{};
  a.x = x->values; a.ldx = x->ld; a.xe = x->exps; a.ldxe = x->ld_exps;
  a.w = w->values; a.ldw = w->ld; a.we = w->exps; a.ldwe = w->ld_exps;
  a.y = static_cast<uint16_t*>(y); a.ldy = ldy;
  a.T = x->rows; a.N = w->rows;
  a.nkb = (int32_t)q8_blocks(x->width);
  launch_matmul(a, (flags & LORA_MATMUL_ACCUMULATE) != 0, static_cast<hipStream_t>(stream));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(LORA_DEVICE_ERROR, "q8_matmul launch failed: %s", hipGetErrorString(e));
  return LORA_OK;
}

// Host-only: the kernel that a product takes (lora_inspect.h)
extern "C" int lora_inspect_matmul(int32_t num_tokens, int32_t width, int32_t h_out, lora_matmul_kernel_t* out) {
  clear_error();
  if (!out) return set_error(LORA_INVALID_ARGUMENT, "out is NULL");
  if (num_tokens <= 0 || width <= 0 || h_out <= 0 || (width & 7) || (h_out & 7))
    return set_error(LORA_INVALID_ARGUMENT, "num_tokens (%d), width (%d) and h_out (%d) must be positive, the widths multiples of 8",
                     num_tokens, width, h_out);
  const int32_t nkb = (int32_t)q8_blocks(width);
  const TileChoice* c = choose(num_tokens, h_out, nkb);
  out->kernels = 1 + (int32_t)(sizeof(kTiles) / sizeof(kTiles[0]));
  out->kernel = c ? 1 + (int32_t)(c - kTiles) : 0;
  out->tokens = c ? c->bt : kFewTokens;
  out->columns = c ? c->bn : 16;
  out->groups = c ? c->ks : kFewWaves;
  out->stages = c ? c->stages : 0;
  out->blocks = (nkb + out->groups - 1) / out->groups;
  out->exps = c ? kExpBlocks : 0;
  return LORA_OK;
}
