// lora_q4_matmul.hip -- the frozen projection's product on 4-bit weights and
// 8-bit or 4-bit rows: y[t][j] (+)= sum_k x(t, k) w(j, k), in fp32, rounded
// once to bf16.
//
// All scales are powers of two, and the scaled matrix instruction
// (v_mfma_scale_f32_*_f8f6f4) takes one for each row and 32 columns of either
// operand, which is what the 4-bit form stores: exponent bytes and codes go in
// as they are. With both operands in 4 bits it runs at twice the rate of the
// 8-bit forms; 8-bit rows on 4-bit weights run at the 8-bit rate and read half
// the weights' bytes.
//
// Precision. The accumulators are fp32. Products of two e2m1 values are whole
// multiples of 1/4 up to 36, and their sums inside a block of 32 are exact. With 8-bit
// rows the instruction first adds eight neighbouring products on a grid of 2^-13 of the
// largest one's power of two (2^8 and 2^-5 in a group of eight, -2^8 in the next: 2^-5; with
// 2^-6: 0, each in a group of its own: 2^-6), about 2e-5 of the result on normal inputs,
// which moves one bf16 result in a hundred by a step. The e4m3 rounding of the
// rows is 2^-4 a value and the result's 2^-8, so it is kept: bf16 products of the same
// values would be exact in fp32 at half the matrix rate and an expansion of every fragment.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lora_inspect.h"
#include "lora_internal.h"
#include "lora_q4.h"
#include "lora_q8.h"

namespace lora {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Mat4Args {
  const uint8_t* x;
  int64_t ldx;   // 4-bit rows: bytes between panels; 8-bit rows: between rows
  const uint8_t* xe;
  int64_t ldxe;
  const uint8_t* w;
  int64_t ldw;   // bytes between panels
  const uint8_t* we;
  int64_t ldwe;
  uint16_t* y;
  int64_t ldy;
  int32_t T, N;
  int32_t nkb;   // panels (128 columns) of the sum
  int32_t tiles_t, tiles_n;
};

__device__ __forceinline__ i32x8 frag4(u32x4 a) { return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0}; }
__device__ __forceinline__ i32x8 frag8(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}
// D = A(32x64) B(64x32) + C, A in e2m1, B in e4m3 (X8) or e2m1. Lane l = (m, h) =
// (l % 32, l / 32) supplies row m. 4 bits: columns 32 h .. 32 h + 31, in order from the
// lowest bits up. 8 bits: columns 16 h .. 16 h + 15, then 32 + 16 h .. + 15 (checked
// with single values on the GPU). Byte 2 S of its scale register scales columns 32 h ..
// 32 h + 31 of its row in either type. D[8(i/4) + 4 h + i%4][m] is register i.
template <bool X8, int S>
__device__ __forceinline__ f32x16 mfma4_32(i32x8 a, i32x8 b, f32x16 c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, X8 ? 0 : 4, 2 * S, ea, X8 ? 0 : 2 * S, eb);
}
// The same with 16x16x128: lane (r, g) = (l % 16, l / 16), columns 32 g .. in 4 bits,
// 16 g .. and 64 + 16 g .. in 8 bits, scale of columns 32 g ..; D[4 g + i][r].
template <bool X8>
__device__ __forceinline__ f32x4 mfma4_16(i32x8 a, i32x8 b, f32x4 c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, X8 ? 0 : 4, 0, ea, 0, eb);
}

// LDS-destination loads with explicit waits (load_lds16 has the rules). M0 gets its
// wait state here; descriptors and offsets come from scalar instructions or from
// the start of the kernel, which the instruction-level tests check.
__device__ __forceinline__ void load_piece16(i32x4 rsrc, uint32_t lds_addr, uint32_t voff, uint32_t soff) {
  int m0_out;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds"
               : "={m0}"(m0_out)
               : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory");
  (void)m0_out;
}
__device__ __forceinline__ void load_piece4(i32x4 rsrc, uint32_t lds_addr, uint32_t voff) {
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
__device__ __forceinline__ i32x4 rsrc_words(uint64_t base, int32_t bytes) {
  return i32x4{(int)(uint32_t)base, (int)(uint32_t)(base >> 32), bytes, kRsrcWord3};  // (addresses have 48 bits)
}

// Tile of workgroup b: each XCD (b % 8) takes a contiguous run of the tiles,
// ordered in groups of kGroupT token tiles, so that the tiles an XCD's CUs
// hold at one time share their x and w rows in its L2.
constexpr int kGroupT = 4;
__device__ __forceinline__ void tile_of(const Mat4Args& a, int b, int grid, int& tt, int& tn) {
  const int q = grid >> 3, r = grid & 7, xcd = b & 7;
  const int id = xcd * q + min(xcd, r) + (b >> 3);
  const int per = kGroupT * a.tiles_n, g = id / per, in = id - g * per;
  const int size = min(kGroupT, a.tiles_t - g * kGroupT);
  tn = in / size;
  tt = g * kGroupT + (in - tn * size);
}

// ---------------------------------------------------------------------------
// Tiled product: BT tokens x BN columns per workgroup, the sum in steps of one
// panel through a ring of S LDS stages. A stage holds the panel's w rows (64
// bytes each) and x rows (64 or 128), and their exponents (a dword each). In
// memory a panel's rows follow each other, so every load is a whole run of 1 KB.
// The 16-byte piece c of row r sits at c ^ (r / 4) % 4 (64-byte rows) or
// c ^ (r / 2) % 8 (128-byte rows) in LDS, which puts a fragment's 16 consecutive
// rows on distinct banks. The loads write LDS directly, so the permutation is
// applied to the address that each lane reads from.
//
// What bounds the 256 x 256 tile: a panel is 1024 clocks of the matrix unit in 4 bits
// (2048 with 8-bit x); its 34 (50) KB take the load path half of that, and the
// fragments' reads and the loads' writes 784 (1100) of LDS. So
//  - a half panel's fragments are read in its first half's instructions, so that
//    none is waited for where the waves meet, and the next stage's loads are spread
//    over the rest of both halves: 0.915 -> 0.835 us a panel in 4 bits,
//  - addresses are walked by scalar additions,
//  - three stages: 250 -> 232 us for 8192 tokens 4096 -> 14336 in 4 bits (four: 238), 98
//    -> 90 for 8191 tokens 4096 -> 4096 with 8-bit x (two stages),
//  - y leaves by non-temporal stores: all CUs end their tiles at about the same time; and
//    what is added to comes by non-temporal loads: 284 -> 271 us (y +=, 4 bits), 112 -> 106
//    (8191 tokens, 8-bit x). (Its lines touched 3 to 12 panels before the end, to have them
//    in L2 by then, was 2-5% slower.)
// 8192 tokens 4096 -> 14336: 232-236 us in 4 bits (4.1 PFLOP/s), 316-327 with 8-bit x
// (3.0); the library's product of 4-bit operands reaches 3.0 for 8192^3. In the steps
// it is 4.7 PFLOP/s on random values and 7.2 on constant ones. The launch takes 436
// thousand clocks on either, the matrix unit busy in 53% of them, at 1.9 GHz on random
// and 2.4 on constant values: power sets the clock, and fewer clocks are in part paid
// back by a lower one. (The matrix instructions alone, from registers, reach 6.8-7.0
// PFLOP/s on random values at 1.7 GHz and 9.0 on constant ones at 2.3; with 8-bit x
// 4.0-4.2 and 4.9.) Each tile's start and end are 6.4 us of 33; workgroups that walk
// over the tiles and load the next one's first stages under them took as long in 4 bits
// (234 us) and longer with 8-bit x (99 us instead of 93 for 8191 tokens 4096 -> 4096).
//
// Exponents of 8-bit rows (one for each 128 columns, row after row in memory) are
// fetched once for kExpBlocks blocks, as a row's dwords are far apart.
//
// Small products cut the sum into KS parts: KS groups of waves with a ring each
// walk their own panels side by side and their sums are added in group order.
// ---------------------------------------------------------------------------
template <int BT_, int BN_, int WT_, int WN_, int S_, bool X8_, int KS_ = 1, bool STREAM_ = false>
struct Tile4 {
  static constexpr int BT = BT_, BN = BN_, WT = WT_, WN = WN_, S = S_, KS = KS_;
  static constexpr bool X8 = X8_;
  static constexpr bool STREAM = STREAM_;               // y goes past the caches
  static constexpr int waves = WT * WN;                 // of one group; KS groups share the sum
  static constexpr int TT = BT / WT, TN = BN / WN;      // a wave's tokens and columns
  static constexpr int FT = TT / 32, FN = TN / 32;      // its fragments
  static constexpr int xrow_bytes = X8 ? 128 : 64;
  static constexpr int wpieces = BN / 16, pieces = wpieces + BT * xrow_bytes / 1024;  // 1 KB each
  static constexpr int vloads = (pieces + waves - 1) / waves;                          // of a wave
  static constexpr int xoff = BN * 64, eoff = vloads * waves * 1024;
  static constexpr int wslots = (BN + 63) / 64, xslots = X8 ? 0 : (BT + 63) / 64;  // exponent loads, 64 rows each
  static constexpr int eloads = (wslots + xslots + waves - 1) / waves;             // of a wave
  static constexpr int stage = eoff + eloads * waves * 256;
  static constexpr int loads = vloads + eloads;           // per wave and step
  static constexpr int ring = S * stage;                  // one group's stages
  static constexpr int x8off = KS * ring;
  static constexpr int x8loads = X8 ? BT / (8 * waves) : 0;  // 256 bytes (8 rows) each, per wave
  static constexpr int x8grp = x8loads * waves * 256;   // one group's exponents of 8-bit rows
  static constexpr int eprow = TN * 4 + 16;             // epilogue row of one token (fp32, padded)
  static constexpr int parts = (KS - 1) * BT * BN * 4;  // the other groups' sums
  static constexpr int epi = parts + waves * 32 * eprow;
  static constexpr int used = x8off + KS * x8grp;
  static constexpr int lds = used > epi ? used : epi;
  static_assert(!X8 || BT % (8 * waves) == 0, "whole exponent loads");
  static_assert(TT % 32 == 0 && TN % 32 == 0, "whole fragments");
  static_assert(S >= 3, "with two stages the loads of half 0 would be waited for at once");
  static_assert(lds <= 160 * 1024 && (S - 1) * loads < 64, "fits the LDS and the load counter");
};

// Exponents of 8-bit rows in LDS: rows of 8 dwords of four blocks each, dword d of
// row r at position d ^ (r / 8) % 8 (the bank of a wave's 32 rows then differs),
// refilled every kExpBlocks blocks (the first dword may begin up to three blocks earlier).
constexpr int kExpBlocks = 28;

template <class C, bool ADD>
__global__ __launch_bounds__(64 * C::waves * C::KS) void q4_tile_kernel(Mat4Args a) {
  __shared__ alignas(1024) uint8_t smem[C::lds];
  constexpr bool X8 = C::X8;
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)smem);
  const int lane = threadIdx.x & 63;
  const int wave0 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = C::KS > 1 ? wave0 / C::waves : 0, wave = wave0 - grp * C::waves;
  // panels [k0, k1) of the sum are this group's; all groups make `steps` steps
  const int steps = C::KS > 1 ? (a.nkb + C::KS - 1) / C::KS : a.nkb;
  const int k0 = grp * steps, k1 = min(a.nkb, k0 + steps);
  int tt, tn;
  tile_of(a, blockIdx.x, gridDim.x, tt, tn);
  const int t0 = tt * C::BT, n0 = tn * C::BN;
  const int vt = min(C::BT, a.T - t0), vn = min(C::BN, a.N - n0);  // valid rows of the tile

  // Load p of the wave takes piece p * waves + wave of the stage: 16 rows of 64 bytes
  // (w, then x) or 8 of 128; then loads of 64 rows' exponents. Pieces behind
  // the last one are empty.
  uint32_t vv[C::vloads], ev[C::eloads];
  bool isx[C::vloads], none[C::vloads];
#pragma unroll
  for (int p = 0; p < C::vloads; ++p) {
    const int q = p * C::waves + wave;
    isx[p] = p * C::waves >= C::wpieces || ((p + 1) * C::waves > C::wpieces && q >= C::wpieces);
    none[p] = (p + 1) * C::waves > C::pieces && q >= C::pieces;
    const int qx = isx[p] ? q - C::wpieces : q;
    const uint32_t v4 = (uint32_t)(qx * 1024 + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 4) & 3)) * 16));
    const int r = 8 * qx + (lane >> 3);
    vv[p] = X8 && isx[p] ? (uint32_t)((int64_t)r * a.ldx) + 16u * ((lane & 7) ^ ((r >> 1) & 7)) : v4;
  }
  uint8_t* const ring = smem + grp * C::ring;
  const uint32_t ring0 = lds0 + (uint32_t)(grp * C::ring);
  // Where the loads stand: the next panel's addresses and stage. (Walked by
  // scalar additions: the addresses made from the panel's number took 45 scalar
  // instructions in one place of the step.)
  struct {
    uint64_t w, x, e[C::eloads], estep[C::eloads];
    int32_t wbytes, xbytes, ebytes[C::eloads];
    uint32_t xat, at;
    int left;
  } to;
  to.w = reinterpret_cast<uint64_t>(a.w) + (uint64_t)n0 * 64 + (uint64_t)k0 * a.ldw;
  to.wbytes = vn * 64;
  const uint64_t xbase = reinterpret_cast<uint64_t>(a.x) + (uint64_t)t0 * (X8 ? (uint64_t)a.ldx : 64u);
  const uint64_t xebase = reinterpret_cast<uint64_t>(a.xe) + (uint64_t)t0 * (X8 ? (uint64_t)a.ldxe : 4u);
  to.x = X8 ? xbase : xbase + (uint64_t)k0 * a.ldx;
  to.xbytes = X8 ? (int32_t)((int64_t)(vt - 1) * a.ldx + (int64_t)a.nkb * 128) : vt * 64;
  to.xat = k0 < k1 ? (uint32_t)k0 * 128u : 0u;
#pragma unroll
  for (int p = 0; p < C::eloads; ++p) {
    const int q = p * C::waves + wave;
    const bool isx = q >= C::wslots;
    ev[p] = 4u * (uint32_t)(lane + 64 * (isx ? q - C::wslots : q));
    to.estep[p] = (uint64_t)(isx ? a.ldxe : a.ldwe);
    to.e[p] = (isx ? xebase : reinterpret_cast<uint64_t>(a.we) + (uint64_t)n0 * 4) + (uint64_t)k0 * to.estep[p];
    to.ebytes[p] = (isx ? (X8 ? 0 : vt) : vn) * 4;
  }
  to.at = ring0;
  to.left = k1 - k0;
  // Load p of the panel; behind the group's last one the descriptors are empty and
  // the loads write zeros, so that every step issues (and waits for) the same
  // number without a branch between them. An empty descriptor needs a scalar offset of
  // 0: the range of a load ends at its bytes less that offset, which must not pass
  // below 0.
  auto load = [&](int p) {
    const bool live = to.left > 0;
    if (p < C::vloads) {
      const int32_t bytes = isx[p] ? to.xbytes : to.wbytes;
      load_piece16(rsrc_words(isx[p] ? to.x : to.w, live && !none[p] ? bytes : 0), to.at + (p * C::waves + wave) * 1024, vv[p],
                   X8 && isx[p] && !none[p] ? to.xat : 0);
    } else {
      const int q = p - C::vloads;
      load_piece4(rsrc_words(to.e[q], live ? to.ebytes[q] : 0), to.at + C::eoff + (q * C::waves + wave) * 256, ev[q]);
    }
  };
  auto next_panel = [&] {
    to.w += (uint64_t)a.ldw;
    if constexpr (X8) to.xat = to.left > 1 ? to.xat + 128u : 0u;
    else to.x += (uint64_t)a.ldx;
#pragma unroll
    for (int p = 0; p < C::eloads; ++p) to.e[p] += to.estep[p];
    to.at = to.at == ring0 + (C::S - 1) * C::stage ? ring0 : to.at + C::stage;
    --to.left;
  };
  // 8-bit rows: the dwords with blocks kb0 .. of the group. What lies behind a
  // row's last block is never used.
  const uint32_t* const xs = reinterpret_cast<const uint32_t*>(smem + C::x8off + grp * C::x8grp);
  const uint32_t xs0 = lds0 + (uint32_t)(C::x8off + grp * C::x8grp);
  auto load_exps = [&](int kb0) {
    const int dwords = (a.nkb + 3) >> 2;
    const i32x4 xer = rsrc_words(xebase, (int32_t)((int64_t)(vt - 1) * a.ldxe + 4 * dwords));
#pragma unroll
    for (int p = 0; p < C::x8loads; ++p) {
      const int r0 = 8 * (p * C::waves + wave), r = r0 + (lane >> 3);
      load_piece4(xer, xs0 + r0 * 32, (uint32_t)((int64_t)r * a.ldxe) + 4u * ((lane & 7) ^ ((r >> 3) & 7)) + (uint32_t)(kb0 & ~3));
    }
  };

  const int wt = wave / C::WN, wn = wave % C::WN;
  const int m = lane & 31, h = lane >> 5;
  const int wrow = wn * C::TN + m, xrow = wt * C::TT + m;
  f32x16 acc[C::FT][C::FN];
#pragma unroll
  for (int i = 0; i < C::FT; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = zero_acc16();

  struct Exps {
    int w[C::FN], x[C::FT];
  };
  const int p4 = (h ^ ((m >> 2) & 3)) * 16;
  const int p80 = (h ^ ((m >> 1) & 7)) * 16, p81 = ((2 + h) ^ ((m >> 1) & 7)) * 16;
  auto read_w = [&](int at, int s, int f) {
    return frag4(*reinterpret_cast<const u32x4*>(ring + at + (wrow + 32 * f) * 64 + (p4 ^ (32 * s))));
  };
  auto read_x = [&](int at, int s, int f) {
    const uint8_t* p = ring + at + C::xoff + (xrow + 32 * f) * C::xrow_bytes;
    if constexpr (X8)
      return frag8(*reinterpret_cast<const u32x4*>(p + (p80 ^ (64 * s))), *reinterpret_cast<const u32x4*>(p + (p81 ^ (64 * s))));
    else
      return frag4(*reinterpret_cast<const u32x4*>(p + (p4 ^ (32 * s))));
  };
  // The dwords that hold a step's exponents; shifted into place apart from the
  // read, which takes its time: bytes 0 and 2 are then a lane's own in the two halves.
  auto read_exps = [&](int at, int kb, int kb0, Exps& e) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(ring + at + C::eoff);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) e.w[j] = (int)p[wrow + 32 * j];
#pragma unroll
    for (int i = 0; i < C::FT; ++i) {
      if constexpr (X8) {
        const int d = (kb >> 2) - (kb0 >> 2), r = xrow + 32 * i;
        e.x[i] = (int)xs[r * 8 + ((d ^ (r >> 3)) & 7)];
      } else {
        e.x[i] = (int)p[64 * C::wslots + xrow + 32 * i];
      }
    }
  };
  // Behind the group's last block an 8-bit row's exponent is 0 (2^-127), not the byte
  // that happens to follow: 255 there would make the empty stage's zeros NaN.
  auto shift_exps = [&](int kb, const Exps& e) {
    Exps o;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) o.w[j] = (int)((uint32_t)e.w[j] >> (8 * h));
#pragma unroll
    for (int i = 0; i < C::FT; ++i) {
      if constexpr (X8) o.x[i] = (int)__builtin_amdgcn_ubfe((uint32_t)e.x[i], 8 * (kb & 3), kb < k1 ? 8 : 0);
      else o.x[i] = (int)((uint32_t)e.x[i] >> (8 * h));
    }
    return o;
  };
  i32x8 fw[2][C::FN], fx[2][C::FT];
  // Half s of the group's step i, whose stage is at `at` (the next one's at `nx`):
  // multiplies fragment set s and reads set s ^ 1 (the next half), early, so that
  // nothing is outstanding where the waves meet. The stage of step i is read
  // by then, and takes the panel of step i + S: the first loads in half 1, the
  // others in half 0 of step i + 1.
  constexpr int M = C::FT * C::FN, F = C::FN + C::FT;
  constexpr int early = (F + (M > 1 ? M / 2 : 1) - 1) / (M > 1 ? M / 2 : 1);
  constexpr int ahead = C::loads / 2;  // loads of half 1
  auto half = [&](auto sc, const Exps& e, int at, int nx, int kb, int kb0, Exps& raw) {
    constexpr int s = decltype(sc)::value;
#pragma unroll
    for (int n = 0; n < M; ++n) {
      const int t = n / C::FN, j = n % C::FN;
      acc[t][j] = mfma4_32<X8, s>(fw[s][j], fx[s][t], acc[t][j], e.w[j], e.x[t]);
#pragma unroll
      for (int f = n * early; f < (n + 1) * early && f < F; ++f) {
        if (f < C::FN) fw[s ^ 1][f] = read_w(s ? nx : at, s ^ 1, f);
        else fx[s ^ 1][f - C::FN] = read_x(s ? nx : at, s ^ 1, f - C::FN);
      }
      // (behind the last panel this reads a row that nothing uses)
      if (s == 1 && n == M / 2) read_exps(nx, kb + 1, kb0, raw);
      if (n >= M / 2) {
        constexpr int R = M - M / 2, first = s ? 0 : ahead, count = s ? ahead : C::loads - ahead;
        const int q = n - M / 2;
#pragma unroll
        for (int p = first + q * count / R; p < first + (q + 1) * count / R; ++p) load(p);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if constexpr (X8) load_exps(k0);
#pragma unroll
  for (int s = 0; s < C::S; ++s) {
#pragma unroll
    for (int p = 0; p < (s < C::S - 1 ? C::loads : ahead); ++p) load(p);
    if (s < C::S - 1) next_panel();
  }
  wait_vm<(C::S - 2) * C::loads + ahead>();
  wait_lds();
  ring_barrier<C::waves>();
#pragma unroll
  for (int j = 0; j < C::FN; ++j) fw[0][j] = read_w(0, 0, j);
#pragma unroll
  for (int i = 0; i < C::FT; ++i) fx[0][i] = read_x(0, 0, i);
  const int span = X8 ? kExpBlocks : steps;
  int at = 0;
  for (int i0 = 0; i0 < steps; i0 += span) {
    const int kb0 = k0 + i0;
    if (X8 && i0) {
      load_exps(kb0);
      wait_vm<0>();
      ring_barrier<C::waves>();
    }
    Exps raw;
    read_exps(at, kb0, kb0, raw);
    Exps e = shift_exps(kb0, raw);
    const int i1 = min(steps, i0 + span);
    for (int i = i0; i < i1; ++i) {
      const int nx = at == (C::S - 1) * C::stage ? 0 : at + C::stage;
      half(std::integral_constant<int, 0>{}, e, at, nx, k0 + i, kb0, raw);
      next_panel();
      // step i is in registers; step i + 1 has landed (the later ones may still
      // be in flight); the barrier makes both true for every wave
      wait_vm<(C::S - 2) * C::loads>();
      wait_lds();
      ring_barrier<C::waves>();
      __builtin_amdgcn_sched_barrier(0);
      half(std::integral_constant<int, 1>{}, e, at, nx, k0 + i, kb0, raw);
      e = shift_exps(k0 + i + 1, raw);
      at = nx;
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
  // Epilogue through LDS, so that a row's columns leave in whole lines: 32 tokens
  // at a time in fp32, 8 columns per lane back. What is added to is read before
  // the first store: a load behind a store would wait its whole latency.
  uint8_t* ep = smem + C::parts + wave * 32 * C::eprow;
  constexpr int LPR = C::TN / 8;        // lanes per row
  constexpr int NP = LPR / 2;           // passes over 32 LPR pieces of 8 columns
  auto place = [&](int i, int p, int& r, int& c, uint16_t*& yp) -> bool {
    r = (64 * p + lane) / LPR;
    c = (64 * p + lane) % LPR;
    const int t = t0 + wt * C::TT + 32 * i + r, ncol = n0 + wn * C::TN + 8 * c;
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
        if (place(i, p, r, c, yp))
          old[i][p] = C::STREAM ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(yp)) : ld16(yp);
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
// owns 16 columns and up to 16 tokens; its 8 waves take every eighth panel of
// the sum straight from memory into fragments (16 rows of a panel are one run of
// 1 KB) and their parts are added in wave order. 1 token (8-bit x), us: 2560 -> 2560 2.8,
// which is one launch, 2560 -> 19456 6.4 (4.1 TB/s), 9728 -> 2560 5.8 (ten panels a
// wave, one behind the other). Two to four panels in flight a wave or 16 waves were
// slower where 1216 workgroups fill the GPU (6.4 -> 7.1-9.4 for 2560 -> 19456); with 160
// of them (2560 columns) that was not measured.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;
constexpr int kFewTokens = 16;

template <bool X8, bool ADD>
__global__ __launch_bounds__(64 * kFewWaves) void q4_few_kernel(Mat4Args a) {
  __shared__ alignas(16) float part[kFewWaves][kFewTokens][16 + 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int vn = min(16, a.N - n0), vt = a.T;
  const bool row = r < vt;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < a.nkb; kb += kFewWaves) {
    const __amdgpu_buffer_rsrc_t wr = mk_rsrc(a.w + (int64_t)kb * a.ldw + (int64_t)n0 * 64, vn * 64);
    const __amdgpu_buffer_rsrc_t wer = mk_rsrc(a.we + (int64_t)kb * a.ldwe + (int64_t)n0 * 4, vn * 4);
    const u32x4 w0 = bld16(wr, r * 64 + g * 16);
    const uint32_t ew = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(wer, r * 4, 0, 0) >> (8 * g);
    i32x8 x;
    uint32_t ex;
    if constexpr (X8) {
      const __amdgpu_buffer_rsrc_t xr = mk_rsrc(a.x, (int64_t)(vt - 1) * a.ldx + (int64_t)a.nkb * 128);
      const __amdgpu_buffer_rsrc_t xer = mk_rsrc(a.xe, (int64_t)(vt - 1) * a.ldxe + a.nkb);
      const uint32_t xo = row ? (uint32_t)((int64_t)r * a.ldx) + (uint32_t)kb * 128u + 16u * g : kOff;
      x = frag8(bld16(xr, xo), bld16(xr, xo + 64));
      ex = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(xer, row ? (int)((int64_t)r * a.ldxe) + kb : (int)kOff, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t xr = mk_rsrc(a.x + (int64_t)kb * a.ldx, vt * 64);
      const __amdgpu_buffer_rsrc_t xer = mk_rsrc(a.xe + (int64_t)kb * a.ldxe, vt * 4);
      x = frag4(bld16(xr, r * 64 + g * 16));
      ex = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(xer, r * 4, 0, 0) >> (8 * g);
    }
    acc = mfma4_16<X8>(frag4(w0), x, acc, (int)ew, (int)ex);
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
void launch_tile(Mat4Args a, bool add, hipStream_t s) {
  a.tiles_t = (a.T + C::BT - 1) / C::BT;
  a.tiles_n = (a.N + C::BN - 1) / C::BN;
  const dim3 grid((unsigned)a.tiles_t * (unsigned)a.tiles_n), blk(64 * C::waves * C::KS);
  if (add) hipLaunchKernelGGL((q4_tile_kernel<C, true>), grid, blk, 0, s, a);
  else hipLaunchKernelGGL((q4_tile_kernel<C, false>), grid, blk, 0, s, a);
}

template <bool X8>
void launch_few(const Mat4Args& a, bool add, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 15) / 16)), blk(64 * kFewWaves);
  if (add) hipLaunchKernelGGL((q4_few_kernel<X8, true>), grid, blk, 0, s, a);
  else hipLaunchKernelGGL((q4_few_kernel<X8, false>), grid, blk, 0, s, a);
}

// Tiles to choose from. A workgroup of a tile takes about fixed + step * (its
// panels of the sum) microseconds while `slots` of them run, so a product takes
// that times the rounds its tiles need: a fit to these times on 256 CUs (us, 8-bit x /
// 4-bit x; tiles are tokens x columns, :n the groups of waves that share the sum), of calls
// repeated on the same operands, which the caches then hold.
//   37, 2560, 2560       64x64 7.1/5.8    64x96:2 7.1/6.5   64x64:4 6.6/5.5    32x64:4 5.0/4.5    32x32:4 4.4/3.9
//   37, 9728, 2560       64x64 20.1/15.2  64x96:2 16.1/14.6 64x64:4 13.0/10.2  32x64:4 9.9/8.7    32x32:4 8.0/6.5
//   100, 9728, 2560      64x64 20.1/15.3  64x96:2 16.7/14.7 64x64:4 13.6/10.3  32x64:4 10.2/8.8   32x32:4 14.0/9.2
//   128, 2560, 19456     128x160 12.7/10.9 128x128 11.4/9.8 128x96 10.5/9.4    64x64 15.1/10.6    64x96:2 14.7/10.6
//   256, 9728, 2560      64x64 20.2/15.4  64x96:2 17.0/14.9 64x64:4 14.2/10.9  32x64:4 19.4/13.6  32x32:4 20.9/14.3
//   256, 2560, 19456     256x128 17.5/13.2 128x160 13.6/11.8 128x128 18.0/13.5 128x96 19.3/13.5   64x64 22.3/16.0
//   512, 2560, 2560      128x128 10.7/9.2 128x96 10.0/9.0   64x64 9.0/7.7      64x96:2 7.9/7.0    64x64:4 13.0/10.5
//   512, 4096, 14336     256x128 27.0/21.5 128x160 33.3/27.7 128x128 28.1/22.0 128x96 40.5/28.4
//   2048, 4096, 4096     256x128 28.5/22.1 128x160 33.3/27.8 128x128 29.1/24.1 128x96 41.5/29.4
//   8191, 4096, 4096     256x256 94/69    256x128 117/75    128x128 115/80
//   8192, 4096, 14336    256x256 324/236  256x128 398/249   128x128 386/276
// Over the 34 products it is made from, the choice is the fastest tile of the list or within
// 7% of it, for operands in the caches. Nothing in it stands for the weights' bytes: on
// weights from memory, as a model's layers bring them, it was not fitted. (128x160 has four
// stages: with its operands from memory 256, 2560, 19456 takes 17.3/14.1, with three
// 18.0/15.4, with five 17.7/14.5.)
struct TileChoice {
  int bt, bn, ks, stages, slots;
  float fixed, step;
  void (*launch)(Mat4Args, bool, hipStream_t);
};
template <class C>
constexpr TileChoice choice(int slots, float fixed, float step) {
  return TileChoice{C::BT, C::BN, C::KS, C::S, slots, fixed, step, launch_tile<C>};
}
const TileChoice kTiles8[] = {
    choice<Tile4<256, 256, 2, 2, 3, true, 1, true>>(256, 6.5f, 1.05f),
    choice<Tile4<256, 128, 4, 1, 3, true>>(256, 5.2f, 0.62f),
    choice<Tile4<128, 160, 4, 1, 4, true>>(256, 5.0f, 0.39f),
    choice<Tile4<128, 128, 2, 2, 3, true>>(256, 3.6f, 0.34f),
    choice<Tile4<128, 96, 4, 1, 4, true>>(256, 4.0f, 0.30f),
    choice<Tile4<64, 64, 2, 2, 4, true>>(512, 3.2f, 0.23f),
    choice<Tile4<64, 96, 2, 1, 3, true, 2>>(256, 4.1f, 0.32f),
    choice<Tile4<64, 64, 2, 1, 3, true, 4>>(256, 4.0f, 0.50f),
    choice<Tile4<32, 64, 1, 2, 3, true, 4>>(256, 2.8f, 0.38f),
    choice<Tile4<32, 32, 1, 1, 4, true, 4>>(256, 2.3f, 0.27f),
};
const TileChoice kTiles4[] = {
    choice<Tile4<256, 256, 2, 2, 3, false, 1, true>>(256, 6.2f, 0.66f),
    choice<Tile4<256, 128, 4, 1, 3, false>>(256, 4.8f, 0.41f),
    choice<Tile4<128, 160, 4, 1, 4, false>>(256, 4.7f, 0.32f),
    choice<Tile4<128, 128, 2, 2, 3, false>>(256, 2.8f, 0.27f),
    choice<Tile4<128, 96, 4, 1, 4, false>>(256, 3.1f, 0.23f),
    choice<Tile4<64, 64, 2, 2, 4, false>>(512, 2.7f, 0.17f),
    choice<Tile4<64, 96, 2, 1, 3, false, 2>>(256, 2.8f, 0.30f),
    choice<Tile4<64, 64, 2, 1, 3, false, 4>>(256, 3.6f, 0.36f),
    choice<Tile4<32, 64, 1, 2, 3, false, 4>>(256, 1.6f, 0.33f),
    choice<Tile4<32, 32, 1, 1, 4, false, 4>>(256, 1.2f, 0.20f),
};
constexpr int kTileCount = (int)(sizeof(kTiles8) / sizeof(kTiles8[0]));
static_assert(sizeof(kTiles8) == sizeof(kTiles4), "as many of each");

constexpr int64_t kMaxTiles = 0xffffffffll / 512;

// The tile for T tokens, N columns and a sum of nkb panels; null: the few-token kernel.
const TileChoice* choose(bool x8, int32_t T, int32_t N, int32_t nkb) {
  // Up to one matrix fragment of tokens the weights' bytes are all that counts, as
  // long as x is small: every 16 columns read all of it again. us, few-token kernel
  // and the fastest tile:
  //   tokens, k, n        8-bit x       4-bit x     x read, MB
  //   1, 2560, 2560      2.8   4.2     2.8   3.8       0.4
  //   1, 2560, 19456     6.4   7.6     6.7   7.1         3
  //   1, 9728, 2560      5.8   7.0     5.8   6.3       1.6
  //   16, 2560, 2560     3.7   4.3     2.9   3.8         7
  //   16, 9728, 2560     8.1   7.2     5.9   6.3        25
  //   16, 2560, 19456   10.1   8.0     6.6   7.4        50
  //   16, 4096, 14336   14.8   8.4     7.6   8.0        59
  // (MB of 8-bit x, half as many of 4-bit x.) The border of 32 MB is wrong for the
  // fifth line alone. (A launch holds fewer than 2^32 threads, 512 of them per workgroup.)
  const int64_t again = (int64_t)T * nkb * (x8 ? 128 : 64) * ((N + 15) / 16);
  if (T <= kFewTokens && N <= 1 << 26 && again <= 32 << 20) return nullptr;
  const TileChoice* const all = x8 ? kTiles8 : kTiles4;
  const TileChoice* best = &all[0];  // (its grid is checked by the caller)
  double least = 0.;
  for (int i = 0; i < kTileCount; ++i) {
    const TileChoice& c = all[i];
    const int64_t tiles = ((int64_t)T + c.bt - 1) / c.bt * (((int64_t)N + c.bn - 1) / c.bn);
    const double t = (double)((tiles + c.slots - 1) / c.slots) * (c.fixed + (double)c.step * ((nkb + c.ks - 1) / c.ks));
    if (i == 0 || (t < least && tiles <= kMaxTiles)) best = &c, least = t;
  }
  return best;
}

// The checks that both forms of x share, and the launch.
int product(Mat4Args a, bool x8, const lora_q4_t* w, int32_t x_rows, int32_t x_width, const uint8_t* x_values, void* y,
            int64_t ldy, uint32_t flags, void* stream) {
  int st = check_q4(w, "w");
  if (st) return st;
  if (flags & ~LORA_MATMUL_ACCUMULATE) return set_error(LORA_INVALID_ARGUMENT, "unknown flags 0x%x", flags);
  if (x_width != w->width)
    return set_error(LORA_INVALID_ARGUMENT, "x is %d wide and w %d: the sum runs over both", x_width, w->width);
  if (w->rows & 7) return set_error(LORA_INVALID_ARGUMENT, "w has %d rows (the width of y): a multiple of 8 is needed", w->rows);
  if (x_rows == 0 || w->rows == 0) return LORA_OK;
  if ((st = check_bf16_rows(y, ldy, w->rows, "y"))) return st;
  if (y == x_values || y == w->values) return set_error(LORA_INVALID_ARGUMENT, "y starts at an operand");
  if (((int64_t)x_rows + 255) / 256 * (((int64_t)w->rows + 255) / 256) > kMaxTiles || x_rows > kQ4Most)
    return set_error(LORA_UNSUPPORTED, "y of %d x %d is too large for one call", x_rows, w->rows);
  a.w = w->values; a.ldw = w->ld; a.we = w->exps; a.ldwe = w->ld_exps;
  a.y = static_cast<uint16_t*>(y); a.ldy = ldy;
  a.T = x_rows; a.N = w->rows;
  a.nkb = (int32_t)q4_panels(w->width);
  const bool add = (flags & LORA_MATMUL_ACCUMULATE) != 0;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (const TileChoice* c = choose(x8, a.T, a.N, a.nkb)) c->launch(a, add, s);
  else if (x8) launch_few<true>(a, add, s);
  else launch_few<false>(a, add, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(LORA_DEVICE_ERROR, "q4_matmul launch failed: %s", hipGetErrorString(e));
  return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_q4_matmul(const lora_q4_t* x, const lora_q4_t* w, void* y, int64_t ldy, uint32_t flags, void* stream) {
  clear_error();
  const int st = check_q4(x, "x");
  if (st) return st;
  Mat4Args a{};
  a.x = x->values; a.ldx = x->ld; a.xe = x->exps; a.ldxe = x->ld_exps;
  return product(a, false, w, x->rows, x->width, x->values, y, ldy, flags, stream);
}

extern "C" int lora_q4_matmul_q8(const lora_q8_t* x, const lora_q4_t* w, void* y, int64_t ldy, uint32_t flags, void* stream) {
  clear_error();
  const int st = check_q8(x, "x", 1);
  if (st) return st;
  // a tile's 8-bit rows are addressed with 32-bit offsets from its first row
  const int64_t most = 0x7fffff00 / 256;
  if (x->ld > most || x->ld_exps > most)
    return set_error(LORA_UNSUPPORTED, "row strides above %lld bytes are not supported", (long long)most);
  Mat4Args a{};
  a.x = x->values; a.ldx = x->ld; a.xe = x->exps; a.ldxe = x->ld_exps;
  return product(a, true, w, x->rows, x->width, x->values, y, ldy, flags, stream);
}

// Host-only: the kernel that a product takes (lora_inspect.h)
extern "C" int lora_inspect_matmul4(int32_t x_bits, int32_t num_tokens, int32_t width, int32_t h_out, lora_matmul_kernel_t* out) {
  clear_error();
  if (!out || (x_bits != 8 && x_bits != 4)) return set_error(LORA_INVALID_ARGUMENT, "out is NULL or x_bits (%d) not 8 or 4", x_bits);
  if (num_tokens <= 0 || width <= 0 || h_out <= 0 || (width & 7) || (h_out & 7))
    return set_error(LORA_INVALID_ARGUMENT, "num_tokens (%d), width (%d) and h_out (%d) must be positive, the widths multiples of 8",
                     num_tokens, width, h_out);
  const int32_t nkb = (int32_t)q4_panels(width);
  const TileChoice* c = choose(x_bits == 8, num_tokens, h_out, nkb);
  out->kernels = 1 + kTileCount;
  out->kernel = c ? 1 + (int32_t)(c - (x_bits == 8 ? kTiles8 : kTiles4)) : 0;
  out->tokens = c ? c->bt : kFewTokens;
  out->columns = c ? c->bn : 16;
  out->groups = c ? c->ks : kFewWaves;
  out->stages = c ? c->stages : 0;
  out->blocks = (nkb + out->groups - 1) / out->groups;
  out->exps = c && x_bits == 8 ? kExpBlocks : 0;
  return LORA_OK;
}
