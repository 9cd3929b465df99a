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
__device__ __forceinline__ void load_lds16_at(i32x4 rsrc, uint32_t lds_addr, uint32_t voff, uint32_t soff) {
  int m0_out;
  asm volatile("s_mov_b32 m0, %1\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds"
               : "={m0}"(m0_out)
               : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory");
  (void)m0_out;
}
__device__ __forceinline__ void load_lds4_at(i32x4 rsrc, uint32_t lds_addr, uint32_t voff, uint32_t soff) {
  int m0_out;
  asm volatile("s_mov_b32 m0, %1\n\tbuffer_load_dword %2, %3, %4 offen lds"
               : "={m0}"(m0_out)
               : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory");
  (void)m0_out;
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

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
// Tiled product: BT tokens x BN columns per workgroup of WT x WN waves, the
// sum in steps of one 128-column block through an S-deep ring of LDS stages.
// A stage holds the w rows, the x rows (128 bytes each) and one dword (four
// blocks' exponents) per token and per 128 columns. The 16-byte piece c of row
// r sits at position c ^ swizzle(r), which spreads the 32 rows of a fragment
// over the LDS banks; the loads write LDS directly, so the permutation is
// applied to the address each lane reads from.
// ---------------------------------------------------------------------------
template <int BT_, int BN_, int WT_, int WN_, int S_>
struct Tile {
  static constexpr int BT = BT_, BN = BN_, WT = WT_, WN = WN_, S = S_;
  static constexpr int waves = WT * WN;
  static constexpr int TT = BT / WT, TN = BN / WN;      // a wave's tokens and columns
  static constexpr int FT = TT / 32, FN = TN / 32;      // its fragments
  static constexpr int xoff = BN * 128, eoff = xoff + BT * 128;
  static constexpr int edw = (BT + 64 + 64 * waves - 1) / (64 * waves) * 64 * waves;  // exponent dwords, whole waves
  static constexpr int stage = eoff + edw * 4;
  static constexpr int loads = (BT + BN) / 8 / waves + edw / 64 / waves;  // per wave and stage
  static constexpr int eprow = TN * 4 + 16;             // epilogue row of one token (fp32, padded)
  static constexpr int epi = waves * 32 * eprow;
  static constexpr int lds = S * stage > epi ? S * stage : epi;
  static_assert((BT + BN) % (8 * waves) == 0 && TT % 32 == 0 && TN % 32 == 0, "whole loads and fragments");
  static_assert(lds <= 160 * 1024, "fits the LDS");
};

__device__ __forceinline__ int swizzle(int row) { return row & 7; }

template <class C, bool ADD>
__global__ __launch_bounds__(64 * C::waves) void q8_tile_kernel(MatArgs a) {
  __shared__ alignas(1024) uint8_t smem[C::lds];
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)smem);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tt, tn;
  tile_of(a, blockIdx.x, gridDim.x, tt, tn);
  const int t0 = tt * C::BT, n0 = tn * C::BN;
  const int vt = min(C::BT, a.T - t0), vn = min(C::BN, a.N - n0);  // valid rows of the tile
  const int64_t kbytes = (int64_t)a.nkb * 128;
  const i32x4 wr = mk_rsrc_words(a.w + (int64_t)n0 * a.ldw, (int64_t)(vn - 1) * a.ldw + kbytes);
  const i32x4 xr = mk_rsrc_words(a.x + (int64_t)t0 * a.ldx, (int64_t)(vt - 1) * a.ldx + kbytes);
  const i32x4 xer = mk_rsrc_words(a.xe + (int64_t)t0 * a.ldxe, (int64_t)(vt - 1) * a.ldxe + ((a.nkb + 3) & ~3));
  const int eb0 = n0 >> 7, vb = ((n0 + vn - 1) >> 7) - eb0 + 1;
  const i32x4 wer = mk_rsrc_words(a.we + (int64_t)eb0 * a.ldwe, (int64_t)(vb - 1) * a.ldwe + ((a.nkb + 3) & ~3));

  constexpr int PW = (C::BN + C::BT) / 8 / C::waves;  // 1 KB pieces (8 rows) per wave
  // Piece p of the wave: rows 8 (p * waves + wave) .. + 7 of the stage (w rows, then x rows).
  uint32_t voff[PW];
#pragma unroll
  for (int p = 0; p < PW; ++p) {
    const int r = 8 * (p * C::waves + wave) + (lane >> 3);
    const int c = (lane & 7) ^ swizzle(r);
    const bool isx = 8 * (p * C::waves + wave) >= C::BN;
    voff[p] = (uint32_t)(isx ? (int64_t)(r - C::BN) * a.ldx : (int64_t)r * a.ldw) + 16u * c;
  }
  constexpr int PE = C::edw / 64 / C::waves;
  uint32_t eoffs[PE];
#pragma unroll
  for (int p = 0; p < PE; ++p) {
    const int i = 64 * (p * C::waves + wave);  // first dword of the piece
    const bool isx = i < C::BT;
    const int r = isx ? i + lane : i + lane - C::BT;
    eoffs[p] = (uint32_t)((int64_t)r * (isx ? a.ldxe : a.ldwe));
  }
  auto issue = [&](int kb) {
    const uint32_t st = lds0 + (uint32_t)(kb % C::S) * C::stage;
#pragma unroll
    for (int p = 0; p < PW; ++p) {
      const int piece = p * C::waves + wave;
      const bool isx = 8 * piece >= C::BN;
      i32x4 r = wr;
      if (isx) r = xr;
      load_lds16_at(r, st + piece * 1024, voff[p], (uint32_t)kb * 128u);
    }
#pragma unroll
    for (int p = 0; p < PE; ++p) {
      const int i = 64 * (p * C::waves + wave);
      i32x4 r = wer;
      if (i < C::BT) r = xer;
      load_lds4_at(r, st + C::eoff + i * 4, eoffs[p], (uint32_t)(kb & ~3));
    }
  };

  const int wt = wave / C::WN, wn = wave % C::WN;
  const int m = lane & 31, h = lane >> 5;
  const int wrow = wn * C::TN + m, xrow = wt * C::TT + m;
  const int edw_w = C::BT + (((n0 + wn * C::TN) >> 7) - eb0);
  f32x16 acc[C::FT][C::FN];
#pragma unroll
  for (int i = 0; i < C::FT; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = zero_acc16();

#pragma unroll
  for (int s = 0; s < C::S - 1; ++s)
    if (s < a.nkb) issue(s);
  for (int kb = 0; kb < a.nkb; ++kb) {
    // stage kb has landed (the later ones may still be in flight), and every
    // wave is done with the stage that the next loads overwrite
    if (kb + C::S - 1 <= a.nkb) wait_vm<(C::S - 2) * C::loads>();
    else wait_vm<0>();
    wait_lds();
    __builtin_amdgcn_s_barrier();
    if (kb + C::S - 1 < a.nkb) issue(kb + C::S - 1);
    const uint8_t* st = smem + (kb % C::S) * C::stage;
    const uint32_t* es = reinterpret_cast<const uint32_t*>(st + C::eoff);
    const int sh = 8 * (kb & 3);
    const int ew = (int)(es[edw_w] >> sh);
    int ex[C::FT];
#pragma unroll
    for (int i = 0; i < C::FT; ++i) ex[i] = (int)(es[xrow + 32 * i] >> sh);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int c0 = ((4 * s + 2 * h) ^ swizzle(m)) * 16, c1 = ((4 * s + 2 * h + 1) ^ swizzle(m)) * 16;
      i32x8 fw[C::FN], fx[C::FT];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const uint8_t* p = st + (wrow + 32 * j) * 128;
        fw[j] = frag(*reinterpret_cast<const u32x4*>(p + c0), *reinterpret_cast<const u32x4*>(p + c1));
      }
#pragma unroll
      for (int i = 0; i < C::FT; ++i) {
        const uint8_t* p = st + C::xoff + (xrow + 32 * i) * 128;
        fx[i] = frag(*reinterpret_cast<const u32x4*>(p + c0), *reinterpret_cast<const u32x4*>(p + c1));
      }
#pragma unroll
      for (int i = 0; i < C::FT; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = mfma8_32(fw[j], fx[i], acc[i][j], ew, ex[i]);
    }
  }
  // Epilogue through LDS, so that a row's columns leave in whole lines:
  // 32 tokens at a time in fp32, 8 columns per lane back.
  wait_lds();
  __builtin_amdgcn_s_barrier();
  uint8_t* ep = smem + wave * 32 * C::eprow;
  constexpr int LPR = C::TN / 8;        // lanes per row
  constexpr int RPP = 64 / LPR;         // rows per pass
  const int ncol = n0 + wn * C::TN + 8 * (lane % LPR);
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
    for (int p = 0; p < 32 / RPP; ++p) {
      const int r = p * RPP + lane / LPR;
      const int t = t0 + wt * C::TT + 32 * i + r;
      const f32x4 v0 = *reinterpret_cast<const f32x4*>(ep + r * C::eprow + (lane % LPR) * 32);
      const f32x4 v1 = *reinterpret_cast<const f32x4*>(ep + r * C::eprow + (lane % LPR) * 32 + 16);
      if (t < a.T && ncol < a.N) {
        uint16_t* yp = a.y + (int64_t)t * a.ldy + ncol;
        float f[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
        if constexpr (ADD) {
          float o[8];
          unpack8(ld16(yp), o);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] += o[e];
        }
        st16(yp, pack8(f));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Few tokens: the weights are read once and that is the floor. A workgroup
// owns 16 columns and up to 16 TF tokens; its 8 waves take every eighth block
// of the sum straight from memory into fragments (no LDS on the way, each w
// row in whole 128-byte lines) and their parts are added in wave order.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;
constexpr int kFewDepth = 2;  // blocks whose loads a wave has in flight

template <int TF, bool ADD>
__global__ __launch_bounds__(64 * kFewWaves) void q8_few_kernel(MatArgs a) {
  __shared__ alignas(16) float part[kFewWaves][TF * 16][16 + 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * (16 * TF);
  const int vn = min(16, a.N - n0), vt = min(16 * TF, a.T - t0);
  const int64_t kbytes = (int64_t)a.nkb * 128;
  const __amdgpu_buffer_rsrc_t wr = mk_rsrc(a.w + (int64_t)n0 * a.ldw, (int64_t)(vn - 1) * a.ldw + kbytes);
  const __amdgpu_buffer_rsrc_t xr = mk_rsrc(a.x + (int64_t)t0 * a.ldx, (int64_t)(vt - 1) * a.ldx + kbytes);
  const __amdgpu_buffer_rsrc_t xer = mk_rsrc(a.xe + (int64_t)t0 * a.ldxe, (int64_t)(vt - 1) * a.ldxe + a.nkb);
  const __amdgpu_buffer_rsrc_t wer = mk_rsrc(a.we + (int64_t)(n0 >> 7) * a.ldwe, a.nkb);
  f32x4 acc[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kb0 = wave; kb0 < a.nkb; kb0 += kFewWaves * kFewDepth) {
    u32x4 w[kFewDepth][2], x[kFewDepth][TF][2];
    int ew[kFewDepth], ex[kFewDepth][TF];
#pragma unroll
    for (int d = 0; d < kFewDepth; ++d) {
      const int kb = kb0 + d * kFewWaves;
      const bool in = kb < a.nkb;
      const uint32_t k = (uint32_t)kb * 128u + 32u * g;
      const uint32_t wo = in ? (uint32_t)((int64_t)r * a.ldw) + k : kOff;
      w[d][0] = bld16(wr, wo);
      w[d][1] = bld16(wr, wo + 16);
      ew[d] = __builtin_amdgcn_raw_buffer_load_b8(wer, in ? kb : (int)kOff, 0, 0);
#pragma unroll
      for (int f = 0; f < TF; ++f) {
        const uint32_t xo = in && 16 * f + r < vt ? (uint32_t)((int64_t)(16 * f + r) * a.ldx) + k : kOff;
        x[d][f][0] = bld16(xr, xo);
        x[d][f][1] = bld16(xr, xo + 16);
        ex[d][f] = __builtin_amdgcn_raw_buffer_load_b8(
            xer, in && 16 * f + r < vt ? (int)((int64_t)(16 * f + r) * a.ldxe) + kb : (int)kOff, 0, 0);
      }
    }
#pragma unroll
    for (int d = 0; d < kFewDepth; ++d)
#pragma unroll
      for (int f = 0; f < TF; ++f)
        acc[f] = mfma8_16(frag(w[d][0], w[d][1]), frag(x[d][f][0], x[d][f][1]), acc[f], ew[d], ex[d][f]);
  }
#pragma unroll
  for (int f = 0; f < TF; ++f) *reinterpret_cast<f32x4*>(&part[wave][16 * f + r][4 * g]) = acc[f];
  __syncthreads();
  for (int i = threadIdx.x; i < TF * 32; i += 64 * kFewWaves) {
    const int t = i >> 1, c = (i & 1) * 8;
    if (t >= vt || n0 + c >= a.N) continue;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
#pragma unroll
    for (int wv = 0; wv < kFewWaves; ++wv)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += part[wv][t][c + e];
    uint16_t* yp = a.y + (int64_t)(t0 + t) * a.ldy + n0 + c;
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
  const dim3 grid((unsigned)a.tiles_t * (unsigned)a.tiles_n), blk(64 * C::waves);
  if (add) hipLaunchKernelGGL((q8_tile_kernel<C, true>), grid, blk, 0, s, a);
  else hipLaunchKernelGGL((q8_tile_kernel<C, false>), grid, blk, 0, s, a);
}

template <int TF>
void launch_few(const MatArgs& a, bool add, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.T + 16 * TF - 1) / (16 * TF))), blk(64 * kFewWaves);
  if (add) hipLaunchKernelGGL((q8_few_kernel<TF, true>), grid, blk, 0, s, a);
  else hipLaunchKernelGGL((q8_few_kernel<TF, false>), grid, blk, 0, s, a);
}

using Tile256 = Tile<256, 256, 2, 4, 2>;
using Tile128 = Tile<128, 128, 2, 2, 2>;

void launch_matmul(const MatArgs& a, bool add, hipStream_t s) {
  if (a.T <= 16) launch_few<1>(a, add, s);
  else if (a.T <= 32) launch_few<2>(a, add, s);
  else if (a.T <= 64) launch_few<4>(a, add, s);
  else if ((int64_t)((a.T + 255) / 256) * ((a.N + 255) / 256) >= 256) launch_tile<Tile256>(a, add, s);
  else launch_tile<Tile128>(a, add, s);
}

}  // namespace
}  // namespace lora

#ifndef LORA_Q8_KERNELS_ONLY
using namespace lora;

extern "C" int lora_q8_matmul(const lora_q8_t* x, const lora_q8_t* w, void* y, int64_t ldy, uint32_t flags, void* stream) {
  set_error(LORA_OK, "%s", "");
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
#endif
