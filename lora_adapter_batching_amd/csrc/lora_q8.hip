// lora_q8.hip -- rows and weights stored in 8 bits (e4m3 with one
// power-of-two scale per block of 128), their restore, and the gated
// activation between two projections, which can write its result straight
// into the 8-bit form that the next projection reads.
//
// All of these are one pass over the data: their floor is the bytes they
// move. A chunk is 8 columns of one row (16 bytes of bf16, 8 of e4m3); 16
// consecutive lanes hold the 16 chunks of one 128-column block, so a block's
// largest magnitude is four DPP steps and never touches memory.
#include <hip/hip_runtime.h>

#include "lora_internal.h"
#include "lora_q8.h"

namespace lora {
namespace {

constexpr int kRowThreads = 256;

// (row, chunk) of a linear chunk index, counted over rows of cpr chunks.
// The workgroup's first chunk is divided in 64 bits (scalar), what lies
// inside the workgroup in 32.
struct ChunkAt {
  int64_t row;
  int chunk;
};
struct ChunkBase {
  int64_t row0;
  uint32_t in_row, cpr;
  __device__ __forceinline__ ChunkBase(int64_t first, uint32_t chunks_per_row) {
    row0 = first / chunks_per_row;
    in_row = (uint32_t)(first - row0 * chunks_per_row);
    cpr = chunks_per_row;
  }
  __device__ __forceinline__ ChunkAt at(uint32_t i) const {
    const uint32_t j = in_row + i, r = j / cpr;
    return ChunkAt{row0 + r, (int)(j - r * cpr)};
  }
};

// 16 bytes of bf16 that the launch touches once. In large batches (NT) they go
// past the caches, which then keep the 8-bit rows for the kernel that reads them
// next: 65536 x 3584 stored and restored 254 -> 225 us, the activation of 16384 x
// 9728 and its restore 285 -> 254, its gradient 285 -> 255 (6.25 TB/s). Small ones
// keep plain accesses: their output is the next kernel's input.
template <bool NT>
__device__ __forceinline__ u32x4 ld_once(const uint16_t* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  else return ld16(p);
}
template <bool NT>
__device__ __forceinline__ void st_once(uint16_t* p, u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  else st16(p, v);
}

// Stores 8 floats of one chunk in 8 bits; every lane of the chunk's block
// takes part.
__device__ __forceinline__ void store_chunk(const float (&f)[8], bool live, uint8_t* values, int64_t ld, uint8_t* exps,
                                            int64_t ld_exps, int64_t row, int chunk) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, finite_abs(f[i]));
  m = max_over_16(m);
  const uint32_t e = q8_exponent(m);
  const float inv = q8_scale(254u - e);  // 2^(127 - e): the quotient is exact
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = pack_e4m3(f[4 * h] * inv, f[4 * h + 1] * inv, f[4 * h + 2] * inv, f[4 * h + 3] * inv);
  if (live) {
    *reinterpret_cast<uint2*>(values + row * ld + 8 * chunk) = make_uint2(w[0], w[1]);
    if ((chunk & 15) == 0) exps[row * ld_exps + (chunk >> 4)] = (uint8_t)e;
  }
}

struct RowsArgs {
  const uint16_t* x;
  int64_t ldx;
  uint8_t* values;
  int64_t ld;
  uint8_t* exps;
  int64_t ld_exps;
  int64_t chunks;  // rows * cpr
  uint32_t cpr;    // chunks per stored row (16 per block)
  int32_t width;
};

template <int U>
__global__ __launch_bounds__(kRowThreads) void q8_rows_kernel(RowsArgs a) {
  const int64_t first = (int64_t)blockIdx.x * (kRowThreads * U);
  const ChunkBase base(first, a.cpr);
  ChunkAt at[U];
  bool live[U];
  u32x4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = threadIdx.x + kRowThreads * u;
    at[u] = base.at(i);
    live[u] = first + i < a.chunks;
    v[u] = zero16();
    if (live[u] && 8 * at[u].chunk < a.width) v[u] = ld_once<(U > 1)>(a.x + at[u].row * a.ldx + 8 * at[u].chunk);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float f[8];
    unpack8(v[u], f);
    store_chunk(f, live[u], a.values, a.ld, a.exps, a.ld_exps, at[u].row, at[u].chunk);
  }
}

struct RestoreArgs {
  const uint8_t* values;
  int64_t ld;
  const uint8_t* exps;
  int64_t ld_exps;
  uint16_t* x;
  int64_t ldx;
  int64_t chunks;  // rows * cpr
  uint32_t cpr;    // chunks of 8 columns per restored row
  int32_t row_shift;  // exponent row = row >> row_shift (0 rows, 7 weights)
};

// e4m3 times a power of two has 4 significant bits: its bf16 value is exact.
__device__ __forceinline__ u32x4 restore8(uint2 q, float scale) {
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, scale, false));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, scale, true));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, scale, false));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, scale, true));
  return v;
}

template <int U>
__global__ __launch_bounds__(kRowThreads) void q8_restore_kernel(RestoreArgs a) {
  const int64_t first = (int64_t)blockIdx.x * (kRowThreads * U);
  const ChunkBase base(first, a.cpr);
  ChunkAt at[U];
  uint2 q[U];
  uint32_t e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = threadIdx.x + kRowThreads * u;
    at[u] = base.at(i);
    q[u] = make_uint2(0u, 0u);
    e[u] = 1;
    if (first + i < a.chunks) {
      q[u] = *reinterpret_cast<const uint2*>(a.values + at[u].row * a.ld + 8 * at[u].chunk);
      e[u] = a.exps[(at[u].row >> a.row_shift) * a.ld_exps + (at[u].chunk >> 4)];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (first + threadIdx.x + kRowThreads * u < a.chunks)
      st_once<(U > 1)>(a.x + at[u].row * a.ldx + 8 * at[u].chunk, restore8(q[u], q8_scale(e[u])));
}

// Weights: one workgroup per 128 x 128 block, which writes the block in both
// orientations (the product's and its gradient's), with the same exponent. Read
// once, so bound by memory: 19456 x 2560 29.9 us (5.0 TB/s), 42 us with the
// transposed store (4.7 TB/s; its bytes go through LDS one by one, which that
// time holds); 2560 x 2560, 400 workgroups, 6.6 and 8.9 us.
struct WeightsArgs {
  const uint16_t* w;
  int64_t ldw;
  int32_t rows, width;
  uint8_t* values;
  int64_t ld;
  uint8_t* exps;
  int64_t ld_exps;
  uint8_t* values_t;  // or null
  int64_t ld_t;
  uint8_t* exps_t;
  int64_t ld_exps_t;
  int32_t col_blocks;
};

__global__ __launch_bounds__(256) void q8_weights_kernel(WeightsArgs a) {
  __shared__ float wave_max[4];
  __shared__ alignas(16) uint8_t tile[128][128 + 4];
  const int rb = blockIdx.x / a.col_blocks, cb = blockIdx.x - rb * a.col_blocks;
  const int chunk = threadIdx.x & 15, r0 = threadIdx.x >> 4;  // 16 rows per pass
  u32x4 v[8];
  float m = 0.f;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = rb * 128 + r0 + 16 * p, c = cb * 128 + 8 * chunk;
    v[p] = zero16();
    if (r < a.rows && c < a.width) v[p] = ld16(a.w + (int64_t)r * a.ldw + c);
    float f[8];
    unpack8(v[p], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, finite_abs(f[i]));
  }
  m = max_over_16(m);
  m = __builtin_fmaxf(m, __shfl_xor(m, 16));
  m = __builtin_fmaxf(m, __shfl_xor(m, 32));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
  __syncthreads();
  m = __builtin_fmaxf(__builtin_fmaxf(wave_max[0], wave_max[1]), __builtin_fmaxf(wave_max[2], wave_max[3]));
  const uint32_t e = q8_exponent(m);
  const float inv = q8_scale(254u - e);
  if (threadIdx.x == 0) {
    a.exps[rb * a.ld_exps + cb] = (uint8_t)e;
    if (a.values_t) a.exps_t[cb * a.ld_exps_t + rb] = (uint8_t)e;
  }
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    float f[8];
    unpack8(v[p], f);
    const int lr = r0 + 16 * p, r = rb * 128 + lr;
    const uint32_t q0 = pack_e4m3(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    const uint32_t q1 = pack_e4m3(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    if (r < a.rows)
      *reinterpret_cast<uint2*>(a.values + (int64_t)r * a.ld + cb * 128 + 8 * chunk) = make_uint2(q0, q1);
    *reinterpret_cast<uint32_t*>(&tile[lr][8 * chunk]) = q0;
    *reinterpret_cast<uint32_t*>(&tile[lr][8 * chunk + 4]) = q1;
  }
  if (!a.values_t) return;
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int lc = r0 + 16 * p, c = cb * 128 + lc;  // row of the transposed block
    uint32_t q[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i >> 2] |= (uint32_t)tile[8 * chunk + i][lc] << (8 * (i & 3));
    if (c < a.width)
      *reinterpret_cast<uint2*>(a.values_t + (int64_t)c * a.ld_t + rb * 128 + 8 * chunk) = make_uint2(q[0], q[1]);
  }
}

// ---------------------------------------------------------------------------
// Gated activation
// ---------------------------------------------------------------------------
// sigma(g) with the hardware's exp2 and reciprocal (an ulp or two each; the
// results are rounded to 8 bits of mantissa or fewer).
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
}

struct GateArgs {
  const uint16_t* gate_up;
  int64_t ld;
  const uint16_t* dh;  // backward only
  int64_t lddh;
  uint16_t* out;  // h, or dgate_up; or null
  int64_t ldo;
  uint8_t* values;  // 8-bit rows; or null
  int64_t ldq;
  uint8_t* exps;
  int64_t ld_exps;
  int64_t chunks;
  uint32_t cpr;
  int32_t width;  // F
};

// 16384 x 9728: bf16 rows 156 us, 8-bit rows 142, both 193 (5.6 to 6.1 TB/s); 256 x
// 9728 5.1 to 5.9.
template <int U, bool BF, bool Q>
__global__ __launch_bounds__(kRowThreads) void swiglu_kernel(GateArgs a) {
  const int64_t first = (int64_t)blockIdx.x * (kRowThreads * U);
  const ChunkBase base(first, a.cpr);
  ChunkAt at[U];
  bool live[U], in[U];
  u32x4 g[U], p[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = threadIdx.x + kRowThreads * u;
    at[u] = base.at(i);
    live[u] = first + i < a.chunks;
    in[u] = live[u] && 8 * at[u].chunk < a.width;
    g[u] = p[u] = zero16();
    if (in[u]) {
      const uint16_t* r = a.gate_up + at[u].row * a.ld + 8 * at[u].chunk;
      g[u] = ld_once<(U > 1)>(r);
      p[u] = ld_once<(U > 1)>(r + a.width);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float gf[8], pf[8], h[8];
    unpack8(g[u], gf);
    unpack8(p[u], pf);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = gf[i] * sigmoid(gf[i]) * pf[i];
    if constexpr (BF) {
      if (in[u]) st_once<(U > 1)>(a.out + at[u].row * a.ldo + 8 * at[u].chunk, pack8(h));
    }
    if constexpr (Q) store_chunk(h, live[u], a.values, a.ldq, a.exps, a.ld_exps, at[u].row, at[u].chunk);
  }
}

// dh meets sigma first: a closed gate's sigma then takes its size down before the
// other factor can take the product out of fp32's range (dh u past 3.4e38 was
// infinite, and times a sigma of 0 not a number).
__device__ __forceinline__ void gate_grad(u32x4 g, u32x4 p, u32x4 d, float (&dg)[8], float (&dp)[8]) {
  float gf[8], pf[8], df[8];
  unpack8(g, gf);
  unpack8(p, pf);
  unpack8(d, df);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = sigmoid(gf[i]);
    const float t = df[i] * s;
    dg[i] = t * pf[i] * (1.f + gf[i] * (1.f - s));
    dp[i] = t * gf[i];
  }
}

// One chunk of gate and the same chunk of up per lane; with 8-bit output the
// two halves' blocks are whole (F a multiple of 128). 16384 x 9728: bf16 253 us,
// 8 bits 228, both 330 (5.6 to 6.3 TB/s); 256 x 9728 6.1 to 7.5.
template <bool NT, bool BF, bool Q>
__global__ __launch_bounds__(kRowThreads) void swiglu_backward_kernel(GateArgs a) {
  const int64_t first = (int64_t)blockIdx.x * kRowThreads;
  const ChunkAt at = ChunkBase(first, a.cpr).at(threadIdx.x);
  const bool live = first + threadIdx.x < a.chunks;
  u32x4 g = zero16(), p = g, d = g;
  if (live) {
    const uint16_t* r = a.gate_up + at.row * a.ld + 8 * at.chunk;
    g = ld_once<NT>(r);
    p = ld_once<NT>(r + a.width);
    d = ld_once<NT>(a.dh + at.row * a.lddh + 8 * at.chunk);
  }
  float dg[8], dp[8];
  gate_grad(g, p, d, dg, dp);
  if constexpr (BF) {
    if (live) {
      uint16_t* o = a.out + at.row * a.ldo + 8 * at.chunk;
      st_once<NT>(o, pack8(dg));
      st_once<NT>(o + a.width, pack8(dp));
    }
  }
  if constexpr (Q) {
    store_chunk(dg, live, a.values, a.ldq, a.exps, a.ld_exps, at.row, at.chunk);
    store_chunk(dp, live, a.values, a.ldq, a.exps, a.ld_exps, at.row, at.chunk + (a.width >> 3));
  }
}

// F not a multiple of 128: a block of the 8-bit row may hold the end of the
// gate half and the start of the up half, so each lane makes one chunk of
// the whole row. The inputs are read once for each half, the second time from the
// caches at best, and both gradients computed for each: 16384 x 9736 takes 313 us
// into 8 bits and 402 into both forms, where whole halves (9728) take 228 and 330.
template <bool BF>
__global__ __launch_bounds__(kRowThreads) void swiglu_backward_split_kernel(GateArgs a) {
  const int64_t first = (int64_t)blockIdx.x * kRowThreads;
  const ChunkBase base(first, a.cpr);
  const ChunkAt at = base.at(threadIdx.x);
  const bool live = first + threadIdx.x < a.chunks;
  const int fc = a.width >> 3;  // chunks of one half
  const bool in = live && at.chunk < 2 * fc;
  const bool up = at.chunk >= fc;
  u32x4 g = zero16(), p = g, d = g;
  if (in) {
    const int c = 8 * (up ? at.chunk - fc : at.chunk);
    const uint16_t* r = a.gate_up + at.row * a.ld + c;
    g = ld16(r);
    p = ld16(r + a.width);
    d = ld16(a.dh + at.row * a.lddh + c);
  }
  float dg[8], dp[8], o[8];
  gate_grad(g, p, d, dg, dp);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = up ? dp[i] : dg[i];
  if constexpr (BF) {
    if (in) st16(a.out + at.row * a.ldo + 8 * at.chunk, pack8(o));
  }
  store_chunk(o, live, a.values, a.ldq, a.exps, a.ld_exps, at.row, at.chunk);
}

// Large batches (8 M elements) keep several chunks per thread in flight and
// stream; small ones spread over as many workgroups as they have.
constexpr int kManyChunks = 4;
bool many(int64_t chunks) { return chunks >= (int64_t)1 << 20; }

int64_t groups(int64_t chunks, int per_thread) {
  return (chunks + (int64_t)kRowThreads * per_thread - 1) / ((int64_t)kRowThreads * per_thread);
}

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(LORA_DEVICE_ERROR, "%s launch failed: %s", what, hipGetErrorString(e));
  return LORA_OK;
}

// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxGroups = 0xffffffffll / kRowThreads;
bool too_many(int64_t chunks) { return groups(chunks, many(chunks) ? 2 : 1) > kMaxGroups; }

}  // namespace

int check_bf16_rows(const void* p, int64_t ld, int64_t width, const char* name) {
  if (!p) return set_error(LORA_INVALID_ARGUMENT, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & 15u) return set_error(LORA_INVALID_ARGUMENT, "%s is not 16-byte aligned", name);
  if (ld < width)
    return set_error(LORA_INVALID_ARGUMENT, "row stride of %s (%lld) is below its width %lld", name, (long long)ld,
                     (long long)width);
  if (ld & 7) return set_error(LORA_INVALID_ARGUMENT, "row stride of %s (%lld) is not a multiple of 8", name, (long long)ld);
  return LORA_OK;
}

int check_q8(const lora_q8_t* q, const char* name, int block_rows) {
  if (!q) return set_error(LORA_INVALID_ARGUMENT, "%s is NULL", name);
  if (q->rows < 0 || q->width <= 0 || (q->width & 7))
    return set_error(LORA_INVALID_ARGUMENT, "%s: rows (%d) must be >= 0 and width (%d) a positive multiple of 8", name,
                     q->rows, q->width);
  if (q->block_rows != 1 && q->block_rows != kQ8Block)
    return set_error(LORA_INVALID_ARGUMENT, "%s: block_rows must be 1 or 128, got %d", name, q->block_rows);
  if (block_rows && q->block_rows != block_rows)
    return set_error(LORA_INVALID_ARGUMENT, "%s: block_rows must be %d here, got %d", name, block_rows, q->block_rows);
  if (q->ld < q8_blocks(q->width) * kQ8Block || (q->ld & 15))
    return set_error(LORA_INVALID_ARGUMENT, "%s: row stride %lld must be a multiple of 16 and hold %lld bytes (whole blocks of 128)",
                     name, (long long)q->ld, (long long)(q8_blocks(q->width) * kQ8Block));
  if (q->ld_exps < q8_blocks(q->width) || (q->ld_exps & 3))
    return set_error(LORA_INVALID_ARGUMENT, "%s: exponent stride %lld must be a multiple of 4 and hold %lld blocks", name,
                     (long long)q->ld_exps, (long long)q8_blocks(q->width));
  if (q->rows == 0) return LORA_OK;
  if (!q->values || !q->exps) return set_error(LORA_INVALID_ARGUMENT, "%s: values/exps is NULL", name);
  if ((reinterpret_cast<uintptr_t>(q->values) & 15u) || (reinterpret_cast<uintptr_t>(q->exps) & 3u))
    return set_error(LORA_INVALID_ARGUMENT, "%s: values must be 16-byte and exps 4-byte aligned", name);
  return LORA_OK;
}

}  // namespace lora

using namespace lora;

extern "C" int lora_q8_quantize(const void* x, int64_t ldx, const lora_q8_t* out, const lora_q8_t* out_t, void* stream) {
  clear_error();
  int st = check_q8(out, "out", 0);
  if (st) return st;
  if (out_t) {
    if (out->block_rows != kQ8Block)
      return set_error(LORA_INVALID_ARGUMENT, "a transposed store needs 128 x 128 blocks (out->block_rows = 128)");
    if ((st = check_q8(out_t, "out_t", kQ8Block))) return st;
    if (out_t->rows != out->width || out_t->width != out->rows)
      return set_error(LORA_INVALID_ARGUMENT, "out_t is %d x %d, the transpose of out is %d x %d", out_t->rows, out_t->width,
                       out->width, out->rows);
  }
  if (out->rows == 0) return LORA_OK;
  if ((st = check_bf16_rows(x, ldx, out->width, "x"))) return st;
  if (x == out->values || (out_t && (x == out_t->values || out->values == out_t->values)))
    return set_error(LORA_INVALID_ARGUMENT, "a store starts at x or at the other store");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (out->block_rows == kQ8Block) {
    WeightsArgs a{};
    a.w = static_cast<const uint16_t*>(x); a.ldw = ldx;
    a.rows = out->rows; a.width = out->width;
    a.values = out->values; a.ld = out->ld; a.exps = out->exps; a.ld_exps = out->ld_exps;
    if (out_t) {
      a.values_t = out_t->values; a.ld_t = out_t->ld; a.exps_t = out_t->exps; a.ld_exps_t = out_t->ld_exps;
    }
    a.col_blocks = (int)q8_blocks(out->width);
    const int64_t n = q8_blocks(out->rows) * a.col_blocks;
    if (n > kMaxGroups) return set_error(LORA_UNSUPPORTED, "x of %d x %d is too large for one call", out->rows, out->width);
    hipLaunchKernelGGL(q8_weights_kernel, dim3((unsigned)n), dim3(256), 0, s, a);
    return launched("q8_weights");
  }
  RowsArgs a{};
  a.x = static_cast<const uint16_t*>(x); a.ldx = ldx;
  a.values = out->values; a.ld = out->ld; a.exps = out->exps; a.ld_exps = out->ld_exps;
  a.width = out->width;
  a.cpr = (uint32_t)q8_blocks(out->width) * 16;
  a.chunks = (int64_t)out->rows * a.cpr;
  if (too_many(a.chunks)) return set_error(LORA_UNSUPPORTED, "x of %d x %d is too large for one call", out->rows, out->width);
  if (many(a.chunks))
    hipLaunchKernelGGL(q8_rows_kernel<kManyChunks>, dim3((unsigned)groups(a.chunks, kManyChunks)), dim3(kRowThreads), 0, s, a);
  else
    hipLaunchKernelGGL(q8_rows_kernel<1>, dim3((unsigned)groups(a.chunks, 1)), dim3(kRowThreads), 0, s, a);
  return launched("q8_rows");
}

extern "C" int lora_q8_dequantize(const lora_q8_t* q, void* x, int64_t ldx, void* stream) {
  clear_error();
  int st = check_q8(q, "q", 0);
  if (st) return st;
  if (q->rows == 0) return LORA_OK;
  if ((st = check_bf16_rows(x, ldx, q->width, "x"))) return st;
  if (x == q->values) return set_error(LORA_INVALID_ARGUMENT, "x starts at the store");
  RestoreArgs a{};
  a.values = q->values; a.ld = q->ld; a.exps = q->exps; a.ld_exps = q->ld_exps;
  a.x = static_cast<uint16_t*>(x); a.ldx = ldx;
  a.cpr = (uint32_t)q->width / 8;
  a.chunks = (int64_t)q->rows * a.cpr;
  a.row_shift = q->block_rows == kQ8Block ? 7 : 0;
  if (too_many(a.chunks)) return set_error(LORA_UNSUPPORTED, "q of %d x %d is too large for one call", q->rows, q->width);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (many(a.chunks))
    hipLaunchKernelGGL(q8_restore_kernel<kManyChunks>, dim3((unsigned)groups(a.chunks, kManyChunks)), dim3(kRowThreads), 0, s, a);
  else
    hipLaunchKernelGGL(q8_restore_kernel<1>, dim3((unsigned)groups(a.chunks, 1)), dim3(kRowThreads), 0, s, a);
  return launched("q8_restore");
}

// Checks shared by the two directions of the gated activation; out_width is
// the width of its outputs (F or 2F).
static int gate_checks(const void* gate_up, int64_t ld, int32_t tokens, int32_t width, const void* out, int64_t ldo,
                       const lora_q8_t* outq, int64_t out_width, const char* oname, const char* qname) {
  if (tokens < 0 || width <= 0 || (width & 7))
    return set_error(LORA_INVALID_ARGUMENT, "num_tokens (%d) must be >= 0 and width (%d) a positive multiple of 8", tokens, width);
  if (width > 0x3fffffff) return set_error(LORA_UNSUPPORTED, "width %d is too large", width);
  if (!out && !outq) return set_error(LORA_INVALID_ARGUMENT, "%s and %s are both NULL", oname, qname);
  int st;
  if (outq) {
    if ((st = check_q8(outq, qname, 1))) return st;
    if (outq->rows != tokens || outq->width != out_width)
      return set_error(LORA_INVALID_ARGUMENT, "%s is %d x %d, expected %d x %lld", qname, outq->rows, outq->width, tokens,
                       (long long)out_width);
  }
  if (tokens == 0) return LORA_OK;
  if ((st = check_bf16_rows(gate_up, ld, 2 * (int64_t)width, "gate_up"))) return st;
  if (out && (st = check_bf16_rows(out, ldo, out_width, oname))) return st;
  if (out == gate_up) return set_error(LORA_INVALID_ARGUMENT, "%s starts at gate_up", oname);
  if (outq && (outq->values == gate_up || outq->values == out))
    return set_error(LORA_INVALID_ARGUMENT, "%s starts at gate_up or at %s", qname, oname);
  return LORA_OK;
}

extern "C" int lora_swiglu(const void* gate_up, int64_t ld, int32_t num_tokens, int32_t width, void* h, int64_t ldh,
                           const lora_q8_t* hq, void* stream) {
  clear_error();
  int st = gate_checks(gate_up, ld, num_tokens, width, h, ldh, hq, width, "h", "hq");
  if (st || num_tokens == 0) return st;
  GateArgs a{};
  a.gate_up = static_cast<const uint16_t*>(gate_up); a.ld = ld;
  a.out = static_cast<uint16_t*>(h); a.ldo = ldh;
  if (hq) { a.values = hq->values; a.ldq = hq->ld; a.exps = hq->exps; a.ld_exps = hq->ld_exps; }
  a.width = width;
  a.cpr = hq ? (uint32_t)q8_blocks(width) * 16 : (uint32_t)width / 8;
  a.chunks = (int64_t)num_tokens * a.cpr;
  if (too_many(a.chunks)) return set_error(LORA_UNSUPPORTED, "%d tokens of width %d are too many for one call", num_tokens, width);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool m = many(a.chunks);
  const dim3 grid((unsigned)groups(a.chunks, m ? 2 : 1)), blk(kRowThreads);
  if (h && hq) {
    if (m) hipLaunchKernelGGL((swiglu_kernel<2, true, true>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((swiglu_kernel<1, true, true>), grid, blk, 0, s, a);
  } else if (hq) {
    if (m) hipLaunchKernelGGL((swiglu_kernel<2, false, true>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((swiglu_kernel<1, false, true>), grid, blk, 0, s, a);
  } else {
    if (m) hipLaunchKernelGGL((swiglu_kernel<2, true, false>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((swiglu_kernel<1, true, false>), grid, blk, 0, s, a);
  }
  return launched("swiglu");
}

extern "C" int lora_swiglu_backward(const void* gate_up, int64_t ld, const void* dh, int64_t lddh, int32_t num_tokens,
                                    int32_t width, void* dgate_up, int64_t lddg, const lora_q8_t* dgate_up_q, void* stream) {
  clear_error();
  int st = gate_checks(gate_up, ld, num_tokens, width, dgate_up, lddg, dgate_up_q, 2 * (int64_t)width, "dgate_up", "dgate_up_q");
  if (st || num_tokens == 0) return st;
  if ((st = check_bf16_rows(dh, lddh, width, "dh"))) return st;
  if (dgate_up == dh || (dgate_up_q && dgate_up_q->values == dh))
    return set_error(LORA_INVALID_ARGUMENT, "an output starts at dh");
  GateArgs a{};
  a.gate_up = static_cast<const uint16_t*>(gate_up); a.ld = ld;
  a.dh = static_cast<const uint16_t*>(dh); a.lddh = lddh;
  a.out = static_cast<uint16_t*>(dgate_up); a.ldo = lddg;
  const lora_q8_t* q = dgate_up_q;
  if (q) { a.values = q->values; a.ldq = q->ld; a.exps = q->exps; a.ld_exps = q->ld_exps; }
  a.width = width;
  const bool split = q && (width % kQ8Block);
  a.cpr = split ? (uint32_t)q8_blocks(2 * (int64_t)width) * 16 : (uint32_t)width / 8;
  a.chunks = (int64_t)num_tokens * a.cpr;
  if (groups(a.chunks, 1) > kMaxGroups) return set_error(LORA_UNSUPPORTED, "%d tokens of width %d are too many for one call", num_tokens, width);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)groups(a.chunks, 1)), blk(kRowThreads);
  const bool m = many(a.chunks);
  if (split) {
    if (dgate_up) hipLaunchKernelGGL(swiglu_backward_split_kernel<true>, grid, blk, 0, s, a);
    else hipLaunchKernelGGL(swiglu_backward_split_kernel<false>, grid, blk, 0, s, a);
  } else if (q && dgate_up) {
    if (m) hipLaunchKernelGGL((swiglu_backward_kernel<true, true, true>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((swiglu_backward_kernel<false, true, true>), grid, blk, 0, s, a);
  } else if (q) {
    if (m) hipLaunchKernelGGL((swiglu_backward_kernel<true, false, true>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((swiglu_backward_kernel<false, false, true>), grid, blk, 0, s, a);
  } else {
    if (m) hipLaunchKernelGGL((swiglu_backward_kernel<true, true, false>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((swiglu_backward_kernel<false, true, false>), grid, blk, 0, s, a);
  }
  return launched("swiglu_backward");
}
