// lora_q4.hip -- rows and weights stored in 4 bits (e2m1 with one power-of-two
// scale per 32 columns, in panels of 128 columns) and their restore.
//
// One pass over the data each: the floor is the bytes. A chunk is 8 columns of
// one row (16 bytes of bf16, 4 of e2m1); the 4 lanes of a quad hold one scale's
// 32 columns, 16 lanes one row of a panel, so the largest magnitude of a block
// is two DPP steps and a panel row's 64 bytes leave as one access.
#include <hip/hip_runtime.h>

#include "lora_internal.h"
#include "lora_q4.h"
#include "lora_q8.h"

namespace lora {
namespace {

constexpr int kThreads = 256;

// A workgroup takes 4 panels of 4 kRows rows: each wave reads 1 KB runs of one row
// and writes neighbouring rows of the panels, which follow each other.
constexpr int kRows = 2;  // of a wave, loaded together (one, four, eight: 5, 2, 9% slower to store 32768 x 4096)
struct Q4Args {
  const uint16_t* x;  // quantise: source; restore: target (cast)
  int64_t ldx;
  uint8_t* values;
  int64_t ld;
  uint8_t* exps;
  int64_t ld_exps;
  int32_t rows, width;
  int32_t panels;
  int32_t tiles_p;  // groups of 4 panels
};

struct Place {
  int row0, panel, chunk;
};
__device__ __forceinline__ Place place_of(const Q4Args& a) {
  const int tr = blockIdx.x / a.tiles_p, tp = blockIdx.x - tr * a.tiles_p;
  return Place{(tr * 4 + (int)(threadIdx.x >> 6)) * kRows, tp * 4 + ((int)(threadIdx.x >> 4) & 3), (int)threadIdx.x & 15};
}

// us (TB/s), x past the caches (NT) where it is too large for them: 256 x 2560 2.3, 2560 x
// 2560 4.4, 8192 x 4096 14.1 (6.0; 16.3 with NT: x was in the Infinity Cache), 19456
// x 2560 23.6 (5.4; 24.8 without), 32768 x 4096 55 (6.1; 58).
template <bool NT>
__global__ __launch_bounds__(kThreads) void q4_rows_kernel(Q4Args a) {
  constexpr int U = kRows;
  const Place p = place_of(a);
  const int col = p.panel * kQ4Panel + 8 * p.chunk;
  u32x4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    v[u] = zero16();
    if (p.row0 + u < a.rows && col < a.width) {
      const uint16_t* src = a.x + (int64_t)(p.row0 + u) * a.ldx + col;
      if constexpr (NT) v[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src));
      else v[u] = ld16(src);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t e = q4_exponent(max_over_4(abs_bits8(v[u])));
    float f[8];
    unpack8(v[u], f);
    const uint32_t q = e == kQ4NoNumber ? 0u : pack_e2m1(f, q4_inverse(e));
    const uint32_t es = gather_exps(e);
    const int64_t row = p.row0 + u;
    if (row < a.rows && p.panel < a.panels) {
      *reinterpret_cast<uint32_t*>(a.values + p.panel * a.ld + row * kQ4RowBytes + 4 * p.chunk) = q;
      if (p.chunk == 0) *reinterpret_cast<uint32_t*>(a.exps + p.panel * a.ld_exps + row * 4) = es;
    }
  }
}

// us (TB/s), the restored rows past the caches (NT) in all but small matrices: 256 x 2560
// 2.5, 2048 x 4096 3.8 (5.7; 5.0 without NT), 19456 x 2560 19.7 (6.4; 26), 32768 x 4096
// 48 (7.0; 62).
template <bool NT>
__global__ __launch_bounds__(kThreads) void q4_restore_kernel(Q4Args a) {
  constexpr int U = kRows;
  const Place p = place_of(a);
  const int col = p.panel * kQ4Panel + 8 * p.chunk;
  if (col >= a.width) return;
  uint32_t q[U], e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = p.row0 + u;
    q[u] = e[u] = 0;
    if (row < a.rows) {
      q[u] = *reinterpret_cast<const uint32_t*>(a.values + p.panel * a.ld + row * kQ4RowBytes + 4 * p.chunk);
      e[u] = a.exps[p.panel * a.ld_exps + row * 4 + (p.chunk >> 2)];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (p.row0 + u >= a.rows) return;
    u32x4* dst = reinterpret_cast<u32x4*>(const_cast<uint16_t*>(a.x) + (int64_t)(p.row0 + u) * a.ldx + col);
    const u32x4 r = restore_e2m1(q[u], e[u]);
    if constexpr (NT) __builtin_nontemporal_store(r, dst);
    else *dst = r;
  }
}

// Weights in both orientations: one workgroup per 128 x 128 block (a panel of
// each store), the scale shared by 32 x 32 values so that both hold the same
// numbers. us (TB/s): 2560 x 2560 7.4, 19456 x 2560 32.5 (4.7), 32768 x 4096 79 (5.2).
struct Q4PairArgs {
  Q4Args a;
  uint8_t* values_t;
  int64_t ld_t;
  uint8_t* exps_t;
  int64_t ld_exps_t;
};

__global__ __launch_bounds__(kThreads) void q4_pair_kernel(Q4PairArgs b) {
  const Q4Args& a = b.a;
  __shared__ uint32_t top[4][4][4];  // [row block][column block][wave]
  __shared__ alignas(16) uint32_t tile[128][16 + 1];  // a chunk's 8 codes each
  const int rb = blockIdx.x / a.panels, cb = blockIdx.x - rb * a.panels;
  const int chunk = threadIdx.x & 15, r0 = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int col = cb * kQ4Panel + 8 * chunk;
  u32x4 v[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = rb * 128 + r0 + 16 * p;
    v[p] = zero16();
    if (r < a.rows && col < a.width) v[p] = ld16(a.x + (int64_t)r * a.ldx + col);
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {  // rows 32 g .. are passes 2 g and 2 g + 1
    uint32_t m = max_over_4(max(abs_bits8(v[2 * g]), abs_bits8(v[2 * g + 1])));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((threadIdx.x & 51) == 0) top[g][chunk >> 2][wave] = m;  // lanes 0, 4, 8, 12
  }
  __syncthreads();
  uint32_t e[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t* t = top[g][chunk >> 2];
    e[g] = q4_exponent(max(max(t[0], t[1]), max(t[2], t[3])));
  }
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    float f[8];
    unpack8(v[p], f);
    const uint32_t ex = e[p >> 1];
    const uint32_t q = ex == kQ4NoNumber ? 0u : pack_e2m1(f, q4_inverse(ex));
    const int lr = r0 + 16 * p;
    const int64_t r = rb * 128 + lr;
    const uint32_t es = gather_exps(ex);
    tile[lr][chunk] = q;
    if (r < a.rows) {
      *reinterpret_cast<uint32_t*>(a.values + cb * a.ld + r * kQ4RowBytes + 4 * chunk) = q;
      if (chunk == 0) *reinterpret_cast<uint32_t*>(a.exps + cb * a.ld_exps + r * 4) = es;
    }
  }
  __syncthreads();
  // Row c of the transposed panel rb: its dword i holds rows 8 i .. 8 i + 7 of
  // column c. A thread turns an 8 x 8 block of codes (one dword of each of 8
  // rows), so that it reads 8 dwords and writes 8.
  const int i = threadIdx.x & 15, c8 = threadIdx.x >> 4;
  uint32_t w[8], o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = tile[8 * i + k][c8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    o[j] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[j] |= ((w[k] >> (4 * j)) & 15u) << (4 * k);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t c = cb * 128 + 8 * c8 + j;
    if (c < a.width) *reinterpret_cast<uint32_t*>(b.values_t + rb * b.ld_t + c * kQ4RowBytes + 4 * i) = o[j];
  }
  if (threadIdx.x < 128) {
    const int64_t c = cb * 128 + (int)threadIdx.x;
    uint32_t es = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t* t = top[g][threadIdx.x >> 5];
      es |= q4_exponent(max(max(t[0], t[1]), max(t[2], t[3]))) << (8 * g);
    }
    if (c < a.width) *reinterpret_cast<uint32_t*>(b.exps_t + rb * b.ld_exps_t + c * 4) = es;
  }
}

// Matrices whose bf16 rows pass the caches: read from 80 MB on, written from 8 MB on (the
// times are at the kernels).
constexpr int64_t kStreamRead = (int64_t)40 << 20, kStreamWrite = (int64_t)4 << 20;  // values
bool at_least(const lora_q4_t* q, int64_t values) { return (int64_t)q->rows * q->width >= values; }

// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxGroups = 0xffffffffll / kThreads;

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(LORA_DEVICE_ERROR, "%s launch failed: %s", what, hipGetErrorString(e));
  return LORA_OK;
}

Q4Args args_of(const void* x, int64_t ldx, const lora_q4_t* q) {
  Q4Args a{};
  a.x = static_cast<const uint16_t*>(x); a.ldx = ldx;
  a.values = q->values; a.ld = q->ld; a.exps = q->exps; a.ld_exps = q->ld_exps;
  a.rows = q->rows; a.width = q->width;
  a.panels = (int32_t)q4_panels(q->width);
  a.tiles_p = (a.panels + 3) / 4;
  return a;
}
int64_t tiles(const Q4Args& a) { return ((int64_t)a.rows + 4 * kRows - 1) / (4 * kRows) * a.tiles_p; }

}  // namespace

int check_q4(const lora_q4_t* q, const char* name) {
  if (!q) return set_error(LORA_INVALID_ARGUMENT, "%s is NULL", name);
  if (q->rows < 0 || q->width <= 0 || (q->width & 7))
    return set_error(LORA_INVALID_ARGUMENT, "%s: rows (%d) must be >= 0 and width (%d) a positive multiple of 8", name,
                     q->rows, q->width);
  if (q->rows > kQ4Most || q->width > kQ4Most)
    return set_error(LORA_UNSUPPORTED, "%s: %d x %d is larger than %d in one direction", name, q->rows, q->width, kQ4Most);
  if (q->rows == 0) return LORA_OK;
  if (q->ld < (int64_t)q->rows * kQ4RowBytes || (q->ld & 15))
    return set_error(LORA_INVALID_ARGUMENT, "%s: panel stride %lld must be a multiple of 16 and hold %d rows of 64 bytes", name,
                     (long long)q->ld, q->rows);
  if (q->ld_exps < (int64_t)q->rows * 4 || (q->ld_exps & 3))
    return set_error(LORA_INVALID_ARGUMENT, "%s: exponent panel stride %lld must be a multiple of 4 and hold %d rows of 4 bytes",
                     name, (long long)q->ld_exps, q->rows);
  if (!q->values || !q->exps) return set_error(LORA_INVALID_ARGUMENT, "%s: values/exps is NULL", name);
  if ((reinterpret_cast<uintptr_t>(q->values) & 15u) || (reinterpret_cast<uintptr_t>(q->exps) & 3u))
    return set_error(LORA_INVALID_ARGUMENT, "%s: values must be 16-byte and exps 4-byte aligned", name);
  return LORA_OK;
}

}  // namespace lora

using namespace lora;

extern "C" int lora_q4_quantize(const void* x, int64_t ldx, const lora_q4_t* out, const lora_q4_t* out_t, void* stream) {
  clear_error();
  int st = check_q4(out, "out");
  if (st) return st;
  if (out_t) {
    if ((st = check_q4(out_t, "out_t"))) return st;
    if (out_t->rows != out->width || out_t->width != out->rows)
      return set_error(LORA_INVALID_ARGUMENT, "out_t is %d x %d, the transpose of out is %d x %d", out_t->rows, out_t->width,
                       out->width, out->rows);
  }
  if (out->rows == 0) return LORA_OK;
  if ((st = check_bf16_rows(x, ldx, out->width, "x"))) return st;
  if (x == out->values || (out_t && (x == out_t->values || out->values == out_t->values)))
    return set_error(LORA_INVALID_ARGUMENT, "a store starts at x or at the other store");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Q4Args a = args_of(x, ldx, out);
  if (out_t) {
    Q4PairArgs b{};
    b.a = a;
    b.values_t = out_t->values; b.ld_t = out_t->ld; b.exps_t = out_t->exps; b.ld_exps_t = out_t->ld_exps;
    const int64_t n = q4_panels(out->rows) * a.panels;
    if (n > kMaxGroups) return set_error(LORA_UNSUPPORTED, "x of %d x %d is too large for one call", out->rows, out->width);
    hipLaunchKernelGGL(q4_pair_kernel, dim3((unsigned)n), dim3(kThreads), 0, s, b);
    return launched("q4_pair");
  }
  const int64_t n = tiles(a);
  if (n > kMaxGroups) return set_error(LORA_UNSUPPORTED, "x of %d x %d is too large for one call", out->rows, out->width);
  if (at_least(out, kStreamRead)) hipLaunchKernelGGL(q4_rows_kernel<true>, dim3((unsigned)n), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(q4_rows_kernel<false>, dim3((unsigned)n), dim3(kThreads), 0, s, a);
  return launched("q4_rows");
}

extern "C" int lora_q4_dequantize(const lora_q4_t* q, void* x, int64_t ldx, void* stream) {
  clear_error();
  int st = check_q4(q, "q");
  if (st) return st;
  if (q->rows == 0) return LORA_OK;
  if ((st = check_bf16_rows(x, ldx, q->width, "x"))) return st;
  if (x == q->values) return set_error(LORA_INVALID_ARGUMENT, "x starts at the store");
  const Q4Args a = args_of(x, ldx, q);
  const int64_t n = tiles(a);
  if (n > kMaxGroups) return set_error(LORA_UNSUPPORTED, "q of %d x %d is too large for one call", q->rows, q->width);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (at_least(q, kStreamWrite)) hipLaunchKernelGGL(q4_restore_kernel<true>, dim3((unsigned)n), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(q4_restore_kernel<false>, dim3((unsigned)n), dim3(kThreads), 0, s, a);
  return launched("q4_restore");
}
