// lora_qk.hip -- the root-mean-square norm of every query and key head and the
// rotation by its token's position, in one pass over the rows that the q and k
// projections leave, and its gradient.
//
// Per head x of a token at position p, with weight w:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w,
//   (out_i, out_j) = (n_i cos a - n_j sin a, n_j cos a + n_i sin a),  a = p f_i
// over the pairs (i, j) of the first rot_dim columns. Back, with m the gradient
// turned the other way and g = m w:
//   dw += m x r,   dx = r (g - x r mean(g x r)).
//
// One pass over the data: the floor is the bytes. 8 columns of a head are one
// lane's 16 bytes and a head is 4 to 32 neighbouring lanes, so a wave holds 2
// to 16 heads of one token; the sums over a head stay in registers.
#include <hip/hip_runtime.h>

#include <math.h>

#include "lora_internal.h"
#include "lora_q8.h"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct QKArgs {
  const uint16_t *q, *k;
  int64_t ldq, ldk;
  const uint16_t *gq, *gk;  // backward: the outputs' gradients
  int64_t ldgq, ldgk;
  uint16_t *oq, *ok;        // outputs, or the inputs' gradients
  int64_t ldoq, ldok;
  const uint16_t *wq, *wk;
  const double* freqs;
  const int32_t* positions;
  float* parts;             // backward: the workgroups' shares of dweight, or null
  int32_t tokens, heads_q, heads, dim, rot;
  int32_t per_token;        // items of one token
  float eps;
};

// Sum over the L lanes of a head, in each of them.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ float sum_over(float v) {
  v = dpp_add<0xB1>(v);                              // quad_perm 1,0,3,2
  v = dpp_add<0x4E>(v);                              // quad_perm 2,3,0,1
  if constexpr (L >= 8) v = dpp_add<0x141>(v);       // row_half_mirror
  if constexpr (L >= 16) v = dpp_add<0x140>(v);      // row_mirror
  if constexpr (L >= 32) v += __shfl_xor(v, 16);
  return v;
}

// What a lane needs of its token's rotation. The angle is taken in 64 bits and
// reduced to part of a turn before it is rounded: position 131071 times a
// frequency near 1 has no bits of the turn left in 32.
template <bool NB>
struct Turn {
  static constexpr int N = NB ? 4 : 8;  // a lane's pairs
  float c[N], s[N];
  __device__ __forceinline__ void set(const QKArgs& a, int position, int chunk) {
    const int half = a.rot >> 1;
    const bool in = 8 * chunk < a.rot;
    const int first = NB ? 4 * chunk : (8 * chunk < half ? 8 * chunk : 8 * chunk - half);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
      if (in) {
        const double t = (double)position * (a.freqs[first + i] * 0.15915494309189533577);
        const float half_turns = (float)(2. * (t - __builtin_rint(t)));
        sincospif(half_turns, &s[i], &c[i]);
      }
    }
  }
};

// The rotation of a lane's 8 columns (BACK: the other way). halves: `other` is the
// pair's other member, from the lane that holds it; `upper` lanes hold the
// second members.
template <bool NB, bool BACK>
__device__ __forceinline__ void turn8(float (&v)[8], const float (&other)[8], const Turn<NB>& t, bool upper) {
  if constexpr (NB) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1], s = BACK ? -t.s[i] : t.s[i];
      v[2 * i] = x * t.c[i] - y * s;
      v[2 * i + 1] = y * t.c[i] + x * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = (upper != BACK) ? t.s[i] : -t.s[i];
      v[i] = v[i] * t.c[i] + other[i] * s;
    }
  }
}

// 16 bytes from another lane of the wave.
__device__ __forceinline__ u32x4 from_lane(u32x4 v, int lane) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * lane, (int)v[i]);
  return o;
}

// A lane's place: its chunk of the head, the lane that holds the other members of its
// pairs, and its share of the wave's items.
template <int L, bool NB>
struct Lane {
  int chunk, head0, other;
  bool in, upper;
  __device__ __forceinline__ explicit Lane(const QKArgs& a) {
    const int lane = threadIdx.x & 63;
    chunk = lane & (L - 1);
    head0 = lane / L;
    in = 8 * chunk < a.dim;
    const int h = a.rot >> 4;  // chunks of half the turned columns
    upper = chunk >= h;
    other = NB || 8 * chunk >= a.rot ? lane : upper ? lane - h : lane + h;
  }
};

// sum(x^2) past fp32's range: x is taken 2^-80 as large (its norm does not change).
__device__ __forceinline__ bool past_range(float ss) { return !(ss < __builtin_inff()); }
constexpr float kDown = 0x1p-80f;

// U groups of 64 / L heads of one token per wave, all loaded before the first is
// used.
template <int L, bool NB, int U>
__global__ __launch_bounds__(kThreads) void qk_forward_kernel(QKArgs a) {
  constexpr int H = 64 / L;  // heads a wave holds at once
  const int item = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int token = item / a.per_token, part = item - token * a.per_token;
  if (token >= a.tokens) return;
  const Lane<L, NB> me(a);
  u32x4 x[U];
  bool live[U], key[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int head = (part * U + u) * H + me.head0;
    key[u] = head >= a.heads_q;
    live[u] = me.in && head < a.heads;
    x[u] = zero16();
    if (live[u]) {
      const uint16_t* row = key[u] ? a.k + (int64_t)token * a.ldk + (int64_t)(head - a.heads_q) * a.dim
                                   : a.q + (int64_t)token * a.ldq + (int64_t)head * a.dim;
      x[u] = ld16(row + 8 * me.chunk);
    }
  }
  u32x4 wq = zero16(), wk = zero16();
  if (me.in && a.heads_q > 0) wq = ld16(a.wq + 8 * me.chunk);
  if (me.in && a.heads > a.heads_q) wk = ld16(a.wk + 8 * me.chunk);
  const u32x4 oq = from_lane(wq, me.other), ok = from_lane(wk, me.other);
  Turn<NB> t;
  t.set(a, a.positions[token], me.chunk);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float f[8], w[8], p[8], pw[8];
    unpack8(x[u], f);
    unpack8(key[u] ? wk : wq, w);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
    ss = sum_over<L>(ss);
    float down = 1.f;
    if (__any(past_range(ss))) {
      down = past_range(ss) ? kDown : 1.f;
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += (f[i] * down) * (f[i] * down);
      ss = sum_over<L>(ss);
    }
    const float r = down * __builtin_amdgcn_rsqf(ss / (float)a.dim + a.eps * down * down);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
    if constexpr (!NB) {
      unpack8(from_lane(x[u], me.other), p);
      unpack8(key[u] ? ok : oq, pw);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = me.other == (int)(threadIdx.x & 63) ? 0.f : p[i] * r * pw[i];
    }
    turn8<NB, false>(f, p, t, me.upper);
    if (live[u]) {
      const int head = (part * U + u) * H + me.head0;
      uint16_t* row = key[u] ? a.ok + (int64_t)token * a.ldok + (int64_t)(head - a.heads_q) * a.dim
                             : a.oq + (int64_t)token * a.ldoq + (int64_t)head * a.dim;
      st16(row + 8 * me.chunk, pack8(f));
    }
  }
}

// One group of 64 / L heads per item; the waves of the grid take the items in
// turn, so that a lane's share of dweight is summed over its items before it
// meets the others' (in a fixed order: lanes, waves, then workgroups).
template <int L, bool NB, bool DW>
__global__ __launch_bounds__(kThreads) void qk_backward_kernel(QKArgs a) {
  constexpr int H = 64 / L;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Lane<L, NB> me(a);
  u32x4 wq = zero16(), wk = zero16();
  if (me.in && a.heads_q > 0) wq = ld16(a.wq + 8 * me.chunk);
  if (me.in && a.heads > a.heads_q) wk = ld16(a.wk + 8 * me.chunk);
  float dwq[8], dwk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;
  for (int token = blockIdx.x * kWaves + wave; token < a.tokens; token += gridDim.x * kWaves) {
    Turn<NB> t;
    t.set(a, a.positions[token], me.chunk);
    for (int part = 0; part < a.per_token; ++part) {
      const int head = part * H + me.head0;
      const bool key = head >= a.heads_q, live = me.in && head < a.heads;
      const int kh = head - a.heads_q;
      u32x4 x = zero16(), g = zero16();
      if (live) {
        x = ld16((key ? a.k + (int64_t)token * a.ldk + (int64_t)kh * a.dim : a.q + (int64_t)token * a.ldq + (int64_t)head * a.dim) + 8 * me.chunk);
        g = ld16((key ? a.gk + (int64_t)token * a.ldgk + (int64_t)kh * a.dim : a.gq + (int64_t)token * a.ldgq + (int64_t)head * a.dim) + 8 * me.chunk);
      }
      float f[8], m[8], p[8], w[8];
      unpack8(x, f);
      unpack8(g, m);
      unpack8(key ? wk : wq, w);
      if constexpr (!NB) {
        unpack8(from_lane(g, me.other), p);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = me.other == (int)(threadIdx.x & 63) ? 0.f : p[i];
      }
      turn8<NB, true>(m, p, t, me.upper);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
      ss = sum_over<L>(ss);
      float down = 1.f;
      if (__any(past_range(ss))) {
        down = past_range(ss) ? kDown : 1.f;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= down, ss += f[i] * f[i];
        ss = sum_over<L>(ss);
      }
      const float r = __builtin_amdgcn_rsqf(ss / (float)a.dim + a.eps * down * down);
      float along = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] *= r;  // x / rms
        if constexpr (DW) {
          dwq[i] += key ? 0.f : m[i] * f[i];
          dwk[i] += key ? m[i] * f[i] : 0.f;
        }
        m[i] *= w[i];
        along += m[i] * f[i];
      }
      along = sum_over<L>(along) / (float)a.dim;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = (m[i] - f[i] * along) * r * down;
      if (live)
        st16((key ? a.ok + (int64_t)token * a.ldok + (int64_t)kh * a.dim : a.oq + (int64_t)token * a.ldoq + (int64_t)head * a.dim) + 8 * me.chunk,
             pack8(m));
    }
  }
  if constexpr (DW) {
    __shared__ float sum[kWaves][2][8 * L];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int d = L; d < 64; d *= 2) {
        dwq[i] += __shfl_xor(dwq[i], d);
        dwk[i] += __shfl_xor(dwk[i], d);
      }
      if (me.head0 == 0) {
        sum[wave][0][8 * me.chunk + i] = dwq[i];
        sum[wave][1][8 * me.chunk + i] = dwk[i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.dim; c += kThreads) {
      const int which = c >= a.dim, col = c - which * a.dim;
      a.parts[(int64_t)blockIdx.x * 2 * a.dim + c] =
          (sum[0][which][col] + sum[1][which][col]) + (sum[2][which][col] + sum[3][which][col]);
    }
  }
}

// dweight = the workgroups' shares, 16 columns a workgroup: 16 threads take every
// sixteenth share of a column, and their sums are added in order.
__global__ __launch_bounds__(256) void qk_weight_kernel(const float* parts, int32_t n, int32_t cols, float* out, int32_t accumulate) {
  __shared__ float sum[16][16 + 1];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float s = 0.f;
  if (col < cols)
    for (int i = r; i < n; i += 16) s += parts[(int64_t)i * cols + col];
  sum[r][c] = s;
  __syncthreads();
  if (r == 0 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sum[i][c];
    out[col] = accumulate ? out[col] + s : s;
  }
}

constexpr int kBackwardGroups = 1024;
constexpr int32_t kMostTokens = 0x7fff0000;  // a token's number and one grid more stay below 2^31
int backward_groups(int32_t tokens) { return (int)min((int64_t)kBackwardGroups, ((int64_t)tokens + kWaves - 1) / kWaves); }

int lanes_of(int32_t dim) { return dim <= 32 ? 4 : dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// Calls f(lanes, neighbours) with both as compile-time constants.
template <class F>
void with_form(const lora_qk_heads_t& h, F f) {
  auto lanes = [&](auto nb) {
    switch (lanes_of(h.head_dim)) {
      case 4: f(std::integral_constant<int, 4>{}, nb); break;
      case 8: f(std::integral_constant<int, 8>{}, nb); break;
      case 16: f(std::integral_constant<int, 16>{}, nb); break;
      default: f(std::integral_constant<int, 32>{}, nb); break;
    }
  };
  if (h.neighbours) lanes(std::true_type{});
  else lanes(std::false_type{});
}

int check_heads(const lora_qk_heads_t* h) {
  if (!h) return set_error(LORA_INVALID_ARGUMENT, "heads is NULL");
  if (h->heads_q < 0 || h->heads_k < 0 || (h->heads_q == 0 && h->heads_k == 0))
    return set_error(LORA_INVALID_ARGUMENT, "heads_q (%d) and heads_k (%d) must be >= 0 and not both 0", h->heads_q, h->heads_k);
  if (h->heads_q > 65536 || h->heads_k > 65536)
    return set_error(LORA_UNSUPPORTED, "more than 65536 heads (%d, %d) are not supported", h->heads_q, h->heads_k);
  if (h->head_dim <= 0 || (h->head_dim & 7))
    return set_error(LORA_INVALID_ARGUMENT, "head_dim (%d) must be a positive multiple of 8", h->head_dim);
  if (h->head_dim > 256) return set_error(LORA_UNSUPPORTED, "head_dim %d is above 256", h->head_dim);
  if (h->rot_dim < 0 || h->rot_dim > h->head_dim || (h->rot_dim & 15))
    return set_error(LORA_INVALID_ARGUMENT, "rot_dim (%d) must be a multiple of 16 from 0 to head_dim (%d)", h->rot_dim, h->head_dim);
  if (!(h->eps >= 1.17549435e-38f) || !(h->eps <= 3.4e38f))
    return set_error(LORA_INVALID_ARGUMENT, "eps (%g) must be a positive normal number", (double)h->eps);
  if ((h->heads_q && !h->weight_q) || (h->heads_k && !h->weight_k))
    return set_error(LORA_INVALID_ARGUMENT, "the weight of heads that there are is NULL");
  if ((reinterpret_cast<uintptr_t>(h->weight_q) | reinterpret_cast<uintptr_t>(h->weight_k)) & 15u)
    return set_error(LORA_INVALID_ARGUMENT, "a weight is not 16-byte aligned");
  if (h->rot_dim && (!h->freqs || (reinterpret_cast<uintptr_t>(h->freqs) & 7u)))
    return set_error(LORA_INVALID_ARGUMENT, "freqs is NULL or not 8-byte aligned");
  return LORA_OK;
}

// The rows of both kinds of heads of one argument pair.
int check_rows(const lora_qk_heads_t* h, const void* q, int64_t ldq, const void* k, int64_t ldk, const char* qn, const char* kn) {
  int st = LORA_OK;
  if (h->heads_q) st = check_bf16_rows(q, ldq, (int64_t)h->heads_q * h->head_dim, qn);
  if (!st && h->heads_k) st = check_bf16_rows(k, ldk, (int64_t)h->heads_k * h->head_dim, kn);
  return st;
}

int check_call(const lora_qk_heads_t* h, const int32_t* positions, int32_t tokens) {
  const int st = check_heads(h);
  if (st) return st;
  if (tokens < 0) return set_error(LORA_INVALID_ARGUMENT, "num_tokens (%d) must be >= 0", tokens);
  if (tokens > kMostTokens) return set_error(LORA_UNSUPPORTED, "num_tokens %d is above %d", tokens, kMostTokens);
  if (tokens && (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u)))
    return set_error(LORA_INVALID_ARGUMENT, "positions is NULL or not 4-byte aligned");
  return LORA_OK;
}

QKArgs args_of(const lora_qk_heads_t* h, const void* q, int64_t ldq, const void* k, int64_t ldk, const int32_t* positions,
               int32_t tokens, void* oq, int64_t ldoq, void* ok, int64_t ldok) {
  QKArgs a{};
  a.q = static_cast<const uint16_t*>(q); a.ldq = ldq;
  a.k = static_cast<const uint16_t*>(k); a.ldk = ldk;
  a.oq = static_cast<uint16_t*>(oq); a.ldoq = ldoq;
  a.ok = static_cast<uint16_t*>(ok); a.ldok = ldok;
  a.wq = static_cast<const uint16_t*>(h->weight_q);
  a.wk = static_cast<const uint16_t*>(h->weight_k);
  a.freqs = h->freqs;
  a.positions = positions;
  a.tokens = tokens;
  a.heads_q = h->heads_q; a.heads = h->heads_q + h->heads_k;
  a.dim = h->head_dim; a.rot = h->rot_dim;
  a.eps = h->eps;
  return a;
}

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(LORA_DEVICE_ERROR, "%s launch failed: %s", what, hipGetErrorString(e));
  return LORA_OK;
}

// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxGroups = 0xffffffffll / kThreads;

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_qk_norm_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, const lora_qk_heads_t* heads,
                                 const int32_t* positions, int32_t num_tokens, void* q_out, int64_t ldqo, void* k_out,
                                 int64_t ldko, void* stream) {
  clear_error();
  int st = check_call(heads, positions, num_tokens);
  if (st || num_tokens == 0) return st;
  if ((st = check_rows(heads, q, ldq, k, ldk, "q", "k"))) return st;
  if ((st = check_rows(heads, q_out, ldqo, k_out, ldko, "q_out", "k_out"))) return st;
  const bool both = heads->heads_q && heads->heads_k;
  if (both && (q_out == k_out || q_out == k || k_out == q))
    return set_error(LORA_INVALID_ARGUMENT, "an output starts at the other output or at the other input");
  if ((heads->heads_q && q_out == q && ldqo != ldq) || (heads->heads_k && k_out == k && ldko != ldk))
    return set_error(LORA_INVALID_ARGUMENT, "an output that takes its input's place needs its row stride");
  QKArgs a = args_of(heads, q, ldq, k, ldk, positions, num_tokens, q_out, ldqo, k_out, ldko);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int per = 64 / lanes_of(a.dim), groups = (a.heads + per - 1) / per;
  const int u = (int64_t)num_tokens * groups >= 16384 ? 4 : 1;
  a.per_token = (groups + u - 1) / u;
  const int64_t n = ((int64_t)num_tokens * a.per_token + kWaves - 1) / kWaves;
  if (n > kMaxGroups) return set_error(LORA_UNSUPPORTED, "%d tokens of %d heads are too many for one call", num_tokens, a.heads);
  with_form(*heads, [&](auto lanes, auto nb) {
    const dim3 grid((unsigned)n), blk(kThreads);
    if (u == 4) hipLaunchKernelGGL((qk_forward_kernel<lanes(), nb(), 4>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((qk_forward_kernel<lanes(), nb(), 1>), grid, blk, 0, s, a);
  });
  return launched("qk_norm_rope");
}

extern "C" int lora_workspace_size_qk(const lora_qk_heads_t* heads, int32_t num_tokens, size_t* bytes) {
  clear_error();
  const int st = check_heads(heads);
  if (st) return st;
  if (!bytes || num_tokens < 0) return set_error(LORA_INVALID_ARGUMENT, "bytes is NULL or num_tokens (%d) below 0", num_tokens);
  *bytes = (size_t)backward_groups(num_tokens) * 2 * (size_t)heads->head_dim * sizeof(float);
  return LORA_OK;
}

extern "C" int lora_qk_norm_rope_backward(const void* q, int64_t ldq, const void* k, int64_t ldk, const lora_qk_heads_t* heads,
                                          const int32_t* positions, int32_t num_tokens, const void* dq_out, int64_t lddqo,
                                          const void* dk_out, int64_t lddko, void* dq, int64_t lddq, void* dk, int64_t lddk,
                                          float* dweight, uint32_t flags, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  int st = check_call(heads, positions, num_tokens);
  if (st) return st;
  if (flags & ~LORA_GRAD_ACCUMULATE) return set_error(LORA_INVALID_ARGUMENT, "unknown flags 0x%x", flags);
  if (dweight && (reinterpret_cast<uintptr_t>(dweight) & 3u)) return set_error(LORA_INVALID_ARGUMENT, "dweight is not 4-byte aligned");
  if (num_tokens) {
    if ((st = check_rows(heads, q, ldq, k, ldk, "q", "k"))) return st;
    if ((st = check_rows(heads, dq_out, lddqo, dk_out, lddko, "dq_out", "dk_out"))) return st;
    if ((st = check_rows(heads, dq, lddq, dk, lddk, "dq", "dk"))) return st;
    if ((heads->heads_q && (dq == q || dq == dq_out)) || (heads->heads_k && (dk == k || dk == dk_out)) ||
        (heads->heads_q && heads->heads_k && (dq == dk || dq == k || dq == dk_out || dk == q || dk == dq_out)))
      return set_error(LORA_INVALID_ARGUMENT, "a gradient starts at an input or at the other gradient");
    if (dweight) {
      const size_t need = (size_t)backward_groups(num_tokens) * 2 * (size_t)heads->head_dim * sizeof(float);
      if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15u)) return set_error(LORA_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
      if (ws_bytes < need)
        return set_error(LORA_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, %zu are needed", ws_bytes, need);
    }
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int cols = 2 * heads->head_dim;
  const int groups = backward_groups(num_tokens);
  if (num_tokens) {
    QKArgs a = args_of(heads, q, ldq, k, ldk, positions, num_tokens, dq, lddq, dk, lddk);
    a.gq = static_cast<const uint16_t*>(dq_out); a.ldgq = lddqo;
    a.gk = static_cast<const uint16_t*>(dk_out); a.ldgk = lddko;
    a.parts = static_cast<float*>(ws);
    const int per = 64 / lanes_of(a.dim);
    a.per_token = (a.heads + per - 1) / per;
    with_form(*heads, [&](auto lanes, auto nb) {
      const dim3 grid((unsigned)groups), blk(kThreads);
      if (dweight) hipLaunchKernelGGL((qk_backward_kernel<lanes(), nb(), true>), grid, blk, 0, s, a);
      else hipLaunchKernelGGL((qk_backward_kernel<lanes(), nb(), false>), grid, blk, 0, s, a);
    });
    if ((st = launched("qk_norm_rope_backward"))) return st;
  }
  if (dweight) {
    hipLaunchKernelGGL(qk_weight_kernel, dim3((unsigned)((cols + 15) / 16)), dim3(256), 0, s, static_cast<const float*>(ws),
                       groups, cols, dweight, (flags & LORA_GRAD_ACCUMULATE) ? 1 : 0);
    return launched("qk_weight");
  }
  return LORA_OK;
}
