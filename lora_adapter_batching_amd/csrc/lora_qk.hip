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
// lane's 16 bytes and a head is 4 to 32 neighbouring lanes, so a wave holds a
// group of 2 to 16 heads of one token; the sums over a head stay in registers. The
// cosines and sines of a token are the same for all its heads: a workgroup
// makes them once, one pair a thread, and its waves read them from LDS.
#include <hip/hip_runtime.h>

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "lora_internal.h"
#include "lora_q8.h"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct QKArgs {
  const uint16_t* x[2];     // rows of the queries and of the keys
  int64_t ldx[2];
  const uint16_t* g[2];     // backward: the outputs' gradients
  int64_t ldg[2];
  uint16_t* o[2];           // outputs, or the inputs' gradients
  int64_t ldo[2];
  const uint16_t* w[2];
  const double* freqs;
  const int32_t* positions;
  float* parts;             // backward: the workgroups' shares of dweight, or null
  int32_t heads[2];
  int32_t tokens, dim, rot;
  float eps, mean;          // mean = 1 / dim
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

// cos and sin of the pairs of W tokens.
constexpr int kMostPairs = 128;
template <int W>
struct Turns {
  alignas(16) float c[W][kMostPairs], s[W][kMostPairs];
};
// Fills it for tokens token0 ..; the caller synchronises. The angle is taken in 64
// bits and reduced to part of a turn before it is rounded: position 131071 times
// a frequency near 1 has few bits of the turn left in 32.
template <int W>
__device__ __forceinline__ void make_turns(const QKArgs& a, int token0, Turns<W>& t) {
  const int half = a.rot >> 1;
  for (int i = threadIdx.x; i < W * half; i += kThreads) {
    const int k = i / half, pair = i - k * half;
    if (token0 + k < a.tokens) {
      const double turns = (double)a.positions[token0 + k] * (a.freqs[pair] * 0.15915494309189533577);
      const float half_turns = (float)(2. * (turns - __builtin_rint(turns)));
      sincospif(half_turns, &t.s[k][pair], &t.c[k][pair]);
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

// A lane's place in its group of heads: its chunk of 8 columns, its head, and the
// lane with the other members of its pairs (itself, where they are its own).
template <int L, bool NB>
struct Lane {
  int chunk, head, other;
  bool in, turned, upper, part;
  __device__ __forceinline__ explicit Lane(const QKArgs& a) {
    const int lane = threadIdx.x & 63;
    chunk = lane & (L - 1);
    head = lane / L;
    in = 8 * chunk < a.dim;
    turned = 8 * chunk < a.rot;
    part = a.rot < a.dim;
    const int h = a.rot >> 4;  // chunks of half the turned columns
    upper = chunk >= h;
    other = NB || !turned ? lane : upper ? lane - h : lane + h;
  }
  // The rotation of its columns: column e becomes c[e] times itself plus s[e] times
  // its pair's other member (-0 times it where there is none, which leaves any sum as it is).
  template <int W>
  __device__ __forceinline__ void turn(const QKArgs& a, const Turns<W>& t, int k, float (&c)[8], float (&s)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = -0.f;
    if (!turned) return;
    if constexpr (NB) {
      const f32x4 vc = *reinterpret_cast<const f32x4*>(&t.c[k][4 * chunk]), vs = *reinterpret_cast<const f32x4*>(&t.s[k][4 * chunk]);
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = vc[e >> 1], s[e] = e & 1 ? vs[e >> 1] : -vs[e >> 1];
    } else {
      const int first = 8 * chunk - (upper ? a.rot >> 1 : 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = t.c[k][first + e], s[e] = upper ? t.s[k][first + e] : -t.s[k][first + e];
    }
  }
  // The other members of its pairs; 0 for columns without one, whose neighbours may hold
  // anything (0 times an infinity or NaN is NaN).
  __device__ __forceinline__ void pairs(u32x4 v, const float (&f)[8], float (&p)[8]) const {
    if constexpr (NB) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = f[e ^ 1];
      if (part) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = turned ? p[e] : 0.f;
      }
    } else {
      u32x4 o = from_lane(v, other);
      if (part) o = turned ? o : zero16();
      unpack8(o, p);
    }
  }
};

// Rows that the launch touches once. NT 1: what it writes goes past the caches, NT 2:
// what it reads too.
template <int NT>
__device__ __forceinline__ u32x4 ld_row(const uint16_t* p) {
  if constexpr (NT >= 2) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  else return ld16(p);
}
template <int NT>
__device__ __forceinline__ void st_row(uint16_t* p, u32x4 v) {
  if constexpr (NT >= 1) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  else st16(p, v);
}

// sum(x^2) past fp32's range: x is taken 2^-80 as large (its norm does not change).
__device__ __forceinline__ bool past_range(float ss) { return !(ss < __builtin_inff()); }
constexpr float kDown = 0x1p-80f;
constexpr int kDownPlaces = -80;

// A workgroup takes W tokens: one for each wave (W = 4), or one whose groups of heads
// the waves take in turn. U groups are loaded before the first is used. Bound by
// memory in large batches; 32 + 8 heads of 128 columns, us (TB/s): 16384 tokens 63
// (5.3), 4096 15.0 (5.6), 1000 6.5, 64 4.2, which is one launch and its chain of
// loads. Angles made by every lane for itself and weights applied apart from the
// rotation took 82 for 16384 tokens: the vector unit was busy most of that. Four
// waves a SIMD (128 registers) instead of three: 4096 tokens 17.2 -> 15.0.
template <int L, bool NB, int W, int U, int NT>
__global__ __launch_bounds__(kThreads, 4) void qk_forward_kernel(QKArgs a) {
  constexpr int H = 64 / L, STEP = W > 1 ? 1 : kWaves;
  __shared__ Turns<W> turns;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k = W > 1 ? wave : 0, g0 = W > 1 ? 0 : wave;
  const int token = blockIdx.x * W + k;
  const bool there = token < a.tokens;
  const Lane<L, NB> me(a);
  auto load = [&](int kind, int g) {
    const int head = g * H + me.head;
    if (!there || !me.in || head >= a.heads[kind]) return zero16();
    return ld_row<NT>(a.x[kind] + (int64_t)token * a.ldx[kind] + (int64_t)head * a.dim + 8 * me.chunk);
  };
  u32x4 x[2][U], w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int u = 0; u < U; ++u) x[i][u] = load(i, g0 + STEP * u);
    w[i] = me.in && a.heads[i] ? ld16(a.w[i] + 8 * me.chunk) : zero16();
  }
  make_turns(a, blockIdx.x * W, turns);
  __syncthreads();
  if (!there) return;
  float c[8], s[8];
  me.turn(a, turns, k, c, s);
  auto heads_of = [&](auto kind_) {
    constexpr int kind = decltype(kind_)::value;
    // The weight goes into the rotation: column e of the output is
    // A[e] r x[e] + B[e] r x[its pair's other].
    float A[8], B[8];
    unpack8(w[kind], A);
    me.pairs(w[kind], A, B);
#pragma unroll
    for (int e = 0; e < 8; ++e) A[e] *= c[e], B[e] *= s[e];
    for (int g = g0; g * H < a.heads[kind]; g += STEP * U) {
      u32x4 next[U];
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = load(kind, g + STEP * (U + u));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[8], p[8];
        unpack8(x[kind][u], f);
        me.pairs(x[kind][u], f, p);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
        ss = sum_over<L>(ss);
        float down = 1.f;
        if (__any(past_range(ss))) {
          down = past_range(ss) ? kDown : 1.f;
          ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= down, p[e] *= down, ss += f[e] * f[e];
          ss = sum_over<L>(ss);
        }
        const float r = __builtin_amdgcn_rsqf(ss * a.mean + a.eps * down * down);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = r * f[e] * A[e] + r * p[e] * B[e];  // (x w alone can leave the range)
        const int head = (g + STEP * u) * H + me.head;
        if (me.in && head < a.heads[kind])
          st_row<NT>(a.o[kind] + (int64_t)token * a.ldo[kind] + (int64_t)head * a.dim + 8 * me.chunk, pack8(f));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) x[kind][u] = next[u];
    }
  };
  heads_of(std::integral_constant<int, 0>{});
  heads_of(std::integral_constant<int, 1>{});
}

// The largest magnitude of 8 bf16, as its bits.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t largest(u32x4 v) {
  u16x2 m = {0, 0};
#pragma unroll
  for (int q = 0; q < 4; ++q) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[q] & 0x7fff7fffu));
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

// The gradient multiplies gradients by weights by r, whose product can be in range where
// two of them are not. Weights are taken as they are while the largest is within
// kWeightWindow binary places of 1, gradients while a head's largest is within kGradWindow;
// otherwise in units of their own, the power of two of that largest, and the result gets
// the units' exponents with r's in one step. So a column of dx is right to its rounding, and to
// 2^-50 of what the head's largest gradient and largest weight give (2^-64 2^-32 is 2^53
// times the smallest fp32 number). The look at the gradients costs no time: 16384 tokens,
// 32 + 8 heads of 128, 98-100 us a pass with dweight, with it and without.
constexpr int kWeightWindow = 32, kGradWindow = 64;
template <int WINDOW>
__device__ __forceinline__ bool outside(uint32_t top) {  // (of a magnitude's bits; 0 is inside)
  constexpr uint32_t low = (127u - WINDOW) << 7, high = (127u + WINDOW) << 7;
  return top - low >= high - low && top != 0;
}
// Exponent of the unit for the largest magnitude's bits: its own, as far as its power and the
// reciprocal are normal numbers; 0 where it is no number.
__device__ __forceinline__ int unit_of(uint32_t top) {
  const int e = (int)(top >> 7);
  return e == 255 ? 0 : min(max(e, 1), 253) - 127;
}
__device__ __forceinline__ float power(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }

// Brings weights to their unit and returns its exponent.
__device__ __forceinline__ int weight_unit(u32x4& w) {
  uint32_t top = largest(w);
  if (!__any(outside<kWeightWindow>(top))) return 0;
#pragma unroll
  for (int l = 1; l < 64; l *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, l));
  const int u = unit_of(__builtin_amdgcn_readfirstlane(top));
  float f[8];
  unpack8(w, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= power(-u);
  w = pack8(f);
  return u;
}

// The gradient. The grid is bounded and its workgroups take the tokens in turn, so
// that a lane's share of dweight is summed over its tokens before it meets the
// others' (in a fixed order: lanes, waves, then workgroups). The turns of a
// workgroup's next tokens are made in the LDS half that the current ones leave.
// 32 + 8 heads of 128 columns, us (TB/s): 16384 tokens 98 without dweight (5.1),
// 101 with it (5.0), 1000 tokens 9 and 14. The sums of dweight hold 16 registers:
// three waves a SIMD and 768 workgroups, all of them resident (1024 in four waves
// with fewer registers: 105); without them four waves and 1024 (in three: 4096
// tokens 26 instead of 24).
template <int L, bool NB, int W, bool DW, int NT>
__global__ __launch_bounds__(kThreads, DW ? 3 : 4) void qk_backward_kernel(QKArgs a) {
  constexpr int H = 64 / L, STEP = W > 1 ? 1 : kWaves;
  __shared__ Turns<W> turns[2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k = W > 1 ? wave : 0, g0 = W > 1 ? 0 : wave;
  const Lane<L, NB> me(a);
  u32x4 w[2];
  int unit[2];
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = me.in && a.heads[i] ? ld16(a.w[i] + 8 * me.chunk) : zero16();
    unit[i] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  }
  int buf = 0;
  for (int token0 = blockIdx.x * W; token0 < a.tokens; token0 += gridDim.x * W, buf ^= 1) {
    const int token = token0 + k;
    const bool there = token < a.tokens;
    auto load = [&](int kind, int g, u32x4& x, u32x4& d) {
      const int head = g * H + me.head;
      x = d = zero16();
      if (!there || !me.in || head >= a.heads[kind]) return;
      x = ld_row<NT>(a.x[kind] + (int64_t)token * a.ldx[kind] + (int64_t)head * a.dim + 8 * me.chunk);
      d = ld_row<NT>(a.g[kind] + (int64_t)token * a.ldg[kind] + (int64_t)head * a.dim + 8 * me.chunk);
    };
    u32x4 x[2], d[2];
    load(0, g0, x[0], d[0]);
    load(1, g0, x[1], d[1]);
    make_turns(a, token0, turns[buf]);
    if (token0 == (int)blockIdx.x * W) {  // (behind the first loads)
      unit[0] = weight_unit(w[0]);
      unit[1] = weight_unit(w[1]);
    }
    __syncthreads();
    if (!there) continue;
    float c[8], s[8];
    me.turn(a, turns[buf], k, c, s);
    auto heads_of = [&](auto kind_) {
      constexpr int kind = decltype(kind_)::value;
      for (int g = g0; g * H < a.heads[kind]; g += STEP) {
        u32x4 nx, nd;
        load(kind, g + STEP, nx, nd);
        float f[8], m[8], p[8], wf[8];
        unpack8(x[kind], f);
        unpack8(d[kind], m);
        unpack8(w[kind], wf);
        me.pairs(d[kind], m, p);
        int gu = 0;
        const bool far = __any(outside<kGradWindow>(largest(d[kind])));
        if (far) {
          uint32_t top = largest(d[kind]);
#pragma unroll
          for (int l = 1; l < L; l *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, l));
          gu = unit_of(top);
#pragma unroll
          for (int e = 0; e < 8; ++e) m[e] *= power(-gu), p[e] *= power(-gu);
        }
        float ss = 0.f, along = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
        ss = sum_over<L>(ss);
        float down = 1.f;
        if (__any(past_range(ss))) {
          down = past_range(ss) ? kDown : 1.f;
          ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= down, ss += f[e] * f[e];
          ss = sum_over<L>(ss);
        }
        const float r = __builtin_amdgcn_rsqf(ss * a.mean + a.eps * down * down);
        float mw[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          mw[e] = m[e] * c[e] - p[e] * s[e];  // turned back
          f[e] *= r;                          // x / rms
          if constexpr (DW) {
            if (far) dw[kind][e] += __builtin_ldexpf(mw[e] * f[e], gu);
            else dw[kind][e] += mw[e] * f[e];
          }
          mw[e] *= wf[e];
          along += mw[e] * f[e];
        }
        along = sum_over<L>(along) * a.mean;
        if (!far && unit[kind] == 0) {
          const float outer = r * down;
#pragma unroll
          for (int e = 0; e < 8; ++e) mw[e] = (mw[e] - f[e] * along) * outer;
        } else {
          const float fraction = __builtin_amdgcn_frexp_mantf(r);
          const int places = __builtin_amdgcn_frexp_expf(r) + (down == 1.f ? 0 : kDownPlaces) + gu + unit[kind];
#pragma unroll
          for (int e = 0; e < 8; ++e) mw[e] = __builtin_ldexpf((mw[e] - f[e] * along) * fraction, places);
        }
        const int head = g * H + me.head;
        if (me.in && head < a.heads[kind])
          st_row<NT>(a.o[kind] + (int64_t)token * a.ldo[kind] + (int64_t)head * a.dim + 8 * me.chunk, pack8(mw));
        x[kind] = nx;
        d[kind] = nd;
      }
    };
    heads_of(std::integral_constant<int, 0>{});
    heads_of(std::integral_constant<int, 1>{});
  }
  if constexpr (DW) {
    __shared__ float sum[kWaves][2][8 * L];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int l = L; l < 64; l *= 2) dw[i][e] += __shfl_xor(dw[i][e], l);
        if (me.head == 0) sum[wave][i][8 * me.chunk + e] = dw[i][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.dim; c += kThreads) {
      const int which = c >= a.dim, col = c - which * a.dim;
      a.parts[(int64_t)blockIdx.x * 2 * a.dim + c] =
          (sum[0][which][col] + sum[1][which][col]) + (sum[2][which][col] + sum[3][which][col]);
    }
  }
}

// dweight = the workgroups' shares, 16 columns a workgroup: 64 threads take every
// 64th share of a column, and their sums are added in order.
__global__ __launch_bounds__(1024) void qk_weight_kernel(const float* parts, int32_t n, int32_t cols, float* out, int32_t accumulate) {
  __shared__ float sum[64][16 + 1];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int i = r; i < n; i += 64) s += parts[(int64_t)i * cols + col];
  }
  sum[r][c] = s;
  __syncthreads();
  if (r < 4) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sum[16 * r + i][c];
  }
  __syncthreads();
  if (r < 4) sum[r][c] = s;
  __syncthreads();
  if (r == 0 && col < cols) {
    s = (sum[0][c] + sum[1][c]) + (sum[2][c] + sum[3][c]);
    out[col] = accumulate ? out[col] + s : s;
  }
}

// Tokens of a workgroup: one a wave where there are enough of them to fill the GPU so.
// 32 + 8 heads of 128, forward, us, one token and four: 1024 tokens 6.5 and 7.0, 2048 10.2
// and 8.7.
constexpr int32_t kOneTokenBelow = 2048;
int tokens_of(int32_t tokens) { return tokens >= kOneTokenBelow ? kWaves : 1; }
constexpr int32_t kMostTokens = 0x7fff0000;  // a token's number and one grid more stay below 2^31
int64_t forward_groups(int32_t tokens) { return ((int64_t)tokens + tokens_of(tokens) - 1) / tokens_of(tokens); }
// Workgroups of the gradient: as many as run at once. With dweight and one token each, fewer,
// as their shares are all read again (1000 tokens: 512 take 13.8 us, 1024 16.7, 256 16.5).
int backward_groups(int32_t tokens, bool dw) {
  return (int)std::min<int64_t>(!dw ? 1024 : tokens_of(tokens) > 1 ? 768 : 512, forward_groups(tokens));
}
// Large batches pass the caches: what they write from kOneTokenBelow tokens on (4096 tokens 17
// -> 15 us), what they read too where all of it exceeds the Infinity Cache (16384 tokens,
// forward 66 -> 63, gradient 111 -> 105; 4096 tokens forward 15.0 -> 16.5).
constexpr int64_t kInfinityCache = 256 << 20;

int lanes_of(int32_t dim) { return dim <= 32 ? 4 : dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// Calls f(lanes, neighbours, tokens of a workgroup, NT) with all as compile-time constants.
template <class F>
void with_form(const lora_qk_heads_t& h, int32_t tokens, int64_t bytes, F f) {
  auto all = [&](auto lanes) {
    auto rest = [&](auto nb) {
      if (tokens_of(tokens) == 1) f(lanes, nb, std::integral_constant<int, 1>{}, std::integral_constant<int, 0>{});
      else if (bytes < kInfinityCache) f(lanes, nb, std::integral_constant<int, kWaves>{}, std::integral_constant<int, 1>{});
      else f(lanes, nb, std::integral_constant<int, kWaves>{}, std::integral_constant<int, 2>{});
    };
    if (h.neighbours) rest(std::true_type{});
    else rest(std::false_type{});
  };
  switch (lanes_of(h.head_dim)) {
    case 4: all(std::integral_constant<int, 4>{}); break;
    case 8: all(std::integral_constant<int, 8>{}); break;
    case 16: all(std::integral_constant<int, 16>{}); break;
    default: all(std::integral_constant<int, 32>{}); break;
  }
}
// Bytes of one matrix of all heads' rows.
int64_t rows_bytes(const lora_qk_heads_t& h, int32_t tokens) {
  return (int64_t)tokens * ((int64_t)h.heads_q + h.heads_k) * h.head_dim * 2;
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
  // (the mean and eps together stay in fp32's range: a mean is at most an eighth of it)
  if (!(h->eps >= 1.17549435e-38f) || !(h->eps <= 1e30f))
    return set_error(LORA_INVALID_ARGUMENT, "eps (%g) must be a positive normal number of at most 1e30", (double)h->eps);
  if ((h->heads_q && !h->weight_q) || (h->heads_k && !h->weight_k))
    return set_error(LORA_INVALID_ARGUMENT, "the weight of heads that there are is NULL");
  if ((h->heads_q && (reinterpret_cast<uintptr_t>(h->weight_q) & 15u)) || (h->heads_k && (reinterpret_cast<uintptr_t>(h->weight_k) & 15u)))
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
  a.x[0] = static_cast<const uint16_t*>(q); a.ldx[0] = ldq;
  a.x[1] = static_cast<const uint16_t*>(k); a.ldx[1] = ldk;
  a.o[0] = static_cast<uint16_t*>(oq); a.ldo[0] = ldoq;
  a.o[1] = static_cast<uint16_t*>(ok); a.ldo[1] = ldok;
  a.w[0] = static_cast<const uint16_t*>(h->weight_q);
  a.w[1] = static_cast<const uint16_t*>(h->weight_k);
  a.freqs = h->freqs;
  a.positions = positions;
  a.heads[0] = h->heads_q; a.heads[1] = h->heads_k;
  a.tokens = tokens;
  a.dim = h->head_dim; a.rot = h->rot_dim;
  a.eps = h->eps; a.mean = 1.f / (float)h->head_dim;
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
  if (num_tokens > 1 && ((heads->heads_q && q_out == q && ldqo != ldq) || (heads->heads_k && k_out == k && ldko != ldk)))
    return set_error(LORA_INVALID_ARGUMENT, "an output that takes its input's place needs its row stride");
  QKArgs a = args_of(heads, q, ldq, k, ldk, positions, num_tokens, q_out, ldqo, k_out, ldko);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n = forward_groups(num_tokens);
  if (n > kMaxGroups) return set_error(LORA_UNSUPPORTED, "%d tokens are too many for one call", num_tokens);
  with_form(*heads, num_tokens, 2 * rows_bytes(*heads, num_tokens), [&](auto lanes, auto nb, auto w, auto nt) {
    hipLaunchKernelGGL((qk_forward_kernel<lanes(), nb(), w(), (w() > 1 ? 4 : 1), nt()>), dim3((unsigned)n), dim3(kThreads), 0, s, a);
  });
  return launched("qk_norm_rope");
}

extern "C" int lora_workspace_size_qk(const lora_qk_heads_t* heads, int32_t num_tokens, size_t* bytes) {
  clear_error();
  const int st = check_heads(heads);
  if (st) return st;
  if (!bytes || num_tokens < 0) return set_error(LORA_INVALID_ARGUMENT, "bytes is NULL or num_tokens (%d) below 0", num_tokens);
  *bytes = (size_t)backward_groups(num_tokens, true) * 2 * (size_t)heads->head_dim * sizeof(float);
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
      const size_t need = (size_t)backward_groups(num_tokens, true) * 2 * (size_t)heads->head_dim * sizeof(float);
      if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15u)) return set_error(LORA_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
      if (ws_bytes < need)
        return set_error(LORA_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, %zu are needed", ws_bytes, need);
    }
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int cols = 2 * heads->head_dim;
  const int groups = backward_groups(num_tokens, dweight != nullptr);
  if (num_tokens) {
    QKArgs a = args_of(heads, q, ldq, k, ldk, positions, num_tokens, dq, lddq, dk, lddk);
    a.g[0] = static_cast<const uint16_t*>(dq_out); a.ldg[0] = lddqo;
    a.g[1] = static_cast<const uint16_t*>(dk_out); a.ldg[1] = lddko;
    a.parts = static_cast<float*>(ws);
    with_form(*heads, num_tokens, 3 * rows_bytes(*heads, num_tokens), [&](auto lanes, auto nb, auto w, auto nt) {
      const dim3 grid((unsigned)groups), blk(kThreads);
      if (dweight) hipLaunchKernelGGL((qk_backward_kernel<lanes(), nb(), w(), true, nt()>), grid, blk, 0, s, a);
      else hipLaunchKernelGGL((qk_backward_kernel<lanes(), nb(), w(), false, nt()>), grid, blk, 0, s, a);
    });
    if ((st = launched("qk_norm_rope_backward"))) return st;
  }
  if (dweight) {
    // (no tokens: no shares, and zeros or nothing to add)
    hipLaunchKernelGGL(qk_weight_kernel, dim3((unsigned)((cols + 15) / 16)), dim3(1024), 0, s, static_cast<const float*>(ws),
                       groups, cols, dweight, (flags & LORA_GRAD_ACCUMULATE) ? 1 : 0);
    return launched("qk_weight");
  }
  return LORA_OK;
}
