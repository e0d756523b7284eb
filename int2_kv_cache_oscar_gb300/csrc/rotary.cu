// Rotary positions of queries and keys (sm_103a): one launch turns the query
// and the key rows of a run of tokens, half or interleaved layout, over the
// first rotary_dim channels of the 128-channel heads.
//
//   (y_a, y_b) = m (x_a cos t - x_b sin t, x_a sin t + x_b cos t),
//   t = position * frequency(pair); the transpose (the gradient) takes -t.
//
// Angles.  A float32 angle of position 131,072 is off by up to 4e-3 rad, and
// float64 products are slow on this chip, so the angle is kept as a phase, in
// turns modulo one, in 64-bit fixed point: phase = position * F mod 2^64 with
// F = frequency / (2 pi) * 2^64, exact integer arithmetic (off by 2^-33 of a
// turn at position 2^31).  Its top 32 bits give the quadrant and the remainder
// (at most an eighth of a turn) for sincospif; as a float32 that is off by
// 2^-28 of a turn at most.
//
// What bounds it: every element is read and written once, so HBM for long
// runs and the launch for one token.  A block computes the cosines and sines
// of its few tokens once for all heads (shared memory) after it has requested
// its rows, so the loads and that arithmetic overlap.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace oscar {
namespace {

constexpr int kRotThreads = 128;
// Threads, row pieces in flight per thread and blocks per SM, measured on a
// bf16 chunk of 8,192 tokens and a float32 run of 2,053: 128 x 2 x 8 27.7 and
// 9.2 us; 256 x 4 x 3 28.5 and 10.3; 128 x 3 x 6 27.6 and 9.6; 256 x 2 x 4 32.5
// and 10.6; 128 x 2 x 10 28.8 and 11.0.
constexpr int kRotItems = 2;
constexpr int kRotBlocks = 8;
constexpr int kRotMaxTokens = 32;   // tokens of one block

// cos and sin of a phase (turns, 2^64 to the turn)
__device__ __forceinline__ float2 phase_cos_sin(uint64_t phase) {
  const uint32_t x = (uint32_t)(phase >> 32) + 0x20000000u;   // + 1/8 turn: quadrant by rounding
  const int32_t r = (int32_t)(x & 0x3fffffffu) - 0x20000000;  // remainder, 2^-32 turns
  float s, c;
  sincospif((float)r * 0x1p-31f, &s, &c);
  switch (x >> 30) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
  }
}

template <bool F32>
struct Row;   // 16 bytes of a row, as float32 values
template <>
struct Row<false> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void widen(const uint4& u, float* f) {
    f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
    f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
  }
  static __device__ __forceinline__ uint4 narrow(const float* f) {   // nearest even: the output type
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Row<true> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ void widen(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 narrow(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// A row is cut into items of two 16-byte pieces: in the half layout piece i of
// the first half and of the second half of the rotated channels, in the
// interleaved layout (and behind the rotated channels) two neighbours.  A
// thread keeps its item of the row and walks over the rows (token, head) of
// the block; an item's cosines and sines are V / 2 float4 (two pairs each),
// stored so that the threads of a row read neighbouring ones.
template <bool F32, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotThreads, kRotBlocks) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using R = Row<F32>;
  constexpr int V = R::kVec;
  constexpr int kRowItems = kHeadDim / (2 * V);
  __shared__ __align__(16) float4 table[kRotMaxTokens][V / 2][kRowItems];   // (cos, cos, sin, sin)
  const int64_t t0 = (int64_t)blockIdx.x * p.block_tokens;
  const int tokens = (int)min((int64_t)p.block_tokens, (int64_t)p.n - t0);
  const int rows = p.q.heads + p.k.heads;
  const int rot_items = p.dim / (2 * V);
  const int half = p.dim / 2;
  const int j = threadIdx.x % kRowItems;
  const bool turned = j < rot_items;
  // byte offsets of the two pieces
  const int at_a = (!INTERLEAVED && turned ? V * j : 2 * V * j) * (16 / V);
  const int at_b = !INTERLEAVED && turned ? at_a + half * (16 / V) : at_a + 16;
  int tok = (int)(threadIdx.x / kRowItems) / rows;
  int h = (int)(threadIdx.x / kRowItems) - tok * rows;

  grid_dependency_wait();
  allow_dependents();
  bool first = true;
  for (int done = 0; done < tokens * rows; done += kRotThreads / kRowItems * kRotItems) {
    uint4 xa[kRotItems], xb[kRotItems];
    uint8_t* dst[kRotItems];
    int tk[kRotItems];
#pragma unroll
    for (int i = 0; i < kRotItems; ++i) {
      tk[i] = tok;
      if (tok < tokens) {
        const bool isq = h < p.q.heads;
        const RotaryRows& x = isq ? p.q : p.k;
        const int64_t head = isq ? h : h - p.q.heads;
        const uint8_t* src = x.in + (t0 + tok) * x.in_token + head * x.in_head;
        dst[i] = x.out + (t0 + tok) * x.out_token + head * x.out_head;
        xa[i] = *reinterpret_cast<const uint4*>(src + at_a);
        xb[i] = *reinterpret_cast<const uint4*>(src + at_b);
      }
      h += p.step_rows;
      tok += p.step_tokens;
      if (h >= rows) {
        h -= rows;
        ++tok;
      }
    }
    if (first) {
      first = false;
      for (int i = threadIdx.x; i < tokens * half; i += kRotThreads) {
        const int t = i / half, pair = i - t * half;
        const uint64_t pos = (uint64_t)(int64_t)p.positions[t0 + t];
        const float2 cs = phase_cos_sin(pos * p.freq[pair]);
        float* e = reinterpret_cast<float*>(&table[t][(pair % V) / 2][pair / V]) + (pair & 1);
        e[0] = cs.x * p.factor;
        e[2] = cs.y * (p.transpose ? -p.factor : p.factor);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kRotItems; ++i) {
      if (tk[i] >= tokens) continue;
      uint4 ya = xa[i], yb = xb[i];
      if (turned) {
        float u[2 * V];
        R::widen(ya, u);
        R::widen(yb, u + V);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {   // pairs 2 e, 2 e + 1 of the item
          const float4 w = table[tk[i]][e][j];
          const float2 c = make_float2(w.x, w.y), s = make_float2(w.z, w.w);
          const int a0 = INTERLEAVED ? 4 * e : 2 * e, b0 = INTERLEAVED ? 4 * e + 1 : V + 2 * e;
          const int a1 = INTERLEAVED ? 4 * e + 2 : 2 * e + 1, b1 = INTERLEAVED ? 4 * e + 3 : V + 2 * e + 1;
          const float2 a = make_float2(u[a0], u[a1]), b = make_float2(u[b0], u[b1]);
          const float2 bs = __fmul2_rn(b, s), bc = __fmul2_rn(b, c);
          const float2 y = __ffma2_rn(a, c, make_float2(-bs.x, -bs.y)), z = __ffma2_rn(a, s, bc);
          u[a0] = y.x;
          u[a1] = y.y;
          u[b0] = z.x;
          u[b1] = z.y;
        }
        ya = R::narrow(u);
        yb = R::narrow(u + V);
      }
      *reinterpret_cast<uint4*>(dst[i] + at_a) = ya;
      *reinterpret_cast<uint4*>(dst[i] + at_b) = yb;
    }
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& params, bool f32, bool interleaved, int sms, cudaStream_t stream) {
  RotaryParams p = params;
  const int rows = p.q.heads + p.k.heads;
  if (p.n <= 0 || rows <= 0) return cudaSuccess;
  const int per_token = rows * (kHeadDim / (2 * (f32 ? Row<true>::kVec : Row<false>::kVec)));
  // as many tokens as give every thread its kRotItems pieces; between one and
  // two waves of blocks, as many as make it one
  const int64_t slots = (int64_t)kRotBlocks * sms;
  int64_t tokens = std::max<int64_t>(1, kRotThreads * kRotItems / per_token);
  if (p.n <= tokens * 2 * slots) tokens = (p.n + slots - 1) / slots;
  tokens = std::max<int64_t>(1, std::min<int64_t>(tokens, kRotMaxTokens));
  p.block_tokens = (int32_t)tokens;
  const int step = kRotThreads / (kHeadDim / (2 * (f32 ? Row<true>::kVec : Row<false>::kVec)));   // rows per round
  p.step_tokens = step / rows;
  p.step_rows = step % rows;
  const unsigned grid = (unsigned)((p.n + tokens - 1) / tokens);
  const auto kernel = f32 ? (interleaved ? rotary_kernel<true, true> : rotary_kernel<true, false>)
                          : (interleaved ? rotary_kernel<false, true> : rotary_kernel<false, false>);
  return launch_dependent(kernel, dim3(grid), dim3(kRotThreads), 0, stream, 1, p);
}

}  // namespace oscar
