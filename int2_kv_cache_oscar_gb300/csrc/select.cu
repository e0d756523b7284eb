// Choosing the groups worth attending (sm_103a): an 8-bit summary of every
// quantised group, a score of each group for a new query, and the largest
// scores of each KV head.
//
// Summary of a group (keys k_hat = code s + z of norm n): every channel's
// lowest and highest value, lo = z and hi = fl32(z + 3 s), in whole steps of
// 2^e (nearest even), e the smallest exponent >= -100 that keeps them within
// +-127, and the largest and smallest norm times 2^e:
//   lo8, hi8 = rne(lo 2^-e), rne(hi 2^-e);  w_max, w_min = fl32(n 2^e).
//
// Score of a group for the query heads of a KV head:
//   a = rne(q 2^(22 - E)), E the smallest exponent >= -100 with |q| < 2^E over
//   those heads; b = Hu a (unnormalised Walsh-Hadamard, whole numbers);
//   q8 = floor(b / 2^B + 1/2), B >= 0 the smallest shift with |b| <= 127 2^B;
//   S = max over heads of sum_c max(q8_c lo8_c, q8_c hi8_c);
//   score = S w_max if S >= 0, else S w_min.
// Up to the 8-bit steps this is the largest score that a key inside the
// group's box could reach.  Everything up to S is whole numbers and the score
// is a 22-bit times a 24-bit number in float64, so scores are exact, the order
// does not depend on how the sums are split, and ties are true ties (the
// lowest group wins).
//
// Bound by latency for a few rows (a score pass over 264 bytes a group, then a
// radix selection in shared memory), by HBM / L2 for many.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace oscar {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelBatch = 4;   // groups in flight per warp
constexpr int kIdxThreads = 256;
constexpr int kIdxMinExp = -100;

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ float finite_or_zero(float x) {
  return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? 0.0f : x;
}

// ----------------------------------------------------------- summaries
// One warp per group: lane l summarises channels 4 l .. 4 l + 3.
template <int MAXS, bool M16>
__global__ void __launch_bounds__(kIdxThreads)
    index_kernel(const __grid_constant__ IndexParams<MAXS> p, const uint8_t* __restrict__ arena) {
  using B = Blk<M16>;
  using MR = Meta<M16>;
  const IndexSeq sq = p.seq[blockIdx.z];
  const int g = sq.first + (int)(blockIdx.x * (kIdxThreads / 32) + (threadIdx.x >> 5));
  if (g >= sq.end) return;
  const int lane = threadIdx.x & 31;
  const int64_t at = ((int64_t)sq.slot * gridDim.y + blockIdx.y) * p.max_groups + g;
  const uint8_t* blk = arena + p.blocks_off + at * (int64_t)B::kBytes;
  const float2 s0 = MR::two(blk + B::kKScale, 4 * lane), s1 = MR::two(blk + B::kKScale, 4 * lane + 2);
  const float2 z0 = MR::two(blk + B::kKZero, 4 * lane), z1 = MR::two(blk + B::kKZero, 4 * lane + 2);
  const float2 n0 = MR::two(blk + B::kKNorm, 4 * lane), n1 = MR::two(blk + B::kKNorm, 4 * lane + 2);
  const float s[4] = {s0.x, s0.y, s1.x, s1.y};
  const float z[4] = {z0.x, z0.y, z1.x, z1.y};
  float lo[4], hi[4], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = finite_or_zero(z[i]);
    hi[i] = finite_or_zero(__fmaf_rn(3.0f, s[i], z[i]));
    top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
  }
  const float n[4] = {finite_or_zero(n0.x), finite_or_zero(n0.y), finite_or_zero(n1.x), finite_or_zero(n1.y)};
  // non-negative floats order as their bit patterns
  const uint32_t tb = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  const uint32_t nmax = __reduce_max_sync(
      0xffffffffu, __float_as_uint(fmaxf(fmaxf(fabsf(n[0]), fabsf(n[1])), fmaxf(fabsf(n[2]), fabsf(n[3])))));
  const uint32_t nmin = __reduce_min_sync(
      0xffffffffu, __float_as_uint(fminf(fminf(fabsf(n[0]), fabsf(n[1])), fminf(fabsf(n[2]), fabsf(n[3])))));
  // top = m 2^x, m in [1/2, 1): 127 2^(x - 7) >= top where m <= 127/128
  int e = (int)(tb >> 23) - 126 - ((tb & 0x7fffffu) <= 0x7e0000u ? 7 : 6);
  e = tb == 0u ? kIdxMinExp : max(e, kIdxMinExp);
  const float f = exp2i(-e);
  uint32_t wl = 0, wh = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wl |= ((uint32_t)__float2int_rn(lo[i] * f) & 0xffu) << (8 * i);
    wh |= ((uint32_t)__float2int_rn(hi[i] * f) & 0xffu) << (8 * i);
  }
  p.codes[at * 32 + lane] = make_uint2(wl, wh);
  if (lane == 0) p.weights[at] = make_float2(__uint_as_float(nmax) * exp2i(e), __uint_as_float(nmin) * exp2i(e));
}

// ------------------------------------------------------------ selection

// Order-preserving bits of a float64 (no NaN; -0 already made +0).
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

struct SelSmem {
  uint32_t red[kSelThreads / 32];
  uint64_t red64[2][kSelThreads / 32];
  uint32_t hist[256];
  uint32_t cnt[2][kSelThreads / 32];
  uint32_t digit, above, inbin;
};

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kSelThreads / 32; ++i) m = max(m, red[i]);
  return m;
}

template <int MAXS>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelectParams<MAXS> p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ SelSmem S;
  const int b = blockIdx.x / p.hkv, j = blockIdx.x % p.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ng = p.seq[b].ng, gqa = p.q_group;
  int32_t* out = p.out + ((int64_t)b * p.hkv + j) * p.n_select;
  const int m = min(p.n_select, ng);
  for (int i = m + tid; i < p.n_select; i += kSelThreads) out[i] = -1;
  if (ng <= p.n_select) {
    for (int i = tid; i < ng; i += kSelThreads) out[i] = i;
    return;
  }
  // dynamic shared memory: [gqa][32] rotated queries (4 channels a lane), [gqa][32] their bytes (parts above and
  // below zero), [ng] score keys
  int4* turned = reinterpret_cast<int4*>(smem_raw);
  int2* q8 = reinterpret_cast<int2*>(turned + (size_t)gqa * 32);
  uint64_t* keys = reinterpret_cast<uint64_t*>(q8 + (size_t)gqa * 32);

  // ---- the queries in 8 bits, one step size for the heads of the KV head
  const uint16_t* q = p.q + ((int64_t)b * p.hq + (int64_t)j * gqa) * kHeadDim;
  auto load_q = [&](int h, float* f) {
    const uint2 raw = *reinterpret_cast<const uint2*>(q + h * kHeadDim + 4 * lane);
    f[0] = finite_or_zero(bf16_lo(raw.x));
    f[1] = finite_or_zero(bf16_hi(raw.x));
    f[2] = finite_or_zero(bf16_lo(raw.y));
    f[3] = finite_or_zero(bf16_hi(raw.y));
  };
  uint32_t top = 0;
  for (int h = warp; h < gqa; h += kSelThreads / 32) {
    float f[4];
    load_q(h, f);
    top = max(top, __float_as_uint(fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])))));
  }
  top = block_max(top, S.red);
  const float up = exp2i(22 - max((int)(top >> 23) - 126, kIdxMinExp));
  uint32_t big = 0;
  for (int h = warp; h < gqa; h += kSelThreads / 32) {
    float f[4];
    load_q(h, f);
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float2int_rn(f[i] * up);
    const int a0 = v[0] + v[1], a1 = v[0] - v[1], a2 = v[2] + v[3], a3 = v[2] - v[3];
    v[0] = a0 + a2;
    v[1] = a1 + a3;
    v[2] = a0 - a2;
    v[3] = a1 - a3;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int other = __shfl_xor_sync(0xffffffffu, v[i], o);
        v[i] = upper ? other - v[i] : v[i] + other;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) big = max(big, (uint32_t)abs(v[i]));
    turned[h * 32 + lane] = make_int4(v[0], v[1], v[2], v[3]);
  }
  big = block_max(big, S.red);
  int shift = 0;
  while (big > (127u << shift)) ++shift;
  const int round = (1 << shift) >> 1;
  for (int h = warp; h < gqa; h += kSelThreads / 32) {
    const int4 t = turned[h * 32 + lane];
    const int v[4] = {(t.x + round) >> shift, (t.y + round) >> shift, (t.z + round) >> shift, (t.w + round) >> shift};
    uint32_t pos = 0, neg = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pos |= (uint32_t)(max(v[i], 0) & 0xff) << (8 * i);
      neg |= (uint32_t)(min(v[i], 0) & 0xff) << (8 * i);
    }
    q8[h * 32 + lane] = make_int2((int)pos, (int)neg);
  }
  __syncthreads();

  // ---- scores: one warp per group, kSelBatch groups in flight
  const int64_t row = (int64_t)p.seq[b].slot * p.hkv + j;
  const uint2* codes = p.codes + row * p.max_groups * 32;
  const float2* weights = p.weights + row * p.max_groups;
  uint64_t kmin = ~0ull, kmax = 0;
  for (int g0 = warp * kSelBatch; g0 < ng; g0 += kSelThreads / 32 * kSelBatch) {
    uint2 c[kSelBatch];
#pragma unroll
    for (int i = 0; i < kSelBatch; ++i)
      c[i] = g0 + i < ng ? codes[(int64_t)(g0 + i) * 32 + lane] : make_uint2(0u, 0u);
    float2 w = make_float2(0.0f, 0.0f);
    if (lane < kSelBatch && g0 + lane < ng) w = weights[g0 + lane];
    int best[kSelBatch];
#pragma unroll
    for (int i = 0; i < kSelBatch; ++i) best[i] = INT32_MIN;
    for (int h = 0; h < gqa; ++h) {
      const int2 qq = q8[h * 32 + lane];
#pragma unroll
      for (int i = 0; i < kSelBatch; ++i) {
        const int s = __reduce_add_sync(0xffffffffu, __dp4a((int)c[i].y, qq.x, __dp4a((int)c[i].x, qq.y, 0)));
        best[i] = max(best[i], s);
      }
    }
    int s = best[0];
#pragma unroll
    for (int i = 1; i < kSelBatch; ++i) s = lane == i ? best[i] : s;
    const int g = g0 + lane;
    if (lane < kSelBatch && g < ng) {
      const double score = (double)s * (double)(s >= 0 ? w.x : w.y) + 0.0;   // -0 + 0 = +0
      const bool kept = g < p.keep_first || g >= ng - p.keep_last;
      const uint64_t key = kept ? ~0ull : order_key(score);
      keys[g] = key;
      if (!kept) {
        kmin = min(kmin, key);
        kmax = max(kmax, key);
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    kmin = min(kmin, __shfl_xor_sync(0xffffffffu, kmin, o));
    kmax = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
  }
  if (lane == 0) {
    S.red64[0][warp] = kmin;
    S.red64[1][warp] = kmax;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSelThreads / 32; ++i) {
    kmin = min(kmin, S.red64[0][i]);
    kmax = max(kmax, S.red64[1][i]);
  }

  // ---- the m-th largest key, 8 bits at a time from the first bit in which
  // the scored keys differ; kept groups are above every one of them
  const int forced = min(ng, p.keep_first) + min(max(ng - p.keep_first, 0), p.keep_last);
  int need = m - forced;                   // still to choose among the scored groups with `prefix`
  int bits = kmax > kmin ? 64 - __clzll((long long)(kmin ^ kmax)) : 0;   // undecided low bits
  uint64_t prefix = bits < 64 ? kmin >> bits : 0;                        // the bits above them
  bool all = false;                        // every key with the prefix is chosen
  while (bits > 0 && need > 0 && !all) {
    const int d = min(bits, 8), low = bits - d;
    if (tid < 256) S.hist[tid] = 0;
    __syncthreads();
    for (int g = tid; g < ng; g += kSelThreads) {
      const uint64_t k = keys[g];
      if (k != ~0ull && (bits == 64 || (k >> bits) == prefix)) atomicAdd(&S.hist[(uint32_t)(k >> low) & ((1u << d) - 1)], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l owns digits 255 - 8 l .. 248 - 8 l, the largest first
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = S.hist[255 - 8 * lane - i];
        sum += c[i];
      }
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up2 = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += up2;
      }
      before -= sum;                       // keys in larger digits than this lane's
      if (before < (uint32_t)need && (uint32_t)need <= before + sum) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < (uint32_t)need && (uint32_t)need <= before + c[i]) {
            S.digit = 255 - 8 * lane - i;
            S.above = before;
            S.inbin = c[i];
          }
          before += c[i];
        }
      }
    }
    __syncthreads();
    need -= (int)S.above;
    all = (uint32_t)need == S.inbin;
    prefix = (prefix << d) | S.digit;
    bits = low;
  }
  // chosen: keys whose top bits are above the prefix; of those equal to it all,
  // or (every bit decided) the `need` lowest groups
  const uint64_t limit = prefix;
  if (all) need = INT32_MAX;

  // ---- the chosen groups in ascending order
  int done_gt = 0, done_eq = 0;
  for (int g0 = 0; g0 < ng; g0 += kSelThreads) {
    const int g = g0 + tid;
    bool gt = false, eq = false;
    if (g < ng) {
      const uint64_t k = keys[g];
      const uint64_t t = bits < 64 ? k >> bits : 0;
      gt = k == ~0ull || t > limit;
      eq = !gt && t == limit;
    }
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) {
      S.cnt[0][warp] = __popc(bg);
      S.cnt[1][warp] = __popc(be);
    }
    __syncthreads();
    int ngt = done_gt, neq = done_eq;
#pragma unroll
    for (int i = 0; i < kSelThreads / 32; ++i) {
      const int x = S.cnt[0][i], y = S.cnt[1][i];
      if (i < warp) {
        ngt += x;
        neq += y;
      }
      done_gt += x;
      done_eq += y;
    }
    const uint32_t below = (1u << lane) - 1;
    ngt += __popc(bg & below);
    neq += __popc(be & below);
    if (gt || (eq && neq < need)) out[ngt + min(neq, need)] = g;
  }
}

template <int MAXS, bool M16>
cudaError_t launch_index_t(const IndexParams<MAXS>& p, const uint8_t* arena, int groups, cudaStream_t stream) {
  constexpr int per = kIdxThreads / 32;
  index_kernel<MAXS, M16><<<dim3((groups + per - 1) / per, p.hkv, p.n_seqs), kIdxThreads, 0, stream>>>(p, arena);
  return cudaGetLastError();
}

}  // namespace

template <int MAXS>
cudaError_t launch_index(const IndexParams<MAXS>& p, const uint8_t* arena, bool meta16, cudaStream_t stream) {
  int groups = 0;
  for (int i = 0; i < p.n_seqs; ++i) groups = std::max(groups, p.seq[i].end - p.seq[i].first);
  if (groups <= 0) return cudaSuccess;
  return meta16 ? launch_index_t<MAXS, true>(p, arena, groups, stream)
                : launch_index_t<MAXS, false>(p, arena, groups, stream);
}

size_t select_smem_bytes(int q_group, int groups) {
  return (size_t)q_group * 32 * (sizeof(int4) + sizeof(int2)) + (size_t)groups * sizeof(uint64_t);
}

template <int MAXS>
cudaError_t launch_select(const SelectParams<MAXS>& p, cudaStream_t stream) {
  int groups = 0;
  for (int i = 0; i < p.n_seqs; ++i) groups = std::max(groups, p.seq[i].ng);
  const size_t smem = groups > p.n_select ? select_smem_bytes(p.q_group, groups) : 0;
  static bool attr_done[64] = {};
  cudaError_t e = ensure_smem_attr(select_kernel<MAXS>, kSelectMaxSmem, attr_done);
  if (e != cudaSuccess) return e;
  select_kernel<MAXS><<<(unsigned)(p.n_seqs * p.hkv), kSelThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

#define OSCAR_INSTANTIATE(N)                                                                                  \
  template cudaError_t launch_index<N>(const IndexParams<N>&, const uint8_t*, bool, cudaStream_t);            \
  template cudaError_t launch_select<N>(const SelectParams<N>&, cudaStream_t);
OSCAR_INSTANTIATE(kDecodeSeqsSmall)
OSCAR_INSTANTIATE(kDecodeSeqsLarge)
#undef OSCAR_INSTANTIATE

}  // namespace oscar
