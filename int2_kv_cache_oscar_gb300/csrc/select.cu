// Choosing the groups worth attending (sm_103a): an 8-bit summary of every
// quantised group, a score of each group for a new query, and the largest
// scores of each KV head.
//
// Summary of a group (keys k_hat = code s + z of norm n): every channel's
// lowest and highest value, lo = z and hi = fl32(z + 3 s), in whole steps of
// 2^e (nearest even), e the smallest exponent >= -100 that keeps them within
// +-127, and the largest and smallest norm times 2^e:
//   lo8, hi8 = rne(lo 2^-e), rne(hi 2^-e);  w_max, w_min = fl32(n 2^e), at most
//   the largest float32.  What is not finite counts as 0.
//
// Score of a group for the query heads of a KV head:
//   a = rne(q 2^(22 - E)), E the smallest exponent >= -100 with |q| < 2^E over
//   those heads; b = Hu a (unnormalised Walsh-Hadamard, whole numbers);
//   q8 = floor(b / 2^B + 1/2), B >= 0 the smallest shift with |b| <= 127 2^B;
//   S = max over heads of sum_c max(q8_c lo8_c, q8_c hi8_c);
//   score = S w_max if S >= 0, else S w_min.
// Up to the 8-bit steps this is the largest score that a key inside the
// group's box could reach.  Everything up to S is whole numbers and the score
// is a 21-bit times a 24-bit number, so scores are exact, the order does not
// depend on how the sums are split, and ties are true ties (the lowest group
// wins).
//
// Selection: a cluster of 1 to 8 blocks per (sequence, KV head) row, each
// scoring a contiguous slice of its groups and storing the scores' keys into
// the first block's shared memory; that block then chooses.  A slice's codes
// come by bulk copies of up to 256 groups (64 KB), two in flight, requested
// before the queries are turned.  Four lanes score a group: each holds a
// quarter of the query bytes of four heads in registers (a warp per group,
// with a warp sum per head, took four times the instructions), then each makes
// the key of one of its warp's four batches (8.9 -> 8.3 us for 256 rows of 256
// groups; every lane making every key costs four times the key's operations).
// The m-th largest key is found by a radix histogram, starting at the first
// bit in which the row's keys differ, and, once at most 32 keys share a digit,
// by ranking those.  Everything is latency and, for many rows, instructions.
#include <algorithm>
#include <cfloat>
#include <cstddef>

#include "common.cuh"
#include "launch.h"

namespace oscar {
namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelHeads = 4;      // query heads scored at once
constexpr int kSelChunk = 256;    // groups of one bulk copy at most: 4 batches of 8 a warp
constexpr int kSelStages = 2;     // copies in flight
constexpr int kSelRank = 32;      // keys ranked directly
static_assert(kSelThreads == 256, "one thread per digit of the histogram");
static_assert(kSelChunk == 4 * 8 * kSelWarps, "a lane per group of a chunk");
constexpr int kIdxThreads = 256;
constexpr int kIdxMinExp = -100;

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ float finite_or_zero(float x) {
  return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? 0.0f : x;
}

// ----------------------------------------------------------- summaries
// One warp per group; lane l summarises channels 4 l .. 4 l + 3.  Bound by HBM:
// 1,536 (768) bytes read and 264 written per group.  (Two or four groups in
// flight per warp took as long, within 2 %.)
template <bool M16>
__device__ __forceinline__ float4 meta4(const uint8_t* section, int lane) {   // elements 4 lane .. + 3
  if constexpr (M16) {
    const uint2 h = *reinterpret_cast<const uint2*>(section + 8 * lane);
    return make_float4(half_lo_to_float(h.x), half_hi_to_float(h.x), half_lo_to_float(h.y), half_hi_to_float(h.y));
  } else {
    return *reinterpret_cast<const float4*>(section + 16 * lane);
  }
}

template <int MAXS, bool M16>
__global__ void __launch_bounds__(kIdxThreads)
    index_kernel(const __grid_constant__ IndexParams<MAXS> p, const uint8_t* __restrict__ arena) {
  using B = Blk<M16>;
  grid_dependency_wait();
  allow_dependents();
  const IndexSeq sq = p.seq[blockIdx.z];
  const int g = sq.first + (int)(blockIdx.x * (kIdxThreads / 32) + (threadIdx.x >> 5));
  if (g >= sq.end) return;
  const int lane = threadIdx.x & 31;
  const int64_t at = ((int64_t)sq.slot * gridDim.y + blockIdx.y) * p.max_groups + g;
  const uint8_t* blk = arena + p.blocks_off + at * (int64_t)B::kBytes;
  const float4 s4 = meta4<M16>(blk + B::kKScale, lane), z4 = meta4<M16>(blk + B::kKZero, lane),
               n4 = meta4<M16>(blk + B::kKNorm, lane);
  const float s[4] = {s4.x, s4.y, s4.z, s4.w};
  const float z[4] = {z4.x, z4.y, z4.z, z4.w};
  const float n[4] = {fabsf(finite_or_zero(n4.x)), fabsf(finite_or_zero(n4.y)), fabsf(finite_or_zero(n4.z)),
                      fabsf(finite_or_zero(n4.w))};
  float lo[4], hi[4], top = 0.0f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    lo[c] = finite_or_zero(z[c]);
    hi[c] = finite_or_zero(__fmaf_rn(3.0f, s[c], z[c]));
    top = fmaxf(top, fmaxf(fabsf(lo[c]), fabsf(hi[c])));
  }
  // non-negative floats order as their bit patterns
  const uint32_t tb = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  const uint32_t nmax = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fmaxf(n[0], n[1]), fmaxf(n[2], n[3]))));
  const uint32_t nmin = __reduce_min_sync(0xffffffffu, __float_as_uint(fminf(fminf(n[0], n[1]), fminf(n[2], n[3]))));
  // top = m 2^x, m in [1/2, 1): 127 2^(x - 7) >= top where m <= 127/128
  int e = (int)(tb >> 23) - 126 - ((tb & 0x7fffffu) <= 0x7e0000u ? 7 : 6);
  e = tb == 0u ? kIdxMinExp : max(e, kIdxMinExp);
  const float f = exp2i(-e);
  uint32_t wl = 0, wh = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    wl |= ((uint32_t)__float2int_rn(lo[c] * f) & 0xffu) << (8 * c);
    wh |= ((uint32_t)__float2int_rn(hi[c] * f) & 0xffu) << (8 * c);
  }
  p.codes[at * 32 + lane] = make_uint2(wl, wh);
  if (lane == 0)
    p.weights[at] = make_float2(fminf(__uint_as_float(nmax) * exp2i(e), FLT_MAX),
                                fminf(__uint_as_float(nmin) * exp2i(e), FLT_MAX));
}

// ------------------------------------------------------------ selection

// Order-preserving key of the exact product s w (|s| <= 2^22, w >= 0 finite):
// sign, exponent and the product's 46 bits, in whole-number operations (as
// float64 products, whose instructions cost a warp 64 to 76 cycles on this
// chip, 256 rows of 256 groups took 10.0 us instead of 8.9).
__device__ __forceinline__ uint64_t score_key(int s, float w) {
  const uint32_t wb = __float_as_uint(w);
  const uint32_t ex = wb >> 23;
  const uint32_t mant = ex ? (wb & 0x7fffffu) | 0x800000u : wb;      // w = mant 2^(max(ex, 1) - 150)
  const uint64_t p = (uint64_t)(uint32_t)abs(s) * mant;
  if (p == 0) return 1ull << 63;
  const int lz = __clzll((long long)p);
  const uint64_t mag = ((uint64_t)(max(ex, 1u) + 63 - lz) << 46) | (((p << lz) >> 17) & ((1ull << 46) - 1));
  return s >= 0 ? (1ull << 63) | mag : ~((1ull << 63) | mag);
}

struct SelSmem {
  alignas(8) uint64_t full[kSelStages];
  uint64_t cand[kSelRank];         // keys to rank
  int32_t cand_group[kSelRank];
  uint64_t limit_key;
  alignas(16) uint32_t hist[256];   // read as uint4
  uint32_t red[4][kSelWarps];
  uint32_t cnt[2][2][kSelWarps];
  uint32_t n_cand;
  uint32_t digit, above, inbin;
  int32_t limit_group;
  int abort_flag;
};
static_assert(offsetof(SelSmem, hist) % 16 == 0 && offsetof(SelSmem, full) % 8 == 0 && alignof(SelSmem) >= 16,
              "vector loads of the histogram, 8-byte barriers");

// Address of a shared variable in block `rank` of the cluster.
template <typename T>
__device__ __forceinline__ T* in_block(T* p, int rank) {
  uint64_t a;
  asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(a);
}

template <int MAXS>
__global__ void __launch_bounds__(kSelThreads)
    select_kernel(const __grid_constant__ SelectParams<MAXS> p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ SelSmem S;
  const int blocks = p.blocks;
  const int rank = blocks > 1 ? (int)(blockIdx.x % (unsigned)blocks) : 0;
  const int row_id = blocks > 1 ? (int)(blockIdx.x / (unsigned)blocks) : (int)blockIdx.x;
  const int b = row_id / p.hkv, j = row_id - b * p.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ng = p.seq[b].ng, gqa = p.q_group;
  int32_t* out = p.out + ((int64_t)b * p.hkv + j) * p.n_select;
  const int m = min(p.n_select, ng);
  const int slice = blocks > 1 ? (ng + blocks - 1) / blocks : ng;
  const int first = min(ng, rank * slice), n = min(ng, first + slice) - first;   // this block's groups
  // dynamic shared memory: staged codes, [gqa][32] rotated queries (4 channels
  // a lane), [gqa][32] their bytes (parts below and above zero), [ng] score
  // keys (the first block's; the others use it for their weights)
  uint8_t* stages = smem_raw;
  int4* turned = reinterpret_cast<int4*>(stages + (size_t)p.stages * p.stage_bytes);
  int2* q8 = reinterpret_cast<int2*>(turned + (size_t)gqa * 32);
  uint64_t* keys = reinterpret_cast<uint64_t*>(q8 + (size_t)gqa * 32);
  if (tid == 0) {
    for (int s = 0; s < kSelStages; ++s) mbar_init(&S.full[s], 1);
    S.n_cand = 0;
    S.abort_flag = 0;
    fence_mbar_init();
  }
  S.hist[tid] = 0;
  __syncthreads();
  // every block of the cluster runs before another one stores into it
  if (blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  grid_dependency_wait();      // q and the index are outputs of earlier kernels, `out` may be read by one
  allow_dependents();
  if (rank == 0)
    for (int i = m + tid; i < p.n_select; i += kSelThreads) out[i] = -1;
  if (ng <= p.n_select) {
    for (int i = tid; i < n; i += kSelThreads) out[first + i] = first + i;
    if (blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return;
  }

  const int64_t row = ((int64_t)p.seq[b].slot * p.hkv + j) * p.max_groups + first;
  const int chunks = (n + kSelChunk - 1) / kSelChunk;
  int issued = 0;                  // chunks requested (thread 0)
  auto request = [&](int c) {      // chunk c into its stage
    const int s = c % p.stages;
    issued = c + 1;
    if (p.fault && blockIdx.x == 0 && c == 0) return;
    const uint32_t bytes = (uint32_t)min(kSelChunk, n - c * kSelChunk) * 256;
    mbar_arrive_expect_tx(&S.full[s], bytes);
    bulk_g2s(stages + (size_t)s * p.stage_bytes, p.codes + (row + c * kSelChunk) * 32, bytes, &S.full[s]);
  };
  if (tid == 0)
    for (int c = 0; c < min(chunks, p.stages); ++c) request(c);

  // ---- the queries in 8 bits, one step size for the heads of the KV head
  const uint16_t* q = p.q + ((int64_t)b * p.hq + (int64_t)j * gqa) * kHeadDim;
  auto load_q = [&](int h, float* f) {
    const uint2 raw = *reinterpret_cast<const uint2*>(q + h * kHeadDim + 4 * lane);
    f[0] = finite_or_zero(bf16_lo(raw.x));
    f[1] = finite_or_zero(bf16_hi(raw.x));
    f[2] = finite_or_zero(bf16_lo(raw.y));
    f[3] = finite_or_zero(bf16_hi(raw.y));
  };
  auto block_max = [&](uint32_t v, uint32_t* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    uint32_t r = red[0];
#pragma unroll
    for (int i = 1; i < kSelWarps; ++i) r = max(r, red[i]);
    return r;
  };
  uint32_t top = 0;
  for (int h = warp; h < gqa; h += kSelWarps) {
    float f[4];
    load_q(h, f);
    top = max(top, __float_as_uint(fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])))));
  }
  // this block's weights, in place of its keys (block 0) or at the front
  for (int i = tid; i < n; i += kSelThreads) keys[i] = reinterpret_cast<const uint64_t*>(p.weights)[row + i];
  top = block_max(top, S.red[0]);
  const float up = exp2i(22 - max((int)(top >> 23) - 126, kIdxMinExp));
  uint32_t big = 0;
  for (int h = warp; h < gqa; h += kSelWarps) {
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
  big = block_max(big, S.red[1]);
  int shift = max(0, 25 - __clz((int)big));      // big < 2^(shift + 7)
  if (big > (127u << shift)) ++shift;
  const int round = (1 << shift) >> 1;
  for (int h = warp; h < gqa; h += kSelWarps) {
    const int4 t = turned[h * 32 + lane];
    const int v[4] = {(t.x + round) >> shift, (t.y + round) >> shift, (t.z + round) >> shift, (t.w + round) >> shift};
    uint32_t pos = 0, neg = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pos |= (uint32_t)(max(v[i], 0) & 0xff) << (8 * i);
      neg |= (uint32_t)(min(v[i], 0) & 0xff) << (8 * i);
    }
    q8[h * 32 + lane] = make_int2((int)neg, (int)pos);
  }
  __syncthreads();

  // ---- scores: four lanes per group, lane part `part` takes the 16-byte
  // pieces part + 4 k (channels 8 (part + 4 k) .. + 7)
  const int part = lane & 3;
  const int4* q8v = reinterpret_cast<const int4*>(q8);     // [gqa][16 pieces]
  uint64_t* dst = rank == 0 ? keys : in_block(keys, 0);
  if (blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  uint32_t hmin = ~0u, hmax = 0;      // upper words of the smallest and the largest scored key
  int4 qr[kSelHeads][4];
  auto load_heads = [&](int h0) {
#pragma unroll
    for (int h = 0; h < kSelHeads; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        qr[h][k] = q8v[min(h0 + h, gqa - 1) * 16 + part + 4 * k];    // (a head twice changes no maximum)
  };
  load_heads(0);
  for (int c = 0; c < chunks; ++c) {
    const int s = c % p.stages;
    mbar_wait_bounded(&S.full[s], (uint32_t)((c / p.stages) & 1), &S.abort_flag, p.err_word, p.spin_limit);
    const int4* codes = reinterpret_cast<const int4*>(stages + (size_t)s * p.stage_bytes);
    const int here = min(kSelChunk, n - c * kSelChunk);
    // batches of 8 groups, warp by warp: t 8 + warp; lane `part` then makes the
    // key of its group of batch `part`
    int best = INT32_MIN;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int g0 = (t * kSelWarps + warp) * 8;
      if (g0 >= here) break;
      const int gl = g0 + (lane >> 2);    // behind the last group: whatever the stage holds, not used
      int4 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = codes[gl * 16 + part + 4 * k];
      int top_s = INT32_MIN;
      for (int h0 = 0; h0 < gqa; h0 += kSelHeads) {
        if (gqa > kSelHeads) load_heads(h0);
#pragma unroll
        for (int h = 0; h < kSelHeads; ++h) {
          int a = 0, d = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            a = __dp4a(w[k].x, qr[h][k].x, a);
            d = __dp4a(w[k].y, qr[h][k].y, d);
            a = __dp4a(w[k].z, qr[h][k].z, a);
            d = __dp4a(w[k].w, qr[h][k].w, d);
          }
          a += d;
          a += __shfl_xor_sync(0xffffffffu, a, 1);
          a += __shfl_xor_sync(0xffffffffu, a, 2);
          top_s = max(top_s, a);
        }
      }
      if (part == t) best = top_s;
    }
    const int gl = (part * kSelWarps + warp) * 8 + (lane >> 2);
    if (gl < here) {
      const int i = c * kSelChunk + gl, g = first + i;
      const float2 wt = *reinterpret_cast<const float2*>(&keys[i]);
      const bool kept = g < p.keep_first || g >= ng - p.keep_last;
      const uint64_t key = kept ? ~0ull : score_key(best, best >= 0 ? wt.x : wt.y);
      dst[g] = key;
      if (!kept) {
        hmin = min(hmin, (uint32_t)(key >> 32));
        hmax = max(hmax, (uint32_t)(key >> 32));
      }
    }
    if (c + p.stages < chunks) {
      __syncthreads();          // everyone is done with the stage
      if (tid == 0 && !S.abort_flag) request(c + p.stages);
    }
  }
  if (S.abort_flag && tid == 0) {
    // a wait gave up and nothing was requested since: wait (bounded) for the
    // copies that may still be in flight, the last of each stage
    for (int c = max(0, issued - p.stages); c < issued; ++c)
      for (uint32_t i = 0; i < p.spin_limit; ++i)
        if (mbar_try_wait(&S.full[c % p.stages], (uint32_t)((c / p.stages) & 1))) break;
  }
  if (blocks > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;      // nothing reads this block's shared memory
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int i = n + tid; i < ng; i += kSelThreads) {
      const uint64_t k = keys[i];
      if (k != ~0ull) {
        hmin = min(hmin, (uint32_t)(k >> 32));
        hmax = max(hmax, (uint32_t)(k >> 32));
      }
    }
  }
  hmin = __reduce_min_sync(0xffffffffu, hmin);
  hmax = __reduce_max_sync(0xffffffffu, hmax);
  if (lane == 0) {
    S.red[2][warp] = hmin;
    S.red[3][warp] = hmax;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) {
    hmin = min(hmin, S.red[2][i]);
    hmax = max(hmax, S.red[3][i]);
  }

  // ---- the m-th largest key, 8 bits at a time from the first bit in which
  // the scored keys' upper words differ; kept groups are above every one of them
  const int forced = min(ng, p.keep_first) + min(max(ng - p.keep_first, 0), p.keep_last);
  int need = m - forced;                   // still to choose among the scored groups with `prefix`
  int bits = 64 - __clz((int)(hmin ^ hmax));      // undecided low bits, at least 32
  uint64_t prefix = bits < 64 ? (uint64_t)hmin >> (bits - 32) : 0;       // the bits above them
  int inbin = INT32_MAX;                   // scored groups with the prefix, once counted
  auto has_prefix = [&](uint64_t k) { return k != ~0ull && (bits == 64 || (k >> bits) == prefix); };
  while (bits > 0 && need > 0 && need != inbin && inbin > kSelRank) {
    const int d = min(bits, 8), low = bits - d;
    for (int i = tid; i < ng; i += kSelThreads) {
      const uint64_t k = keys[i];
      if (has_prefix(k)) atomicAdd(&S.hist[(uint32_t)(k >> low) & ((1u << d) - 1)], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l owns digits 255 - 8 l .. 248 - 8 l, the largest first
      const uint4 x = reinterpret_cast<const uint4*>(S.hist)[2 * (31 - lane) + 1];
      const uint4 y = reinterpret_cast<const uint4*>(S.hist)[2 * (31 - lane)];
      const uint32_t c[8] = {x.w, x.z, x.y, x.x, y.w, y.z, y.y, y.x};
      const uint32_t sum = x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w;
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t lower = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += lower;
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
    inbin = (int)S.inbin;
    prefix = (prefix << d) | S.digit;
    bits = low;
    S.hist[tid] = 0;
    __syncthreads();
  }
  // chosen: keys whose top bits are above the prefix; of those equal to it
  // all, or the `need` first by (key, group): where at most kSelRank share the
  // prefix they are ranked; where every bit is decided they are equal
  uint64_t limit_key = 0;       // the last chosen (key, group) of the ranked ones
  int limit_group = INT32_MAX;
  bool ranked = false;
  if (need == inbin) {
    need = INT32_MAX;
  } else if (bits > 0 && need > 0) {
    ranked = true;
    for (int i = tid; i < ng; i += kSelThreads) {
      const uint64_t k = keys[i];
      if (has_prefix(k)) {
        const uint32_t at = atomicAdd(&S.n_cand, 1u);
        if (at < (uint32_t)kSelRank) {
          S.cand[at] = k;
          S.cand_group[at] = i;
        }
      }
    }
    __syncthreads();
    if (warp == 0) {
      const bool on = lane < inbin;
      const uint64_t k = on ? S.cand[lane] : 0;
      const int g = on ? S.cand_group[lane] : INT32_MAX;
      int before = 0;
      for (int i = 0; i < inbin; ++i) {
        const uint64_t ki = S.cand[i];
        before += ki > k || (ki == k && S.cand_group[i] < g);
      }
      if (on && before == need - 1) {
        S.limit_key = k;
        S.limit_group = g;
      }
    }
    __syncthreads();
    limit_key = S.limit_key;
    limit_group = S.limit_group;
  }

  // ---- the chosen groups in ascending order: `above` are chosen, of those
  // `at` the limit (equal keys, or the whole bin) the first `need`
  int done2 = 0, done1 = 0;
  for (int i0 = 0, turn = 0; i0 < ng; i0 += kSelThreads, turn ^= 1) {
    const int i = i0 + tid;
    bool above = false, at = false;
    if (i < ng) {
      const uint64_t k = keys[i];
      const uint64_t t = bits < 64 ? k >> bits : 0;
      above = k == ~0ull || t > prefix;
      if (!above && t == prefix) {
        if (ranked) above = k > limit_key || (k == limit_key && i <= limit_group);
        else at = true;
      }
    }
    const uint32_t b2 = __ballot_sync(0xffffffffu, above), b1 = __ballot_sync(0xffffffffu, at);
    if (lane == 0) {
      S.cnt[turn][0][warp] = __popc(b2);
      S.cnt[turn][1][warp] = __popc(b1);
    }
    __syncthreads();
    int n2 = done2, n1 = done1;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      const int x = S.cnt[turn][0][w], y = S.cnt[turn][1][w];
      if (w < warp) {
        n2 += x;
        n1 += y;
      }
      done2 += x;
      done1 += y;
    }
    const uint32_t below = (1u << lane) - 1;
    n2 += __popc(b2 & below);
    n1 += __popc(b1 & below);
    if (above || (at && n1 < need)) out[n2 + min(n1, need)] = i;
  }
}

template <int MAXS, bool M16>
cudaError_t launch_index_t(const IndexParams<MAXS>& p, const uint8_t* arena, int groups, cudaStream_t stream) {
  constexpr int per = kIdxThreads / 32;
  return launch_dependent(index_kernel<MAXS, M16>, dim3((groups + per - 1) / per, p.hkv, p.n_seqs), dim3(kIdxThreads),
                          0, stream, 1, p, arena);
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

template <int MAXS>
cudaError_t launch_select(const SelectParams<MAXS>& params, int sms, cudaStream_t stream) {
  SelectParams<MAXS> p = params;
  int groups = 0;
  for (int i = 0; i < p.n_seqs; ++i) groups = std::max(groups, p.seq[i].ng);
  if (groups <= p.n_select) groups = 0;
  const int rows = p.n_seqs * p.hkv;
  // blocks of a row: more while each keeps at least 64 groups and the grid
  // stays within two blocks per SM
  int blocks = 1;
  while (blocks < kSelMaxBlocks && groups >= 128 * blocks && (int64_t)rows * blocks <= sms) blocks *= 2;
  const int slice = (groups + blocks - 1) / blocks, chunks = (slice + kSelChunk - 1) / kSelChunk;
  p.blocks = blocks;
  // (whole batches: lanes behind the last group read the stage too)
  p.stage_bytes = std::max(8, std::min((slice + 7) & ~7, kSelChunk)) * 256;
  const auto smem = [&](int stages) {
    return (size_t)stages * p.stage_bytes + (size_t)p.q_group * 32 * (sizeof(int4) + sizeof(int2)) +
           (size_t)groups * sizeof(uint64_t);
  };
  static_assert(kSelChunk * 256 + kSelectMaxHeads * 32 * 24 + kSelectMaxGroups * 8 <= kSelectMaxSmem,
                "the largest selection fits with one stage");
  p.stages = chunks < 2 || smem(kSelStages) > (size_t)kSelectMaxSmem ? 1 : kSelStages;
  static bool attr_done[64] = {};
  cudaError_t e = ensure_smem_attr(select_kernel<MAXS>, kSelectMaxSmem, attr_done);
  if (e != cudaSuccess) return e;
  return launch_dependent(select_kernel<MAXS>, dim3((unsigned)(rows * blocks)), dim3(kSelThreads), smem(p.stages),
                          stream, (unsigned)blocks, p);
}

#define OSCAR_INSTANTIATE(N)                                                                                  \
  template cudaError_t launch_index<N>(const IndexParams<N>&, const uint8_t*, bool, cudaStream_t);            \
  template cudaError_t launch_select<N>(const SelectParams<N>&, int, cudaStream_t);
OSCAR_INSTANTIATE(kSelectSeqsSmall)
OSCAR_INSTANTIATE(kDecodeSeqsLarge)
#undef OSCAR_INSTANTIATE

}  // namespace oscar
