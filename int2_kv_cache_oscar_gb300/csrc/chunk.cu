// Attention within a new chunk (sm_103a tcgen05): packed documents of bf16
// queries, keys and values; a token attends to the keys of its own document up
// to itself, or up to the document's prefix where that reaches further:
//   x_t = scale q . k_t,  x_t = cap tanh(x_t / cap),  x_t -= slope |i - t|,
//   o = sum exp(x_t) v_t / sum exp(x_t),  t < max(i + 1, prefix),
// and is merged with the row that it got over what precedes the chunk.
//
// A CTA takes up to two tiles of 128 (token, query head) rows of one document
// and KV head (row = token * gqa + head: the heads of a group share every key
// tile, and a causal tile's diagonal is 128 / gqa tokens wide), and walks over
// the document's keys 128 at a time.  12 warps:
//   * warps 0-3 and 4-7: softmax of the two row tiles, thread = row.  Scores
//     are read from TMEM once, kept in registers, and P (bf16) is written back
//     over them as the A operand of P.V.  The output accumulator stays in TMEM
//     and is rescaled only when a row's maximum grows by more than 8 (log2
//     units); by then its last P.V is done, since the scores of a step are
//     issued behind the P.V of the step before;
//   * warp 8: one thread issues every tcgen05.mma.  S = Q K^T and O += P V of
//     the two tiles alternate, so that one tile's products run while the other
//     tile's softmax does;
//   * warp 9: one thread loads key and value tiles by TMA (128-byte swizzle)
//     into a ring of five 32 KB slots;
//   * warps 10, 11: look through the value rows of tiles with hidden keys.  A
//     hidden key has p = 0, but 0 times an infinite or NaN value would still
//     spoil every row of the tile: such value rows are cleared in shared
//     memory, and rows that do see them add them on the CUDA cores.
// Bound: 4 * 128 flops per visible (row, key) on the tensor cores for long
// documents; launch and pipeline latency for short ones.
// P is rounded to bf16 (the type of V: the tensor cores take both operands of a
// product in one type), relative 2^-9 a weight; row sums are of the float32
// weights, scores and outputs accumulate in float32.
#include <cstddef>

#include "common.cuh"
#include "launch.h"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace oscar {
namespace {

constexpr int kChRows = 128;                  // rows of a tile (M)
constexpr int kChKeys = 128;                  // keys of a step (N)
constexpr int kChThreads = 12 * 32;
constexpr int kChSlots = 5;
constexpr int kBox = 64 * 2 * 128;            // 128 rows of 64 channels
constexpr int kTileBytes = 2 * kBox;
// TMEM columns of tile i: scores (then P in the first 64), output accumulator
__host__ __device__ constexpr uint32_t col_s(int i) { return 128u * i; }
__host__ __device__ constexpr uint32_t col_o(int i) { return 256u + 128u * i; }
constexpr uint32_t kTmemCols = 512;
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;   // registers of a thread: warps 0-7, warps 8-11
constexpr float kGrowth = 8.0f;               // see above
constexpr float kLn2 = 0.69314718055994530942f;

struct ChunkSmem {
  alignas(1024) uint8_t q[2][kTileBytes];
  alignas(1024) uint8_t ring[kChSlots][kTileBytes];
  alignas(8) uint64_t full[kChSlots];
  uint64_t empty[kChSlots];
  uint64_t s_full[2];         // scores of a tile's step are done (and the P.V before them)
  uint64_t p_ready[2][2];     // P of the step's first and second 64 keys is in TMEM
  uint64_t o_done[2];
  uint64_t v_clean[4];        // value rows of a step with hidden keys have been looked through
  uint64_t drained;           // everything issued is done (only where a wait gave up)
  uint32_t bad[4][4];         // value rows cleared there, a bit each
  uint32_t issued[kChSlots];  // uses of each slot requested so far
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(ChunkSmem) + 1024 <= 232448, "one CTA per SM");

// 128-byte-swizzled shared-memory matrix descriptor: start, leading and stride byte offsets.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor: float32 accumulator, bf16 operands, M = N = 128, A
// K-major, B K-major (keys) or N-major (values).
constexpr uint32_t kIdescQK = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint32_t tld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return r;
}

// Byte offset of 16-byte chunk c (of 16) of row r in a tile of two swizzled boxes.
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (uint32_t)((c >> 3) * kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Ring position of key and value tiles: K0, K1, V0, K2, V1, ...
__device__ __forceinline__ int key_pos(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int value_pos(int j, int steps) { return j == steps - 1 ? 2 * steps - 1 : 2 * j + 2; }

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a CTA works on.
struct ChunkTile {
  int row0, len, prefix;     // the document: first token, tokens, prefix
  int head;                  // KV head
  int first_row;             // of the CTA, within the document's rows
  int rows;                  // of the document
  int steps[2];              // key steps of each tile (0: no rows)
  int plain[2];              // leading steps in which its rows see every key
};

template <int MAXS>
__device__ __forceinline__ ChunkTile locate(const ChunkParams<MAXS>& p) {
  ChunkTile t;
  const int u = (int)(blockIdx.x / (unsigned)p.hkv);
  t.head = (int)(blockIdx.x - (unsigned)u * (unsigned)p.hkv);
  int lo = 0, hi = p.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.seq[mid].tbase <= u) lo = mid; else hi = mid - 1;
  }
  const ChunkSeq s = p.seq[lo];
  t.row0 = s.row0;
  t.len = s.len;
  t.prefix = s.prefix;
  t.rows = s.len * p.gqa;
  const int tiles = (t.rows + p.cta_rows - 1) / p.cta_rows;
  t.first_row = (tiles - 1 - (u - s.tbase)) * p.cta_rows;     // the longest ones first
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r0 = t.first_row + i * kChRows;
    const bool live = i * kChRows < p.cta_rows && r0 < t.rows;
    const int first = r0 / p.gqa, last = (min(r0 + kChRows, t.rows) - 1) / p.gqa;
    const int lim = min(max(last + 1, t.prefix), t.len);
    t.steps[i] = live ? (lim + kChKeys - 1) / kChKeys : 0;
    t.plain[i] = live ? min(max(first + 1, t.prefix), t.len) / kChKeys : t.steps[0];
  }
  return t;
}

// Rows of the warp add the value rows that were cleared (bits of `bad`, keys k0
// .. + 127 of the document) times their weights, read from P in TMEM, to the
// output accumulator (started from zero where `fresh`).
__device__ __noinline__ void add_cleared(uint32_t t_p, uint32_t t_o, const uint32_t* bad, int visible, bool fresh,
                                         const uint16_t* v, int64_t v_token) {
  for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
    uint32_t o[32];
    if (fresh) {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0u;
    } else {
      tld32(t_o + c0, o);
      tld_wait();
    }
    for (int t = 0; t < kChKeys; ++t) {
      if (!((bad[t >> 5] >> (t & 31)) & 1u)) continue;
      const uint32_t pair = tld1(t_p + t / 2);
      tld_wait();
      if (t < visible) {
        const float w = (t & 1) ? bf16_hi(pair) : bf16_lo(pair);
        const uint16_t* row = v + (int64_t)t * v_token + c0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          o[i] = __float_as_uint(fmaf(w, __uint_as_float((uint32_t)row[i] << 16), __uint_as_float(o[i])));
      }
      __syncwarp();
    }
    tst32(t_o + c0, o);
    tst_wait();
  }
}

template <int MAXS, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kChThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkParams<MAXS> p, const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  ChunkSmem& S = *reinterpret_cast<ChunkSmem*>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const ChunkTile T = locate(p);
  const int steps = max(T.steps[0], T.steps[1]);
  const int plain = min(T.plain[0], T.plain[1]);      // steps before this one hide no key from any row

  // the n-th load of the ring: K0, K1, V0, K2, V1, ...
  auto load = [&](int n) {
    const int s = n % kChSlots;
    const bool val = n == 2 * steps - 1 || (n > 0 && (n & 1) == 0);
    const int j = n == 2 * steps - 1 ? steps - 1 : val ? (n - 2) / 2 : (n + 1) / 2;
    const CUtensorMap* m = val ? &tmv : &tmk;
    mbar_arrive_expect_tx(&S.full[s], kTileBytes);
    tma_load_3d(S.ring[s], m, 0, T.head, T.row0 + j * kChKeys, &S.full[s]);
    tma_load_3d(S.ring[s] + kBox, m, 64, T.head, T.row0 + j * kChKeys, &S.full[s]);
    reinterpret_cast<volatile uint32_t*>(S.issued)[s] = (uint32_t)(n / kChSlots) + 1;
  };
  const int early = min(kChSlots, 2 * steps);     // loads that no slot has to be waited for

  if (warp == 9 && lane == 0) {
    for (int i = 0; i < kChSlots; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
      S.issued[i] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_ready[i][0], 4);
      mbar_init(&S.p_ready[i][1], 4);
      mbar_init(&S.o_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&S.v_clean[i], 2);
    mbar_init(&S.drained, 1);
    S.abort_flag = 0;
    fence_mbar_init();
    grid_dependency_wait();
    for (int n = 0; n < early; ++n) load(n);
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  grid_dependency_wait();
  allow_dependents();
  if (warp < 8) {
    // the queries of the rows, 16 lanes a row (rows behind the last one repeat
    // it), all of a thread's loads in flight at once
    const int i = warp >> 2;
    if (T.steps[i] > 0) {
      const int first = T.first_row + i * kChRows, t0 = first / p.gqa, rest = first - t0 * p.gqa;
      const int c = tid & 15, r0 = (tid & 127) >> 4;
      const float inv = 1.0f / (float)p.gqa;
      const uint16_t* base = p.q + (int64_t)(T.row0 + t0) * p.q_token + (int64_t)(T.head * p.gqa) * p.q_head + 8 * c;
      uint4 u[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int at = rest + min(r0 + 8 * x, T.rows - 1 - first);
        // at / gqa: below 2^17, where the half keeps the product off whole numbers
        const int tok = (int)(((float)at + 0.5f) * inv), h = at - tok * p.gqa;
        u[x] = *reinterpret_cast<const uint4*>(base + (int64_t)tok * p.q_token + (int64_t)h * p.q_head);
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) *reinterpret_cast<uint4*>(S.q[i] + tile_off(r0 + 8 * x, c)) = u[x];
      async_fence();
    }
  }
  tfence_before();
  __syncthreads();
  tfence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---------------------------------------------------------- MMA issuer
      const uint64_t dq[2] = {desc128(smem_u32(S.q[0]), 16, 1024), desc128(smem_u32(S.q[1]), 16, 1024)};
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, &S.abort_flag, nullptr));
        tfence_after();
        return ok;
      };
      // scores of tile i from the keys in a slot; `freed`: the slot's last use
      auto scores = [&](int i, int slot, bool freed) {
        const uint64_t dk = desc128(smem_u32(S.ring[slot]), 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint64_t off = (uint64_t)(((ks >> 2) * kBox + (ks & 3) * 32) >> 4);
            mma_ss(tmem + col_s(i), dq[i] + off, dk + off, kIdescQK, ks > 0);
          }
          mma_commit(&S.s_full[i]);
          if (freed) mma_commit(&S.empty[slot]);
        }
        __syncwarp();
      };
      bool ok = wait(&S.full[0], 0);
      if (ok) {
        if (T.steps[0] > 0) scores(0, 0, T.steps[1] == 0);
        if (T.steps[1] > 0) scores(1, 0, true);
      }
      for (int j = 0; ok && j < steps; ++j) {
        const int kn = key_pos(j + 1), vn = value_pos(j, steps);
        const int vs = vn % kChSlots, ksl = kn % kChSlots;
        const bool more = j + 1 < steps;
        const bool hidden = j >= plain;
        ok = wait(&S.full[vs], (vn / kChSlots) & 1);
        if (ok && more) ok = wait(&S.full[ksl], (kn / kChSlots) & 1);
        bool keep = j > 0;
        if (ok && hidden) {
          ok = wait(&S.v_clean[j & 3], ((j - plain) >> 2) & 1);
          keep = keep || (S.bad[j & 3][0] | S.bad[j & 3][1] | S.bad[j & 3][2] | S.bad[j & 3][3]) != 0u;
        }
        // values are N-major: 64 channels a box, 16 keys a k-step
        const uint64_t dv = desc128(smem_u32(S.ring[vs]), kBox, 1024);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!ok || j >= T.steps[i]) continue;
          const bool last = i == 1 || j >= T.steps[1];       // the step's last tile
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && wait(&S.p_ready[i][half], j & 1);
            if (!ok) continue;
            if (elect_one()) {
#pragma unroll
              for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                mma_ts(tmem + col_o(i), tmem + col_s(i) + 8 * ks, dv + (uint64_t)((ks * 2048) >> 4), kIdescPV, keep || ks > 0);
              if (half == 1) {
                if (last) mma_commit(&S.empty[vs]);
                if (j + 1 >= T.steps[i]) mma_commit(&S.o_done[i]);
              }
            }
            __syncwarp();
          }
          if (ok && j + 1 < T.steps[i]) scores(i, ksl, last);
        }
        // (a tile that ends before the other: the other one's scores free the keys)
      }
      if (!ok) {
        // gave up: what has been issued completes before TMEM is freed (bounded)
        if (elect_one()) mma_commit(&S.drained);
        for (uint32_t n = 0; n < kSpinLimit; ++n)
          if (mbar_try_wait(&S.drained, 0)) break;
      }
    } else if (warp == 9 && lane == 0) {
      // -------------------------------------------------------------- loads
      int n = early;
      for (; n < 2 * steps; ++n) {
        if (!mbar_wait_bounded(&S.empty[n % kChSlots], ((n / kChSlots) - 1) & 1, &S.abort_flag, nullptr)) break;
        load(n);
      }
      if (S.abort_flag) {
        // gave up: the copies in flight get their time (bounded)
        for (int x = max(0, n - kChSlots); x < n; ++x)
          for (uint32_t i = 0; i < kSpinLimit; ++i)
            if (mbar_try_wait(&S.full[x % kChSlots], (x / kChSlots) & 1)) break;
      }
    } else if (warp >= 10) {
      // ----------------------------------------- value rows of partial steps
      const int w = warp - 10;
      for (int j = plain; j < steps; ++j) {
        const int vn = value_pos(j, steps), vs = vn % kChSlots;
        // (these warps do not follow a slot's earlier uses: its phase is waited for once it exists)
        const bool ok = wait_issued(&S.issued[vs], (uint32_t)(vn / kChSlots), &S.abort_flag, nullptr) &&
                        mbar_wait_bounded(&S.full[vs], (vn / kChSlots) & 1, &S.abort_flag, nullptr);
        if (!__all_sync(0xffffffffu, ok)) break;
        bool cleared = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 64 * w + 32 * i + lane;
          uint32_t any = 0u;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint4 u = *reinterpret_cast<const uint4*>(S.ring[vs] + tile_off(r, c));
            // an exponent of all ones carries into bit 15 of its half
            any |= (((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
                    ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u)) &
                   0x80008000u;
          }
          const uint32_t bits = __ballot_sync(0xffffffffu, any != 0u);
          if (lane == 0) S.bad[j & 3][2 * w + i] = bits;
          if (any != 0u) {
#pragma unroll 1
            for (int c = 0; c < 16; ++c) *reinterpret_cast<uint4*>(S.ring[vs] + tile_off(r, c)) = make_uint4(0, 0, 0, 0);
          }
          cleared = cleared || bits != 0u;
        }
        if (cleared) async_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.v_clean[j & 3]);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2;
    const int my_steps = i ? T.steps[1] : T.steps[0], my_plain = i ? T.plain[1] : T.plain[0];
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + col_s(i) + lanes, tO = tmem + col_o(i) + lanes;
    const int r = T.first_row + i * kChRows + 32 * (warp & 3) + lane;
    const bool live = r < T.rows;
    const int row = min(r, T.rows - 1);
    const int tok = row / p.gqa, h = T.head * p.gqa + row - tok * p.gqa;
    const int limit = min(max(tok + 1, T.prefix), T.len);     // visible keys: [0, limit)
    const float slope2 = BIAS ? p.slopes[h] * 1.4426950408889634f : 0.0f;
    // scores to log2 units: a factor here, the rule's arithmetic otherwise
    const float sl = CAP || BIAS ? 1.0f : p.scale_log2;
    float m = -INFINITY, l = 0.0f;     // running maximum (before sl) and sum
    bool ok = true;
    for (int j = 0; j < my_steps; ++j) {
      ok = mbar_wait_bounded(&S.s_full[i], j & 1, &S.abort_flag, nullptr);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tfence_after();
      float s[kChKeys];
#pragma unroll
      for (int c = 0; c < kChKeys; c += 32) tld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&s[c]));
      tld_wait();
      if constexpr (CAP) {
        // cap tanh(x / cap) = cap - 2 cap / (1 + exp(2 x / cap)), in log2 units
#pragma unroll
        for (int c = 0; c < kChKeys; ++c)
          s[c] = fmaf(p.cap_out, rcp_approx(1.0f + tc_exp2(s[c] * p.cap_in)), p.cap_log2);
      }
      if constexpr (BIAS) {
        const float d0 = (float)(j * kChKeys - tok);
#pragma unroll
        for (int c = 0; c < kChKeys; ++c)
          s[c] = fmaf(-slope2, fabsf(d0 + (float)c), CAP ? s[c] : s[c] * p.scale_log2);
      }
      if (j >= my_plain) {
        const int vis = limit - j * kChKeys;
#pragma unroll
        for (int c = 0; c < kChKeys; ++c) s[c] = c < vis ? s[c] : -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < kChKeys; c += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (c + 4 + e < kChKeys)
            asm("max.f32 %0, %0, %1, %2;" : "+f"(mx[e]) : "f"(s[c + e]), "f"(s[c + 4 + e]));
          else
            mx[e] = fmaxf(mx[e], s[c + e]);
        }
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      // a larger maximum takes effect where it is far above the one in use
      const bool grow = (top - m) * sl > kGrowth || m == -INFINITY;
      const float m_new = grow ? fmaxf(m, top) : m;
      if (__any_sync(0xffffffffu, grow && j > 0)) {
        const float f = m_new == -INFINITY ? 1.0f : tc_exp2((m - m_new) * sl);
        l *= f;
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 16) {
          uint32_t o[16];
          tld16(tO + c, o);
          tld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tst16(tO + c, o);
        }
        tst_wait();
      }
      m = m_new;
      const float base = m == -INFINITY ? 0.0f : -m * sl;
      const float2 sl2 = make_float2(sl, sl), base2 = make_float2(base, base);
      float2 sum0 = make_float2(0.0f, 0.0f), sum1 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int c = 64 * half + 2 * e;
          const float2 a = __ffma2_rn(make_float2(s[c], s[c + 1]), sl2, base2);
          const float2 b = __ffma2_rn(make_float2(s[c + 2], s[c + 3]), sl2, base2);
          const float2 pa = make_float2(tc_exp2(a.x), tc_exp2(a.y)), pb = make_float2(tc_exp2(b.x), tc_exp2(b.y));
          sum0 = __fadd2_rn(sum0, pa);
          sum1 = __fadd2_rn(sum1, pb);
          pk[e] = pack_bf16x2(pa.x, pa.y);
          pk[e + 1] = pack_bf16x2(pb.x, pb.y);
        }
        tst32(tS + 32 * half, pk);
        if (half == 0 && j < plain) {
          tst_wait();
          tfence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.p_ready[i][0]);
        }
      }
      tst_wait();
      if (j >= plain) {
        // hidden keys in this step: values that had to be cleared are added here
        ok = mbar_wait_bounded(&S.v_clean[j & 3], ((j - plain) >> 2) & 1, &S.abort_flag, nullptr);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t* bad = S.bad[j & 3];
        if ((bad[0] | bad[1] | bad[2] | bad[3]) != 0u)
          add_cleared(tS, tO, bad, limit - j * kChKeys, j == 0,
                      p.v + (int64_t)(T.row0 + j * kChKeys) * p.v_token + (int64_t)T.head * p.v_head, p.v_token);
        tfence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_ready[i][0]);
      } else {
        tfence_before();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&S.p_ready[i][1]);
      l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
    }
    if (my_steps > 0) {
      // o / l, merged with the row over what precedes the chunk.  Rows pass
      // through the tile's query memory (free by now), a warp's 32 rows by itself:
      // 16 lanes a row in global memory, a thread a row in between.
      uint8_t* rows = S.q[i];
      const int w0 = T.first_row + i * kChRows + 32 * (warp & 3);     // the warp's first row
      const int t0 = w0 / p.gqa, rest = w0 - t0 * p.gqa, c = lane & 15, r0 = lane >> 4;
      const float inv = 1.0f / (float)p.gqa;
      const int64_t base = ((int64_t)(T.row0 + t0) * p.hq + T.head * p.gqa) * kHeadDim + 8 * c;
      // element of row w0 + r, chunk c
      auto place = [&](int r) {
        const int at = rest + r, tk = (int)(((float)at + 0.5f) * inv);
        return base + ((int64_t)tk * p.hq + (at - tk * p.gqa)) * kHeadDim;
      };
      const int64_t at = (int64_t)(T.row0 + tok) * p.hq + h;
      float before = -INFINITY;
      uint4 u[16];
      if (p.prior_lse != nullptr) {
        before = p.prior_lse[at];
#pragma unroll
        for (int x = 0; x < 16; ++x)
          u[x] = w0 + r0 + 2 * x < T.rows ? *reinterpret_cast<const uint4*>(p.prior_out + place(r0 + 2 * x))
                                          : make_uint4(0, 0, 0, 0);
      }
      if (ok) {
        ok = mbar_wait_bounded(&S.o_done[i], 0, &S.abort_flag, nullptr);
        ok = __all_sync(0xffffffffu, ok);
        tfence_after();
      }
      if (p.prior_lse != nullptr) {
#pragma unroll
        for (int x = 0; x < 16; ++x) *reinterpret_cast<uint4*>(rows + tile_off(32 * (warp & 3) + r0 + 2 * x, c)) = u[x];
        __syncwarp();
      }
      float lse = ok ? fmaf(m, sl * kLn2, logf(l)) : NAN;
      float fo = ok ? 1.0f / l : NAN, fp = 0.0f;
      if (before != -INFINITY) {
        const float top = fmaxf(lse, before);
        const float a = expf(lse - top), b = expf(before - top);
        fp = b / (a + b);
        fo *= a / (a + b);
        lse = top + logf(a + b);
      }
#pragma unroll 1
      for (int c4 = 0; c4 < 16; c4 += 4) {
        uint32_t o[32];
        if (ok) {
          tld32(tO + 8 * c4, o);
          tld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0x7fc00000u;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4* mine = reinterpret_cast<uint4*>(rows + tile_off(32 * (warp & 3) + lane, c4 + e));
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[8 * e + k]) * fo;
          if (fp != 0.0f) {     // (also NaN)
            const uint4 b = *mine;
            x[0] = fmaf(bf16_lo(b.x), fp, x[0]);
            x[1] = fmaf(bf16_hi(b.x), fp, x[1]);
            x[2] = fmaf(bf16_lo(b.y), fp, x[2]);
            x[3] = fmaf(bf16_hi(b.y), fp, x[3]);
            x[4] = fmaf(bf16_lo(b.z), fp, x[4]);
            x[5] = fmaf(bf16_hi(b.z), fp, x[5]);
            x[6] = fmaf(bf16_lo(b.w), fp, x[6]);
            x[7] = fmaf(bf16_hi(b.w), fp, x[7]);
          }
          *mine = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                             pack_bf16x2(x[6], x[7]));
        }
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < 16; ++x)
        if (w0 + r0 + 2 * x < T.rows)
          *reinterpret_cast<uint4*>(p.out + place(r0 + 2 * x)) =
              *reinterpret_cast<const uint4*>(rows + tile_off(32 * (warp & 3) + r0 + 2 * x, c));
      if (live && p.lse != nullptr) p.lse[at] = lse;
    }
  }

  tfence_before();
  __syncthreads();
  if (warp == 8) {
    tfence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// Rows [token][head][128 channels] of bf16: box = 64 channels of one head, 128 tokens.
bool encode_chunk_map(CUtensorMap* map, const void* base, uint64_t tokens, uint64_t heads, uint64_t token_bytes,
                      uint64_t head_bytes) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {kHeadDim, heads, tokens};
  const cuuint64_t strides[2] = {head_bytes, token_bytes};
  const cuuint32_t box[3] = {64, 1, kChKeys};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MAXS, bool CAP, bool BIAS>
cudaError_t launch_chunk_t(const ChunkParams<MAXS>& p, const CUtensorMap& tmk, const CUtensorMap& tmv, unsigned grid,
                           cudaStream_t stream) {
  static bool attr_done[64] = {};
  const int smem = (int)sizeof(ChunkSmem) + 1024;
  cudaError_t e = ensure_smem_attr(chunk_kernel<MAXS, CAP, BIAS>, smem, attr_done);
  if (e != cudaSuccess) return e;
  // the warps' shares of the registers must fit in what the block is launched with
  static const int regs = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, chunk_kernel<MAXS, CAP, BIAS>) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs * kChThreads < 256 * kSoftmaxRegs + 128 * kOtherRegs) return cudaErrorInvalidConfiguration;
  return launch_dependent(chunk_kernel<MAXS, CAP, BIAS>, dim3(grid), dim3(kChThreads), (size_t)smem, stream, 1, p, tmk, tmv);
}

}  // namespace

template <int MAXS>
cudaError_t launch_chunk(ChunkParams<MAXS>& p, const uint16_t* k, int64_t k_token, int64_t k_head, int64_t tokens,
                         int sms, cudaStream_t stream) {
  CUtensorMap tmk, tmv;
  if (!encode_chunk_map(&tmk, k, tokens, p.hkv, 2 * k_token, 2 * k_head) ||
      !encode_chunk_map(&tmv, p.v, tokens, p.hkv, 2 * p.v_token, 2 * p.v_head))
    return cudaErrorInvalidValue;
  // two row tiles a CTA share its key tiles; one each while that leaves SMs without work
  int64_t tiles = 0;
  for (p.cta_rows = 2 * kChRows;; p.cta_rows = kChRows) {
    tiles = 0;
    for (int i = 0; i < p.n_seqs; ++i) {
      p.seq[i].tbase = (int32_t)tiles;
      tiles += ((int64_t)p.seq[i].len * p.gqa + p.cta_rows - 1) / p.cta_rows;
    }
    if (p.cta_rows == kChRows || tiles * p.hkv >= sms) break;
  }
  const unsigned grid = (unsigned)(tiles * p.hkv);
  const bool cap = p.cap_log2 != 0.0f, bias = p.slopes != nullptr;
  if (cap) return bias ? launch_chunk_t<MAXS, true, true>(p, tmk, tmv, grid, stream)
                       : launch_chunk_t<MAXS, true, false>(p, tmk, tmv, grid, stream);
  return bias ? launch_chunk_t<MAXS, false, true>(p, tmk, tmv, grid, stream)
              : launch_chunk_t<MAXS, false, false>(p, tmk, tmv, grid, stream);
}

template cudaError_t launch_chunk<kDecodeSeqsSmall>(ChunkParams<kDecodeSeqsSmall>&, const uint16_t*, int64_t, int64_t,
                                                    int64_t, int, cudaStream_t);
template cudaError_t launch_chunk<kDecodeSeqsLarge>(ChunkParams<kDecodeSeqsLarge>&, const uint16_t*, int64_t, int64_t,
                                                    int64_t, int, cudaStream_t);

}  // namespace oscar
