// Attention within a new chunk (sm_103a tcgen05): packed documents of bf16
// queries, keys and values; a token attends to the keys of its own document up
// to itself, or up to the document's prefix where that reaches further:
//   x_t = scale q . k_t,  x_t = cap tanh(x_t / cap),  x_t -= slope |i - t|,
//   o = sum exp(x_t) v_t / sum exp(x_t),  t < max(i + 1, prefix),
// and is merged with the row that it got over what precedes the chunk.
//
// A piece of work is up to two tiles of 128 (token, query head) rows of one
// document and KV head (row = token * gqa + head: the heads of a group share every
// key tile, and a causal tile's diagonal is 128 / gqa tokens wide) against the
// document's keys, 128 at a time.  A CTA an SM takes pieces from the list of all,
// the longest first, in rounds of alternating direction (piece k of CTA b of G: k G
// + b, or (k + 1) G - 1 - b): set-up is paid once, and the loads and first scores
// of the next piece run while this one's rows are written.  12 warps:
//   * warps 0-3 and 4-7: softmax of the two row tiles, thread = row.  Scores
//     are read from TMEM once, kept in registers, and P (bf16) is written back
//     over them as the A operand of P.V.  The output accumulator stays in TMEM
//     and is rescaled only when a row's maximum grows by more than 8 (log2
//     units); by then its last P.V is done, since the scores of a step are
//     issued behind the P.V of the step before;
//   * warp 8 issues every tcgen05.mma.  S = Q K^T and O += P V of the two tiles
//     alternate, so that one tile's products run while the other tile's softmax does;
//   * warp 9: one thread loads key and value tiles by TMA (128-byte swizzle) into a
//     ring of four 32 KB slots, and describes the pieces of work to the others.
//     Queries come by TMA too where 128 rows are whole tokens (gqa divides 128),
//     requested by the softmax warps once the last scores of a piece are there,
//     else by 16-byte copies (64 documents of 128 tokens 42 against 47 us);
//   * warps 10, 11: look through the value rows of tiles with hidden keys.  A
//     hidden key has p = 0, but 0 times an infinite or NaN value would still
//     spoil every row of the tile: such value rows are cleared in shared
//     memory, and rows that do see them add them on the CUDA cores.
// Bound: 4 * 128 flops per visible (row, key) on the tensor cores for long
// documents; launch and pipeline latency for short ones.  A step of 128 keys takes
// some 2,900 cycles for two tiles, 2,048 of them products: a tile's chain is 1,500 cycles
// of softmax, then the second half of its P.V and the next scores (768), and the way
// from one to the other and back (700): 8,192 tokens of 32 heads take 358 us, 1,530
// TFLOP/s.  A piece of a single step takes 9,000 cycles, most of them the softmax
// warps' own: 3,000 of softmax with a mask, 4,000 of output rows on their way out
// (64 bytes of a row at a time: 32 or 128 of them 2 to 6 % slower).  Tried when the
// former took 374 us, and slower: a second warpgroup a tile for half of the keys (533
// us: 104 registers a thread do not hold a half), pieces handed out by cluster launch
// control (407 us), a piece a CTA (379 us, and 78 against 57 for the 64 documents).
// P is rounded to bf16 (the type of V: the tensor cores take both operands of a
// product in one type), relative 2^-8 a weight; row sums are of the float32
// weights, scores and outputs accumulate in float32.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace oscar {
namespace {

constexpr int kChRows = 128;                  // rows of a tile (M)
constexpr int kChKeys = 128;                  // keys of a step (N)
constexpr int kChThreads = 12 * 32;
constexpr int kChSlots = 4;
constexpr int kWorkReaders = 11;              // warps that read a piece: issuer, two that look through values, softmax
constexpr int kStageRow = 64;                // bytes of a row that pass through shared memory at a time
constexpr int kBox = 64 * 2 * 128;            // 128 rows of 64 channels
constexpr int kTileBytes = 2 * kBox;
// TMEM columns of tile i: scores (then P in the first 64), output accumulator
__host__ __device__ constexpr uint32_t col_s(int i) { return 128u * i; }
__host__ __device__ constexpr uint32_t col_o(int i) { return 256u + 128u * i; }
constexpr uint32_t kTmemCols = 512;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;   // registers of a thread: warps 0-7, warps 8-11
constexpr float kGrowth = 8.0f;               // see above
constexpr float kFarBase = 0x1p20f;           // log2 units: a base beyond is not exact to 2^-4
constexpr float kCapSmall = 0.25f / 0.6f;     // a quarter of the cap, in units of 0.6 of it (see cap_small)
constexpr float kLn2 = 0.69314718055994530942f;

// cap tanh(x / cap) of a raw score, in log2 units: cap - 2 cap / (1 + exp(2 x /
// cap)), off by cap 2^-22 at most (`in` = 2 x / cap of a raw score of 1 in log2 units,
// `out` = -2 cap).
__device__ __forceinline__ float cap_far(float s, float in, float out, float cap) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s * in));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return fmaf(out, r, cap);
}

// The same within 0.6 of the cap, two scores: tanh(x) = x (1 + c1 x^2 + .. + c4 x^8),
// the smallest largest relative error over that range (2^-23.5), with the scale and
// the cap in the coefficients.
__device__ __forceinline__ float2 cap_near(float2 s, const float (&c)[5]) {
  const float2 y = __fmul2_rn(s, s);
  auto two = [](float v) { return make_float2(v, v); };
  float2 t = __ffma2_rn(two(c[4]), y, two(c[3]));
  t = __ffma2_rn(t, y, two(c[2]));
  t = __ffma2_rn(t, y, two(c[1]));
  return __fmul2_rn(s, __ffma2_rn(t, y, two(c[0])));
}

// The same within a quarter of the cap: two terms less, relative error 2^-21 (cap
// 2^-23).
template <typename P>
__device__ __forceinline__ float2 cap_small(float2 s, const P& p) {
  const float2 y = __fmul2_rn(s, s);
  auto two = [](float v) { return make_float2(v, v); };
  const float2 t = __ffma2_rn(two(p.cap_d[2]), y, two(p.cap_d[1]));
  return __fmul2_rn(s, __ffma2_rn(t, y, two(p.cap_d[0])));
}

// A piece of work.
struct ChunkTile {
  int row0, len, prefix;     // the document: first token, tokens, prefix
  int head;                  // KV head
  int first_row;             // of the piece, within the document's rows
  int rows;                  // of the document
  int steps[2];              // key steps of each tile (0: no rows)
  int plain[2];              // leading steps in which its rows see every key
  int there;                 // 0: no more work
};

struct ChunkSmem {
  alignas(1024) uint8_t q[2][kTileBytes];
  alignas(1024) uint8_t ring[kChSlots][kTileBytes];
  alignas(128) uint8_t stage[8][32 * kStageRow];   // of a softmax warp: channels of its rows on their way
  alignas(8) uint64_t full[kChSlots];
  uint64_t empty[kChSlots];
  uint64_t s_full[2];         // scores of a tile's step are done (and the P.V before them)
  uint64_t p_ready[2][2];     // P of the step's first and second 64 keys is in TMEM
  uint64_t o_done[2];
  uint64_t v_clean[4];        // value rows of a step with hidden keys have been looked through
  uint64_t q_ready[2];        // queries of a tile are in place
  uint64_t w_full[2], w_empty[2];   // pieces of work: described, read by every role
  uint64_t drained;           // everything issued is done (only where a wait gave up)
  uint32_t bad[4][4];         // value rows cleared there, a bit each
  ChunkTile work[2];
  uint32_t issued[kChSlots];  // uses of each slot requested so far
  uint32_t tmem_base;
  int abort_flag;
  int stopped;                // first piece of the CTA that a wait which gave up left out
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

// A wait that may take as long as the other roles need for a whole piece, whose length
// is the document's: bounded like the others, but by polls during which no tile was
// requested into the slot that `issued` counts.
template <typename Ready>
__device__ __forceinline__ bool wait_for_piece(Ready ready, const volatile uint32_t* issued, volatile int* abort_flag,
                                               uint32_t limit) {
  uint32_t seen = 0;
  for (uint32_t i = 0; i < limit; ++i) {
    if (ready()) return true;
    if (*abort_flag) return false;
    if (i % 64 == 63 && *issued != seen) {
      seen = *issued;
      i = 0;
    }
  }
  *abort_flag = 1;
  return false;
}

// Ring position of key and value tiles: K0, K1, V0, K2, V1, ...
__device__ __forceinline__ int key_pos(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int value_pos(int j, int steps) { return j == steps - 1 ? 2 * steps - 1 : 2 * j + 2; }

template <int MAXS>
__device__ __forceinline__ ChunkTile locate(const ChunkParams<MAXS>& p, int work) {
  ChunkTile t;
  t.there = 1;
  const int u = (int)((unsigned)work / (unsigned)p.hkv);
  t.head = work - u * p.hkv;
  int lo = 0, hi = p.n_seqs - 1, tile = -1;
  if (p.sorted) {
    lo = (int)(p.order[u] >> 22);
    tile = (int)(p.order[u] & 0x3fffffu);
  } else {
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.seq[mid].tbase <= u) lo = mid; else hi = mid - 1;
    }
  }
  const ChunkSeq s = p.seq[lo];
  t.row0 = s.row0;
  t.len = s.len;
  t.prefix = s.prefix;
  t.rows = s.len * p.gqa;
  const int tiles = (t.rows + p.cta_rows - 1) / p.cta_rows;
  if (tile < 0) tile = tiles - 1 - (u - s.tbase);     // the longest ones first
  t.first_row = tile * p.cta_rows;
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

// Which of the step's keys c .. c + 31 a row sees, of which the first `visible` are
// visible: a bit a key (tested in fewer instructions than a comparison each).
__device__ __forceinline__ uint32_t seen_of(int visible, int c) {
  return visible >= c + 32 ? 0xffffffffu : visible <= c ? 0u : (1u << (visible - c)) - 1u;
}

// 16 bytes from global to shared memory, without a register in between.
__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// UNIT: raw scores are taken times a power of two before the slopes (see ChunkParams)
template <int MAXS, bool CAP, bool BIAS, bool UNIT>
__global__ void __launch_bounds__(kChThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkParams<MAXS> p, const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  ChunkSmem& S = *reinterpret_cast<ChunkSmem*>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  // the n-th load of a piece of work, K0, K1, V0, K2, V1, ..., into ring use `use`
  auto load = [&](const ChunkTile& T, int steps, int n, uint32_t use) {
    const int s = (int)(use % kChSlots);
    const bool val = n == 2 * steps - 1 || (n > 0 && (n & 1) == 0);
    const int j = n == 2 * steps - 1 ? steps - 1 : val ? (n - 2) / 2 : (n + 1) / 2;
    const CUtensorMap* m = val ? &tmv : &tmk;
    if (p.fault && blockIdx.x == 0 && use == 1) return;     // (failure-path test)
    mbar_arrive_expect_tx(&S.full[s], kTileBytes);
    tma_load_3d(S.ring[s], m, 0, T.head, T.row0 + j * kChKeys, &S.full[s]);
    tma_load_3d(S.ring[s] + kBox, m, 64, T.head, T.row0 + j * kChKeys, &S.full[s]);
    reinterpret_cast<volatile uint32_t*>(S.issued)[s] = use / kChSlots + 1;
  };

  // ---- a softmax warp's place: tile i, rows 32 (warp & 3) .. of it
  const int i = warp >> 2, wr = 32 * (warp & 3);
  const int c16 = lane & 15, r16 = lane >> 4;        // 16 lanes a query row in global memory
  // The warp's 32 query rows of a piece (rows behind the last one repeat it): a
  // lane works out where its own row is, 16 lanes copy a row.
  auto load_queries = [&](const ChunkTile& T) {
    const int row = min(T.first_row + i * kChRows + wr + lane, T.rows - 1), tok = row / p.gqa;
    const int64_t off = (int64_t)(T.row0 + tok) * p.q_token + (int64_t)(T.head * p.gqa + row - tok * p.gqa) * p.q_head;
#pragma unroll 2
    for (int x = 0; x < 16; ++x)
      copy16_async(S.q[i] + tile_off(wr + r16 + 2 * x, c16), p.q + __shfl_sync(0xffffffffu, off, r16 + 2 * x) + 8 * c16);
  };

  // The same of a whole tile by one thread, where a tile is whole tokens (rows of
  // tokens behind the document's are loaded as they are, or as 0 behind the last).
  auto load_tile = [&](const ChunkTile& T, int i) {
    const int tok = T.row0 + (T.first_row + i * kChRows) / p.gqa;
    mbar_arrive_expect_tx(&S.q_ready[i], kTileBytes);
    tma_load_3d(S.q[i], &tmq, 0, T.head * p.gqa, tok, &S.q_ready[i]);
    tma_load_3d(S.q[i] + kBox, &tmq, 64, T.head * p.gqa, tok, &S.q_ready[i]);
  };

  uint32_t loaded = 0;     // ring uses issued so far (warp 9, lane 0)
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
      mbar_init(&S.q_ready[i], p.whole_tokens ? 1 : 4);
      mbar_init(&S.w_full[i], 1);
      mbar_init(&S.w_empty[i], kWorkReaders);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&S.v_clean[i], 2);
    mbar_init(&S.drained, 1);
    S.abort_flag = 0;
    S.stopped = INT32_MAX;
    fence_mbar_init();
    // the first loads, for which no slot has to be waited
    grid_dependency_wait();
    const ChunkTile T = locate(p, (int)blockIdx.x);
    const int steps = max(T.steps[0], T.steps[1]);
    S.work[0] = T;
    mbar_arrive(&S.w_full[0]);
    for (int i = 0; i < 2; ++i)
      if (p.whole_tokens && T.steps[i] > 0) load_tile(T, i);
    for (; (int)loaded < min(kChSlots, 2 * steps); ++loaded) load(T, steps, (int)loaded, loaded);
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  grid_dependency_wait();
  allow_dependents();
  if (warp < 8 && !p.whole_tokens) {
    const ChunkTile T = locate(p, (int)blockIdx.x);
    if ((i ? T.steps[1] : T.steps[0]) > 0) load_queries(T);
  }
  tfence_before();
  __syncthreads();
  tfence_after();
  const uint32_t tmem = S.tmem_base;

  // the number of the CTA's k-th piece (-1: no more)
  auto piece_of = [&](int k) {
    const unsigned G = gridDim.x, b = blockIdx.x, w = (unsigned)k * G + ((k & 1) ? G - 1 - b : b);
    return w < (unsigned)p.pieces ? (int)w : -1;
  };
  // The CTA's k-th piece (its `there` is 0 behind the last one, or when a wait
  // gave up); every reading warp takes and releases each piece once.
  auto take = [&](int k) {
    bool ok = wait_for_piece([&] { return mbar_try_wait(&S.w_full[k & 1], (k >> 1) & 1); }, &S.issued[0], &S.abort_flag,
                             p.spin_limit);
    ok = __all_sync(0xffffffffu, ok);
    ChunkTile T = S.work[k & 1];
    if (!ok) T.there = 0;
    return T;
  };
  auto release = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.w_empty[k & 1]);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---------------------------------------------------------- MMA issuer
      const uint64_t dq[2] = {desc128(smem_u32(S.q[0]), 16, 1024), desc128(smem_u32(S.q[1]), 16, 1024)};
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, &S.abort_flag, nullptr, p.spin_limit); };
      auto slot_full = [&](uint32_t use) { return wait(&S.full[use % kChSlots], (use / kChSlots) & 1); };
      // after the waits for what the next products read: the warp goes on together
      auto go_on = [&](bool ok) {
        ok = __all_sync(0xffffffffu, ok);
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
      bool ok = true;
      uint32_t base = 0, hid = 0, step[2] = {0, 0}, tiles[2] = {0, 0};   // ring uses, steps with hidden keys, of each tile place
      for (int k = 0;; ++k) {
        int my[2], plain;
        {
          const ChunkTile T = take(k);
          release(k);
          // (reductions: values that the compiler knows to be the whole warp's)
          if (!__reduce_or_sync(0xffffffffu, (unsigned)T.there)) break;
          my[0] = __reduce_max_sync(0xffffffffu, T.steps[0]);
          my[1] = __reduce_max_sync(0xffffffffu, T.steps[1]);
          plain = __reduce_max_sync(0xffffffffu, min(T.plain[0], T.plain[1]));
        }
        const int steps = max(my[0], my[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!ok || my[i] == 0) continue;
          ok = go_on(slot_full(base) && wait(&S.q_ready[i], tiles[i] & 1));
          ++tiles[i];
          if (ok) scores(i, base % kChSlots, i == 1 || my[1] == 0);
        }
        for (int j = 0; ok && j < steps; ++j) {
          const uint32_t kn = base + key_pos(j + 1), vn = base + value_pos(j, steps);
          const int vs = vn % kChSlots, ksl = kn % kChSlots;
          bool keep = j > 0;
          // values are N-major: 64 channels a box, 16 keys a k-step
          const uint64_t dv = desc128(smem_u32(S.ring[vs]), kBox, 1024);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || j >= my[i]) continue;
            const bool last = i == 1 || my[1] == 0;       // the step's last tile (the second one has no fewer steps)
            const uint32_t turn = step[i] & 1;
            ++step[i];
            ok = wait(&S.p_ready[i][0], turn);
            if (i == 0 || my[0] <= j) {       // the step's first tile: its values, and the next keys
              ok = ok && slot_full(vn) && (j + 1 >= steps || slot_full(kn));
              if (j >= plain) ok = ok && wait(&S.v_clean[hid & 3], (hid >> 2) & 1);
            }
            ok = go_on(ok);
            if (!ok) continue;
            if (j == 0 && j >= plain)
              keep = (S.bad[hid & 3][0] | S.bad[hid & 3][1] | S.bad[hid & 3][2] | S.bad[hid & 3][3]) != 0u;
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_ts(tmem + col_o(i), tmem + col_s(i) + 8 * ks, dv + (uint64_t)((ks * 2048) >> 4), kIdescPV, keep || ks > 0);
            }
            __syncwarp();
            ok = go_on(wait(&S.p_ready[i][1], turn));
            if (!ok) continue;
            if (elect_one()) {
#pragma unroll
              for (int ks = 4; ks < 8; ++ks)
                mma_ts(tmem + col_o(i), tmem + col_s(i) + 8 * ks, dv + (uint64_t)((ks * 2048) >> 4), kIdescPV, true);
              if (last) mma_commit(&S.empty[vs]);
              if (j + 1 >= my[i]) mma_commit(&S.o_done[i]);
            }
            __syncwarp();
            if (j + 1 < my[i]) scores(i, ksl, last);
          }
          if (j >= plain) ++hid;
        }
        if (!ok) break;
        base += 2 * steps;
      }
      if (S.abort_flag) {
        // gave up: what has been issued completes before TMEM is freed (bounded)
        if (elect_one()) mma_commit(&S.drained);
        for (uint32_t n = 0; n < p.spin_limit; ++n)
          if (mbar_try_wait(&S.drained, 0)) break;
      }
    } else if (warp == 9 && lane == 0) {
      // -------------------------------------------------------------- loads
      int n = (int)loaded;      // (of the first piece, requested above)
      bool ok = true;
      ChunkTile T = S.work[0];
      for (int k = 1;; ++k) {
        const int steps = max(T.steps[0], T.steps[1]);
        for (; n < 2 * steps; ++n, ++loaded) {
          ok = loaded < kChSlots ||
               mbar_wait_bounded(&S.empty[loaded % kChSlots], ((loaded / kChSlots) - 1) & 1, &S.abort_flag, nullptr, p.spin_limit);
          if (!ok) break;
          load(T, steps, n, loaded);
        }
        n = 0;
        if (!ok || !T.there) break;
        const int w = piece_of(k);
        if (w >= 0) {
          T = locate(p, w);
        } else {
          T.there = T.steps[0] = T.steps[1] = 0;
        }
        if (k >= 2) ok = mbar_wait_bounded(&S.w_empty[k & 1], ((k >> 1) - 1) & 1, &S.abort_flag, nullptr, p.spin_limit);
        if (!ok) break;
        S.work[k & 1] = T;
        mbar_arrive(&S.w_full[k & 1]);
      }
      if (S.abort_flag) {
        // gave up: the copies in flight get their time (bounded)
        for (uint32_t x = loaded > kChSlots ? loaded - kChSlots : 0; x < loaded; ++x)
          for (uint32_t i = 0; i < p.spin_limit; ++i)
            if (mbar_try_wait(&S.full[x % kChSlots], (x / kChSlots) & 1)) break;
      }
    } else if (warp >= 10) {
      // ----------------------------------------- value rows of partial steps
      const int half = warp - 10;
      uint32_t base = 0, hid = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const ChunkTile T = take(k);
        release(k);
        if (!T.there) break;
        const int steps = max(T.steps[0], T.steps[1]), plain = min(T.plain[0], T.plain[1]);
        for (int j = plain; j < steps; ++j, ++hid) {
          const uint32_t vn = base + value_pos(j, steps);
          const int vs = vn % kChSlots;
          // (these warps do not follow a slot's earlier uses: its phase is waited for once it exists)
          const volatile uint32_t* uses = &S.issued[vs];
          ok = wait_for_piece([&] { return *uses > vn / kChSlots; }, uses, &S.abort_flag, p.spin_limit) &&
               mbar_wait_bounded(&S.full[vs], (vn / kChSlots) & 1, &S.abort_flag, nullptr, p.spin_limit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          bool cleared = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 64 * half + 32 * i + lane;
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
            if (lane == 0) S.bad[hid & 3][2 * half + i] = bits;
            if (any != 0u) {
#pragma unroll 1
              for (int c = 0; c < 16; ++c) *reinterpret_cast<uint4*>(S.ring[vs] + tile_off(r, c)) = make_uint4(0, 0, 0, 0);
            }
            cleared = cleared || bits != 0u;
          }
          if (cleared) async_fence();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.v_clean[hid & 3]);
        }
        base += 2 * steps;
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const uint32_t lanes = (uint32_t)wr << 16;
    const uint32_t tS = tmem + col_s(i) + lanes, tO = tmem + col_o(i) + lanes;
    uint8_t* stage = S.stage[warp];
    // scores to log2 units: a factor here (slopes are divided by it), the cap's arithmetic otherwise
    const float sl = CAP ? 1.0f : UNIT ? p.unit_log2 : p.scale_log2;

    auto queries_loaded = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      async_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.q_ready[i]);
    };

    bool ok = true;
    uint32_t step = 0, hid = 0, done = 0;     // steps of this tile place, steps with hidden keys, tiles
    uint32_t tiles = 0;                       // whose queries have been requested
    {
      const ChunkTile T = S.work[0];
      tiles = (i ? T.steps[1] : T.steps[0]) > 0;
      if (tiles > 0 && !p.whole_tokens) queries_loaded();
    }
    // what the lane's row needs of a piece
    struct Row {
      int steps, plain_steps, plain;       // of this tile; steps before `plain` hide no key from any row of the piece
      int tok, limit;                      // visible keys: [0, limit)
      uint32_t at;                         // the row in the outputs
      float slope;
    };
    auto row_of = [&](const ChunkTile& T) {
      Row r;
      r.steps = i ? T.steps[1] : T.steps[0];
      r.plain_steps = i ? T.plain[1] : T.plain[0];
      r.plain = min(T.plain[0], T.plain[1]);
      const int row = min(T.first_row + i * kChRows + wr + lane, T.rows - 1);
      r.tok = row / p.gqa;
      r.limit = min(max(r.tok + 1, T.prefix), T.len);
      r.at = (uint32_t)(T.row0 + r.tok) * p.hq + T.head * p.gqa + row - r.tok * p.gqa;
      r.slope = 0.0f;
      if constexpr (BIAS) r.slope = p.slopes[T.head * p.gqa + row - r.tok * p.gqa] * p.slope_unit;
      return r;
    };
    Row next;
    {
      const ChunkTile T = take(0);
      next = row_of(T);
    }
    for (int k = 0;; ++k) {
      const int my_steps = next.steps, my_plain = next.plain_steps, plain = next.plain, tok0 = next.tok, limit = next.limit;
      const uint32_t orow = next.at;
      const float slope2 = next.slope;
      float m = -INFINITY, l = 0.0f;     // running maximum (before sl) and sum
      uint32_t hj = hid;
      for (int j = 0; j < my_steps; ++j, ++step) {
        ok = ok && mbar_wait_bounded(&S.s_full[i], step & 1, &S.abort_flag, nullptr, p.spin_limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tfence_after();
        float s[kChKeys];
        float top = -INFINITY;
        {
#pragma unroll
          for (int c = 0; c < kChKeys; c += 32) tld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&s[c]));
          tld_wait();
          if constexpr (CAP) {
            float hi = fmaxf(s[0], s[1]), lo = fminf(s[0], s[1]);
#pragma unroll
            for (int c = 2; c < kChKeys; c += 2) {
              asm("max.f32 %0, %0, %1, %2;" : "+f"(hi) : "f"(s[c]), "f"(s[c + 1]));
              asm("min.f32 %0, %0, %1, %2;" : "+f"(lo) : "f"(s[c]), "f"(s[c + 1]));
            }
            // (the scores of a model with a cap mostly stay well within it, hidden ones too)
            const float reach = fmaxf(hi, -lo) * p.cap_near;
            if (__all_sync(0xffffffffu, reach <= kCapSmall)) {
#pragma unroll
              for (int c = 0; c < kChKeys; c += 2) {
                const float2 y = cap_small(make_float2(s[c], s[c + 1]), p);
                s[c] = y.x;
                s[c + 1] = y.y;
              }
              top = cap_small(make_float2(hi, hi), p).x;
            } else {
              // A row takes the form that the scores which it sees ask for, by itself:
              // neither hidden keys nor the warp's other rows have a part in its bits
              // (the short polynomial is the long one with zeros for its last terms).
              // Branches by row cost what each takes (8,192 capped tokens: 454 us where
              // all scores are small, 556 within 0.6 of the cap, 826 all beyond, 990 to
              // 1,180 with rows of every kind in a warp; with one form a warp, chosen by
              // what its rows do not see as well, 449, 515, 751 and 777 to 856).
              float own = reach;
              if (j >= my_plain) {
                const int vis = limit - j * kChKeys;
                own = 0.0f;
#pragma unroll
                for (int c = 0; c < kChKeys; c += 32) {
                  const uint32_t seen = seen_of(vis, c);
#pragma unroll
                  for (int e = 0; e < 32; ++e) own = (seen >> e) & 1u ? fmaxf(own, fabsf(s[c + e])) : own;
                }
                own *= p.cap_near;
              }
              float c[5];
#pragma unroll
              for (int e = 0; e < 5; ++e) c[e] = !(own <= kCapSmall) ? p.cap_c[e] : e < 3 ? p.cap_d[e] : 0.0f;
              if (__all_sync(0xffffffffu, own <= 1.0f)) {
#pragma unroll
                for (int k = 0; k < kChKeys; k += 2) {
                  const float2 y = cap_near(make_float2(s[k], s[k + 1]), c);
                  s[k] = y.x;
                  s[k + 1] = y.y;
                }
                top = cap_near(make_float2(hi, hi), c).x;
              } else if (own <= 1.0f) {
#pragma unroll
                for (int k = 0; k < kChKeys; k += 2) {
                  const float2 y = cap_near(make_float2(s[k], s[k + 1]), c);
                  s[k] = y.x;
                  s[k + 1] = y.y;
                }
                top = cap_near(make_float2(hi, hi), c).x;
              } else {
#pragma unroll
                for (int k = 0; k < kChKeys; ++k) s[k] = cap_far(s[k], p.cap_in, p.cap_out, p.cap_log2);
                top = cap_far(hi, p.cap_in, p.cap_out, p.cap_log2);
              }
              __syncwarp();
            }
          }
          if constexpr (UNIT) {
#pragma unroll
            for (int c = 0; c < kChKeys; ++c) s[c] *= p.score_unit;
          }
          if constexpr (BIAS) {
            const float2 slope = make_float2(-slope2, -slope2);
            float2 d[4];     // distances, tok0 - key
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float d0 = (float)(tok0 - j * kChKeys - 2 * e);
              d[e] = make_float2(d0, d0 - 1.0f);
            }
            auto lower = [&](auto both_ways) {
#pragma unroll
              for (int c = 0; c < kChKeys; c += 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  float2 y = make_float2(s[c + 2 * e], s[c + 2 * e + 1]);
                  y = __ffma2_rn(slope, decltype(both_ways)::value ? make_float2(fabsf(d[e].x), fabsf(d[e].y)) : d[e], y);
                  s[c + 2 * e] = y.x;
                  s[c + 2 * e + 1] = y.y;
                  d[e] = __fadd2_rn(d[e], make_float2(-8.0f, -8.0f));
                }
              }
            };
            if (__any_sync(0xffffffffu, tok0 < (j + 1) * kChKeys - 1)) lower(std::true_type{});   // keys behind the query's token
            else lower(std::false_type{});
          }
          if (j >= my_plain) {
            const int vis = limit - j * kChKeys;
#pragma unroll
            for (int c = 0; c < kChKeys; c += 32) {
              const uint32_t seen = seen_of(vis, c);
#pragma unroll
              for (int e = 0; e < 32; ++e) s[c + e] = (seen >> e) & 1u ? s[c + e] : -INFINITY;
            }
          }
          if (BIAS || !CAP || j >= my_plain) {
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
            top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          }
        }
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
        float base = m == -INFINITY ? 0.0f : -m * sl;
        if constexpr (BIAS || !CAP) {
          // scores far from zero: -m sl is rounded by more than an exponent bears (the same
          // for all of a row's weights, so it does not matter before); the maximum is taken off first
          const bool far = fabsf(base) > kFarBase;
          if (__any_sync(0xffffffffu, far)) {
            const float off = far ? -m : 0.0f;
#pragma unroll
            for (int c = 0; c < kChKeys; ++c) s[c] += off;
            if (far) base = 0.0f;
          }
        }
        const float2 sl2 = make_float2(sl, sl), base2 = make_float2(base, base);
        float2 sum0 = make_float2(0.0f, 0.0f), sum1 = make_float2(0.0f, 0.0f);
        auto weights = [&](const float* x, uint32_t* pk) {     // of 4 scores
          const float2 a = __ffma2_rn(make_float2(x[0], x[1]), sl2, base2), b = __ffma2_rn(make_float2(x[2], x[3]), sl2, base2);
          const float2 pa = make_float2(tc_exp2(a.x), tc_exp2(a.y)), pb = make_float2(tc_exp2(b.x), tc_exp2(b.y));
          sum0 = __fadd2_rn(sum0, pa);
          sum1 = __fadd2_rn(sum1, pb);
          pk[0] = pack_bf16x2(pa.x, pa.y);
          pk[1] = pack_bf16x2(pb.x, pb.y);
        };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; e += 2) weights(&s[64 * half + 2 * e], &pk[e]);
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
          ok = mbar_wait_bounded(&S.v_clean[hj & 3], (hj >> 2) & 1, &S.abort_flag, nullptr, p.spin_limit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t* bad = S.bad[hj & 3];
          ++hj;
          if ((bad[0] | bad[1] | bad[2] | bad[3]) != 0u) {
            const ChunkTile T = S.work[k & 1];
            add_cleared(tS, tO, bad, limit - j * kChKeys, j == 0,
                        p.v + (int64_t)(T.row0 + j * kChKeys) * p.v_token + (int64_t)T.head * p.v_head, p.v_token);
          }
        }
        tfence_before();
        __syncwarp();
        if (lane == 0) {
          if (j >= plain) mbar_arrive(&S.p_ready[i][0]);
          mbar_arrive(&S.p_ready[i][1]);
        }
        l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
      }
      const ChunkTile T = S.work[k & 1];
      release(k);
      hid += max(T.steps[0], T.steps[1]) - plain;

      // every product with this piece's queries is done (its last scores were):
      // the next piece's take their place meanwhile
      bool more, queries;
      {
        const ChunkTile N = take(k + 1);
        more = N.there != 0;
        queries = more && (i ? N.steps[1] : N.steps[0]) > 0;
        if (more) next = row_of(N);
        if (queries && ok) {
          ++tiles;
          if (!p.whole_tokens) load_queries(N);
          else if ((warp & 3) == 0 && lane == 0) load_tile(N, i);
        }
      }
      if (my_steps > 0) {
        // o / l, merged with the row over what precedes the chunk.  A warp's rows pass
        // through its part of shared memory, kStageRow bytes at a time (a loop of few
        // instructions: they are fetched anew for every piece): kLanes lanes a row in
        // global memory, a thread a row in between.
        const int rows = T.rows - (T.first_row + i * kChRows + wr);     // rows of the warp that exist
        constexpr int kLanes = kStageRow / 16, kTogether = 32 / kLanes;
        const int cx = lane % kLanes, rx = lane / kLanes;
        uint32_t from[kLanes];     // rows rx, rx + kTogether, ... of the outputs (rows behind the last one repeat it)
#pragma unroll
        for (int x = 0; x < kLanes; ++x) from[x] = __shfl_sync(0xffffffffu, orow, rx + kTogether * x);
        // 16-byte chunk c of row x in shared memory: 8 lanes of either order touch every bank once
        auto staged = [&](int x, int c) {
          return reinterpret_cast<uint4*>(stage + x * kStageRow + ((c ^ ((x * kLanes / 8) & (kLanes - 1))) << 4));
        };
        const bool merge = p.prior_lse != nullptr;
        const float before = merge ? p.prior_lse[orow] : -INFINITY;
        // rows to merge with, requested early
        uint4 u[kLanes];
        auto load_prior = [&](int c) {
#pragma unroll
          for (int x = 0; x < kLanes; ++x)
            u[x] = *reinterpret_cast<const uint4*>(p.prior_out + (int64_t)from[x] * kHeadDim + c + 8 * cx);
        };
        if (merge) load_prior(0);
        if (ok) {
          ok = mbar_wait_bounded(&S.o_done[i], done & 1, &S.abort_flag, nullptr, p.spin_limit);
          ok = __all_sync(0xffffffffu, ok);
          tfence_after();
        }
        ++done;
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
        for (int c = 0; c < kHeadDim; c += kStageRow / 2) {
          if (merge) {
#pragma unroll
            for (int x = 0; x < kLanes; ++x) *staged(rx + kTogether * x, cx) = u[x];
            __syncwarp();
            if (c + kStageRow / 2 < kHeadDim) load_prior(c + kStageRow / 2);
          }
          uint32_t o[kStageRow / 2];
          if (ok) {
#pragma unroll
            for (int d = 0; d < kStageRow / 2; d += 32) tld32(tO + c + d, *reinterpret_cast<uint32_t(*)[32]>(&o[d]));
            tld_wait();
          } else {
#pragma unroll
            for (int q = 0; q < kStageRow / 2; ++q) o[q] = 0x7fc00000u;
          }
#pragma unroll
          for (int d = 0; d < kLanes; ++d) {
            uint4* mine = staged(lane, d);
            float x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = __uint_as_float(o[8 * d + q]) * fo;
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
          __syncwarp();
#pragma unroll
          for (int x = 0; x < kLanes; ++x)
            if (rx + kTogether * x < rows)
              *reinterpret_cast<uint4*>(p.out + (int64_t)from[x] * kHeadDim + c + 8 * cx) = *staged(rx + kTogether * x, cx);
          __syncwarp();
        }
        tfence_before();
        if (lane < rows && p.lse != nullptr) p.lse[orow] = lse;
      }
      if (!more || !ok) {
        if (S.abort_flag && lane == 0) atomicMin(&S.stopped, k + 1);
        break;
      }
      if (queries && !p.whole_tokens) queries_loaded();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (S.abort_flag && p.whole_tokens && tiles > 0)     // (bounded: the last queries' copy gets its time)
      for (uint32_t n = 0; n < p.spin_limit; ++n)
        if (mbar_try_wait(&S.q_ready[i], (tiles - 1) & 1)) break;
    named_bar_sync(1, 256);
    if (S.abort_flag) {
      // gave up: the rows of the pieces that were not begun (the others' are written)
      for (int k = S.stopped; k < INT32_MAX && piece_of(k) >= 0; ++k) {
        const ChunkTile T = locate(p, piece_of(k));
        const int rows = min(p.cta_rows, T.rows - T.first_row);
        for (int x = tid; x < 16 * rows; x += 256) {
          const int row = T.first_row + x / 16, tok = row / p.gqa;
          const int64_t at = (int64_t)(T.row0 + tok) * p.hq + T.head * p.gqa + row - tok * p.gqa;
          const uint32_t nan2 = 0x7fc07fc0u;
          *reinterpret_cast<uint4*>(p.out + at * kHeadDim + 8 * (x % 16)) = make_uint4(nan2, nan2, nan2, nan2);
          if (x % 16 == 0 && p.lse != nullptr) p.lse[at] = NAN;
        }
      }
    }
  }

  tfence_before();
  __syncthreads();
  if (warp == 8) {
    tfence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// Rows [token][head][128 channels] of bf16: box = 64 channels of 128 rows, box_heads heads a token.
bool encode_chunk_map(CUtensorMap* map, const void* base, uint64_t tokens, uint64_t heads, uint64_t token_bytes,
                      uint64_t head_bytes, uint32_t box_heads = 1) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {kHeadDim, heads, tokens};
  const cuuint64_t strides[2] = {head_bytes, token_bytes};
  const cuuint32_t box[3] = {64, box_heads, kChRows / box_heads};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static_assert(sizeof(ChunkParams<kDecodeSeqsLarge>) + 3 * sizeof(CUtensorMap) + 64 <= 32764, "kernel parameter limit");

template <int MAXS, bool CAP, bool BIAS, bool UNIT = false>
cudaError_t launch_chunk_t(const ChunkParams<MAXS>& p, const CUtensorMap& tmk, const CUtensorMap& tmv, const CUtensorMap& tmq, unsigned grid,
                           cudaStream_t stream) {
  static bool attr_done[64] = {};
  const int smem = (int)sizeof(ChunkSmem) + 1024;
  cudaError_t e = ensure_smem_attr(chunk_kernel<MAXS, CAP, BIAS, UNIT>, smem, attr_done);
  if (e != cudaSuccess) return e;
  // the warps' shares of the registers must fit in what the block is launched with
  static const int regs = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, chunk_kernel<MAXS, CAP, BIAS, UNIT>) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs * kChThreads < 256 * kSoftmaxRegs + 128 * kOtherRegs) return cudaErrorInvalidConfiguration;
  return launch_dependent(chunk_kernel<MAXS, CAP, BIAS, UNIT>, dim3(grid), dim3(kChThreads), (size_t)smem, stream, 1, p, tmk, tmv, tmq);
}

}  // namespace

int64_t chunk_tiles(const ChunkSeq* docs, int n, int gqa, int hkv, int sms, int32_t* cta_rows) {
  // two row tiles a CTA share its key tiles; one each while that leaves SMs without work
  for (*cta_rows = 2 * kChRows;; *cta_rows = kChRows) {
    int64_t tiles = 0;
    for (int i = 0; i < n; ++i) tiles += ((int64_t)docs[i].len * gqa + *cta_rows - 1) / *cta_rows;
    if (*cta_rows == kChRows || tiles * hkv >= sms) return tiles;
  }
}

template <int MAXS>
cudaError_t launch_chunk(ChunkParams<MAXS>& p, int64_t tokens, int sms, cudaStream_t stream) {
  CUtensorMap tmk, tmv, tmq{};
  if (!encode_chunk_map(&tmk, p.k, tokens, p.hkv, 2 * p.k_token, 2 * p.k_head) ||
      !encode_chunk_map(&tmv, p.v, tokens, p.hkv, 2 * p.v_token, 2 * p.v_head))
    return cudaErrorInvalidValue;
  p.whole_tokens = kChRows % p.gqa == 0;
  if (p.whole_tokens && !encode_chunk_map(&tmq, p.q, tokens, p.hq, 2 * p.q_token, 2 * p.q_head, p.gqa))
    return cudaErrorInvalidValue;
  int64_t tiles = chunk_tiles(p.seq, p.n_seqs, p.gqa, p.hkv, sms, &p.cta_rows);
  p.pieces = (int32_t)(tiles * p.hkv);
  tiles = 0;
  for (int i = 0; i < p.n_seqs; ++i) {
    p.seq[i].tbase = (int32_t)tiles;
    tiles += ((int64_t)p.seq[i].len * p.gqa + p.cta_rows - 1) / p.cta_rows;
  }
  // several rounds over documents of different lengths: pieces in descending order
  // of their steps (without the table, document by document: 24 documents of 1 to
  // 1,531 tokens took 1.3 times as long)
  p.sorted = p.pieces > sms && p.n_seqs > 1 && tiles <= ChunkParams<MAXS>::kOrder;
  if (p.sorted) {
    struct Entry {
      int32_t steps;
      uint32_t what;
    } list[ChunkParams<MAXS>::kOrder];
    int n = 0;
    for (int i = 0; i < p.n_seqs; ++i) {
      const int64_t rows = (int64_t)p.seq[i].len * p.gqa;
      for (int64_t r = 0; r < rows; r += p.cta_rows) {
        const int last = (int)((std::min<int64_t>(r + p.cta_rows, rows) - 1) / p.gqa);
        const int lim = std::min(std::max(last + 1, p.seq[i].prefix), p.seq[i].len);
        list[n++] = Entry{(lim + kChKeys - 1) / kChKeys, (uint32_t)i << 22 | (uint32_t)(r / p.cta_rows)};
      }
    }
    std::sort(list, list + n, [](const Entry& a, const Entry& b) {
      return a.steps != b.steps ? a.steps > b.steps : a.what < b.what;
    });
    for (int i = 0; i < n; ++i) p.order[i] = list[i].what;
  }
  const unsigned grid = (unsigned)std::min<int64_t>(p.pieces, sms);
  const bool cap = p.cap_log2 != 0.0f, bias = p.slopes != nullptr;
  if (cap) return bias ? launch_chunk_t<MAXS, true, true>(p, tmk, tmv, tmq, grid, stream)
                       : launch_chunk_t<MAXS, true, false>(p, tmk, tmv, tmq, grid, stream);
  if constexpr (MAXS == kDecodeSeqsLarge)
    if (bias && p.score_unit != 1.0f) return launch_chunk_t<MAXS, false, true, true>(p, tmk, tmv, tmq, grid, stream);
  return bias ? launch_chunk_t<MAXS, false, true>(p, tmk, tmv, tmq, grid, stream)
              : launch_chunk_t<MAXS, false, false>(p, tmk, tmv, tmq, grid, stream);
}

template cudaError_t launch_chunk<kDecodeSeqsSmall>(ChunkParams<kDecodeSeqsSmall>&, int64_t, int, cudaStream_t);
template cudaError_t launch_chunk<kDecodeSeqsLarge>(ChunkParams<kDecodeSeqsLarge>&, int64_t, int, cudaStream_t);

}  // namespace oscar
