// Attention within a chunk whose documents have at most 32 tokens (drafted tokens
// under verification, single steps): the same call as in chunk.cu, laid out for
// latency (sm_103a).
//
// A warp takes 16 (token, query head) rows of one document and KV head against all
// of its keys, by itself: no barrier, no tensor memory, and about a tenth of the
// instructions of the tiled kernel, of whose time on such documents more than half
// goes into fetching its code.  All of its loads are in flight at once; scores and
// values run on mma.sync m16n8k16:
//   scores: A = queries, B = keys, straight from 16-byte loads (the channels in any
//           order, the same for both);
//   values: A = the weights where the scores were accumulated, in two bf16 terms (16
//           bits), B = values through shared memory (ldmatrix.trans), copied there
//           without registers in between: 168 a thread instead of 220, 12 warps an SM
//           instead of 8 (1,000 documents of 32 tokens 371 -> 255 us; 16 warps, with
//           spills, 285).
// Rows leave through shared memory, 16 lanes a row.  Values that are not finite and
// that some row does not see would spoil it through 0 times infinity: a warp that
// finds one clears the token's values there, and rows that do see it add them on the
// CUDA cores.
// Beside longer documents it runs behind the tiled kernel, whose rows it has no part in,
// without waiting for it to end (500 documents of 5 tokens beside one of 300: 33 us,
// all of them tiled 135; 5 tokens beside 33: 8.1, tiled 7.1).
// 8 documents of 5 tokens, 32 heads, merged: 7.9 us in the tiled kernel, 4.3 here; 64
// documents of 32 tokens 22 us (of 40, tiled: 28).  Bound by latency: a warp's loads,
// scores, weights and rows follow one another.
#include "common.cuh"
#include "launch.h"

namespace oscar {
namespace {

constexpr int kShortRows = 16;
constexpr int kShortWarps = 4;
constexpr int kVPitch = kHeadDim * 2 + 16;        // bytes of a value row in shared memory
constexpr int kOPitch = kHeadDim + 4;             // floats of an output row there

// KEYS: 16 or 32, at least the longest document's tokens
template <int KEYS>
struct ShortSmem {
  static constexpr int kValues = KEYS * kVPitch, kOut = kShortRows * kOPitch * 4;
  alignas(16) uint8_t v[kValues > kOut ? kValues : kOut];   // values, then the rows' outputs in float32
  float p[kShortRows][KEYS];                      // weights (of a warp that has cleared values)
  float prior[kShortRows];                        // factor of the row to merge with
};
static_assert(kShortWarps * sizeof(ShortSmem<kChunkShort>) <= 48 * 1024, "static shared memory");

// 16 bytes from global to shared memory, or 0 there.
__device__ __forceinline__ void copy16_or_zero(void* dst, const void* src, bool copy) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(copy ? 16 : 0) : "memory");
}

template <int MAXS, int KEYS>
__global__ void __launch_bounds__(32 * kShortWarps, KEYS == 32 ? 3 : 4)
    chunk_short_kernel(const __grid_constant__ ChunkParams<MAXS> p) {
  __shared__ ShortSmem<KEYS> smem[kShortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = (int)blockIdx.x * kShortWarps + warp;
  if (piece >= p.pieces) return;
  ShortSmem<KEYS>& S = smem[warp];
  constexpr int kTiles = KEYS / 8;
  // the piece: document, KV head, rows
  const int u = piece / p.hkv;
  int lo = 0, hi = p.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.seq[mid].tbase <= u) lo = mid; else hi = mid - 1;
  }
  const ChunkSeq d = p.seq[lo];
  const int rows = d.len * p.gqa, tiles = (rows + kShortRows - 1) / kShortRows;
  // (the pieces of a head side by side: they share keys and values)
  const int at_doc = piece - d.tbase * p.hkv, j = at_doc / tiles;
  const int first = (at_doc - j * tiles) * kShortRows;
  const int last_tok = (min(first + kShortRows, rows) - 1) / p.gqa;
  const int keys = min(max(last_tok + 1, d.prefix), d.len);
  const int g = lane >> 2, tig = lane & 3;
  int tok[2], limit[2];
  const uint16_t* q[2];
  float slope2[2] = {0.0f, 0.0f};
  const int r16 = lane >> 4, c16 = lane & 15;       // 16 lanes a row: values, prior, outputs
  // the row of the outputs that lane l < 16 stands for (rows behind the last one repeat it)
  const int mine = min(first + (lane & 15), rows - 1), mtok = mine / p.gqa;
  const uint32_t orow = (uint32_t)(d.row0 + mtok) * p.hq + j * p.gqa + mine - mtok * p.gqa;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int row = min(first + g + 8 * x, rows - 1);
    tok[x] = row / p.gqa;
    limit[x] = min(max(tok[x] + 1, d.prefix), d.len);
    const int h = j * p.gqa + row - tok[x] * p.gqa;
    q[x] = p.q + (int64_t)(d.row0 + tok[x]) * p.q_token + (int64_t)h * p.q_head + 8 * tig;
  }
  if (!p.late) {
    grid_dependency_wait();
    allow_dependents();
  }

  // ---- everything that is read
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 qa[4], qb[4], kf[kTiles][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    qa[i] = *reinterpret_cast<const uint4*>(q[0] + 32 * i);
    qb[i] = *reinterpret_cast<const uint4*>(q[1] + 32 * i);
  }
  const uint16_t* kbase = p.k + (int64_t)d.row0 * p.k_token + (int64_t)j * p.k_head + 8 * tig;
#pragma unroll
  for (int nt = 0; nt < kTiles; ++nt) {
    const int key = 8 * nt + g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      kf[nt][i] = key < keys ? *reinterpret_cast<const uint4*>(kbase + key * p.k_token + 32 * i) : zero;
  }
  const uint16_t* vbase = p.v + (int64_t)d.row0 * p.v_token + (int64_t)j * p.v_head + 8 * c16;
#pragma unroll
  for (int x = 0; x < KEYS / 2; ++x)
    copy16_or_zero(S.v + (2 * x + r16) * kVPitch + 16 * c16, vbase + min(2 * x + r16, keys - 1) * p.v_token,
                   2 * x + r16 < keys);
  if (p.rule.slopes != nullptr) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = min(first + g + 8 * x, rows - 1);
      slope2[x] = p.rule.slopes[j * p.gqa + row - tok[x] * p.gqa] * 1.4426950408889634f;
    }
  }
  const bool merge = p.prior_lse != nullptr;
  uint4 pr[kShortRows / 2];
  float before[2] = {-INFINITY, -INFINITY};
  if (merge) {
#pragma unroll
    for (int x = 0; x < 2; ++x) before[x] = p.prior_lse[__shfl_sync(0xffffffffu, orow, g + 8 * x)];
#pragma unroll
    for (int x = 0; x < kShortRows / 2; ++x)
      pr[x] = *reinterpret_cast<const uint4*>(p.prior_out + (int64_t)__shfl_sync(0xffffffffu, orow, 2 * x + r16) * kHeadDim + 8 * c16);
  }

  // ---- scores of rows g and g + 8, keys 8 nt + 2 tig, + 1, under the rule
  float s[kTiles][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int nt = 0; nt < kTiles; ++nt) {
    s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
    if (8 * nt < keys) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mma_bf16_16816(s[nt], qa[i].x, qb[i].x, qa[i].y, qb[i].y, kf[nt][i].x, kf[nt][i].y);
        mma_bf16_16816(s[nt], qa[i].z, qb[i].z, qa[i].w, qb[i].w, kf[nt][i].z, kf[nt][i].w);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float2 y = make_float2(s[nt][2 * x] * p.scale_log2, s[nt][2 * x + 1] * p.scale_log2);
      if (p.rule.cap != 0.0f) y = capped(y, p.rule, false);
      const int key = 8 * nt + 2 * tig;
      y.x = fmaf(-slope2[x], fabsf((float)(tok[x] - key)), y.x);
      y.y = fmaf(-slope2[x], fabsf((float)(tok[x] - key - 1)), y.y);
      s[nt][2 * x] = key < limit[x] ? y.x : -INFINITY;
      s[nt][2 * x + 1] = key + 1 < limit[x] ? y.y : -INFINITY;
      m[x] = fmaxf(m[x], fmaxf(s[nt][2 * x], s[nt][2 * x + 1]));
    }
  }
  // ---- the values are in shared memory: a lane looks through what it copied
  auto mine_of = [&](int x) { return reinterpret_cast<uint4*>(S.v + (2 * x + r16) * kVPitch + 16 * c16); };
  auto not_finite = [](uint4 w) {
    // an exponent of all ones carries into bit 15 of its half
    return ((((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
             ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u)) &
            0x80008000u) != 0u;
  };
  bool odd = false;
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
  for (int x = 0; x < KEYS / 2; ++x) odd = odd || not_finite(*mine_of(x));
  odd = __any_sync(0xffffffffu, odd);
  uint32_t bad = 0u;                       // tokens whose values are not finite, cleared there
  if (odd) {
#pragma unroll 1
    for (int x = 0; x < KEYS / 2; ++x) {
      const uint32_t lanes = __ballot_sync(0xffffffffu, not_finite(*mine_of(x)));
      bad |= ((lanes & 0xffffu) != 0u ? 1u : 0u) << (2 * x) | ((lanes >> 16) != 0u ? 1u : 0u) << (2 * x + 1);
      if ((bad >> (2 * x + r16)) & 1u) *mine_of(x) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    m[x] = fmaxf(m[x], __shfl_xor_sync(0xffffffffu, m[x], 1));
    m[x] = fmaxf(m[x], __shfl_xor_sync(0xffffffffu, m[x], 2));
    const float base = m[x] == -INFINITY ? 0.0f : m[x];
#pragma unroll
    for (int nt = 0; nt < kTiles; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[nt][2 * x + e] = exp2f(s[nt][2 * x + e] - base);
        l[x] += s[nt][2 * x + e];
      }
    }
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
  }
  // ---- factors of the row and of the one to merge with
  float fo[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float lse = fmaf(m[x], 0.69314718055994530942f, logf(l[x])), fp = 0.0f;
    fo[x] = 1.0f / l[x];
    if (before[x] != -INFINITY) {
      const float top = fmaxf(lse, before[x]);
      const float a = expf(lse - top), b = expf(before[x] - top);
      fp = b / (a + b);
      fo[x] *= a / (a + b);
      lse = top + logf(a + b);
    }
    const uint32_t at = __shfl_sync(0xffffffffu, orow, g + 8 * x);
    if (tig == 0) {
      S.prior[g + 8 * x] = fp;
      if (p.lse != nullptr && first + g + 8 * x < rows) p.lse[at] = lse;
    }
  }
  __syncwarp();
  float* out = reinterpret_cast<float*>(S.v);
  float o[16][4];
#pragma unroll
  for (int t = 0; t < 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.0f;
#pragma unroll
  for (int kk = 0; kk < KEYS / 16; ++kk) {
    if (16 * kk >= keys) break;
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {       // rows g, g + 8 of keys 2 tig .., then of keys 2 tig + 8 ..
      const float* x = &s[2 * kk + (e >> 1)][2 * (e & 1)];
      ph[e] = pack_bf16x2(x[0], x[1]);
      pl[e] = pack_bf16x2(x[0] - bf16_lo(ph[e]), x[1] - bf16_hi(ph[e]));
    }
    const uint32_t at = smem_u32(S.v) + (16 * kk + (lane & 15)) * kVPitch + 16 * (lane >> 4);
#pragma unroll
    for (int t = 0; t < 16; t += 2) {
      uint32_t b0, b1, b2, b3;
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(b0), "=r"(b1), "=r"(b2), "=r"(b3)
                   : "r"(at + 16 * t));
      mma_bf16_16816(o[t], ph[0], ph[1], ph[2], ph[3], b0, b1);
      mma_bf16_16816(o[t + 1], ph[0], ph[1], ph[2], ph[3], b2, b3);
      mma_bf16_16816(o[t], pl[0], pl[1], pl[2], pl[3], b0, b1);
      mma_bf16_16816(o[t + 1], pl[0], pl[1], pl[2], pl[3], b2, b3);
    }
  }
  __syncwarp();                          // the values have been read
#pragma unroll
  for (int t = 0; t < 16; ++t) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
      *reinterpret_cast<float2*>(out + (g + 8 * x) * kOPitch + 8 * t + 2 * tig) =
          make_float2(o[t][2 * x] * fo[x], o[t][2 * x + 1] * fo[x]);
  }
  if (odd) {
    // rows that see a cleared token add its values by their weights; the others keep
    // the bits that they have whatever it holds
#pragma unroll
    for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) S.p[g + 8 * (x >> 1)][8 * nt + 2 * tig + (x & 1)] = s[nt][x] * fo[x >> 1];
    __syncwarp();
#pragma unroll 1
    for (int r = 0; r < kShortRows; ++r) {
      const int see = min(max(min(first + r, rows - 1) / p.gqa + 1, d.prefix), d.len);
      uint32_t left = see >= 32 ? bad : bad & ((1u << see) - 1u);
      if (left == 0u) continue;
      float4 a = *reinterpret_cast<const float4*>(out + r * kOPitch + 4 * lane);
      for (; left != 0u; left &= left - 1u) {
        const int t = __ffs((int)left) - 1;
        const uint2 w = *reinterpret_cast<const uint2*>(p.v + (int64_t)(d.row0 + t) * p.v_token + (int64_t)j * p.v_head + 4 * lane);
        const float f = S.p[r][t];
        a.x = fmaf(f, bf16_lo(w.x), a.x);
        a.y = fmaf(f, bf16_hi(w.x), a.y);
        a.z = fmaf(f, bf16_lo(w.y), a.z);
        a.w = fmaf(f, bf16_hi(w.y), a.w);
      }
      *reinterpret_cast<float4*>(out + r * kOPitch + 4 * lane) = a;
    }
  }
  __syncwarp();
  // ---- rows out, merged
#pragma unroll
  for (int x = 0; x < kShortRows / 2; ++x) {
    const int r = 2 * x + r16;
    const float4 a = *reinterpret_cast<const float4*>(out + r * kOPitch + 8 * c16);
    const float4 b = *reinterpret_cast<const float4*>(out + r * kOPitch + 8 * c16 + 4);
    float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const float fp = S.prior[r];
    if (merge && fp != 0.0f) {             // (also NaN)
      const uint4 w = pr[x];
      y[0] = fmaf(bf16_lo(w.x), fp, y[0]);
      y[1] = fmaf(bf16_hi(w.x), fp, y[1]);
      y[2] = fmaf(bf16_lo(w.y), fp, y[2]);
      y[3] = fmaf(bf16_hi(w.y), fp, y[3]);
      y[4] = fmaf(bf16_lo(w.z), fp, y[4]);
      y[5] = fmaf(bf16_hi(w.z), fp, y[5]);
      y[6] = fmaf(bf16_lo(w.w), fp, y[6]);
      y[7] = fmaf(bf16_hi(w.w), fp, y[7]);
    }
    const int64_t to = (int64_t)__shfl_sync(0xffffffffu, orow, r) * kHeadDim + 8 * c16;
    if (first + r < rows)
      *reinterpret_cast<uint4*>(p.out + to) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                         pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
  }
  if (p.late) {
    grid_dependency_wait();
    allow_dependents();
  }
}

}  // namespace

template <int MAXS>
cudaError_t launch_chunk_short(ChunkParams<MAXS>& p, cudaStream_t stream) {
  int64_t tiles = 0;
  for (int i = 0; i < p.n_seqs; ++i) {
    p.seq[i].tbase = (int32_t)tiles;
    tiles += ((int64_t)p.seq[i].len * p.gqa + kShortRows - 1) / kShortRows;
  }
  p.pieces = (int32_t)(tiles * p.hkv);
  const unsigned grid = (unsigned)((p.pieces + kShortWarps - 1) / kShortWarps);
  // (the longest document is the first)
  return launch_dependent(p.seq[0].len <= 16 ? chunk_short_kernel<MAXS, 16> : chunk_short_kernel<MAXS, kChunkShort>, dim3(grid),
                          dim3(32 * kShortWarps), 0, stream, 1, p);
}

template cudaError_t launch_chunk_short<kDecodeSeqsSmall>(ChunkParams<kDecodeSeqsSmall>&, cudaStream_t);
template cudaError_t launch_chunk_short<kDecodeSeqsLarge>(ChunkParams<kDecodeSeqsLarge>&, cudaStream_t);

}  // namespace oscar
