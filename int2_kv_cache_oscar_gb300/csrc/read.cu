// Tokens of the cache read back (sm_103a): keys and values of a range of each
// sequence, as bf16 or float32 rows.
//
//   group tokens:  k_t = H_d (n_t (code_t s + z)),  v_t = code^V_t s^V_t + z^V_t
//   window tokens: the stored bf16 rows.
//
// H_d is its own inverse, so reading a key back is one more Walsh-Hadamard
// transform: 7 x 64 packed adds per token against 256 bytes written, on the
// CUDA cores; the matrix-product form (128 x 128 x 128 per group on the tensor
// cores, the float32 scales split into two fp16 terms) would need the scaled
// codes expanded into operand tiles, which costs more than the transform.
//
// One block of 128 threads per (128-token tile, KV head), taken from a list of
// tiles in a persistent grid; the next tile's packed block (13,824 or 11,008
// bytes) is on its way into a second shared-memory stage (one bulk copy)
// meanwhile.  The values come first: one barrier between the two parts of a
// tile is enough, and warps drift apart by up to a part.
//   keys:   thread = token.  Its codes are 8 words; channels c and c + 64 sit
//           at the same bit of two of them and share a packed pair, so six
//           transform stages are packed adds in registers and the last one is
//           within the pairs.  The thread puts its row into shared memory (rows
//           16 bytes apart in banks) and sends it off with one bulk store:
//           stored from registers, 32 rows of different lines a warp, the keys
//           kept the load/store unit busy for a quarter of the time.
//   values: thread = 8 channels x 16 tokens (8 words), so that 16 lanes write
//           one token's row.
// Bound by HBM writes (512 or 1,024 bytes written per 108 or 86 read).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace oscar {
namespace {

constexpr int kReadThreads = 128;
constexpr int kReadStages = 2;
constexpr float kTwo23 = 8388608.0f;
constexpr uint32_t kTwo23Bits = 0x4B000000u;

template <bool M16, bool F32>
struct ReadSmem {
  static constexpr int kRow = kHeadDim * (F32 ? 4 : 2);
  static constexpr int kPitch = kRow + 16;
  alignas(128) uint8_t stage[kReadStages][Blk<M16>::kBytes];
  alignas(16) uint8_t krow[kGroup][kPitch];   // key rows on their way out
  alignas(16) float4 kp[kReadStages][kHeadDim / 2];   // channels (c, c + 64): scale 2^-b (2), zero (2), b the codes' bit
  alignas(8) uint64_t full[kReadStages];
  int abort_flag;
};

static_assert(sizeof(ReadSmem<false, true>) <= 113 * 1024 && sizeof(ReadSmem<false, false>) <= 75 * 1024,
              "two and three blocks per SM");
static_assert(ReadSmem<false, false>::kPitch % 16 == 0 && ReadSmem<true, true>::kPitch % 16 == 0, "bulk stores");

// Bit of the code of column c within its (half) word once the upper 16 bits
// have been shifted down for odd columns: 4 kk + 2 hf.
__host__ __device__ constexpr int col_bit(int c) { return 4 * ((c >> 4) & 3) + 2 * ((c >> 3) & 1); }

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// code * 2^b exactly, from a word with the code at bits b, b + 1 (b <= 14)
__device__ __forceinline__ float2 codes2(uint32_t w0, uint32_t w1, int b) {
  const float2 f = make_float2(__uint_as_float((w0 & (3u << b)) | kTwo23Bits),
                               __uint_as_float((w1 & (3u << b)) | kTwo23Bits));
  return __fadd2_rn(f, make_float2(-kTwo23, -kTwo23));
}

// One row from shared to global memory (bytes a multiple of 16), in this
// thread's current bulk group.
__device__ __forceinline__ void bulk_s2g(void* gmem_dst, const void* smem_src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(gmem_dst), "r"(smem_u32(smem_src)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void st_row32(void* p, uint4 lo, uint4 hi) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(lo.x), "r"(lo.y), "r"(lo.z),
               "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
               : "memory");
}

// 8 channels of a row (32-byte store pieces in float32, one 16-byte one in bf16)
template <bool F32>
__device__ __forceinline__ void store8(void* row, int c, const float* f, bool wide) {
  if constexpr (F32) {
    float* d = static_cast<float*>(row) + c;
    const uint4 lo = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    const uint4 hi = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    if (wide) {      // 32-byte aligned: whole sectors
      st_row32(d, lo, hi);
    } else {
      reinterpret_cast<uint4*>(d)[0] = lo;
      reinterpret_cast<uint4*>(d)[1] = hi;
    }
  } else {   // nearest even: the output type
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + c) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
}

// Tile u of the list: sequence, KV head, 128-token tile.
template <int MAXS>
__device__ __forceinline__ void locate_tile(const ReadParams<MAXS>& p, int64_t u, int& b, int& j, int& tile) {
  int lo = 0, hi = p.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.seq[mid].ubase <= u) lo = mid; else hi = mid - 1;
  }
  b = lo;
  const int64_t off = u - p.seq[b].ubase;
  const int64_t i = off / p.hkv;
  j = (int)(off - i * p.hkv);
  tile = p.seq[b].start / kGroup + (int)i;
}

template <int MAXS, bool M16, bool F32>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams<MAXS> p,
                                                            const uint8_t* __restrict__ arena) {
  using B = Blk<M16>;
  using MR = Meta<M16>;
  using Out = typename std::conditional<F32, float, uint16_t>::type;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using Smem = ReadSmem<M16, F32>;
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kReadStages; ++s) mbar_init(&S.full[s], 1);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  uint32_t* err = reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(arena));

  // requests the block of tile u (window tiles need none)
  auto request = [&](int64_t u, int s) {
    int b, j, tile;
    locate_tile(p, u, b, j, tile);
    if ((tile + 1) * (int64_t)kGroup > p.seq[b].len) {
      mbar_arrive(&S.full[s]);
      return;
    }
    const uint8_t* src =
        arena + p.blocks_off + (((int64_t)p.seq[b].slot * p.hkv + j) * p.max_groups + tile) * (int64_t)B::kBytes;
    if (p.fault && u == 0) return;
    mbar_arrive_expect_tx(&S.full[s], B::kBytes);
    bulk_g2s(S.stage[s], src, B::kBytes, &S.full[s]);
  };

  int64_t u = blockIdx.x;
  if (tid == 0 && u < p.n_tiles) request(u, 0);
  for (uint32_t it = 0; u < p.n_tiles; ++it, u += gridDim.x) {
    const int s = it & 1;
    int b, j, tile;
    locate_tile(p, u, b, j, tile);
    const ReadSeq sq = p.seq[b];
    // rows of the outputs: token tile * 128 + t goes to row0 + t
    const int64_t row0 = sq.row0 + ((int64_t)tile * kGroup - sq.start);
    const int lo = max(0, sq.start - tile * kGroup);
    const int hi = (int)min((int64_t)kGroup, (int64_t)sq.end - (int64_t)tile * kGroup);
    Out* kout = static_cast<Out*>(p.k_out);
    Out* vout = static_cast<Out*>(p.v_out);
    auto out_row = [&](Out* base, int t) { return base + ((row0 + t) * p.hkv + j) * kHeadDim; };

    const bool late = !mbar_wait_bounded(&S.full[s], (it >> 1) & 1, &S.abort_flag, err, p.spin_limit);
    const bool packed = (tile + 1) * (int64_t)kGroup <= sq.len;
    const uint8_t* blk = S.stage[s];
    if (packed && tid < kHeadDim / 2) {
      const float f = exp2i(-col_bit(tid));
      S.kp[s][tid] = make_float4(MR::one(blk + B::kKScale, tid) * f, MR::one(blk + B::kKScale, tid + 64) * f,
                                 MR::one(blk + B::kKZero, tid), MR::one(blk + B::kKZero, tid + 64));
    }
    if (!packed) {
      // ---- window rows: 16 lanes a row
      const uint16_t* wk = reinterpret_cast<const uint16_t*>(arena + p.windows_off +
                                                             ((int64_t)sq.slot * p.hkv + j) * kWindowBytes);
      const uint16_t* wv = wk + kGroup * kHeadDim;
      for (int t = lo + (tid >> 4); t < hi; t += kReadThreads / 16) {
        const int c = 8 * (tid & 15);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          Out* base = kv ? vout : kout;
          if (base == nullptr) continue;
          const uint4 w = *reinterpret_cast<const uint4*>((kv ? wv : wk) + t * kHeadDim + c);
          if constexpr (F32) {
            const float f[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                                bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
            store8<true>(out_row(base, t), c, f, p.wide);
          } else {
            *reinterpret_cast<uint4*>(out_row(base, t) + c) = w;
          }
        }
      }
    } else if (vout != nullptr) {
      // ---- values: channels 8 c8 .. + 7, tokens of (token half jt, tig)
      const int c8 = lane & 15, x = 2 * warp + (lane >> 4);
      const int tig = x & 3, jt = x >> 2;
      const uint32_t* words = reinterpret_cast<const uint32_t*>(blk + B::kVCodes) +
                              ((((c8 >> 1) * 2 + jt) * 32 + tig) * 2 + (c8 & 1));
      uint32_t w[8];
#pragma unroll
      for (int g = 0; g < 8; ++g) w[g] = words[8 * g];
      const int t0 = 64 * jt + 2 * tig;      // this thread's tokens are t0 + 8 q + e
      const int m0 = t0 * 4 + (c8 >> 2);     // and their scales and zeros (see vmeta_row: e swaps where q is odd)
      Out* row0p = out_row(vout, t0) + 8 * c8;
      const int64_t pitch = (int64_t)p.hkv * kHeadDim;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (e) {
#pragma unroll
          for (int g = 0; g < 8; ++g) w[g] >>= 16;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {   // kk = q >> 1, hf = q & 1
          const int bit = 4 * (q >> 1) + 2 * (q & 1);
          const int at = m0 + 4 * (8 * q + (M16 ? e : e ^ (q & 1)));
          const float sc = MR::one(blk + B::kVScale, at) * exp2i(-bit), ze = MR::one(blk + B::kVZero, at);
          float f[8];
#pragma unroll
          for (int g = 0; g < 8; g += 2) {
            const float2 v = __ffma2_rn(codes2(w[g], w[g + 1], bit), make_float2(sc, sc), make_float2(ze, ze));
            f[g] = v.x;
            f[g + 1] = v.y;
          }
          const int t = t0 + 8 * q + e;
          if (t >= lo && t < hi) store8<F32>(row0p + (8 * q + e) * pitch, 0, f, p.wide);
        }
      }
    }

    // One barrier a tile: the parameter table is complete, and everyone is done
    // with the previous tile, whose stage takes the next one.
    if (__syncthreads_or(late)) {
      // a wait gave up: leave (no copy of a later tile has been requested; this
      // tile's gets its time, bounded)
      if (tid == 0)
        for (uint32_t n = 0; n < p.spin_limit; ++n)
          if (mbar_try_wait(&S.full[s], (it >> 1) & 1)) break;
      break;
    }
    if (tid == 0 && u + gridDim.x < p.n_tiles) request(u + gridDim.x, s ^ 1);

    if (packed && kout != nullptr) {
      // ---- keys: token tid
      const int t = tid, mt = t >> 4, r = (t >> 3) & 1, g = t & 7;
      const uint32_t* words = reinterpret_cast<const uint32_t*>(blk + kOffKCodes);
      float2 x[64];   // channels (c, c + 64)
#pragma unroll
      for (int tig = 0; tig < 4; ++tig) {
        uint32_t w0 = words[(mt * 32 + 4 * g + tig) * 4 + r];
        uint32_t w1 = words[(mt * 32 + 4 * g + tig) * 4 + 2 + r];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (e) {
            w0 >>= 16;
            w1 >>= 16;
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int c = 8 * q + 2 * tig + e;
            const float4 kp = S.kp[s][c];
            x[c] = __ffma2_rn(codes2(w0, w1, 4 * (q >> 1) + 2 * (q & 1)), make_float2(kp.x, kp.y),
                              make_float2(kp.z, kp.w));
          }
        }
      }
#pragma unroll
      for (int hb = 0; hb < 6; ++hb) {
#pragma unroll
        for (int n = 0; n < 32; ++n) {
          const int h = 1 << hb;
          const int i = ((n >> hb) << (hb + 1)) | (n & (h - 1));
          const float2 a = x[i], d = x[i + h];
          x[i] = __fadd2_rn(a, d);
          x[i + h] = __ffma2_rn(d, make_float2(-1.0f, -1.0f), a);   // a - d (no negated packed operand)
        }
      }
      // last stage within the pairs, times n / sqrt(128)
      const float n = MR::one(blk + B::kKNorm, t) * 0.088388347648318440550f;
#pragma unroll
      for (int i = 0; i < 64; ++i) x[i] = __fmul2_rn(x[i], make_float2(n, n));
      // (this thread's previous row has been read from shared memory)
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      uint8_t* srow = S.krow[t];
#pragma unroll
      for (int up = 0; up < 2; ++up) {
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[i] = up ? x[c + i].x - x[c + i].y : x[c + i].x + x[c + i].y;
          }
          store8<F32>(srow, 64 * up + c, f, false);
        }
      }
      if (t >= lo && t < hi) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        bulk_s2g(out_row(kout, t), srow, Smem::kRow);
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // the last rows are written
}

template <int MAXS, bool M16, bool F32>
cudaError_t launch_read_t(const ReadParams<MAXS>& p, const uint8_t* arena, int sms, cudaStream_t stream) {
  if (p.n_tiles <= 0) return cudaSuccess;
  const int smem = (int)sizeof(ReadSmem<M16, F32>);
  static bool attr_done[64] = {};
  cudaError_t e = ensure_smem_attr(read_kernel<MAXS, M16, F32>, smem, attr_done);
  if (e != cudaSuccess) return e;
  // resident blocks per SM: registers allow three, a float32 row buffer two
  const unsigned grid = (unsigned)std::min<int64_t>(p.n_tiles, (F32 ? 2 : 3) * (int64_t)sms);
  return launch_dependent(read_kernel<MAXS, M16, F32>, dim3(grid), dim3(kReadThreads), (size_t)smem, stream, 1, p, arena);
}

}  // namespace

template <int MAXS>
cudaError_t launch_read(const ReadParams<MAXS>& p, const uint8_t* arena, bool meta16, bool f32, int sms,
                        cudaStream_t stream) {
  if (meta16)
    return f32 ? launch_read_t<MAXS, true, true>(p, arena, sms, stream)
               : launch_read_t<MAXS, true, false>(p, arena, sms, stream);
  return f32 ? launch_read_t<MAXS, false, true>(p, arena, sms, stream)
             : launch_read_t<MAXS, false, false>(p, arena, sms, stream);
}

template cudaError_t launch_read<kDecodeSeqsSmall>(const ReadParams<kDecodeSeqsSmall>&, const uint8_t*, bool, bool,
                                                   int, cudaStream_t);
template cudaError_t launch_read<kReadSeqsLarge>(const ReadParams<kReadSeqsLarge>&, const uint8_t*, bool, bool,
                                                   int, cudaStream_t);

}  // namespace oscar
