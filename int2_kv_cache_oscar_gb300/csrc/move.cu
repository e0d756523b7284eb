// Sequences copied to other slots and compacted (sm_103a): group blocks,
// window rows and maxima, moved as they are.
//
//   copy (source and destination slots differ): a block of threads takes a
//     group's block of one KV head, 32 bytes a thread and load, and stores it to
//     every destination that wants it, so that forks of one sequence read it
//     once; its next block is on its way meanwhile.  Then the window rows and
//     the maxima, a (destination, KV head) at a time.
//   in place: destination i of the kept groups g_0 < g_1 < ... is a place at or
//     before g_i, so the blocks of a (slot, KV head) have to move in order.  They
//     do so in parallel over their bytes: a block of threads owns a slice of 128
//     to 512 bytes of every block, reads the slices of many groups, and after a
//     barrier writes them.  A read of group g_k, k > i, is never of place i <
//     g_k, so the reads of the next groups are requested before the writes.
// Bound by HBM: every moved byte is read and written once.  Four forks of 128K tokens
// (8 KV heads, 113 MB read, 453 written) 95 us a call, 99 without stores that leave the
// L2 first; half of 128K kept 21 us (57 MB; the kernel alone, caches cold, 19); blocks
// an SM: 4 as 6, 8 slower (120 us).
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace oscar {
namespace {

constexpr int kCopyThreads = 216;      // 432 pieces of 32 bytes, 344 with 16-bit metadata
constexpr int kCopyLoads = 2;
constexpr int kCopyBlocksPerSm = 6;

struct Piece {
  uint32_t w[8];
};

__device__ __forceinline__ Piece load32(const uint8_t* p) {
  Piece r;
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                 "=r"(r.w[7])
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ void store32(uint8_t* p, const Piece& r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
               "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
               : "memory");
}

// The same where more is written than the L2 cache holds: it leaves the cache first.
__device__ __forceinline__ void store32_passing(uint8_t* p, const Piece& r) {
  asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]),
               "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
               : "memory");
}

// Source group of destination group g of a task.
template <int TASKS, int RUNS>
__device__ __forceinline__ int source_group(const MoveParams<TASKS, RUNS>& p, const MoveTask& t, int g) {
  if (t.n_runs == 0) return g;
  int lo = t.run0, hi = t.run0 + t.n_runs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.run[mid].dst <= g) lo = mid; else hi = mid - 1;
  }
  return p.run[lo].src + (g - p.run[lo].dst);
}

// A block of the copy's list: its source, and where it goes.
struct CopyUnit {
  const uint8_t* src;
  int dst0, n_dst, g, j;
};

template <int TASKS, int RUNS>
__device__ __forceinline__ CopyUnit copy_unit(const MoveParams<TASKS, RUNS>& p, const uint8_t* blocks, int64_t u) {
  int lo = 0, hi = p.n_tasks - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.task[mid].ubase <= u) lo = mid; else hi = mid - 1;
  }
  const MoveTask t = p.task[lo];
  const int64_t off = u - t.ubase;
  CopyUnit r;
  r.j = (int)(off / t.groups);
  r.g = t.g0 + (int)(off - (int64_t)r.j * t.groups);
  r.src = blocks + (((int64_t)t.src * p.hkv + r.j) * p.max_groups + source_group(p, t, r.g)) * (int64_t)p.block_bytes;
  r.dst0 = t.dst0;
  r.n_dst = t.n_dst;
  return r;
}

template <int TASKS, int RUNS>
__global__ void __launch_bounds__(kCopyThreads, kCopyBlocksPerSm)
    copy_kernel(const __grid_constant__ MoveParams<TASKS, RUNS> p, uint8_t* __restrict__ arena) {
  grid_dependency_wait();
  allow_dependents();
  const int tid = threadIdx.x;
  uint8_t* blocks = arena + p.blocks_off;
  const int pieces = p.block_bytes / 32;
  Piece next[kCopyLoads];
  auto request = [&](const CopyUnit& c) {
#pragma unroll
    for (int i = 0; i < kCopyLoads; ++i)
      if (tid + i * kCopyThreads < pieces) next[i] = load32(c.src + 32 * (tid + i * kCopyThreads));
  };
  int64_t u = blockIdx.x;
  CopyUnit c;
  if (u < p.n_units) {
    c = copy_unit(p, blocks, u);
    request(c);
  }
  while (u < p.n_units) {
    const CopyUnit at = c;
    Piece now[kCopyLoads];
#pragma unroll
    for (int i = 0; i < kCopyLoads; ++i) now[i] = next[i];
    u += gridDim.x;
    if (u < p.n_units) {
      c = copy_unit(p, blocks, u);
      request(c);
    }
    // the destinations of a task are in descending order of their groups
    for (int d = at.dst0; d < at.dst0 + at.n_dst && p.dst[d].groups > at.g; ++d) {
      uint8_t* to = blocks + (((int64_t)p.dst[d].slot * p.hkv + at.j) * p.max_groups + at.g) * (int64_t)p.block_bytes;
#pragma unroll
      for (int i = 0; i < kCopyLoads; ++i)
        if (tid + i * kCopyThreads < pieces) {
          if (p.passing) store32_passing(to + 32 * (tid + i * kCopyThreads), now[i]);
          else store32(to + 32 * (tid + i * kCopyThreads), now[i]);
        }
    }
  }
  // ---- window rows (8 pieces a row) and maxima
  for (int64_t x = blockIdx.x; x < (int64_t)p.n_dst * p.hkv; x += gridDim.x) {
    const int d = (int)(x / p.hkv), j = (int)(x - (int64_t)d * p.hkv);
    const MoveDst to = p.dst[d];
    if (to.src == to.slot) continue;
    const int64_t from_row = (int64_t)to.src * p.hkv + j, to_row = (int64_t)to.slot * p.hkv + j;
    const uint8_t* ws = arena + p.windows_off + from_row * kWindowBytes;
    uint8_t* wd = arena + p.windows_off + to_row * kWindowBytes;
    const int n = 8 * to.wlen;
    for (int i = tid; i < 2 * n; i += kCopyThreads) {
      const int off = i < n ? 32 * i : kWindowBytes / 2 + 32 * (i - n);
      store32(wd + off, load32(ws + off));
    }
    if (tid < 2) {
      uint32_t* m = reinterpret_cast<uint32_t*>(arena + (tid ? p.zmax_off : kMetaHeader));
      m[to_row] = m[from_row];
    }
  }
}

constexpr int kPlaceThreads = 256;
constexpr int kPlaceLoads = 4;

template <int TASKS, int RUNS>
__global__ void __launch_bounds__(kPlaceThreads)
    compact_kernel(const __grid_constant__ MoveParams<TASKS, RUNS> p, uint8_t* arena, int lanes) {
  grid_dependency_wait();
  allow_dependents();
  // a (task, KV head, slice): thread = (group of a batch, 32-byte piece of the slice)
  const int pieces = p.block_bytes / 32, slices = (pieces + lanes - 1) / lanes;
  const int64_t x = blockIdx.x / slices;
  const MoveTask t = p.task[x / p.hkv];
  const int j = (int)(x % p.hkv);
  const int piece = (int)(blockIdx.x % slices) * lanes + (int)threadIdx.x % lanes;
  const int row = (int)threadIdx.x / lanes, rows = kPlaceThreads / lanes;
  const bool mine = piece < pieces;
  uint8_t* base = arena + p.blocks_off + ((int64_t)t.src * p.hkv + j) * p.max_groups * (int64_t)p.block_bytes + 32 * piece;
  const int end = t.g0 + t.groups, step = rows * kPlaceLoads;
  Piece next[kPlaceLoads];
  auto request = [&](int g0) {
#pragma unroll
    for (int i = 0; i < kPlaceLoads; ++i) {
      const int g = g0 + row + rows * i;
      if (mine && g < end) next[i] = load32(base + (int64_t)source_group(p, t, g) * p.block_bytes);
    }
  };
  request(t.g0);
  for (int g0 = t.g0; g0 < end; g0 += step) {
    Piece now[kPlaceLoads];
#pragma unroll
    for (int i = 0; i < kPlaceLoads; ++i) now[i] = next[i];
    if (g0 + step < end) request(g0 + step);
    __syncthreads();       // the slices of this batch have been read by everyone
#pragma unroll
    for (int i = 0; i < kPlaceLoads; ++i) {
      const int g = g0 + row + rows * i;
      if (mine && g < end) store32(base + (int64_t)g * p.block_bytes, now[i]);
    }
  }
}

}  // namespace

template <int TASKS, int RUNS>
cudaError_t launch_move(const MoveParams<TASKS, RUNS>& p, uint8_t* arena, int sms, cudaStream_t stream) {
  const int64_t most = std::max<int64_t>(p.n_units, (int64_t)p.n_dst * p.hkv);
  const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)kCopyBlocksPerSm * sms);
  if (grid == 0) return cudaSuccess;
  return launch_dependent(copy_kernel<TASKS, RUNS>, dim3(grid), dim3(kCopyThreads), 0, stream, 1, p, arena);
}

template <int TASKS, int RUNS>
cudaError_t launch_compact(const MoveParams<TASKS, RUNS>& p, uint8_t* arena, int sms, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.n_tasks * p.hkv;
  if (rows == 0) return cudaSuccess;
  // slices of 512 bytes, smaller ones where those leave SMs without work
  const int pieces = p.block_bytes / 32;
  int lanes = 16;
  while (lanes > 4 && rows * ((pieces + lanes - 1) / lanes) < sms) lanes /= 2;
  const int64_t grid = rows * ((pieces + lanes - 1) / lanes);
  return launch_dependent(compact_kernel<TASKS, RUNS>, dim3((unsigned)grid), dim3(kPlaceThreads), 0, stream, 1, p, arena,
                          lanes);
}

template cudaError_t launch_move<kMoveTasksSmall, kMoveRunsSmall>(const MoveParams<kMoveTasksSmall, kMoveRunsSmall>&,
                                                                 uint8_t*, int, cudaStream_t);
template cudaError_t launch_move<kMoveTasksLarge, kMoveRunsLarge>(const MoveParams<kMoveTasksLarge, kMoveRunsLarge>&,
                                                                 uint8_t*, int, cudaStream_t);
template cudaError_t launch_compact<kMoveTasksSmall, kMoveRunsSmall>(const MoveParams<kMoveTasksSmall, kMoveRunsSmall>&,
                                                                    uint8_t*, int, cudaStream_t);
template cudaError_t launch_compact<kMoveTasksLarge, kMoveRunsLarge>(const MoveParams<kMoveTasksLarge, kMoveRunsLarge>&,
                                                                    uint8_t*, int, cudaStream_t);

}  // namespace oscar
