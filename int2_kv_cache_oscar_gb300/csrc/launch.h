// Host-side launch interface between the C ABI (oscar_api.cu) and the kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace oscar {

// One 128-token group of one sequence that fills during an append (all KV
// heads run it, grid.y = head).  Tokens 0..n_win-1 of the group come from
// the window, the rest from input rows in_row, in_row + 1, ...  When
// tail_count > 0 the same CTA afterwards writes input rows tail_in_row ...
// into window positions tail_pos ... (the window it has just read).
struct QuantTask {
  int32_t slot;
  int32_t group;
  int32_t n_win;
  int32_t in_row;
  int32_t tail_pos;
  int32_t tail_count;
  int32_t tail_in_row;
  int32_t kind;  // 0 = quantise a group (+ optional tail), 1 = window append only
};

// A QuantTask as the kernel reads it, 16 bytes, so that a whole 128K-token
// append (1,024 tasks) fits in one launch's parameters:
//   a = slot | n_win << 24 | kind << 31   (kind 1: the n_win bits hold
//                                          tail_pos mod 128)
//   b = group | tail_count << 24
//   c = in_row, d = tail_in_row
// A kind-0 task's tail always starts on a group boundary (tail_pos mod 128
// = 0).  slot and group are below 2^24 (max_batch * Hkv <= 2^24; groups of
// an int32 length), n_win and tail_count below 128.
struct PackedTask {
  uint32_t a, b;
  int32_t c, d;
  __host__ __device__ int slot() const { return (int)(a & 0xFFFFFFu); }
  __host__ __device__ int kind() const { return (int)(a >> 31); }
  __host__ __device__ int n_win() const { return kind() ? 0 : (int)((a >> 24) & 0x7Fu); }
  __host__ __device__ int tail_pos_mod() const { return kind() ? (int)((a >> 24) & 0x7Fu) : 0; }
  __host__ __device__ int group() const { return (int)(b & 0xFFFFFFu); }
  __host__ __device__ int tail_count() const { return (int)((b >> 24) & 0x7Fu); }
  __host__ __device__ int in_row() const { return c; }
  __host__ __device__ int tail_in_row() const { return d; }
};
static_assert(sizeof(PackedTask) == 16, "16-byte tasks");

inline PackedTask pack_task(const QuantTask& t) {
  PackedTask p;
  const uint32_t low7 = (uint32_t)(t.kind ? (t.tail_pos & 127) : t.n_win) & 0x7Fu;
  p.a = ((uint32_t)t.slot & 0xFFFFFFu) | (low7 << 24) | ((uint32_t)(t.kind & 1) << 31);
  p.b = ((uint32_t)(t.kind ? 0 : t.group) & 0xFFFFFFu) | (((uint32_t)t.tail_count & 0x7Fu) << 24);
  p.c = t.in_row;
  p.d = t.tail_in_row;
  return p;
}

constexpr int kQuantPlanSmall = 64;
constexpr int kQuantPlanLarge = 2000;   // 32 + 2000 * 16 bytes of plan: within the 32,764-byte parameter limit

template <int CAP>
struct QuantPlan {
  int32_t n_tasks;
  int32_t hkv;
  int32_t max_groups;
  int32_t wide;          // 1: k and v are 32-byte aligned (32-byte row loads)
  int64_t blocks_off;
  int64_t windows_off;
  int64_t zmax_off;      // per (slot, head) largest |value zero| (float bits, atomicMax)
  PackedTask t[CAP];
};
static_assert(sizeof(QuantPlan<kQuantPlanLarge>) + 3 * sizeof(void*) <= 32764, "kernel parameter limit");

// meta16: the float16-metadata block layout (see include/oscar.h)
cudaError_t launch_quantize_small(const QuantPlan<kQuantPlanSmall>& plan, uint8_t* arena, const uint16_t* k,
                                  const uint16_t* v, bool meta16, cudaStream_t stream);
cudaError_t launch_quantize_large(const QuantPlan<kQuantPlanLarge>& plan, uint8_t* arena, const uint16_t* k,
                                  const uint16_t* v, bool meta16, cudaStream_t stream);

// ------------------------------------------------------------------ decode

// Per-sequence data of one decode launch.  Work units are (sequence, KV head,
// unit) triples in that order (a unit is one 128-token group of the INT2
// cache, or one 64-token tile of the bf16 reference cache); sequence b owns
// units [ubase, ubase + hkv * units_b).
struct DecodeSeq {
  int32_t slot;
  int32_t len;
  int64_t ubase;  // first unit of this sequence
  int32_t rank;   // number of earlier sequences with >= 1 unit
  // INT2: groups 0..settled-1 of each of this sequence's rows were written by
  // kernels that have completed before this launch can start (the host tracks
  // appends), so their blocks may be copied before the grid dependency wait
  int32_t settled;
};

struct DecodeHeader {
  int32_t n_seqs;
  int32_t hkv;
  int32_t gqa;           // query heads of each KV head served by this launch (<= kMaxGqa BF16, kMaxGqaInt2 INT2)
  int32_t hq;
  int32_t max_groups;    // INT2: groups per (slot, head); bf16: max_seq_len
  int32_t n_ctas;        // main-kernel CTAs (N)
  int32_t bf16_mode;     // 1: bf16 reference cache (64-token units, no window)
  int32_t q_group;       // query heads per KV head in the q / out layout (hq / hkv >= gqa)
  int64_t n_units;       // T
  int64_t blocks_off;
  int64_t windows_off;
  float scale_log2;      // softmax_scale * log2(e)
  int32_t q_head0;       // this launch's first query head within each KV head's group
  const uint16_t* q;
  uint16_t* out;
  float* partials;
  uint32_t* err_word;
  // fused append: when set, each (sequence, KV head) row's newest window
  // token (window row len mod 128 - 1) is taken from these [n_seqs, hkv, d]
  // bf16 rows instead of the arena, and stored into the arena window
  const uint16_t* k_new;
  const uint16_t* v_new;
  // combine staging, sized by the host for this launch: window rows (the
  // longest window of the batch) and bytes of partial records per chunk
  int32_t comb_wrows;
  int32_t comb_part_bytes;
  int32_t out_f32;       // the combine writes float32 outputs (else bf16)
  // bounded waits of the INT2 main kernel give up after this many polls; a
  // test of that path sets fault_unit >= 0: CTA 0's producer then leaves that
  // unit's copy unissued (its consumer's wait runs out), and a small limit
  uint32_t spin_limit;
  int32_t fault_unit;
  // INT2 over listed groups: a row's units are the n_sel entries of
  // groups[(sequence * hkv + head) * n_sel], an entry outside [0, groups of
  // the sequence) is skipped (NULL: a row's units are its groups)
  const int32_t* groups;
  int32_t n_sel;
  int32_t comb_row;      // listed groups: the combine's CTAs take a KV head (else a query head)
  float* lse;            // [n_seqs, hq] natural-log log-sum-exp of the rows, or NULL
  ScoreRule rule;        // every group only (not with `groups`)
};

template <int MAXS>
struct DecodeParams {
  DecodeHeader h;
  DecodeSeq seq[MAXS];
};

constexpr int kDecodeSeqsSmall = 16;
constexpr int kDecodeSeqsLarge = 1024;

// Floats of one partial record (o[128], m, l, 2 pad) per query head.
constexpr int kPartialFloats = 132;

// ------------------------------------------------------------------ rotary

// Rows of one tensor [n, heads, 128]: strides in bytes, in and out.
struct RotaryRows {
  const uint8_t* in;
  uint8_t* out;
  int64_t in_token, in_head;
  int64_t out_token, out_head;
  int32_t heads;
};

struct RotaryParams {
  RotaryRows q, k;            // heads 0: absent
  const int32_t* positions;   // [n]
  int64_t n;
  int32_t dim;                // rotated channels
  int32_t block_tokens;       // set by the launch: tokens of a block,
  int32_t step_tokens;        // and a thread's step from one of its rows to
  int32_t step_rows;          // the next, tokens and heads
  int32_t transpose;
  float factor;
  uint64_t freq[kHeadDim / 2];   // turns per position, 2^64 to the turn
};

cudaError_t launch_rotary(const RotaryParams& p, bool f32, bool interleaved, int sms, cudaStream_t stream);

// -------------------------------------------------------------------- read

// Tokens [start, end) of one sequence; its output rows begin at row0.  Tiles
// of 128 tokens (the last one may be the window) times KV heads, head fastest,
// are numbered from ubase.
struct ReadSeq {
  int32_t slot;
  int32_t len;
  int32_t start;
  int32_t end;
  int64_t row0;
  int64_t ubase;
};

constexpr int kReadSeqsLarge = 512;   // sequences of one launch (within the kernel parameter limit)

template <int MAXS>
struct ReadParams {
  int32_t n_seqs;      // sequences with a non-empty range
  int32_t hkv;
  int32_t max_groups;
  int32_t wide;        // 1: both outputs are 32-byte aligned (float32: 32-byte stores of
                       // values and window rows)
  int64_t blocks_off;
  int64_t windows_off;
  int64_t n_tiles;
  void* k_out;         // rows of 128 channels, or NULL
  void* v_out;
  int32_t late;        // 1: nothing of the kernel before this one is read or written over; it is
                       // waited for at the end only (that kernel has waited for those before it)
  int32_t reserved;
  int64_t row_pitch;   // elements from one row of an output to the next, and from
  int64_t head_pitch;  // one KV head to the next
  uint32_t spin_limit; // polls of a bounded wait; the test hook's `fault` (1) leaves
  int32_t fault;       // the copy of tile 0 unissued, with a small limit
  ReadSeq seq[MAXS];
};

template <int MAXS>
cudaError_t launch_read(const ReadParams<MAXS>& p, const uint8_t* arena, bool meta16, bool f32, int sms,
                        cudaStream_t stream);

// ------------------------------------------------------------------ select

struct IndexSeq {
  int32_t slot;
  int32_t first;   // groups [first, end) are summarised
  int32_t end;
};

template <int MAXS>
struct IndexParams {
  int32_t n_seqs;
  int32_t hkv;
  int32_t max_groups;
  int64_t blocks_off;
  uint2* codes;        // [slot][KV head][group][lane]: 4 channels' lowest and highest values
  float2* weights;     // [slot][KV head][group]: largest and smallest norm, times the step
  IndexSeq seq[MAXS];
};

struct SelectSeq {
  int32_t slot;
  int32_t ng;
};

template <int MAXS>
struct SelectParams {
  int32_t n_seqs;
  int32_t hkv;
  int32_t hq;
  int32_t q_group;
  int32_t max_groups;
  int32_t n_select;
  int32_t keep_first;
  int32_t keep_last;
  int32_t blocks;      // of a row (a cluster), set by the launch
  int32_t stages;      // copies in flight and the bytes of each, set by the launch
  int32_t stage_bytes;
  uint32_t spin_limit; // as in ReadParams; `fault`: chunk 0 of block 0
  int32_t fault;
  uint32_t* err_word;
  const uint2* codes;
  const float2* weights;
  const uint16_t* q;   // [n_seqs, hq, 128]
  int32_t* out;        // [n_seqs, hkv, n_select]
  SelectSeq seq[MAXS];
};

constexpr int kSelectSeqsSmall = 64;     // a small launch's sequences (index and selection)
constexpr int kSelectMaxSmem = 224 * 1024;
constexpr int kSelectMaxHeads = 64;       // query heads per KV head
constexpr int kSelectMaxGroups = 12000;   // groups of a sequence to choose among (their keys in shared memory)
constexpr int kSelMaxBlocks = 8;          // blocks of a row

template <int MAXS>
cudaError_t launch_index(const IndexParams<MAXS>& p, const uint8_t* arena, bool meta16, cudaStream_t stream);
template <int MAXS>
cudaError_t launch_select(const SelectParams<MAXS>& p, int sms, cudaStream_t stream);

// ----------------------------------------------------------------- prefill

// One chunked-prefill attention launch: n_q queries of one sequence against
// every token in its cache.  Rows are (query, head) pairs, query-major.
struct PrefillParams {
  int32_t slot;
  int32_t hkv;
  int32_t gqa;
  int32_t hq;
  int32_t rows;          // n_q * gqa (per KV head)
  int32_t ng;            // full groups in the cache
  int32_t wlen;          // window tokens
  int32_t max_groups;
  int64_t blocks_off;
  int64_t windows_off;
  int64_t zmax_off;      // per (slot, head) largest |value zero| quantised so far (float bits)
  float scale_log2;      // softmax_scale * log2(e)
  ScoreRule rule;
  int32_t n_parts;       // the groups are split into this many parts (grid.z); 1: no split
  const uint16_t* q;     // [n_q, hq, d] bf16
  uint16_t* out;         // [n_q, hq, d] bf16
  float* lse;            // [n_q, hq] fp32 natural-log log-sum-exp, or NULL
  uint32_t* err_word;
  // n_parts > 1: partial records [part][KV head][row][kPrefillRecFloats]
  // (o unnormalised = sum p v, then m in log2 units and l), merged by a
  // second kernel
  float* parts;
};

// Floats of one partial prefill record (o[128], m, l, 2 pad).
constexpr int kPrefillRecFloats = 132;

cudaError_t launch_prefill(const PrefillParams& p, const uint8_t* arena, bool meta16, cudaStream_t stream);
// the tcgen05 history kernel (prefill_tc.cu); launch_prefill adds the merge of split parts
cudaError_t launch_prefill_tc(const PrefillParams& p, const uint8_t* arena, bool meta16, cudaStream_t stream);

// -------------------------------------------------------------------- move

// Groups g0 .. g0 + groups - 1 of the destinations dst0 .. dst0 + n_dst - 1 of
// one source slot: the same groups of the source, or (n_runs > 0) those of its
// runs.  A copy's units are (KV head, group), numbered from ubase.
struct MoveTask {
  int32_t src;
  int32_t dst0, n_dst;
  int32_t g0, groups;
  int32_t run0, n_runs;
  int64_t ubase;
};

struct MoveDst {
  int32_t src, slot;     // equal: compacted in place (window and maxima stay)
  int32_t groups;        // of the destination; a task's destinations in descending order
  int32_t wlen;          // window rows copied
};

struct MoveRun {         // destination groups dst, dst + 1, ... are source groups src, src + 1, ...
  int32_t dst, src;
};

template <int TASKS, int RUNS>
struct MoveParams {
  int32_t n_tasks;
  int32_t n_dst;
  int32_t hkv;
  int32_t max_groups;
  int32_t block_bytes;
  int32_t passing;       // a copy writes more than the L2 cache keeps
  int64_t n_units;
  int64_t blocks_off;
  int64_t windows_off;
  int64_t zmax_off;
  MoveTask task[TASKS];
  MoveDst dst[TASKS];
  MoveRun run[RUNS];
};

constexpr int kMoveTasksSmall = 32, kMoveRunsSmall = 64;
constexpr int kMoveTasksLarge = 400, kMoveRunsLarge = 1200;
static_assert(sizeof(MoveParams<kMoveTasksLarge, kMoveRunsLarge>) + 16 <= 32764, "kernel parameter limit");

template <int TASKS, int RUNS>
cudaError_t launch_move(const MoveParams<TASKS, RUNS>& p, uint8_t* arena, int sms, cudaStream_t stream);
template <int TASKS, int RUNS>
cudaError_t launch_compact(const MoveParams<TASKS, RUNS>& p, uint8_t* arena, int sms, cudaStream_t stream);

// ------------------------------------------------------------------- chunk

// One document of a packed chunk: its first token, tokens, the prefix that
// every token sees, and the first of its row tiles in the launch.
struct ChunkSeq {
  int32_t row0;
  int32_t len;
  int32_t prefix;
  int32_t tbase;       // set by the launch
};

template <int MAXS>
struct ChunkParams {
  int32_t n_seqs;      // documents with tokens, the longest first
  int32_t hkv;
  int32_t gqa;
  int32_t hq;
  int32_t cta_rows;    // (token, head) rows of a piece of work, 128 or 256, and
  int32_t pieces;      // how many pieces; set by the launch
  int32_t whole_tokens;   // 128 rows are whole tokens: queries come by TMA; set by the launch
  uint32_t spin_limit; // polls of a bounded wait; the test hook's `fault` (1) leaves
  int32_t fault;       // the second copy of CTA 0 unissued, with a small limit
  float scale_log2;    // softmax_scale * log2(e)
  float cap_in;        // 2 softmax_scale log2(e) / cap
  float cap_out;       // -2 cap log2(e)
  float cap_log2;      // cap log2(e); 0: no cap
  float cap_near;      // softmax_scale / (0.6 cap): |raw score| times it up to 1 takes the polynomial
  float cap_c[5];      // of the raw score (x times a polynomial of x^2)
  float cap_d[3];      // the same of a shorter one, up to a quarter of the cap
  const float* slopes; // [hq], or NULL
  float slope_unit;    // log2(e) with a cap (scores in log2 units), score_unit / softmax_scale without
  float score_unit;    // what raw scores are taken times before the slopes: 1, under a scale so small that a slope
  float unit_log2;     // over it might overflow its power of two (the large block only); scale_log2 / score_unit
  int32_t late;        // short documents beside the tiled kernel of the same call, just before: nothing of its
                       // is read or written over, so it is waited for at the end only (it has waited for those
                       // before).  Here, where it moves no pair of the values above off 8 bytes: further up it
                       // made the capped kernel spill (8,192 capped tokens 453 -> 470 us)
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;   // strides in elements
  ScoreRule rule;              // as the kernel of short documents takes it
  const uint16_t* prior_out;   // [tokens, hq, 128], with prior_lse or both NULL
  const float* prior_lse;      // [tokens, hq]
  uint16_t* out;               // [tokens, hq, 128]
  float* lse;                  // [tokens, hq], or NULL
  ChunkSeq seq[MAXS];
  // row tiles in the order in which they are taken (document << 22 | tile), set by
  // the launch where there is one
  static constexpr int kOrder = MAXS <= kDecodeSeqsSmall ? 496 : 2000;
  int32_t sorted;
  uint32_t order[kOrder];
};

constexpr int kChunkShort = 32;    // documents of up to so many tokens are chunk_short.cu's

// Row tiles of a KV head in the tiled kernel's launch, and their rows.
int64_t chunk_tiles(const ChunkSeq* docs, int n, int gqa, int hkv, int sms, int32_t* cta_rows);
template <int MAXS>
cudaError_t launch_chunk(ChunkParams<MAXS>& p, int64_t tokens, int sms, cudaStream_t stream);
template <int MAXS>
cudaError_t launch_chunk_short(ChunkParams<MAXS>& p, cudaStream_t stream);

int num_sms(int device);
int decode_int2_ctas_per_sm();
int decode_bf16_ctas_per_sm();

template <int MAXS>
cudaError_t launch_decode_int2(const DecodeParams<MAXS>& p, const uint8_t* arena, bool meta16, cudaStream_t stream,
                               cudaEvent_t ev_start, cudaEvent_t ev_stop);
template <int MAXS>
cudaError_t launch_decode_bf16(const DecodeParams<MAXS>& p, const uint16_t* kc, const uint16_t* vc,
                               cudaStream_t stream, cudaEvent_t ev_start, cudaEvent_t ev_stop);
template <int MAXS>
cudaError_t launch_combine(const DecodeParams<MAXS>& p, const uint8_t* arena, cudaStream_t stream);

}  // namespace oscar
