// Kernel launchers called by the C ABI layer after host-side validation.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "realign_params.h"

namespace sd {

struct GreedyParams {
  const void *logits;
  int dtype;
  int64_t row_stride;
  int B, D, V;
  const int32_t *draft;
  int32_t *accept_len, *next_token, *target_tok;
  // workspace, one kAtomicLine-byte line per word: keys[r * kKeyStride] for
  // r < B*(D+1), counters[b * kCountStride] for b < B
  unsigned long long *keys;
  unsigned int *counters;
  int32_t *status;
  bool vec;                   // 16-byte aligned rows: vector loads
  // trees (launch_verify_tree_greedy): D + 1 nodes per row
  const int32_t *parent;      // [B][D+1]
  int32_t *path;              // [B][depth+1]
  int depth;                  // nodes below the root that a row accepts at most
};

// Words that many workgroups update with device-scope atomics each get a
// 128-byte line of their own: atomics that share a line are serialized by the
// memory system, so packed words queue for microseconds where a lone word's
// round trip takes a few hundred nanoseconds.
constexpr int kAtomicLine = 128;
constexpr int kKeyStride = kAtomicLine / 8;
constexpr int kCountStride = kAtomicLine / 4;

// Trees of drafted tokens (see tree_common.h).
constexpr int kMaxNodes = 256;           // nodes of a tree
constexpr int kMaxTreeLen = 1 << 30;     // content positions a tree's root may stand at
constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 16;          // tokens one rotary workgroup turns at most

// Tree attention.
constexpr int kMaxAttnRows = 1024;       // batch rows (every wave reads all their lengths, 64 at a time)

// Query rows of a workgroup: rw waves of rt 16-row tiles, times kw waves that
// take other keys; the head size is padded to dhp.
struct AttnShape {
  int dhp, rt, rw, kw;
  int rows() const { return rw * rt * 16; }
  // a part's results in the workspace: per query row O, then max and sum
  size_t part_bytes() const { return (size_t)rows() * (dhp + 4) * 4; }
};

// Whether waves of an instance share keys through LDS (of which three tiles and
// more have to fit), and the waves that take other keys beside four that share.
constexpr bool attn_shared(int dtype, int dhp) { return !(dtype == 0 && dhp == 256); }
constexpr int attn_share_keys(int dtype, int dhp) { return dhp * (dtype == 0 ? 2 : 1) <= 128 ? 2 : 1; }
// Tiles in 128 KiB of LDS (per key wave), at most eight.
constexpr int attn_stages(int bytes) { return 131072 / bytes >= 8 ? 8 : 131072 / bytes; }
// Workgroups per CU of four waves that share none: two of 256 registers, or one
// of 512 where the keys of a tile or two take more.
constexpr int attn_direct_wgs(int dtype, int dhp) { return dhp * (dtype == 0 ? 2 : 1) <= 128 ? 2 : 1; }
// 16-row query tiles that a wave holds at most.
constexpr int attn_most_tiles(int dtype, int dhp) { return dhp * (dtype == 0 ? 2 : 1) <= 128 ? 2 : 1; }
AttnShape attn_shape(int dtype, int Dh, int M);
int attn_resident(int dtype, const AttnShape &a);  // workgroups that the device holds at once

struct TreeAttnParams {
  const void *q;                         // strided (row, node, query head), Dh contiguous
  void *out;
  int64_t qs[3], os[3];                  // in elements
  const void *k_old, *v_old;             // this layer's K and V: rows of Dh elements
  const void *k_new, *v_new;             // [B][H][N][Dh]
  const int32_t *table;                  // paged: [n_rows][max_blocks], else NULL
  int max_blocks, page, n_pages;
  const int32_t *len, *rows, *width;     // [n_rows]; [B] or NULL; rectangle widths or NULL
  int n_rows, cap, group;
  const int32_t *parent;                 // [B][N]
  int B, N, H, G, Dh;
  float scale;                           // its size times log2(e)
  bool negate;                           // it was negative
  unsigned int *counters;                // workspace: a line per slot, zero between calls
  int4 *cuts;                            // the number of segments in several parts, then (first part's slot, parts, row, segment)
  void *partial;
  int partial_bytes, blocks, resident, grid;  // query blocks per head, workgroups
  int32_t *status;
  FastDiv page_div, g_div;
};

struct TreePosParams {
  const int32_t *parent, *len, *rows;    // [B][N], [n_rows], [B] (nullable = identity)
  int B, N, n_rows;
  int32_t *pos, *status;                 // [B][N]
};

struct RopeParams {
  const void *x;
  void *out;
  int64_t xs[3], os[3];                  // strides of row, node, head in elements
  int dtype, B, N, heads, Dh, rot;
  const int32_t *pos;                    // [B][N]
  const double *freq;                    // [rot / 2] radians per position
  float factor;
  bool interleaved;
  int ve;                                // elements per access that pointers and strides allow (1 to 16 bytes)
  int tokens;                            // per workgroup (set by the launcher, with the divisors)
  FastDiv half_div, head_div, token_div, node_div;
};

struct CompactParams {
  const void *kv_new;                    // [seqs / H][B][H][N][units * 16 bytes]
  void *kv_path;                         // [seqs / H][B][H][depth + 1][units * 16 bytes]
  int seqs, B, H, N, depth, units;       // seqs = layers * 2 * heads
  const int32_t *draft, *path, *accept_len;  // [B][N], [B][depth + 1], [B]
  int32_t *draft_path, *status;          // [B][depth]
  FastDiv unit_div, head_div;
};

struct SampleParams {
  const float *p, *q;
  int B, D, V;
  int R, S;                   // ids per run, splits (workgroups) per batch row
  const int32_t *draft;
  const float *u_accept, *u_draw;
  int32_t *accept_len, *next_token, *status;
  // workspace: one block of kSampleRowBytes per batch row, at a place that
  // depends on the row alone: a counter line (zero between calls), then the
  // (residual, p) mass of each of the row's S splits (kSampleSplits slots),
  // then of each of its S * kSampleThreads runs
  char *ws;
};

constexpr int kSampleThreads = 256;  // threads per sampled-verification workgroup (one run each)
constexpr int kSampleSplits = 16;    // workgroups per batch row at most (runs grow with V beyond 32768)
constexpr size_t kSampleRowBytes = kAtomicLine + (size_t)kSampleSplits * 16 + (size_t)kSampleSplits * kSampleThreads * 16;
void sample_shape(int V, int &R, int &S);

struct TreeSampleParams {
  const float *p;             // [B][N][V]
  int B, N, V, depth;
  int R, S;                   // as for sampled verification of a chain, the workspace too
  const int32_t *draft, *parent;         // [B][N]
  const float *u_accept, *u_draw;        // [B][N]
  int32_t *accept_len, *next_token, *path, *status;
  char *ws;
};

struct SampleLogitsParams {
  const void *target, *draftl;  // logits [B][D+1][V] and [B][D][V] of `dtype`
  int dtype, B, D, V;
  int S;                        // splits of kSlChunk logits per stop row (mass and draw)
  int Ss;                       // splits of kSlStatChunk logits per row (statistics)
  double inv_t;                 // 1 / temperature
  float top_p;                  // nucleus mass, in (0, 1]
  bool nucleus;                 // top_p < 1: cut every row to its nucleus
  bool vec;                     // rows 16-byte aligned: vector loads
  const int32_t *draft;
  const float *u_accept, *u_draw;
  int32_t *accept_len, *next_token, *status;
  double *stats;                // workspace [B][2D+1][Ss] x (max, exp-sum)
  float *gath;                  // workspace [B][D] x (target logit, draft logit) at the draft token
  double *part;                 // workspace [B][S] x (residual mass, target mass) of the stop row
  double *thr;                  // workspace [B][S][kSlThreads] x the same per thread run
  double *rowinfo;              // workspace [B] x 8: (M, 1/Z) of the stop row's target and draft rows,
                                // their nucleus thresholds, the draw's uniform, the stop position
  double *nuc;                  // workspace [B][2D+1] x 4: (M, 1/Z, threshold) of every nucleus
  float *cutoff;                // optional out [B][2D+1]: every row's threshold (-inf: no nucleus)
};

// Sampled verification from logits.  The statistics kernel reads each row in
// splits of kSlStatChunk logits (kSlStatThreads threads of kSlStatPer logits);
// the mass and draw kernels cut the stop row into splits of kSlChunk logits, a
// run of kSlChunk / kSlThreads consecutive ids per thread.  Compile-time knobs
// (measured defaults).
#ifndef SPECDEC_SL_STAT_THREADS
#define SPECDEC_SL_STAT_THREADS 256
#endif
#ifndef SPECDEC_SL_STAT_PER
#define SPECDEC_SL_STAT_PER 16
#endif
#ifndef SPECDEC_SL_THREADS
#define SPECDEC_SL_THREADS 512
#endif
#ifndef SPECDEC_SL_CHUNK
#define SPECDEC_SL_CHUNK 4096
#endif
constexpr int kSlStatThreads = SPECDEC_SL_STAT_THREADS;
constexpr int kSlStatPer = SPECDEC_SL_STAT_PER;
constexpr int kSlStatChunk = kSlStatThreads * kSlStatPer;
constexpr int kSlChunk = SPECDEC_SL_CHUNK;
constexpr int kSlThreads = SPECDEC_SL_THREADS;



constexpr int kPagedAppend = 0, kPagedGather = 1, kPagedAdmit = 2, kPagedRetire = 3;
constexpr int kPagedMaxGrid = 4096;   // workgroups of one append or admit launch at most
// Arrival counting of append / admit: workgroups in groups of kArriveGroup
// consecutive ids, one counter line per group plus the root line (group
// sizes 8 to 64 measured alike on MI355X).
constexpr int kArriveGroup = 32;
constexpr int kSyncStride = kAtomicLine / 4;  // int32 words between two counters
constexpr int kPagedSyncWords = (1 + kPagedMaxGrid / kArriveGroup) * kSyncStride;

struct PagedParams {
  int op;                      // kPaged*
  void *pages;                 // [L][2][n_pages][H][page][units * 16 bytes]
  int32_t *bt;                 // [rows][max_blocks] page ids, -1 = none
  int32_t *free_pages;         // [n_pages] free-page stack
  int32_t *n_free;             // [1] entries of the stack in use
  int32_t *tokens;             // [rows][max_blocks * page]
  int32_t *len;                // [rows]
  int32_t *sync;               // [kPagedSyncWords] arrival counters of append / admit (one per
                               // kSyncStride words), zero between calls
  int layers, heads, units, n_pages, page, max_blocks, rows;
  const int32_t *rowmap;       // [B] pool row of each batch entry, nullable = identity
  int B, D;
  const void *kv_new;          // append: [L][2][B][H][D+1][units * 16 bytes]
  const int32_t *draft, *accept_len, *next_token;
  int32_t pad_token;
  // the rectangle side: the view an append writes, a gather's output, an admit's input
  void *rect_kv;               // [L][2][B][H][rect_cap][units * 16 bytes]
  int32_t *rect_tok, *rect_pos, *rect_len, *rect_width;
  int8_t *rect_mask;
  int rect_cap;
  const int32_t *in_len, *in_width;  // admit: content lengths [B] and the rectangle's width [1]
  int32_t *width_out;          // append: S'
  int32_t *status;
  int kv_wgs;                  // workgroups that copy KV (set by the launcher)
};

struct GroupParams {
  const int32_t *len;
  const int32_t *ids;          // nullable: entry i is pool row ids[i] (len read there, order lists ids)
  int N, group;
  int32_t *order, *uniform, *width, *n_uniform;
};

constexpr int kMaxPoolSlots = 4096;  // pool rows a grouping or a lifecycle call handles

struct PoolParams {
  // the pool (left-aligned rows)
  void *kv;                    // [L][2][slots][H][cap][units * 16 bytes]
  int32_t *tokens, *len;       // [slots][cap], [slots]
  int layers, heads, units, slots, cap;
  // scheduling state
  int32_t *active, *n_active, *free_slots, *n_free, *q_head;
  // finish
  const int32_t *rows, *accept_len;
  int B, D;
  int32_t eos_id, max_len;
  int32_t *retired, *n_retired;
  // admit: the prompt queue [L][2][Q][H][pcap][units * 16 bytes], tokens [Q][pcap], lengths [Q]
  const void *pkv;
  const int32_t *ptok, *plen;
  int Q, pcap;
  int32_t *admitted, *n_admitted;
  int32_t *status;
};

hipError_t launch_verify_greedy(const GreedyParams &p, hipStream_t s);
hipError_t launch_verify_tree_greedy(const GreedyParams &p, hipStream_t s);
hipError_t launch_verify_sample(const SampleParams &p, hipStream_t s);
hipError_t launch_verify_tree_sample(const TreeSampleParams &p, hipStream_t s);
hipError_t launch_verify_sample_logits(const SampleLogitsParams &p, hipStream_t s);
hipError_t launch_group_by_len(const GroupParams &p, hipStream_t s);
hipError_t launch_paged(const PagedParams &p, hipStream_t s);
hipError_t launch_pool_finish(const PoolParams &p, hipStream_t s);
hipError_t launch_pool_admit(const PoolParams &p, hipStream_t s);
hipError_t launch_tree_positions(const TreePosParams &p, hipStream_t s);
hipError_t launch_tree_attention_f32(const TreeAttnParams &p, hipStream_t s);
hipError_t launch_tree_attention_f16(const TreeAttnParams &p, hipStream_t s);
hipError_t launch_tree_attention_bf16(const TreeAttnParams &p, hipStream_t s);
hipError_t launch_rope(const RopeParams &p, hipStream_t s);
hipError_t launch_tree_compact(CompactParams p, hipStream_t s);
hipError_t launch_zero(void *ptr, size_t bytes, hipStream_t s);
hipError_t static_scratch(void **out, hipStream_t s);

}  // namespace sd
