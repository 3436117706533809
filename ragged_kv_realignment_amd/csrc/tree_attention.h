// Attention of a tree of drafted nodes over a row's cache and the nodes' own
// ancestors, for caches in pages, left-padded rectangles and pools.
//
// For node i of row b and query head h of KV head k = h / G:
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j),
// j over the row's cached positions [0, len) and the nodes from i to the root.
//
// The G N query rows of one (row, KV head) share its keys, so a wave multiplies
// them together with matrix instructions while the keys stream by once:
//  - S^T = K Q^T: a lane holds 8 consecutive elements of one key (16 bytes as
//    they lie in memory), which is the instruction's layout for K.
//  - The softmax weights come out as S^T, a lane holding one query and 8 keys of
//    a 32-key tile; with the contraction's keys numbered in that order the same
//    registers, rounded to the cache's type, are the operand of
//  - O^T += V^T P^T.  For it a lane loads, for each of its 8 keys, its NE =
//    Dh / 16 elements (a row of V is read by 16 lanes, whole), and 8 x NE
//    elements turn into NE operands by byte permutes: element e of all 8 keys is
//    the operand of the output rows dh = NE (lane mod 16) + e.
// The running maximum is only raised when some score passes it by more than
// 2^kSlack: below that the weights stay under 2^kSlack, exact enough in every
// type, and the accumulators need no rescaling.  Weights, sums and O are fp32.
// The weights are rounded to the cache's type for the second product (8 bits of
// mantissa for bf16); their sum is taken of the rounded ones, so the roundings
// mostly cancel in the quotient: against 64 bits the output is off by 2.2e-3 of
// its size (bf16), of which its own rounding is 1.7e-3.
//
// Two forms (attn_shape has the rule, with both measured):
//  - Few query rows: the waves of a workgroup take keys in turn, straight from
//    memory to registers, a tile ahead.  Bound by memory and by latency: 79 MB of
//    8 rows x 32 heads of 128 to 1024 positions in 22 us (3.5 TB/s; a large copy
//    reaches 5.1), of which the split's plan takes 1.5, the first loads 1.5, and
//    the parts' sums and joins at the end 5.
//  - More: keys pass once through a ring of tiles in LDS for all the waves of a
//    workgroup, by loads that write LDS directly.  Bound by instruction issue: per
//    32-key tile and 16 query rows 17 matrix instructions beside about 110 others.
//    16 sequences of 256 to 2048 positions, 8 heads of 96 query rows: 36 us, 82
//    MB; 2 of 40001 and 65537, 2 heads of 1024 query rows: 142 us, 686 TFLOP/s
//    (a large product of hipBLASLt: 1208), at which power takes the clock from 2.4
//    to 2.0 GHz.
//
// A segment that is cut into parts (see plan) leaves (max, sum, O) of each in the
// workspace.  In the first form the last workgroup to arrive adds them; in the
// second another kernel does.  Either adds in part order, so results do not depend
// on timing.  The order of completion in the first form uses the same scheme as
// verification: sums stored past the non-coherent L2 (sc1), completed (vmcnt)
// before the count, loaded only after the count has returned.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "coherent.h"
#include "device_common.h"
#include "launch.h"
#include "specdec.h"
#include "tree_common.h"
#include "wave_dpp.h"

namespace sd {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

namespace {

constexpr int kTile = 32;       // keys of a wave's step
constexpr float kSlack = 8.0f;  // log2 of the largest weight before the maximum is raised
constexpr int kWindow = 1024;   // page ids in LDS
constexpr int kMinUnits = 2;    // of a part (see plan)
constexpr int kJoin = 16;       // parts that one workgroup adds at once
constexpr float kLow = -1e30f;  // running maximum before the first key

template <int DT> constexpr int es() { return DT == 0 ? 4 : 2; }

// One matrix instruction of the cache's type: 16x16 outputs over 32 (2-byte
// types) or 16 (fp32: four instructions of 4) contracted elements, a and b
// holding 16 bytes per lane.
template <int DT>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == 1) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else if constexpr (DT == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[k]), __uint_as_float(b[k]), c, 0, 0, 0);
    return c;
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  if constexpr (DT == 1) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), f16x2));
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
  }
}

// The largest of eight scores; NaN, whose query's result is NaN in any case, stays.
// (fmaxf, which passes NaN over, would first canonicalise each operand.)
__device__ __forceinline__ float max8(f32x4 a, f32x4 b) {
  auto larger = [](float x, float y) { return __builtin_elementwise_maximum(x, y); };
  return larger(larger(larger(larger(a[0], a[1]), a[2]), larger(larger(a[3], b[0]), b[1])), larger(b[2], b[3]));
}

template <int DT>
__device__ __forceinline__ float widen(const char *p) {
  if constexpr (DT == 0) return *reinterpret_cast<const float *>(p);
  else if constexpr (DT == 1) return f16_bits_to_f32(*reinterpret_cast<const uint16_t *>(p));
  else return bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(p));
}

// Whether either 16-bit element of a dword (or the dword) has an exponent of all
// ones, in the sign bits of the result: one more unit of exponent carries there.
template <int DT>
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) {
  constexpr uint32_t kExp = DT == 0 ? 0x7F800000u : DT == 1 ? 0x7C007C00u : 0x7F807F80u;
  constexpr uint32_t kOne = DT == 0 ? 0x00800000u : DT == 1 ? 0x04000400u : 0x00800080u;
  return (w & kExp) + kOne;
}

// The dword with zero in the place of its elements that are not finite.
template <int DT>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  const uint32_t odd = odd_bits<DT>(w);
  if constexpr (DT == 0) {
    return odd & 0x80000000u ? 0u : w;
  } else {
    return (odd & 0x80000000u ? 0u : w & 0xFFFF0000u) | (odd & 0x8000u ? 0u : w & 0xFFFFu);
  }
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// 16-byte stores and loads of partial sums through the coherence point.
__device__ __forceinline__ void st_f4(__amdgpu_buffer_rsrc_t r, uint32_t off, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4v, v), r, off, 0, kCoherentPolicy);
}
__device__ __forceinline__ f32x4 ld_f4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kCoherentPolicy));
}

// Elements e .. e+7 (a, then d) of query row `row` of (b, h), times f.
template <int DT>
__device__ __forceinline__ void write_out(const TreeAttnParams &p, int b, int h, int row, int e, f32x4 a, f32x4 d, float f) {
  const int n = (int)fdiv((uint32_t)row, p.g_div), gq = row - n * p.G;
  char *dst = static_cast<char *>(p.out) + ((int64_t)b * p.os[0] + (int64_t)n * p.os[1] +
                                            (int64_t)(h * p.G + gq) * p.os[2] + e) * es<DT>();
  a *= f;
  d *= f;
  if constexpr (DT == 0) {
    *reinterpret_cast<f32x4 *>(dst) = a;
    if (e + 4 < p.Dh) *reinterpret_cast<f32x4 *>(dst + 16) = d;
  } else {
    *reinterpret_cast<u32x4 *>(dst) =
        u32x4{pack2<DT>(a[0], a[1]), pack2<DT>(a[2], a[3]), pack2<DT>(d[0], d[1]), pack2<DT>(d[2], d[3])};
  }
}

// The same unless the row's node is not part of the tree (anc: the nodes'
// ancestor bits).
template <int DT>
__device__ __forceinline__ void store_out(const TreeAttnParams &p, int b, int h, int row, int e, f32x4 a, f32x4 d, float f,
                                          const uint32_t (*anc)[kMaxNodes / 32]) {
  if (anc[fdiv((uint32_t)row, p.g_div)][0] & 1u) write_out<DT>(p, b, h, row, e, a, d, f);
}

// The values of V that are not finite, of the nodes of tiles [t0, t1) that query
// row `row` attends to, added to its elements e .. e+7: a weight is positive, so
// an infinity stays one of its sign.  (Slow, and never taken for finite values.)
template <int DT>
__device__ __forceinline__ void add_odd(const TreeAttnParams &p, const char *v, int row, int e, int Dh, int t0, int t1,
                                     const uint32_t (*anc)[kMaxNodes / 32], f32x4 &a, f32x4 &d) {
  const int n = (int)fdiv((uint32_t)row, p.g_div);
  for (int j = t0 > 0 ? t0 * kTile : 0; j < t1 * kTile && j <= n; ++j) {
    if (!((anc[n][j >> 5] >> (j & 31)) & 1u)) continue;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = e + k < Dh ? widen<DT>(v + ((size_t)j * Dh + e + k) * es<DT>()) : 0.0f;
      if (!(fabsf(x) < INFINITY)) (k < 4 ? a : d)[k & 3] += x;
    }
  }
}

}  // namespace

namespace {

// Ancestor bits of every node (itself included) from its raw parent, a node per
// thread, by pointer doubling in LDS: after round k a node holds the bits of 2^k
// generations and the pointer past them.  A node outside the tree gets none.
__device__ __forceinline__ void tree_parents(int N, int raw, int32_t *status, int *ptr, uint32_t (*anc)[kMaxNodes / 32]) {
  const int t = threadIdx.x, words = (N + 31) / 32;
  bool bad = false;
  if (t < N) {
    ptr[t] = node_parent(t, raw, bad);
    for (int k = 0; k < words; ++k) anc[t][k] = (t >> 5) == k ? 1u << (t & 31) : 0u;
  }
  if (bad) set_status(status, SPECDEC_S_TREE);
}
__device__ __forceinline__ void tree_ancestors(int N, int *ptr, uint32_t (*anc)[kMaxNodes / 32]) {
  const int t = threadIdx.x, words = (N + 31) / 32;
  for (int span = 1; span < N; span <<= 1) {
    __syncthreads();
    int q = 0;
    uint32_t up[kMaxNodes / 32] = {};
    if (t < N) {
      q = ptr[t];
      if (q > 0) {
        for (int k = 0; k < words; ++k) up[k] = anc[q][k];
        q = ptr[q];
      }
    }
    __syncthreads();
    if (t < N) {
      ptr[t] = q;
      for (int k = 0; k < words; ++k) anc[t][k] |= up[k];
    }
  }
  if (t < N) {
    for (int k = 0; k < words; ++k) anc[t][k] = ptr[t] < 0 ? 0u : k == 0 ? anc[t][k] | 1u : anc[t][k];
  }
  __syncthreads();
}

// Loads that write LDS directly: lane i's 16 bytes go to byte `to` (the same in all
// lanes) of LDS + 16 i.  They have no output register; wait_loads() waits for them.
// (The compiler, which would know the builtin's write to LDS, has every read of LDS
// wait for all of them, the next tiles' too.  It keeps nothing in M0 from one
// instruction to another; the s_nop is the wait state that a read of M0 needs after
// its write.)
__device__ __forceinline__ void load_lds(const void *from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(to) : "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}
// At most N of this wave's loads are still out (they return in order); N is
// rounded down to what the instruction can say.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N > 63 ? 63 : N) : "memory");
}
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <class T>
__device__ __forceinline__ T lds_read(uint32_t at) {
  return *(const __attribute__((address_space(3))) T *)(uintptr_t)at;
}

// How the pieces of a row of P are turned among its slots in LDS (256 bytes are
// all banks: two rows of 8 pieces, or 16 pieces of a longer row).
template <int P>
__device__ __forceinline__ int swz(int row) {
  return P == 8 ? (row >> 1) & 7 : row & 15;
}

// Waits for the queries, here instead of with every use in a loop (where the
// wait would cover the keys on their way), and flips their signs where the scale
// was negative.
template <int DT, int RT, int KS>
__device__ __forceinline__ void settle(u32x4 (&q)[RT][KS], bool negate) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int s = 0; s < KS; ++s) asm volatile("" : "+v"(q[rt][s]));
  if (!negate) return;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int s = 0; s < KS; ++s) q[rt][s] ^= (u32x4)(DT == 0 ? 0x80000000u : 0x80008000u);
}

// What one workgroup does: units [unit0, unit1) (of KW key tiles) of segment
// `seg` (head x query block) of batch row b; as the part of a segment in several
// parts, its slot in the workspace, the segment's first slot and its parts.
struct Chunk {
  int b, seg, row, len, start;
  int unit0, unit1;
  int slot, slot0, parts;  // slot -1: the whole segment
  int cut, cuts;           // its number among the segments in several parts; theirs (known to part 0)
};

// The split.  A segment (batch row, KV head, query block) is cut into parts of at
// most `u` units, and a workgroup takes one part: a part ends in about 4 us of
// sums, stores and joins, so no workgroup takes pieces of two segments.
//  - With fewer segments than resident workgroups, u is about the least for which
//    every part gets a resident workgroup (the estimate counts half a part lost
//    per segment, and grows by an eighth until the parts fit).
//  - With more, u is a resident workgroup's share of the work: long rows are cut
//    to it, the others stay whole, and the launch runs them as places fall free.
//  - Parts under kMinUnits gain nothing: one token over 300, 700, 2000 and 8000
//    positions of 8 heads takes 8.1, 9.9, 12.0 and 17.0 us with at least 4 units,
//    8.7, 8.9, 10.8 and 15.8 with 2, 7.9, 8.7, 12.1 and 16.6 with 1.
// Every wave works it out by itself from the lengths, 64 rows at a time, a row per
// lane.  Returns false where there is nothing for this workgroup.
template <int KW>
__device__ __forceinline__ bool plan(const TreeAttnParams &p, int HR, int tree_tiles, Chunk &k) {
  const int lane = threadIdx.x & (kWave - 1);
  struct Row {
    int row, len, start;
    bool bad;
    int units;
  };
  auto load = [&](int b0) {
    Row x{};
    const int b = b0 + lane;
    if (b < p.B) {
      x.row = p.rows ? p.rows[b] : b;
      const bool in = x.row >= 0 && x.row < p.n_rows;
      x.len = in ? p.len[x.row] : -1;
      x.start = p.width ? p.width[p.group > 0 ? b / p.group : 0] - x.len : 0;
      x.bad = x.len < 0 || x.start < 0 || (long long)x.start + x.len > p.cap;
      x.units = x.bad ? 0 : ((x.len + kTile - 1) / kTile + tree_tiles + KW - 1) / KW;
    }
    return x;
  };
  const Row one = load(0);  // all there is for B <= 64
  auto rows_at = [&](int b0) { return b0 ? load(b0) : one; };
  double total = 0.0;
  int longest = 0;
  bool bad = false;
  for (int b0 = 0; b0 < p.B; b0 += kWave) {
    const Row x = rows_at(b0);
    bad |= x.bad;
    total += wave_total_f64((double)x.units);
    longest = max(longest, x.units);
  }
  if (__any(bad) || total * HR >= 1073741824.0) {
    if (threadIdx.x == 0) set_status(p.status, SPECDEC_S_LEN_RANGE);
    if (threadIdx.x == 0 && blockIdx.x == 0) p.cuts[0].x = 0;
    return false;
  }
  const int segs = p.B * HR;
  const float room = p.resident > segs ? (float)p.resident - 0.5f * (float)segs : (float)p.resident;
  // rounded up past the float's errors: no fewer units than an even share
  int u = max((int)((float)total * (float)HR / room * 1.00001f) + 1, kMinUnits);
  auto parts_of = [&](int units) { return (int)((uint32_t)(units + u - 1) / (uint32_t)u); };
  int all = 0;
  for (int tries = 0;; ++tries) {
    all = 0;
    for (int b0 = 0; b0 < p.B; b0 += kWave) all += wave_total_i32(parts_of(rows_at(b0).units));
    all *= HR;
    if (all <= p.resident || p.resident <= segs || !__any(longest > u)) break;
    u = tries < 16 ? u + (u + 7) / 8 : 1 << 30;
  }
  // consecutive parts on one XCD (workgroups go to the 8 XCDs in turn)
  const int per_xcd = (all + 7) / 8, on_xcd = (int)(blockIdx.x >> 3);
  const int w = (int)(blockIdx.x & 7) * per_xcd + on_xcd;
  if (on_xcd >= per_xcd || w >= all) return false;
  // all parts, in order of batch row, head, key and query block; those of cut
  // segments have slots, in order of segment and key
  k.cuts = 0;
  if (w == 0)
    for (int b0 = 0; b0 < p.B; b0 += kWave) k.cuts += HR * __popcll(__ballot(parts_of(rows_at(b0).units) > 1));
  int before = 0, slots = 0, cuts = 0;
  for (int b0 = 0; b0 < p.B; b0 += kWave) {
    const Row x = rows_at(b0);
    const int n = parts_of(x.units), mine = n * HR, cut = n > 1 ? mine : 0;
    const int incl = wave_scan_i32(mine), icut = wave_scan_i32(cut);
    const unsigned long long hit = __ballot(before + incl > w);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      k.b = b0 + at;
      k.row = __builtin_amdgcn_readlane(x.row, at);
      k.len = __builtin_amdgcn_readlane(x.len, at);
      k.start = __builtin_amdgcn_readlane(x.start, at);
      const int units = __builtin_amdgcn_readlane(x.units, at), np = __builtin_amdgcn_readlane(n, at);
      const int rel = w - before - __builtin_amdgcn_readlane(incl - mine, at);
      // of a head: by part, then by query block, so that blocks that share keys
      // run side by side on one XCD and share its L2
      const int h = uniform((int)((uint32_t)rel / (uint32_t)(np * p.blocks))), in_head = rel - h * np * p.blocks;
      const int part = uniform((int)((uint32_t)in_head / (uint32_t)p.blocks));
      k.seg = h * p.blocks + in_head - part * p.blocks;
      // even parts: the first `units % np` are one longer
      const int each = uniform((int)((uint32_t)units / (uint32_t)np)), longer = units - each * np;
      k.unit0 = part * each + min(part, longer);
      k.unit1 = k.unit0 + each + (part < longer);
      k.parts = np;
      k.slot0 = np > 1 ? slots + __builtin_amdgcn_readlane(icut - cut, at) + k.seg * np : 0;
      k.slot = np > 1 ? k.slot0 + part : -1;
      k.cut = cuts + HR * __popcll(__ballot(n > 1) & ((1ull << at) - 1ull)) + k.seg;
      return true;
    }
    cuts += HR * __popcll(__ballot(n > 1));
    before += __builtin_amdgcn_readlane(incl, kWave - 1);
    slots += __builtin_amdgcn_readlane(icut, kWave - 1);
  }
  return false;
}

}  // namespace

// RT 16-query tiles per wave, RW waves across queries times KW across keys; DHP
// the head size, or with PAD the next of 64, 128 and 256.
template <int DT, int DHP, int RT, int RW, int KW, bool PAGED, bool PAD>
__global__ __launch_bounds__(RW * KW * kWave, RW > 1 ? (RW * KW + 3) / 4 : attn_direct_wgs(DT, DHP)) void k_tree_attention(TreeAttnParams p) {
  constexpr int NW = RW * KW, NT = NW * kWave;
  constexpr bool SHARED = RW > 1;         // keys pass through LDS, for the waves that share them
  constexpr int ES = es<DT>();
  constexpr bool NEXT = !SHARED && RT == 1 && DHP * ES <= 512;  // registers for a second tile
  constexpr int EL = 16 / ES;             // elements of a 16-byte piece
  constexpr int KS = DHP / (4 * EL);      // contraction steps of S (4 lane groups x EL elements)
  constexpr int NE = DHP / 16;            // elements of V a lane holds per key
  constexpr int VD = NE * ES / 4;         // dwords of them
  constexpr int ROWS = RW * RT * 16;      // query rows of a workgroup
  constexpr int LROW = DHP + 4;           // floats of an LDS row of O
  // LDS of the keys: per stage and key wave 32 rows of K, then of V
  constexpr int P = DHP * ES / 16;        // 16-byte pieces of a row
  constexpr int TILE_BYTES = 2 * kTile * P * 16;
  constexpr int ST = SHARED ? attn_stages(KW * TILE_BYTES) : 4, U = (ST - 1) / 2;
  constexpr int PASS = (kTile * P + RW * kWave - 1) / (RW * kWave);  // wave-loads of K (of V) that a wave makes at most
  constexpr int KEY_BYTES = SHARED ? ST * KW * TILE_BYTES : 0;
  constexpr int O_BYTES = KW > 1 ? NW * RT * 16 * LROW * 4 : 0;

  __shared__ uint32_t s_page[SHARED && PAGED ? kWindow : 1];
  __shared__ __align__(1024) char s_mem[KEY_BYTES > O_BYTES ? KEY_BYTES : O_BYTES > 0 ? O_BYTES : 16];
  __shared__ uint32_t s_anc[kMaxNodes][kMaxNodes / 32];
  __shared__ int s_ptr[kMaxNodes], s_last, s_odd, s_hole;
  __shared__ float s_ml[NW][RT * 16][2];

  const int t = threadIdx.x, lane = t & (kWave - 1), wave = uniform(t / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int kw = wave % KW, rw = wave / KW;
  const int N = p.N, G = p.G, H = p.H, Dh = PAD ? p.Dh : DHP, M = N * G;
  const int tree_tiles = (N + kTile - 1) / kTile;
  const int RB = p.blocks, HR = H * RB;
  const size_t row_bytes = (size_t)Dh * ES;

  // The split of the work (see plan).  Every wave finds it from the lengths.
  Chunk k;
  if (!plan<KW>(p, HR, tree_tiles, k)) return;
  if constexpr (SHARED) {  // for the kernel that joins the parts
    if (threadIdx.x == 0 && k.cuts >= 0 && blockIdx.x == 0) p.cuts[0].x = k.cuts;
    if (threadIdx.x == 0 && k.slot >= 0 && k.slot == k.slot0) p.cuts[1 + k.cut] = int4{k.slot0, k.parts, k.b, k.seg};
  }
  const int b = k.b, h = k.seg / RB, rb = k.seg - h * RB, r = k.row, len = k.len, start = k.start;
  const int cache_tiles = (len + kTile - 1) / kTile, tiles = cache_tiles + tree_tiles;
  const int t0 = k.unit0 * KW, t1 = min(tiles, k.unit1 * KW);

  // the tree's parents come with the first loads
  const bool need_anc = t1 > cache_tiles;
  int raw_parent = 0;
  if (need_anc && t < N) raw_parent = p.parent[(size_t)b * N + t];
  if (t == 0) s_odd = s_hole = 0;
  bool bad_page = false;

  // Key i of tile tl: the page id to look up, and its row index (in units of Dh
  // elements) from that.  Past the last key the last one is read again.  A bad
  // page's keys take no part: the read stays inside the cache.
  const uint32_t old0 = (uint32_t)((r * H + h) * p.cap + start), new0 = (uint32_t)((b * H + h) * N);
  const int *table = PAGED ? p.table + (size_t)r * p.max_blocks : nullptr;
  auto page_of = [&](int tl, int i) -> int {
    if constexpr (!PAGED) return 0;
    else return table[fdiv((uint32_t)max(min(tl * kTile + i, len - 1), 0), p.page_div)];
  };
  auto row_of = [&](int tl, int i, int page, bool &in) -> uint32_t {
    if (tl >= cache_tiles) return new0 + (uint32_t)min((tl - cache_tiles) * kTile + i, N - 1);
    const uint32_t pos = (uint32_t)min(tl * kTile + i, len - 1);
    if constexpr (!PAGED) return old0 + pos;
    else {
      in = (uint32_t)page < (uint32_t)p.n_pages;
      return ((in ? (uint32_t)page : 0u) * H + h) * p.page + (pos - fdiv(pos, p.page_div) * p.page);
    }
  };

  // queries of this wave: row rt * 16 + c of its block, 16 bytes per step
  u32x4 q[RT][KS];
  const int rbase = rb * ROWS + rw * RT * 16;
  auto load_q = [&] {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = rbase + rt * 16 + c;
      const int n = row < M ? (int)fdiv((uint32_t)row, p.g_div) : 0, gq = row - n * G;
      const char *src = static_cast<const char *>(p.q) +
                        ((int64_t)b * p.qs[0] + (int64_t)n * p.qs[1] + (int64_t)(h * G + gq) * p.qs[2]) * ES;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int dh = (s * 4 + g) * EL;
        q[rt][s] = row < M && (!PAD || dh < Dh) ? *reinterpret_cast<const u32x4 *>(src + dh * ES) : (u32x4)(0u);
      }
    }
  };

  f32x4 o[RT][NE];
  float m[RT];
  f32x4 l[RT];  // every element the sum of the query's weights (fp32: of this lane's)
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = kLow;
    l[rt] = (f32x4)(0.0f);
#pragma unroll
    for (int e = 0; e < NE; ++e) o[rt][e] = (f32x4)(0.0f);
  }

  // A tile's keys as the products take them: K of key kt * 16 + c, piece s * 4 +
  // g; V of keys kt * 16 + g * 4 + 0 .. 3, NE elements from c * NE.
  struct Keys {
    u32x4 k[2][KS];
    uint32_t v[8][VD];
  };
  auto split_v = [](uint32_t *v, const char *src, bool in, auto piece_in) {
    if constexpr (VD == 2) {
      const u32x2 w = in ? *reinterpret_cast<const u32x2 *>(src) : (u32x2)(0u);
      v[0] = w[0];
      v[1] = w[1];
    } else {
#pragma unroll
      for (int d = 0; d < VD / 4; ++d) {
        const u32x4 w = piece_in(d) ? *reinterpret_cast<const u32x4 *>(src + d * 16) : (u32x4)(0u);
#pragma unroll
        for (int y = 0; y < 4; ++y) v[d * 4 + y] = w[y];
      }
    }
  };
  auto load_k = [&](Keys &x, int tl, uint32_t rho) {
    const char *kb = static_cast<const char *>(tl < cache_tiles ? p.k_old : p.k_new);
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      const char *src = kb + (size_t)__shfl(rho, kt * 16 + c) * row_bytes + g * 16;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        x.k[kt][s] = !PAD || (s * 4 + g) * EL < Dh ? *reinterpret_cast<const u32x4 *>(src + s * 64) : (u32x4)(0u);
    }
  };
  auto load_v = [&](Keys &x, int tl, uint32_t rho) {
    const char *vb = static_cast<const char *>(tl < cache_tiles ? p.v_old : p.v_new);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      split_v(x.v[i], vb + (size_t)__shfl(rho, (i >> 2) * 16 + g * 4 + (i & 3)) * row_bytes + c * NE * ES,
              !PAD || c * NE < Dh, [&](int d) { return !PAD || c * NE + d * EL < Dh; });
  };
  // The parts of a tile's work.  s[rt][kt][y] is of query c and key kt * 16 + g * 4
  // + y: scores, then weights.
  using Scores = f32x4[RT][2];
  auto scores = [&](const Keys &x, Scores &s) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        s[rt][kt] = (f32x4)(0.0f);
#pragma unroll
        for (int y = 0; y < KS; ++y) s[rt][kt] = mma<DT>(x.k[kt][y], q[rt][y], s[rt][kt]);
      }
  };
  // Keys that exist (vm) and, in the tree, that are part of it: what other nodes
  // hold must not meet a zero weight as NaN.
  auto existing = [&](int tl, uint32_t vm) -> uint32_t {
    if (tl < cache_tiles) return vm;
    const int j = (tl - cache_tiles) * kTile + (lane & (kTile - 1));
    return vm & (uint32_t)__ballot(j < N && (s_anc[min(j, N - 1)][0] & 1u));
  };
  auto mask_scores = [&](Scores &s, int tl, uint32_t vm) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      uint32_t see = vm;
      if (tl >= cache_tiles) {
        const int row = rbase + rt * 16 + c;
        see = row < M ? s_anc[fdiv((uint32_t)row, p.g_div)][tl - cache_tiles] : 0u;
      }
      see >>= g * 4;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[rt][kt][y] = see & (1u << (kt * 16 + y)) ? s[rt][kt][y] : -INFINITY;
    }
  };
  auto mask_values = [&](Keys &x, int tl, uint32_t vm) {
    const uint32_t there = existing(tl, vm) >> (g * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t on = there & (1u << ((i >> 2) * 16 + (i & 3))) ? 0xFFFFFFFFu : 0u;
#pragma unroll
      for (int d = 0; d < VD; ++d) x.v[i][d] &= on;
    }
    // In the tree a node's V may only reach its descendants, but zero times
    // infinity is NaN: where a tile holds a value that is not finite, zero takes
    // its place here and the rows that attend to it add it at the end.
    if (tl >= cache_tiles) {
      uint32_t odd = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int d = 0; d < VD; ++d) odd |= odd_bits<DT>(x.v[i][d]);
      if (__any(odd & (DT == 0 ? 0x80000000u : 0x80008000u))) {
        s_odd = 1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int d = 0; d < VD; ++d) x.v[i][d] = finite_only<DT>(x.v[i][d]);
      }
    }
  };
  auto raise = [&](const Scores &s) {
    float top[RT];
    bool up = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      top[rt] = max8(s[rt][0], s[rt][1]) * p.scale;
      up |= top[rt] > m[rt] + kSlack;
    }
    if (!__any(up)) return;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      top[rt] = fmaxf(top[rt], __shfl_xor(top[rt], 16));
      top[rt] = fmaxf(top[rt], __shfl_xor(top[rt], 32));
      const float to = fmaxf(m[rt], top[rt]), f = __builtin_amdgcn_exp2f(m[rt] - to);
      m[rt] = to;
      l[rt] *= f;
#pragma unroll
      for (int e = 0; e < NE; ++e) o[rt][e] *= f;
    }
  };
  auto weights = [&](Scores &s, u32x4 (&w)[RT]) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[rt][kt][y] = __builtin_amdgcn_exp2f(fmaf(s[rt][kt][y], p.scale, -m[rt]));
      if constexpr (DT == 0) {
        l[rt][0] += ((s[rt][0][0] + s[rt][0][1]) + (s[rt][0][2] + s[rt][0][3])) +
                    ((s[rt][1][0] + s[rt][1][1]) + (s[rt][1][2] + s[rt][1][3]));
      } else {
        w[rt] = u32x4{pack2<DT>(s[rt][0][0], s[rt][0][1]), pack2<DT>(s[rt][0][2], s[rt][0][3]),
                      pack2<DT>(s[rt][1][0], s[rt][1][1]), pack2<DT>(s[rt][1][2], s[rt][1][3])};
        // the sum of the rounded weights, by a product with ones: their roundings
        // then mostly cancel in the quotient
        constexpr uint32_t kOnes = DT == 1 ? 0x3C003C00u : 0x3F803F80u;
        l[rt] = mma<DT>((u32x4)(kOnes), w[rt], l[rt]);
      }
    }
  };
  // O^T += V^T P^T
  auto products = [&](const Keys &x, const Scores &s, const u32x4 (&w)[RT]) {
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            o[rt][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.v[i][e]), s[rt][i >> 2][i & 3], o[rt][e], 0,
                                                            0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
        u32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = __builtin_amdgcn_perm(x.v[2 * i + 1][e / 2], x.v[2 * i][e / 2], sel);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) o[rt][e] = mma<DT>(a, w[rt], o[rt][e]);
      }
    }
  };
  const int whole_tiles = min(t1, len / kTile);

  if constexpr (!SHARED) {
    // Keys straight into registers.  While a tile is multiplied the next is on its
    // way, in registers of its own (NEXT) or in the same ones as they fall free.
    // Page ids are looked up one tile further ahead, before the loads that need
    // not wait for them (loads return in order).
    auto find = [&](int tl, bool &valid) -> uint32_t {
      const int i = lane & (kTile - 1);
      bool in = true;
      const uint32_t rho = row_of(tl, i, page_of(tl, i), in);
      bad_page |= !in;
      valid = in && (tl < cache_tiles ? tl * kTile + i < len : (tl - cache_tiles) * kTile + i < N);
      return rho;
    };
    Keys x0, x1;
    bool valid = false, valid_next = false;
    uint32_t rho = 0, rho_next = 0;
    int tl = t0 + kw;
    if (tl < t1) {
      rho = find(tl, valid);
      if (tl + KW < t1) rho_next = find(tl + KW, valid_next);
      load_q();
      load_k(x0, tl, rho);
      load_v(x0, tl, rho);
    }
    if (need_anc) {
      tree_parents(N, raw_parent, p.status, s_ptr, s_anc);
      tree_ancestors(N, s_ptr, s_anc);
    }
    settle<DT>(q, p.negate);
    uint32_t vm = (uint32_t)__ballot(valid);  // keys of the tile that exist
    auto step = [&](auto plain) {
      const uint32_t vm_now = vm, at_next = rho_next;
      const bool more = tl + KW < t1;
      vm = (uint32_t)__ballot(valid_next);
      if (tl + 2 * KW < t1) rho_next = find(tl + 2 * KW, valid_next);
      if constexpr (NEXT) {
        if (more) {
          load_k(x1, tl + KW, at_next);
          load_v(x1, tl + KW, at_next);
        }
      }
      Scores s;
      u32x4 w[RT];
      scores(x0, s);
      if constexpr (!NEXT) {
        if (more) load_k(x0, tl + KW, at_next);
      }
      if constexpr (!decltype(plain)::value) {
        mask_scores(s, tl, vm_now);
        mask_values(x0, tl, vm_now);
      }
      raise(s);
      weights(s, w);
      products(x0, s, w);
      if constexpr (NEXT) {
        x0 = x1;
      } else {
        if (more) load_v(x0, tl + KW, at_next);
      }
      tl += KW;
    };
    while (tl < whole_tiles && vm == 0xFFFFFFFFu) step(std::true_type{});
    while (tl < t1) step(std::false_type{});
  } else {
    // Keys through LDS, each piece loaded once for the RW waves that share it, by
    // loads that write LDS directly and hold no register.  A wave-load fills 64
    // slots of 16 bytes in a row; which piece of its row a slot holds is turned by
    // swz(row), so that the 16 rows that one read of K touches lie in different
    // banks.  LDS holds ST >= 2 U + 1 tiles (per key wave) in a ring.  A step
    // multiplies V of tile i and K of tile i + 1 and starts the loads of tile i + U +
    // 1; the waves meet every U steps, where the tiles up to i + U must have come and
    // nobody reads the ones before i any more.  Between, they drift apart, and one's
    // softmax runs beside another's products.
    const int in_group = rw * kWave + lane;
    auto tile_of = [&](int i) { return t0 + kw + i * KW; };
    const int mine = tile_of(0) < t1 ? (t1 - tile_of(0) + KW - 1) / KW : 0;  // tiles of this key wave
    const int steps = (t1 - t0 + KW - 1) / KW;
    // The page ids of the next kWindow blocks (as row indexes) are kept in LDS:
    // looked up tile by tile they would return in order with the keys that are on
    // their way.
    int window = 0, filled = 0;  // its first block; the first tile that is not all in it
    const uint32_t lds0 = lds_offset(s_mem) + kw * TILE_BYTES;
    // The page ids of tiles i0 .. i1 are in the window.  Every wave of the
    // workgroup comes here, past a barrier: the window moves for all together.
    auto need_pages = [&](int i0, int i1) {
      const int first = t0 + i0 * KW, end = min(t0 + (i1 + 1) * KW, cache_tiles);
      if (!PAGED || first >= end || end <= filled) return;
      window = (int)fdiv((uint32_t)(first * kTile), p.page_div);
      const int blocks = (int)fdiv((uint32_t)(len - 1), p.page_div) + 1, n = min(kWindow, blocks - window);
      for (int i = t; i < n; i += NT) {
        const int page = table[window + i];
        const bool in = (uint32_t)page < (uint32_t)p.n_pages;
        if (!in) bad_page = s_hole = true;
        s_page[i] = ((in ? (uint32_t)page : 0u) * H + h) * p.page;
      }
      filled = window + n == blocks ? cache_tiles : (window + n) * p.page / kTile;
      barrier();
    };
    static_assert(PASS <= 2, "two rows of K, and of V, per lane and tile");
    // This lane's rows of the tile to be fetched next: position, block and place in
    // it, moved on from tile to tile; past the last key the last one is read again.
    const int by = KW * kTile, by_blocks = PAGED ? (int)fdiv((uint32_t)by, p.page_div) : 0, by_rest = by - by_blocks * p.page;
    const int end_block = PAGED && len > 0 ? (int)fdiv((uint32_t)(len - 1), p.page_div) : 0;
    const int end_slot = len - 1 - end_block * p.page;
    int pos[PASS], blk[PASS], slot[PASS];
#pragma unroll
    for (int j = 0; j < PASS; ++j) {
      pos[j] = tile_of(0) * kTile + (in_group + j * RW * kWave) / P;
      blk[j] = PAGED ? (int)fdiv((uint32_t)pos[j], p.page_div) : 0;
      slot[j] = pos[j] - blk[j] * p.page;
    }
    // the rows of the blocks that those lie in
    auto pages = [&](uint32_t (&at)[PASS]) {
#pragma unroll
      for (int j = 0; j < PASS; ++j)  // (tiles of the tree need none, and may find no window)
        at[j] = PAGED ? s_page[min((uint32_t)((pos[j] < len ? blk[j] : end_block) - window), kWindow - 1u)] : 0u;
    };
    // the loads of tile i, with those
    auto fetch = [&](int i, const uint32_t (&page)[PASS]) {
      const int tl = tile_of(i);
      const bool is_old = tl < cache_tiles;
      const char *kb = static_cast<const char *>(is_old ? p.k_old : p.k_new);
      const char *vb = static_cast<const char *>(is_old ? p.v_old : p.v_new);
      const uint32_t to = lds0 + (uint32_t)((i % ST) * KW * TILE_BYTES + rw * (kWave * 16));
#pragma unroll
      for (int j = 0; j < PASS; ++j) {
        const int row = (in_group + j * RW * kWave) / P;
        if (kTile * P % (RW * kWave) != 0 && row >= kTile) break;  // whole waves, where RW is 6
        const int piece = (in_group + j * RW * kWave) % P ^ swz<P>(row);
        uint32_t rho;
        if (!is_old) rho = new0 + (uint32_t)min((tl - cache_tiles) * kTile + row, N - 1);
        else if constexpr (PAGED) rho = page[j] + (uint32_t)(pos[j] < len ? slot[j] : end_slot);
        else rho = old0 + (uint32_t)min(pos[j], len - 1);
        if (i < mine && (!PAD || piece * EL < Dh)) {
          load_lds(kb + piece * 16 + (size_t)rho * row_bytes, to + j * RW * kWave * 16);
          load_lds(vb + piece * 16 + (size_t)rho * row_bytes, to + j * RW * kWave * 16 + kTile * P * 16);
        }
        pos[j] += by;
        if constexpr (PAGED) {
          blk[j] += by_blocks;
          slot[j] += by_rest;
          const bool next = slot[j] >= p.page;
          blk[j] += next;
          slot[j] -= next ? p.page : 0;
        }
      }
    };
    // Where this lane's pieces lie: K of row c, piece g of step 0 (step s: bits of
    // 64 s turned), V of row g * 4 and its first piece (row g * 4 + i: bits of 16 i
    // turned, i rows on; piece d likewise).  Tiles start at multiples of 1 KiB.
    constexpr int HALF = 16 * P * 16;  // bytes from a tile's first 16 rows to its others
    const uint32_t k_at = (uint32_t)(c * P * 16 + ((g ^ swz<P>(c)) << 4));
    const uint32_t v_at = (uint32_t)((kTile + g * 4) * P * 16 + (((c * NE * ES >> 4) ^ swz<P>(g * 4)) << 4) + c * NE * ES % 16);
    auto read_k = [&](Keys &x, uint32_t tile) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t a = tile + (k_at ^ (64u * s));
        x.k[0][s] = lds_read<u32x4>(a);
        x.k[1][s] = lds_read<u32x4>(a + HALF);
      }
    };
    auto read_v = [&](Keys &x, uint32_t tile) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // row g * 4 + i: its turn is (g * 4 + i) & 15, or of two rows of 8 pieces (g * 2 + i / 2) & 7
        const uint32_t turn = (uint32_t)(P == 8 ? i >> 1 : i) * 16u;
#pragma unroll
        for (int d = 0; d < (VD < 4 ? 1 : VD / 4); ++d)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t a = tile + ((v_at ^ turn ^ (16u * d)) + i * P * 16 + y * HALF);
            if constexpr (VD == 2) {
              const u32x2 w = lds_read<u32x2>(a);
              x.v[y * 4 + i][0] = w[0];
              x.v[y * 4 + i][1] = w[1];
            } else {
              const u32x4 w = lds_read<u32x4>(a);
#pragma unroll
              for (int z = 0; z < 4; ++z) x.v[y * 4 + i][d * 4 + z] = w[z];
            }
          }
      }
    };
    if constexpr (PAD) {  // pieces past Dh are never written: they read as zeros
      for (int i = t; i < ST * KW * TILE_BYTES / 16; i += NT) reinterpret_cast<u32x4 *>(s_mem)[i] = (u32x4)(0u);
    }
    load_q();
    __syncthreads();  // s_hole, and the zeros
    need_pages(0, U);
    // the last waits for other loads: the keys on their way would be waited for too
    if (need_anc) tree_parents(N, raw_parent, p.status, s_ptr, s_anc);
    settle<DT>(q, p.negate);
#pragma unroll 1
    for (int i = 0; i <= U; ++i) {
      uint32_t page[PASS];
      pages(page);
      fetch(i, page);
    }
    if (need_anc) tree_ancestors(N, s_ptr, s_anc);
    // keys of a tile that exist: all but the last ones, unless some page was bad
    auto existing_keys = [&](int tl, bool hole) -> uint32_t {
      const int n = tl < cache_tiles ? len - tl * kTile : N - (tl - cache_tiles) * kTile;
      uint32_t vm = n >= kTile ? 0xFFFFFFFFu : (1u << n) - 1u;
      if (hole && tl < cache_tiles) {
        bool in = true;
        row_of(tl, lane & (kTile - 1), page_of(tl, lane & (kTile - 1)), in);
        vm &= (uint32_t)__ballot(in);
      }
      return vm;
    };
    Scores s;
    Keys x;
    auto tile_at = [&](int i) { return lds0 + (uint32_t)((i % ST) * KW * TILE_BYTES); };
    // of tile i, all but its weights
    auto begin = [&](int i, bool hole) {
      const int tl = tile_of(i);
      read_k(x, tile_at(i));
      scores(x, s);
      read_v(x, tile_at(i));
      const uint32_t vm = existing_keys(tl, hole);
      if (tl >= cache_tiles || vm != 0xFFFFFFFFu) {
        mask_scores(s, tl, vm);
        mask_values(x, tl, vm);
      }
      raise(s);
    };
    bool hole = false;
    int i = 0, due = 0;
    auto meet = [&] {
      due += U;
      wait_loads<0>();  // this wave's share of the tiles up to i + U
      barrier();        // the others', and all are past the tiles before i
      hole = uniform(s_hole) != 0;
      need_pages(i + U + 1, i + 2 * U);
    };
    meet();
    if (mine > 0) begin(0, hole);
    // A step reads the next tile's K while V is multiplied, and its V beside the
    // softmax, where there are registers for both.
    constexpr bool AHEAD = DHP * ES <= 256;
    for (; tile_of(i + 1) < whole_tiles; ++i) {  // whole tiles, and one after them
      if (i == due) meet();
      if (PAGED && hole) break;
      u32x4 w[RT];
      uint32_t page[PASS];
      pages(page);
      weights(s, w);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      if constexpr (AHEAD) read_k(x, tile_at(i + 1));
      __builtin_amdgcn_sched_barrier(0);
      products(x, s, w);
      fetch(i + U + 1, page);
      __builtin_amdgcn_sched_barrier(0);  // V's registers are free before K's fill
      if constexpr (!AHEAD) read_k(x, tile_at(i + 1));
      scores(x, s);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      read_v(x, tile_at(i + 1));
      __builtin_amdgcn_sched_barrier(0);
      raise(s);
    }
    for (; i < steps; ++i) {
      if (i == due) meet();
      if (i >= mine) continue;
      u32x4 w[RT];
      uint32_t page[PASS];
      pages(page);
      weights(s, w);
      fetch(i + U + 1, page);
      products(x, s, w);
      if (i + 1 < mine) begin(i + 1, hole);
    }
    __syncthreads();  // the keys' LDS is free
  }
  if (bad_page) set_status(p.status, SPECDEC_S_LEN_RANGE);

  // The end: every query's maximum and sum over lane groups and key waves, then
  // O over the key waves.
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float sum = l[rt][0];
    if constexpr (DT == 0) {
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
    }
    if (g == 0) {
      s_ml[wave][rt * 16 + c][0] = m[rt];
      s_ml[wave][rt * 16 + c][1] = sum;
    }
  }
  __syncthreads();
  const __amdgpu_buffer_rsrc_t wsr = coherent_rsrc(p.partial, p.partial_bytes);
  constexpr uint32_t kSlotBytes = ROWS * LROW * 4;  // per row: O, then max and sum (16-byte rows)
  const uint32_t slot = (uint32_t)k.slot * kSlotBytes;
  const bool odd = s_odd;
  const char *nv = static_cast<const char *>(p.v_new) + (size_t)(b * H + h) * N * row_bytes;
  // elements e .. e+7 of a block's row: to the output, or to the workspace
  auto finish = [&](int brow, int e, f32x4 a, f32x4 d, float mx, float sum) {
    const int row = rb * ROWS + brow;
    if (row >= M || e >= Dh) return;
    if (odd) add_odd<DT>(p, nv, row, e, Dh, t0 - cache_tiles, t1 - cache_tiles, s_anc, a, d);
    if (k.slot < 0) {
      store_out<DT>(p, b, h, row, e, a, d, 1.0f / sum, s_anc);
    } else {
      const uint32_t off = slot + (uint32_t)(brow * LROW) * 4u;
      if constexpr (SHARED) {
        char *to = static_cast<char *>(p.partial) + off;
        *reinterpret_cast<f32x4 *>(to + e * 4) = a;
        *reinterpret_cast<f32x4 *>(to + e * 4 + 16) = d;
        // a sum below zero says that the node is not part of the tree
        const bool out = need_anc && !(s_anc[fdiv((uint32_t)row, p.g_div)][0] & 1u);
        if (e == 0) *reinterpret_cast<f32x4 *>(to + DHP * 4) = f32x4{mx, out ? -1.0f : sum, 0.0f, 0.0f};
      } else {
        st_f4(wsr, off + (uint32_t)e * 4u, a);
        st_f4(wsr, off + (uint32_t)e * 4u + 16u, d);
        if (e == 0) st_f4(wsr, off + DHP * 4u, f32x4{mx, sum, 0.0f, 0.0f});
      }
    }
  };
  if constexpr (KW == 1) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float mx = m[rt], sum = s_ml[wave][rt * 16 + c][1];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < NE; e += NE < 8 ? NE : 8) {
          if constexpr (NE >= 8) {
            finish((rw * RT + rt) * 16 + c, (g * 4 + x) * NE + e,
                   f32x4{o[rt][e][x], o[rt][e + 1][x], o[rt][e + 2][x], o[rt][e + 3][x]},
                   f32x4{o[rt][e + 4][x], o[rt][e + 5][x], o[rt][e + 6][x], o[rt][e + 7][x]}, mx, sum);
          } else if (x % 2 == 0) {  // Dh = 64: eight elements are two rows of the product
            finish((rw * RT + rt) * 16 + c, (g * 4 + x) * NE,
                   f32x4{o[rt][0][x], o[rt][1][x], o[rt][2][x], o[rt][3][x]},
                   f32x4{o[rt][0][x + 1], o[rt][1][x + 1], o[rt][2][x + 1], o[rt][3][x + 1]}, mx, sum);
          }
        }
    }
  } else {
    float(*s_o)[RT * 16][LROW] = reinterpret_cast<float(*)[RT * 16][LROW]>(s_mem);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float top = kLow;
#pragma unroll
      for (int i = 0; i < KW; ++i) top = fmaxf(top, s_ml[rw * KW + i][rt * 16 + c][0]);
      const float f = __builtin_amdgcn_exp2f(m[rt] - top);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < NE; e += 4)
          *reinterpret_cast<f32x4 *>(&s_o[wave][rt * 16 + c][(g * 4 + x) * NE + e]) =
              f32x4{o[rt][e][x], o[rt][e + 1][x], o[rt][e + 2][x], o[rt][e + 3][x]} * f;
    }
    __syncthreads();
    constexpr int PIECES = DHP / 8;  // of 8 elements: a thread's share of a row
    const int most = min(ROWS, M - rb * ROWS);
    for (int i = t; i < most * PIECES; i += NT) {
      const int e = i % PIECES * 8, brow = i / PIECES, wq = brow / (RT * 16), rr = brow % (RT * 16);
      f32x4 a = (f32x4)(0.0f), d = (f32x4)(0.0f);
      float mx = kLow, sum = 0.0f;
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        a += *reinterpret_cast<const f32x4 *>(&s_o[wq * KW + j][rr][e]);
        d += *reinterpret_cast<const f32x4 *>(&s_o[wq * KW + j][rr][e + 4]);
        mx = fmaxf(mx, s_ml[wq * KW + j][rr][0]);
      }
#pragma unroll
      for (int j = 0; j < KW; ++j)
        sum += s_ml[wq * KW + j][rr][1] * __builtin_amdgcn_exp2f(s_ml[wq * KW + j][rr][0] - mx);
      finish(brow, e, a, d, mx, sum);
    }
  }
  if (SHARED || k.slot < 0) return;

  // One of several workgroups of the segment: the last to arrive adds them.  Of
  // more than kJoin parts, first the last of each kJoin in turn adds those into the
  // first one's slot, then the last of these adds the sums: 130 parts of 16 rows by
  // one workgroup alone took 30 us.
  constexpr int PIECES = DHP / 8, NB = 4;  // parts whose loads are in flight together
  const int most = min(ROWS, M - rb * ROWS);
  // Whether this is the last of n workgroups; what it stored before is there then.
  auto last_of = [&](int n, int line) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (t == 0) {
      unsigned int *count = p.counters + (size_t)line * kCountStride;
      const bool last = atomicAdd(count, 1u) == (unsigned)(n - 1);
      if (last) store_agent(count, 0u);
      s_last = last;
    }
    __syncthreads();
    return s_last != 0;
  };
  // Slots from, from + step, ...: n of them, to the output or to the first.  (The
  // pieces of a row are of one wave, which has read them all when it writes.)
  static_assert(kWave % PIECES == 0, "a row's pieces in one wave");
  auto join = [&](int from, int step, int n, bool final) {
    for (int i = t; i < most * PIECES; i += NT) {
      const int e = i % PIECES * 8, brow = i / PIECES;
      if (e >= Dh) continue;
      f32x4 a = (f32x4)(0.0f), d = (f32x4)(0.0f);
      float mx = kLow, sum = 0.0f;
      const uint32_t off = (uint32_t)from * kSlotBytes + (uint32_t)(brow * LROW) * 4u;
      for (int j0 = 0; j0 < n; j0 += NB) {
        f32x4 ml[NB], pa[NB], pd[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const uint32_t at = off + (uint32_t)(min(j0 + j, n - 1) * step) * kSlotBytes;
          ml[j] = ld_f4(wsr, at + DHP * 4u);
          pa[j] = ld_f4(wsr, at + (uint32_t)e * 4u);
          pd[j] = ld_f4(wsr, at + (uint32_t)e * 4u + 16u);
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          if (j0 + j >= n) break;
          const float up = fmaxf(mx, ml[j][0]), fo = __builtin_amdgcn_exp2f(mx - up), fn = __builtin_amdgcn_exp2f(ml[j][0] - up);
          a = a * fo + pa[j] * fn;
          d = d * fo + pd[j] * fn;
          sum = sum * fo + ml[j][1] * fn;
          mx = up;
        }
      }
      if (final) {
        store_out<DT>(p, b, h, rb * ROWS + brow, e, a, d, 1.0f / sum, s_anc);
      } else {
        st_f4(wsr, off + (uint32_t)e * 4u, a);
        st_f4(wsr, off + (uint32_t)e * 4u + 16u, d);
        if (e == 0) st_f4(wsr, off + DHP * 4u, f32x4{mx, sum, 0.0f, 0.0f});
      }
    }
  };
  const int first = (k.slot - k.slot0) / kJoin * kJoin, here = min(kJoin, k.parts - first);
  if (!last_of(here, k.slot0 + first)) return;
  if (k.parts > kJoin) {
    join(k.slot0 + first, 1, here, false);
    if (!last_of((k.parts + kJoin - 1) / kJoin, k.slot0 + 1)) return;
  }
  if (!need_anc) {
    tree_parents(N, t < N ? p.parent[(size_t)b * N + t] : 0, p.status, s_ptr, s_anc);
    tree_ancestors(N, s_ptr, s_anc);
  }
  if (k.parts > kJoin) join(k.slot0, kJoin, (k.parts + kJoin - 1) / kJoin, true);
  else join(k.slot0, 1, k.parts, true);
}

// Joins the parts of cut segments where those are of many rows: one workgroup for
// 256 pieces (of 8 elements) of a segment's rows, added in part order.  Bound by
// the round trips to its cut, to the parts and out: 5 us for segments of 4 parts
// of 96 rows, 9 us for 64 parts of 256 (34 MB).  (The last part's workgroup would
// take 60 us for 16 parts of 256 rows by itself; for up to 32 rows the join in the
// kernel above is quicker than a second launch.)
template <int DT, int DHP>
__global__ __launch_bounds__(kBlock) void k_tree_join(TreeAttnParams p, int rows) {
  const int4 cut = p.cuts[1 + blockIdx.x];  // with the count, in one round trip
  if ((int)blockIdx.x >= p.cuts[0].x) return;
  constexpr int PIECES = DHP / 8, LROW = DHP + 4, NB = 4;
  const int i = (int)(blockIdx.y * kBlock + threadIdx.x), e = i % PIECES * 8, brow = i / PIECES;
  const int h = cut.w / p.blocks, row = (cut.w - h * p.blocks) * rows + brow;
  if (brow >= rows || row >= p.N * p.G || e >= p.Dh) return;
  const size_t part_floats = (size_t)rows * LROW;
  const float *from = static_cast<const float *>(p.partial) + cut.x * part_floats + (size_t)brow * LROW;
  f32x4 a = (f32x4)(0.0f), d = (f32x4)(0.0f);
  float mx = kLow, sum = 0.0f;
  bool out = false;
  for (int j0 = 0; j0 < cut.y; j0 += NB) {
    f32x4 ml[NB], pa[NB], pd[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const float *at = from + min(j0 + j, cut.y - 1) * part_floats;
      ml[j] = *reinterpret_cast<const f32x4 *>(at + DHP);
      pa[j] = *reinterpret_cast<const f32x4 *>(at + e);
      pd[j] = *reinterpret_cast<const f32x4 *>(at + e + 4);
    }
    // all of them on their way before the first is waited for
#pragma unroll
    for (int j = 0; j < NB; ++j) asm volatile("" : "+v"(ml[j]), "+v"(pa[j]), "+v"(pd[j]));
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (j0 + j >= cut.y) break;
      out |= ml[j][1] < 0.0f;
      const float up = fmaxf(mx, ml[j][0]), fo = __builtin_amdgcn_exp2f(mx - up), fn = __builtin_amdgcn_exp2f(ml[j][0] - up);
      a = a * fo + pa[j] * fn;
      d = d * fo + pd[j] * fn;
      sum = sum * fo + ml[j][1] * fn;
      mx = up;
    }
  }
  if (!out) write_out<DT>(p, cut.z, h, row, e, a, d, 1.0f / sum);
}

template <int DT, int DHP, int RT, int RW, int KW>
static hipError_t launch_attn(const TreeAttnParams &p, hipStream_t s) {
  const dim3 grid((unsigned)p.grid), block(RW * KW * kWave);
  if (p.table && p.Dh == DHP)
    hipLaunchKernelGGL((k_tree_attention<DT, DHP, RT, RW, KW, true, false>), grid, block, 0, s, p);
  else if (p.table)
    hipLaunchKernelGGL((k_tree_attention<DT, DHP, RT, RW, KW, true, true>), grid, block, 0, s, p);
  else if (p.Dh == DHP)
    hipLaunchKernelGGL((k_tree_attention<DT, DHP, RT, RW, KW, false, false>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((k_tree_attention<DT, DHP, RT, RW, KW, false, true>), grid, block, 0, s, p);
  if constexpr (RW > 1) {
    constexpr int kRows = RW * RT * 16;
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 parts((unsigned)min((long)p.resident, (long)p.B * p.H * p.blocks), (kRows * (DHP / 8) + kBlock - 1) / kBlock);
    hipLaunchKernelGGL((k_tree_join<DT, DHP>), parts, dim3(kBlock), 0, s, p, kRows);
  }
  return hipGetLastError();
}

// The instance of a shape (see attn_shape).
template <int DT, int DHP>
static hipError_t launch_attn_dh(const TreeAttnParams &p, const AttnShape &a, hipStream_t s) {
  constexpr int kMost = attn_most_tiles(DT, DHP);
  if (a.rw == 1 && a.rt == 1) return launch_attn<DT, DHP, 1, 1, 4>(p, s);
  if constexpr (kMost == 2) {
    if (a.rw == 1) return launch_attn<DT, DHP, 2, 1, 4>(p, s);
    if (a.rt == 2) return launch_attn<DT, DHP, 2, 8, 1>(p, s);
    if (a.rw == 6) return launch_attn<DT, DHP, 1, 6, 2>(p, s);
  }
  if constexpr (attn_shared(DT, DHP)) {
    if constexpr (attn_share_keys(DT, DHP) == 2)
      if (a.rw == 4) return launch_attn<DT, DHP, 1, 4, 2>(p, s);
    if (a.rw == 8) return launch_attn<DT, DHP, 1, 8, 1>(p, s);
  }
  return hipErrorInvalidValue;
}

template <int DT>
static hipError_t launch_attn_dt(const TreeAttnParams &p, hipStream_t s) {
  const AttnShape a = attn_shape(DT, p.Dh, p.N * p.G);
  if (a.dhp == 64) return launch_attn_dh<DT, 64>(p, a, s);
  if (a.dhp == 128) return launch_attn_dh<DT, 128>(p, a, s);
  return launch_attn_dh<DT, 256>(p, a, s);
}

}  // namespace sd
