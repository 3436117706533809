// Attention of a tree of drafted nodes over a row's cache and the nodes' own
// ancestors, for caches in pages, left-padded rectangles and pools.
//
// For node i of row b and query head h of KV head k = h / G:
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j),
// j over the row's cached positions [0, len) and the nodes from i to the root.
//
// The G N query rows of one (row, KV head) share its keys, so a wave multiplies
// them together with matrix instructions while the keys stream by once:
//  - S^T = K Q^T: a lane holds 8 consecutive elements of one key straight from
//    memory (16 bytes), which is the instruction's layout for K; the keys need
//    no LDS.
//  - The softmax weights come out as S^T, a lane holding one query and 8 keys of
//    a 32-key tile; with the contraction's keys numbered in that order the same
//    registers, rounded to the cache's type, are the operand of
//  - O^T += V^T P^T.  For it a lane loads, for each of its 8 keys, its NE =
//    Dh / 16 elements (a row of V is read by 16 lanes, whole), and 8 x NE
//    elements turn into NE operands by byte permutes: element e of all 8 keys is
//    the operand of the output rows dh = NE (lane mod 16) + e.  V needs no LDS
//    either.
// The running maximum is only raised when some score passes it by more than
// 2^kSlack: below that the weights stay under 2^kSlack, exact enough in every
// type, and the accumulators need no rescaling.  Weights and sums are fp32.
// The weights are rounded to the cache's type for the second product (8 bits of
// mantissa for bf16): their errors average over the keys to less than the
// output's own rounding.
//
// Work split.  Rows have ragged lengths, so the key tiles of all (row, KV head,
// query block) segments are laid end to end and every workgroup takes an equal
// run of them (in units of one tile per key wave), whatever segments that
// crosses.  A segment within one workgroup is finished there; otherwise its
// workgroups leave (max, sum, O) in the workspace and the last to arrive adds
// them in workgroup order, so results do not depend on timing.  The order of
// completion uses the same scheme as verification: sums stored past the
// non-coherent L2 (sc1), completed (vmcnt) before the count, loaded only after
// the count has returned.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "coherent.h"
#include "device_common.h"
#include "launch.h"
#include "specdec.h"
#include "tree_common.h"

namespace sd {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 32;        // keys of a wave's step
constexpr float kSlack = 8.0f;   // log2 of the largest weight before the maximum is raised
constexpr float kLow = -1e30f;   // running maximum before the first key

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
  if constexpr (DT == 1) {
    const _Float16 a = (_Float16)lo, b = (_Float16)hi;
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
  } else {
    const __bf16 a = (__bf16)lo, b = (__bf16)hi;
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
  }
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

// Inclusive prefix sums of n <= NT * 4 values into pre[1..n], pre[0] = 0.
template <typename F>
__device__ __forceinline__ void block_prefix(int n, long long *pre, long long *scratch, F value) {
  const int per = (n + kThreads - 1) / kThreads, t = threadIdx.x, lane = t & (kWave - 1);
  long long own = 0;
  for (int k = 0; k < per; ++k) {
    const int i = t * per + k;
    if (i < n) own += value(i);
  }
  long long incl = own;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const long long y = __shfl_up(incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == kWave - 1) scratch[t / kWave] = incl;
  __syncthreads();
  long long run = incl - own;
  for (int k = 0; k < t / kWave; ++k) run += scratch[k];
  for (int k = 0; k < per; ++k) {
    const int i = t * per + k;
    if (i < n) {
      run += value(i);
      pre[i + 1] = run;
    }
  }
  if (t == 0) pre[0] = 0;
  __syncthreads();
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// 16-byte stores and loads of partial sums through the coherence point.
__device__ __forceinline__ void st_f4(__amdgpu_buffer_rsrc_t r, uint32_t off, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4v, v), r, off, 0, kCoherentPolicy);
}
__device__ __forceinline__ f32x4 ld_f4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kCoherentPolicy));
}

// The workgroup whose run [total w / W, total (w + 1) / W) holds unit x.
__device__ __forceinline__ int first_wg(long long x, long long total, int W) {
  return (int)(((x + 1) * W - 1) / total);
}

// Elements e .. e+7 (a, then d) of query row `row` of (b, h), unless its node
// is not part of the tree (anc: the nodes' ancestor bits).
template <int DT>
__device__ __forceinline__ void store_out(const TreeAttnParams &p, int b, int h, int row, int e, f32x4 a, f32x4 d, float f,
                                          const uint32_t (*anc)[kMaxNodes / 32]) {
  const int n = (int)fdiv((uint32_t)row, p.g_div), gq = row - n * p.G;
  if (!(anc[n][0] & 1u)) return;
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

// RT 16-query tiles per wave, RW waves across query blocks, KW = 4 / RW waves
// across keys; DHP the head size, or with PAD the next of 64, 128 and 256.
template <int DT, int DHP, int RT, int RW, bool PAD>
__global__ __launch_bounds__(kThreads, attn_wgs_per_cu(RT, DHP)) void k_tree_attention(TreeAttnParams p) {
  constexpr int KW = kWaves / RW;
  constexpr int ES = es<DT>();
  constexpr int EL = 16 / ES;             // elements of a 16-byte piece
  constexpr int KS = DHP / (4 * EL);      // contraction steps of S (4 lane groups x EL elements)
  constexpr int NE = DHP / 16;            // elements of V a lane holds per key
  constexpr int VP = (NE * ES + 15) / 16; // 16-byte pieces of them (8 bytes where NE * ES is 8)
  constexpr int VD = NE * ES / 4;         // dwords of them
  constexpr int ROWS = RW * RT * 16;      // query rows of a workgroup
  constexpr int LROW = DHP + 4;           // floats of an LDS row of O

  __shared__ long long s_pre[kMaxAttnRows + 1], s_scan[kWaves];
  __shared__ uint32_t s_anc[2][kMaxNodes][kMaxNodes / 32];
  __shared__ int s_ptr[kMaxNodes], s_red[kWaves], s_last, s_odd;
  __shared__ float s_ml[kWaves][RT * 16][2];
  __shared__ __align__(16) float s_o[kWaves][16][LROW];

  const int t = threadIdx.x, lane = t & (kWave - 1), wave = uniform(t / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int kw = wave % KW, rw = wave / KW;
  const int N = p.N, G = p.G, H = p.H, Dh = PAD ? p.Dh : DHP, M = N * G;
  const int tree_tiles = (N + kTile - 1) / kTile;
  const int RB = (M + ROWS - 1) / ROWS;
  const size_t row_bytes = (size_t)Dh * ES;

  // lengths of every row: the split of the work, and whether there is any
  auto row_of = [&](int b) { return p.rows ? p.rows[b] : b; };
  auto start_of = [&](int b, int len) { return p.width ? p.width[p.group > 0 ? b / p.group : 0] - len : 0; };
  int bad = 0;
  for (int b = t; b < p.B; b += kThreads) {
    const int r = row_of(b);
    if (r < 0 || r >= p.n_rows) {
      bad = 1;
    } else {
      const int len = p.len[r], s = start_of(b, len);
      bad |= len < 0 || s < 0 || (long long)s + len > p.cap;
    }
  }
  if (block_or_int<kThreads>(bad, s_red)) {
    if (t == 0) set_status(p.status, SPECDEC_S_LEN_RANGE);
    return;
  }
  block_prefix(p.B, s_pre, s_scan, [&](int b) {
    const long long tiles = (p.len[row_of(b)] + kTile - 1) / kTile + tree_tiles;
    return (tiles + KW - 1) / KW;
  });
  const long long HR = (long long)H * RB, total = s_pre[p.B] * HR;
  const int W = (int)min((long long)gridDim.x, total);
  // consecutive runs of work on one XCD (workgroups go to the 8 XCDs in turn),
  // so query blocks that share keys share an L2
  const int per_xcd = (W + 7) / 8, on_xcd = (int)(blockIdx.x >> 3);
  const int w = (int)(blockIdx.x & 7) * per_xcd + on_xcd;
  if (on_xcd >= per_xcd || w >= W) return;
  const long long begin = total * w / W, end = total * (w + 1) / W;

  const __amdgpu_buffer_rsrc_t wsr = coherent_rsrc(p.partial, p.partial_bytes);
  constexpr int kSlotFloats = ROWS * (DHP + 4);  // per row: O, then max and sum (16-byte rows)
  int anc_of = -1;

  for (long long at = begin; at < end;) {
    // the segment at `at`: batch row b, head h, query block rb
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_pre[mid] * HR <= at) lo = mid;
      else hi = mid;
    }
    const int b = uniform(lo);
    const long long units = s_pre[b + 1] - s_pre[b], rem = at - s_pre[b] * HR;
    const int seg = uniform((int)(rem / units));
    const long long u0 = rem - seg * units, seg0 = at - u0, seg1 = seg0 + units;
    const long long u1 = min(units, u0 + (end - at));
    at += u1 - u0;
    const int h = seg / RB, rb = seg - h * RB;
    const int r = uniform(row_of(b)), len = uniform(p.len[r]), start = uniform(start_of(b, len));
    const int cache_tiles = (len + kTile - 1) / kTile, tiles = cache_tiles + tree_tiles;
    const int t0 = (int)(u0 * KW), t1 = (int)min((long long)tiles, u1 * KW);

    // which nodes each node attends: a bit per ancestor, by pointer doubling
    if (t1 > cache_tiles && anc_of != b) {
      __syncthreads();  // the last segment's readers
      const int words = (N + 31) / 32;
      bool bad_tree = false;
      if (t < N) {
        s_ptr[t] = node_parent(t, p.parent[(size_t)b * N + t], bad_tree);
        for (int k = 0; k < words; ++k) s_anc[0][t][k] = (t >> 5) == k ? 1u << (t & 31) : 0u;
      }
      if (bad_tree) set_status(p.status, SPECDEC_S_TREE);
      int side = 0;
      for (int span = 1; span < N; span <<= 1, side ^= 1) {
        __syncthreads();
        int q = 0;
        if (t < N) {
          q = s_ptr[t];
          for (int k = 0; k < words; ++k) s_anc[side ^ 1][t][k] = s_anc[side][t][k] | (q > 0 ? s_anc[side][q][k] : 0u);
          if (q > 0) q = s_ptr[q];
        }
        __syncthreads();
        if (t < N) s_ptr[t] = q;
      }
      __syncthreads();
      // a node that reached the root sees it; one that did not sees nothing
      if (t < N) {
        for (int k = 0; k < words; ++k) {
          const uint32_t m = s_anc[side][t][k];
          s_anc[side ^ 1][t][k] = s_ptr[t] < 0 ? 0u : k == 0 ? m | 1u : m;
        }
      }
      side ^= 1;
      __syncthreads();
      if (t < N && side)
        for (int k = 0; k < words; ++k) s_anc[0][t][k] = s_anc[1][t][k];
      __syncthreads();
      anc_of = b;
    }

    // queries of this wave: row rt * 16 + c of its block, 16 bytes per step
    const int rbase = rb * ROWS + rw * RT * 16;
    u32x4 q[RT][KS];
    int node[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = rbase + rt * 16 + c;
      const int n = row < M ? (int)fdiv((uint32_t)row, p.g_div) : 0, gq = row - n * G;
      node[rt] = row < M ? n : -1;
      const char *src = static_cast<const char *>(p.q) +
                        ((int64_t)b * p.qs[0] + (int64_t)n * p.qs[1] + (int64_t)(h * G + gq) * p.qs[2]) * ES;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int dh = (s * 4 + g) * EL;
        q[rt][s] = row < M && (!PAD || dh < Dh) ? *reinterpret_cast<const u32x4 *>(src + dh * ES) : (u32x4)(0u);
      }
    }

    f32x4 o[RT][NE];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = kLow;
      l[rt] = 0.0f;
#pragma unroll
      for (int e = 0; e < NE; ++e) o[rt][e] = (f32x4)(0.0f);
    }

    if (t == 0) s_odd = 0;
    __syncthreads();
    bool bad_page = false;

    // Row index (in units of Dh elements) of key lane & 31 of tile tl, and
    // whether there is such a key.  A tile of the cache holds at least one.
    auto find = [&](int tl, bool &valid) -> uint32_t {
      const int k = lane & (kTile - 1);
      if (tl < cache_tiles) {
        const int pos = tl * kTile + k;
        valid = pos < len;
        const int at_pos = valid ? pos : len - 1;
        if (!p.table) return (uint32_t)((r * H + h) * p.cap + start + at_pos);
        const int blk = (int)fdiv((uint32_t)at_pos, p.page_div), slot = at_pos - blk * p.page;
        int pg = p.table[(size_t)r * p.max_blocks + blk];
        if (pg < 0 || pg >= p.n_pages) {  // takes no part; the read stays inside the cache
          pg = 0;
          valid = false;
          bad_page = true;
        }
        return (uint32_t)((pg * H + h) * p.page + slot);
      }
      const int j = (tl - cache_tiles) * kTile + k;
      valid = j < N && tl < tiles && (s_anc[0][min(j, N - 1)][0] & 1u);
      return (uint32_t)((b * H + h) * N + min(j, N - 1));
    };
    u32x4 kr[2][KS];
    uint32_t vr[8][VD];
    auto load_k = [&](int tl, uint32_t rho) {
      const char *base = static_cast<const char *>(tl < cache_tiles ? p.k_old : p.k_new);
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const char *src = base + (size_t)__shfl(rho, kt * 16 + c) * row_bytes;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int dh = (s * 4 + g) * EL;
          kr[kt][s] = !PAD || dh < Dh ? *reinterpret_cast<const u32x4 *>(src + dh * ES) : (u32x4)(0u);
        }
      }
    };
    auto load_v = [&](int tl, uint32_t rho) {
      const char *base = static_cast<const char *>(tl < cache_tiles ? p.v_old : p.v_new);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const char *src = base + (size_t)__shfl(rho, (k >> 2) * 16 + g * 4 + (k & 3)) * row_bytes + c * NE * ES;
        if constexpr (VD == 2) {
          const u32x2 v = !PAD || c * NE < Dh ? *reinterpret_cast<const u32x2 *>(src) : (u32x2)(0u);
          vr[k][0] = v[0];
          vr[k][1] = v[1];
        } else {
#pragma unroll
          for (int d = 0; d < VP; ++d) {
            const u32x4 v = !PAD || c * NE + d * EL < Dh ? *reinterpret_cast<const u32x4 *>(src + d * 16) : (u32x4)(0u);
#pragma unroll
            for (int x = 0; x < 4; ++x) vr[k][d * 4 + x] = v[x];
          }
        }
      }
    };

    bool valid = false, valid_next = false;
    uint32_t rho = 0, rho_next = 0;
    int tl = t0 + kw;
    if (tl < t1) {
      rho = find(tl, valid);
      load_k(tl, rho);
      load_v(tl, rho);
      if (tl + KW < t1) rho_next = find(tl + KW, valid_next);
    }
    for (; tl < t1; tl += KW) {
      const bool more = tl + KW < t1;
      const uint32_t vm = (uint32_t)__ballot(valid);  // keys of the tile that exist
      const bool in_tree = tl >= cache_tiles;
      // scores: s[rt][kt][x] of query c and key kt * 16 + g * 4 + x
      f32x4 s[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          s[rt][kt] = (f32x4)(0.0f);
#pragma unroll
          for (int x = 0; x < KS; ++x) s[rt][kt] = mma<DT>(kr[kt][x], q[rt][x], s[rt][kt]);
        }
      if (more) load_k(tl + KW, rho_next);
      const uint32_t mine = g * 4;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) s[rt][kt] *= p.scale;  // log2(e) / sqrt(Dh), or the caller's
        if (in_tree || vm != 0xFFFFFFFFu) {
          uint32_t see = vm;
          if (in_tree) see = node[rt] >= 0 ? s_anc[0][node[rt]][tl - cache_tiles] : 0u;
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (!((see >> (kt * 16 + mine + x)) & 1u)) s[rt][kt][x] = -INFINITY;
        }
        float top = fmaxf(fmaxf(fmaxf(s[rt][0][0], s[rt][0][1]), fmaxf(s[rt][0][2], s[rt][0][3])),
                          fmaxf(fmaxf(s[rt][1][0], s[rt][1][1]), fmaxf(s[rt][1][2], s[rt][1][3])));
        if (__any(top > m[rt] + kSlack)) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const float up = fmaxf(m[rt], top), f = __builtin_amdgcn_exp2f(m[rt] - up);
          m[rt] = up;
          l[rt] *= f;
#pragma unroll
          for (int e = 0; e < NE; ++e) o[rt][e] *= f;
        }
        float sum = 0.0f;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            s[rt][kt][x] = __builtin_amdgcn_exp2f(s[rt][kt][x] - m[rt]);
            sum += s[rt][kt][x];
          }
        l[rt] += sum;
      }

      // V of keys that do not exist must not meet their zero weights as NaN
      if (vm != 0xFFFFFFFFu) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool on = (vm >> ((k >> 2) * 16 + mine + (k & 3))) & 1u;
#pragma unroll
          for (int d = 0; d < VD; ++d) vr[k][d] = on ? vr[k][d] : 0u;
        }
      }
      // In the tree a node's V may only reach its descendants, but zero times
      // infinity is NaN: where a tile holds a value that is not finite, zero takes
      // its place here and the rows that attend to it add it at the segment's end.
      if (in_tree) {
        uint32_t odd = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int d = 0; d < VD; ++d) odd |= odd_bits<DT>(vr[k][d]);
        if (__any(odd & (DT == 0 ? 0x80000000u : 0x80008000u))) {
          s_odd = 1;
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int d = 0; d < VD; ++d) vr[k][d] = finite_only<DT>(vr[k][d]);
        }
      }

      // O^T += V^T P^T
      if constexpr (DT == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              o[rt][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vr[k][e]), s[rt][k >> 2][k & 3], o[rt][e], 0,
                                                              0, 0);
      } else {
        u32x4 w8[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          w8[rt] = u32x4{pack2<DT>(s[rt][0][0], s[rt][0][1]), pack2<DT>(s[rt][0][2], s[rt][0][3]),
                         pack2<DT>(s[rt][1][0], s[rt][1][1]), pack2<DT>(s[rt][1][2], s[rt][1][3])};
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
          u32x4 a;
#pragma unroll
          for (int k = 0; k < 4; ++k) a[k] = __builtin_amdgcn_perm(vr[2 * k + 1][e / 2], vr[2 * k][e / 2], sel);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) o[rt][e] = mma<DT>(a, w8[rt], o[rt][e]);
        }
      }
      if (more) {
        load_v(tl + KW, rho_next);
        rho = rho_next;
        valid = valid_next;
        if (tl + 2 * KW < t1) rho_next = find(tl + 2 * KW, valid_next);
      }
    }

    if (bad_page) set_status(p.status, SPECDEC_S_LEN_RANGE);
    // The segment's end: sums over lane groups, then over the key waves.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] += __shfl_xor(l[rt], 16);
      l[rt] += __shfl_xor(l[rt], 32);
      if (g == 0) {
        s_ml[wave][rt * 16 + c][0] = m[rt];
        s_ml[wave][rt * 16 + c][1] = l[rt];
      }
    }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == units;
    // this workgroup's slot: its run's first segment if that began earlier, its
    // last if it goes on
    const uint32_t slot = (uint32_t)(w * 2 + (u0 == 0)) * (uint32_t)(kSlotFloats * 4);
    // 16-byte pieces of a tile's rows: thread -> (row, first element)
    constexpr int PIECES = DHP / 8;  // of 8 elements
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float top = kLow;
#pragma unroll
      for (int k = 0; k < KW; ++k) top = fmaxf(top, s_ml[rw * KW + k][rt * 16 + c][0]);
      const float f = __builtin_amdgcn_exp2f(m[rt] - top);
      if (rt) __syncthreads();
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < NE; e += 4)
          *reinterpret_cast<f32x4 *>(&s_o[wave][c][(g * 4 + x) * NE + e]) =
              f32x4{o[rt][e][x], o[rt][e + 1][x], o[rt][e + 2][x], o[rt][e + 3][x]} * f;
      __syncthreads();
      for (int i = t; i < RW * 16 * PIECES; i += kThreads) {
        const int e = i % PIECES * 8, rr = i / PIECES, wq = rr / 16, rc = rr % 16;
        const int brow = (wq * RT + rt) * 16 + rc, row = rb * ROWS + brow;
        if (row >= M || e >= Dh) continue;
        f32x4 a = (f32x4)(0.0f), d = (f32x4)(0.0f);
        float mx = kLow, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          a += *reinterpret_cast<const f32x4 *>(&s_o[wq * KW + k][rc][e]);
          d += *reinterpret_cast<const f32x4 *>(&s_o[wq * KW + k][rc][e + 4]);
          mx = fmaxf(mx, s_ml[wq * KW + k][rt * 16 + rc][0]);
        }
#pragma unroll
        for (int k = 0; k < KW; ++k)
          sum += s_ml[wq * KW + k][rt * 16 + rc][1] * __builtin_amdgcn_exp2f(s_ml[wq * KW + k][rt * 16 + rc][0] - mx);
        if (s_odd)
          add_odd<DT>(p, static_cast<const char *>(p.v_new) + (size_t)(b * H + h) * N * row_bytes, row, e, Dh, t0 - cache_tiles,
                      t1 - cache_tiles, s_anc[0], a, d);
        if (whole) {
          store_out<DT>(p, b, h, row, e, a, d, 1.0f / sum, s_anc[0]);
        } else {
          const uint32_t off = slot + (uint32_t)(brow * (DHP + 4)) * 4u;
          st_f4(wsr, off + (uint32_t)e * 4u, a);
          st_f4(wsr, off + (uint32_t)e * 4u + 16u, d);
          if (e == 0) st_f4(wsr, off + DHP * 4u, f32x4{mx, sum, 0.0f, 0.0f});
        }
      }
    }
    if (!whole) {
      // the segment's workgroups: the first holds its unit 0, the last its end
      const int w0 = first_wg(seg0, total, W), w1 = first_wg(seg1 - 1, total, W);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (t == 0) {
        unsigned int *count = p.counters + (size_t)w0 * kCountStride;
        const bool last = atomicAdd(count, 1u) == (unsigned)(w1 - w0);
        if (last) store_agent(count, 0u);
        s_last = last;
      }
      __syncthreads();
      if (s_last) {
        if (anc_of != b) {
          // only whether a node is used matters here
          __syncthreads();
          bool bt = false;
          if (t < N) s_ptr[t] = node_parent(t, p.parent[(size_t)b * N + t], bt);
          for (int span = 1; span < N; span <<= 1) {
            __syncthreads();
            const int q1 = t < N && s_ptr[t] > 0 ? s_ptr[s_ptr[t]] : t < N ? s_ptr[t] : 0;
            __syncthreads();
            if (t < N) s_ptr[t] = q1;
          }
          if (t < N) s_anc[0][t][0] = s_ptr[t] == 0;
          __syncthreads();
          anc_of = -1;
        }
        for (int i = t; i < ROWS * PIECES; i += kThreads) {
          const int e = i % PIECES * 8, brow = i / PIECES, row = rb * ROWS + brow;
          if (row >= M || e >= Dh) continue;
          f32x4 a = (f32x4)(0.0f), d = (f32x4)(0.0f);
          float mx = kLow, sum = 0.0f;
          for (int k = w0; k <= w1; ++k) {
            const uint32_t off = (uint32_t)(k * 2 + (k == w0)) * (uint32_t)(kSlotFloats * 4) + (uint32_t)(brow * (DHP + 4)) * 4u;
            const f32x4 ml = ld_f4(wsr, off + DHP * 4u);
            const f32x4 ka = ld_f4(wsr, off + (uint32_t)e * 4u), kd = ld_f4(wsr, off + (uint32_t)e * 4u + 16u);
            const float up = fmaxf(mx, ml[0]), fo = __builtin_amdgcn_exp2f(mx - up), fn = __builtin_amdgcn_exp2f(ml[0] - up);
            a = a * fo + ka * fn;
            d = d * fo + kd * fn;
            sum = sum * fo + ml[1] * fn;
            mx = up;
          }
          store_out<DT>(p, b, h, row, e, a, d, 1.0f / sum, s_anc[0]);
        }
      }
    }
    __syncthreads();  // s_ml, s_o and s_anc are free again
  }
}

template <int DT, int DHP, int RT, int RW>
static hipError_t launch_attn(const TreeAttnParams &p, hipStream_t s) {
  if (p.Dh == DHP)
    hipLaunchKernelGGL((k_tree_attention<DT, DHP, RT, RW, false>), dim3((unsigned)p.grid), dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL((k_tree_attention<DT, DHP, RT, RW, true>), dim3((unsigned)p.grid), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

// The instance of a shape (see attn_shape).
template <int DT, int DHP>
static hipError_t launch_attn_dh(const TreeAttnParams &p, const AttnShape &a, hipStream_t s) {
  constexpr int kMost = attn_most_tiles(DT, DHP);
  if (a.rw == 1) {
    if (a.rt == 1) return launch_attn<DT, DHP, 1, 1>(p, s);
    if constexpr (kMost >= 2)
      if (a.rt == 2) return launch_attn<DT, DHP, 2, 1>(p, s);
    if constexpr (kMost >= 4)
      if (a.rt == 4) return launch_attn<DT, DHP, 4, 1>(p, s);
  }
  if constexpr (kMost >= 4)
    if (a.rt == 3 && a.rw == 2) return launch_attn<DT, DHP, 3, 2>(p, s);
  if (a.rt == kMost && a.rw == 2) return launch_attn<DT, DHP, kMost, 2>(p, s);
  if (a.rt == kMost && a.rw == 4) return launch_attn<DT, DHP, kMost, 4>(p, s);
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
