// Tree speculation around the model's attention: positions of the nodes,
// rotary positions, and compaction of the accepted path.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "launch.h"
#include "specdec.h"
#include "tree_common.h"

namespace sd {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ positions

// pos[b][i] = len + depth of node i.  One workgroup per batch row, a node per
// thread; the depths by pointer doubling.  A few hundred bytes per row: the
// call is a launch, two round trips and log2 N steps in LDS, 3.5 us for 16 rows
// of 24 nodes and 3.8 us for 64 of 64.
__global__ __launch_bounds__(kMaxNodes) void k_tree_positions(TreePosParams p) {
  __shared__ int s_ptr[kMaxNodes], s_steps[kMaxNodes], s_red[kMaxNodes / kWave];
  const int b = blockIdx.x, i = threadIdx.x;
  // every workgroup looks at every row's length, so a bad one stops them all
  int bad_len = 0;
  for (int k = i; k < p.B; k += kMaxNodes) {
    const int r = p.rows ? p.rows[k] : k;
    const bool in = r >= 0 && r < p.n_rows;
    const int n = in ? p.len[r] : -1;
    bad_len |= n < 0 || n > kMaxTreeLen;
  }
  bool bad = false;
  if (i < p.N) {
    s_ptr[i] = node_parent(i, p.parent[(size_t)b * p.N + i], bad);
    s_steps[i] = i > 0;
  }
  const int flags = block_or_int<kMaxNodes>((bad_len ? SPECDEC_S_LEN_RANGE : 0) | (bad ? SPECDEC_S_TREE : 0), s_red);
  if (i == 0) set_status(p.status, flags);
  if (flags & SPECDEC_S_LEN_RANGE) return;
  tree_depths<kMaxNodes>(p.N, s_ptr, s_steps);
  const int len = p.len[p.rows ? p.rows[b] : b];
  if (i < p.N) p.pos[(size_t)b * p.N + i] = s_ptr[i] == 0 ? len + s_steps[i] : -1;
}

hipError_t launch_tree_positions(const TreePosParams &p, hipStream_t s) {
  hipLaunchKernelGGL(k_tree_positions, dim3((unsigned)p.B), dim3(kMaxNodes), 0, s, p);
  return hipGetLastError();
}

// ----------------------------------------------------------------------- rope

template <int DT> struct RopeElem { using T = uint16_t; };
template <> struct RopeElem<0> { using T = uint32_t; };

template <int DT>
__device__ __forceinline__ float rope_widen(uint32_t bits) {
  if constexpr (DT == 0) return __uint_as_float(bits);
  else if constexpr (DT == 1) return f16_bits_to_f32(bits);
  else return bf16_bits_to_f32(bits);
}

template <int DT>
__device__ __forceinline__ uint32_t rope_narrow(float v) {
  // the empty asm keeps the fp32 result apart from its conversion: fused into a
  // mixed-precision multiply-add it rounds once in some access widths' code and
  // twice in others'
  if constexpr (DT == 1) asm("" : "+v"(v));
  if constexpr (DT == 0) return __float_as_uint(v);
  else if constexpr (DT == 1) return __builtin_bit_cast(uint16_t, (_Float16)v);
  else return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// The turned pair, the products' roundings spelled out so that every access
// width gives the same bytes.
__device__ __forceinline__ float turn0(float x0, float x1, float2 w) { return fmaf(x0, w.x, -(x1 * w.y)); }
__device__ __forceinline__ float turn1(float x0, float x1, float2 w) { return fmaf(x1, w.x, x0 * w.y); }

// VE elements as they lie in memory: one load or store of up to 16 bytes, or
// VE of one element where AL says that the addresses are aligned to elements
// only.
template <int DT, int VE, bool AL>
struct alignas(sizeof(typename RopeElem<DT>::T) * (AL ? VE : 1)) RopeVec {
  typename RopeElem<DT>::T e[VE];
};

// One workgroup rotates `tokens` consecutive (row, node) pairs.  First the
// angles: pair k of a token turns by pos * freq[k], formed in fp64 and reduced
// to turns there (at position 131072 an fp32 product would be off by 1e-2
// radians), its sine and cosine then in fp32 of the reduced turn; they are
// shared by all heads through LDS.  Then the heads, VE elements per access: the
// half layout takes the vectors at k and k + rot/2 together, the interleaved
// one holds whole pairs in a vector.  A pair is read before it is written, by
// the same thread, so x and out may be the same tensor.  A token with a
// negative position is passed over.
// 4.2 us for 384 tokens of 40 heads x 128 (6.6 MB: a launch, the angles and one
// round trip); 10.5 us for 4096 tokens of 32 heads x 96 (41 MB, 3.9 TB/s: by
// memory).  With 4-byte accesses in place of 16 a thread has a quarter of the
// bytes in flight, so the widest that divides every piece is taken.
template <int DT, int VE, bool AL, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeParams p) {
  using Vec = RopeVec<DT, VE, AL>;
  using T = typename RopeElem<DT>::T;
  extern __shared__ float2 s_cs[];  // [tokens][half]
  __shared__ int s_pos[kRopeTokens];
  const int half = p.rot / 2;
  const int64_t first = (int64_t)blockIdx.x * p.tokens;
  const int nt = (int)min((int64_t)p.tokens, (int64_t)p.B * p.N - first);
  if ((int)threadIdx.x < nt) s_pos[threadIdx.x] = p.pos[first + threadIdx.x];
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int t = (int)fdiv((uint32_t)i, p.half_div), k = i - t * half;
    constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
    double turn = (double)s_pos[t] * p.freq[k] * kTurn;
    turn -= rint(turn);
    float sn, cs;
    sincospif(2.0f * (float)turn, &sn, &cs);
    s_cs[i] = make_float2(cs * p.factor, sn * p.factor);
  }
  __syncthreads();
  // work items of a token: its heads' pair vectors, then the vectors past rot
  const int pair_items = INTER ? p.rot / VE : half / VE;
  const int per_head = pair_items + (p.Dh - p.rot) / VE;
  const int per_token = p.heads * per_head;
  for (int i = threadIdx.x; i < nt * per_token; i += kRopeThreads) {
    const int t = (int)fdiv((uint32_t)i, p.token_div), r = i - t * per_token;
    const int h = (int)fdiv((uint32_t)r, p.head_div), v = r - h * per_head;
    if (s_pos[t] < 0) continue;
    const uint32_t tok = (uint32_t)(first + t);
    const uint32_t b = fdiv(tok, p.node_div), n = tok - b * (uint32_t)p.N;
    const T *x = static_cast<const T *>(p.x) + (b * p.xs[0] + n * p.xs[1] + h * p.xs[2]);
    T *y = static_cast<T *>(p.out) + (b * p.os[0] + n * p.os[1] + h * p.os[2]);
    const float2 *cs = s_cs + t * half;
    if (v >= pair_items) {  // past the rotated part: copied
      const int at = p.rot + (v - pair_items) * VE;
      *reinterpret_cast<Vec *>(y + at) = *reinterpret_cast<const Vec *>(x + at);
    } else if constexpr (INTER) {
      const int at = v * VE;
      Vec a = *reinterpret_cast<const Vec *>(x + at);
#pragma unroll
      for (int e = 0; e < VE; e += 2) {
        const float2 w = cs[at / 2 + e / 2];
        const float x0 = rope_widen<DT>(a.e[e]), x1 = rope_widen<DT>(a.e[e + 1]);
        a.e[e] = (T)rope_narrow<DT>(turn0(x0, x1, w));
        a.e[e + 1] = (T)rope_narrow<DT>(turn1(x0, x1, w));
      }
      *reinterpret_cast<Vec *>(y + at) = a;
    } else {
      const int at = v * VE;
      Vec a = *reinterpret_cast<const Vec *>(x + at), c = *reinterpret_cast<const Vec *>(x + at + half);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float2 w = cs[at + e];
        const float x0 = rope_widen<DT>(a.e[e]), x1 = rope_widen<DT>(c.e[e]);
        a.e[e] = (T)rope_narrow<DT>(turn0(x0, x1, w));
        c.e[e] = (T)rope_narrow<DT>(turn1(x0, x1, w));
      }
      *reinterpret_cast<Vec *>(y + at) = a;
      *reinterpret_cast<Vec *>(y + at + half) = c;
    }
  }
}

template <int DT, int VE, bool AL, bool INTER>
static hipError_t launch_rope_ve(RopeParams p, hipStream_t s) {
  const int half = p.rot / 2;
  const int per_head = (INTER ? p.rot / VE : half / VE) + (p.Dh - p.rot) / VE;
  const int64_t all = (int64_t)p.B * p.N;
  // tokens per workgroup: two accesses per thread where a token is small
  int tokens = (int)((2 * kRopeThreads) / ((int64_t)p.heads * per_head));
  tokens = tokens < 1 ? 1 : tokens > kRopeTokens ? kRopeTokens : tokens;
  p.tokens = tokens;
  p.half_div = host_fast_div((uint32_t)(half > 0 ? half : 1));
  p.head_div = host_fast_div((uint32_t)per_head);
  p.token_div = host_fast_div((uint32_t)(p.heads * per_head));
  p.node_div = host_fast_div((uint32_t)p.N);
  hipLaunchKernelGGL((k_rope<DT, VE, AL, INTER>), dim3((unsigned)((all + tokens - 1) / tokens)), dim3(kRopeThreads),
                     (size_t)tokens * half * sizeof(float2), s, p);
  return hipGetLastError();
}

template <int DT, bool INTER>
static hipError_t launch_rope_dt(const RopeParams &p, hipStream_t s) {
  // the widest access that every piece is a whole number of (p.ve: by the
  // pointers and strides); Dh and rot are even, so pairs always are
  int ve = p.ve;
  while (ve > 1 && ((INTER ? p.rot : p.rot / 2) % ve || (p.Dh - p.rot) % ve)) ve /= 2;
  if constexpr (DT != 0) {
    if (ve == 8) return launch_rope_ve<DT, 8, true, INTER>(p, s);
  }
  if (ve == 4) return launch_rope_ve<DT, 4, true, INTER>(p, s);
  if (ve == 2) return launch_rope_ve<DT, 2, true, INTER>(p, s);
  return launch_rope_ve<DT, INTER ? 2 : 1, false, INTER>(p, s);
}

hipError_t launch_rope(const RopeParams &p, hipStream_t s) {
  if (p.interleaved)
    return p.dtype == 0 ? launch_rope_dt<0, true>(p, s) : p.dtype == 1 ? launch_rope_dt<1, true>(p, s)
                                                                       : launch_rope_dt<2, true>(p, s);
  return p.dtype == 0 ? launch_rope_dt<0, false>(p, s) : p.dtype == 1 ? launch_rope_dt<1, false>(p, s)
                                                                      : launch_rope_dt<2, false>(p, s);
}

// -------------------------------------------------------------------- compact

// Entries path[b][0 .. accept_len[b]] of row b's N speculative entries become
// its first ones, and the accepted nodes' token ids with them.  A workgroup
// serves one batch row: its path in LDS, then an equal share of the row's
// (layer, K|V, head) sequences x kept entries x 16-byte units, four in flight
// per thread.  Bound by the launch and dependent round trips (path, entries)
// up to about 10 MB, by HBM beyond: 4.1 us for one row of 32 layers x 32 heads x
// 128 (5 MB), 7.2 us for 16 rows of 36 layers x 8 heads x 128 (17 MB).
__global__ __launch_bounds__(kBlock) void k_tree_compact(CompactParams p) {
  __shared__ int s_path[kMaxNodes], s_red[kBlock / kWave];
  const int b = blockIdx.y, P = p.depth + 1;
  const int acc = p.accept_len[b];
  int bad = acc < 0 || acc > p.depth;
  if ((int)threadIdx.x < P) {
    const int at = p.path[(size_t)b * P + threadIdx.x];
    s_path[threadIdx.x] = at;
    bad |= (int)threadIdx.x <= acc && (at < 0 || at >= p.N);
  }
  if (block_or_int(bad, s_red)) {  // nothing of this row is written
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, SPECDEC_S_TREE);
    return;
  }
  const int kept = acc + 1;
  if (blockIdx.x == 0 && (int)threadIdx.x < acc)
    p.draft_path[(size_t)b * p.depth + threadIdx.x] = p.draft[(size_t)b * p.N + s_path[threadIdx.x + 1]];
  const uint32_t run = (uint32_t)(kept * p.units);  // a sequence's kept units, contiguous in the output
  const FastDiv run_div = fast_div(run);
  const uint32_t total = (uint32_t)p.seqs * run, step = gridDim.x * kBlock;
  constexpr int NB = 4;
  for (uint32_t i0 = blockIdx.x * kBlock + threadIdx.x; i0 < total; i0 += NB * step) {
    u32x4 v[NB];
    size_t to[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const uint32_t i = min(i0 + k * step, total - 1);
      const uint32_t s = fdiv(i, run_div), r = i - s * run;
      const uint32_t j = fdiv(r, p.unit_div), u = r - j * (uint32_t)p.units;
      const uint32_t lk = fdiv(s, p.head_div), h = s - lk * (uint32_t)p.H;
      const size_t seq = ((size_t)lk * p.B + b) * p.H + h;
      v[k] = __builtin_nontemporal_load(static_cast<const u32x4 *>(p.kv_new) + (seq * p.N + s_path[j]) * p.units + u);
      to[k] = (seq * P + j) * p.units + u;
    }
#pragma unroll
    for (int k = 0; k < NB; ++k)
      if (i0 + k * step < total) static_cast<u32x4 *>(p.kv_path)[to[k]] = v[k];
  }
}

hipError_t launch_tree_compact(CompactParams p, hipStream_t s) {
  p.unit_div = host_fast_div((uint32_t)p.units);
  p.head_div = host_fast_div((uint32_t)p.H);
  // workgroups per row: enough that every thread has four units, up to eight
  // workgroups per CU over the whole batch
  const int64_t most = (int64_t)p.seqs * (p.depth + 1) * p.units;
  int64_t wgs = (most + 4 * kBlock - 1) / (4 * kBlock);
  const int64_t cap = (8LL * device_cus() + p.B - 1) / p.B;
  wgs = wgs < 1 ? 1 : wgs > cap ? cap : wgs;
  hipLaunchKernelGGL(k_tree_compact, dim3((unsigned)wgs, (unsigned)p.B), dim3(kBlock), 0, s, p);
  return hipGetLastError();
}

}  // namespace sd
