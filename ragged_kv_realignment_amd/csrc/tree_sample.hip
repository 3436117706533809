// Sampled verification of a tree of drafts from the target's probabilities.
//
// At a node whose target distribution is p, the children's tokens x_1, x_2, ...
// (in index order, a repeated token once) are tried in turn against what is
// left of p: child k is taken with probability p(x_k) / (1 - p(x_1) - ... -
// p(x_{k-1})), and if none is taken the row's next token is drawn from p with
// those tokens removed.  Whatever the tree, the token that follows the node is
// then distributed as p: P(x_k) is the product of the k - 1 refusals, which
// telescopes to 1 - p(x_1) - ... - p(x_{k-1}), times the chance above, and any
// other token keeps p's ratio to its remaining mass.  No draft distribution
// enters, so a tree may hold the draft model's best tokens or drawn ones alike.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <math.h>
#include "coherent.h"
#include "device_common.h"
#include "launch.h"
#include "specdec.h"
#include "tree_common.h"
#include "wave_dpp.h"

namespace sd {

typedef float f32x4 __attribute__((ext_vector_type(4)));

namespace {

constexpr int NT = kSampleThreads;
constexpr int NW = NT / kWave;
constexpr int kBatch = 8;  // 16-byte vectors a thread has in flight over a long run

__device__ __forceinline__ double mass(float x) { return x > 0.0f ? (double)x : 0.0; }

// Whether id v is one of the n removed tokens.
__device__ __forceinline__ bool is_gone(const int *gone, int n, int v) {
  bool hit = false;
  for (int k = 0; k < n; ++k) hit |= gone[k] == v;
  return hit;
}

// A thread's run of ids [lo, hi) of the stop row, its probabilities in batches
// of NB vectors (VW = 4) or scalars: each(v, x, kept) sees every id in order and
// says whether to go on.  `n` removed tokens are looked for only where n > 0.
template <int VW, int NB, typename F>
__device__ __forceinline__ void each_id(const float *p, int lo, int hi, const int *gone, int n, F each) {
  if constexpr (VW == 4) {
    for (int v0 = lo; v0 < hi; v0 += 4 * NB) {
      f32x4 x[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k)  // in range: a repeated load, never used
        x[k] = *reinterpret_cast<const f32x4 *>(p + min(v0 + 4 * k, hi - 4));
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (v0 + 4 * k >= hi) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = v0 + 4 * k + e;
          if (!each(v, mass(x[k][e]), n == 0 || !is_gone(gone, n, v))) return;
        }
      }
    }
  } else {
    for (int v = lo; v < hi; ++v)
      if (!each(v, mass(p[v]), n == 0 || !is_gone(gone, n, v))) return;
  }
}

}  // namespace

// Batch row b's stop row is cut into S splits of NT runs of R consecutive ids,
// a workgroup per split (numbered split-major) and a run per thread.
//  1. Every workgroup of row b decides the walk, alike in all of them: a node
//     per thread, its token's target probability at its parent gathered in one
//     round trip; each thread then goes over its earlier siblings in LDS for the
//     mass that is left (fp64, subtracted in index order from 1) and marks
//     itself in its parent's slot if it is accepted (the lowest stays); thread 0
//     follows the slots from the root to the stop node.
//  2. Each thread sums its run in id order in fp64: without the stop node's
//     refused children, and with them (the fallback where nothing else has
//     mass).  The workgroup's totals and, for runs over 8 ids, the runs' sums go
//     to the row's workspace block.
//  3. The last of the row's workgroups to count itself draws u * total: the
//     split by a scan of the totals across lanes, the run by a scan of its sums
//     in thread order, the id by walking the run again with step 2's additions.
// Stores and loads of the sums pass the non-coherent L2 (sc1), and the count is
// issued after the stores have completed, as in verification of a chain.
// Bound by latency: the dependent loads (draft and parent, the gathered
// probabilities, the stop row, the totals, the crossing run) and two barriers
// between each.  8.1 us for one row of 9 nodes and 32000 ids, 10.9 us for 32 rows
// of 24 nodes (4 MB).
template <int VW, int NB, bool STORE_RUNS>
__global__ __launch_bounds__(NT) void k_verify_tree_sample(TreeSampleParams p, FastDiv b_div) {
  const int B = p.B, S = p.S, R = p.R, N = p.N, V = p.V;
  const int split = (int)fdiv(blockIdx.x, b_div);
  const int b = (int)blockIdx.x - split * B;
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = t / kWave;
  __shared__ int s_par[kMaxNodes], s_x[kMaxNodes], s_next[kMaxNodes], s_gone[kMaxNodes];
  __shared__ double s_p[kMaxNodes];
  __shared__ int s_flags, s_last, s_sel, s_stop, s_acc, s_ngone;
  __shared__ double s_w[NW], s_f[NW];
  __shared__ int s_i[NW];
  __shared__ float s_ud;
  if (t == 0) s_flags = s_ngone = 0;
  // 1. the walk
  int par = -1, x = 0;
  float u = 0.0f, ud = 0.0f;
  double px = 0.0;
  bool bad = false, out = false;
  if (t < N) {
    const size_t at = (size_t)b * N + t;
    const int raw = p.parent[at];
    x = p.draft[at];
    u = p.u_accept[at];
    ud = p.u_draw[at];
    if (t > 0) par = node_parent(t, raw, bad);
    out = par >= 0 && (x < 0 || x >= V);
    if (par >= 0 && !out) px = mass(p.p[((size_t)b * N + par) * V + x]);
    s_par[t] = par;
    s_x[t] = x;
    s_p[t] = px;
    s_next[t] = N;
  }
  __syncthreads();
  if (bad || out) atomicOr(&s_flags, (bad ? SPECDEC_S_TREE : 0) | (out ? SPECDEC_S_DRAFT_RANGE : 0));
  if (par >= 0) {  // a token that an earlier sibling has counts once
    bool again = false;
    for (int j = par + 1; j < t; ++j) again |= s_par[j] == par && s_x[j] == x;
    if (again) px = 0.0;
  }
  __syncthreads();
  if (par >= 0) s_p[t] = px;
  __syncthreads();
  if (par >= 0) {
    double left = 1.0;
    for (int j = par + 1; j < t; ++j) left -= s_par[j] == par ? s_p[j] : 0.0;
    if ((double)u * left < px) atomicMin(&s_next[par], t);
  }
  __syncthreads();
  if (t == 0) {
    int cur = 0, a = 0;
    int32_t *path = p.path + (size_t)b * (p.depth + 1);
    if (split == 0) path[0] = 0;
    while (a < p.depth && s_next[cur] < N) {
      cur = s_next[cur];
      ++a;
      if (split == 0) path[a] = cur;
    }
    s_stop = cur;
    s_acc = a;
  }
  __syncthreads();
  const int stop = s_stop, acc = s_acc;
  if (split == 0 && t > acc && t <= p.depth) p.path[(size_t)b * (p.depth + 1) + t] = -1;
  if (t == stop) s_ud = ud;
  // the refused children of the stop node (at the depth limit none was tried)
  if (par == stop && acc < p.depth && !out) s_gone[atomicAdd(&s_ngone, 1)] = x;
  __syncthreads();
  const int ngone = s_ngone;
  const float *row = p.p + ((size_t)b * N + stop) * V;
  char *blk = p.ws + (size_t)b * kSampleRowBytes;
  unsigned int *counter = reinterpret_cast<unsigned int *>(blk);
  const __amdgpu_buffer_rsrc_t rt = coherent_rsrc(blk + kAtomicLine, kSampleSplits * 16);
  const __amdgpu_buffer_rsrc_t rr = coherent_rsrc(blk + kAtomicLine + kSampleSplits * 16, kSampleSplits * NT * 16);

  // how many removed tokens lie in [lo, hi): only such runs look for them
  auto gone_in = [&](int lo, int hi) {
    int n = 0;
    for (int k = 0; k < ngone; ++k) n += s_gone[k] >= lo && s_gone[k] < hi;
    return n ? ngone : 0;
  };
  auto run_sums = [&](int lo, int hi, double &w, double &f) {
    double cw = 0.0, cf = 0.0;
    each_id<VW, NB>(row, lo, hi, s_gone, gone_in(lo, hi), [&](int, double m, bool kept) {
      cw += kept ? m : 0.0;
      cf += m;
      return true;
    });
    w = cw;
    f = cf;
  };

  // 2. this thread's run, and the split's totals
  {
    const int g = split * NT + t;
    const int lo = (int)min((long)V, (long)g * R), hi = min(V, lo + R);
    double w, f;
    run_sums(lo, hi, w, f);
    if constexpr (STORE_RUNS) st_pair(rr, (uint32_t)g * 16u, w, f);
    const double ww = wave_total_f64(w), wf = wave_total_f64(f);
    if (lane == 0) {
      s_w[wv] = ww;
      s_f[wv] = wf;
    }
    if constexpr (STORE_RUNS) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (t == 0) {
      double tw = 0.0, tf = 0.0;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        tw += s_w[k];
        tf += s_f[k];
      }
      st_pair(rt, (uint32_t)split * 16u, tw, tf);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      s_last = atomicAdd(counter, 1u) == (unsigned)(S - 1);
    }
  }
  __syncthreads();
  if (!s_last) return;

  // 3. the draw; lane k of every wave holds split k's totals (S <= 16)
  double mw, mf;
  ld_pair(rt, (uint32_t)min(lane, S - 1) * 16u, mw, mf);
  if (lane >= S) mw = mf = 0.0;
  const double iw = wave_scan_f64(mw), jf = wave_scan_f64(mf);
  const double Tw = lane_f64(iw, kWave - 1), Tf = lane_f64(jf, kWave - 1);
  const bool full = !(Tw > 0.0);  // nothing left: the whole of p
  const double T = full ? Tf : Tw;
  int j = 0;
  if (T > 0.0) {
    const double target = (double)s_ud * T;
    const double ms = full ? mf : mw, is = full ? jf : iw;
    const unsigned long long hit = __ballot(ms > 0.0 && is > target), some = __ballot(ms > 0.0);
    const int ss = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some);
    const double P = lane_f64(is - ms, ss);
    const double tgt = hit ? target : INFINITY;  // no crossing by rounding: the last id with mass
    const int g = ss * NT + t;
    const int lo = (int)min((long)V, (long)g * R), hi = min(V, lo + R);
    double w, f;
    if constexpr (STORE_RUNS) ld_pair(rr, (uint32_t)g * 16u, w, f);
    else run_sums(lo, hi, w, f);
    const double m = full ? f : w;
    const double incl = wave_scan_f64(m);
    if (lane == kWave - 1) s_w[wv] = incl;
    __syncthreads();
    double e = 0.0;
#pragma unroll
    for (int k = 0; k < NW; ++k)
      if (k < wv) e += s_w[k];
    const double before = P + (e + (incl - m));
    const bool cross = m > 0.0 && before + m > tgt;
    const int who = block_first<NT>(cross, s_i);
    const int me = who != INT_MAX ? who : block_last<NT>(m > 0.0, s_i);
    if (t == me) {
      const double to = who != INT_MAX ? tgt : INFINITY;
      int at = 0;
      double c = 0.0;
      each_id<VW, NB>(row, lo, hi, s_gone, full ? 0 : gone_in(lo, hi), [&](int v, double q, bool kept) {
        const double d = kept ? q : 0.0;
        c += d;
        if (d > 0.0) at = v;
        return !(before + c > to);
      });
      s_sel = at;
    }
    __syncthreads();
    j = s_sel;
  } else if (t == 0) {
    atomicOr(&s_flags, SPECDEC_S_PROB);
  }
  __syncthreads();
  if (t == 0) {
    p.accept_len[b] = acc;
    p.next_token[b] = j;
    store_agent(counter, 0u);
    set_status(p.status, s_flags);
  }
}

hipError_t launch_verify_tree_sample(const TreeSampleParams &p, hipStream_t s) {
  const bool vec = p.V % 4 == 0 && reinterpret_cast<uintptr_t>(p.p) % 16 == 0;
  const dim3 grid((unsigned)((long)p.B * p.S));
  const FastDiv b_div = host_fast_div((uint32_t)p.B);
  // runs of 8 ids: summed again by the drawing workgroup instead of stored
  if (vec && p.R == 8)
    hipLaunchKernelGGL((k_verify_tree_sample<4, 2, false>), grid, dim3(NT), 0, s, p, b_div);
  else if (vec)
    hipLaunchKernelGGL((k_verify_tree_sample<4, kBatch, true>), grid, dim3(NT), 0, s, p, b_div);
  else
    hipLaunchKernelGGL((k_verify_tree_sample<1, 1, true>), grid, dim3(NT), 0, s, p, b_div);
  return hipGetLastError();
}

}  // namespace sd
