// Which drafted nodes are kept, and the token that follows (definition in include/mla_prefill.h).
//
// Mathematics.  Drawn children: with target p and draft q at a node, the residual after k refusals is
// proportional to (p - a_k q)+, a_0 = 0, a_1 = 1, a_{k+1} = a_k + F(a_k), F(a) = sum (p - a q)+: from
// r_{k+1} = (r_k - q)+ with r_k = (p - a_k q)+ / F(a_k) the factor 1 / F(a_k) comes out in front.  So one
// number stands for all refusals so far, and each needs one pass over the two rows.  Given children: the
// residual is p without their tokens, and needs none.  The next token is drawn by inverse sums from what
// is left at the last kept node.
//
// Sums are integers in units of 2^-43: exact whatever their order, so that the token does not depend on
// how the row is split; an entry is off by half a unit at most, at random.  An entry's integer comes from two
// additions of constants, whose results' low bits it is (a conversion of fp32 to 64 bits takes eight times as long
// here).  (p - a q)+ is made by two fp32 multiply-adds with a in two fp32 parts (2^-48 of it): off by 2^-24 of p at
// most, at random, and so are, by less, the sums of them and the a of the next refusal.
//
// One launch; a cluster of up to eight CTAs has a request, each a slice of the vocabulary.  Every CTA walks
// the tree by itself (its few numbers are loaded at once, for all nodes) and comes to the same end; only
// sums over the vocabulary, and the search in them, are shared out.  A warp sums 512 entries at a time and
// leaves each such sum in shared memory, so that the search looks at the sums and one group of entries.
// What bounds it: for few requests latencies, one behind the other (the nodes, the row's slice, the cluster's
// sum, the group); for many the reading of the last nodes' rows.  (Replayed graphs: 1 request of 5 given nodes over 32,003
// entries 8.7 us; 64 of up to 16 drawn ones over 131,072 28.1-28.7 us, of which the rows that are read, 67 MB, take 10 at a copy's rate: a node's
// refusals are one pass over its rows each, and the next pass starts from the last one's sum.)
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int THREADS = 256, NWARPS = THREADS / 32;
constexpr int BLOCKS = 4;                  // of an SM: 64 requests' clusters of eight are all there at once
constexpr int GROUP = 512;                 // entries of one sum
constexpr int LOADED = 512;                // nodes whose numbers are held in shared memory
constexpr int MAX_CLUSTER = 8;
constexpr int SLICE = 4096;                // entries for which another CTA is worth its barriers
constexpr unsigned ALL = 0xffffffffu;
constexpr double UNIT = 1.0 / 8796093022208.0;   // 2^-43

__device__ __forceinline__ float probability(float x) { return __saturatef(x); }   // (a NaN: 0)
__device__ __forceinline__ float at(const float* p) { return probability(__ldg(p)); }
__device__ __forceinline__ float at(const __nv_bfloat16* p) { return probability(__bfloat162float(*p)); }

// x in [0, 1] as two integers, of units of 2^-20 (rounded) and of the rest in units of 2^-43: x + 8 has its last bit
// at 2^-20, the rest + 1.5 * 2^-20 at 2^-43.  Sums of up to 2^8 of them are exact in 32 bits each.
struct Fixed {
  uint32_t high, low;
  __device__ void add(float x) {
    const float t = x + 8.f, u = (x - (t - 8.f)) + 1.5f / 1048576.f;
    high += __float_as_uint(t) - __float_as_uint(8.f);
    low += __float_as_uint(u) - __float_as_uint(1.5f / 1048576.f);
  }
  __device__ uint64_t value() const { return ((uint64_t)high << 23) + (uint64_t)(int64_t)(int32_t)low; }
};
__device__ __forceinline__ uint64_t fixed(float x) {
  Fixed f{0, 0};
  f.add(x);
  return f.value();
}
// What is left of p after `a` times q, a = hi + lo.
__device__ __forceinline__ float left_of(float p, float q, float hi, float lo) {
  return __saturatef(fmaf(-lo, q, fmaf(-hi, q, p)));
}

// Sixteen bytes of a row as values.
__device__ __forceinline__ void unpack(const uint4& v, float* x, const float*) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = probability(__uint_as_float(w[i]));
}
__device__ __forceinline__ void unpack(const uint4& v, float* x, const __nv_bfloat16*) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = probability(__uint_as_float(w[i] << 16));
    x[2 * i + 1] = probability(__uint_as_float(w[i] & 0xffff0000u));
  }
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(ALL, v, d);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {   // sums up to and with each lane
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t o = __shfl_up_sync(ALL, v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ uint64_t load_cluster(const uint64_t* mine, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_addr(mine), rank)) : "memory");
  return v;
}

// The sum of one group of 512 entries, of which those below `vocab` exist.
template <class T>
__device__ __forceinline__ uint64_t group_sum(const T* p, const T* q, int64_t first, int64_t vocab, bool wide, float hi, float lo,
                                              int lane) {
  constexpr int EACH = 16 / sizeof(T), STEPS = GROUP / 32 / EACH;
  Fixed s{0, 0};
  if (wide) {
#pragma unroll
    for (int i = 0; i < STEPS; i += 2) {   // (two steps' loads at a time: more registers would halve the CTAs of an SM)
      uint4 a[2], b[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t e = first + (32 * (i + k) + lane) * EACH;
        const bool there = e < vocab;   // (all of the sixteen bytes: the vocabulary is a multiple of them)
        a[k] = there ? __ldg(reinterpret_cast<const uint4*>(p + e)) : make_uint4(0, 0, 0, 0);
        b[k] = there && q ? __ldg(reinterpret_cast<const uint4*>(q + e)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[EACH], y[EACH];
        unpack(a[k], x, p);
        unpack(b[k], y, p);
#pragma unroll
        for (int j = 0; j < EACH; ++j) s.add(left_of(x[j], y[j], hi, lo));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < GROUP / 32; i += 8) {
      float x[8], y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t e = first + 32 * (i + k) + lane;
        x[k] = e < vocab ? at(p + e) : 0.f;
        y[k] = e < vocab && q ? at(q + e) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s.add(left_of(x[k], y[k], hi, lo));
    }
  }
  return warp_sum(s.value());
}

// What the walk asks of all threads: a sum over the vocabulary, or the search in it, at a node with `a` times
// its draft (or its given children) taken off.
struct Ask {
  int pick, given, node;
  double a;
};
struct Node {
  int parent, token;   // parent -1: never kept
  float u, p, q;       // the uniform; target and draft of its token at its parent
};

template <class T>
__global__ void __launch_bounds__(THREADS, BLOCKS) verify_kernel(const __grid_constant__ VerifyParams v) {
  extern __shared__ uint64_t sums[];              // of the slice's groups
  __shared__ int parent_s[LOADED], token_s[LOADED];
  __shared__ float u_s[LOADED], p_s[LOADED], q_s[LOADED];
  __shared__ Ask ask;
  __shared__ uint64_t total_s[2], part_s[NWARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank(), ranks = (uint32_t)v.ranks;
  const int r = (int)(blockIdx.x / ranks);
  const int64_t V = v.vocab;
  const T* target = static_cast<const T*>(v.target);
  const T* draft = static_cast<const T*>(v.draft);
  const int64_t groups = (V + GROUP - 1) / GROUP, each = (groups + ranks - 1) / ranks;
  const int64_t g0 = min((int64_t)rank * each, groups), g1 = min(g0 + each, groups);
  int32_t* path = v.accepted + (int64_t)r * v.max_accepted;
  const int q0 = __ldg(v.qo + r), q1 = __ldg(v.qo + r + 1);
  const bool rows_ok = q0 >= 0 && q1 >= q0 && q1 <= v.total_rows;
  const int n = rows_ok ? q1 - q0 : 0;
  if (n == 0) {   // (the whole cluster returns)
    for (int64_t i = tid + (int64_t)rank * THREADS; i < v.max_accepted; i += ranks * THREADS) path[i] = -1;
    if (rank == 0 && tid == 0) {
      v.counts[r] = 0;
      v.next[r] = -1;
      if (!rows_ok && v.status) atomicOr(v.status, MLA_DEVSTAT_BAD_INDEX);
    }
    return;
  }
  if (rank == 0 && tid == 0) v.next[r] = -1;   // (whoever finds a token writes it behind a cluster's barrier)
  auto load = [&](int j, bool report) {
    Node d;
    d.parent = v.parents ? __ldg(v.parents + q0 + j) : j - 1;
    d.token = __ldg(v.tokens + q0 + j);
    d.u = fmaxf(__ldg(v.uniforms + q0 + j), 0.f);
    const bool parent_ok = j == 0 || (d.parent >= -1 && d.parent < j), token_ok = d.token >= 0 && d.token < V;
    if (report && v.status && (!parent_ok || (j > 0 && !token_ok))) atomicOr(v.status, MLA_DEVSTAT_BAD_INDEX);
    if (j == 0 || !parent_ok || !token_ok) d.parent = -1;
    d.p = d.q = 0.f;
    if (d.parent >= 0) {
      const int64_t e = (q0 + (int64_t)d.parent) * V + d.token;
      d.p = at(target + e);
      if (draft) d.q = at(draft + e);
    }
    return d;
  };
  for (int j = tid; j < n; j += THREADS) {
    const Node d = load(j, rank == 0);
    if (j < LOADED) {
      parent_s[j] = d.parent;
      token_s[j] = d.token;
      u_s[j] = d.u;
      p_s[j] = d.p;
      q_s[j] = d.q;
    }
  }
  auto node = [&](int j) { return j < LOADED ? Node{parent_s[j], token_s[j], u_s[j], p_s[j], q_s[j]} : load(j, false); };
  // Whether a sibling of `d` between its parent and node j has its token.
  auto same_before = [&](const Node& d, int j, int first, int step) {
    bool same = false;
    for (int k = d.parent + 1 + first; k < j && !same; k += step) {
      const Node e = node(k);
      same = e.parent == d.parent && e.token == d.token;
    }
    return same;
  };

  // The walk, of warp 0: from where it stands to its next question.
  int cur = 0, from = 1, length = 1;
  double a = 0.0, mass = 1.0;
  auto walk = [&]() {
    bool pick = length >= v.max_accepted;   // (a full path: as if `cur` had no children)
    bool full = pick, sum = false;
    while (!pick && !sum) {
      int child = -1;
      for (; from < n && child < 0; from += 32) {
        const int j = from + lane;
        const unsigned m = __ballot_sync(ALL, j < n && node(j).parent == cur);
        if (m) child = from + __ffs(m) - 1;
      }
      if (child < 0) {
        pick = true;
        break;
      }
      from = child + 1;
      const Node d = node(child);
      bool passes;
      if (draft) {
        passes = (double)d.u * (double)d.q * mass < fmax((double)d.p - a * (double)d.q, 0.0);
      } else {
        const double p = __any_sync(ALL, same_before(d, child, lane, 32)) ? 0.0 : (double)d.p;
        passes = (double)d.u * mass < p;
        if (!passes) mass -= p;
      }
      if (passes) {
        if (rank == 0 && lane == 0) path[length] = child;
        cur = child;
        ++length;
        a = 0.0;
        mass = 1.0;
        full = pick = length >= v.max_accepted;
      } else if (draft) {
        a += mass;
        sum = true;
      }
    }
    if (lane == 0) ask = Ask{pick, pick && !full && !draft, cur, a};
  };
  int sweeps = 0;
  uint64_t before = 0;   // what the slices before this one have
  // The sum over the vocabulary of what is left at a node, by the whole cluster.
  auto sweep = [&](int at_node, double times, bool given) {
    const T* p = target + (q0 + (int64_t)at_node) * V;
    const T* q = times != 0.0 ? draft + (q0 + (int64_t)at_node) * V : nullptr;
    const float hi = (float)times, lo = (float)(times - (double)hi);
    uint64_t mine = 0;
    for (int64_t g = g0 + warp; g < g1; g += NWARPS) {
      const uint64_t s = group_sum(p, q, g * GROUP, V, v.wide != 0, hi, lo, lane);
      if (lane == 0) sums[g - g0] = s;
      mine += s;
    }
    if (lane == 0) part_s[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      uint64_t off = 0;
      if (given) {   // the children's tokens are gone, each once
        for (int j = at_node + 1 + lane; j < n; j += 32) {
          const Node d = node(j);
          const int64_t g = d.token / GROUP;
          if (d.parent != at_node || g < g0 || g >= g1 || same_before(d, j, 0, 1)) continue;
          const uint64_t f = fixed(d.p);
          atomicAdd(reinterpret_cast<unsigned long long*>(sums + (g - g0)), 0ull - (unsigned long long)f);
          off += f;
        }
      }
      const uint64_t s = warp_sum((lane < NWARPS ? part_s[lane] : 0ull) - off);
      if (lane == 0) total_s[sweeps & 1] = s;
    }
    __syncwarp();
    cluster_sync();
    uint64_t all = 0;
    before = 0;
    for (uint32_t k = 0; k < ranks; ++k) {
      const uint64_t s = load_cluster(&total_s[sweeps & 1], k);
      if (k < rank) before += s;
      all += s;
    }
    ++sweeps;   // (the other total is free: every CTA has read it before it arrived here)
    return all;
  };
  __syncthreads();
  if (warp == 0) walk();
  __syncthreads();
  // A child that does not pass takes one sweep, so there are less than n of them.
  int swept = -1;   // the node that the sums are of (with what the last child left of it)
  uint64_t all = 0;
  for (int i = 0; i < n && !ask.pick; ++i) {
    swept = ask.node;
    all = sweep(ask.node, ask.a, false);
    if (warp == 0) {
      mass = (double)all * UNIT;
      __syncwarp();
      walk();
    }
    __syncthreads();
  }
  const Ask last = ask;
  const T* p = target + (q0 + (int64_t)last.node) * V;
  double times = last.a;
  bool given = last.given;
  if (swept != last.node) all = sweep(last.node, times, given);   // (its last child's refusal asked for them already)
  if (all == 0 && (times != 0.0 || given)) {   // nothing is left: p itself
    times = 0.0;
    given = false;
    all = sweep(last.node, times, given);
  }
  if (warp == 0 && rank == 0) {
    if (lane == 0) path[0] = 0;
    for (int i = length + lane; i < v.max_accepted; i += 32) path[i] = -1;
    if (lane == 0) v.counts[r] = length;
  }
  if (warp == 0 && all > 0) {
    const double u = fminf(fmaxf(__ldg(v.final_uniforms + r), 0.f), 1.f);
    uint64_t goal = (uint64_t)(u * (double)all);   // the least token whose sum passes u * all, and so its floor
    if (goal >= all) goal = all - 1;
    const uint64_t mine = __shfl_sync(ALL, total_s[(sweeps - 1) & 1], 0);
    if (goal >= before && goal - before < mine) {
      goal -= before;
      // the group
      uint64_t done = 0;
      int64_t g = g0;
      for (; g < g1; g += 32) {
        const uint64_t s = warp_scan(g + lane < g1 ? sums[g + lane - g0] : 0ull, lane) + done;
        const unsigned m = __ballot_sync(ALL, s > goal);
        if (m) {
          const int k = __ffs(m) - 1;
          const uint64_t below = __shfl_up_sync(ALL, s, 1);
          if (k > 0) done = __shfl_sync(ALL, below, k);
          g += k;
          break;
        }
        done = __shfl_sync(ALL, s, 31);
      }
      // the entry: sixteen in a row for each lane
      const T* q = times != 0.0 ? draft + (q0 + (int64_t)last.node) * V : nullptr;
      const float hi = (float)times, lo = (float)(times - (double)hi);
      const int64_t e0 = g * GROUP + lane * (GROUP / 32);
      float f[GROUP / 32];
#pragma unroll
      for (int i = 0; i < GROUP / 32; ++i) {
        const int64_t e = e0 + i;
        f[i] = e < V ? left_of(at(p + e), q ? at(q + e) : 0.f, hi, lo) : 0.f;
      }
      if (given) {
        for (int j = last.node + 1; j < n; ++j) {
          const Node d = node(j);
          if (d.parent != last.node || d.token < e0 || d.token >= e0 + GROUP / 32) continue;
#pragma unroll
          for (int i = 0; i < GROUP / 32; ++i)
            if (e0 + i == d.token) f[i] = 0.f;
        }
      }
      Fixed mine_f{0, 0};
#pragma unroll
      for (int i = 0; i < GROUP / 32; ++i) mine_f.add(f[i]);
      const uint64_t sum = mine_f.value();
      __syncwarp();
      const uint64_t s = warp_scan(sum, lane) + done;
      const unsigned m = __ballot_sync(ALL, s > goal);
      if (m && lane == __ffs(m) - 1) {
        uint64_t at_now = s - sum;
        int k = 0;
#pragma unroll
        for (int i = 0; i < GROUP / 32; ++i) {
          at_now += fixed(f[i]);
          if (at_now <= goal) k = i + 1;
        }
        v.next[r] = (int32_t)(e0 + k);
      }
    }
  }
  __syncwarp();
  cluster_sync();   // (nobody leaves while others read its total)
}

}  // namespace

int verify_ranks(int64_t vocab) {
  int ranks = 1;
  while (ranks < MAX_CLUSTER && vocab > (int64_t)ranks * SLICE) ranks *= 2;
  return ranks;
}

cudaError_t launch_verify(VerifyParams v, int batch, bool bf16, cudaStream_t stream) {
  const int size = bf16 ? 2 : 4;
  auto fits = [&](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
  v.wide = fits(v.target) && fits(v.draft) && v.vocab * size % 16 == 0;
  v.ranks = verify_ranks(v.vocab);
  const int64_t groups = (v.vocab + GROUP - 1) / GROUP, each = (groups + v.ranks - 1) / v.ranks;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)v.ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)batch * (unsigned)v.ranks);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)each * sizeof(uint64_t);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, v) : cudaLaunchKernelEx(&cfg, verify_kernel<float>, v);
}

}  // namespace mla
