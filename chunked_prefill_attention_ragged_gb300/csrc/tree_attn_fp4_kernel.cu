// Tree attention over a cache of 4-bit entries: the mathematics, the split of the work, the products and the
// softmax of tree_attn_kernel.cu (a cluster of two CTAs runs a unit of 128 pairs with cta_group::2 products),
// over keys and values that are made bf16 on their way into shared memory.
//
// Eight warps make them: four the CTA's 64 keys of a tile as the half of S's B operand, four the tile's 128
// keys x 256 of the value columns.  A lane has four 32-value groups (16 bytes,
// one scale) at a time: it loads them into registers while the products read the tile before, waits until four
// panels are free, and writes 64 bytes of each in the swizzle that the products expect.  Entries go straight from L2 to registers: there is no
// room for them in shared memory beside Q (72 KB), a tile (136 KB) and P.
//   warp 0     Q producer
//   warp 1     even CTA: issues every product
//   warp 2     brings rows of the tiles to come into L2
//   warp 3     TMEM allocation; ropes
//   warps 4-7  softmax
//   warps 8-11 keys, 12-15 values
// A code becomes bf16 by moving its bits to a bf16's low exponent bits and one product by 2^126 times the
// scale, exact; scales above 2, where that factor has no bf16, take two products (a tile in which a warp
// meets one).  A row with a scale byte above 252 has NaN in its rope, which only S sees, and zeros for values,
// so that it cannot reach rows that do not see it.  Rows that are not there are zeros.
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "tree_core.cuh"

namespace mla {
namespace {

constexpr int NTHREADS = 512;
constexpr int LAUNCH_REGS = 128;
constexpr int REGS_CTRL = 88, REGS_SOFTMAX = 216, REGS_ROWS = 104;
static_assert(REGS_CTRL + REGS_SOFTMAX + 2 * REGS_ROWS <= 4 * LAUNCH_REGS, "register split exceeds the launch allocation");
constexpr int AHEAD = 2;   // tiles between the one being made and the one brought into L2

template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
// Bytes of a word above 252 (in their top bits).
__device__ __forceinline__ uint32_t above252(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x03030303u) & w & 0x80808080u; }

// A group's 32 values to four 16-byte pieces.  Each code is multiplied by `m` and, where the scales are `big`,
// by `m2`.
__device__ __forceinline__ void put_group(const uint32_t* at, uint32_t flip, uint32_t more, const uint4& w, bool big, uint32_t m,
                                          uint32_t m2) {
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  uint32_t r[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    fp4_fields(words[i], r[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) r[i][k] = mul_bf16x2(r[i][k], m);
  }
  if (big) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) r[i][k] = mul_bf16x2(r[i][k], m2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) st_shared_v4((at[i] ^ flip) + more, r[i][0], r[i][1], r[i][2], r[i][3]);
}

// A warp's part of what it writes is there: handed to the products' proxy, told to the even CTA.
__device__ __forceinline__ void tell(const Ctx& c, int b, int lane) {
  fence_async_shared();
  __syncwarp();
  if (lane == 0) {
    if (c.rank) mbar_arrive_remote(mapa_shared(c.bar(b), 0));
    else mbar_arrive(c.bar(b));
  }
}

// What the eight warps do is a line of stages, two for each tile: four panels of 64 rows each.  Keys (warps
// 8-11): panels 0-3 and 4-7 of the CTA's 64 keys; values (warps 12-15): the CTA's four panels, of the tile's
// first and second 64 keys.  A warp has 16 rows.  The bytes of the stage after next are loaded when a stage is done: most of a tile's time before they are needed.  One loop
// for both, and short: straight code for a tile of each did not stay in the instruction cache (see below).
//
// Lane (panel, row % 4, half) = (l / 8, l / 2 % 4, l % 2) has a piece of rows 4 j + row % 4 of the warp's, j < 4:
// a load takes 128 bytes of four rows, and eight lanes of a store have eight different bank groups.
struct Stage {
  uint4 code[4];
  uint32_t scale[4];
};
__device__ void run_rows(const Ctx& c, const TreeLaunch& p, Parts parts, bool values, volatile int* begun) {
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3, r4 = (lane >> 1) & 3;
  const int group = 2 * (lane >> 3) + (lane & 1);   // of the stage's eight
  const uint32_t dst = c.sbase + (values ? OFF_V : OFF_K);
  uint32_t at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) at[i] = dst + (lane >> 3) * QP + (16 * w4 + r4) * 128 + (((4 * (lane & 1) + i) ^ r4) << 4);
  const int full = values ? VF : KF, empty = values ? VE : KE;
  // The key of stage 0 that this lane looks up (lanes 0-15: the warp's rows), how much further stage 1's is,
  // and where a stage's bytes lie in an entry.
  const int first = (values ? 0 : 64 * (int)c.rank) + 16 * w4 + (lane & 15), second = values ? 64 : 0;
  const int part = values ? (int)c.rank : 0, step = values ? 0 : 1;
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(p.t.cache);
  int tiles = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    const int64_t end = min((int64_t)u.hi * KEYS, (int64_t)u.q.kv);
    // A block as the table has it: looked at a tile later, so that nothing waits for it here.
    auto find = [&](int64_t key) {
      return key < end ? __ldg(p.t.block_table + (int64_t)u.r * p.t.max_blocks + block_of(p, (int)key)) : 0;
    };
    auto get = [&](int32_t blk, int64_t key, int s, Stage* to) {
      const int32_t mine = key < end ? block_row(p, blk == PAST_END ? -1 : blk, key) : p.oob_row;
      const int at_code = 128 * (part + step * s) + 16 * group, at_scale = FP4_SCALES + 8 * (part + step * s) + group;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t row = __shfl_sync(0xffffffffu, mine, 4 * j + r4);
        to->code[j] = make_uint4(0, 0, 0, 0);
        to->scale[j] = 0;
        if (row != p.oob_row) {
          const uint8_t* e = cache + (int64_t)row * FP4_ENTRY;
          to->code[j] = load16(e + at_code);
          to->scale[j] = __ldg(e + at_scale);
        }
      }
    };
    int64_t key = (int64_t)u.lo * KEYS + first;
    Stage now, next;
    get(find(key), key, 0, &now);
    get(find(key + second), key + second, 1, &next);
    key += KEYS;
    int32_t blk0 = find(key), blk1 = find(key + second);   // of the two stages after those
#pragma unroll 1
    for (int n = 0; n < 2 * (u.hi - u.lo); ++n) {
      const int s = n & 1;
      if (s == 0 && !values && w4 == 0 && lane == 0) *begun = tiles;
      __syncwarp();
      if (tiles > 0 && !c.wait_warp(empty + s, (tiles - 1) & 1)) {
        ok = false;
        break;
      }
      const uint32_t most = max(max(now.scale[0], now.scale[1]), max(now.scale[2], now.scale[3]));
      const bool big = __any_sync(0xffffffffu, most > 128);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t b = now.scale[j];
        // 2^126 times the scale, or one after the other; values of a row that is NaN are zeros
        uint32_t m = big ? 0x7e80u : (b + 126) << 7;
        if (b > FP4_MAX_SCALE) m = 0;
        put_group(at, (j & 1) << 6, s * 4 * QP + j * 512, now.code[j], big, m | m << 16,
                  scale_bf16x2(b > FP4_MAX_SCALE ? 0 : b));
      }
      tell(c, full + s, lane);
      now = next;
      const int64_t k = key + (s ? second : 0);
      get(s ? blk1 : blk0, k, s, &next);
      if (s == 0) {
        blk0 = find(k + KEYS);
      } else {
        blk1 = find(k + KEYS);
        key += KEYS;
        ++tiles;
      }
    }
  }
}

// Warp 3: the ropes of the CTA's 64 keys, K's last panel.  Lane i has 16 bytes of rows 4 j + i / 8; a row with
// a scale byte above 252 gets NaN.
__device__ void run_ropes(const Ctx& c, const TreeLaunch& p, Parts parts) {
  const int lane = threadIdx.x & 31, ch = lane & 7;
  const uint32_t dst = c.sbase + OFF_K + 8 * QP;
  int tiles = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    int64_t key0 = (int64_t)u.lo * KEYS + 64 * c.rank;
    KeyBlocks b = find_blocks(p, u, key0, lane);
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++tiles, key0 += KEYS) {
      const KeyRows k = find_rows(p, b, key0, lane);
      if (t + 1 < u.hi) b = find_blocks(p, u, key0 + KEYS, lane);
      // which of a lane's two rows are NaN
      uint32_t bad[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 s = make_uint4(0, 0, 0, 0);
        if (k.r[i] != p.oob_row) s = load16(reinterpret_cast<const uint8_t*>(p.t.cache) + (int64_t)k.r[i] * FP4_ENTRY + FP4_SCALES);
        bad[i] = __ballot_sync(0xffffffffu, (above252(s.x) | above252(s.y) | above252(s.z) | above252(s.w)) != 0);
      }
      if (tiles > 0 && !c.wait_warp(KE + 2, (tiles - 1) & 1)) {
        ok = false;
        break;
      }
#pragma unroll 2
      for (int j = 0; j < 16; ++j) {
        const int key = 4 * j + (lane >> 3);
        const int32_t row = __shfl_sync(0xffffffffu, j < 8 ? k.r[0] : k.r[1], key & 31);
        const bool there = row != p.oob_row;
        const uint8_t* src = (there ? reinterpret_cast<const uint8_t*>(p.t.cache) + (int64_t)row * FP4_ENTRY + FP4_ROPE
                                    : reinterpret_cast<const uint8_t*>(p.t.q)) + ch * 16;
        cp_async16(dst + key * 128 + ((ch ^ (key & 7)) << 4), src, there ? 16 : 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      if (bad[0] | bad[1]) {
        __syncwarp();   // (a row's pieces are other lanes' copies)
        for (int j = 0; j < 16; ++j) {
          const int key = 4 * j + (lane >> 3);
          if ((bad[j >> 3] >> (key & 31)) & 1)
            st_shared_v4(dst + key * 128 + ch * 16, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        }
      }
      tell(c, KF + 2, lane);
    }
  }
}

__device__ void run_queries(const Ctx& c, Parts parts, const CUtensorMap* tq) {
  const int lane = threadIdx.x & 31;
  int units = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    if (lane == 0) {
      if (units > 0) ok = c.wait(QE, (units - 1) & 1);
      if (ok) {
        expect_both(c, QF, NP * QP);
        tma_load_3d_pair(c.sbase + OFF_Q, tq, mapa_shared(c.bar(QF), 0), 0, (int32_t)(u.pair0 + 64 * c.rank), 0);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) ++units;
  }
  if (lane == 0) {
    if (c.rank == 0) {
      if (units) c.drain(QF, (units - 1) & 1);
    } else if (!ok) {
      settle();
    }
  }
}

// Warp 2: this CTA's keys of the tiles to come into L2, a lane an entry.  It follows the keys' count of
// tiles and gives up quietly.
__device__ void run_prefetch(const Ctx& c, const TreeLaunch& p, Parts parts, const volatile int* begun) {
  const int lane = threadIdx.x & 31;
  int tiles = 0;
  Part u;
  while (parts.next(&u)) {
    for (int t = u.lo; t < u.hi; ++t, ++tiles) {
      const uint64_t t0 = global_timer_ns();
      while (*begun < tiles) {
        __nanosleep(200);
        if (*c.abort_flag || global_timer_ns() - t0 > p.wait_limit_ns) return;
      }
      __syncwarp();
      if (t + AHEAD < u.hi) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t key = (int64_t)(t + AHEAD) * KEYS + 64 * c.rank + 32 * i + lane;
          if (key < u.q.kv) {
            const int32_t row = block_row(p, table_block(p, u, key), key);
            const uint8_t* e = reinterpret_cast<const uint8_t*>(p.t.cache) + (int64_t)row * FP4_ENTRY;
            if (row != p.oob_row)
              asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(e), "r"(FP4_ENTRY) : "memory");
          }
        }
      }
    }
  }
}

__global__ void __launch_bounds__(NTHREADS, 1)
tree_attn_fp4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ TreeLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ StartRec start;
  __shared__ int64_t count;
  __shared__ JoinRec join;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + OFF_MISC + 4);
  int* begun = reinterpret_cast<int*>(smem + OFF_MISC + 8);   // tiles that the keys' first warp has begun, less one
  const uint32_t rank = cluster_ctarank();
  const int worker = blockIdx.x >> 1;
  const Ctx c{smem_addr(smem), abort_flag, p.t.status, p.wait_limit_ns, rank};
  ReqWords words{0, 0, 0};   // (on their way while the barriers are made)
  if ((int)threadIdx.x < p.t.batch) words = load_words(p.t, threadIdx.x);
  if (warp == 1) {
    // P: every softmax warp of both CTAs; maxima: the two warps of 32 rows; keys and values: four warps of
    // each CTA; ropes: one.
    static_assert(NBAR <= 32, "a lane each");
    const bool rows = lane == KF || lane == KF + 1 || lane == VF || lane == VF + 1;
    if (lane < NBAR) mbar_init(c.bar(lane), lane == PR || rows ? 8 : lane == KF + 2 || lane == XB || lane == XB + 1 ? 2 : 1);
    if (lane == 0) {
      *abort_flag = 0;
      *begun = -1;
    }
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tm_q);
  if (warp == 3) {   // one warp of each CTA of the pair, together
    tmem_alloc_pair(smem_addr(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  if (warp == 3) cluster_arrive();   // (see tree_attn_kernel)
  else cluster_arrive_relaxed();
  find_piece<NTHREADS>(p.t, words, worker, p.workers, blockIdx.x == 0, &start, &count, &join);
  char* ws = static_cast<char*>(p.t.workspace);
  if (threadIdx.x == 0 && rank == 0) reinterpret_cast<JoinRec*>(ws)[worker] = join;
  __syncwarp();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const Parts parts(p.t, start, count);
  if (warp < 4) {
    setmaxnreg_dec<REGS_CTRL>();
    if (warp == 0) run_queries(c, parts, &tm_q);
    else if (warp == 1 && rank == 0) run_mma<FP4>(c, p, parts, tmem);
    else if (warp == 2) run_prefetch(c, p, parts, begun);
    else if (warp == 3) run_ropes(c, p, parts);
  } else if (warp < 8) {
    setmaxnreg_inc<REGS_SOFTMAX>();
    run_softmax(c, p, parts, tmem, ws + WS_SLOTS + (size_t)worker * 2 * SLOT_BYTES, smem);
  } else {
    setmaxnreg_dec<REGS_ROWS>();
    run_rows(c, p, parts, warp >= 12, begun);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // Neither CTA leaves (freeing shared memory and TMEM) while the even CTA's products may still
  // read or write the other's.
  cluster_sync();
  tc_fence_after();
  if (warp == 3) {
    __syncwarp();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

cudaLaunchConfig_t pair_config(cudaLaunchAttribute* attr, int workers, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * workers, 1, 1);
  cfg.blockDim = dim3(NTHREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters that run at once on the current device (0 on error), no more than the workspace has room for.
int max_workers() {
  static PerDeviceOnce configured;
  static int workers[PerDeviceOnce::kMaxDevices] = {};
  const cudaError_t e = configured.run([] {
    cudaError_t r = cudaFuncSetAttribute(tree_attn_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (r != cudaSuccess) return r;
    // The split of the registers takes for granted that every thread starts with LAUNCH_REGS.
    cudaFuncAttributes attrs;
    r = cudaFuncGetAttributes(&attrs, tree_attn_fp4_kernel);
    if (r != cudaSuccess) return r;
    if (attrs.numRegs != LAUNCH_REGS) return cudaErrorInvalidConfiguration;
    int dev = 0, n = 0;
    r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pair_config(attr, 1, nullptr);
    r = cudaOccupancyMaxActiveClusters(&n, tree_attn_fp4_kernel, &cfg);
    if (r != cudaSuccess) return r;
    const int64_t room = (tree_workspace_bytes() - (int64_t)WS_SLOTS) / (int64_t)(2 * SLOT_BYTES);
    workers[dev] = (int)std::min<int64_t>(n, std::min<int64_t>(room, MAX_WORKERS));
    return r;
  });
  int dev = 0;
  if (e != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return 0;
  return workers[dev];
}

}  // namespace

cudaError_t launch_tree_attention_fp4(const TreeParams& t, cudaStream_t stream) {
  const int64_t pairs = (t.total_rows * t.num_heads + t.batch - 1) / t.batch;   // of a request, on average
  if (pairs <= 32) return launch_tree_attention_fp4_few(t, (int)pairs, stream);
  const TreeLaunch p = tree_launch(t, max_workers());
  if (p.workers <= 0) return cudaErrorInvalidConfiguration;
  CUtensorMap tq;
  const uint64_t dims[3] = {64, (uint64_t)t.total_rows * (uint64_t)t.num_heads, NP}, strides[2] = {576 * 2, 64 * 2};
  const uint32_t box[3] = {64, 64, NP};   // 64 rows, panel by panel
  if (make_tensor_map_bf16(&tq, t.q, 3, dims, strides, box) != MLA_OK) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pair_config(attr, p.workers, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_attn_fp4_kernel, tq, p);
  return e != cudaSuccess ? e : launch_tree_join(p, stream);
}

}  // namespace mla
