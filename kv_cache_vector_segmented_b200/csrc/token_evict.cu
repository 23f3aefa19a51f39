// Eviction from the exact token cache (ri_token_evict): every (sequence, KV
// head) keeps its `keep` tokens of highest rank, and the kept tokens behind
// row `keep` move into the rows of the dropped ones.
//
// The order is total: held tokens (first and most recent positions) before
// all others, then larger weight, then lower row.  A token's rank is a 32-bit
// key (the order-preserving image of its weight, all ones when held), so the
// keep-th largest key is found by four 8-bit digits (radix selection), and
// ties on it are settled by counting in row order.  Every step is a count or
// a prefix sum: the result does not depend on the order in which threads run.
//
// One thread-block cluster per (sequence, KV head), one launch.  A block
// holds a contiguous slice of the rows' keys in shared memory (read once);
// the blocks add up their digit counts through distributed shared memory,
// with one cluster barrier per digit.  Bound: reading 8 bytes per token and
// moving 2 x 512 bytes per token that changes its row.
#include "common.cuh"
#include "internal.h"

namespace ri {

namespace {

constexpr int kThreads = 512;  // two blocks per SM at 64 registers
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
// rows whose keys and positions a block holds (8 bytes each); a longer slice
// (caches of more than 16 x this) is read again from global memory instead
constexpr int kMaxHeld = 24576;

struct EvictParams {
  ri_token_cache c, o;
  int budget, first, recent;
  int cluster;     // blocks per unit
  int32_t* holes;  // [units][W]: rows below keep whose tokens are dropped, in order
  int32_t* moved;  // [units][W]: rows from keep on whose tokens stay, in order
  int* status;
};

// Largest key for held tokens; a NaN weight ranks as -inf, -0 as +0.
__device__ __forceinline__ uint32_t rank_key(float w, int pos, int first, long long recent_from) {
  if (pos < first || pos > recent_from) return 0xFFFFFFFFu;
  if (w != w) w = -__int_as_float(0x7f800000);
  return float_order_key(w + 0.f);
}

// Shared memory every block of a cluster may read.
struct Exchange {
  int hist[4][256];  // counts of one digit each
  int newest;
  int ties;          // rows of the threshold key in this slice
  int holes, moved;  // of this slice
  int total[256];
  int digit, above, count;
  int warp_a[kWarps], warp_b[kWarps];
};

__device__ __forceinline__ int remote_int(const int* p, int rank) {
  uint32_t a;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Barrier over the unit's blocks (one: the block's own).
__device__ __forceinline__ void unit_sync(int cluster) {
  if (cluster == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
  }
}

// Sum over the warps before this one, and over all, of a per-warp count.
__device__ __forceinline__ int warps_before(int count, int* sums, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sums[warp] = count;
  __syncthreads();
  const int v = lane < kWarps ? sums[lane] : 0;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  *all = __shfl_sync(~0u, x, 31);
  return __shfl_sync(~0u, x - v, warp);
}

// kHeld: the slice's keys stay in shared memory.
template <bool kHeld>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t held[];  // keys, then positions, of the slice
  __shared__ Exchange x;
  const int n_blocks = p.cluster;
  const int unit = blockIdx.x / n_blocks, rank = blockIdx.x - unit * n_blocks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = p.c.capacity;
  const int W = min(p.budget, cap);
  int len = p.c.lens[unit];
  if (len < 0 || len > cap) {
    if (tid == 0) record_status(p.status, RI_ERR_INVALID_ARG);
    len = len < 0 ? 0 : cap;
  }
  const int keep = min(len, p.budget);
  // rows of this block, a multiple of 32 each but for the last
  const int slice = ((len + n_blocks - 1) / n_blocks + 31) & ~31;
  const int r0 = min(len, rank * slice), r1 = min(len, r0 + slice), rows = r1 - r0;
  const int32_t* pos = p.c.pos + (size_t)unit * cap;
  const float* weight = p.c.weight + (size_t)unit * cap;
  uint32_t* keys = held;
  uint32_t* poss = held + slice;
  const bool leaves = keep < len;

  int need_ties = 0;
  uint32_t key = 0;
  long long recent_from = 0;
  auto key_of = [&](int i) {  // row r0 + i
    return kHeld ? keys[i] : rank_key(weight[r0 + i], pos[r0 + i], p.first, recent_from);
  };
  if (leaves) {
    // ---- the newest position, over the unit
    int newest = INT_MIN;
    for (int i = tid; i < rows; i += kThreads) {
      const int q = pos[r0 + i];
      if (kHeld) {
        poss[i] = (uint32_t)q;
        keys[i] = __float_as_uint(weight[r0 + i]);
      }
      newest = max(newest, q);
    }
    for (int i = tid; i < 4 * 256; i += kThreads) (&x.hist[0][0])[i] = 0;
    if (tid == 0) x.newest = INT_MIN;
    __syncthreads();
    newest = __reduce_max_sync(~0u, newest);
    if (lane == 0) atomicMax(&x.newest, newest);
    unit_sync(n_blocks);
    newest = INT_MIN;
    for (int b = 0; b < n_blocks; ++b) newest = max(newest, remote_int(&x.newest, b));
    recent_from = (long long)newest - p.recent;

    // ---- the keep-th largest key, digit by digit from the top
    uint32_t mask = 0;
    int above = 0, count = 0;  // keys above the prefix; keys of it
#pragma unroll 1
    for (int d = 0; d < 4; ++d) {
      const int shift = 24 - 8 * d;
      for (int i = tid; i < rows; i += kThreads) {
        uint32_t k;
        if (kHeld && d == 0) {
          k = rank_key(__uint_as_float(keys[i]), (int)poss[i], p.first, recent_from);
          keys[i] = k;
        } else {
          k = key_of(i);
        }
        if ((k & mask) == key) atomicAdd(&x.hist[d][(k >> shift) & 255], 1);
      }
      unit_sync(n_blocks);
      if (tid < 256) {
        int sum = 0;
        for (int b = 0; b < n_blocks; ++b) sum += remote_int(&x.hist[d][tid], b);
        x.total[255 - tid] = sum;  // largest digit first
      }
      __syncthreads();
      if (warp == 0) {
        int v[8], mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += v[i] = x.total[8 * lane + i];
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(~0u, upto, o);
          if (lane >= o) upto += y;
        }
        int before = above + upto - mine;
        if (before < keep && keep <= before + mine) {  // one lane: the digit is among its 8
          int i = 0;
          while (before + v[i] < keep) before += v[i++];
          x.digit = 255 - (8 * lane + i);
          x.above = before;
          x.count = v[i];
        }
      }
      __syncthreads();
      key |= (uint32_t)x.digit << shift;
      mask |= 255u << shift;
      above = x.above;
      count = x.count;
    }
    need_ties = keep - above;  // rows of that key kept, in row order
    if (need_ties == count) need_ties = INT_MAX;  // all of them: no counting
  }

  // A warp takes 32 * steps rows in a row, so ranks come from ballots.
  const int steps = (rows + kThreads - 1) / kThreads;
  const int w0 = warp * 32 * steps;  // first row of the warp in the slice
  auto row_in = [&](int s) { return w0 + 32 * s + lane; };
  int tie_base = 0;
  if (leaves && need_ties != INT_MAX) {
    int n = 0;
    for (int s = 0; s < steps; ++s) {
      const int i = row_in(s);
      n += __popc(__ballot_sync(~0u, i < rows && key_of(i) == key));
    }
    int all;
    tie_base = warps_before(n, x.warp_a, &all);
    if (tid == 0) x.ties = all;
    unit_sync(n_blocks);
    for (int b = 0; b < rank; ++b) tie_base += remote_int(&x.ties, b);
  }
  // the row's token stays; `t` counts the ties met by the warp
  auto kept_row = [&](int i, int* t) {
    if (!leaves) return i < rows;
    const uint32_t k = i < rows ? key_of(i) : 0u;
    bool kept = i < rows && k > key;
    const bool tie = i < rows && k == key;
    const uint32_t ties = __ballot_sync(~0u, tie);
    if (tie) kept = tie_base + *t + __popc(ties & ((1u << lane) - 1)) < need_ties;
    *t += __popc(ties);
    return kept;
  };

  int n_moves = 0;
  int32_t* holes = p.holes + (size_t)unit * W;
  int32_t* moved = p.moved + (size_t)unit * W;
  if (leaves) {
    // ---- ranks of the holes below keep and of the kept rows from keep on
    int t = 0, nh = 0, nm = 0;
    for (int s = 0; s < steps; ++s) {
      const int i = row_in(s), r = r0 + i;
      const bool kept = kept_row(i, &t);
      nh += __popc(__ballot_sync(~0u, i < rows && r < keep && !kept));
      nm += __popc(__ballot_sync(~0u, r >= keep && kept));
    }
    int all_h, all_m;
    int h = warps_before(nh, x.warp_a, &all_h), m = warps_before(nm, x.warp_b, &all_m);
    if (tid == 0) {
      x.holes = all_h;
      x.moved = all_m;
    }
    unit_sync(n_blocks);
    for (int b = 0; b < n_blocks; ++b) {
      const int bh = remote_int(&x.holes, b), bm = remote_int(&x.moved, b);
      if (b < rank) {
        h += bh;
        m += bm;
      }
      n_moves += bh;
    }
    t = 0;
    for (int s = 0; s < steps; ++s) {
      const int i = row_in(s), r = r0 + i;
      const bool kept = kept_row(i, &t);
      const bool hole = i < rows && r < keep && !kept, move = r >= keep && kept;
      const uint32_t bh = __ballot_sync(~0u, hole), bm = __ballot_sync(~0u, move);
      const uint32_t lt = (1u << lane) - 1;
      if (hole) holes[h + __popc(bh & lt)] = r;
      if (move) moved[m + __popc(bm & lt)] = r;
      h += __popc(bh);
      m += __popc(bm);
    }
  }
  // the lists are complete, nothing reads the old state by rank from here on,
  // and no block's shared memory is read any more
  unit_sync(n_blocks);
  if (rank == 0 && tid == 0) p.o.lens[unit] = keep;

  const size_t src0 = (size_t)unit * cap, dst0 = (size_t)unit * p.o.capacity;
  const uint4* kv_src = reinterpret_cast<const uint4*>(lane < 16 ? p.c.K : p.c.V);
  uint4* kv_dst = reinterpret_cast<uint4*>(lane < 16 ? p.o.K : p.o.V);
  const int ch = lane & 15;
  // ---- kept rows below keep, where an array of the result is another one
  const bool kv_apart = kv_src != kv_dst, any_kv = __any_sync(~0u, kv_apart);
  const bool pos_apart = p.c.pos != p.o.pos, weight_apart = p.c.weight != p.o.weight;
  if (any_kv || pos_apart || weight_apart) {
    int t = 0;
    for (int s = 0; s < steps; ++s) {
      if (r0 + w0 + 32 * s >= keep) break;  // uniform over the warp
      const int i = row_in(s), r = r0 + i;
      const bool stays = kept_row(i, &t) && r < keep;
      if (stays && pos_apart) p.o.pos[dst0 + r] = pos[r];
      if (stays && weight_apart) p.o.weight[dst0 + r] = weight[r];
      uint32_t left = any_kv ? __ballot_sync(~0u, stays) : 0u;
      while (left) {
        uint4 v[4];
        int row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          row[j] = -1;
          if (left) {
            row[j] = r0 + w0 + 32 * s + __ffs(left) - 1;
            left &= left - 1;
          }
          if (row[j] >= 0 && kv_apart) v[j] = kv_src[(src0 + row[j]) * 16 + ch];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (row[j] >= 0 && kv_apart) kv_dst[(dst0 + row[j]) * 16 + ch] = v[j];
      }
    }
  }
  // (keys read from memory again must not meet a moved token's)
  if (!kHeld) unit_sync(n_blocks);
  // ---- moved[k] -> holes[k], four rows in flight per warp.  Sources lie at
  // or behind keep, destinations before it: no move reads what another writes.
  const int warps = n_blocks * kWarps;
  for (int k0 = rank * kWarps + warp; k0 < n_moves; k0 += 4 * warps) {
    int from = 0, to = 0;
    if (lane < 4 && k0 + lane * warps < n_moves) {
      from = moved[k0 + lane * warps];
      to = holes[k0 + lane * warps];
      p.o.pos[dst0 + to] = pos[from];
      p.o.weight[dst0 + to] = weight[from];
    }
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int f = __shfl_sync(~0u, from, j);
      if (k0 + j * warps < n_moves) v[j] = kv_src[(src0 + f) * 16 + ch];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = __shfl_sync(~0u, to, j);
      if (k0 + j * warps < n_moves) kv_dst[(dst0 + d) * 16 + ch] = v[j];
    }
  }
}

}  // namespace

size_t token_evict_bytes(const ri_token_cache& c, int budget) {
  const size_t units = (size_t)c.batch * c.num_kv_heads;
  const size_t W = budget < c.capacity ? budget : c.capacity;
  return align_up(kStatusBytesHost + 2 * units * W * sizeof(int32_t), 256);
}

cudaError_t launch_token_evict(const TokenEvictArgs& a, cudaStream_t s) {
  EvictParams p;
  p.c = a.c;
  p.o = a.out;
  p.budget = a.budget;
  p.first = a.keep_first;
  p.recent = a.keep_recent;
  p.status = reinterpret_cast<int*>(a.ws);
  const int units = a.c.batch * a.c.num_kv_heads;
  const int cap = a.c.capacity, W = a.budget < cap ? a.budget : cap;
  p.holes = reinterpret_cast<int32_t*>(a.ws + kStatusBytesHost);
  p.moved = p.holes + (size_t)units * W;
  // Blocks per unit: more while a block has over 4 rows per thread and the
  // grid is within two blocks per SM.
  int cluster = 1;
  while (cluster < kMaxCluster && cap > cluster * 4 * kThreads &&
         (long long)units * cluster * 2 <= 2 * num_sms())
    cluster *= 2;
  while (cluster < kMaxCluster && cap > (long long)cluster * (kMaxHeld - 32)) cluster *= 2;
  p.cluster = cluster;
  const int slice = ((cap + cluster - 1) / cluster + 31) & ~31;
  const bool held = slice <= kMaxHeld;
  void (*kernel)(EvictParams) = held ? evict_kernel<true> : evict_kernel<false>;
  cudaError_t e = set_smem_once(6, reinterpret_cast<const void*>(evict_kernel<true>), kMaxHeld * 8);
  if (e == cudaSuccess)
    e = allow_large_clusters(6, reinterpret_cast<const void*>(evict_kernel<true>));
  if (e == cudaSuccess)
    e = allow_large_clusters(7, reinterpret_cast<const void*>(evict_kernel<false>));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = held ? (size_t)slice * 8 : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace ri
