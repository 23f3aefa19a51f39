// Eviction from the exact token cache (ri_token_evict): every (sequence, KV
// head) keeps its `keep` tokens of highest rank, and the kept tokens behind
// row `keep` move into the rows of the dropped ones.
//
// The order is total: held tokens (first and most recent positions) before
// all others, by row among themselves; then larger weight, then lower row.  A
// token's rank is a 32-bit key (the order-preserving image of its weight, all
// ones when held).  The keep-th token is found by counting: the keys' range is
// cut into 1024 equal buckets, the bucket that holds the keep-th key is cut again while it has
// more than 256 keys (one cut is usual: a float's bits spread the weights over
// the range by their logarithm), and its keys are then ranked one against the
// other.  Every step is a count, a prefix sum or a comparison: the result does
// not depend on the order in which threads run.
//
// One thread-block cluster per (sequence, KV head).  A block holds a
// contiguous slice of the rows' keys in shared memory (read once); blocks
// exchange counts and candidates through distributed shared memory.  The same
// launch moves the rows, or a second one where the clusters leave much of the
// machine idle.
//
// Bound: reading 8 bytes per token, and 1 KB of traffic per token that changes
// its row.  Measured: 128 heads of 8K tokens halved 65 us, of which the moves'
// 262 MB take about 45 (5.8 TB/s) and the selection, latency after latency, 20;
// 8 heads of 128K reduced to 8K 45 us (29 of them the selection on 64 SMs); one
// token out of each of 128 heads 11.5 us.
#include "common.cuh"
#include "internal.h"

namespace ri {

namespace {

constexpr int kThreads = 1024;
constexpr int kBucketBits = 10;  // 1 << kBucketBits == kThreads
constexpr int kWarps = kThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kRowsInFlight = 8;
constexpr int kRowsPerThread = 2;
// Rows per unit from which a launch of its own for the moves pays: 8 heads of
// 128K rows to 1024, 2048, 4096, 8192 in one launch 31, 33, 38, 45 us, in two 33,
// 35, 37, 41.
constexpr int kApartRows = 2048;
constexpr int kMaxCluster = 16;
// rows whose keys and positions a block holds (8 bytes each); a longer slice
// (caches of more than 16 x this) is read again from global memory instead
constexpr int kMaxHeld = 23552;

struct EvictParams {
  ri_token_cache c, o;
  int budget, first, recent;
  int cluster;     // blocks per unit
  int32_t* holes;  // [units][W]: rows below keep whose tokens are dropped, in order
  int32_t* moved;  // [units][W]: rows from keep on whose tokens stay, in order
  int32_t* listed; // [units]: rows to move; -n: rows 0 .. n - 1, each to its own number
  bool apart;      // a second launch moves the rows
  int* status;
};

// Largest key for held tokens; a NaN weight ranks as -inf, -0 as +0.
__device__ __forceinline__ uint32_t rank_key(float w, int pos, int first, long long recent_from) {
  if (pos < first || pos > recent_from) return 0xFFFFFFFFu;
  if (w != w) w = -__int_as_float(0x7f800000);
  return float_order_key(w + 0.f);
}

constexpr int kBuckets = kThreads;  // one thread sums one bucket
constexpr int kPasses = 4;          // kBucketBits each, of 32
static_assert(kBuckets == 1 << kBucketBits, "");
constexpr int kRanked = 256;        // most candidates ranked directly, by four threads each
static_assert(kThreads == 4 * kRanked, "");

// Shared memory every block of a cluster may read.
struct Exchange {
  int hist[kPasses][kBuckets];
  unsigned long long mine[kRanked], all[kRanked];  // candidates: key, then ~row
  int n_mine;
  int newest;
  uint32_t low, high;  // raw keys of the slice
  int held;
  int ties, cut;       // mass ties of the slice; the last kept row among them
  int holes, moved;    // of this slice
  int bucket, above, count;
  uint32_t cut_key;
  int warp_a[kWarps], warp_b[kWarps];
};

__device__ __forceinline__ int remote_int(const int* p, int rank) {
  uint32_t a;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ unsigned long long remote_u64(const unsigned long long* p, int rank) {
  uint32_t a;
  unsigned long long v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// Lane b's copy of a word of block b of the unit's n (0 from lane n on), so
// that all blocks' words arrive in one round trip.
__device__ __forceinline__ int gather_int(const int* p, int n) {
  const int lane = threadIdx.x & 31;
  if (n == 1) return lane == 0 ? *p : 0;  // the block's own
  return lane < n ? remote_int(p, lane) : 0;
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

// Row moved[k] -> row holes[k] of a unit, for the rows of one warp of `warps`:
// up to 32 in a row, their numbers in one load, their K and V kRowsInFlight
// rows in flight.  Sources of moves lie at or behind keep, destinations before it: no
// move reads what another writes.
__device__ __forceinline__ void move_rows(const EvictParams& p, int unit, int n_rows, int warp,
                                          int warps) {
  const int lane = threadIdx.x & 31, ch = lane & 15;
  const int cap = p.c.capacity, W = min(p.budget, cap);
  const bool list = n_rows >= 0;
  if (!list) n_rows = -n_rows;
  const int32_t* holes = p.holes + (size_t)unit * W;
  const int32_t* moved = p.moved + (size_t)unit * W;
  const size_t src0 = (size_t)unit * cap, dst0 = (size_t)unit * p.o.capacity;
  const int32_t* pos = p.c.pos + src0;
  const float* weight = p.c.weight + src0;
  const bool pos_apart = p.c.pos != p.o.pos, weight_apart = p.c.weight != p.o.weight;
  const uint4* kv_src = reinterpret_cast<const uint4*>(lane < 16 ? p.c.K : p.c.V);
  uint4* kv_dst = reinterpret_cast<uint4*>(lane < 16 ? p.o.K : p.o.V);
  const int run = min(32, (n_rows + warps - 1) / warps);
  int k0 = warp * run;
  auto numbers = [&](int k, int* from, int* to) {  // of row k + lane of the list
    *from = *to = k + lane;
    if (list && lane < min(run, n_rows - k)) {
      *from = moved[k + lane];
      *to = holes[k + lane];
    }
  };
  int from, to;
  numbers(k0, &from, &to);
  while (k0 < n_rows) {
    const int n = min(run, n_rows - k0), next = k0 + warps * run;
    int next_from, next_to;
    numbers(next, &next_from, &next_to);  // on their way meanwhile
    if (lane < n) {
      if (from != to || pos_apart) p.o.pos[dst0 + to] = pos[from];
      if (from != to || weight_apart) p.o.weight[dst0 + to] = weight[from];
    }
    for (int j0 = 0; j0 < n; j0 += kRowsInFlight) {
      uint4 v[kRowsInFlight];
#pragma unroll
      for (int j = 0; j < kRowsInFlight; ++j) {
        const int f = __shfl_sync(~0u, from, (j0 + j) & 31);
        if (j0 + j < n) v[j] = __ldcs(kv_src + (src0 + f) * 16 + ch);
      }
#pragma unroll
      for (int j = 0; j < kRowsInFlight; ++j) {
        const int d = __shfl_sync(~0u, to, (j0 + j) & 31);
        if (j0 + j < n) __stcs(kv_dst + (dst0 + d) * 16 + ch, v[j]);
      }
    }
    from = next_from;
    to = next_to;
    k0 = next;
  }
}

// kHeld: the slice's keys stay in shared memory.
template <bool kHeld>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  // kHeld: the slice's keys, its positions; then one bit per row
  extern __shared__ uint32_t held[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  uint32_t* bits = kHeld ? poss + slice : held;
  const bool leaves = keep < len;

  // a row's token stays: its key is above cut_key, or equal and not behind cut_row
  uint32_t cut_key = 0;
  int cut_row = INT_MAX;
  long long recent_from = 0;
  auto key_of = [&](int i) {  // row r0 + i
    return kHeld ? keys[i] : rank_key(weight[r0 + i], pos[r0 + i], p.first, recent_from);
  };
  // A warp takes 32 * steps rows in a row, so ranks come from ballots.
  const int steps = (rows + kThreads - 1) / kThreads;
  const int w0 = warp * 32 * steps;  // first row of the warp in the slice
  auto row_in = [&](int s) { return w0 + 32 * s + lane; };
  if (leaves) {
    // ---- the newest position and the keys' range, over the unit
    for (int i = tid; i < kPasses * kBuckets; i += kThreads) (&x.hist[0][0])[i] = 0;
    if (tid == 0) {
      x.newest = INT_MIN;
      x.low = 0xFFFFFFFFu;
      x.high = 0;
      x.n_mine = x.held = 0;
      x.cut = -1;
    }
    int newest = INT_MIN;
    uint32_t low = 0xFFFFFFFFu, high = 0;
#pragma unroll 8
    for (int i = tid; i < rows; i += kThreads) {
      const int q = pos[r0 + i];
      const uint32_t k = rank_key(weight[r0 + i], 0, 0, 0);  // as if not held
      if (kHeld) {
        poss[i] = (uint32_t)q;
        keys[i] = k;
      }
      newest = max(newest, q);
      low = min(low, k);
      high = max(high, k);
    }
    newest = __reduce_max_sync(~0u, newest);
    low = __reduce_min_sync(~0u, low);
    high = __reduce_max_sync(~0u, high);
    __syncthreads();
    if (lane == 0) {
      atomicMax(&x.newest, newest);
      atomicMin(&x.low, low);
      atomicMax(&x.high, high);
    }
    unit_sync(n_blocks);
    {
      const int a = gather_int(&x.newest, n_blocks);
      const uint32_t b = (uint32_t)gather_int(reinterpret_cast<int*>(&x.low), n_blocks);
      const uint32_t c = (uint32_t)gather_int(reinterpret_cast<int*>(&x.high), n_blocks);
      newest = __reduce_max_sync(~0u, lane < n_blocks ? a : INT_MIN);
      low = __reduce_min_sync(~0u, lane < n_blocks ? b : 0xFFFFFFFFu);
      high = __reduce_max_sync(~0u, lane < n_blocks ? c : 0u);
    }
    recent_from = (long long)newest - p.recent;

    // ---- the bucket of the keep-th key, narrowed down
    const uint32_t span = high - low;
    int shift = span < kBuckets ? 0 : 32 - __clz(span) - kBucketBits;  // span >> shift < kBuckets
    uint32_t range = span;  // keys of interest: low .. low + range
    int above = 0, count = 0;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      int held_mine = 0;
      for (int i = tid; i < rows; i += kThreads) {
        uint32_t k;
        if (kHeld && pass == 0) {
          const int q = (int)poss[i];
          k = q < p.first || q > recent_from ? 0xFFFFFFFFu : keys[i];
          keys[i] = k;
        } else {
          k = key_of(i);
        }
        if (k == 0xFFFFFFFFu) ++held_mine;
        else if (k >= low && k - low <= range) atomicAdd(&x.hist[pass][(k - low) >> shift], 1);
      }
      if (pass == 0) {
        held_mine = __reduce_add_sync(~0u, held_mine);
        if (lane == 0 && held_mine) atomicAdd(&x.held, held_mine);
      }
      unit_sync(n_blocks);
      if (pass == 0) above = __reduce_add_sync(~0u, gather_int(&x.held, n_blocks));
      if (above >= keep) {  // the held ones alone are enough
        count = INT_MAX;
        low = 0xFFFFFFFFu;
        above = 0;
        break;
      }
      // thread t sums bucket kBuckets - 1 - t, so that a prefix sum runs from the top
      int sum = 0;
      if (n_blocks == 1) {
        sum = x.hist[pass][kBuckets - 1 - tid];
      } else {
        int v[kMaxCluster];
#pragma unroll
        for (int b = 0; b < kMaxCluster; ++b)
          v[b] = b < n_blocks ? remote_int(&x.hist[pass][kBuckets - 1 - tid], b) : 0;
#pragma unroll
        for (int b = 0; b < kMaxCluster; ++b) sum += v[b];
      }
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += y;
      }
      int all;
      const int warp_total = __shfl_sync(~0u, upto, 31);
      const int before = above + warps_before(warp_total, x.warp_a, &all) + upto - sum;
      if (before < keep && keep <= before + sum) {  // one thread of the block
        x.bucket = kBuckets - 1 - tid;
        x.above = before;
        x.count = sum;
      }
      __syncthreads();
      low += (uint32_t)x.bucket << shift;
      above = x.above;
      count = x.count;
      range = (1u << shift) - 1;  // of this bucket
      if (count <= kRanked || shift == 0) break;
      shift = shift > kBucketBits ? shift - kBucketBits : 0;
    }
    const int need = keep - above;  // of the bucket's keys, in order

    if (count <= kRanked) {
      // ---- the bucket's keys are ranked one against the other
      for (int i = tid; i < rows; i += kThreads) {
        const uint32_t k = key_of(i);
        if (k != 0xFFFFFFFFu && k >= low && k - low <= range)
          x.mine[atomicAdd(&x.n_mine, 1)] = (unsigned long long)k << 32 | (uint32_t)~(r0 + i);
      }
      unit_sync(n_blocks);
      const unsigned long long* all = x.mine;
      if (n_blocks > 1) {
        int n = gather_int(&x.n_mine, n_blocks), first = 0;  // lane b: block b's
        for (int b = 0; b < n_blocks; ++b) {
          const int nb = __shfl_sync(~0u, n, b);
          for (int i = tid; i < nb; i += kThreads) x.all[first + i] = remote_u64(&x.mine[i], b);
          first += nb;
        }
        __syncthreads();
        all = x.all;
      }
      {
        const unsigned long long me = (tid >> 2) < count ? all[tid >> 2] : 0ull;
        int larger = 0;
#pragma unroll 4
        for (int j = tid & 3; j < count; j += 4) larger += all[j] > me;
        larger += __shfl_xor_sync(~0u, larger, 1);
        larger += __shfl_xor_sync(~0u, larger, 2);
        if ((tid >> 2) < count && (tid & 3) == 0 && larger == need - 1) {
          x.cut_key = (uint32_t)(me >> 32);
          x.above = (int)~(uint32_t)me;  // its row
        }
      }
      __syncthreads();
      cut_key = x.cut_key;
      cut_row = x.above;
    } else {
      // ---- many rows of one key: the need-th of them, in row order
      cut_key = low;
      int n = 0;
      for (int s = 0; s < steps; ++s) {
        const int i = row_in(s);
        n += __popc(__ballot_sync(~0u, i < rows && key_of(i) == cut_key));
      }
      int all;
      int t = warps_before(n, x.warp_b, &all);
      if (tid == 0) x.ties = all;
      unit_sync(n_blocks);
      const int before = gather_int(&x.ties, n_blocks);
      t += __reduce_add_sync(~0u, lane < rank ? before : 0);
      for (int s = 0; s < steps; ++s) {
        const int i = row_in(s);
        const uint32_t m = __ballot_sync(~0u, i < rows && key_of(i) == cut_key);
        if ((m >> lane & 1) && t + __popc(m & ((1u << lane) - 1)) == need - 1) x.cut = r0 + i;
        t += __popc(m);
      }
      unit_sync(n_blocks);
      const int c = gather_int(&x.cut, n_blocks);
      cut_row = __reduce_max_sync(~0u, lane < n_blocks ? c : -1);
    }
  }
  auto kept_key = [&](int i) {
    const uint32_t k = key_of(i);
    return k > cut_key || (k == cut_key && r0 + i <= cut_row);
  };

  // K or V of the result in another array: rows that stay are copied as well,
  // listed behind the moves (a row's rank among them: the rows below it that
  // are no holes)
  const bool kv_apart = p.c.K != p.o.K || p.c.V != p.o.V;
  int n_moves = 0;
  int32_t* holes = p.holes + (size_t)unit * W;
  int32_t* moved = p.moved + (size_t)unit * W;
  if (leaves) {
    // ---- one bit per row: its token stays; holes below keep and kept rows
    // from keep on are counted per warp, then ranked
    auto masks = [&](int i0, uint32_t kept, uint32_t* hole, uint32_t* move) {
      const int low = min(max(keep - (r0 + i0), 0), 32);  // the word's rows below keep
      const uint32_t below = low == 32 ? ~0u : (1u << low) - 1;
      *hole = below & ~kept;  // (keep <= len: rows below keep are all live)
      *move = ~below & kept;
    };
    uint32_t hole, move;
    int nh = 0, nm = 0;
    for (int s = 0; s < steps; ++s) {
      const int i = row_in(s), i0 = w0 + 32 * s;
      if (i0 >= rows) break;  // uniform over the warp
      const uint32_t kept = __ballot_sync(~0u, i < rows && kept_key(i));
      if (lane == 0) bits[i0 >> 5] = kept;
      masks(i0, kept, &hole, &move);
      nh += __popc(hole);
      nm += __popc(move);
    }
    int all_h, all_m;
    int h = warps_before(nh, x.warp_a, &all_h), m = warps_before(nm, x.warp_b, &all_m);
    if (tid == 0) {
      x.holes = all_h;
      x.moved = all_m;
    }
    unit_sync(n_blocks);
    const int bh = gather_int(&x.holes, n_blocks), bm = gather_int(&x.moved, n_blocks);
    n_moves = __reduce_add_sync(~0u, bh);
    h += __reduce_add_sync(~0u, lane < rank ? bh : 0);
    m += __reduce_add_sync(~0u, lane < rank ? bm : 0);
    const uint32_t lt = (1u << lane) - 1;
    for (int s = 0; s < steps; ++s) {
      const int i0 = w0 + 32 * s, r = r0 + i0 + lane;
      if (i0 >= rows) break;
      masks(i0, bits[i0 >> 5], &hole, &move);
      const int hb = h + __popc(hole & lt);
      if (hole >> lane & 1) holes[hb] = r;
      else if (move >> lane & 1) moved[m + __popc(move & lt)] = r;
      else if (kv_apart && r < keep) holes[n_moves + r - hb] = moved[n_moves + r - hb] = r;
      h += __popc(hole);
      m += __popc(move);
    }
    __syncthreads();  // bits of other warps are read below
  }
  // the lists are complete, nothing ranks by the old state from here on, and
  // no block's shared memory is read any more
  unit_sync(n_blocks);
  if (rank == 0 && tid == 0) p.o.lens[unit] = keep;

  const size_t dst0 = (size_t)unit * p.o.capacity;
  const bool pos_apart = p.c.pos != p.o.pos, weight_apart = p.c.weight != p.o.weight;
  // ---- positions and weights of rows that stay, where only these are apart
  if (!kv_apart && (pos_apart || weight_apart)) {
    const int end = min(rows, keep - r0);
#pragma unroll 4
    for (int i = tid; i < end; i += kThreads) {
      const int q = pos[r0 + i];
      const float f = weight[r0 + i];
      if (!leaves || (bits[i >> 5] >> (i & 31) & 1)) {
        p.o.pos[dst0 + r0 + i] = q;
        p.o.weight[dst0 + r0 + i] = f;
      }
    }
  }
  // (nothing leaves: the rows are their own list)
  const int n_rows = kv_apart ? (leaves ? keep : -keep) : n_moves;
  if (p.apart) {
    if (rank == 0 && tid == 0) p.listed[unit] = n_rows;
  } else {
    move_rows(p, unit, n_rows, rank * kWarps + warp, n_blocks * kWarps);
  }
}

// (One block per SM as the compiler's bound: it then keeps all loads of a batch
// in flight, 107 registers; with 76 the 128K prompt took 49 us instead of 45.)
__global__ void __launch_bounds__(kMoveThreads, 1)
    move_kernel(const __grid_constant__ EvictParams p, int parts) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = blockIdx.x / parts, part = blockIdx.x - unit * parts;
  constexpr int kPerBlock = kMoveThreads / 32;
  move_rows(p, unit, p.listed[unit], part * kPerBlock + (threadIdx.x >> 5), parts * kPerBlock);
}

}  // namespace

size_t token_evict_bytes(const ri_token_cache& c, int budget) {
  const size_t units = (size_t)c.batch * c.num_kv_heads;
  const size_t W = budget < c.capacity ? budget : c.capacity;
  return align_up(kStatusBytesHost + (2 * units * W + units) * sizeof(int32_t), 256);
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
  p.listed = p.moved + (size_t)units * W;
  // Blocks per unit: more while a block has over kRowsPerThread rows per thread
  // and the grid is within a block per SM.
  // Of 8 at most, unless the slices get too long for shared memory: clusters of
  // 16 took longer, 128K rows of 1, 4, 8 heads 41, 43, 86 us against 33, 37, 41.
  int cluster = 1;
  while (cluster < 8 && cap > cluster * kRowsPerThread * kThreads &&
         (long long)units * cluster * 2 <= num_sms())
    cluster *= 2;
  while (cluster < kMaxCluster && cap > (long long)cluster * (kMaxHeld - 32)) cluster *= 2;
  p.cluster = cluster;
  const int slice = ((cap + cluster - 1) / cluster + 31) & ~31;
  const bool held = slice <= kMaxHeld;
  void (*kernel)(EvictParams) = held ? evict_kernel<true> : evict_kernel<false>;
  cudaError_t e = set_smem_once(6, reinterpret_cast<const void*>(evict_kernel<true>),
                                kMaxHeld * 8 + kMaxHeld / 8);
  if (e == cudaSuccess)
    e = set_smem_once(7, reinterpret_cast<const void*>(evict_kernel<false>),
                      kEvictMaxCapacity / kMaxCluster / 8 + 4);
  if (e == cudaSuccess)
    e = allow_large_clusters(6, reinterpret_cast<const void*>(evict_kernel<true>));
  if (e == cudaSuccess)
    e = allow_large_clusters(7, reinterpret_cast<const void*>(evict_kernel<false>));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (held ? (size_t)slice * 8 : 0) + slice / 8;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Where the clusters leave much of the machine idle (8 heads of a 128K
  // prompt: 64 blocks), a second launch over all of it moves the rows.  8K rows
  // halved, one launch and two: 96 blocks (96 heads) 64 and 57 us, 128 blocks (32,
  // 64, 128 heads) 28 and 31, 47 and 45, 72 and 68.
  p.apart = units * cluster * 4 < 3 * num_sms() && W > kApartRows;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess || !p.apart) return e;
  const int parts = (4 * num_sms() + units - 1) / units;
  cudaLaunchConfig_t mc = {};
  mc.gridDim = dim3((unsigned)(units * parts));
  mc.blockDim = dim3(kMoveThreads);
  mc.stream = s;
  cudaLaunchAttribute after[1];
  after[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  after[0].val.programmaticStreamSerializationAllowed = 1;
  mc.attrs = after;
  mc.numAttrs = 1;
  return cudaLaunchKernelEx(&mc, move_kernel, p, parts);
}

}  // namespace ri
