// Eviction from the exact token cache (ri_token_evict): every (sequence, KV
// head) keeps its `keep` tokens of highest rank, and the kept tokens behind
// row `keep` move into the rows of the dropped ones.
//
// The order is total: held tokens (first and most recent positions) before
// all others, then larger weight, then lower row.  A token's rank is a 32-bit
// key (the order-preserving image of its weight, all ones when held), so the
// keep-th largest key is found digit by digit (radix selection), and ties on
// it are settled by counting in row order.  Every step is a count or a scan:
// the result does not depend on the order in which threads run.
#include "common.cuh"
#include "internal.h"

namespace ri {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

struct EvictParams {
  ri_token_cache c, o;
  int budget, first, recent;
  int32_t* place;  // [units][min(budget, capacity)]: source row of each kept row
  int32_t* holes;  // the same size: rows below keep whose tokens are dropped
  int* status;
};

// Largest key for held tokens; a NaN weight ranks as -inf, -0 as +0.
__device__ __forceinline__ uint32_t rank_key(float w, int pos, int first, long long recent_from) {
  if (pos < first || pos > recent_from) return 0xFFFFFFFFu;
  if (w != w) w = -__int_as_float(0x7f800000);
  return float_order_key(w + 0.f);
}

// Exclusive sum over the block of one small count per thread; *total gets the
// block's sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kWarps; ++i) {
    const int s = warp_sums[i];
    if (i < warp) before += s;
    all += s;
  }
  *total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictParams p) {
  __shared__ int warp_sums[kWarps];
  __shared__ int hist[256];
  __shared__ int sh_newest, sh_digit, sh_above;
  const int unit = blockIdx.x, tid = threadIdx.x;
  const int cap = p.c.capacity;
  const int W = min(p.budget, cap);
  int len = p.c.lens[unit];
  if (len < 0 || len > cap) {
    if (tid == 0) record_status(p.status, RI_ERR_INVALID_ARG);
    len = len < 0 ? 0 : cap;
  }
  const int keep = min(len, p.budget);
  const int32_t* pos = p.c.pos + (size_t)unit * cap;
  const float* weight = p.c.weight + (size_t)unit * cap;
  int32_t* place = p.place + (size_t)unit * W;
  int32_t* holes = p.holes + (size_t)unit * W;
  if (keep == len) {  // nothing leaves
    for (int i = tid; i < keep; i += kThreads) place[i] = i;
    __syncthreads();
    if (tid == 0) p.o.lens[unit] = keep;
    return;
  }
  if (tid == 0) sh_newest = INT_MIN;
  __syncthreads();
  int newest = INT_MIN;
  for (int i = tid; i < len; i += kThreads) newest = max(newest, pos[i]);
  atomicMax(&sh_newest, newest);
  __syncthreads();
  const long long recent_from = (long long)sh_newest - p.recent;

  // the keep-th largest key: its digits from the top, `above` keys larger
  uint32_t key = 0, mask = 0;
  int above = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < len; i += kThreads) {
      const uint32_t k = rank_key(weight[i], pos[i], p.first, recent_from);
      if ((k & mask) == key) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int sum = above, d = 255;
      while (sum + hist[d] < keep) sum += hist[d--];
      sh_digit = d;
      sh_above = sum;
    }
    __syncthreads();
    key |= (uint32_t)sh_digit << shift;
    mask |= 255u << shift;
    above = sh_above;
    __syncthreads();
  }
  const int ties = keep - above;  // tokens of that key kept, in row order

  int n_tie = 0, n_hole = 0, n_src = 0;
  for (int base = 0; base < len; base += kThreads) {
    const int i = base + tid;
    const uint32_t k =
        i < len ? rank_key(weight[i], pos[i], p.first, recent_from) : 0;
    const bool tie = i < len && k == key;
    int total;
    const int t = n_tie + block_scan(tie, warp_sums, &total);
    n_tie += total;
    const bool kept = i < len && (k > key || (tie && t < ties));
    const bool hole = i < keep && !kept, src = i >= keep && kept;
    const int hr = n_hole + block_scan(hole, warp_sums, &total);
    n_hole += total;
    if (i < keep && kept) place[i] = i;
    if (hole) holes[hr] = i;
    const int sr = n_src + block_scan(src, warp_sums, &total);  // its barriers order holes[]
    n_src += total;
    // sources lie behind every hole: all holes up to rank sr are listed
    if (src) place[holes[sr]] = i;
  }
  if (tid == 0) p.o.lens[unit] = keep;
}

// One warp per kept row and turn: moves the row's K, V, position and weight
// where its source is another row or the destination another array.
__global__ void __launch_bounds__(256) evict_move_kernel(EvictParams p, int chunks) {
  const int unit = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int lane = threadIdx.x & 31;
  const int cap = p.c.capacity, ocap = p.o.capacity;
  const int W = min(p.budget, cap);
  const int keep = p.o.lens[unit];
  const int32_t* place = p.place + (size_t)unit * W;
  const bool kv_same = p.c.K == p.o.K, v_same = p.c.V == p.o.V;
  for (int j = chunk * 8 + (threadIdx.x >> 5); j < keep; j += chunks * 8) {
    const int i = place[j];
    const size_t src = (size_t)unit * cap + i, dst = (size_t)unit * ocap + j;
    const bool moved = i != j;
    const uint4* s = reinterpret_cast<const uint4*>(lane < 16 ? p.c.K : p.c.V) + src * 16;
    uint4* d = reinterpret_cast<uint4*>(lane < 16 ? p.o.K : p.o.V) + dst * 16;
    if (moved || !(lane < 16 ? kv_same : v_same)) d[lane & 15] = s[lane & 15];
    if (lane == 0 && (moved || p.c.pos != p.o.pos)) p.o.pos[dst] = p.c.pos[src];
    if (lane == 16 && (moved || p.c.weight != p.o.weight)) p.o.weight[dst] = p.c.weight[src];
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
  const int W = a.budget < a.c.capacity ? a.budget : a.c.capacity;
  p.place = reinterpret_cast<int32_t*>(a.ws + kStatusBytesHost);
  p.holes = p.place + (size_t)units * W;
  evict_select_kernel<<<units, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  int chunks = (W + 63) / 64;
  if ((long long)chunks * units > 4096) chunks = 4096 / units > 0 ? 4096 / units : 1;
  evict_move_kernel<<<units * chunks, 256, 0, s>>>(p, chunks);
  return cudaGetLastError();
}

}  // namespace ri
