// Attention of one token per sequence over a shared prefix and the sequence's
// own cached tokens (ri_token_attend): three launches.
//
//  prefix_kernel  all query rows of a KV head against the head's prefix, on
//                 the 5th-generation tensor cores (the batch's rows make one
//                 tall matrix, so the prefix is read once for all of them);
//  own_kernel     each (sequence, KV head)'s G rows against its own tokens,
//                 on warp-level tensor-core tiles (8 rows do not fill a tall
//                 tile); keeps the scores when weights are to be added;
//  merge_kernel   joins the shares by log-sum-exp, writes out and lse, and
//                 adds the own tokens' probabilities to their weights.
//
// A NaN or +inf among a row's scores makes its sums NaN, and so the row: out,
// lse and the weights that it adds to.
//
// Every share is (reference m, sums l and r, numerator) in units of log2, with
// s = q.k log2(e) / sqrt(d), p_i = 2^(s_i - m) and p'_i = p_i rounded to bf16:
//   l = sum_i p_i,  r = sum_i p'_i,  num = sum_i p'_i v_i;
// the merge takes M = max m, l = sum 2^(m - M) l, r and num likewise, and gives
// out = num / r, lse = M + log2 l.  Scores, sums and numerators are fp32; only
// the probabilities enter the value product as bf16 (the tensor cores take two
// bf16 operands; an own token's as a sum of two).  Dividing by the sum of the
// rounded ones takes out what they are off by in common: a token that holds
// nearly all weight gives its value.
// (Summed for every tile, r cost the prefix kernel 7 %; where no key counts
// for an eighth of its row, the unrounded sum goes into r instead.)  What is left
// of the prefix's roundings is as much as the output's own: behind a long prefix
// the output is off from 64 bits by 0.0023 of its norm, of which its rounding
// to bf16 alone makes 0.0017.  Own tokens alone are off by the latter.
//
// What bounds it: up to about 100 query rows per KV head the prefix's bytes,
// beyond that the tensor cores beside the special function unit (a tile's two
// products take 1024 cycles of the one, its exponentials 1024 of the other),
// under the power limit.  Measured: 64 sequences of 4 query heads behind 128K
// tokens of 8 heads 200-216 us in all (157 us for the prefix alone at 1965 MHz:
// 0.9 PFLOP/s; tensor pipe active 50 %, special functions 47 %), 16 behind 32K
// 59-61 us (4.1 TB/s over all three launches; the merge and its start take 10).
// Not kept: part of the exponentials as polynomials on the FMA pipe (184-204
// against 177 us for the prefix of the largest case: more instructions, more
// power), an issuing warp per slot (187), one own-token warp with a deeper
// ring in place of two.
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace ri {

namespace {

constexpr float kScaleLog2 = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kD = kHeadDim;
constexpr float kLazy = 8.f;  // log2: the reference moves when the maximum passes it by this
// The least reference: of a row that has met scores of -inf only, whose
// probabilities are then 2^-inf = 0 (and not 2^(-inf + inf), NaN).
constexpr float kLowest = -3.402823466e38f;
constexpr int kTile = 128;                  // query rows, keys of a tile
constexpr int kTileBytes = kTile * kD * 2;  // 32 KB of bf16
constexpr int kHalfTile = kTileBytes / 2;   // 64 of the 128 columns, 128-byte rows

// ---------------------------------------------------------------- work split
// The prefix is cut into tiles of 128 keys, the query rows of a KV head
// (b, g in order) into tiles of 128.  A unit is a KV head and two row tiles
// that share each key tile from shared memory (the last unit of an odd count
// has one); its work is 2 (or 1) per key tile.  Block c takes the work from
// chunk * c to chunk * (c + 1) of all units in a row, so every block carries
// the same share to within a tile, whatever the lengths.  Block c's share of
// unit u lies in slots 2 (c + u) and 2 (c + u) + 1, which no other (c, u)
// has, as u grows with c.
struct PrefixPlan {
  int rows;            // B * G, rows per KV head
  int tiles;           // row tiles per KV head
  int per_head;        // units per KV head
  int units;           // over all KV heads
  int key_tiles;
  int blocks, chunk;   // chunk: work of a block
  int head_work, total;  // work per KV head, in all
  __host__ __device__ int work_per_tile(int u) const {
    return (u % per_head) * 2 + 1 < tiles ? 2 : 1;
  }
  __host__ __device__ int start(int u) const {
    return (u / per_head) * head_work + (u % per_head) * 2 * key_tiles;
  }
  __host__ __device__ int tile_at(int u, int x) const {  // first key tile at or past work x
    const int s = x - start(u);
    if (s <= 0) return 0;
    const int w = work_per_tile(u);
    const int t = (s >> (w - 1)) + (s & (w - 1));
    return t < key_tiles ? t : key_tiles;
  }
  __host__ __device__ int from(int c) const { return c < blocks ? c * chunk : total; }
  __host__ __device__ int unit_of(int x) const {  // the unit holding work x
    const int h = x / head_work;
    const int i = (x - h * head_work) / (2 * key_tiles);
    return h * per_head + (i < per_head ? i : per_head - 1);
  }
};

// False when the work of all units does not fit 31 bits.
bool plan_prefix(const ri_token_cache& c, int prefix_len, PrefixPlan* p) {
  *p = PrefixPlan{};
  p->rows = c.batch * c.group_size;
  p->tiles = (p->rows + kTile - 1) / kTile;
  p->per_head = (p->tiles + 1) / 2;
  p->units = c.num_kv_heads * p->per_head;
  p->key_tiles = (prefix_len + kTile - 1) / kTile;
  const long long total = (long long)p->tiles * p->key_tiles * c.num_kv_heads;
  if (total > (1ll << 31) - (1 << 24)) return false;
  p->head_work = p->tiles * p->key_tiles;
  p->total = (int)total;
  if (!prefix_len) return true;
  const long long pieces = (long long)p->units * p->key_tiles;
  const int blocks = (int)(pieces < num_sms() ? pieces : num_sms());
  p->chunk = (p->total + blocks - 1) / blocks;
  p->blocks = (p->total + p->chunk - 1) / p->chunk;
  return true;
}

constexpr int kMaxSplits = 512;  // bounds the merge's shared memory (8 x (SMs + 512) floats)

struct AttendLayout {
  int splits;  // shares of a (sequence, KV head)'s own tokens, a warp's work each
  // prefix shares: ml fp32 [slots][128][4] (m, l, r, 0), num fp32 [slots][128
  // rows][128]; own shares: ml [units][splits][G][4], num [units][splits][G][128];
  // score fp32 [units][capacity][Gp], Gp = 4 or 8
  size_t off_pml, off_pnum, off_ml, off_num, off_score, total;
};

AttendLayout layout(const ri_token_cache& c, const PrefixPlan& pp) {
  AttendLayout L;
  const size_t units = (size_t)c.batch * c.num_kv_heads;
  // own shares: tasks for 8 warps per SM, two rounds of them, of 64 tokens or
  // more of a full cache; without a prefix (beside which the rounds run into
  // one another) up to four, the count whose last round is fullest, the fewest
  // of about equal ones.  Against two rounds always: 512 heads of 1.7K tokens 89
  // us (92), 800 of 1K 83 (88), 128 of 4K 56.5 (59); where the rounds were full
  // anyhow, 128 heads of 1.5K 30.5 us (29.7).
  const long long warps = 8ll * num_sms(), n = (long long)units;
  long long most = (c.capacity + 63) / 64;
  if (most > kMaxSplits) most = kMaxSplits;
  long long splits = (2 * warps + n - 1) / n;
  if (splits > most) splits = most;
  double best = 0.0;
  for (long long s = splits, end = (4 * warps + n - 1) / n; s <= end && s <= most && !pp.blocks; ++s) {
    const long long rounds = (n * s + warps - 1) / warps;
    const double full = (double)(n * s) / (double)(rounds * warps);
    if (full > best + 0.02) {
      best = full;
      splits = s;
    }
  }
  L.splits = (int)splits;
  const size_t slots = pp.blocks ? 2 * (size_t)(pp.blocks + pp.units) : 0;
  size_t off = kStatusBytesHost;
  L.off_pml = off;
  off = align_up(off + slots * kTile * sizeof(float4), 256);
  L.off_pnum = off;
  off = align_up(off + slots * kTile * kD * sizeof(float), 256);
  L.off_ml = off;
  off = align_up(off + units * splits * c.group_size * sizeof(float4), 256);
  L.off_num = off;
  off = align_up(off + units * splits * c.group_size * kD * sizeof(float), 256);
  L.off_score = off;
  off = align_up(off + units * c.capacity * (c.group_size <= 4 ? 4 : 8) * sizeof(float), 256);
  L.total = off;
  return L;
}

constexpr size_t kTaskCounter = 128;  // byte of the status region: own tasks taken

struct AttendParams {
  ri_token_cache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  float4* pml;
  float* pnum;
  float4* ml;
  float* num;
  float* score;
  int* status;
  PrefixPlan plan;  // blocks == 0: no prefix
  int prefix_len;
  int* next_task;  // own tasks taken, in the workspace's status region; 0 between calls
  int tasks;       // own tasks: units * splits
  int splits, add_weight;
  unsigned long long wait_ns;  // limit of a wait in the prefix kernel
  int hand_off;    // self-test: what the prefix's first block leaves undone (0: nothing)
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
struct f2 {
  unsigned long long v;
};
__device__ __forceinline__ f2 make_f2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(f2 a, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(a.v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Towards zero.
__device__ __forceinline__ uint32_t pack_bf16_down(float lo, float hi) {
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
constexpr float kLeast = 9.1835496e-41f;  // 2^-133, the least bf16 above 0

// The two values of a packed pair.
__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

// True in one lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// --------------------------------------------------------------- own tokens
// A warp's task: one share of a (sequence, KV head)'s own tokens, in tiles of
// 16 tokens through a ring of asynchronous copies.  S = Q K^T on m16n8k16
// tiles (the G <= 8 query rows of 16), whose fragment is, as it stands, the
// B operand of num^T += V^T P^T.
constexpr int kOwnWarps = 4;
constexpr int kOwnThreads = kOwnWarps * 32;
constexpr int kOwnTokens = 16;
constexpr int kOwnTile = kOwnTokens * kD * 2;  // 4 KB of K, as much of V
constexpr int kOwnStages = 3;        // of a block of its own
constexpr int kOwnStagesBeside = 2;  // of a warp beside the prefix
constexpr size_t own_ring_bytes(int stages) { return (size_t)stages * 2 * kOwnTile; }
constexpr size_t kOwnSmem = kOwnWarps * own_ring_bytes(kOwnStages);

__device__ __forceinline__ void cp_async16_zero(uint32_t smem, const void* g, bool valid) {
  const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(g), "r"(n)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int live_len(const ri_token_cache& c, int unit, int* status) {
  int len = c.lens[unit];
  if (len < 0 || len > c.capacity) {
    record_status(status, RI_ERR_INVALID_ARG);
    len = len < 0 ? 0 : c.capacity;
  }
  return len;
}

template <int kStages>
__device__ __forceinline__ void own_task(const AttendParams& p, int task, uint32_t buf) {
  const int unit = task / p.splits, split = task - unit * p.splits;
  const int G = p.c.group_size, Gp = G <= 4 ? 4 : 8;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;  // score row (query) and column pair of a thread
  const int cap = p.c.capacity;
  const int len = live_len(p.c, unit, p.status);
  // whole tiles of 16 tokens, split evenly
  const int tiles = (len + kOwnTokens - 1) / kOwnTokens;
  const int t0 = (int)((long long)tiles * split / p.splits);
  const int t1 = (int)((long long)tiles * (split + 1) / p.splits);
  float4* ml = p.ml + ((size_t)unit * p.splits + split) * G;
  if (t0 >= t1) {
    if (lane < G) ml[lane] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    return;
  }
  const uint8_t* K = static_cast<const uint8_t*>(p.c.K) + (size_t)unit * cap * kD * 2;
  const uint8_t* V = static_cast<const uint8_t*>(p.c.V) + (size_t)unit * cap * kD * 2;

  // chunk c (16 bytes) of row r of a tile, XOR-swizzled for ldmatrix
  auto at = [](int r, int c) { return (uint32_t)(r * 256 + ((c ^ (r & 7)) << 4)); };
  auto copy = [&](int t, int stage) {
    const uint32_t dst = buf + stage * 2 * kOwnTile;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // two whole rows per instruction
      const int r = 2 * i + (lane >> 4), c = lane & 15;
      const int tok = t * kOwnTokens + r;
      const bool valid = tok < len;
      const size_t src = valid ? (size_t)tok * 256 + c * 16 : 0;
      cp_async16_zero(dst + at(r, c), K + src, valid);
      cp_async16_zero(dst + kOwnTile + at(r, c), V + src, valid);
    }
  };
  __syncwarp();  // the ring's last readers (the warp's task before) are through
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (t0 + i < t1) copy(t0 + i, i);
    cp_async_commit();
  }
  // query rows as the A operand: rows g (valid below G), rows 8..15 are zero
  uint32_t qa[8][2];
  const uint32_t* q = reinterpret_cast<const uint32_t*>(
      p.q + ((size_t)unit * G + (g < G ? g : 0)) * kD);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    qa[k][0] = g < G ? q[k * 8 + tq] : 0u;
    qa[k][1] = g < G ? q[k * 8 + 4 + tq] : 0u;
  }
  float m = kLowest, l = 0.f;  // of query g, over this thread's columns for l
  float o[8][4];                 // numerator^T: rows d = 16 i + lane / 4 (+ 8), columns 2 tq, + 1
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

  int stage = 0;
#pragma unroll 1
  for (int t = t0; t < t1; ++t) {
    if (t + kStages - 1 < t1)
      copy(t + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
    cp_async_commit();
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t kb = buf + stage * 2 * kOwnTile, vb = kb + kOwnTile;
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // matrices: keys 0-7 / 8-15 (lane bit 4) x the two halves of 16 d (bit 3)
      uint32_t b[4];
      ldsm_x4(b, kb + at((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
      mma16816(s[0], qa[k][0], 0u, qa[k][1], 0u, b[0], b[1]);
      mma16816(s[1], qa[k][0], 0u, qa[k][1], 0u, b[2], b[3]);
    }
    float x[4] = {s[0][0] * kScaleLog2, s[0][1] * kScaleLog2, s[1][0] * kScaleLog2,
                  s[1][1] * kScaleLog2};
    const int tok = t * kOwnTokens + 2 * tq;  // tokens tok, tok + 1, tok + 8, tok + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ti = tok + (i & 1) + (i >> 1) * 8;
      if (ti >= len) x[i] = -INFINITY;
      else if (p.add_weight && g < G) p.score[((size_t)unit * cap + ti) * Gp + g] = x[i];
    }
    float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
    const bool grow = top > m + kLazy;
    if (__any_sync(~0u, grow)) {
      const float mn = grow ? top : m;
      const float f = exp2_approx(m - mn);
      m = mn;
      l *= f;
      const float f0 = __shfl_sync(~0u, f, 8 * tq), f1 = __shfl_sync(~0u, f, 8 * tq + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f1;
        o[i][2] *= f0;
        o[i][3] *= f1;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = exp2_approx(x[i] - m);
    l += (x[0] + x[1]) + (x[2] + x[3]);
    // the probabilities and what their rounding left, as two products: the
    // copies are the bound here, not the tensor cores.  Rounded towards zero,
    // and what is left not below kLeast, so that neither part of a probability
    // is 0 or negative: both products of an infinite value are that infinity.
    const uint32_t p0 = pack_bf16_down(x[0], x[1]), p1 = pack_bf16_down(x[2], x[3]);
    auto left = [](float v, float part) { return fmaxf(v - part, fminf(v, kLeast)); };
    const uint32_t q0 = pack_bf16(left(x[0], bf16_lo(p0)), left(x[1], bf16_hi(p0)));
    const uint32_t q1 = pack_bf16(left(x[2], bf16_lo(p1)), left(x[3], bf16_hi(p1)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // V^T: matrices keys 0-7 / 8-15 (lane bit 4) x d halves of 16 (bit 3)
      uint32_t a[4];
      ldsm_x4_t(a, vb + at((lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)));
      mma16816(o[i], a[0], a[1], a[2], a[3], p0, p1);
      mma16816(o[i], a[0], a[1], a[2], a[3], q0, q1);
    }
    __syncwarp();
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  l += __shfl_xor_sync(~0u, l, 1);
  l += __shfl_xor_sync(~0u, l, 2);
  if (tq == 0 && g < G) ml[g] = make_float4(m, l, l, 0.f);  // p' = p to 2^-15
  float* num = p.num + ((size_t)unit * p.splits + split) * G * kD;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (2 * tq + e < G)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        num[(2 * tq + e) * kD + 16 * i + g] = o[i][e];
        num[(2 * tq + e) * kD + 16 * i + g + 8] = o[i][2 + e];
      }
}

// The next task of the shared counter (p.tasks or more: none is left).  A
// task's result is the same whoever takes it.
__device__ __forceinline__ int take_task(const AttendParams& p) {
  int t = 0;
  if ((threadIdx.x & 31) == 0) t = atomicAdd(p.next_task, 1);
  return __shfl_sync(~0u, t, 0);
}

// The own tokens without a prefix, or what the warps beside the prefix have
// left of them: those blocks start as the prefix's blocks end.
__global__ void __launch_bounds__(kOwnThreads)
    own_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  // behind a prefix launch everything older is complete (it has waited)
  if (!p.plan.blocks) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  const uint32_t buf = smem_u32(smem) + warp * own_ring_bytes(kOwnStages);
  if (p.plan.blocks) {
    for (int t = take_task(p); t < p.tasks; t = take_task(p)) own_task<kOwnStages>(p, t, buf);
  } else {
    // the first tasks are the warps' own numbers; the next one is asked for
    // before a task and needed after it
    const int first = gridDim.x * kOwnWarps;
    int t = blockIdx.x * kOwnWarps + warp;
    while (t < p.tasks) {
      int next = p.tasks;
      if ((threadIdx.x & 31) == 0 && first < p.tasks) next = first + atomicAdd(p.next_task, 1);
      own_task<kOwnStages>(p, t, buf);
      t = __shfl_sync(~0u, next, 0);
    }
  }
  // this launch completes after the prefix launch, so that the merge, which
  // waits for this one, has both
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------ prefix kernel
// K / V tiles in flight: 4 beside two query tiles; with one row tile per KV
// head (the memory-bound case) the second query tile's room is a fifth
constexpr int kRingPair = 4, kRingSingle = 5;
constexpr int kSoftmaxWarps = 8;          // two warpgroups, one per slot
constexpr int kWarpMma = 8, kWarpLoad = 9;
constexpr int kWarpOwn = 10;              // warps 10 and 11: own tokens meanwhile
constexpr int kPrefixThreads = 384;
// Registers: 168 per thread at launch (384 x 168 = 64512); the softmax
// warpgroups hold a row's 128 scores and take 192 each, the third goes down
// to 112: 256 x 192 + 128 x 112 = 63488.
constexpr int kRegsSoftmax = 192, kRegsRest = 112;
// TMEM columns: scores (and, over them, the probabilities) of slot i, then
// the numerators.  A tile's scores go over the probabilities of the slot's tile
// before: one thread issues both products, and its MMAs run in issue order.
constexpr uint32_t kColS = 0, kColO = 256;

struct PrefixShared {
  uint64_t full[kRingSingle], empty[kRingSingle];
  uint64_t q_full, s_full[2], p_full[2][2], o_full[2], drain;
  uint32_t tmem;
  int done;  // the block's prefix work is through: no more own shares are taken
};
constexpr size_t kPrefixSmem = 1024 + (2 + kRingPair) * (size_t)kTileBytes +
                               2 * own_ring_bytes(kOwnStagesBeside) + sizeof(PrefixShared);

// V tile [key][d] as the B operand of num += P V (N = d contiguous, "MN
// major"): 128-byte swizzle, 64 columns of d per half tile; adjacent halves
// kHalfTile apart (leading offset), adjacent groups of 8 keys 1024 bytes
// apart (stride offset).
__device__ __forceinline__ uint64_t umma_desc_v(uint32_t addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(kHalfTile >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// D[tmem] (+)= A[tmem] B[smem], A = probabilities, two bf16 per column.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One K or V tile: 128 tokens from token `y` on, as two halves of 64 columns.
__device__ __forceinline__ void tma_load_tile(void* dst, const CUtensorMap* map, int y, int head,
                                              uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(0), "r"(head),
      "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A share of one unit: key tiles [t0, t1), one or two row tiles.  With two
// row tiles ("pair") both slots see every key tile; with one, the slots take
// the key tiles in turn, so that one's softmax runs beside the other's
// products here too, and are joined at the end.
struct Share {
  int head, row0, t0, t1;
  bool pair;
};

// In the place of a share that a wait's expiry left incomplete (whatever its
// numerators hold).  Joined with any other, its reference is the greatest, so
// the sums are l = -inf, which no true share has, and r = NaN: out is NaN.
__device__ __forceinline__ float4 lost_share() {
  return make_float4(-kLowest, -INFINITY, __int_as_float(0x7fffffff), 0.f);
}

template <int kQTiles>
__device__ __forceinline__ Share share_of(const PrefixPlan& p, int u, int x0, int x1) {
  Share s;
  s.head = u / p.per_head;
  s.row0 = (u % p.per_head) * 2 * kTile;
  s.t0 = p.tile_at(u, x0);
  s.t1 = p.tile_at(u, x1);
  s.pair = kQTiles == 2 && p.work_per_tile(u) == 2;
  return s;
}

template <int kRing>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ AttendParams p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~1023ull);
  constexpr int kQTiles = kRing == kRingSingle ? 1 : 2;
  static_assert(kQTiles + kRing == 2 + kRingPair, "one layout of shared memory");
  uint8_t* sq = base;                             // kQTiles query tiles
  uint8_t* ring = base + kQTiles * kTileBytes;    // kRing K / V tiles
  uint8_t* own = ring + kRing * kTileBytes;       // the rings of warps 10 and 11
  PrefixShared* sh =
      reinterpret_cast<PrefixShared*>(own + 2 * own_ring_bytes(kOwnStagesBeside));
  // (shuffled: uniform over the warp for the compiler too)
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const PrefixPlan& plan = p.plan;

  if (warp == kWarpMma) {
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    mbar_init(&sh->q_full, kSoftmaxWarps * 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_full[i][0], 4);
      mbar_init(&sh->p_full[i][1], 4);
      mbar_init(&sh->o_full[i], 1);
    }
    mbar_init(&sh->drain, 1);
    sh->done = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, sh->tmem, 0);
  // what came before on the stream is complete from here on; only then may
  // the own tokens' launch start, which reads what that wrote without a wait
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int x0 = plan.from(blockIdx.x), x1 = plan.from(blockIdx.x + 1);
  const int u0 = plan.unit_of(x0);
  const int last_tile = plan.key_tiles - 1;
  // A wait that expires is recorded; its role then runs on without waiting,
  // copying or multiplying, so every loop and barrier still ends, and the
  // softmax warps give their shares out as lost ones.
  bool ok = true;
  auto withheld = [&](int hand_off) { return p.hand_off == hand_off && blockIdx.x == 0; };

  if (warp >= kSoftmaxWarps) {
    // one instruction for the whole warpgroup
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------- loads
      if (lane == 0) {
        int n = 0;  // tiles loaded
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
        auto load = [&](const CUtensorMap* map, int t, int head) {
          const int st = n % kRing;
          if (n == 1 && withheld(RI_TOKEN_WAIT_TILE)) ok = false;
          if (ok && n >= kRing &&
              !mbar_wait(&sh->empty[st], (uint32_t)((n / kRing - 1) & 1), p.wait_ns)) {
            record_status(p.status, RI_ERR_TIMEOUT);
            ok = false;
          }
          if (!ok) return;
          uint8_t* dst = ring + st * kTileBytes;
          mbar_arrive_expect_tx(&sh->full[st], kTileBytes);
          tma_load_tile(dst, map, t * kTile, head, &sh->full[st]);
          ++n;
        };
        for (int u = u0; u < plan.units && plan.start(u) < x1; ++u) {
          const Share s = share_of<kQTiles>(plan, u, x0, x1);
          const int ahead = s.pair ? 1 : 2;  // key tiles before the first value tile
          for (int t = s.t0; t < s.t1 && t < s.t0 + ahead; ++t) load(&map_k, t, s.head);
          for (int t = s.t0; t < s.t1; ++t) {
            load(&map_v, t, s.head);
            if (t + ahead < s.t1) load(&map_k, t + ahead, s.head);
          }
        }
        // every copy has landed before the block's shared memory goes away
        for (int i = n > kRing ? n - kRing : 0; i < n; ++i)
          if (!mbar_wait(&sh->full[i % kRing], (uint32_t)((i / kRing) & 1)))
            record_status(p.status, RI_ERR_TIMEOUT);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      // -------------------------------------------------------- MMA issuer
      // The whole warp runs the loop and one elected lane issues: with the
      // control flow and the addresses uniform over the warp an MMA takes a
      // few issue slots (from a lane-0 branch: about 130 cycles each, more
      // than the MMA itself).
      {
        constexpr uint32_t idesc_s = umma_idesc_bf16_f32(kTile, kTile);
        constexpr uint32_t idesc_o = umma_idesc_bf16_f32(kTile, kD) | (1u << 16);  // B: MN major
        const uint32_t q_addr = smem_u32(sq), ring_addr = smem_u32(ring);
        int n = 0;  // tiles consumed
        uint32_t q_phase = 0, p_phases = 0;  // bit i of p_phases: slot i
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (ok) {
            ok = __all_sync(~0u, mbar_wait(bar, parity, p.wait_ns));
            if (!ok && lane == 0) record_status(p.status, RI_ERR_TIMEOUT);
          }
        };
        auto wait_tile = [&](int i) { wait(&sh->full[i % kRing], (uint32_t)((i / kRing) & 1)); };
        auto commit = [&](uint64_t* bar) {
          if (ok && elect_one()) umma_commit(bar);
        };
        // S[slot] = Q K^T for the tile in ring slot i % kRing
        auto scores = [&](int slot, int qtile, int i) {
          if (!ok) return;
          tc_fence_after();
          const uint64_t a = umma_desc_sw128(q_addr + qtile * kTileBytes);
          const uint64_t b = umma_desc_sw128(ring_addr + (i % kRing) * kTileBytes);
          const uint32_t d = tmem + kColS + slot * kTile;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t off = ((k >> 2) * kHalfTile + (k & 3) * 32) >> 4;
              umma_bf16(d, a + off, b + off, idesc_s, k > 0);
            }
            if (!withheld(RI_TOKEN_WAIT_SCORES)) umma_commit(&sh->s_full[slot]);
          }
          __syncwarp();
        };
        // O[slot] += P[slot] V, the first 64 keys while the others are in the works
        auto values = [&](int slot, int i, bool first) {
          const uint64_t b = umma_desc_v(ring_addr + (i % kRing) * kTileBytes);
          const uint32_t d = tmem + kColO + slot * kD, a = tmem + kColS + slot * kTile;
          const uint32_t phase = (p_phases >> slot) & 1;
          p_phases ^= 1u << slot;
          wait_tile(i);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            wait(&sh->p_full[slot][half], phase);
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; ++k)
                umma_ts(d, a + 8 * k, b + k * (2048 >> 4), idesc_o, k > 0 || !first);
            }
            __syncwarp();
          }
        };
        auto release = [&](int i) { commit(&sh->empty[i % kRing]); };
        for (int u = u0; u < plan.units && plan.start(u) < x1; ++u) {
          const Share s = share_of<kQTiles>(plan, u, x0, x1);
          const int T = s.t1 - s.t0;
          if (T <= 0) continue;
          wait(&sh->q_full, q_phase);
          q_phase ^= 1;
          if (s.pair) {
            wait_tile(n);
            scores(0, 0, n);
            scores(1, 1, n);
            release(n++);
            for (int j = 0; j < T; ++j) {
              const int v = n++;
              const int k = j + 1 < T ? n++ : -1;
#pragma unroll 1
              for (int slot = 0; slot < 2; ++slot) {
                values(slot, v, j == 0);
                if (slot == 1) release(v);
                if (k >= 0) {
                  if (slot == 0) wait_tile(k);
                  scores(slot, slot, k);
                  if (slot == 1) release(k);
                } else {
                  commit(&sh->o_full[slot]);
                }
              }
            }
          } else {
            for (int j = 0; j < 2 && j < T; ++j) {
              wait_tile(n);
              scores(j, 0, n);
              release(n++);
            }
            for (int j = 0; j < T; ++j) {
              const int slot = j & 1;
              const int v = n++;
              const int k = j + 2 < T ? n++ : -1;
              values(slot, v, j < 2);
              release(v);
              if (k >= 0) {
                wait_tile(k);
                scores(slot, 0, k);
                release(k);
              } else {
                commit(&sh->o_full[slot]);
              }
            }
          }
        }
        // nothing of the tensor pipe is in flight when the memory is freed
        if (elect_one()) umma_commit(&sh->drain);
        if (!mbar_wait(&sh->drain, 0)) record_status(p.status, RI_ERR_TIMEOUT);
      }
      __syncwarp();
    } else {
      // ------------------------------------------ own tokens, meanwhile
      const uint32_t buf = smem_u32(own) + (warp - kWarpOwn) * own_ring_bytes(kOwnStagesBeside);
      while (!*reinterpret_cast<volatile int*>(&sh->done)) {
        const int t = take_task(p);
        if (t >= p.tasks) break;
        own_task<kOwnStagesBeside>(p, t, buf);
      }
      cp_async_wait<0>();
    }
  } else {
    // ----------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int slot = warp >> 2;
    const int row = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_addr + kColS + slot * kTile;
    const uint32_t t_o = tmem + lane_addr + kColO + slot * kD;
    uint32_t s_phase = 0, o_phase = 0, unit_phase = 0;  // unit: of o_full[0]
    const int H = p.c.num_kv_heads, G = p.c.group_size;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(~0u, mbar_wait(bar, parity, p.wait_ns));
      if (!ok && lane == 0) record_status(p.status, RI_ERR_TIMEOUT);
    };
    for (int u = u0; u < plan.units && plan.start(u) < x1; ++u) {
      const Share s = share_of<kQTiles>(plan, u, x0, x1);
      const int T = s.t1 - s.t0;
      if (T <= 0) continue;
      // the unit's query rows, into the K-major 128-byte swizzle: a thread
      // takes chunk tid % 16 of every 16th row, eight loads in flight
      for (int tile = 0; tile < (s.pair ? 2 : 1); ++tile) {
        uint4 v[8];
        const int ch = tid & 15;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int qr = s.row0 + tile * kTile + i * 16 + (tid >> 4);
          const int qb = qr / G;
          v[i] = make_uint4(0, 0, 0, 0);
          if (qr < plan.rows)
            v[i] = ldg_nc_v4(p.q + (((size_t)qb * H + s.head) * G + (qr - qb * G)) * kD + ch * 8);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 16 + (tid >> 4);
          *reinterpret_cast<uint4*>(sq + tile * kTileBytes + (ch >> 3) * kHalfTile + r * 128 +
                                    (((ch & 7) ^ (r & 7)) << 4)) = v[i];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh->q_full);

      const int row_tile0 = s.row0 + (s.pair ? slot * kTile : 0);
      const bool live = row_tile0 + (warp & 3) * 32 < plan.rows;  // any row of this warp
      const int step = s.pair ? 1 : 2;
      float m = 0.f, l = 0.f, rs = 0.f;
      bool any = false;
      for (int t = s.t0 + (s.pair ? 0 : slot); t < s.t1; t += step) {
        wait(&sh->s_full[slot], s_phase);
        s_phase ^= 1;
        if (ok && live) {
          tc_fence_after();
          uint32_t x[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_nowait(t_s + c * 32, x[c]);
          tmem_wait_ld();
          if (t == last_tile) {
            const int n = p.prefix_len - t * kTile;  // valid keys, >= 1
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c * 32 + i >= n) x[c][i] = 0xff800000u;  // -inf
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = __uint_as_float(x[c][0]);
#pragma unroll
            for (int i = 1; i < 31; i += 2)
              mx[c] = fmax3f(mx[c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
            mx[c] = fmaxf(mx[c], __uint_as_float(x[c][31]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kScaleLog2;
          if (!any) {
            m = fmaxf(top, kLowest);
          } else {
            // the numerator is complete up to the previous tile here: the
            // commit that signalled these scores covers every MMA before it
            const bool grow = top > m + kLazy;
            if (__any_sync(~0u, grow)) {
              const float mn = grow ? top : m;
              const float f = exp2_approx(m - mn);
              m = mn;
              l *= f;
              rs *= f;
              uint32_t o[16];
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {  // 16 columns: the scores stay in registers
                tmem_ld16(t_o + c * 16, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(t_o + c * 16, o);
              }
            }
          }
          any = true;
          const f2 scale = make_f2(kScaleLog2, kScaleLog2), shift = make_f2(-m, -m);
          // The rounded sum is worth its cost where one key may count for much
          // of a row (an eighth of what it has gathered): there the probabilities
          // are read back; elsewhere their errors average out and the exact
          // sum stands in for it.
          const bool heavy = __any_sync(~0u, exp2_approx(top - m) * 8.f > l);
          f2 sum[2] = {make_f2(0.f, 0.f), make_f2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const f2 v = fma2(make_f2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])),
                          scale, shift);
              float a, b;
              split(v, &a, &b);
              a = exp2_approx(a);
              b = exp2_approx(b);
              sum[i & 1] = add2(sum[i & 1], make_f2(a, b));
              pk[i] = pack_bf16(a, b);
            }
            tmem_st16(t_s + c * 16, pk);
            if (c == 1) {  // 64 keys are through: their products may start
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh->p_full[slot][0]);
            }
          }
          float s0, s1, s2, s3;
          split(sum[0], &s0, &s1);
          split(sum[1], &s2, &s3);
          s0 = (s0 + s1) + (s2 + s3);
          l += s0;
          tmem_wait_st();
          if (heavy) {
            s0 = 0.f;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t pk[16];
              tmem_ld16(t_s + c * 16, pk);
#pragma unroll
              for (int i = 0; i < 16; ++i) s0 += bf16_lo(pk[i]) + bf16_hi(pk[i]);
            }
          }
          rs += s0;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->p_full[slot][1]);
        } else if (lane == 0) {
          mbar_arrive(&sh->p_full[slot][0]);
          mbar_arrive(&sh->p_full[slot][1]);
        }
        __syncwarp();
      }

      // -------------------------------------------- the unit's share goes out
      const bool used = s.pair || s.t0 + slot < s.t1;  // this slot had a tile
      if (used) {
        wait(&sh->o_full[slot], o_phase);
        o_phase ^= 1;
      } else {
        // the other slot's products read the query tile, which the share goes over
        wait(&sh->o_full[0], unit_phase);
      }
      const float4 mine = !ok    ? lost_share()
                          : used ? make_float4(m, l, rs, 0.f)
                                 : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      // Through shared memory (the query tiles are free: an equal part per
      // warp), so that rows leave as whole 128- or 256-byte pieces: a thread
      // holds a row, and 32 rows' 16-byte stores would each touch 32 lines.
      constexpr int kCols = 32 * kQTiles, kChunks = kCols / 4;  // columns at a time
      const size_t out_slot = 2 * ((size_t)blockIdx.x + u) + (s.pair ? slot : 0);
      float* num = p.pnum + out_slot * kTile * kD;
      float4* ml = p.pml + out_slot * kTile;
      uint8_t* stage = sq + warp * (32 * kCols * 4);
      const int warp_row = (warp & 3) * 32;
      const int n_rows = min(32, plan.rows - row_tile0 - warp_row);  // <= 0: none live
      auto put = [&](int i, uint4 v) {  // 16-byte chunk i of this thread's row
        *reinterpret_cast<uint4*>(stage + lane * (kCols * 4) +
                                  ((i ^ (lane & (kChunks - 1))) << 4)) = v;
      };
      auto send = [&](int col) {  // the warp's rows, kCols columns from col on
        __syncwarp();
        const int c = lane & (kChunks - 1);
        for (int r = lane / kChunks; r < n_rows; r += 32 / kChunks)
          *reinterpret_cast<uint4*>(num + (warp_row + r) * kD + col + c * 4) =
              *reinterpret_cast<const uint4*>(stage + r * (kCols * 4) +
                                              ((c ^ (r & (kChunks - 1))) << 4));
        __syncwarp();
      };
      if (s.pair) {
        named_barrier(1, kSoftmaxWarps * 32);  // both slots' scores are through
        if (live) {
          tc_fence_after();
          if (lane < n_rows) ml[row] = mine;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t a[32];
            tmem_ld32_nowait(t_o + c * 32, a);
            tmem_wait_ld();
            const int part = c * 32 % kCols / 4;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              put(part + i, make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]));
            if ((c + 1) * 32 % kCols == 0) send((c + 1) * 32 - kCols);
          }
          tc_fence_before();
        }
      } else {
        // both slots hold the same rows: (m, l, r) change hands, and each
        // warpgroup joins half of the columns of both numerators
        float4* ex = reinterpret_cast<float4*>(sq);  // [2][128]
        ex[slot * kTile + row] = mine;
        named_barrier(1, kSoftmaxWarps * 32);
        const float4 e0 = ex[row], e1 = ex[kTile + row];
        named_barrier(1, kSoftmaxWarps * 32);
        const float M = fmaxf(e0.x, e1.x);
        const float f0 = exp2_approx(e0.x - M), f1 = exp2_approx(e1.x - M);
        const bool both = s.t1 - s.t0 > 1;
        if (live) {
          tc_fence_after();
          if (lane < n_rows && slot == 0)
            ml[row] = make_float4(M, f0 * e0.y + f1 * e1.y, f0 * e0.z + f1 * e1.z, 0.f);
          const uint32_t t_num = tmem + lane_addr + kColO + slot * 64;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t a[32], b[32];
            tmem_ld32_nowait(t_num + c * 32, a);
            if (both) tmem_ld32_nowait(t_num + kD + c * 32, b);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float v = f0 * __uint_as_float(a[i]);
              if (both) v = fmaf(f1, __uint_as_float(b[i]), v);
              a[i] = __float_as_uint(v);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              put(c * 32 % kCols / 4 + i,
                  make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]));
            if ((c + 1) * 32 % kCols == 0) send(slot * 64 + (c + 1) * 32 - kCols);
          }
          tc_fence_before();
        }
      }
      // the numerators are read and the query tiles done with (their last
      // scores were waited for) before the next unit replaces either
      named_barrier(1, kSoftmaxWarps * 32);
      unit_phase ^= 1;
    }
    if (tid == 0) *reinterpret_cast<volatile int*>(&sh->done) = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// -------------------------------------------------------------------- merge
// One block per (sequence, KV head) and chunk of its own tokens.  Every block
// joins the references and sums of its G rows (a warp per row, its lanes over
// the shares, whose factors 2^(m - M) stay in shared memory); the unit's
// blocks share out the rows' numerators, four columns per lane.
constexpr int kMergeThreads = 256;
constexpr int kMergeTokens = 4 * kMergeThreads;  // own tokens of a chunk, at least

// log2 scores of one own token, Gp = 4 or 8 of them
struct Scores {
  float4 a, b;
};
__device__ __forceinline__ Scores load_scores(const AttendParams& p, size_t row, int G) {
  const float4* s = reinterpret_cast<const float4*>(p.score) + row * (G <= 4 ? 1 : 2);
  Scores r;
  r.a = s[0];
  r.b = G > 4 ? s[1] : make_float4(0.f, 0.f, 0.f, 0.f);
  return r;
}

__global__ void __launch_bounds__(kMergeThreads, 4)
    merge_kernel(const __grid_constant__ AttendParams p, int chunks) {
  extern __shared__ float factor[];  // [G][shares]
  __shared__ float sh_lse[kMaxGroup], sh_r[kMaxGroup];
  __shared__ int sh_n[kMaxGroup], sh_slot[kMaxGroup];  // prefix shares, the first one's slot
  __shared__ float4 sh_part[kMergeThreads / 32][32];
  const int unit = blockIdx.x / chunks, chunk = blockIdx.x - unit * chunks;
  const int G = p.c.group_size, H = p.c.num_kv_heads;
  const int b = unit / H, h = unit - b * H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PrefixPlan& plan = p.plan;
  const int shares = plan.blocks + p.splits;  // room per row; most rows use fewer
  // (the lengths are older than the two launches before this one)
  const int len = live_len(p.c, unit, p.status);
  const int per_chunk = (p.c.capacity + chunks - 1) / chunks;
  const int i0 = chunk * per_chunk + threadIdx.x;
  const int end = p.add_weight ? min(len, (chunk + 1) * per_chunk) : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.next_task = 0;  // every task has been taken
  // the first own tokens' scores and weights, on their way meanwhile
  constexpr int kAhead = 2;
  const size_t row0 = (size_t)unit * p.c.capacity;
  Scores ahead[kAhead];
  float weight[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = i0 + j * kMergeThreads;
    if (i < end) {
      ahead[j] = load_scores(p, row0 + i, G);
      weight[j] = p.c.weight[row0 + i];
    }
  }
  if (warp < G) {
    const int g = warp, r = b * G + g, row = r % kTile;
    int c0 = 0, n_prefix = 0, u = 0, slot = 0;
    if (plan.blocks) {
      // the blocks whose work meets the row's unit
      u = h * plan.per_head + r / (2 * kTile);
      const int s0 = plan.start(u), s1 = s0 + plan.work_per_tile(u) * plan.key_tiles;
      c0 = s0 / plan.chunk;
      n_prefix = (s1 + plan.chunk - 1) / plan.chunk - c0;
      slot = 2 * (c0 + u) + (r / kTile & 1);
    }
    float* f = factor + g * shares;
    float m = -INFINITY, l = 0.f, rs = 0.f;
    for (int i = lane; i < n_prefix + p.splits; i += 32) {
      float4 v = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      if (i < n_prefix) {
        // (a block on the unit's edge may have no tile of it)
        if (plan.tile_at(u, plan.from(c0 + i)) < plan.tile_at(u, plan.from(c0 + i + 1)))
          v = p.pml[(size_t)(slot + 2 * i) * kTile + row];
      } else {
        v = p.ml[((size_t)unit * p.splits + i - n_prefix) * G + g];
      }
      f[i] = v.x;
      if (v.x > m) {
        const float e = exp2_approx(m - v.x);
        l = l * e + v.y;
        rs = rs * e + v.z;
        m = v.x;
      } else if (v.x > -INFINITY) {
        const float e = exp2_approx(v.x - m);
        l += v.y * e;
        rs += v.z * e;
      }
    }
    float M = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    const float e = m > -INFINITY ? exp2_approx(m - M) : 0.f;
    l *= e;
    rs *= e;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      l += __shfl_xor_sync(~0u, l, o);
      rs += __shfl_xor_sync(~0u, rs, o);
    }
    for (int i = lane; i < n_prefix + p.splits; i += 32)
      f[i] = f[i] > -INFINITY ? exp2_approx(f[i] - M) : -1.f;  // -1: nothing was written
    if (lane == 0) {
      sh_r[g] = rs;
      // (a sum of NaN: NaN; with a lost share: +inf, so that the row's
      // probabilities, 2^(score - lse), add nothing to the weights)
      sh_lse[g] = l == 0.f ? -INFINITY : l == -INFINITY ? INFINITY : M + log2f(l);
      sh_n[g] = n_prefix;
      sh_slot[g] = slot;
    }
  }
  __syncthreads();
  // The numerators: row g is joined by block g mod chunks of the unit, by
  // `per_row` warps that take its shares in turn, kFlight loads in flight each.
  constexpr int kFlight = 4;
  const int rows_here = chunk < G ? (G - chunk + chunks - 1) / chunks : 0;
  if (rows_here) {
    const int per_row = rows_here <= 1 ? 8 : rows_here <= 2 ? 4 : rows_here <= 4 ? 2 : 1;
    const int g = chunk + warp / per_row * chunks, part = warp % per_row;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g < G) {
      const int n = sh_n[g], all = n + p.splits;
      const float* f = factor + g * shares;
      const float4* prefix = reinterpret_cast<const float4*>(p.pnum) +
                             ((size_t)sh_slot[g] * kTile + (b * G + g) % kTile) * (kD / 4) + lane;
      const float4* own = reinterpret_cast<const float4*>(p.num) +
                          ((size_t)unit * p.splits * G + g) * (kD / 4) + lane;
      for (int f0 = part; f0 < all; f0 += kFlight * per_row) {
        float4 v[kFlight];
        float w[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
          const int i = f0 + j * per_row;
          w[j] = i < all ? f[i] : -1.f;
          v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          // (read with a factor of 0 too: a numerator of NaN counts all the same)
          if (!(w[j] < 0.f))
            v[j] = *(i < n ? prefix + (size_t)i * 2 * kTile * (kD / 4)
                           : own + (size_t)(i - n) * G * (kD / 4));
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
          acc.x = fmaf(w[j], v[j].x, acc.x);
          acc.y = fmaf(w[j], v[j].y, acc.y);
          acc.z = fmaf(w[j], v[j].z, acc.z);
          acc.w = fmaf(w[j], v[j].w, acc.w);
        }
      }
    }
    if (per_row > 1) {
      sh_part[warp][lane] = acc;
      __syncthreads();
      if (part == 0)
        for (int i = 1; i < per_row; ++i) {
          const float4 v = sh_part[warp + i][lane];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
    }
    if (g < G && part == 0) {
      const float inv = sh_r[g] == 0.f ? 0.f : 1.f / sh_r[g];  // (a sum of NaN: NaN)
      const size_t row = (size_t)unit * G + g;
      *reinterpret_cast<uint2*>(p.out + row * kD + lane * 4) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (p.lse && lane == 0)
        p.lse[row] = sh_lse[g] < INFINITY ? sh_lse[g] * kLn2 : __int_as_float(0x7fffffff);
    }
  }
  if (i0 >= end) return;
  float lse[kMaxGroup];
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g)  // (-inf: every score is -inf, and adds 2^-inf)
    lse[g] = g < G && sh_lse[g] != -INFINITY ? sh_lse[g] : 0.f;
  auto added = [&](const Scores& s) {  // (entries from G on were never written)
    float w = exp2_approx(s.a.x - lse[0]);
    if (G > 1) w += exp2_approx(s.a.y - lse[1]);
    if (G > 2) w += exp2_approx(s.a.z - lse[2]);
    if (G > 3) w += exp2_approx(s.a.w - lse[3]);
    if (G > 4) w += exp2_approx(s.b.x - lse[4]);
    if (G > 5) w += exp2_approx(s.b.y - lse[5]);
    if (G > 6) w += exp2_approx(s.b.z - lse[6]);
    if (G > 7) w += exp2_approx(s.b.w - lse[7]);
    return w;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = i0 + j * kMergeThreads;
    if (i < end) p.c.weight[row0 + i] = weight[j] + added(ahead[j]);
  }
#pragma unroll 2
  for (int i = i0 + kAhead * kMergeThreads; i < end; i += kMergeThreads)
    p.c.weight[row0 + i] += added(load_scores(p, row0 + i, G));
}

// --------------------------------------------------------------------- host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(ptr);
    return static_cast<EncodeTiledFn>(nullptr);
  }();
  return fn;
}

// [heads][length][128] bf16 with the prefix's strides, seen as [heads][2][length]
// [64]: a box is 128 tokens of both halves, each half 128-byte swizzled; rows
// past the length read as zero.
cudaError_t encode_prefix(CUtensorMap* map, const void* base, const ri_token_prefix& p,
                          int heads) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[4] = {64, (cuuint64_t)p.length, 2, (cuuint64_t)heads};
  cuuint64_t strides[3] = {(cuuint64_t)p.stride_t * 2, 128, (cuuint64_t)p.stride_h * 2};
  cuuint32_t box[4] = {64, kTile, 2, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <typename... Args, typename... Given>
cudaError_t launch_dependent(void (*kernel)(Args...), int blocks, int threads, size_t smem,
                             cudaStream_t s, const Given&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

size_t token_attend_bytes(const ri_token_cache& c, int prefix_len) {
  PrefixPlan plan;
  if (!plan_prefix(c, prefix_len, &plan)) return 0;
  return layout(c, plan).total;
}

cudaError_t launch_token_attend(const TokenAttendArgs& a, cudaStream_t s) {
  AttendParams p;
  memset(&p, 0, sizeof(p));
  if (!plan_prefix(a.c, a.p.length, &p.plan)) return cudaErrorInvalidValue;
  const AttendLayout L = layout(a.c, p.plan);
  p.c = a.c;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.pml = reinterpret_cast<float4*>(a.ws + L.off_pml);
  p.pnum = reinterpret_cast<float*>(a.ws + L.off_pnum);
  p.ml = reinterpret_cast<float4*>(a.ws + L.off_ml);
  p.num = reinterpret_cast<float*>(a.ws + L.off_num);
  p.score = reinterpret_cast<float*>(a.ws + L.off_score);
  p.status = reinterpret_cast<int*>(a.ws);
  p.next_task = reinterpret_cast<int*>(a.ws + kTaskCounter);
  p.prefix_len = a.p.length;
  p.splits = L.splits;
  const int units = a.c.batch * a.c.num_kv_heads;
  p.tasks = units * L.splits;
  p.add_weight = a.add_weight;
  p.wait_ns = a.wait_ns;
  p.hand_off = a.hand_off;
  cudaError_t e = set_smem_once(5, reinterpret_cast<const void*>(own_kernel), (int)kOwnSmem);
  if (e != cudaSuccess) return e;
  if (p.plan.blocks) {
    CUtensorMap mk, mv;
    const bool single = p.plan.tiles == 1;
    void (*kernel)(CUtensorMap, CUtensorMap, AttendParams) =
        single ? prefix_kernel<kRingSingle> : prefix_kernel<kRingPair>;
    e = set_smem_once(single ? 4 : 12, reinterpret_cast<const void*>(kernel), (int)kPrefixSmem);
    if (e == cudaSuccess) e = encode_prefix(&mk, a.p.K, a.p, a.c.num_kv_heads);
    if (e == cudaSuccess) e = encode_prefix(&mv, a.p.V, a.p, a.c.num_kv_heads);
    if (e == cudaSuccess)
      e = launch_dependent(kernel, p.plan.blocks, kPrefixThreads, kPrefixSmem, s, mk, mv, p);
    if (e != cudaSuccess) return e;
  }
  // Every launch sets up while the one before it ends (programmatic dependent
  // launch).  Behind a prefix the own tokens' blocks take the SMs that it
  // leaves; the merge waits for both.
  const int fill = 2 * num_sms(), want = (p.tasks + kOwnWarps - 1) / kOwnWarps;
  e = launch_dependent(own_kernel, want < fill ? want : fill, kOwnThreads, kOwnSmem, s, p);
  if (e == cudaSuccess) {
    // about one round of blocks, four per SM: a block per row of the group, or
    // per kMergeTokens own tokens, while there is room
    int chunks = a.add_weight ? (a.c.capacity + kMergeTokens - 1) / kMergeTokens : 1;
    if (chunks < a.c.group_size) chunks = a.c.group_size;
    const int most = 4 * num_sms() / units;
    if (chunks > most) chunks = most > 1 ? most : 1;
    const size_t smem = (size_t)a.c.group_size * (p.plan.blocks + L.splits) * sizeof(float);
    e = launch_dependent(merge_kernel, units * chunks, kMergeThreads, smem, s, p, chunks);
  }
  // without its merge a launch leaves the counter standing
  if (e != cudaSuccess) cudaMemsetAsync(p.next_task, 0, sizeof(int), s);
  return e;
}

}  // namespace ri
