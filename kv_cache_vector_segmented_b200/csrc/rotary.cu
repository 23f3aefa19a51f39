// Rotary positions: the rotation of query and key heads, alone (ri_rotary)
// and fused with the append to the exact token cache (ri_token_append).
//
// Mathematics: pair (a, b) of a head at position p turns by p * f_i radians.
// A position far out (p * f of 10^6 radians) loses all its fraction in fp32,
// so the table holds f / 2 pi as a 64-bit fraction of a turn: the product
// with the position, modulo 2^64, IS the angle's fraction of a turn, exact to
// 2^-64 * p, in two integer multiplications.  Its top 32 bits as a signed
// number of half turns go to sincospif.  The rotation runs in fp32 and is
// rounded once to the tensor's type.
//
// What bounds it: memory (each element read and written once); the angle of a
// pair is computed once per thread and used for every head the thread takes.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace ri {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void turn_angle(unsigned long long turns, int pos, float magnitude,
                                           float* c, float* s) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * turns;
  // [-2^31, 2^31) of 2^-31 half turns; the cut bits are 2^-32 of a turn
  const float half_turns = static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f;
  float sv, cv;
  sincospif(half_turns, &sv, &cv);
  *c = cv * magnitude;
  *s = sv * magnitude;
}

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f<__half>(__half v) {
  return __half2float(v);
}
template <>
__device__ __forceinline__ float to_f<float>(float v) {
  return v;
}
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}

// VEC elements moved by one access (16 bytes, or one element).
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Pack {
  T v[VEC];
};

// A head's accesses ("items"): rotated ones first, then copies of the rest.
//  half layout  item i turns elements [i VEC, +VEC) with those n further on;
//  interleaved  item i turns the pairs inside elements [i W, +W), W = VEC (at
//               least a pair).
// VEC is 16 bytes' worth of elements where every row and both halves start on
// 16 bytes, else 1.
template <typename T, int VEC, bool INTER>
struct Item {
  static constexpr int W = VEC > 1 ? VEC : 2;
  static constexpr int kPairs = INTER ? W / 2 : VEC;
  static constexpr int kElems = INTER ? W : 2 * VEC;
  int n;       // pairs of a head
  int at;      // first element
  bool turns;

  static __host__ __device__ int turned(int rotary_dim) {
    return INTER ? rotary_dim / W : rotary_dim / 2 / VEC;
  }
  static __host__ __device__ int count(int rotary_dim, int d) {
    return turned(rotary_dim) + (d - rotary_dim) / VEC;
  }
  __device__ __forceinline__ Item(int item, int rotary_dim) : n(rotary_dim / 2) {
    const int k = turned(rotary_dim);
    turns = item < k;
    at = turns ? item * (INTER ? W : VEC) : rotary_dim + (item - k) * VEC;
  }
  __device__ __forceinline__ void angles(const ri_rope& rope, int pos, float sign,
                                         float (&c)[kPairs], float (&s)[kPairs]) const {
    if (!turns) return;
    const unsigned long long* turns_of =
        reinterpret_cast<const unsigned long long*>(rope.turns) + (INTER ? at / 2 : at);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      turn_angle(__ldg(turns_of + i), pos, rope.magnitude, &c[i], &s[i]);
      s[i] *= sign;
    }
  }
  __device__ __forceinline__ void load(const T* row, T (&e)[kElems]) const {
    take<VEC>(row + at, e, 0);
    if (turns) {
      if (!INTER) take<VEC>(row + at + n, e, VEC);
      else if (VEC == 1) take<1>(row + at + 1, e, 1);
    }
  }
  __device__ __forceinline__ void store(T* row, const T (&e)[kElems]) const {
    put<VEC>(row + at, e, 0);
    if (turns) {
      if (!INTER) put<VEC>(row + at + n, e, VEC);
      else if (VEC == 1) put<1>(row + at + 1, e, 1);
    }
  }
  __device__ __forceinline__ void turn(T (&e)[kElems], const float (&c)[kPairs],
                                       const float (&s)[kPairs]) const {
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + VEC;
      const float a = to_f(e[ia]), b = to_f(e[ib]);
      e[ia] = from_f<T>(a * c[i] - b * s[i]);
      e[ib] = from_f<T>(b * c[i] + a * s[i]);
    }
  }

 private:
  template <int N>
  static __device__ __forceinline__ void take(const T* p, T (&e)[kElems], int to) {
    const Pack<T, N> v = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) e[to + i] = v.v[i];
  }
  template <int N>
  static __device__ __forceinline__ void put(T* p, const T (&e)[kElems], int from) {
    Pack<T, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.v[i] = e[from + i];
    *reinterpret_cast<Pack<T, N>*>(p) = v;
  }
};

// A block's 256 threads: `lanes` items of a row, fastest, so that a row is one
// contiguous access; then `row_slots` rows; then tokens.  A thread computes
// its item's angles once and uses them for every row of its token and group
// that falls to its slot, kBatch rows in flight.
struct Shape {
  int lanes, row_slots;  // powers of two
  int items;
  int group_rows;        // rows (heads) of a group, blockIdx.y counts the groups
};
constexpr int kBatch = 4;
constexpr int kMaxGridDim = 65535;  // of y and z

// Rows of a token and how many of them a group takes: the largest group whose
// grid still gives every SM four blocks.
Shape shape_of(int items, int tokens, int batch, int units, int rows_per_unit) {
  Shape s;
  s.items = items;
  s.lanes = 1;
  while (s.lanes < items && s.lanes < kThreads) s.lanes *= 2;
  int token_slots = kThreads / s.lanes;
  while (token_slots > 1 && token_slots / 2 >= tokens) token_slots /= 2;
  s.row_slots = kThreads / s.lanes / token_slots;
  const long long blocks = (long long)batch * ((tokens + token_slots - 1) / token_slots);
  int per = units;  // a group: units with their rows
  while (per > 1 && blocks * ((units + per - 1) / per) < 4ll * num_sms()) per = (per + 1) / 2;
  while ((units + per - 1) / per > kMaxGridDim) per *= 2;
  s.group_rows = per * rows_per_unit;
  return s;
}

dim3 grid_of(const Shape& s, int tokens, int batch, int rows) {
  const int token_slots = kThreads / s.lanes / s.row_slots;
  return dim3((unsigned)((tokens + token_slots - 1) / token_slots),
              (unsigned)((rows + s.group_rows - 1) / s.group_rows), (unsigned)batch);
}

template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, const Shape sh) {
  using I = Item<T, VEC, INTER>;
  const int lane = threadIdx.x & (sh.lanes - 1), slot = threadIdx.x / sh.lanes;
  const int token_slots = kThreads / sh.lanes / sh.row_slots;
  const int t = blockIdx.x * token_slots + slot / sh.row_slots;
  if (t >= a.T) return;
  const int r1 = min(a.heads, (int)(blockIdx.y + 1) * sh.group_rows);
  for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
    const int pos = a.pos[b * a.pos_stride + t];
    const T* x = static_cast<const T*>(a.x.data) + b * a.x.stride_b + t * a.x.stride_t;
    T* y = static_cast<T*>(a.out.data) + b * a.out.stride_b + t * a.out.stride_t;
    for (int i = lane; i < sh.items; i += sh.lanes) {
      const I item(i, a.rope.rotary_dim);
      float c[I::kPairs], s[I::kPairs];
      item.angles(a.rope, pos, a.inverse ? -1.f : 1.f, c, s);
      for (int r = blockIdx.y * sh.group_rows + (slot & (sh.row_slots - 1)); r < r1;
           r += kBatch * sh.row_slots) {
        T e[kBatch][I::kElems];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (r + j * sh.row_slots < r1)
            item.load(x + (r + j * sh.row_slots) * a.x.stride_h, e[j]);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (r + j * sh.row_slots < r1) {
            item.turn(e[j], c, s);
            item.store(y + (r + j * sh.row_slots) * a.out.stride_h, e[j]);
          }
      }
    }
  }
}

template <typename T, int VEC, bool INTER>
cudaError_t rotary_typed(const RotaryArgs& a, cudaStream_t s) {
  using I = Item<T, VEC, INTER>;
  const int n = a.rope.rotary_dim;
  // in place the rest of the head stays where it is
  const int items = a.x.data == a.out.data ? I::turned(n) : I::count(n, a.d);
  const Shape sh = shape_of(items, a.T, a.B, a.heads, 1);
  dim3 grid = grid_of(sh, a.T, a.B, a.heads);
  if (grid.z > kMaxGridDim) grid.z = kMaxGridDim;
  rotary_kernel<T, VEC, INTER><<<grid, kThreads, 0, s>>>(a, sh);
  return cudaGetLastError();
}

bool vec_ok(const ri_heads& x, int size) {
  return aligned16(x.data) && x.stride_b * size % 16 == 0 && x.stride_t * size % 16 == 0 &&
         x.stride_h * size % 16 == 0;
}

template <typename T>
cudaError_t rotary_of(const RotaryArgs& a, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const bool inter = a.rope.interleaved;
  const int run = inter ? a.rope.rotary_dim : a.rope.rotary_dim / 2;
  // whole 16-byte accesses where every row and both halves start on one
  const bool vec = run % V == 0 && a.d % V == 0 && a.rope.rotary_dim % V == 0 &&
                   vec_ok(a.x, sizeof(T)) && vec_ok(a.out, sizeof(T));
  if (vec) return inter ? rotary_typed<T, V, true>(a, s) : rotary_typed<T, V, false>(a, s);
  return inter ? rotary_typed<T, 1, true>(a, s) : rotary_typed<T, 1, false>(a, s);
}

// ------------------------------------------------------------------- append
// The rows of a token are dealt by KV head: its G query heads, its key, its
// value.  The value's row takes the same items, copied.
template <int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const AppendTokensArgs a, const Shape sh, int advance) {
  using T = __nv_bfloat16;
  using I = Item<T, VEC, INTER>;
  const int lane = threadIdx.x & (sh.lanes - 1), slot = threadIdx.x / sh.lanes;
  const int token_slots = kThreads / sh.lanes / sh.row_slots;
  const int t = blockIdx.x * token_slots + slot / sh.row_slots;
  const int H = a.c.num_kv_heads, G = a.q.data ? a.c.group_size : 0, cap = a.c.capacity;
  const int per = G + 2;  // rows of a KV head
  const int r0 = blockIdx.y * sh.group_rows, r1 = min(H * per, r0 + sh.group_rows);
  const int n = a.rope.turns ? a.rope.rotary_dim : 0;
  for (int b = blockIdx.z; b < a.c.batch; b += gridDim.z) {
    if (t < a.T) {
      const int pos = a.pos[b * a.pos_stride + t];
      for (int i = lane; i < sh.items; i += sh.lanes) {
        const I item(i, n);
        float c[I::kPairs], s[I::kPairs];
        item.angles(a.rope, pos, 1.f, c, s);
        for (int r = r0 + (slot & (sh.row_slots - 1)); r < r1; r += kBatch * sh.row_slots) {
          T e[kBatch][I::kElems];
          T* dst[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int row = r + j * sh.row_slots;
            dst[j] = nullptr;
            if (row >= r1) continue;
            const int h = row / per, k = row - h * per;
            const T* src;
            if (k < G) {
              src = static_cast<const T*>(a.q.data) + b * a.q.stride_b + t * a.q.stride_t +
                    (long long)(h * G + k) * a.q.stride_h;
              dst[j] = static_cast<T*>(a.q_out) +
                       (((long long)b * a.T + t) * H * G + h * G + k) * kHeadDim;
            } else {
              const long long unit = (long long)b * H + h;
              const int len = a.c.lens[unit];
              const bool live = len >= 0 && len <= cap;
              const int at = live ? len : len < 0 ? 0 : cap;
              const bool room = at + (long long)a.T <= cap;
              if (k == G && i == 0 && t == 0) {
                if (!live) record_status(a.status, RI_ERR_INVALID_ARG);
                if (!room) record_status(a.status, RI_ERR_CAPACITY);
              }
              if (!room) continue;
              const ri_heads& x = k == G ? a.k : a.v;
              src = static_cast<const T*>(x.data) + b * x.stride_b + t * x.stride_t +
                    h * x.stride_h;
              const long long to = unit * cap + at + t;
              dst[j] = static_cast<T*>(k == G ? a.c.K : a.c.V) + to * kHeadDim;
              if (k == G && i == 0) {
                a.c.pos[to] = pos;
                a.c.weight[to] = 0.f;
              }
            }
            item.load(src, e[j]);
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (dst[j]) {
              const int row = r + j * sh.row_slots;
              if (row % per != per - 1) item.turn(e[j], c, s);  // not the value
              item.store(dst[j], e[j]);
            }
        }
      }
    }
    if (advance) {
      // a unit's key and value lie in one block: with one token (or lengths
      // that go elsewhere) this block is the last to need its length
      __syncthreads();
      for (int h = r0 / per + threadIdx.x; h < r1 / per; h += kThreads)
        if (blockIdx.x == 0) {
          const int u = b * H + h, len = min(max(a.c.lens[u], 0), cap);
          a.lens_out[u] = len + (long long)a.T <= cap ? len + a.T : len;
        }
    }
  }
}

// Advances the lengths in place once every token of append_kernel is stored.
__global__ void advance_kernel(int32_t* lens, int units, int cap, int T) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= units) return;
  const int len = min(max(lens[u], 0), cap);
  lens[u] = len + (long long)T <= cap ? len + T : len;
}

template <int VEC, bool INTER>
cudaError_t append_typed(const AppendTokensArgs& a, cudaStream_t s) {
  using I = Item<__nv_bfloat16, VEC, INTER>;
  const int n = a.rope.turns ? a.rope.rotary_dim : 0;
  const int H = a.c.num_kv_heads, per = (a.q.data ? a.c.group_size : 0) + 2;
  const Shape sh = shape_of(I::count(n, kHeadDim), a.T, a.c.batch, H, per);
  dim3 grid = grid_of(sh, a.T, a.c.batch, H * per);
  if (grid.z > kMaxGridDim) grid.z = kMaxGridDim;
  // several tokens in place: other blocks may still read a length, so a second
  // launch advances them
  const bool later = a.lens_out == a.c.lens && a.T > 1;
  append_kernel<VEC, INTER><<<grid, kThreads, 0, s>>>(a, sh, !later);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !later) return e;
  const int units = a.c.batch * H;
  advance_kernel<<<(units + 255) / 256, 256, 0, s>>>(a.c.lens, units, a.c.capacity, a.T);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t s) {
  switch (dtype) {
    case RI_BF16: return rotary_of<__nv_bfloat16>(a, s);
    case RI_FP16: return rotary_of<__half>(a, s);
    default: return rotary_of<float>(a, s);
  }
}

cudaError_t launch_token_append(const AppendTokensArgs& a, cudaStream_t s) {
  const int n = a.rope.turns ? a.rope.rotary_dim : 0;
  const bool inter = n > 0 && a.rope.interleaved;
  const bool vec = (inter ? n : n / 2) % 8 == 0 && n % 8 == 0;
  if (vec) return inter ? append_typed<8, true>(a, s) : append_typed<8, false>(a, s);
  return inter ? append_typed<1, true>(a, s) : append_typed<1, false>(a, s);
}

}  // namespace ri
