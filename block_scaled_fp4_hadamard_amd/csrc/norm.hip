// Layer norm of a matrix's rows, its RMS form, and their backward pass.
//
//   forward    mean = sum x / n, d = x - mean, rstd = (sum d^2 / n + eps)^-1/2,
//              y = d * rstd * w + b                  (RMS: mean = 0, no b)
//   backward   h = (x - mean) * rstd, g = dy * w,
//              dx = rstd * (g - sum(g) / n - h * sum(g h) / n)
//                                                    (RMS: without sum(g) / n)
//              dw = sum over rows of dy * h, db = sum over rows of dy
//
// Everything between the loads and the stores is float32; y and dx are rounded
// once.  The variance is the mean square of d, formed after the mean, from the
// row that is still in registers: no difference of large numbers.  Every sum
// has an order that the sizes alone decide.
//
// Memory-bound: x read and y written once; x and dy read and dx written once.
// A row belongs to G lanes (16, 64: part of a wave or a wave, no LDS; 256,
// 1024: a workgroup or a part of one), N vectors of 16 bytes a lane, so that it
// stays in registers between its sums and its output.  From HBM, launch
// included: forward 8192 x 4096 bf16 25 to 27 us (5.0 to 5.3 TB/s), its RMS form 23
// (5.8), 262144 x 128 21 (6.4), 2001 x 5003 float32 22 (3.6: short of waves);
// backward 8192 x 4096 46 us (4.4), of which the sums' second launch is 5, 4001 x
// 14335 float32 160 (4.3).  A wave for a row of 4096 took 59 us forward: too few
// loads in flight.
//
// 1024 lanes leave 128 registers each, and some kernels of two or four vectors a
// lane do not fit them: the RMS backward of 2049 to 4096 bf16 columns spills 67
// (8192 x 4096: 81 us, 2.5 TB/s), of 129 to 256 and 513 to 1024 columns 115 and 70;
// the forward of 16385 to 32768 bf16 columns 94 (2048 x 20001: 84 us, 2.0 TB/s).
// Rows wider than registers are read again for every sum: 1024 x 33001 bf16 42 us
// forward (3.2 TB/s), 2048 x 20001 backward 126 (1.9).
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "norm_kernels.h"

namespace mx {

namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes wherever a row may start: one access, whatever the row pitch and the width
typedef u32x4 u32x4_any __attribute__((aligned(2)));

struct Bf16 {
  uint16_t bits;
};
template <typename T>
constexpr int kPer = 16 / (int)sizeof(T);          // elements of a 16-byte vector

__device__ __forceinline__ float value(Bf16 v) { return __uint_as_float((uint32_t)v.bits << 16); }
__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}

// The vector's elements at p[at ..]; zeros at and past `cols`.
template <typename T>
__device__ __forceinline__ u32x4 load_raw(const T* p, int at, int cols) {
  if (at + kPer<T> <= cols) return *(const u32x4_any*)(p + at);
  u32x4 r = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < kPer<T>; ++e)
    if (at + e < cols) {
      if constexpr (sizeof(T) == 2) r[e >> 1] |= (uint32_t)p[at + e].bits << (16 * (e & 1));
      else r[e] = __float_as_uint(p[at + e]);
    }
  return r;
}

template <typename T>
__device__ __forceinline__ float part(const u32x4& r, int e) {
  if constexpr (sizeof(T) == 2)
    return __uint_as_float((e & 1) ? r[e >> 1] & 0xFFFF0000u : r[e >> 1] << 16);
  else
    return __uint_as_float(r[e]);
}

// STREAM: past the caches, which the next rows' loads then have for themselves.  Forward: 8192 x 4096 27 us for 28,
// 262144 x 128 21 for 23; backward, long rows: 160 for 163; but 8192 x 4096 49 for 46, where it is left out.
template <bool STREAM, typename T>
__device__ __forceinline__ void store(T* p, int at, int cols, const float (&v)[kPer<T>]) {
  u32x4 r;
  if constexpr (sizeof(T) == 2) r = u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                          pack_bf16(v[6], v[7])};
  else r = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  if (at + kPer<T> <= cols) {
    if constexpr (STREAM) __builtin_nontemporal_store(r, (u32x4_any*)(p + at));
    else *(u32x4_any*)(p + at) = r;
    return;
  }
#pragma unroll
  for (int e = 0; e < kPer<T>; ++e)
    if (at + e < cols) {
      if constexpr (sizeof(T) == 2) p[at + e].bits = (uint16_t)(r[e >> 1] >> (16 * (e & 1)));
      else p[at + e] = v[e];
    }
}

// kPer<T> weights from `at` on (which may be of the other type): ones where there are none, zeros past `cols`.
template <int E>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, float none, int at, int cols, float (&o)[E]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = none;
  } else if (bf16) {
    const Bf16* p = (const Bf16*)w;
    if constexpr (E == 8) {
      const u32x4 r = load_raw(p, at, cols);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = part<Bf16>(r, e);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = at + e < cols ? value(p[at + e]) : 0.0f;
    }
  } else {
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
      const u32x4 r = load_raw((const float*)w, at + 4 * q, cols);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[4 * q + e] = part<float>(r, e);
    }
  }
}

// a pointer that is the same in all lanes of a wave
template <typename T>
__device__ __forceinline__ T* uniform(T* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (T*)(((uint64_t)hi << 32) | lo);
}
// row `row` of a matrix, uniform where a wave has one row (G lanes a row)
template <int G, typename T>
__device__ __forceinline__ T* row_of(T* p, int64_t row, int64_t ld) {
  if constexpr (G >= 64) return uniform(p + row * ld);
  else return p + row * ld;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float swap_add16(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float swap_add32(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
// the sum over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float sum16(float v) {
  v += dpp<0xB1>(v);     // l ^ 1
  v += dpp<0x4E>(v);     // l ^ 2
  v += dpp<0x141>(v);    // 7 - l within 8
  v += dpp<0x140>(v);    // 15 - l within 16
  return v;
}
__device__ __forceinline__ float sum64(float v) { return swap_add32(swap_add16(sum16(v))); }

// The sum over the G lanes of a row.  G > 64: `red` holds one float a wave, and a barrier parts its write from its
// read; whoever calls twice uses two arrays in turn.
template <int G>
__device__ __forceinline__ float row_sum(float v, float* red, int wave, int first) {
  if constexpr (G == 16) {
    return sum16(v);
  } else {
    v = sum64(v);
    if constexpr (G > 64) {
      if ((threadIdx.x & 63) == 0) red[wave] = v;
      __syncthreads();
      v = red[first];
#pragma unroll
      for (int i = 1; i < G / 64; ++i) v += red[first + i];
    }
    return v;
  }
}

constexpr unsigned kGrid = 256 * 8;       // workgroups of 256 lanes that are resident together

template <typename T, int KIND, int G, int N>
__global__ void __launch_bounds__(G < 256 ? 256 : G) norm_kernel(const NormParams p, const bool wbf) {
  constexpr int E = kPer<T>, kThreads = G < 256 ? 256 : G, kRows = kThreads / G;
  __shared__ float red[2][kThreads / 64];
  const int lane = threadIdx.x % G, wave = threadIdx.x / 64, cols = (int)p.cols;
  const float n = (float)cols;       // divided by, not multiplied with its inverse: the mean of equal values is the value
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G; row < p.rows; row += (int64_t)gridDim.x * kRows) {
    const T* x = (const T*)p.x + row * p.ld_x;
    u32x4 raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = load_raw(x, (i * G + lane) * E, cols);
    float mean = 0.0f;
    if constexpr (KIND == MX_NORM_LAYER) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) s += part<T>(raw[i], e);
      mean = row_sum<G>(s, red[0], wave, 0) / n;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = part<T>(raw[i], e) - mean;
        // a place past the row holds zero, and its difference to the mean must not count
        if (KIND == MX_NORM_RMS || (i * G + lane) * E + e < cols) s = fmaf(d, d, s);
      }
    // RMS: one sum a row, in two arrays in turn
    const float var = row_sum<G>(s, red[KIND == MX_NORM_LAYER ? 1 : (row / kRows / gridDim.x) & 1], wave, 0) / n;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (lane == 0) {
      if (KIND == MX_NORM_LAYER && p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    T* y = (T*)p.y + row * p.ld_y;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = (i * G + lane) * E;
      if (at >= cols) continue;
      float w[E], b[E], o[E];
      load_weight<E>(p.weight, wbf, 1.0f, at, cols, w);
      if constexpr (KIND == MX_NORM_LAYER) load_weight<E>(p.bias, wbf, 0.0f, at, cols, b);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float h = (part<T>(raw[i], e) - mean) * rstd;
        o[e] = KIND == MX_NORM_LAYER ? fmaf(h, w[e], b[e]) : h * w[e];
      }
      store<true>(y, at, cols, o);
    }
  }
}

// Rows wider than the registers of a workgroup: each pass reads the row again.
template <typename T, int KIND>
__global__ void __launch_bounds__(1024) norm_wide(const NormParams p, const bool wbf) {
  constexpr int E = kPer<T>;
  __shared__ float red[2][16];
  const int wave = threadIdx.x / 64;
  const int cols = (int)p.cols, step = 1024 * E, from = threadIdx.x * E;
  const float n = (float)cols;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = (const T*)p.x + row * p.ld_x;
    float mean = 0.0f;
    if constexpr (KIND == MX_NORM_LAYER) {
      float s = 0.0f;
      for (int at = from; at < cols; at += step) {
        const u32x4 r = load_raw(x, at, cols);
#pragma unroll
        for (int e = 0; e < E; ++e) s += part<T>(r, e);
      }
      mean = row_sum<1024>(s, red[turn ^= 1], wave, 0) / n;
    }
    float s = 0.0f;
    for (int at = from; at < cols; at += step) {
      const u32x4 r = load_raw(x, at, cols);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = part<T>(r, e) - mean;
        if (at + e < cols) s = fmaf(d, d, s);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<1024>(s, red[turn ^= 1], wave, 0) / n + p.eps);
    if (threadIdx.x == 0) {
      if (KIND == MX_NORM_LAYER && p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    T* y = (T*)p.y + row * p.ld_y;
    for (int at = from; at < cols; at += step) {
      const u32x4 r = load_raw(x, at, cols);
      float w[E], b[E], o[E];
      load_weight<E>(p.weight, wbf, 1.0f, at, cols, w);
      if constexpr (KIND == MX_NORM_LAYER) load_weight<E>(p.bias, wbf, 0.0f, at, cols, b);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float h = (part<T>(r, e) - mean) * rstd;
        o[e] = KIND == MX_NORM_LAYER ? fmaf(h, w[e], b[e]) : h * w[e];
      }
      store<true>(y, at, cols, o);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  One workgroup of 1024 lanes a CU at most (few rows: of 256), of
// kRows = THREADS / G rows at a time; a lane keeps its columns' sums of dy and dy * h over all its rows
// in registers.  At the end the workgroup's rows are added in LDS, one after
// another, and its sums go to the workspace; norm_grad_sum adds the workgroups'
// in order.
constexpr int kGradGrid = 256;
constexpr int kLong = 19456;             // columns whose two sums fit into LDS
constexpr int kLongLanes = 512;          // 1024 leave 128 registers a lane, too few for two rows

template <typename T, int KIND, int G, int N, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_grad_kernel(const NormGradParams p, const bool wbf, float* parts) {
  constexpr int E = kPer<T>, kRows = THREADS / G, kCols = G * N * E;
  __shared__ float red[2][2][THREADS / 64];
  __shared__ float sum[kRows > 1 ? 2 * kCols : 1];
  const int lane = threadIdx.x % G, mine = threadIdx.x / G, wave = threadIdx.x / 64, cols = (int)p.cols;
  const int first = mine * (G / 64);              // the row's first wave (G > 64)
  const float n = (float)cols;
  float dw[N][E], db[N][E];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = db[i][e] = 0.0f;
  // the lane's weights: a load of theirs in the loop would wait for the row asked for before it
  float w[N][E];
#pragma unroll
  for (int i = 0; i < N; ++i) load_weight<E>(p.weight, wbf, 1.0f, (i * G + lane) * E, cols, w[i]);
  int turn = 0;
  // a row, asked for while the one before it is worked on
  struct Row {
    u32x4 x[N], dy[N];
    float mean, rstd;
  };
  auto ask = [&](int64_t row, Row& r) {
    const bool real = row < p.rows;
    const T* x = row_of<G>((const T*)p.x, row, p.ld_x);
    const T* dy = row_of<G>((const T*)p.dy, row, p.ld_dy);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r.x[i] = load_raw(x, (i * G + lane) * E, real ? cols : 0);
      r.dy[i] = load_raw(dy, (i * G + lane) * E, real ? cols : 0);
    }
    r.mean = KIND == MX_NORM_LAYER && real ? p.mean[row] : 0.0f;
    r.rstd = real ? p.rstd[row] : 0.0f;
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  Row ahead;
  ask((int64_t)blockIdx.x * kRows + mine, ahead);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < p.rows; base += step, turn ^= 1) {
    const int64_t row = base + mine;
    const bool real = row < p.rows;
    const Row now = ahead;
    ask(row + step, ahead);
    const auto &rx = now.x, &ry = now.dy;
    const float mean = now.mean, rstd = now.rstd;
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        // past the row's end dy is zero
        const float h = (part<T>(rx[i], e) - mean) * rstd, d = part<T>(ry[i], e), g = d * w[i][e];
        c1 += g;
        c2 = fmaf(g, h, c2);
        dw[i][e] = fmaf(d, h, dw[i][e]);
        db[i][e] += d;
      }
    }
    if constexpr (G == 16) {
      c1 = sum16(c1);
      c2 = sum16(c2);
    } else {
      c1 = sum64(c1);
      c2 = sum64(c2);
      if constexpr (G > 64) {
        if ((threadIdx.x & 63) == 0) {
          red[turn][0][wave] = c1;
          red[turn][1][wave] = c2;
        }
        __syncthreads();
        c1 = red[turn][0][first];
        c2 = red[turn][1][first];
#pragma unroll
        for (int i = 1; i < G / 64; ++i) {
          c1 += red[turn][0][first + i];
          c2 += red[turn][1][first + i];
        }
      }
    }
    c1 = KIND == MX_NORM_LAYER ? c1 / n : 0.0f;
    c2 /= n;
    if (!real) continue;
    T* dx = row_of<G>((T*)p.dx, row, p.ld_dx);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = (i * G + lane) * E;
      if (at >= cols) continue;
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float h = (part<T>(rx[i], e) - mean) * rstd;
        o[e] = (fmaf(part<T>(ry[i], e), w[i][e], -c1) - h * c2) * rstd;
      }
      store<false>(dx, at, cols, o);
    }
  }
  if (parts == nullptr) return;
  // parts: [workgroup][dw, db][cols]
  float* out = parts + (int64_t)blockIdx.x * 2 * p.cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = (i * G + lane) * E + e;
        if (at < cols) {
          out[at] = dw[i][e];
          out[cols + at] = db[i][e];
        }
      }
  } else {
    for (int r = 0; r < kRows; ++r) {
      if (mine == r) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int at = (i * G + lane) * E + e;
            sum[at] = (r ? sum[at] : 0.0f) + dw[i][e];
            sum[kCols + at] = (r ? sum[kCols + at] : 0.0f) + db[i][e];
          }
      }
      __syncthreads();
    }
    for (int at = threadIdx.x; at < cols; at += THREADS) {
      out[at] = sum[at];
      out[cols + at] = sum[kCols + at];
    }
  }
}

// Long rows: one workgroup of 512 lanes takes a row at a time, the next one asked for ahead; the columns' sums live in
// LDS, each lane adding to its own, so that registers hold the rows.
template <typename T, int KIND, int N>
__global__ void __launch_bounds__(kLongLanes) norm_grad_long(const NormGradParams p, const bool wbf, float* parts) {
  constexpr int E = kPer<T>;
  __shared__ float red[2][2][kLongLanes / 64];
  __shared__ __attribute__((aligned(16))) float sum[2][kLong];
  typedef float v4f __attribute__((ext_vector_type(4)));
  const int lane = threadIdx.x, wave = lane / 64, cols = (int)p.cols;
  const float n = (float)cols;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int q = 0; q < E; q += 4) {
      const int at = (i * kLongLanes + lane) * E + q;
      if (at < cols) *(v4f*)&sum[0][at] = *(v4f*)&sum[1][at] = v4f{0.f, 0.f, 0.f, 0.f};
    }
  float w[N][E];
#pragma unroll
  for (int i = 0; i < N; ++i) load_weight<E>(p.weight, wbf, 1.0f, (i * kLongLanes + lane) * E, cols, w[i]);
  struct Row {
    u32x4 x[N], dy[N];
    float mean, rstd;
  };
  auto ask = [&](int64_t row, Row& r) {
    const bool real = row < p.rows;
    const T* x = row_of<kLongLanes>((const T*)p.x, row, p.ld_x);
    const T* dy = row_of<kLongLanes>((const T*)p.dy, row, p.ld_dy);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r.x[i] = load_raw(x, (i * kLongLanes + lane) * E, real ? cols : 0);
      r.dy[i] = load_raw(dy, (i * kLongLanes + lane) * E, real ? cols : 0);
    }
    r.mean = KIND == MX_NORM_LAYER && real ? p.mean[row] : 0.0f;
    r.rstd = real ? p.rstd[row] : 0.0f;
  };
  Row ahead;
  ask(blockIdx.x, ahead);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const Row now = ahead;
    ask(row + gridDim.x, ahead);
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = (i * kLongLanes + lane) * E;
      if (at >= cols) continue;
#pragma unroll
      for (int q = 0; q < E; q += 4) {
        v4f a = *(const v4f*)&sum[0][at + q], b = *(const v4f*)&sum[1][at + q];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float h = (part<T>(now.x[i], q + e) - now.mean) * now.rstd, d = part<T>(now.dy[i], q + e), g = d * w[i][q + e];
          c1 += g;
          c2 = fmaf(g, h, c2);
          a[e] = fmaf(d, h, a[e]);
          b[e] += d;
        }
        *(v4f*)&sum[0][at + q] = a;
        *(v4f*)&sum[1][at + q] = b;
      }
    }
    c1 = row_sum<kLongLanes>(c1, red[turn][0], wave, 0);
    c2 = row_sum<kLongLanes>(c2, red[turn][1], wave, 0) / n;
    c1 = KIND == MX_NORM_LAYER ? c1 / n : 0.0f;
    T* dx = row_of<kLongLanes>((T*)p.dx, row, p.ld_dx);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = (i * kLongLanes + lane) * E;
      if (at >= cols) continue;
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float h = (part<T>(now.x[i], e) - now.mean) * now.rstd;
        o[e] = (fmaf(part<T>(now.dy[i], e), w[i][e], -c1) - h * c2) * now.rstd;
      }
      store<true>(dx, at, cols, o);
    }
  }
  if (parts == nullptr) return;
  float* out = parts + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int at = (i * kLongLanes + lane) * E + e;
      if (at < cols) {
        out[at] = sum[0][at];
        out[cols + at] = sum[1][at];
      }
    }
}

// Wider rows: the two sums of every row first, then columns in strips, each lane one column over a run of rows.
template <typename T, int KIND>
__global__ void __launch_bounds__(1024) norm_grad_wide_rows(const NormGradParams p, const bool wbf, float* c) {
  constexpr int E = kPer<T>;
  __shared__ float red[2][2][16];
  const int wave = threadIdx.x / 64, cols = (int)p.cols;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const T* x = (const T*)p.x + row * p.ld_x;
    const T* dy = (const T*)p.dy + row * p.ld_dy;
    const float mean = KIND == MX_NORM_LAYER ? p.mean[row] : 0.0f, rstd = p.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int at = threadIdx.x * E; at < cols; at += 1024 * E) {
      const u32x4 rx = load_raw(x, at, cols), ry = load_raw(dy, at, cols);
      float w[E];
      load_weight<E>(p.weight, wbf, 1.0f, at, cols, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float g = part<T>(ry, e) * w[e];
        c1 += g;
        c2 = fmaf(g, (part<T>(rx, e) - mean) * rstd, c2);
      }
    }
    c1 = row_sum<1024>(c1, red[turn][0], wave, 0);
    c2 = row_sum<1024>(c2, red[turn][1], wave, 0);
    if (threadIdx.x == 0) {
      c[2 * row] = KIND == MX_NORM_LAYER ? c1 / (float)cols : 0.0f;
      c[2 * row + 1] = c2 / (float)cols;
    }
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(256) norm_grad_wide_cols(const NormGradParams p, const bool wbf, const float* c,
                                                           int64_t run, float* parts) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= p.cols) return;
  const float w = p.weight == nullptr ? 1.0f : wbf ? value(((const Bf16*)p.weight)[at]) : ((const float*)p.weight)[at];
  const int64_t from = blockIdx.y * run, to = from + run < p.rows ? from + run : p.rows;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = from; row < to; ++row) {
    const float mean = KIND == MX_NORM_LAYER ? p.mean[row] : 0.0f, rstd = p.rstd[row];
    const float d = value(((const T*)p.dy)[row * p.ld_dy + at]);
    const float h = (value(((const T*)p.x)[row * p.ld_x + at]) - mean) * rstd;
    dw = fmaf(d, h, dw);
    db += d;
    const float o = (fmaf(d, w, -c[2 * row]) - h * c[2 * row + 1]) * rstd;
    if constexpr (sizeof(T) == 2) ((T*)p.dx)[row * p.ld_dx + at].bits = (uint16_t)pack_bf16(o, 0.0f);
    else ((T*)p.dx)[row * p.ld_dx + at] = o;
  }
  if (parts != nullptr) {
    parts[(int64_t)blockIdx.y * 2 * p.cols + at] = dw;
    parts[((int64_t)blockIdx.y * 2 + 1) * p.cols + at] = db;
  }
}

// Workgroups of norm_grad_sum at most: a launch holds less than 2^32 lanes (one of more wraps around, without an error).
constexpr int64_t kSumGrid = int64_t(1) << 21;

// dweight and dbias from the workgroups' sums: 64 columns a workgroup at a time, its 16 waves a run of the sums each.
__global__ void __launch_bounds__(1024) norm_grad_sum(const float* parts, int count, int64_t cols, float* dweight,
                                                      float* dbias) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* out = blockIdx.y ? dbias : dweight;
  if (out == nullptr) return;
  const int run = (count + 15) / 16, to = min(count, (wave + 1) * run);
  for (int64_t base = (int64_t)blockIdx.x * 64; base < cols; base += (int64_t)gridDim.x * 64) {
    const int64_t at = base + lane;
    const float* x = parts + (int64_t)blockIdx.y * cols + at;
    float s = 0.0f;
    if (at < cols) {
#pragma unroll 4
      for (int i = wave * run; i < to; ++i) s += x[(int64_t)i * 2 * cols];
    }
    if (base >= (int64_t)gridDim.x * 64) __syncthreads();        // the columns before have been added
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && at < cols) {
#pragma unroll
      for (int i = 1; i < 16; ++i) s += red[i][lane];
      out[at] = s;
    }
  }
}

struct Shape {
  int lanes, vectors;            // G and N; lanes 0: rows wider than registers
  int threads;                   // of a workgroup
};

// The lanes of a row, for `cols` elements of e a vector.  A wave for 129 to 192 vectors, which leave half of 256 lanes idle
// (59898 x 516 float32: 42 us forward and 78 backward for 61 and 112).
Shape forward_shape(int64_t cols, int e) {
  const int64_t v = (cols + e - 1) / e;
  if (v <= 16) return {16, 1, 256};
  if (v <= 32) return {16, 2, 256};
  if (v <= 64) return {64, 1, 256};
  if (v <= 128) return {64, 2, 256};
  if (v <= 192) return {64, 3, 256};
  if (v <= 256) return {256, 1, 256};
  if (v <= 512) return {256, 2, 256};
  if (v <= 1024) return {256, 4, 256};
  if (v <= 1536) return {256, 6, 256};
  if (v <= 2048) return {256, 8, 256};
  if (v <= 4096) return {1024, 4, 1024};
  return {0, 0, 1024};
}

// Backward.  Few rows take small workgroups, so that more CUs share them (33 x 4096 RMS: the kernel 9 us for 19.6); many
// take large ones, of which each leaves its sums once.
Shape grad_shape(int64_t cols, int64_t rows, int e) {
  const int64_t v = (cols + e - 1) / e;
  Shape s = {0, 0, 1024};
  if (v <= 32) s = {16, v <= 16 ? 1 : 2, 1024};
  else if (v <= 128) s = {64, v <= 64 ? 1 : 2, 1024};
  else if (v <= 192 && e == 4) s = {64, 3, 1024};       // bf16: its 24 columns a lane leave too few registers
  else if (v <= 512) s = {256, v <= 256 ? 1 : 2, 1024};
  else if (v <= 1024) return {1024, 1, 1024};
  else if (v <= 2048 && e == 4) return {1024, 2, 1024};
  else if (cols <= kLong) return {kLongLanes, (int)((v + 2 * kLongLanes - 1) / (2 * kLongLanes)) * 2, kLongLanes};
  if (s.lanes != 0 && rows <= kGradGrid * (256 / s.lanes)) s.threads = 256;
  return s;
}

constexpr int64_t kWideRuns = 256;                // runs of rows of the kernels for the widest rows at most

// workgroups whose sums the workspace holds
int64_t grad_parts(int64_t rows, const Shape& s) {
  if (s.lanes == 0) return rows < kWideRuns ? rows : kWideRuns;
  const int64_t each = s.threads / s.lanes, need = (rows + each - 1) / each;
  return need < kGradGrid ? need : kGradGrid;
}

template <typename T, int KIND>
hipError_t forward(const NormParams& p, bool wbf, hipStream_t st) {
  const Shape s = forward_shape(p.cols, kPer<T>);
  const int64_t each = s.lanes == 0 || s.lanes >= 256 ? 1 : 256 / s.lanes, need = (p.rows + each - 1) / each;
  const int64_t most = s.lanes == 0 || s.lanes == 1024 ? kGrid / 4 : kGrid;
  const dim3 g((unsigned)(need < most ? need : most));
#define MX_NORM_CASE(LANES, VECTORS)                                                                            \
  if (s.lanes == LANES && s.vectors == VECTORS) {                                                               \
    hipLaunchKernelGGL((norm_kernel<T, KIND, LANES, VECTORS>), g, dim3(LANES < 256 ? 256 : LANES), 0, st, p, wbf); \
    return hipGetLastError();                                                                                   \
  }
  MX_NORM_CASE(16, 1) MX_NORM_CASE(16, 2) MX_NORM_CASE(64, 1) MX_NORM_CASE(64, 2) MX_NORM_CASE(64, 3) MX_NORM_CASE(256, 1)
  MX_NORM_CASE(256, 2) MX_NORM_CASE(256, 4) MX_NORM_CASE(256, 6) MX_NORM_CASE(256, 8) MX_NORM_CASE(1024, 4)
#undef MX_NORM_CASE
  hipLaunchKernelGGL((norm_wide<T, KIND>), g, dim3(1024), 0, st, p, wbf);
  return hipGetLastError();
}

template <typename T, int KIND>
hipError_t backward(const NormGradParams& p, bool wbf, float* ws, hipStream_t st) {
  const bool sums = p.dweight != nullptr || p.dbias != nullptr;
  const Shape s = grad_shape(p.cols, p.rows, kPer<T>);
  const int64_t count = grad_parts(p.rows, s);       // 0 without rows: the sums are zeros
  float* parts = sums ? ws : nullptr;
  const dim3 g((unsigned)count);
#define MX_NORM_CASE(LANES, VECTORS, THREADS)                                                                         \
  if (count > 0 && s.lanes == LANES && s.vectors == VECTORS && s.threads == THREADS)                                  \
    hipLaunchKernelGGL((norm_grad_kernel<T, KIND, LANES, VECTORS, THREADS>), g, dim3(THREADS), 0, st, p, wbf, parts);
  MX_NORM_CASE(16, 1, 256) MX_NORM_CASE(16, 2, 256) MX_NORM_CASE(64, 1, 256) MX_NORM_CASE(64, 2, 256)
  MX_NORM_CASE(256, 1, 256) MX_NORM_CASE(256, 2, 256) MX_NORM_CASE(16, 1, 1024) MX_NORM_CASE(16, 2, 1024)
  MX_NORM_CASE(64, 1, 1024) MX_NORM_CASE(64, 2, 1024) MX_NORM_CASE(256, 1, 1024) MX_NORM_CASE(256, 2, 1024)
  MX_NORM_CASE(1024, 1, 1024)
  if constexpr (sizeof(T) == 4) {
    MX_NORM_CASE(64, 3, 256) MX_NORM_CASE(64, 3, 1024) MX_NORM_CASE(1024, 2, 1024)
  }
#undef MX_NORM_CASE
#define MX_NORM_CASE(VECTORS)                                                                                      \
  if (count > 0 && s.lanes == kLongLanes && s.vectors == VECTORS)                                                  \
    hipLaunchKernelGGL((norm_grad_long<T, KIND, VECTORS>), g, dim3(kLongLanes), 0, st, p, wbf, parts);
  MX_NORM_CASE(6)
  if constexpr (sizeof(T) == 4) {
    MX_NORM_CASE(8) MX_NORM_CASE(10)
  } else {
    MX_NORM_CASE(4)
  }
#undef MX_NORM_CASE
  if (count > 0 && s.lanes == 0) {
    float* c = sums ? ws + 2 * count * p.cols : ws;
    hipLaunchKernelGGL((norm_grad_wide_rows<T, KIND>), dim3((unsigned)(p.rows < 512 ? p.rows : 512)), dim3(1024), 0, st,
                       p, wbf, c);
    const int64_t run = (p.rows + count - 1) / count;
    hipLaunchKernelGGL((norm_grad_wide_cols<T, KIND>), dim3((unsigned)((p.cols + 255) / 256), (unsigned)count),
                       dim3(256), 0, st, p, wbf, c, run, parts);
  }
  if (sums) {
    const int64_t need = (p.cols + 63) / 64;
    hipLaunchKernelGGL(norm_grad_sum, dim3((unsigned)(need < kSumGrid ? need : kSumGrid), 2), dim3(1024), 0, st, parts,
                       (int)count, p.cols, p.dweight, p.dbias);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormParams& p, int type, int weight_type, int kind, hipStream_t s) {
  const bool wbf = weight_type == MX_OUT_BF16;
  if (type == MX_OUT_BF16)
    return kind == MX_NORM_LAYER ? forward<Bf16, MX_NORM_LAYER>(p, wbf, s) : forward<Bf16, MX_NORM_RMS>(p, wbf, s);
  return kind == MX_NORM_LAYER ? forward<float, MX_NORM_LAYER>(p, wbf, s) : forward<float, MX_NORM_RMS>(p, wbf, s);
}

int64_t norm_grad_workspace(int64_t rows, int64_t cols, int type, bool sums) {
  const Shape s = grad_shape(cols, rows, type == MX_OUT_BF16 ? 8 : 4);
  return 4 * ((sums ? 2 * grad_parts(rows, s) * cols : 0) + (s.lanes == 0 ? 2 * rows : 0));
}

hipError_t launch_norm_grad(const NormGradParams& p, int type, int weight_type, int kind, float* workspace,
                            hipStream_t s) {
  const bool wbf = weight_type == MX_OUT_BF16;
  if (type == MX_OUT_BF16)
    return kind == MX_NORM_LAYER ? backward<Bf16, MX_NORM_LAYER>(p, wbf, workspace, s)
                                 : backward<Bf16, MX_NORM_RMS>(p, wbf, workspace, s);
  return kind == MX_NORM_LAYER ? backward<float, MX_NORM_LAYER>(p, wbf, workspace, s)
                               : backward<float, MX_NORM_RMS>(p, wbf, workspace, s);
}

}  // namespace mx
