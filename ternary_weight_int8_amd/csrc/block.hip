// block.hip -- gfx950 kernels of the operators around the ternary product,
// part of libternary_gemm.so (ABI and formulas in include/ternary_gemm.h):
//   ternary_rmsnorm_quantize    residual addition, RMS norm, int8 rows
//   ternary_rmsnorm_backward    its gradients
//   ternary_epilogue_backward   the backward of bias and activation, with the
//                               int8 rows that the dX products take
//   ternary_layernorm_quantize  the same with a layer norm
//   ternary_layernorm_backward  its gradients
//   ternary_gated_backward      the backward of the gated product, with int8 rows
//   ternary_clip_grad_norm      the global norm of many gradients, and the
//                               scaling by it
// (the product's own epilogue is part of the product's kernels).  All of them
// only read and write their operands: HBM bounds them (a copy of 512 MiB
// reaches 5.3 TB/s, read and written, on an MI355X), and the smallest are bound
// by their launches: 2.5 us for a row of 1280, and more than that on the host.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>
#include <vector>

#include "checks.h"
#include "ternary_gemm.h"

// Sums and products are fused only where fma is written, so that a kernel
// rounds alike whatever its widths are compiled for.  The kernels of other row
// lengths and counts add a row, and the columns, up in another order, and the
// looped backward of the norm divides where the register one multiplies by 1 / C:
// the same call repeats its bits, a row among more or fewer rows may not.
#pragma clang fp contract(off)

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kNT = 256;   // threads per workgroup
constexpr int64_t kCUs = 256;                        // compute units of an MI355X
constexpr int64_t kNormWaves = 32, kBwdWaves = 16;   // waves a CU of the row kernels' grids, at most

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
template <class T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// |v| as an integer: the order of the magnitudes, with a NaN above them all
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ int8_t quant1(float y, float s) {
  if (!(s > 0.f && s < __builtin_inff())) return 0;
  const float r = rintf(__fdiv_rn(y, s));
  return (int8_t)(r > 127.f ? 127.f : (r < -127.f ? -127.f : r));
}

// sum and maximum over the workgroup's four waves; `part` has 4 entries and
// is free again when every thread has passed the next barrier
template <class F>
__device__ __forceinline__ F block_sum(F v, F *part) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}
__device__ __forceinline__ float block_max(uint32_t v, uint32_t *part) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = __shfl_xor(v, off);
    v = o > v ? o : v;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t m = part[0];
#pragma unroll
  for (int i = 1; i < kNT / 64; ++i) m = part[i] > m ? part[i] : m;
  return __uint_as_float(m);
}

// ---------------------------------------------------------------------------
// Rows held in registers.  The three row operators need a sum or a maximum
// over a row before they can write it, so a row is read once into registers,
// reduced, and written from them: HBM sees every input and output once.
//
// A wave (W = 1, several rows a workgroup) or a workgroup of 1 to 16 waves (W = 0)
// takes a row, each of its NT threads holding V units of 16 bytes (U elements):
// unit j of thread t is unit t + NT j of the row, so a wave's loads cover whole
// lines.  Rows need not be whole units or aligned:
// loads and stores are element-aligned vectors (gfx950 serves them), and the
// row's last unit is the last U elements, of which the first `dup` also
// belong to the unit before; both threads compute and store the same values
// for them, and only the row's sums and the column sums leave them out.  (A
// store never precedes the reduction that every load of the row precedes, so
// this holds for in-place outputs too.)  Rows of fewer than U elements, and
// rows that no W, V holds, take the looped kernels further down.
// ---------------------------------------------------------------------------
template <class T>
constexpr int kU = 16 / (int)sizeof(T);

template <class T>
struct Raw;
template <>
struct Raw<float> {
  typedef float V __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Raw<uint16_t> {
  typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
};
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32u __attribute__((aligned(1)));

__device__ __forceinline__ void unpack(const Raw<float>::V &r, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = r[i];
}
__device__ __forceinline__ void unpack(const Raw<uint16_t>::V &r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r[i] << 16);
    v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ Raw<float>::V pack(const float (&v)[4]) { return {v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ Raw<uint16_t>::V pack(const float (&v)[8]) {
  Raw<uint16_t>::V r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){v[2 * i], v[2 * i + 1]}, bf16x2));
  return r;
}

// Workgroup barrier for LDS only (outstanding global loads and stores go on)
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Sum and maximum over a wave, the same in every lane: pairs, quads, eights
// and sixteens by data-parallel moves, then the four sixteens through scalar
// registers.  Every lane has to be active.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
__device__ __forceinline__ float lane_f(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kMirror>(__float_as_uint(v)));
  return (lane_f(v, 0) + lane_f(v, 16)) + (lane_f(v, 32) + lane_f(v, 48));
}
// the same in 64 bits
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32 | dpp<CTRL>((uint32_t)b));
}
__device__ __forceinline__ double lane_f(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(b >> 32), l), lo = __builtin_amdgcn_readlane((int)b, l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  return (lane_f(v, 0) + lane_f(v, 16)) + (lane_f(v, 32) + lane_f(v, 48));
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = umax(v, dpp<kXor1>(v));
  v = umax(v, dpp<kXor2>(v));
  v = umax(v, dpp<kHalfMirror>(v));
  v = umax(v, dpp<kMirror>(v));
  const uint32_t a = __builtin_amdgcn_readlane((int)v, 0), b = __builtin_amdgcn_readlane((int)v, 16);
  const uint32_t c = __builtin_amdgcn_readlane((int)v, 32), d = __builtin_amdgcn_readlane((int)v, 48);
  return umax(umax(a, b), umax(c, d));
}
// over a row's threads: a wave by itself, or the workgroup's waves through
// `part` (a word a wave), which every sixteen lanes then reduce.  One barrier:
// a caller alternates between two `part`s from row to row, and the barrier of
// the row between separates the reads of one from the next writes to it.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *part) {
  v = wave_sum(v);
  if constexpr (W == 0) {
    const int lane = threadIdx.x & 63, l = lane & 15;
    if (lane == 0) part[threadIdx.x >> 6] = v;
    lds_barrier();
    v = l < (int)(blockDim.x >> 6) ? part[l] : 0.f;
    v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kHalfMirror>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kMirror>(__float_as_uint(v)));
  }
  return v;
}
// the waves' sums in 64 bits, v the same in every lane of a wave
template <int W>
__device__ __forceinline__ double row_sum_waves(double v, double *part) {
  if constexpr (W == 0) {
    const int lane = threadIdx.x & 63, l = lane & 15;
    if (lane == 0) part[threadIdx.x >> 6] = v;
    lds_barrier();
    v = l < (int)(blockDim.x >> 6) ? part[l] : 0.;
    v += dpp<kXor1>(v);
    v += dpp<kXor2>(v);
    v += dpp<kHalfMirror>(v);
    v += dpp<kMirror>(v);
  }
  return v;
}
template <int W>
__device__ __forceinline__ float row_max(uint32_t v, uint32_t *part) {
  v = wave_max(v);
  if constexpr (W == 0) {
    const int lane = threadIdx.x & 63, l = lane & 15;
    if (lane == 0) part[threadIdx.x >> 6] = v;
    lds_barrier();
    v = l < (int)(blockDim.x >> 6) ? part[l] : 0u;
    v = umax(v, dpp<kXor1>(v));
    v = umax(v, dpp<kXor2>(v));
    v = umax(v, dpp<kHalfMirror>(v));
    v = umax(v, dpp<kMirror>(v));
  }
  return __uint_as_float(v);
}
constexpr int max_t(int W, int V) { return W && V > 1 ? 256 : 1024; }   // threads a workgroup, at most

// A thread's units of a row of C elements
template <class T, int W, int V>
struct Units {
  static constexpr int U = kU<T>;
  int off[V];    // first element of each unit
  int32_t dup;   // of the row's last unit: elements that the unit before has too
  int32_t last;  // j of the thread's unit if that is the row's last and dup > 0, else -1
  int32_t n;     // units of the thread
  __device__ __forceinline__ void init(int32_t C, int t) {
    const int32_t NT = W ? 64 : (int32_t)blockDim.x;
    const int32_t nu = (C + U - 1) / U;
    dup = nu * U - C;
    last = dup && (nu - 1) % NT == t ? (nu - 1) / NT : -1;
    n = t < nu ? (nu - 1 - t) / NT + 1 : 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int32_t o = (t + NT * j) * U;
      off[j] = o + U <= C ? o : C - U;
    }
  }
  __device__ __forceinline__ bool on(int j) const { return j < n; }
};

template <class T>
__device__ __forceinline__ typename Raw<T>::V load_raw(const T *p) {
  return *reinterpret_cast<const typename Raw<T>::V *>(p);
}
template <class T>
__device__ __forceinline__ void store_raw(T *p, const typename Raw<T>::V &v) {
  *reinterpret_cast<typename Raw<T>::V *>(p) = v;
}
template <int U>
__device__ __forceinline__ void load_f(const float *p, float (&v)[U]) {
#pragma unroll
  for (int i = 0; i < U; i += 4) {
    const Raw<float>::V r = load_raw(p + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[i + k] = r[k];
  }
}

// Int8 rows.  With s >= max|y| / 127 rounded and r = 1 / s rounded, the
// quotient y / s correctly rounded takes two corrections of y r (the second
// starts within one unit in the last place, from which one correction with a
// correctly rounded reciprocal is exact); 1.5 2^23 added to it leaves the
// nearest whole number, ties to even, in the low bits, and |y / s| <= 127.0001
// needs no clamp.  That is the IEEE division and rint of the row quantizer in
// six operations where s and r are well inside the normal range (fast_scale);
// elsewhere quant1 divides.
__device__ __forceinline__ bool fast_scale(float s) { return s >= 0x1p-100f && s <= 0x1p120f; }
template <int U>
__device__ __forceinline__ void store_q(int8_t *q, const float (&y)[U], float s, float r, bool fast) {
  uint32_t w[U / 4];
  if (fast) {
#pragma unroll
    for (int k = 0; k < U / 4; ++k) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = y[4 * k + i];
        float p = v * r;
        p = __builtin_fmaf(__builtin_fmaf(-p, s, v), r, p);
        p = __builtin_fmaf(__builtin_fmaf(-p, s, v), r, p);
        b[i] = __float_as_uint(p + 12582912.f);
      }
      // bytes 0 of b[0], b[1] and of b[2], b[3], then the two halves
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
      w[k] = lo | hi;
    }
  } else {
#pragma unroll
    for (int k = 0; k < U / 4; ++k) {
      w[k] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k] |= (uint32_t)(uint8_t)quant1(y[4 * k + i], s) << (8 * i);
    }
  }
  if constexpr (U == 8)
    *reinterpret_cast<u32x2u *>(q) = u32x2u{w[0], w[1]};
  else
    *reinterpret_cast<u32u *>(q) = w[0];
}

// ---------------------------------------------------------------------------
// Norm
// ---------------------------------------------------------------------------
struct NormArgs {
  const void *X, *res;
  const float *gain;
  void *H, *Y;
  float *rstd, *scale;
  int8_t *Q;
  float eps;
  int64_t R, C;
};

// The looped kernel, for rows of fewer elements than a vector or of more than
// 16384: one workgroup per row (grid-stride), three passes over the row: the sum and
// its squares, the largest |y|, the outputs; each thread reads again only
// what it read or wrote itself
template <class T>
__global__ __launch_bounds__(kNT) void norm_rows(NormArgs a) {
  __shared__ float part[4];
  __shared__ uint32_t upart[4];
  const int t = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.X) + row * a.C;
    const T *res = a.res ? static_cast<const T *>(a.res) + row * a.C : nullptr;
    T *h = res ? static_cast<T *>(a.H) + row * a.C : nullptr;
    float ss = 0.f;
    for (int64_t c = t; c < a.C; c += kNT) {
      T v = x[c];
      if (res) {
        v = narrow<T>(widen(v) + widen(res[c]));
        h[c] = v;
      }
      const float f = widen(v);
      ss = __builtin_fmaf(f, f, ss);
    }
    ss = block_sum(ss, part);
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(ss, (float)a.C) + a.eps));
    const T *src = res ? h : x;
    uint32_t m = 0;
    for (int64_t c = t; c < a.C; c += kNT) {
      const uint32_t u = mag((widen(src[c]) * rstd) * a.gain[c]);
      m = u > m ? u : m;
    }
    const float s = __fdiv_rn(block_max(m, upart), 127.f);
    if (t == 0) {
      a.scale[row] = s;
      if (a.rstd) a.rstd[row] = rstd;
    }
    int8_t *q = a.Q + row * a.C;
    T *y = a.Y ? static_cast<T *>(a.Y) + row * a.C : nullptr;
    for (int64_t c = t; c < a.C; c += kNT) {
      const float v = (widen(src[c]) * rstd) * a.gain[c];
      if (y) y[c] = narrow<T>(v);
      q[c] = quant1(v, s);
    }
  }
}

// Rows in registers, grid-stride over them; the gain stays in registers from
// row to row.  Bound by HBM: 16384x1280 bf16 with residual and Y, 189 MB, takes
// 33 us (the looped kernel below 110 us).
template <class T, int W, int V>
__global__ __launch_bounds__(max_t(W, V)) void norm_reg(NormArgs a) {
  constexpr int U = kU<T>;
  __shared__ float part[2][16];
  __shared__ uint32_t upart[2][16];
  const int t = W ? threadIdx.x & 63 : threadIdx.x;
  const int grp = W ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  Units<T, W, V> un;
  un.init((int32_t)a.C, t);
  float gain[V][U];
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (un.on(j)) load_f<U>(a.gain + un.off[j], gain[j]);
  int flip = 0;
  const int groups = W ? (int)(blockDim.x >> 6) : 1;
  for (int64_t row = (int64_t)blockIdx.x * groups + grp; row < a.R; row += (int64_t)gridDim.x * groups, flip ^= 1) {
    const int64_t base = row * a.C;
    const T *x = static_cast<const T *>(a.X) + base;
    typename Raw<T>::V h[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) h[j] = load_raw(x + un.off[j]);
    if (a.res) {
      const T *res = static_cast<const T *>(a.res) + base;
      typename Raw<T>::V r[V];
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) r[j] = load_raw(res + un.off[j]);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) {
          float f[U], g[U];
          unpack(h[j], f);
          unpack(r[j], g);
#pragma unroll
          for (int i = 0; i < U; ++i) f[i] += g[i];
          h[j] = pack(f);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        float f[U];
        unpack(h[j], f);
        if (j == un.last) {
#pragma unroll
          for (int i = 0; i < U; ++i) f[i] = i < un.dup ? 0.f : f[i];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) ss = __builtin_fmaf(f[i], f[i], ss);
      }
    ss = row_sum<W>(ss, part[flip]);
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(ss, (float)a.C) + a.eps));
    if (a.res) {
      T *H = static_cast<T *>(a.H) + base;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) store_raw(H + un.off[j], h[j]);
    }
    float y[V][U];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        unpack(h[j], y[j]);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          y[j][i] = (y[j][i] * rstd) * gain[j][i];
          m = umax(m, mag(y[j][i]));
        }
      }
    const float s = __fdiv_rn(row_max<W>(m, upart[flip]), 127.f), r = __fdiv_rn(1.f, s);
    const bool fast = fast_scale(s);
    if (t == 0) {
      a.scale[row] = s;
      if (a.rstd) a.rstd[row] = rstd;
    }
    int8_t *q = a.Q + base;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) store_q<U>(q + un.off[j], y[j], s, r, fast);
    if (a.Y) {
      T *Y = static_cast<T *>(a.Y) + base;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) store_raw(Y + un.off[j], pack(y[j]));
    }
  }
}

// ---------------------------------------------------------------------------
// Backward of the norm, and of the epilogue.  In registers: one pass over the
// rows, each thread adding its columns' terms up over the rows that its group
// takes; the sums of a workgroup's groups meet in LDS, and its row of P goes
// to col_finish, which adds the workgroups up in order.  At 16384x3456 bf16 the
// norm's 453 MB take 86 us and 4.7 us for col_finish, at the rate of a copy; the
// epilogue's 396 MB 91 us with gelu, whose sigmoid takes about 50 us of vector
// instructions under the loads (sixteen waves a CU hide more of it than eight,
// 121 us; the next row's loads a row ahead gained nothing, 97 us).  Row pass and
// column pass apart read everything twice: 388 and 400 us.
// ---------------------------------------------------------------------------
template <class T, int W, int V>
__device__ __forceinline__ void write_cols(float (&acc)[V][kU<T>], const Units<T, W, V> &un, int grp, float *lds,
                                           float *__restrict__ P) {
  constexpr int U = kU<T>;
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (j != un.last || i >= un.dup) f(un.off[j] + i, acc[j][i]);
      }
  };
  if constexpr (W == 0) {
    each([&](int c, float v) { P[c] = v; });
  } else {
    // group after group adds into LDS
    const int groups = (int)(blockDim.x >> 6);
    for (int g = 0; g < groups; ++g) {
      if (grp == g) {
        if (groups == 1)
          each([&](int c, float v) { P[c] = v; });
        else if (g == 0)
          each([&](int c, float v) { lds[c] = v; });
        else if (g < groups - 1)
          each([&](int c, float v) { lds[c] += v; });
        else
          each([&](int c, float v) { P[c] = lds[c] + v; });
      }
      lds_barrier();
    }
  }
}

// The same by one workgroup for all rows (the passes with two column sums): every
// group's sums lie side by side in LDS, and the threads each add columns up, group
// after group, which takes no turns of the groups.
constexpr int kOneGroups = 16;
template <class T, int V>
__device__ __forceinline__ void write_cols_one(float (&acc)[V][kU<T>], const Units<T, 1, V> &un, int grp, int32_t C,
                                               float *lds, float *__restrict__ out) {
  constexpr int U = kU<T>;
  __syncthreads();   // the sums before these have been read
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (un.on(j)) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (j != un.last || i >= un.dup) lds[grp * (64 * V * U) + un.off[j] + i] = acc[j][i];
    }
  __syncthreads();
  const int groups = (int)(blockDim.x >> 6);
  for (int32_t c = threadIdx.x; c < C; c += blockDim.x) {
    float sum = lds[c];
    for (int g = 1; g < groups; ++g) sum += lds[g * (64 * V * U) + c];
    out[c] = sum;
  }
}

struct NormBwdArgs {
  const void *dY, *H;
  const float *gain, *rstd;
  const void *dH;
  void *dX;
  float *P;      // [gridDim.x][C]
  int64_t R, C;
};

template <class T, int W, int V>
__global__ __launch_bounds__(max_t(W, V)) void norm_bwd_reg(NormBwdArgs a) {
  constexpr int U = kU<T>;
  __shared__ float part[2][16];
  __shared__ float cols[W ? 64 * V * U : 1];
  const int t = W ? threadIdx.x & 63 : threadIdx.x;
  const int grp = W ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  Units<T, W, V> un;
  un.init((int32_t)a.C, t);
  // past one unit a thread, registers are short and every row reads the gain
  // again (from the caches)
  constexpr bool kKeep = V == 1;
  float kept[U], acc[V][U];
  if (kKeep && un.on(0)) load_f<U>(a.gain + un.off[0], kept);
  auto gain_of = [&](int j, float (&g)[U]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < U; ++i) g[i] = kept[i];
    } else {
      load_f<U>(a.gain + un.off[j], g);
    }
  };
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int i = 0; i < U; ++i) acc[j][i] = 0.f;
  }
  const float invC = __fdiv_rn(1.f, (float)a.C);
  int flip = 0;
  const int groups = W ? (int)(blockDim.x >> 6) : 1;
  for (int64_t row = (int64_t)blockIdx.x * groups + grp; row < a.R; row += (int64_t)gridDim.x * groups, flip ^= 1) {
    const int64_t base = row * a.C;
    typename Raw<T>::V dy[V], h[V], dh[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        dy[j] = load_raw(static_cast<const T *>(a.dY) + base + un.off[j]);
        h[j] = load_raw(static_cast<const T *>(a.H) + base + un.off[j]);
      }
    if (a.dH) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) dh[j] = load_raw(static_cast<const T *>(a.dH) + base + un.off[j]);
    }
    const float rstd = a.rstd[row];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        float d[U], f[U], gain[U], part_sum = 0.f;
        gain_of(j, gain);
        unpack(dy[j], d);
        unpack(h[j], f);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float g = d[i] * (f[i] * rstd);
          acc[j][i] += g;
          // left out by not adding it: a zero factor would make an infinity a NaN
          part_sum = (j == un.last && i < un.dup) ? part_sum : __builtin_fmaf(g, gain[i], part_sum);
        }
        sum += part_sum;
      }
    if (W == 0 && a.dH) {
      // dX may be dH itself, and two waves may share a row's last elements:
      // dH is in registers before the barrier that the stores come after
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) asm volatile("" : "+v"(dh[j]));
    }
    const float mean = row_sum<W>(sum, part[flip]) * invC;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        float d[U], f[U], gain[U];
        gain_of(j, gain);
        unpack(dy[j], d);
        unpack(h[j], f);
#pragma unroll
        for (int i = 0; i < U; ++i) d[i] = rstd * __builtin_fmaf(-(f[i] * rstd), mean, d[i] * gain[i]);
        if (a.dH) {
          unpack(dh[j], f);
#pragma unroll
          for (int i = 0; i < U; ++i) d[i] += f[i];
        }
        store_raw(static_cast<T *>(a.dX) + base + un.off[j], pack(d));
      }
  }
  write_cols<T, W, V>(acc, un, grp, cols, a.P + (int64_t)blockIdx.x * a.C);
}

template <class T>
__global__ __launch_bounds__(kNT) void norm_bwd_rows(NormBwdArgs a) {
  __shared__ float part[4];
  const int t = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const T *dy = static_cast<const T *>(a.dY) + row * a.C;
    const T *h = static_cast<const T *>(a.H) + row * a.C;
    const T *dh = a.dH ? static_cast<const T *>(a.dH) + row * a.C : nullptr;
    T *dx = static_cast<T *>(a.dX) + row * a.C;
    const float rstd = a.rstd[row];
    float sum = 0.f;
    for (int64_t c = t; c < a.C; c += kNT) sum = __builtin_fmaf(widen(dy[c]) * a.gain[c], widen(h[c]) * rstd, sum);
    const float mean = __fdiv_rn(block_sum(sum, part), (float)a.C);
    for (int64_t c = t; c < a.C; c += kNT) {
      float v = rstd * (widen(dy[c]) * a.gain[c] - widen(h[c]) * rstd * mean);
      if (dh) v += widen(dh[c]);
      dx[c] = narrow<T>(v);
    }
  }
}

struct EpiBwdArgs {
  const void *dY, *Z;
  void *dZ;
  int8_t *Q;
  float *scale;
  float *P;      // [gridDim.x][C], or null
  int64_t R, C;
  int32_t act;
};

constexpr float kGeluA = 1.5957691216057308f;              // 2 sqrt(2 / pi)
constexpr float kGeluAB = 1.5957691216057308f * 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

// dz = dy * act'(z).  For z sigmoid(u) the slope is p + z p (1 - p) u', p =
// sigmoid(u); silu and gelu differ in four constants and a clamp: with c = z
// held to +-lim,
//     t = c (k0 + k1 c^2),  e = 2^t,  p = 1 / (1 + e),  q = e p = 1 - p
//     act' = p + c (d0 + d1 c^2) q p
// lim (87 for silu, 10 for gelu) is where the slope reaches 0 or 1 to within
// 1e-35 and e is still finite.
struct Sigm {
  float lim, k0, k1, d0, d1;
};
__device__ __forceinline__ Sigm sigm_of(int act) {
  if (act == TGEMM_ACT_SILU) return {87.f, -kLog2e, 0.f, 1.f, 0.f};
  return {10.f, -kGeluA * kLog2e, -kGeluAB * kLog2e, kGeluA, 3.f * kGeluAB};
}
__device__ __forceinline__ float back_sigm(float dy, float z, const Sigm &k) {
  const float c = fminf(fmaxf(z, -k.lim), k.lim), c2 = c * c;
  const float e = __builtin_amdgcn_exp2f(c * __builtin_fmaf(k.k1, c2, k.k0));
  const float p = __builtin_amdgcn_rcpf(1.f + e);
  const float w = c * __builtin_fmaf(k.d1, c2, k.d0) * (e * p);
  const float d = dy * __builtin_fmaf(w, p, p);
  return z == z ? d : z;   // the clamp drops a NaN
}

// relu2's 2 z dy is taken as p + p, p = z dy, which overflows only where the
// product does (2 z or 2 dy alone may do so before); a NaN z stays one
__device__ __forceinline__ float back_relu(float dy, float z) { return dy * (z > 0.f ? 1.f : (z == z ? 0.f : z)); }
__device__ __forceinline__ float back_relu2(float dy, float z) {
  const float p = dy * (z < 0.f ? 0.f : z);
  return p + p;
}
__host__ __device__ __forceinline__ bool is_sigm(int act) { return act >= TGEMM_ACT_SILU; }
static_assert(TGEMM_ACT_GELU_TANH > TGEMM_ACT_SILU && TGEMM_ACT_RELU2 < TGEMM_ACT_SILU, "is_sigm");

__device__ __forceinline__ float back(float dy, float z, int act) {
  if (is_sigm(act)) return back_sigm(dy, z, sigm_of(act));
  return act == TGEMM_ACT_NONE ? dy : act == TGEMM_ACT_RELU ? back_relu(dy, z) : back_relu2(dy, z);
}

// S: silu and gelu_tanh, else the other three, one uniform branch a unit
template <class T, int W, int V, int S>
__global__ __launch_bounds__(max_t(W, V)) void epi_bwd_reg(EpiBwdArgs a) {
  constexpr int U = kU<T>;
  __shared__ uint32_t upart[2][16];
  __shared__ float cols[W ? 64 * V * U : 1];
  const int t = W ? threadIdx.x & 63 : threadIdx.x;
  const int grp = W ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  Units<T, W, V> un;
  un.init((int32_t)a.C, t);
  float acc[V][U];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < U; ++i) acc[j][i] = 0.f;
  const Sigm sg = sigm_of(a.act);
  int flip = 0;
  const int groups = W ? (int)(blockDim.x >> 6) : 1;
  for (int64_t row = (int64_t)blockIdx.x * groups + grp; row < a.R; row += (int64_t)gridDim.x * groups, flip ^= 1) {
    const int64_t base = row * a.C;
    typename Raw<T>::V dy[V], z[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        dy[j] = load_raw(static_cast<const T *>(a.dY) + base + un.off[j]);
        z[j] = load_raw(static_cast<const T *>(a.Z) + base + un.off[j]);
      }
    float d[V][U];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        float f[U];
        unpack(dy[j], d[j]);
        unpack(z[j], f);
        if constexpr (S) {
#pragma unroll
          for (int i = 0; i < U; ++i) d[j][i] = back_sigm(d[j][i], f[i], sg);
        } else if (a.act == TGEMM_ACT_RELU) {
#pragma unroll
          for (int i = 0; i < U; ++i) d[j][i] = back_relu(d[j][i], f[i]);
        } else if (a.act == TGEMM_ACT_RELU2) {
#pragma unroll
          for (int i = 0; i < U; ++i) d[j][i] = back_relu2(d[j][i], f[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          acc[j][i] += d[j][i];
          m = umax(m, mag(d[j][i]));
        }
      }
    const float s = __fdiv_rn(row_max<W>(m, upart[flip]), 127.f), r = __fdiv_rn(1.f, s);
    const bool fast = fast_scale(s);
    if (t == 0) a.scale[row] = s;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        store_raw(static_cast<T *>(a.dZ) + base + un.off[j], pack(d[j]));
        store_q<U>(a.Q + base + un.off[j], d[j], s, r, fast);
      }
  }
  if (a.P) write_cols<T, W, V>(acc, un, grp, cols, a.P + (int64_t)blockIdx.x * a.C);
}

template <class T>
__global__ __launch_bounds__(kNT) void epi_bwd_rows(EpiBwdArgs a) {
  __shared__ uint32_t upart[4];
  const int t = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const T *dy = static_cast<const T *>(a.dY) + row * a.C;
    const T *z = static_cast<const T *>(a.Z) + row * a.C;
    T *dz = static_cast<T *>(a.dZ) + row * a.C;
    int8_t *q = a.Q + row * a.C;
    uint32_t m = 0;
    for (int64_t c = t; c < a.C; c += kNT) {
      const float v = back(widen(dy[c]), widen(z[c]), a.act);
      dz[c] = narrow<T>(v);
      const uint32_t u = mag(v);
      m = u > m ? u : m;
    }
    const float s = __fdiv_rn(block_max(m, upart), 127.f);
    if (t == 0) a.scale[row] = s;
    for (int64_t c = t; c < a.C; c += kNT) q[c] = quant1(back(widen(dy[c]), widen(z[c]), a.act), s);
  }
}

// Partial column sums: workgroup (x, y) takes 256 columns, one a thread, and
// the y-th strip of rows, and writes its sums to row y of P.  NORM: the terms
// are dy * h * rstd; otherwise dy * act'(z).  c0: the launch's first column (a launch
// has fewer than 2^32 threads: launch_columns).
constexpr int64_t kMaxColGrid = 1 << 20;
template <class Launch>
void launch_columns(int64_t C, int64_t each, Launch launch) {   // `each` columns a workgroup
  for (int64_t c0 = 0; c0 < C; c0 += kMaxColGrid * each) {
    const int64_t n = ceil_div(C - c0, each);
    launch((unsigned)(n < kMaxColGrid ? n : kMaxColGrid), c0);
  }
}
template <class T, bool NORM>
__global__ __launch_bounds__(kNT) void col_sums(const T *__restrict__ A, const T *__restrict__ B,
                                                const float *__restrict__ rstd, int32_t act, float *__restrict__ P,
                                                int64_t R, int64_t C, int64_t strip, int64_t c0) {
  const int64_t c = c0 + (int64_t)blockIdx.x * kNT + threadIdx.x;
  if (c >= C) return;
  const int64_t r0 = (int64_t)blockIdx.y * strip, r1 = r0 + strip < R ? r0 + strip : R;
  float sum = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float a = widen(A[r * C + c]), b = widen(B[r * C + c]);
    sum = NORM ? __builtin_fmaf(a, b * rstd[r], sum) : sum + back(a, b, act);
  }
  P[blockIdx.y * C + c] = sum;
}

// ---------------------------------------------------------------------------
// Layer norm.  As the RMS norm, with the mean taken off first: the mean from one
// sum over the row, the variance from a second one over the squares of what is
// left (from the registers: the row is still read once).  A mean far above the
// deviation has to cost neither of them anything.  bfloat16 values of one size add up
// exactly in float32 (8 bits each, at most 2^14 of them), and the mean's rounding is
// 2^-16 of their spacing.  float32 values do not: 1280 of them about 4096 that deviate by
// 0.03 leave a float32 mean off by up to 2% of the deviation, so their sum and the mean
// are held to more bits (Mean), at 3% of the time of 16384x3456 without a residual and
// nothing with one.  A row of one value leaves exact zeros either way.
// Bound by HBM: 16384x1280
// bf16 with residual and Y, 189 MB, 34 us (the RMS norm 33), 16384x3456 float32, 963 MB,
// 188 us.  Column sums of both kinds (dgain, dbeta) cost the backward pass little more
// than one: 16384x3456 bf16 91 us against 84, 16384x1280 float32 62 against 60.  Its float32
// rows past 12288 spill 87 registers: 2048x14336 174 us (a copy's rate: 89), where
// 2048x11008, without, takes 86 (68).
// ---------------------------------------------------------------------------
struct LnArgs {
  const void *X, *res;
  const float *gain, *beta;   // beta may be null
  void *H, *Y;
  float *mean, *rstd, *scale;
  int8_t *Q;
  float eps;
  int64_t R, C;
  double n, inv;   // C and 1 / C
};

// The mean of C values from their sum in 64 bits: hi is its nearest float32, lo the
// rest (sum - C hi is exact by fma, and 0 where hi is the mean).  With d = h - hi,
//     sum (h - mean)^2 / C = sum d^2 / C - lo^2,  (h - mean) rstd = d rstd - lo rstd
// No h, itself a float32, is nearer to the mean than hi, so lo^2 is at most half of
// sum d^2 / C and the difference loses one bit.
struct Mean {
  float hi, lo;
};
__device__ __forceinline__ Mean mean_of(double sum, double C, double invC) {
  const float hi = (float)(sum * invC);
  return {hi, (float)(__builtin_fma(-C, (double)hi, sum) * invC)};
}
__device__ __forceinline__ float ln_rstd(float ss, const Mean &m, float C, float eps) {
  return __fdiv_rn(1.f, __fsqrt_rn(__builtin_fmaf(-m.lo, m.lo, __fdiv_rn(ss, C)) + eps));
}
// shift: -lo rstd
__device__ __forceinline__ float ln_y(float d, float rstd, float shift, float gain, float beta) {
  return __builtin_fmaf(__builtin_fmaf(d, rstd, shift), gain, beta);
}

template <class T>
__global__ __launch_bounds__(kNT) void ln_rows(LnArgs a) {
  __shared__ double part[4];
  __shared__ float part2[4];
  __shared__ uint32_t upart[4];
  const int t = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.X) + row * a.C;
    const T *res = a.res ? static_cast<const T *>(a.res) + row * a.C : nullptr;
    T *h = res ? static_cast<T *>(a.H) + row * a.C : nullptr;
    double sum = 0.;
    for (int64_t c = t; c < a.C; c += kNT) {
      T v = x[c];
      if (res) {
        v = narrow<T>(widen(v) + widen(res[c]));
        h[c] = v;
      }
      sum += (double)widen(v);
    }
    const Mean mean = mean_of(block_sum(sum, part), a.n, a.inv);
    const T *src = res ? h : x;
    float ss = 0.f;
    for (int64_t c = t; c < a.C; c += kNT) {
      const float d = widen(src[c]) - mean.hi;
      ss = __builtin_fmaf(d, d, ss);
    }
    const float rstd = ln_rstd(block_sum(ss, part2), mean, (float)a.C, a.eps), shift = -mean.lo * rstd;
    uint32_t m = 0;
    for (int64_t c = t; c < a.C; c += kNT)
      m = umax(m, mag(ln_y(widen(src[c]) - mean.hi, rstd, shift, a.gain[c], a.beta ? a.beta[c] : 0.f)));
    const float s = __fdiv_rn(block_max(m, upart), 127.f);
    if (t == 0) {
      a.scale[row] = s;
      if (a.rstd) {
        a.mean[row] = mean.hi;
        a.rstd[row] = rstd;
      }
    }
    int8_t *q = a.Q + row * a.C;
    T *y = a.Y ? static_cast<T *>(a.Y) + row * a.C : nullptr;
    for (int64_t c = t; c < a.C; c += kNT) {
      const float v = ln_y(widen(src[c]) - mean.hi, rstd, shift, a.gain[c], a.beta ? a.beta[c] : 0.f);
      if (y) y[c] = narrow<T>(v);
      q[c] = quant1(v, s);
    }
  }
}

template <class T, int W, int V>
__global__ __launch_bounds__(max_t(W, V)) void ln_reg(LnArgs a) {
  constexpr int U = kU<T>;
  // In float32 a workgroup's next row is loaded while it reduces the one in hand
  // (16384x3456 at one unit a lane, residual 177 -> 149 us, without 139 -> 131; four units spill).
  // bfloat16 rows gain nothing from it without a residual and lose with one (89 -> 97 us).
  constexpr bool kAhead = W == 0 && U == 4 && V <= 3;
  constexpr bool kSplit = U == 4;   // the mean in two parts
  __shared__ std::conditional_t<kSplit, double, float> part[2][16];
  __shared__ float part2[2][16];
  __shared__ uint32_t upart[2][16];
  const int t = W ? threadIdx.x & 63 : threadIdx.x;
  const int grp = W ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  Units<T, W, V> un;
  un.init((int32_t)a.C, t);
  float gain[V][U], beta[V][U];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int i = 0; i < U; ++i) beta[j][i] = 0.f;
    if (un.on(j)) {
      load_f<U>(a.gain + un.off[j], gain[j]);
      if (a.beta) load_f<U>(a.beta + un.off[j], beta[j]);
    }
  }
  // kSplit: the lane's elements (0 in lanes past the row), about one over them (lane 0's
  // serves), and the wave's
  const float own = (float)(U * un.n - (un.last >= 0 ? un.dup : 0)), per = __builtin_amdgcn_rcpf(fmaxf(own, 1.f));
  const double wave_own = W ? a.n : (double)wave_sum(own);
  int flip = 0;
  const int groups = W ? (int)(blockDim.x >> 6) : 1;
  const int64_t stride = (int64_t)gridDim.x * groups;
  typename Raw<T>::V hn[V], rn[V];
  auto ahead = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        hn[j] = load_raw(static_cast<const T *>(a.X) + row * a.C + un.off[j]);
        if (a.res) rn[j] = load_raw(static_cast<const T *>(a.res) + row * a.C + un.off[j]);
      }
  };
  if (kAhead && (int64_t)blockIdx.x < a.R) ahead(blockIdx.x);
  for (int64_t row = (int64_t)blockIdx.x * groups + grp; row < a.R; row += stride, flip ^= 1) {
    const int64_t base = row * a.C;
    const T *x = static_cast<const T *>(a.X) + base;
    typename Raw<T>::V h[V], res_row[V];
    if constexpr (kAhead) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[j] = hn[j];
        res_row[j] = rn[j];
      }
      if (row + stride < a.R) ahead(row + stride);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) h[j] = load_raw(x + un.off[j]);
    }
    if (a.res) {
      if constexpr (!kAhead) {
        const T *res = static_cast<const T *>(a.res) + base;
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (un.on(j)) res_row[j] = load_raw(res + un.off[j]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) {
          float f[U], g[U];
          unpack(h[j], f);
          unpack(res_row[j], g);
#pragma unroll
          for (int i = 0; i < U; ++i) f[i] += g[i];
          h[j] = pack(f);
        }
    }
    Mean mean;
    if constexpr (kSplit) {
      // A lane's sum in float32 is of differences from its first value, a wave's of
      // differences from the mean of its lane 0: both are of the size of the deviation.
      float first = 0.f, diff = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) {
          float f[U];
          unpack(h[j], f);
          if (j == 0) first = f[0];
#pragma unroll
          for (int i = 0; i < U; ++i) diff += j == un.last && i < un.dup ? 0.f : f[i] - first;
        }
      const float about = lane_f(__builtin_fmaf(diff, per, first), 0);
      const float rest = wave_sum(__builtin_fmaf(own, first - about, diff));
      double sum = __builtin_fma(wave_own, (double)about, (double)rest);
      if (!(fabsf(rest) < __builtin_inff())) {   // the differences pass float32, or a value is not finite
        sum = 0.;
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (un.on(j)) {
            float f[U];
            unpack(h[j], f);
#pragma unroll
            for (int i = 0; i < U; ++i) sum += (double)(j == un.last && i < un.dup ? 0.f : f[i]);
          }
        sum = wave_sum(sum);
      }
      mean = mean_of(row_sum_waves<W>(sum, part[flip]), a.n, a.inv);
    } else {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) {
          float f[U];
          unpack(h[j], f);
#pragma unroll
          for (int i = 0; i < U; ++i) sum += j == un.last && i < un.dup ? 0.f : f[i];
        }
      mean = {__fdiv_rn(row_sum<W>(sum, part[flip]), (float)a.C), 0.f};
    }
    float y[V][U], ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        unpack(h[j], y[j]);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          y[j][i] -= mean.hi;
          const float d = j == un.last && i < un.dup ? 0.f : y[j][i];
          ss = __builtin_fmaf(d, d, ss);
        }
      }
    ss = row_sum<W>(ss, part2[flip]);
    const float rstd = ln_rstd(ss, mean, (float)a.C, a.eps), shift = kSplit ? -mean.lo * rstd : 0.f;
    if (a.res) {
      T *H = static_cast<T *>(a.H) + base;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) store_raw(H + un.off[j], h[j]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          y[j][i] = ln_y(y[j][i], rstd, shift, gain[j][i], beta[j][i]);
          m = umax(m, mag(y[j][i]));
        }
      }
    const float s = __fdiv_rn(row_max<W>(m, upart[flip]), 127.f), r = __fdiv_rn(1.f, s);
    const bool fast = fast_scale(s);
    if (t == 0) {
      a.scale[row] = s;
      if (a.rstd) {
        a.mean[row] = mean.hi;
        a.rstd[row] = rstd;
      }
    }
    int8_t *q = a.Q + base;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) store_q<U>(q + un.off[j], y[j], s, r, fast);
    if (a.Y) {
      T *Y = static_cast<T *>(a.Y) + base;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) store_raw(Y + un.off[j], pack(y[j]));
    }
  }
}

// Its backward pass: with xhat = (h - mean) rstd and t = dy gain,
//     dX = rstd (t - sum t / C - xhat sum(t xhat) / C) + dH
// Both sums of a row meet in one exchange, and the two column sums lie side by
// side in a workgroup's row of P.
struct LnBwdArgs {
  const void *dY, *H;
  const float *gain, *mean, *rstd;
  const void *dH;
  void *dX;
  float *P, *P2;   // partial sums of dgain and dbeta (P2 null: none), `pitch` apart from workgroup to workgroup
  int64_t pitch;
  int64_t R, C;
};

template <int W>
__device__ __forceinline__ f32x2 row_sum2(float v, float w, f32x2 *part) {
  v = wave_sum(v);
  w = wave_sum(w);
  if constexpr (W == 0) {
    const int lane = threadIdx.x & 63, l = lane & 15;
    if (lane == 0) part[threadIdx.x >> 6] = f32x2{v, w};
    lds_barrier();
    const f32x2 p = l < (int)(blockDim.x >> 6) ? part[l] : f32x2{0.f, 0.f};
    v = p[0];
    w = p[1];
    v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
    w += __uint_as_float(dpp<kXor1>(__float_as_uint(w)));
    v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
    w += __uint_as_float(dpp<kXor2>(__float_as_uint(w)));
    v += __uint_as_float(dpp<kHalfMirror>(__float_as_uint(v)));
    w += __uint_as_float(dpp<kHalfMirror>(__float_as_uint(w)));
    v += __uint_as_float(dpp<kMirror>(__float_as_uint(v)));
    w += __uint_as_float(dpp<kMirror>(__float_as_uint(w)));
  }
  return f32x2{v, w};
}

template <class T, int W, int V, bool ONE = false>
__global__ __launch_bounds__(ONE ? 64 * kOneGroups : max_t(W, V)) void ln_bwd_reg(LnBwdArgs a) {
  constexpr int U = kU<T>;
  __shared__ f32x2 part[2][16];
  __shared__ float cols[ONE ? kOneGroups * 64 * V * U : W ? 64 * V * U : 1];
  const int t = W ? threadIdx.x & 63 : threadIdx.x;
  const int grp = W ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  Units<T, W, V> un;
  un.init((int32_t)a.C, t);
  constexpr bool kKeep = V == 1;   // as in norm_bwd_reg
  float kept[U], acc[V][U], bacc[V][U];
  if (kKeep && un.on(0)) load_f<U>(a.gain + un.off[0], kept);
  auto gain_of = [&](int j, float (&g)[U]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < U; ++i) g[i] = kept[i];
    } else {
      load_f<U>(a.gain + un.off[j], g);
    }
  };
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int i = 0; i < U; ++i) acc[j][i] = bacc[j][i] = 0.f;
  }
  const float invC = __fdiv_rn(1.f, (float)a.C);
  int flip = 0;
  const int groups = W ? (int)(blockDim.x >> 6) : 1;
  for (int64_t row = (int64_t)blockIdx.x * groups + grp; row < a.R; row += (int64_t)gridDim.x * groups, flip ^= 1) {
    const int64_t base = row * a.C;
    typename Raw<T>::V dy[V], h[V], dh[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        dy[j] = load_raw(static_cast<const T *>(a.dY) + base + un.off[j]);
        h[j] = load_raw(static_cast<const T *>(a.H) + base + un.off[j]);
      }
    if (a.dH) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) dh[j] = load_raw(static_cast<const T *>(a.dH) + base + un.off[j]);
    }
    const float rstd = a.rstd[row], mean = a.mean[row];
    float st = 0.f, sx = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        float d[U], f[U], gain[U], pt = 0.f, px = 0.f;
        gain_of(j, gain);
        unpack(dy[j], d);
        unpack(h[j], f);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float g = d[i] * ((f[i] - mean) * rstd);
          acc[j][i] += g;
          bacc[j][i] += d[i];
          // left out by not adding it: a zero factor would make an infinity a NaN
          const bool twice = j == un.last && i < un.dup;
          pt = twice ? pt : __builtin_fmaf(d[i], gain[i], pt);
          px = twice ? px : __builtin_fmaf(g, gain[i], px);
        }
        st += pt;
        sx += px;
      }
    if (W == 0 && a.dH) {
      // as in norm_bwd_reg: dX may be dH itself
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (un.on(j)) asm volatile("" : "+v"(dh[j]));
    }
    const f32x2 sums = row_sum2<W>(st, sx, part[flip]);
    const float mt = sums[0] * invC, mx = sums[1] * invC;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        float d[U], f[U], gain[U];
        gain_of(j, gain);
        unpack(dy[j], d);
        unpack(h[j], f);
#pragma unroll
        for (int i = 0; i < U; ++i)
          d[i] = rstd * __builtin_fmaf(-((f[i] - mean) * rstd), mx, __builtin_fmaf(d[i], gain[i], -mt));
        if (a.dH) {
          unpack(dh[j], f);
#pragma unroll
          for (int i = 0; i < U; ++i) d[i] += f[i];
        }
        store_raw(static_cast<T *>(a.dX) + base + un.off[j], pack(d));
      }
  }
  if constexpr (ONE) {
    write_cols_one<T, V>(acc, un, grp, (int32_t)a.C, cols, a.P);
    if (a.P2) write_cols_one<T, V>(bacc, un, grp, (int32_t)a.C, cols, a.P2);
  } else {
    write_cols<T, W, V>(acc, un, grp, cols, a.P + (int64_t)blockIdx.x * a.pitch);
    if (a.P2) write_cols<T, W, V>(bacc, un, grp, cols, a.P2 + (int64_t)blockIdx.x * a.pitch);
  }
}

template <class T>
__global__ __launch_bounds__(kNT) void ln_bwd_rows(LnBwdArgs a) {
  __shared__ float part[4];
  const int t = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const T *dy = static_cast<const T *>(a.dY) + row * a.C;
    const T *h = static_cast<const T *>(a.H) + row * a.C;
    const T *dh = a.dH ? static_cast<const T *>(a.dH) + row * a.C : nullptr;
    T *dx = static_cast<T *>(a.dX) + row * a.C;
    const float rstd = a.rstd[row], mean = a.mean[row];
    float st = 0.f, sx = 0.f;
    for (int64_t c = t; c < a.C; c += kNT) {
      const float v = widen(dy[c]) * a.gain[c];
      st += v;
      sx = __builtin_fmaf(v, (widen(h[c]) - mean) * rstd, sx);
    }
    const float mt = __fdiv_rn(block_sum(st, part), (float)a.C), mx = __fdiv_rn(block_sum(sx, part), (float)a.C);
    for (int64_t c = t; c < a.C; c += kNT) {
      float v = rstd * __builtin_fmaf(-((widen(h[c]) - mean) * rstd), mx, __builtin_fmaf(widen(dy[c]), a.gain[c], -mt));
      if (dh) v += widen(dh[c]);
      dx[c] = narrow<T>(v);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward of the gated product: row r of Z holds the gate's values z and, C
// further, the up projection's u.
//     dz = dy u act'(z),  du = dy act(z)
// dZ, the int8 rows and the column sums have the same two halves; the int8 rows
// are of (kz dz | ku du), k the scales of the two weight matrices, so that one
// product with both matrices' codes adds the two parts of dX up.  One pass over dY and
// Z, the row's 2 C values kept in registers between its largest magnitude and its int8
// row: 16384x3456 bf16, 680 MB, takes 144 us with silu (4.7 TB/s) and 4.7 for col_finish.
// Past 8192 columns a workgroup's sixteen waves hold two bfloat16 units a lane, or three
// or four float32 ones, in 128 registers, and spill: two 21 to 23 of them, three 21 to
// 26, four 64 to 70.  silu, column sums and all: 4096x11008 bf16 163 us (a copy's rate:
// 102), 4096x14336 193 (133), 4096x16384 209 (152); 2048x11008 float32 128 (94), 2048x14336
// 220 (122).
// ---------------------------------------------------------------------------
struct GatedBwdArgs {
  const void *dY, *Z;
  void *dZ;
  int8_t *Q;
  float *scale;
  float *P;       // [gridDim.x][2 C], or null
  float kz, ku;
  int64_t R, C;
  int32_t act;
};

// (dz, du) of z sigmoid(u(z)), in the terms of back_sigm.  Below -lim act(z) is
// taken there: it is less than 1e-35 from 0, its limit, either way.
__device__ __forceinline__ f32x2 gated_sigm(float dy, float z, float u, const Sigm &k) {
  const float c = fminf(fmaxf(z, -k.lim), k.lim), c2 = c * c;
  const float e = __builtin_amdgcn_exp2f(c * __builtin_fmaf(k.k1, c2, k.k0));
  const float p = __builtin_amdgcn_rcpf(1.f + e);
  const float w = c * __builtin_fmaf(k.d1, c2, k.d0) * (e * p);
  const float dz = (dy * u) * __builtin_fmaf(w, p, p), du = dy * (fmaxf(z, -k.lim) * p);
  return z == z ? f32x2{dz, du} : f32x2{z, z};   // the clamps drop a NaN
}
__device__ __forceinline__ f32x2 gated_poly(float dy, float z, float u, int act) {
  const float t = dy * u;
  if (act == TGEMM_ACT_NONE) return f32x2{t, dy * z};
  const float p = z < 0.f ? 0.f : z;   // a NaN stays one
  return act == TGEMM_ACT_RELU ? f32x2{back_relu(t, z), dy * p} : f32x2{back_relu2(t, z), (dy * p) * p};
}
__device__ __forceinline__ f32x2 gated_back(float dy, float z, float u, int act) {
  return is_sigm(act) ? gated_sigm(dy, z, u, sigm_of(act)) : gated_poly(dy, z, u, act);
}

template <class T, int W, int V, int S, bool ONE = false>
__global__ __launch_bounds__(ONE ? 64 * kOneGroups : max_t(W, V)) void gated_bwd_reg(GatedBwdArgs a) {
  constexpr int U = kU<T>;
  __shared__ uint32_t upart[2][16];
  __shared__ float cols[ONE ? kOneGroups * 64 * V * U : W ? 64 * V * U : 1];
  const int t = W ? threadIdx.x & 63 : threadIdx.x;
  const int grp = W ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  Units<T, W, V> un;
  un.init((int32_t)a.C, t);
  float zacc[V][U], uacc[V][U];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < U; ++i) zacc[j][i] = uacc[j][i] = 0.f;
  const Sigm sg = sigm_of(a.act);
  int flip = 0;
  const int groups = W ? (int)(blockDim.x >> 6) : 1;
  for (int64_t row = (int64_t)blockIdx.x * groups + grp; row < a.R; row += (int64_t)gridDim.x * groups, flip ^= 1) {
    const int64_t base = row * a.C, zbase = 2 * base;
    typename Raw<T>::V dy[V], z[V], u[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        dy[j] = load_raw(static_cast<const T *>(a.dY) + base + un.off[j]);
        z[j] = load_raw(static_cast<const T *>(a.Z) + zbase + un.off[j]);
        u[j] = load_raw(static_cast<const T *>(a.Z) + zbase + a.C + un.off[j]);
      }
    float dz[V][U], du[V][U];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        float d[U];
        unpack(dy[j], d);
        unpack(z[j], dz[j]);
        unpack(u[j], du[j]);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          f32x2 v;
          if constexpr (S)
            v = gated_sigm(d[i], dz[j][i], du[j][i], sg);
          else
            v = gated_poly(d[i], dz[j][i], du[j][i], a.act);
          dz[j][i] = v[0];
          du[j][i] = v[1];
          zacc[j][i] += v[0];
          uacc[j][i] += v[1];
          m = umax(m, umax(mag(v[0] * a.kz), mag(v[1] * a.ku)));
        }
      }
    const float s = __fdiv_rn(row_max<W>(m, upart[flip]), 127.f), r = __fdiv_rn(1.f, s);
    const bool fast = fast_scale(s);
    if (t == 0) a.scale[row] = s;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (un.on(j)) {
        store_raw(static_cast<T *>(a.dZ) + zbase + un.off[j], pack(dz[j]));
        store_raw(static_cast<T *>(a.dZ) + zbase + a.C + un.off[j], pack(du[j]));
#pragma unroll
        for (int i = 0; i < U; ++i) {
          dz[j][i] *= a.kz;
          du[j][i] *= a.ku;
        }
        store_q<U>(a.Q + zbase + un.off[j], dz[j], s, r, fast);
        store_q<U>(a.Q + zbase + a.C + un.off[j], du[j], s, r, fast);
      }
  }
  if constexpr (ONE) {
    if (a.P) {
      write_cols_one<T, V>(zacc, un, grp, (int32_t)a.C, cols, a.P);
      write_cols_one<T, V>(uacc, un, grp, (int32_t)a.C, cols, a.P + a.C);
    }
  } else if (a.P) {
    float *P = a.P + (int64_t)blockIdx.x * 2 * a.C;
    write_cols<T, W, V>(zacc, un, grp, cols, P);
    write_cols<T, W, V>(uacc, un, grp, cols, P + a.C);
  }
}

template <class T>
__global__ __launch_bounds__(kNT) void gated_bwd_rows(GatedBwdArgs a) {
  __shared__ uint32_t upart[4];
  const int t = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const T *dy = static_cast<const T *>(a.dY) + row * a.C;
    const T *z = static_cast<const T *>(a.Z) + 2 * row * a.C, *u = z + a.C;
    T *dz = static_cast<T *>(a.dZ) + 2 * row * a.C;
    int8_t *q = a.Q + 2 * row * a.C;
    uint32_t m = 0;
    for (int64_t c = t; c < a.C; c += kNT) {
      const f32x2 v = gated_back(widen(dy[c]), widen(z[c]), widen(u[c]), a.act);
      dz[c] = narrow<T>(v[0]);
      dz[a.C + c] = narrow<T>(v[1]);
      m = umax(m, umax(mag(v[0] * a.kz), mag(v[1] * a.ku)));
    }
    const float s = __fdiv_rn(block_max(m, upart), 127.f);
    if (t == 0) a.scale[row] = s;
    for (int64_t c = t; c < a.C; c += kNT) {
      const f32x2 v = gated_back(widen(dy[c]), widen(z[c]), widen(u[c]), a.act);
      q[c] = quant1(v[0] * a.kz, s);
      q[a.C + c] = quant1(v[1] * a.ku, s);
    }
  }
}

// Partial column sums of the two looped backward passes, as col_sums: two
// sums a column, C apart in a row of P
struct Cols2Args {
  const void *A, *B;           // dY, and H or Z
  const float *mean, *rstd;    // layer norm
  float *P;                    // [strips][pitch]
  int64_t pitch;               // 2 C, or C for the first sums alone
  int64_t R, C, strip;
  int32_t act;                 // gated
  int64_t c0;                  // the launch's first column
};
template <class T, bool NORM>
__global__ __launch_bounds__(kNT) void col_sums2(Cols2Args k) {
  const int64_t c = k.c0 + (int64_t)blockIdx.x * kNT + threadIdx.x;
  if (c >= k.C) return;
  const T *A = static_cast<const T *>(k.A), *B = static_cast<const T *>(k.B);
  const int64_t r0 = (int64_t)blockIdx.y * k.strip, r1 = r0 + k.strip < k.R ? r0 + k.strip : k.R;
  float s0 = 0.f, s1 = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float a = widen(A[r * k.C + c]);
    if constexpr (NORM) {
      s0 = __builtin_fmaf(a, (widen(B[r * k.C + c]) - k.mean[r]) * k.rstd[r], s0);
      s1 += a;
    } else {
      const f32x2 v = gated_back(a, widen(B[2 * r * k.C + c]), widen(B[(2 * r + 1) * k.C + c]), k.act);
      s0 += v[0];
      s1 += v[1];
    }
  }
  float *P = k.P + blockIdx.y * k.pitch;
  P[c] = s0;
  if (k.pitch > k.C) P[k.C + c] = s1;
}

// the rows of P added up: a workgroup takes 32 columns, its 32 groups of 32
// threads each every 32nd row, eight loads at a time, and the groups' sums
// meet in LDS in order
constexpr int kFinCols = 32, kFinGroups = 32, kFinT = kFinCols * kFinGroups;
// (columns from `split` on go to out2: the sums of two operands side by side)
__global__ __launch_bounds__(kFinT) void col_finish(const float *__restrict__ P, float *__restrict__ out,
                                                    float *__restrict__ out2, int64_t split, int64_t rows, int64_t C,
                                                    int64_t c0) {
  __shared__ float part[kFinGroups][kFinCols + 1];
  const int c = threadIdx.x % kFinCols, g = threadIdx.x / kFinCols;
  const int64_t col = c0 + (int64_t)blockIdx.x * kFinCols + c;
  float sum = 0.f;
  if (col < C)
    for (int64_t r0 = g; r0 < rows; r0 += 8 * kFinGroups) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = r0 + k * kFinGroups < rows ? P[(r0 + k * kFinGroups) * C + col] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += v[k];
    }
  part[g][c] = sum;
  __syncthreads();
  if (g == 0 && col < C) {
#pragma unroll
    for (int i = 1; i < kFinGroups; ++i) sum += part[i][c];
    if (col < split)
      out[col] = sum;
    else
      out2[col - split] = sum;
  }
}

constexpr int64_t kMaxStrips = 512;
int64_t strips_of(int64_t R) { return R < kMaxStrips ? R : kMaxStrips; }

// ---------------------------------------------------------------------------
// Clipping (69.5M bf16: 23.5 us for the sums, 48 us for the scaling, each at the
// rate of a copy).  Two launches over the tensors' chunks: the sums of squares, one
// double a workgroup, then the scaling, whose workgroups each add those
// doubles up again in one order (a few KB from the caches, in place of a
// third launch).  A square of any float32 fits a double, so neither end of
// the range is lost.  The second pass takes the chunks from the last to the
// first: what the first pass read last is still in the caches (256 MB behind
// the L2s), and reading it again costs no HBM.
// ---------------------------------------------------------------------------
constexpr int kGroup = 96;                 // tensors per launch
constexpr int kChunk = 8 * kNT * 4;        // elements per workgroup and step
// Lists of more bytes than this are written past the caches (a nontemporal
// store), which leaves the gradients that the second pass reads in them: 80 MB
// of bf16 29.2 -> 27.8 us, 278 MB 92 -> 78 us, 556 MB of float32 168 -> 140 us.
// Smaller ones stay cached for whatever reads them next.
constexpr int64_t kStreamBytes = 32 << 20;
constexpr int64_t kMaxParts = 1024;        // workgroups of the first pass, over all launches (and one each)

// the tensors of one launch; first[i]: the first chunk of tensor i
struct Tensors {
  const void *in[kGroup];
  void *out[kGroup];
  int64_t size[kGroup];
  int32_t first[kGroup + 1];
  uint8_t bf16[kGroup];
  int32_t count;
};

__device__ __forceinline__ int tensor_of(const Tensors &ts, int32_t chunk) {
  int lo = 0, hi = ts.count;   // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ts.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum_d(double v, double *part) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// the squares of elements e0 .. e1 of a tensor, 16 bytes a load, four in flight
template <class T>
__device__ __forceinline__ double chunk_sumsq(const T *p, int64_t e0, int64_t e1) {
  constexpr int U = kU<T>;
  const int n = (int)(e1 - e0), nu = n / U;
  p += e0;
  double sum = 0.0;
  for (int u0 = threadIdx.x; u0 < nu; u0 += 4 * kNT) {
    typename Raw<T>::V r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (u0 + k * kNT < nu) r[k] = load_raw(p + (u0 + k * kNT) * U);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (u0 + k * kNT < nu) {
        float v[U];
        unpack(r[k], v);
#pragma unroll
        for (int i = 0; i < U; ++i) sum = __builtin_fma((double)v[i], (double)v[i], sum);
      }
  }
  const int e = nu * U + (int)threadIdx.x;   // at most U - 1 elements past the units
  if (e < n) {
    const double v = widen(p[e]);
    sum = __builtin_fma(v, v, sum);
  }
  return sum;
}

__global__ __launch_bounds__(kNT) void sumsq(Tensors ts, double *__restrict__ part) {
  __shared__ double wsum[4];
  double sum = 0.0;
  for (int32_t c = blockIdx.x; c < ts.first[ts.count]; c += gridDim.x) {
    const int i = tensor_of(ts, c);
    const int64_t e0 = (int64_t)(c - ts.first[i]) * kChunk;
    const int64_t e1 = e0 + kChunk < ts.size[i] ? e0 + kChunk : ts.size[i];
    sum += ts.bf16[i] ? chunk_sumsq(static_cast<const uint16_t *>(ts.in[i]), e0, e1)
                      : chunk_sumsq(static_cast<const float *>(ts.in[i]), e0, e1);
  }
  sum = block_sum_d(sum, wsum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// STREAM: the outputs bypass the caches
template <class T, bool STREAM>
__device__ __forceinline__ void chunk_scale(const T *p, T *q, int64_t e0, int64_t e1, float f) {
  constexpr int U = kU<T>;
  const int n = (int)(e1 - e0), nu = n / U;
  p += e0;
  q += e0;
  for (int u0 = threadIdx.x; u0 < nu; u0 += 4 * kNT) {
    typename Raw<T>::V r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (u0 + k * kNT < nu) r[k] = load_raw(p + (u0 + k * kNT) * U);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (u0 + k * kNT < nu) {
        float v[U];
        unpack(r[k], v);
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] *= f;
        typename Raw<T>::V *to = reinterpret_cast<typename Raw<T>::V *>(q + (u0 + k * kNT) * U);
        if constexpr (STREAM)
          __builtin_nontemporal_store(pack(v), to);
        else
          *to = pack(v);
      }
  }
  const int e = nu * U + (int)threadIdx.x;
  if (e < n) q[e] = narrow<T>(widen(p[e]) * f);
}

// `parts` doubles from the first pass; workgroup 0 of the first launch writes the norm
template <bool STREAM>
__global__ __launch_bounds__(kNT) void scale_all(Tensors ts, const double *__restrict__ part, int32_t parts,
                                                 float max_norm, float eps, float *__restrict__ norm) {
  __shared__ double wsum[4];
  double sum = 0.0;
  for (int32_t i = threadIdx.x; i < parts; i += kNT) sum += part[i];
  const float v = (float)__dsqrt_rn(block_sum_d(sum, wsum));
  float f = __fdiv_rn(max_norm, v + eps);
  f = f > 1.f ? 1.f : f;
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  const int32_t chunks = ts.first[ts.count];
  for (int32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const int32_t c = chunks - 1 - k;
    const int i = tensor_of(ts, c);
    const int64_t e0 = (int64_t)(c - ts.first[i]) * kChunk;
    const int64_t e1 = e0 + kChunk < ts.size[i] ? e0 + kChunk : ts.size[i];
    if (ts.bf16[i])
      chunk_scale<uint16_t, STREAM>(static_cast<const uint16_t *>(ts.in[i]), static_cast<uint16_t *>(ts.out[i]), e0, e1, f);
    else
      chunk_scale<float, STREAM>(static_cast<const float *>(ts.in[i]), static_cast<float *>(ts.out[i]), e0, e1, f);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int64_t kMaxRowGrid = 1 << 20;

int check_rc(int kind, int64_t R, int64_t C) {
  if (kind != TGEMM_IN_F32 && kind != TGEMM_IN_BF16) return TGEMM_ERR_KIND;
  if (R < 1 || C < 1 || R > INT64_MAX / C / 8 || ceil_div(C, kNT) > INT32_MAX) return TGEMM_ERR_DIM;
  return TGEMM_OK;
}

// whether an output of the lists overlaps another output or another gradient:
// the ranges sorted by address, each compared with the furthest end of the
// outputs (for a gradient) or of all ranges (for an output) before it
bool lists_overlap(const void *const *grads, void *const *outs, const int64_t *sizes, const int32_t *kinds,
                   int64_t count) {
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  std::vector<Range> r;
  r.reserve(2 * count);
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    const uintptr_t b = (uintptr_t)sizes[i] * (kinds[i] == TGEMM_IN_F32 ? 4 : 2);
    r.push_back({(uintptr_t)outs[i], (uintptr_t)outs[i] + b, true});
    if (grads[i] != outs[i]) r.push_back({(uintptr_t)grads[i], (uintptr_t)grads[i] + b, false});
  }
  std::sort(r.begin(), r.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
  uintptr_t all = 0, written = 0;   // furthest ends so far
  for (const Range &x : r) {
    if (x.lo < (x.out ? all : written)) return true;
    if (x.hi > all) all = x.hi;
    if (x.out && x.hi > written) written = x.hi;
  }
  return false;
}

// the tensors g0 .. of a launch, empty ones left out
void fill(Tensors &ts, const void *const *grads, void *const *outs, const int64_t *sizes, const int32_t *kinds,
          int64_t g0, int64_t count) {
  ts.count = 0;
  ts.first[0] = 0;
  for (int64_t i = g0; i < count && i < g0 + kGroup; ++i) {
    if (sizes[i] == 0) continue;
    const int j = ts.count++;
    ts.in[j] = grads[i];
    ts.out[j] = outs[i];
    ts.size[j] = sizes[i];
    ts.bf16[j] = kinds[i] == TGEMM_IN_BF16;
    ts.first[j + 1] = ts.first[j] + (int32_t)ceil_div(sizes[i], kChunk);
  }
}

int done() { return hipGetLastError() == hipSuccess ? TGEMM_OK : TGEMM_ERR_HIP; }


void launch_finish(const float *P, float *out, int64_t rows, int64_t C, hipStream_t stream) {
  launch_columns(C, kFinCols, [&](unsigned grid, int64_t c0) {
    hipLaunchKernelGGL(col_finish, dim3(grid), dim3(kFinT), 0, stream, P, out, nullptr, C, rows, C, c0);
  });
}
// rows of two sums side by side, C columns each (out2 null: of the first alone)
void launch_finish2(const float *P, float *out, float *out2, int64_t rows, int64_t C, hipStream_t stream) {
  const int64_t n = out2 ? 2 * C : C;
  launch_columns(n, kFinCols, [&](unsigned grid, int64_t c0) {
    hipLaunchKernelGGL(col_finish, dim3(grid), dim3(kFinT), 0, stream, P, out, out2, C, rows, n, c0);
  });
}

// W and V of the register kernels, for rows of U to 16384 elements: a wave a
// row while its lanes hold the row in one unit, or, where no column sums take
// registers too, in four and there are rows for four waves a CU (16384x1280
// bf16: 33.6 us, 37.6 with a workgroup a row; its backward pass 46.9 us against
// 38.1); else a workgroup of as many waves as the row fills with the
// fewest units a thread (3456 bf16: 432 units, 7 waves of one, 4% idle lanes;
// four waves of two leave 16% idle).  For the backward passes (`sums`), at most
// 32 rows of one unit a lane go to one workgroup, whose column sums need no
// workspace and no second launch.  That costs the GPU more from 12 rows on, since the
// workgroup's waves add into LDS one after another (norm, 243 f32, in a graph:
// 8 rows 3.8 against 5.0 us, 12 rows 4.9 and 4.9, 27 rows 6.4 and 5.2; epilogue,
// 512 bf16: 8.2 and 6.0 at 12 rows, 11.8 and 6.3 at 27), but it saves the host
// more than that (norm, 243 f32, calls one after another: 10.4 against 15.0 us),
// up to where the GPU takes as long as the host (64 rows: 7.8 us for the norm of
// 243 f32, 16.4 against 14.4 for the epilogue of 512 bf16).
// v 0: the looped kernels.
struct RowPlan {
  int w, v, bt;
  int64_t grid;   // workgroups
};
RowPlan row_plan(int64_t R, int64_t C, int kind, bool sums, bool one_ok = true) {
  const int U = kind == TGEMM_IN_F32 ? kU<float> : kU<uint16_t>;
  RowPlan p = {0, 0, 0, 0};
  const int64_t nu = ceil_div(C, U);
  if (C < U || C > 16384) return p;
  p.w = nu <= 64 || (nu <= 256 && R >= 1024 && !sums) ? 1 : 0;
  p.v = (int)ceil_div(nu, p.w ? 64 : 1024);
  p.bt = p.w ? 256 : 64 * (int)ceil_div(nu, 64 * p.v);
  const bool one = one_ok && sums && nu <= 64 && R <= 32;
  if (one) p.bt = 64 * (int)(R < 16 ? R : 16);
  const int64_t groups = ceil_div(R, p.w ? p.bt / 64 : 1), per_cu = 64 * (sums ? kBwdWaves : kNormWaves) / p.bt;
  int64_t cap = kCUs * (per_cu > 1 ? per_cu : 1);
  // column sums: at least four rows a workgroup, down to two workgroups a CU (a
  // row of P costs as much as half a row: 1782x729 f32, 1280 workgroups 14.3 us,
  // 512 12.1 us)
  const int64_t least = R / 4 > 2 * kCUs ? R / 4 : 2 * kCUs;
  if (sums && cap > least) cap = least;
  p.grid = one ? 1 : groups < cap ? groups : cap;
  return p;
}

// The layer norm's plan: a row's fixed work (the steps of its three reductions,
// its barriers) is done by every wave of it, so past 256 units a row takes the
// fewest waves that its registers allow, of a number that fills the 16 waves of a
// CU with whole rows. bfloat16: two units a thread but where that is six waves (12
// of 16): 16384x3456 70 -> 50 us (with residual and Y 115 -> 98), 8000x7000 84 ->
// 53, 8000x5000 (five waves) equal, 6000x6000 (six) 45 -> 49 and left. float32:
// three units, but two where those are four, seven or eight waves and three would
// be three, five or six.  At one, two and three units: 16384x1280 58, 33 and 29 us, 8000x2000
// 38, 21 and 23, 16384x3456 168, 79 and 93; at two and three past 4096: 8000x5000 79 and
// 50, 6000x7000 68 and 66, 6000x8192 70 and 73, and with a residual alike (8000x5000 106 and
// 101) but for 8000x4100, 81 and 87.
RowPlan ln_plan(int64_t R, int64_t C, int kind) {
  RowPlan p = row_plan(R, C, kind, false);
  const bool f32 = kind == TGEMM_IN_F32;
  const int64_t nu = ceil_div(C, f32 ? kU<float> : kU<uint16_t>);
  if (!p.v || p.w || nu <= 256) return p;
  const int v = !f32 || (nu > 384 && nu <= 512) || (nu > 768 && nu <= 1024) ? 2 : 3;
  const int waves = (int)ceil_div(nu, 64 * v);
  if (v <= p.v || (!f32 && waves == 6)) return p;
  p.v = v;
  p.bt = 64 * waves;
  const int64_t per = kNormWaves / waves, cap = kCUs * (per > 1 ? per : 1);
  p.grid = R < cap ? R : cap;
  return p;
}

// the row kernel K<T, W, V> of a plan
#define ROW_CASE(W, V) \
  case W * 8 + V: hipLaunchKernelGGL((Kernel::template Of<T, W, V>::run), g, b, 0, stream, a); break;
template <class Kernel, class T>
void row_launch(const RowPlan &p, const typename Kernel::Args &a, hipStream_t stream) {
  const dim3 g((unsigned)p.grid), b((unsigned)p.bt);
  switch (p.w * 8 + p.v) {
    ROW_CASE(1, 1) ROW_CASE(0, 1) ROW_CASE(0, 2)
    default: break;
  }
  if constexpr (!Kernel::kSums) {
    switch (p.w * 8 + p.v) {
      ROW_CASE(1, 2) ROW_CASE(1, 3) ROW_CASE(1, 4)
      default: break;
    }
  }
  if constexpr (kU<T> == 4) {   // float32 rows past 8192
    switch (p.w * 8 + p.v) {
      ROW_CASE(0, 3) ROW_CASE(0, 4)
      default: break;
    }
  }
}
#undef ROW_CASE
#define ROW_KERNEL(NAME, SUMS, ARGS, ...)          \
  struct NAME {                                    \
    typedef ARGS Args;                             \
    static constexpr bool kSums = SUMS;            \
    template <class T, int W, int V>               \
    struct Of {                                    \
      static constexpr auto run = __VA_ARGS__;     \
    };                                             \
  };
ROW_KERNEL(NormReg, false, NormArgs, norm_reg<T, W, V>)
ROW_KERNEL(NormBwdReg, true, NormBwdArgs, norm_bwd_reg<T, W, V>)
ROW_KERNEL(EpiBwdPoly, true, EpiBwdArgs, epi_bwd_reg<T, W, V, 0>)
ROW_KERNEL(EpiBwdSigm, true, EpiBwdArgs, epi_bwd_reg<T, W, V, 1>)
ROW_KERNEL(LnReg, false, LnArgs, ln_reg<T, W, V>)
ROW_KERNEL(LnBwdReg, true, LnBwdArgs, ln_bwd_reg<T, W, V>)
ROW_KERNEL(GatedBwdPoly, true, GatedBwdArgs, gated_bwd_reg<T, W, V, 0>)
ROW_KERNEL(GatedBwdSigm, true, GatedBwdArgs, gated_bwd_reg<T, W, V, 1>)
ROW_KERNEL(LnBwdOne, true, LnBwdArgs, ln_bwd_reg<T, W, V, true>)
ROW_KERNEL(GatedBwdPolyOne, true, GatedBwdArgs, gated_bwd_reg<T, W, V, 0, true>)
ROW_KERNEL(GatedBwdSigmOne, true, GatedBwdArgs, gated_bwd_reg<T, W, V, 1, true>)
#undef ROW_KERNEL
template <class Kernel>
void row_launch(int kind, const RowPlan &p, const typename Kernel::Args &a, hipStream_t stream) {
  if (kind == TGEMM_IN_F32)
    row_launch<Kernel, float>(p, a, stream);
  else
    row_launch<Kernel, uint16_t>(p, a, stream);
}

// The passes with two column sums: their plan is row_plan's but for few rows, which
// one workgroup takes (write_cols_one), up to three units a lane in float32 and two
// in bfloat16.  (Its sixteen waves leave a lane 128 registers: at these largest widths the
// gated pass spills 19 to 24 of them, and the norm's bfloat16 one 2.)  That saves the
// second launch and the workspace: the
// norm, 27x729 f32, 11.4 against 15.9 us a call (8.3 against 5.6 in a graph), 27x243
// 11.4 and 16.0 (4.5 and 6.4), 32x1000 bf16 13.5 and 16.1 (10.9 and 6.1).  The gated
// pass has several times the instructions, and one CU for all of them: past two units
// a lane in float32 and one in bfloat16 it is so up to 16 rows, where the GPU takes as
// long as the host (16x729 f32 12.8 us a call against 17.0, 12.4 against 5.9 in a graph;
// 27 rows 14.9 and 15.2, 32 rows 17.3 and 17.6).  Without dbias there is no second
// launch and no workspace to save, and a few rows are as many workgroups' (in a graph,
// 16x729 f32 3.2 us against 9.8, 32x500 bf16 3.3 against 7.6).
bool one_ok(int64_t R, int64_t C, int kind, bool gated) {
  const bool f32 = kind == TGEMM_IN_F32;
  const int64_t U = f32 ? kU<float> : kU<uint16_t>, units = ceil_div(C, U);
  if (C < U || units > (f32 ? 192 : 128)) return false;
  return R <= (gated && units > (f32 ? 128 : 64) ? 16 : 32);
}
template <class Kernel, class T>
void one_launch(int64_t R, int64_t C, const typename Kernel::Args &a, hipStream_t stream) {
  const dim3 g(1), b((unsigned)(64 * (R < kOneGroups ? R : kOneGroups)));
  switch (ceil_div(ceil_div(C, kU<T>), 64)) {
    case 1: hipLaunchKernelGGL((Kernel::template Of<T, 1, 1>::run), g, b, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((Kernel::template Of<T, 1, 2>::run), g, b, 0, stream, a); break;
    default:
      if constexpr (kU<T> == 4) hipLaunchKernelGGL((Kernel::template Of<T, 1, 3>::run), g, b, 0, stream, a);
      break;
  }
}
template <class Kernel>
void one_launch(int kind, int64_t R, int64_t C, const typename Kernel::Args &a, hipStream_t stream) {
  if (kind == TGEMM_IN_F32)
    one_launch<Kernel, float>(R, C, a, stream);
  else
    one_launch<Kernel, uint16_t>(R, C, a, stream);
}
int64_t two_sums_ws_bytes(int64_t R, int64_t C, bool gated) {
  int64_t rows = 0;
  for (const int kind : {TGEMM_IN_F32, TGEMM_IN_BF16}) {
    const RowPlan p = row_plan(R, C, kind, true);
    const int64_t n = one_ok(R, C, kind, gated) ? 0 : p.v == 0 ? strips_of(R) : p.grid;
    rows = n > rows ? n : rows;
  }
  return 4 * rows * 2 * C;
}

// bytes of P for either kind: a row for each workgroup of the row kernel, or
// each strip of the looped kernels; none where one workgroup takes every row
int64_t col_ws_bytes(int64_t R, int64_t C) {
  int64_t rows = 0;
  for (const int kind : {TGEMM_IN_F32, TGEMM_IN_BF16}) {
    const RowPlan p = row_plan(R, C, kind, true);
    const int64_t n = p.v == 0 ? strips_of(R) : p.grid > 1 ? p.grid : 0;
    rows = n > rows ? n : rows;
  }
  return 4 * rows * C;
}
template <class T, bool NORM>
void launch_cols(const T *A, const T *B, const float *rstd, int act, float *P, float *out, int64_t R, int64_t C,
                 hipStream_t stream) {
  const int64_t strip = ceil_div(R, strips_of(R)), strips = ceil_div(R, strip);
  launch_columns(C, kNT, [&](unsigned grid, int64_t c0) {
    hipLaunchKernelGGL((col_sums<T, NORM>), dim3(grid, (unsigned)strips), dim3(kNT), 0, stream, A, B, rstd, act, P, R, C,
                       strip, c0);
  });
  launch_finish(P, out, strips, C, stream);
}

template <class T, bool NORM>
void launch_cols2(Cols2Args k, float *out, float *out2, hipStream_t stream) {
  k.pitch = out2 ? 2 * k.C : k.C;
  k.strip = ceil_div(k.R, strips_of(k.R));
  const int64_t strips = ceil_div(k.R, k.strip);
  launch_columns(k.C, kNT, [&](unsigned grid, int64_t c0) {
    k.c0 = c0;
    hipLaunchKernelGGL((col_sums2<T, NORM>), dim3(grid, (unsigned)strips), dim3(kNT), 0, stream, k);
  });
  launch_finish2(k.P, out, out2, strips, k.C, stream);
}
template <bool NORM>
void launch_cols2(int kind, const Cols2Args &k, float *out, float *out2, hipStream_t stream) {
  if (kind == TGEMM_IN_F32)
    launch_cols2<float, NORM>(k, out, out2, stream);
  else
    launch_cols2<uint16_t, NORM>(k, out, out2, stream);
}

}  // namespace

extern "C" {

int ternary_rmsnorm_quantize(const void *X, int in_kind, const void *residual, const float *gain, float eps, void *H,
                             void *Y, float *rstd, int8_t *Q, float *scale, int64_t R, int64_t C, hipStream_t stream) {
  if (!X || !gain || !Q || !scale || (residual && !H)) return TGEMM_ERR_NULL;
  const int st = check_rc(in_kind, R, C);
  if (st != TGEMM_OK) return st;
  if (!(eps >= 0.f && eps < __builtin_inff())) return TGEMM_ERR_VALUE;
  if (!residual) H = nullptr;
  const int64_t n = R * C, xb = n * (in_kind == TGEMM_IN_F32 ? 4 : 2);
  const Buf outs[] = {{H, xb}, {Y, xb}, {rstd, 4 * R}, {Q, n}, {scale, 4 * R}};
  const Buf ins[] = {{X, xb}, {residual, xb}, {gain, 4 * C}};
  const void *const same[5][2] = {{X, residual}};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  const NormArgs a = {X, residual, gain, H, Y, rstd, scale, Q, eps, R, C};
  const RowPlan p = row_plan(R, C, in_kind, false);
  if (p.v) {
    row_launch<NormReg>(in_kind, p, a, stream);
    return done();
  }
  const dim3 g((unsigned)(R < kMaxRowGrid ? R : kMaxRowGrid));
  if (in_kind == TGEMM_IN_F32)
    hipLaunchKernelGGL(norm_rows<float>, g, dim3(kNT), 0, stream, a);
  else
    hipLaunchKernelGGL(norm_rows<uint16_t>, g, dim3(kNT), 0, stream, a);
  return done();
}

int ternary_rmsnorm_backward_workspace(int64_t R, int64_t C, int64_t *bytes) {
  if (!bytes) return TGEMM_ERR_NULL;
  const int st = check_rc(TGEMM_IN_F32, R, C);
  if (st != TGEMM_OK) return st;
  *bytes = col_ws_bytes(R, C);
  return TGEMM_OK;
}

int ternary_rmsnorm_backward(const void *dY, const void *H, int in_kind, const float *gain, const float *rstd,
                             const void *dH, void *dX, float *dgain, int64_t R, int64_t C, void *workspace,
                             int64_t workspace_bytes, hipStream_t stream) {
  if (!dY || !H || !gain || !rstd || !dX || !dgain) return TGEMM_ERR_NULL;
  const int st = check_rc(in_kind, R, C);
  if (st != TGEMM_OK) return st;
  const int64_t wb = col_ws_bytes(R, C);
  if (!workspace_ok(workspace, workspace_bytes, wb)) return TGEMM_ERR_WORKSPACE;
  const int64_t xb = R * C * (in_kind == TGEMM_IN_F32 ? 4 : 2);
  const Buf outs[] = {{dX, xb}, {dgain, 4 * C}, {workspace, workspace_bytes > 0 ? workspace_bytes : 0}};
  const Buf ins[] = {{dY, xb}, {H, xb}, {gain, 4 * C}, {rstd, 4 * R}, {dH, xb}};
  const void *const same[3][2] = {{dH, dH}};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  float *P = static_cast<float *>(workspace);
  NormBwdArgs a = {dY, H, gain, rstd, dH, dX, P, R, C};
  const RowPlan p = row_plan(R, C, in_kind, true);
  if (p.v) {
    if (p.grid == 1) a.P = dgain;
    row_launch<NormBwdReg>(in_kind, p, a, stream);
    if (p.grid > 1) launch_finish(P, dgain, p.grid, C, stream);
    return done();
  }
  const dim3 g((unsigned)(R < kMaxRowGrid ? R : kMaxRowGrid));
  if (in_kind == TGEMM_IN_F32) {
    hipLaunchKernelGGL(norm_bwd_rows<float>, g, dim3(kNT), 0, stream, a);
    launch_cols<float, true>(static_cast<const float *>(dY), static_cast<const float *>(H), rstd, 0, P, dgain, R, C,
                             stream);
  } else {
    hipLaunchKernelGGL(norm_bwd_rows<uint16_t>, g, dim3(kNT), 0, stream, a);
    launch_cols<uint16_t, true>(static_cast<const uint16_t *>(dY), static_cast<const uint16_t *>(H), rstd, 0, P, dgain,
                                R, C, stream);
  }
  return done();
}

int ternary_epilogue_backward_workspace(int64_t R, int64_t C, int64_t *bytes) {
  return ternary_rmsnorm_backward_workspace(R, C, bytes);
}

int ternary_epilogue_backward(const void *dY, const void *Z, int in_kind, int act, void *dZ, float *dbias, int8_t *Q,
                              float *scale, int64_t R, int64_t C, void *workspace, int64_t workspace_bytes,
                              hipStream_t stream) {
  if (!dY || !Z || !dZ || !Q || !scale) return TGEMM_ERR_NULL;
  const int st = check_rc(in_kind, R, C);
  if (st != TGEMM_OK) return st;
  if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_VALUE;
  const int64_t wb = dbias ? col_ws_bytes(R, C) : 0;
  if (!workspace_ok(workspace, workspace_bytes, wb)) return TGEMM_ERR_WORKSPACE;
  const int64_t n = R * C, xb = n * (in_kind == TGEMM_IN_F32 ? 4 : 2);
  const Buf outs[] = {{dZ, xb}, {dbias, 4 * C}, {Q, n}, {scale, 4 * R}, {workspace, workspace_bytes > 0 ? workspace_bytes : 0}};
  const Buf ins[] = {{dY, xb}, {Z, xb}};
  const void *const same[5][2] = {};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  float *P = static_cast<float *>(workspace);
  EpiBwdArgs a = {dY, Z, dZ, Q, scale, dbias ? P : nullptr, R, C, act};
  const RowPlan p = row_plan(R, C, in_kind, true);
  if (p.v) {
    if (p.grid == 1) a.P = dbias;
    if (is_sigm(act))
      row_launch<EpiBwdSigm>(in_kind, p, a, stream);
    else
      row_launch<EpiBwdPoly>(in_kind, p, a, stream);
    if (dbias && p.grid > 1) launch_finish(P, dbias, p.grid, C, stream);
    return done();
  }
  const dim3 g((unsigned)(R < kMaxRowGrid ? R : kMaxRowGrid));
  if (in_kind == TGEMM_IN_F32) {
    hipLaunchKernelGGL(epi_bwd_rows<float>, g, dim3(kNT), 0, stream, a);
    if (dbias)
      launch_cols<float, false>(static_cast<const float *>(dY), static_cast<const float *>(Z), nullptr, act, P, dbias,
                                R, C, stream);
  } else {
    hipLaunchKernelGGL(epi_bwd_rows<uint16_t>, g, dim3(kNT), 0, stream, a);
    if (dbias)
      launch_cols<uint16_t, false>(static_cast<const uint16_t *>(dY), static_cast<const uint16_t *>(Z), nullptr, act,
                                   P, dbias, R, C, stream);
  }
  return done();
}

int ternary_layernorm_quantize(const void *X, int in_kind, const void *residual, const float *gain, const float *beta,
                               float eps, void *H, void *Y, float *mean, float *rstd, int8_t *Q, float *scale, int64_t R,
                               int64_t C, hipStream_t stream) {
  if (!X || !gain || !Q || !scale || (residual && !H) || !mean != !rstd) return TGEMM_ERR_NULL;
  const int st = check_rc(in_kind, R, C);
  if (st != TGEMM_OK) return st;
  if (!(eps >= 0.f && eps < __builtin_inff())) return TGEMM_ERR_VALUE;
  if (!residual) H = nullptr;
  const int64_t n = R * C, xb = n * (in_kind == TGEMM_IN_F32 ? 4 : 2);
  const Buf outs[] = {{H, xb}, {Y, xb}, {mean, 4 * R}, {rstd, 4 * R}, {Q, n}, {scale, 4 * R}};
  const Buf ins[] = {{X, xb}, {residual, xb}, {gain, 4 * C}, {beta, 4 * C}};
  const void *const same[6][2] = {{X, residual}};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  const LnArgs a = {X, residual, gain, beta, H, Y, mean, rstd, scale, Q, eps, R, C, (double)C, 1. / (double)C};
  const RowPlan p = ln_plan(R, C, in_kind);
  if (p.v) {
    row_launch<LnReg>(in_kind, p, a, stream);
    return done();
  }
  const dim3 g((unsigned)(R < kMaxRowGrid ? R : kMaxRowGrid));
  if (in_kind == TGEMM_IN_F32)
    hipLaunchKernelGGL(ln_rows<float>, g, dim3(kNT), 0, stream, a);
  else
    hipLaunchKernelGGL(ln_rows<uint16_t>, g, dim3(kNT), 0, stream, a);
  return done();
}

int ternary_layernorm_backward_workspace(int64_t R, int64_t C, int64_t *bytes) {
  if (!bytes) return TGEMM_ERR_NULL;
  const int st = check_rc(TGEMM_IN_F32, R, C);
  if (st != TGEMM_OK) return st;
  *bytes = two_sums_ws_bytes(R, C, false);
  return TGEMM_OK;
}

int ternary_layernorm_backward(const void *dY, const void *H, int in_kind, const float *gain, const float *mean,
                               const float *rstd, const void *dH, void *dX, float *dgain, float *dbeta, int64_t R,
                               int64_t C, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!dY || !H || !gain || !mean || !rstd || !dX || !dgain) return TGEMM_ERR_NULL;
  const int st = check_rc(in_kind, R, C);
  if (st != TGEMM_OK) return st;
  if (!workspace_ok(workspace, workspace_bytes, two_sums_ws_bytes(R, C, false))) return TGEMM_ERR_WORKSPACE;
  const int64_t xb = R * C * (in_kind == TGEMM_IN_F32 ? 4 : 2);
  const Buf outs[] = {{dX, xb}, {dgain, 4 * C}, {dbeta, 4 * C}, {workspace, workspace_bytes > 0 ? workspace_bytes : 0}};
  const Buf ins[] = {{dY, xb}, {H, xb}, {gain, 4 * C}, {mean, 4 * R}, {rstd, 4 * R}, {dH, xb}};
  const void *const same[4][2] = {{dH, dH}};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  float *P = static_cast<float *>(workspace);
  LnBwdArgs a = {dY, H, gain, mean, rstd, dH, dX, P, dbeta ? P + C : nullptr, dbeta ? 2 * C : C, R, C};
  if (one_ok(R, C, in_kind, false)) {
    a.P = dgain;
    a.P2 = dbeta;
    one_launch<LnBwdOne>(in_kind, R, C, a, stream);
    return done();
  }
  const RowPlan p = row_plan(R, C, in_kind, true);
  if (p.v) {
    row_launch<LnBwdReg>(in_kind, p, a, stream);
    launch_finish2(P, dgain, dbeta, p.grid, C, stream);
    return done();
  }
  const dim3 g((unsigned)(R < kMaxRowGrid ? R : kMaxRowGrid));
  if (in_kind == TGEMM_IN_F32)
    hipLaunchKernelGGL(ln_bwd_rows<float>, g, dim3(kNT), 0, stream, a);
  else
    hipLaunchKernelGGL(ln_bwd_rows<uint16_t>, g, dim3(kNT), 0, stream, a);
  launch_cols2<true>(in_kind, {dY, H, mean, rstd, P, 0, R, C, 0, 0, 0}, dgain, dbeta, stream);
  return done();
}

int ternary_gated_backward_workspace(int64_t R, int64_t C, int64_t *bytes) {
  if (!bytes) return TGEMM_ERR_NULL;
  const int st = check_rc(TGEMM_IN_F32, R, C);
  if (st != TGEMM_OK) return st;
  *bytes = two_sums_ws_bytes(R, C, true);
  return TGEMM_OK;
}

int ternary_gated_backward(const void *dY, const void *Z, int in_kind, int act, float gate_scale, float up_scale,
                           void *dZ, float *dbias, int8_t *Q, float *scale, int64_t R, int64_t C, void *workspace,
                           int64_t workspace_bytes, hipStream_t stream) {
  if (!dY || !Z || !dZ || !Q || !scale) return TGEMM_ERR_NULL;
  const int st = check_rc(in_kind, R, C);
  if (st != TGEMM_OK) return st;
  if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_VALUE;
  const int64_t wb = dbias ? two_sums_ws_bytes(R, C, true) : 0;
  if (!workspace_ok(workspace, workspace_bytes, wb)) return TGEMM_ERR_WORKSPACE;
  const int64_t n = R * C, xb = n * (in_kind == TGEMM_IN_F32 ? 4 : 2);
  const Buf outs[] = {{dZ, 2 * xb}, {dbias, 8 * C}, {Q, 2 * n}, {scale, 4 * R},
                      {workspace, workspace_bytes > 0 ? workspace_bytes : 0}};
  const Buf ins[] = {{dY, xb}, {Z, 2 * xb}};
  const void *const same[5][2] = {};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  float *P = static_cast<float *>(workspace);
  GatedBwdArgs a = {dY, Z, dZ, Q, scale, dbias ? P : nullptr, gate_scale, up_scale, R, C, act};
  if (dbias && one_ok(R, C, in_kind, true)) {
    a.P = dbias;
    if (is_sigm(act))
      one_launch<GatedBwdSigmOne>(in_kind, R, C, a, stream);
    else
      one_launch<GatedBwdPolyOne>(in_kind, R, C, a, stream);
    return done();
  }
  const RowPlan p = row_plan(R, C, in_kind, true, dbias != nullptr);
  if (p.v) {
    if (is_sigm(act))
      row_launch<GatedBwdSigm>(in_kind, p, a, stream);
    else
      row_launch<GatedBwdPoly>(in_kind, p, a, stream);
    if (dbias) launch_finish(P, dbias, p.grid, 2 * C, stream);
    return done();
  }
  const dim3 g((unsigned)(R < kMaxRowGrid ? R : kMaxRowGrid));
  if (in_kind == TGEMM_IN_F32)
    hipLaunchKernelGGL(gated_bwd_rows<float>, g, dim3(kNT), 0, stream, a);
  else
    hipLaunchKernelGGL(gated_bwd_rows<uint16_t>, g, dim3(kNT), 0, stream, a);
  if (dbias) launch_cols2<false>(in_kind, {dY, Z, nullptr, nullptr, P, 0, R, C, 0, act, 0}, dbias, dbias + C, stream);
  return done();
}

int ternary_clip_grad_norm_workspace(const int64_t *sizes, int64_t count, int64_t *bytes) {
  if (!sizes || !bytes) return TGEMM_ERR_NULL;
  if (count < 1) return TGEMM_ERR_DIM;
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > INT64_MAX / 16) return TGEMM_ERR_DIM;
    chunks += ceil_div(sizes[i], kChunk);
    if (chunks > INT32_MAX) return TGEMM_ERR_DIM;
  }
  const int64_t launches = ceil_div(count, kGroup);
  *bytes = 8 * ((chunks < kMaxParts ? chunks : kMaxParts) + launches + 1);
  return TGEMM_OK;
}

int ternary_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *sizes, const int32_t *kinds,
                           int64_t count, float max_norm, float eps, float *norm, void *workspace,
                           int64_t workspace_bytes, hipStream_t stream) {
  if (!grads || !outs || !sizes || !kinds || !norm) return TGEMM_ERR_NULL;
  int64_t need = 0;
  const int st = ternary_clip_grad_norm_workspace(sizes, count, &need);
  if (st != TGEMM_OK) return st;
  for (int64_t i = 0; i < count; ++i) {
    if (kinds[i] != TGEMM_IN_F32 && kinds[i] != TGEMM_IN_BF16) return TGEMM_ERR_KIND;
    if (sizes[i] > 0 && (!grads[i] || !outs[i])) return TGEMM_ERR_NULL;
  }
  if (!(max_norm >= 0.f) || !(eps >= 0.f)) return TGEMM_ERR_VALUE;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return TGEMM_ERR_WORKSPACE;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    const int64_t b = sizes[i] * (kinds[i] == TGEMM_IN_F32 ? 4 : 2);
    if (overlap(outs[i], b, norm, 4) || overlap(outs[i], b, workspace, need) || overlap(grads[i], b, norm, 4) ||
        overlap(grads[i], b, workspace, need) || (outs[i] != grads[i] && overlap(outs[i], b, grads[i], b)))
      return TGEMM_ERR_ALIAS;
  }
  try {
    if (lists_overlap(grads, outs, sizes, kinds, count)) return TGEMM_ERR_ALIAS;
  } catch (...) {
    return TGEMM_ERR_DIM;   // more gradients than the host can list
  }
  if (overlap(norm, 4, workspace, need)) return TGEMM_ERR_ALIAS;
  double *part = static_cast<double *>(workspace);
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) total += ceil_div(sizes[i], kChunk);
  // the first pass forwards, the second backwards over the launches too
  int64_t parts = 0;
  Tensors ts;
  for (int64_t g0 = 0; g0 < count; g0 += kGroup) {
    fill(ts, grads, outs, sizes, kinds, g0, count);
    const int64_t chunks = ts.first[ts.count], share = kMaxParts * chunks / (total ? total : 1);
    if (chunks == 0) continue;
    const int64_t grid = chunks < kMaxParts && total <= kMaxParts ? chunks : share > 1 ? share : 1;
    hipLaunchKernelGGL(sumsq, dim3((unsigned)grid), dim3(kNT), 0, stream, ts, part + parts);
    parts += grid;
  }
  int64_t bytes = 0;
  for (int64_t i = 0; i < count; ++i) bytes += sizes[i] * (kinds[i] == TGEMM_IN_F32 ? 4 : 2);
  const bool big = bytes > kStreamBytes;
  bool first = true;
  for (int64_t g0 = (count - 1) / kGroup * kGroup; g0 >= 0; g0 -= kGroup) {
    if (count > kGroup || total == 0) fill(ts, grads, outs, sizes, kinds, g0, count);
    const int64_t chunks = ts.first[ts.count];
    if (chunks == 0 && !(first && g0 == 0)) continue;
    const int64_t cap = kCUs * 8, grid = chunks < 1 ? 1 : chunks < cap ? chunks : cap;
    hipLaunchKernelGGL(big ? scale_all<true> : scale_all<false>, dim3((unsigned)grid), dim3(kNT), 0, stream, ts, part,
                       (int32_t)parts, max_norm, eps, first ? norm : nullptr);
    first = false;
  }
  return done();
}

}  // extern "C"
