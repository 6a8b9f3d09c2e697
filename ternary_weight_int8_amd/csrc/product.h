// product.h -- what the kernels of the int8 products share: loads straight into
// LDS, the decoding of stored weights, the order of the tiles, and the output's
// scales and epilogues.
#ifndef TERNARY_PRODUCT_H
#define TERNARY_PRODUCT_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ternary_gemm.h"

namespace {

typedef int32_t v4i __attribute__((ext_vector_type(4)));

// Workgroup barrier for LDS only: waits for this wave's LDS operations, not
// for its outstanding global loads (which __syncthreads() would also drain,
// defeating the prefetch).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Loads straight into LDS.  They come from inline assembly, so the compiler
// does not drain them at every LDS read; a kernel waits for its own by count
// (memory operations of a wave complete in issue order).
// 16 bytes per lane from sbase + voff into LDS at lds + 16 * lane
__device__ __forceinline__ void dma16(uint32_t lds, uint32_t voff, const void *sbase) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"s"(lds), "v"(voff), "s"(sbase) : "memory", "m0");
}
// 4 bytes per lane from sbase + voff into LDS at lds + 4 * lane
__device__ __forceinline__ void dma4(uint32_t lds, uint32_t voff, const void *sbase) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               ::"s"(lds), "v"(voff), "s"(sbase) : "memory", "m0");
}
// wait until at most N of this wave's memory operations are in flight
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// the same, then this wave's LDS operations, then meet the other waves
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Byte c of this word is the int8 weight of code c: 00, 01, FF, 00, i.e.
// (c & 1) - ((c >> 1) & 1) [P10425 "What this adds"; P10855 PR body].
constexpr uint32_t kCodeTable = 0x00FF0100u;

// ---------------------------------------------------------------------------
// The output of a call: the int32 sums as computed, or the sums scaled into
// f32 or bf16 (the dequantization step that follows the integer product:
// activations quantized per row for the forward and dX, X and dY per column
// for dW [P10855 PR body]).  A scaled element is
//     y = (float(acc) * rs[row]) * cs[col]          (cs null: cscal)
// with the int32 -> float conversion and each product rounded to nearest-even
// in IEEE single precision, in that order; bf16 output then rounds y to the
// nearest bf16, ties to even (v_cvt_pk_bf16_f32; a NaN stays a NaN).
// ---------------------------------------------------------------------------
constexpr float kGeluA = 1.5957691216057308f;              // 2 sqrt(2 / pi)
constexpr float kGeluAB = 1.5957691216057308f * 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;
enum OutKind { OUT_I32 = 0, OUT_F32 = TGEMM_OUT_F32, OUT_BF16 = TGEMM_OUT_BF16 };
static_assert(OUT_F32 != OUT_I32 && OUT_BF16 != OUT_I32 && OUT_F32 != OUT_BF16, "output kinds");

struct Out {
  void *ptr;          // [R][Cc] elements of the kind
  const float *rs;    // per output row (scaled kinds)
  const float *cs;    // per output column, or null: cscal for every column
  float cscal;
  int32_t kind;       // OutKind
  int32_t vec;        // Cc % 4 == 0 and ptr aligned to 4 elements: 4-element stores
  int32_t vec8;       // bf16, Cc % 8 == 0 and ptr 16-byte aligned: 8-element stores
  // the epilogue's (Epi below; unused by the plain and scaled calls)
  const float *bias;  // per output column, or null
  const void *res;    // [R][Cc] elements of the kind, or null
  void *z;            // [R][Cc] elements of the kind, or null
  int32_t act;        // TGEMM_ACT_*
  float cscal2;       // EPI_GATED: the up projection's scale (cscal is the gate's)
};

// What the stores of a kernel compute: EPI_NONE the int32 sums or their
// scaled form; the other two the epilogue of ternary_gemm_s8_epilogue on the
// scaled sum y, in single precision up to the rounding of what is stored,
//     z = y + bias[col],   Y = act(z) + res[row][col]
// with z itself stored too if asked for.  The activations are split in two
// kinds so that a kernel's unrolled stores hold the code of one kind only:
// EPI_POLY   none, relu, relu2: a comparison and a product
// EPI_SIGM   z sigmoid(u(z)), u = z (silu) or a z + b z^3 (gelu's tanh form,
//            0.5 (1 + tanh(t)) = sigmoid(2 t))
// Two flags say where a kernel's epilogue takes its scales from, and what its
// columns are:
// EPI_COLS   a scale per column (o.cs, or 1 for every column where it is null)
//            in place of o.cscal
// EPI_GATED  columns 2 c and 2 c + 1 of the product are the gate and the up
//            projection of output column c (Gated, below)
enum Epi { EPI_NONE = 0, EPI_POLY = 1, EPI_SIGM = 2, EPI_COLS = 4, EPI_GATED = 8 };
constexpr int kEpiAct = 3;   // the bits of the activation's kind
int epi_of(int act) { return act == TGEMM_ACT_SILU || act == TGEMM_ACT_GELU_TANH ? EPI_SIGM : EPI_POLY; }

__device__ __forceinline__ float scaled(int32_t x, float r, float c) {
  return __fmul_rn(__fmul_rn((float)x, r), c);
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// two floats -> two bf16 (round to nearest even) packed low, high
__device__ __forceinline__ uint32_t bf16_pack(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}

// Element-aligned vectors: the epilogue's loads and stores take any width and
// any base (gfx950 serves unaligned global accesses), so a row of an odd
// number of columns still moves four elements at a time.
typedef float v4f_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t v2u_u __attribute__((ext_vector_type(2), aligned(2)));

template <int E>
__device__ __forceinline__ float epi_act(float z, int act) {
#pragma clang fp contract(off)   // every kernel rounds alike
  if constexpr ((E & kEpiAct) == EPI_POLY) {
    if (act == TGEMM_ACT_NONE) return z;
    const float p = z < 0.f ? 0.f : z;   // a NaN stays one
    return act == TGEMM_ACT_RELU ? p : p * p;
  } else {
    // sigmoid(u) = 1 / (1 + 2^t), t = -u log2(e), by the hardware's 2^t and
    // reciprocal (within 1 ulp each; libm's expf and the IEEE divide made the
    // unrolled stores spill).  Rounding t leaves a relative error of about
    // |t| 2^-24 in 2^t, as rounding u does.  Past +-200 the sigmoid is 0 or 1
    // in single precision; the clamp keeps t finite, and the product with z
    // brings back a NaN that it drops.
    const bool silu = act == TGEMM_ACT_SILU;
    const float k0 = silu ? -kLog2e : -kGeluA * kLog2e, k1 = silu ? 0.f : -kGeluAB * kLog2e;
    const float c = __builtin_amdgcn_fmed3f(z, -200.f, 200.f);
    const float t = c * __builtin_fmaf(k1, c * c, k0);
    return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t));
  }
}

__device__ __forceinline__ void store4(void *base, int32_t kind, int64_t e, const float (&y)[4]) {
  if (kind == OUT_F32)
    *reinterpret_cast<v4f_u *>(static_cast<float *>(base) + e) = v4f_u{y[0], y[1], y[2], y[3]};
  else
    *reinterpret_cast<v2u_u *>(static_cast<uint16_t *>(base) + e) = v2u_u{bf16_pack(y[0], y[1]), bf16_pack(y[2], y[3])};
}
__device__ __forceinline__ void store1(void *base, int32_t kind, int64_t e, float y) {
  if (kind == OUT_F32)
    static_cast<float *>(base)[e] = y;
  else
    static_cast<uint16_t *>(base)[e] = __builtin_bit_cast(uint16_t, (__bf16)y);
}

template <int E>
__device__ __forceinline__ float col_scale(const Out &o, int64_t col) {
  if constexpr (E & EPI_COLS) return o.cs ? o.cs[col] : 1.f;
  return o.cscal;
}

// the epilogue of one element, and of four neighbours of a row
template <int E>
__device__ __forceinline__ void epi_put1(const Out &o, int64_t Cc, int64_t row, int64_t col, int32_t x, float r) {
#pragma clang fp contract(off)   // every kernel rounds alike
  const int64_t e = row * Cc + col;
  float z = scaled(x, r, col_scale<E>(o, col));
  if (o.bias) z += o.bias[col];
  if (o.z) store1(o.z, o.kind, e, z);
  float y = epi_act<E>(z, o.act);
  if (o.res)
    y += o.kind == OUT_F32 ? static_cast<const float *>(o.res)[e]
                           : __uint_as_float((uint32_t)static_cast<const uint16_t *>(o.res)[e] << 16);
  store1(o.ptr, o.kind, e, y);
}
template <int E>
__device__ __forceinline__ void epi_put4(const Out &o, int64_t Cc, int64_t row, int64_t col, const v4i &v, float r) {
#pragma clang fp contract(off)   // every kernel rounds alike
  const int64_t e = row * Cc + col;
  float y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = scaled(v[k], r, col_scale<E>(o, col + k));
  if (o.bias) {
    const v4f_u b = *reinterpret_cast<const v4f_u *>(o.bias + col);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] += b[k];
  }
  if (o.z) store4(o.z, o.kind, e, y);
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = epi_act<E>(y[k], o.act);
  if (o.res) {
    if (o.kind == OUT_F32) {
      const v4f_u x = *reinterpret_cast<const v4f_u *>(static_cast<const float *>(o.res) + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] += x[k];
    } else {
      const v2u_u x = *reinterpret_cast<const v2u_u *>(static_cast<const uint16_t *>(o.res) + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] += __uint_as_float(k & 1 ? x[k / 2] & 0xFFFF0000u : x[k / 2] << 16);
    }
  }
  store4(o.ptr, o.kind, e, y);
}

// The epilogue of a wave's FM x FN fragments, four fragments of a row at a
// time (a whole row of them spilled).  Each pass is straight-line code; what
// depends on the arguments (bias, Z, residual) is decided once a pass, not once
// an element: with the decisions inside the unrolled elements, the code was
// over 100 KB and ran 16384x3456x1280 with gelu in 120 us.  It takes 111 us now,
// 84 us without activation and Z: 21 us a tile for the products as in the plain
// forward, and per wave and tile 144 elements of some 17 vector instructions,
// which no MFMA covers, since the CU's waves reach their tiles' ends together.
// Lane moves issued a run ahead spilled (117 us), and two workgroups of 256 x
// 144 a CU, which drift apart, took 123 us.
//   0  lanes: from the MFMA layout (lane l: row l % 16, columns 4 (l / 16) ..
//      + 3) to four neighbouring lanes a row, by ds_bpermute.  float32: 16
//      bytes a lane, 64 a row.  bfloat16: fragments in pairs, first exchanged
//      between lane groups (permlane32_swap, permlane16_swap: group g then
//      holds columns 8 g .. + 3 of the pair's 32 in the first register set, 8 g
//      + 4 .. + 7 in the second), so that a lane has 8 columns, 16 bytes, and
//      a row 64; an odd last fragment has 8 bytes a lane
//   1  z = scaled sum + bias;  2  Z;  3  the activation;  4  + residual;  5  Y
// GUARD: the tile reaches past the output's last row or column.
typedef uint32_t v4u_u __attribute__((ext_vector_type(4), aligned(2)));

// fragments F0 .. F0 + N - 1 of fragment row i; `row` is the lane's output row
template <int E, bool BF, bool GUARD, int F0, int N, int FN>
__device__ __forceinline__ void epi_run(const Out &o, int64_t Cc, const v4i (&acc)[FN], int64_t row, bool in,
                                        int64_t c0, int lane, float rs) {
#pragma clang fp contract(off)   // every kernel rounds alike
  constexpr int kKind = BF ? OUT_BF16 : OUT_F32;
  constexpr int kPairs = BF ? N / 2 : 0;           // fragments 2 k, 2 k + 1 for k < kPairs
  asm volatile("" : "+v"(lane));   // columns and masks anew in each run: kept over all of them they spilled
  const int p = lane & 3, src = 4 * ((lane >> 2) + 16 * p);
  auto col_of = [&](int jj) -> int64_t {           // first of the four columns in register set jj
    return c0 + 16 * F0 + (jj < 2 * kPairs ? 32 * (jj / 2) + 8 * p + 4 * (jj & 1) : 16 * jj + 4 * p);
  };
  float y[N][4];
  auto store = [&](void *base) {
    if (!in) return;
#pragma unroll
    for (int jj = 0; jj < N; ++jj) {
      const int64_t col = col_of(jj), at = row * Cc + col;
      const bool pair = BF && jj < 2 * kPairs;
      if (pair && !(jj & 1) && (!GUARD || col + 7 < Cc)) {
        const float(&w)[4] = y[jj + 1 < N ? jj + 1 : jj];
        *reinterpret_cast<v4u_u *>(static_cast<uint16_t *>(base) + at) =
            v4u_u{bf16_pack(y[jj][0], y[jj][1]), bf16_pack(y[jj][2], y[jj][3]), bf16_pack(w[0], w[1]),
                  bf16_pack(w[2], w[3])};
      } else if (pair && (jj & 1) && (!GUARD || col + 3 < Cc)) {
        // went with the set before it
      } else if (!GUARD || col + 3 < Cc) {
        store4(base, kKind, at, y[jj]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < Cc) store1(base, kKind, at + e, y[jj][e]);
      }
    }
  };
  {
    v4i v[N];
#pragma unroll
    for (int jj = 0; jj < N; ++jj) v[jj] = acc[F0 + jj];
#pragma unroll
    for (int k = 0; k < kPairs; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const auto h = __builtin_amdgcn_permlane32_swap(v[2 * k][e], v[2 * k + 1][e], false, false);
        const auto q = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
        v[2 * k][e] = q[0];
        v[2 * k + 1][e] = q[1];
      }
#pragma unroll
    for (int jj = 0; jj < N; ++jj)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[jj][e] = scaled(__builtin_amdgcn_ds_bpermute(src, v[jj][e]), rs, o.cscal);
  }
  if (o.bias) {
#pragma unroll
    for (int jj = 0; jj < N; ++jj) {
      const int64_t col = col_of(jj);
      if (!GUARD || col + 3 < Cc) {
        const v4f_u b = *reinterpret_cast<const v4f_u *>(o.bias + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[jj][e] += b[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < Cc) y[jj][e] += o.bias[col + e];
      }
    }
  }
  if (o.z) store(o.z);
  if (E != EPI_POLY || o.act != TGEMM_ACT_NONE) {
#pragma unroll
    for (int jj = 0; jj < N; ++jj)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[jj][e] = epi_act<E>(y[jj][e], o.act);
  }
  if (o.res && in) {
#pragma unroll
    for (int jj = 0; jj < N; ++jj) {
      const int64_t col = col_of(jj), at = row * Cc + col;
      if (!GUARD || col + 3 < Cc) {
        if constexpr (BF) {
          const v2u_u v = *reinterpret_cast<const v2u_u *>(static_cast<const uint16_t *>(o.res) + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[jj][e] += __uint_as_float(e & 1 ? v[e / 2] & 0xFFFF0000u : v[e / 2] << 16);
        } else {
          const v4f_u v = *reinterpret_cast<const v4f_u *>(static_cast<const float *>(o.res) + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[jj][e] += v[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < Cc)
            y[jj][e] += BF ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(o.res)[at + e] << 16)
                           : static_cast<const float *>(o.res)[at + e];
      }
    }
  }
  store(o.ptr);
  __builtin_amdgcn_sched_barrier(0);   // the next run's registers do not mix with this one's
}

template <int E, bool BF, bool GUARD, int F0, int FN>
__device__ __forceinline__ void epi_row(const Out &o, int64_t Cc, const v4i (&acc)[FN], int64_t row, bool in,
                                        int64_t c0, int lane, float rs) {
  constexpr int N = FN - F0 < 4 ? FN - F0 : 4;
  epi_run<E, BF, GUARD, F0, N, FN>(o, Cc, acc, row, in, c0, lane, rs);
  if constexpr (F0 + N < FN) epi_row<E, BF, GUARD, F0 + N, FN>(o, Cc, acc, row, in, c0, lane, rs);
}

template <int E, bool BF, bool GUARD, int FM, int FN>
__device__ __forceinline__ void epi_tile(const Out &o, int64_t R, int64_t Cc, const v4i (&acc)[FM][FN], int64_t r0,
                                         int64_t c0, int lane, const float (&rs)[FM]) {
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t row = r0 + (lane >> 2) + 16 * i;
    epi_row<E, BF, GUARD, 0, FN>(o, Cc, acc[i], row, !GUARD || row < R, c0, lane, rs[i]);
  }
}

// ---------------------------------------------------------------------------
// Gated: the product's columns 2 c and 2 c + 1 are the gate and the up projection
// of output column c, so that every lane that has a quad of columns has whole
// pairs, in any kernel and whatever the width.
//     g = (float(acc) rs) cscal + bias[c],  u = (float(acc') rs) cscal2 + bias[No + c]
//     Y[row][c] = act(g) u,  Z[row] = (g | u)
// No is the output's width; Z has 2 No columns, and so has bias.
// ---------------------------------------------------------------------------

// the pairs of columns col, col + 1 of the output, from a quad of the product
template <int E>
__device__ __forceinline__ void gated_put(const Out &o, int64_t No, int64_t row, int64_t col, const v4i &v, float r) {
#pragma clang fp contract(off)   // every kernel rounds alike
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t c = col + k;
    if (c >= No) break;
    float g = scaled(v[2 * k], r, o.cscal), u = scaled(v[2 * k + 1], r, o.cscal2);
    if (o.bias) {
      g += o.bias[c];
      u += o.bias[No + c];
    }
    if (o.z) {
      store1(o.z, o.kind, 2 * row * No + c, g);
      store1(o.z, o.kind, (2 * row + 1) * No + c, u);
    }
    store1(o.ptr, o.kind, row * No + c, epi_act<E>(g, o.act) * u);
  }
}

// columns col .. col + 3 of row `row`, all inside the output (o.vec); r is
// the row's scale (read by the caller; unused for int32)
template <int E>
__device__ __forceinline__ void put4(const Out &o, int64_t Cc, int64_t row, int64_t col, const v4i &v, float r) {
  if constexpr (E != EPI_NONE) {
    epi_put4<E>(o, Cc, row, col, v, r);
    return;
  }
  const int64_t e = row * Cc + col;
  if (o.kind == OUT_I32) {
    *reinterpret_cast<v4i *>(static_cast<int32_t *>(o.ptr) + e) = v;
    return;
  }
  float y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = scaled(v[k], r, o.cs ? o.cs[col + k] : o.cscal);
  if (o.kind == OUT_F32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(o.ptr) + e) = make_float4(y[0], y[1], y[2], y[3]);
  } else {
    uint2 b;
    b.x = bf16_pack(y[0], y[1]);
    b.y = bf16_pack(y[2], y[3]);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.ptr) + e) = b;
  }
}
template <int E>
__device__ __forceinline__ void put1(const Out &o, int64_t Cc, int64_t row, int64_t col, int32_t x, float r) {
  if constexpr (E != EPI_NONE) {
    epi_put1<E>(o, Cc, row, col, x, r);
    return;
  }
  const int64_t e = row * Cc + col;
  if (o.kind == OUT_I32) {
    static_cast<int32_t *>(o.ptr)[e] = x;
    return;
  }
  const float y = scaled(x, r, o.cs ? o.cs[col] : o.cscal);
  if (o.kind == OUT_F32)
    static_cast<float *>(o.ptr)[e] = y;
  else
    static_cast<uint16_t *>(o.ptr)[e] = __builtin_bit_cast(uint16_t, (__bf16)y);
}
__device__ __forceinline__ float row_scale(const Out &o, int64_t row) {
  return o.kind == OUT_I32 ? 0.f : o.rs[row];
}

// ---------------------------------------------------------------------------
// Workgroup -> tile order.  The hardware hands workgroup ids to the XCDs
// round-robin (id % xcds; MI355X has eight), and each XCD has its own L2.
// xcd_tile gives each
// XCD a contiguous range of positions in a linear tile order (a bijection on
// [0, tiles)).  That order runs row by row inside bands of band_cols tile
// columns, band after band, so the tiles an XCD runs together share input
// rows, and with several bands an XCD also touches only its band's columns.
// The host picks the band count that minimises the operand bytes the eight
// XCDs fetch between them.
// ---------------------------------------------------------------------------
__host__ __device__ inline int32_t xcd_tile(int32_t wg, int32_t tiles, int32_t xcds) {
  const int32_t q = tiles / xcds, r = tiles % xcds;
  const int32_t x = wg % xcds, j = wg / xcds;
  return (x < r) ? x * (q + 1) + j : r * (q + 1) + (x - r) * q + j;
}

__host__ __device__ inline void tile_rc(int32_t pos, int32_t tiles_r, int32_t tiles_c,
                                        int32_t band_cols, int32_t *tr, int32_t *tc) {
  const int32_t per_band = tiles_r * band_cols;
  const int32_t band = pos / per_band, rem = pos % per_band;
  const int32_t c0 = band * band_cols;
  const int32_t w = tiles_c - c0 < band_cols ? tiles_c - c0 : band_cols;
  *tr = rem / w;
  *tc = c0 + rem % w;
}

// ---------------------------------------------------------------------------
// Code decode: one packed dword x (code i at bits 2i) -> 16 int8 weights.
// For output dword j (codes 4j .. 4j + 3, byte j of x), one v_perm_b32
// gathers byte j of x and byte j of y = x >> 2 as [x_j, y_j, x_j, y_j]; a
// packed 16-bit right shift by (0, 4) leaves code 4j + k in the low two bits
// of byte k (byte 1: bits 2-3 of x_j, byte 2: bits 4-5, byte 3: bits 6-7);
// masked to those bits, each byte selects its weight from kCodeTable with a
// second v_perm_b32.  Four codes -> four weights in four instructions.
// ---------------------------------------------------------------------------
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4i decode16(uint32_t x) {
  const uint32_t y = x >> 2;
  v4i w;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // selector bytes [j, 4 + j, j, 4 + j]: bytes 0-3 of the pool are x, 4-7 are y
    const uint32_t sel = (uint32_t)j * 0x00010001u + (uint32_t)(4 + j) * 0x01000100u;
    const u16x2 h = __builtin_bit_cast(u16x2, __builtin_amdgcn_perm(y, x, sel)) >> (u16x2){0, 4};
    w[j] = (int32_t)__builtin_amdgcn_perm(0u, kCodeTable, __builtin_bit_cast(uint32_t, h) & 0x03030303u);
  }
  return w;
}

}  // namespace

// The gated product of few rows on the stored codes, in ternary_gemm.hip: whether
// it takes these sizes and this smallest alignment of A and Wpacked, its launch, and
// the call (arguments checked by the caller).
struct GatedCall {
  const int8_t *A;
  const uint8_t *Wpacked;
  const float *row_scale, *bias;
  float gate_scale, up_scale;
  void *Y, *Z;
  int32_t kind, act;
  int64_t M, N, K;
};
__attribute__((visibility("hidden"))) bool gated_few_ok(int64_t M, int64_t N, int64_t K, int64_t align);
__attribute__((visibility("hidden"))) void gated_few_plan(int64_t M, int64_t N, int64_t K, int32_t cus, int32_t xcds,
                                                          tgemm_plan *plan);
__attribute__((visibility("hidden"))) int gated_few(const GatedCall &c, int32_t cus, int32_t xcds, hipStream_t stream);

#endif  // TERNARY_PRODUCT_H
