// block.hip -- gfx950 kernels of the operators around the ternary product,
// part of libternary_gemm.so (ABI and formulas in include/ternary_gemm.h):
//   ternary_rmsnorm_quantize    residual addition, RMS norm, int8 rows
//   ternary_rmsnorm_backward    its gradients
//   ternary_epilogue_backward   the backward of bias and activation, with the
//                               int8 rows that the dX products take
//   ternary_clip_grad_norm      the global norm of many gradients, and the
//                               scaling by it
// (the product's own epilogue is part of the product's kernels).  All four
// only read and write their operands: HBM bounds them, and the smallest are
// bound by their launches.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <new>
#include <vector>

#include "ternary_gemm.h"

// sums and products are fused only where fma is written, so that every variant
// of a kernel rounds alike
#pragma clang fp contract(off)

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kNT = 256;   // threads per workgroup

bool overlap(const void *a, int64_t an, const void *b, int64_t bn) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}
bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
__device__ __forceinline__ float block_sum(float v, float *part) {
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

// one workgroup per row (grid-stride), three passes over the row: the sum and
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

// ---------------------------------------------------------------------------
// Backward of the norm, and of the epilogue: a pass over rows, and one over
// columns for the gradients that are sums over rows.
// ---------------------------------------------------------------------------
struct NormBwdArgs {
  const void *dY, *H;
  const float *gain, *rstd;
  const void *dH;
  void *dX;
  int64_t R, C;
};

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
  int64_t R, C;
  int32_t act;
};

constexpr float kGeluA = 1.5957691216057308f;              // 2 sqrt(2 / pi)
constexpr float kGeluAB = 1.5957691216057308f * 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

// dy * act'(z).  relu2's 2 z is taken as (2 dy) z, which stays finite where
// the product does.  For z sigmoid(u): p + z p (1 - p) u', p = sigmoid(u) = 1 / (1 + e),
// 1 - p = e p with e = exp(-u).  Past +-88 the slope is 0 or 1 in single
// precision (the terms are below 1e-36); the clamp keeps e finite.  It is
// written with comparisons, which keep a NaN.
__device__ __forceinline__ float back(float dy, float z, int act) {
  if (act == TGEMM_ACT_NONE) return dy;
  if (act == TGEMM_ACT_RELU) return dy * (z > 0.f ? 1.f : (z == z ? 0.f : z));
  if (act == TGEMM_ACT_RELU2) return (dy + dy) * (z < 0.f ? 0.f : z);
  const bool silu = act == TGEMM_ACT_SILU;
  const float c = z < -88.f ? -88.f : (z > 88.f ? 88.f : z), c2 = c * c;
  const float u = silu ? c : c * (kGeluA + kGeluAB * c2), du = silu ? 1.f : kGeluA + 3.f * kGeluAB * c2;
  const float e = __builtin_amdgcn_exp2f(fminf(-u * kLog2e, 126.f));
  const float p = __builtin_amdgcn_rcpf(1.f + e);
  return dy * (p + c * p * (e * p) * du);
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
// are dy * h * rstd; otherwise dy * act'(z).
template <class T, bool NORM>
__global__ __launch_bounds__(kNT) void col_sums(const T *__restrict__ A, const T *__restrict__ B,
                                                const float *__restrict__ rstd, int32_t act, float *__restrict__ P,
                                                int64_t R, int64_t C, int64_t strip) {
  const int64_t c = (int64_t)blockIdx.x * kNT + threadIdx.x;
  if (c >= C) return;
  const int64_t r0 = (int64_t)blockIdx.y * strip, r1 = r0 + strip < R ? r0 + strip : R;
  float sum = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float a = widen(A[r * C + c]), b = widen(B[r * C + c]);
    sum = NORM ? __builtin_fmaf(a, b * rstd[r], sum) : sum + back(a, b, act);
  }
  P[blockIdx.y * C + c] = sum;
}

// the strips' sums added in strip order
__global__ __launch_bounds__(kNT) void col_finish(const float *__restrict__ P, float *__restrict__ out, int64_t strips,
                                                  int64_t C) {
  const int64_t c = (int64_t)blockIdx.x * kNT + threadIdx.x;
  if (c >= C) return;
  float sum = 0.f;
  for (int64_t s = 0; s < strips; ++s) sum += P[s * C + c];
  out[c] = sum;
}

constexpr int64_t kMaxStrips = 512;
int64_t strips_of(int64_t R) { return R < kMaxStrips ? R : kMaxStrips; }

// ---------------------------------------------------------------------------
// Clipping
// ---------------------------------------------------------------------------
constexpr int kGroup = 64;             // tensors per launch
constexpr int64_t kChunk = 16384;      // elements per workgroup

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
  int i = 0;
  while (i + 1 < ts.count && ts.first[i + 1] <= chunk) ++i;
  return i;
}

__global__ __launch_bounds__(kNT) void sumsq(Tensors ts, double *__restrict__ part) {
  __shared__ double wsum[4];
  const int i = tensor_of(ts, blockIdx.x);
  const int64_t e0 = (int64_t)(blockIdx.x - ts.first[i]) * kChunk;
  const int64_t e1 = e0 + kChunk < ts.size[i] ? e0 + kChunk : ts.size[i];
  double sum = 0.0;
  for (int64_t e = e0 + threadIdx.x; e < e1; e += kNT) {
    const double v = ts.bf16[i] ? widen(static_cast<const uint16_t *>(ts.in[i])[e]) : static_cast<const float *>(ts.in[i])[e];
    sum = __builtin_fma(v, v, sum);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = (wsum[0] + wsum[1]) + (wsum[2] + wsum[3]);
}

// one workgroup: the partial sums in a fixed order, the norm, the factor
__global__ __launch_bounds__(kNT) void norm_finish(const double *__restrict__ part, int64_t n, float max_norm, float eps,
                                                   float *__restrict__ norm, float *__restrict__ factor) {
  __shared__ double wsum[4];
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kNT) sum += part[i];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    const float v = (float)__dsqrt_rn((wsum[0] + wsum[1]) + (wsum[2] + wsum[3]));
    *norm = v;
    const float f = __fdiv_rn(max_norm, v + eps);
    *factor = f > 1.f ? 1.f : f;
  }
}

__global__ __launch_bounds__(kNT) void scale_all(Tensors ts, const float *__restrict__ factor) {
  const int i = tensor_of(ts, blockIdx.x);
  const int64_t e0 = (int64_t)(blockIdx.x - ts.first[i]) * kChunk;
  const int64_t e1 = e0 + kChunk < ts.size[i] ? e0 + kChunk : ts.size[i];
  const float f = *factor;
  for (int64_t e = e0 + threadIdx.x; e < e1; e += kNT) {
    if (ts.bf16[i])
      static_cast<uint16_t *>(ts.out[i])[e] = narrow<uint16_t>(widen(static_cast<const uint16_t *>(ts.in[i])[e]) * f);
    else
      static_cast<float *>(ts.out[i])[e] = static_cast<const float *>(ts.in[i])[e] * f;
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

struct Buf {
  const void *p;
  int64_t bytes;
};
// whether outs[i] overlaps an input (equal pointers allowed where `same` names
// that input for it) or a later output; NULL buffers overlap nothing
template <int NO, int NI>
bool alias(const Buf (&outs)[NO], const Buf (&ins)[NI], const void *const (&same)[NO][2]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes) &&
          !(outs[i].p == ins[j].p && outs[i].bytes == ins[j].bytes &&
            (ins[j].p == same[i][0] || ins[j].p == same[i][1])))
        return true;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
  }
  return false;
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

int done() { return hipGetLastError() == hipSuccess ? TGEMM_OK : TGEMM_ERR_HIP; }

int64_t col_ws_bytes(int64_t R, int64_t C) { return 4 * strips_of(R) * C; }

template <class T, bool NORM>
void launch_cols(const T *A, const T *B, const float *rstd, int act, float *P, float *out, int64_t R, int64_t C,
                 hipStream_t stream) {
  const int64_t strip = ceil_div(R, strips_of(R)), strips = ceil_div(R, strip);
  const unsigned gx = (unsigned)ceil_div(C, kNT);
  hipLaunchKernelGGL((col_sums<T, NORM>), dim3(gx, (unsigned)strips), dim3(kNT), 0, stream, A, B, rstd, act, P, R, C,
                     strip);
  hipLaunchKernelGGL(col_finish, dim3(gx), dim3(kNT), 0, stream, P, out, strips, C);
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
  if (!workspace || workspace_bytes < wb || !aligned(workspace, 16)) return TGEMM_ERR_WORKSPACE;
  const int64_t xb = R * C * (in_kind == TGEMM_IN_F32 ? 4 : 2);
  const Buf outs[] = {{dX, xb}, {dgain, 4 * C}, {workspace, wb}};
  const Buf ins[] = {{dY, xb}, {H, xb}, {gain, 4 * C}, {rstd, 4 * R}, {dH, xb}};
  const void *const same[3][2] = {{dH, dH}};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  const NormBwdArgs a = {dY, H, gain, rstd, dH, dX, R, C};
  const dim3 g((unsigned)(R < kMaxRowGrid ? R : kMaxRowGrid));
  float *P = static_cast<float *>(workspace);
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
  if (dbias && (!workspace || workspace_bytes < wb || !aligned(workspace, 16))) return TGEMM_ERR_WORKSPACE;
  const int64_t n = R * C, xb = n * (in_kind == TGEMM_IN_F32 ? 4 : 2);
  const Buf outs[] = {{dZ, xb}, {dbias, 4 * C}, {Q, n}, {scale, 4 * R}, {dbias ? workspace : nullptr, wb}};
  const Buf ins[] = {{dY, xb}, {Z, xb}};
  const void *const same[5][2] = {};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  const EpiBwdArgs a = {dY, Z, dZ, Q, scale, R, C, act};
  const dim3 g((unsigned)(R < kMaxRowGrid ? R : kMaxRowGrid));
  float *P = static_cast<float *>(workspace);
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

int ternary_clip_grad_norm_workspace(const int64_t *sizes, int64_t count, int64_t *bytes) {
  if (!sizes || !bytes) return TGEMM_ERR_NULL;
  if (count < 1) return TGEMM_ERR_DIM;
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > INT64_MAX / 16) return TGEMM_ERR_DIM;
    chunks += ceil_div(sizes[i], kChunk);
    if (chunks > INT32_MAX) return TGEMM_ERR_DIM;
  }
  *bytes = 16 + 8 * chunks;
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
  } catch (const std::bad_alloc &) {
    return TGEMM_ERR_DIM;   // more gradients than the host can list
  }
  if (overlap(norm, 4, workspace, need)) return TGEMM_ERR_ALIAS;
  float *factor = static_cast<float *>(workspace);
  double *part = reinterpret_cast<double *>(static_cast<char *>(workspace) + 16);
  for (int pass = 0; pass < 2; ++pass) {
    int64_t done_chunks = 0;
    Tensors ts;
    ts.count = 0;
    ts.first[0] = 0;
    for (int64_t i = 0; i < count; ++i) {
      if (sizes[i] > 0) {
        const int j = ts.count++;
        ts.in[j] = grads[i];
        ts.out[j] = outs[i];
        ts.size[j] = sizes[i];
        ts.bf16[j] = kinds[i] == TGEMM_IN_BF16;
        ts.first[j + 1] = ts.first[j] + (int32_t)ceil_div(sizes[i], kChunk);
      }
      const int32_t chunks = ts.first[ts.count];
      if (chunks > 0 && (ts.count == kGroup || i == count - 1)) {
        if (pass == 0)
          hipLaunchKernelGGL(sumsq, dim3((unsigned)chunks), dim3(kNT), 0, stream, ts, part + done_chunks);
        else
          hipLaunchKernelGGL(scale_all, dim3((unsigned)chunks), dim3(kNT), 0, stream, ts, factor);
        done_chunks += chunks;
        ts.count = 0;
      }
    }
    if (pass == 0)
      hipLaunchKernelGGL(norm_finish, dim3(1), dim3(kNT), 0, stream, part, done_chunks, max_norm, eps, norm, factor);
  }
  return done();
}

}  // extern "C"
