// int8.hip -- gfx950 kernels of two products, part of libternary_gemm.so (ABI and
// formulas in include/ternary_gemm.h):
//   ternary_gemm_s8s8_epilogue  int8 rows times int8 weights, a scale a row and
//                               a scale a column, bias, activation, residual
//   ternary_gemm_s8_gated       int8 rows times the ternary weights of a gate and
//                               of an up projection, act(g) u (few rows are
//                               multiplied in ternary_gemm.hip)

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "checks.h"
#include "product.h"
#include "ternary_gemm.h"

namespace {

// ---------------------------------------------------------------------------
// Tiled kernel (tgemm_int8): both operands are int8 rows along the contraction, of
// whole 16-byte chunks, 16-byte aligned; K products a row are counted, the rest of
// the last step as zeros.  (Ternary weights come decoded, see lay_gated: decoding each
// fragment as it is read, as the ternary kernels do, costs every row of waves 16 vector
// instructions a fragment.  Decoding once a step on the way into LDS was not tried.)
//
// Persistent workgroups of NW = WM x WN waves, one or two a CU, take tiles of BM x BN
// in XCD-contiguous order, in bands of columns.  A step is KS = 128 values: a row's
// 128 bytes are a whole line, and the loads go straight into LDS, into a ring of D
// stages.  Chunk c of row r lies at slot c ^ ((r >> 1) & 7), free of conflicts for the
// fragment reads (16 rows at one chunk) and, the loads' lanes taking slots in order,
// for the loads.  A step has U = 2 substeps of one v_mfma_i32_16x16x64_i8 a fragment
// pair; during one, the fragments of the next are read.  The step's one barrier
// stands before its last substep: by then every wave has read all of stage g, so the
// loads of step g + D go into it from there on, and the barrier publishes stage g + 1,
// which the last substep reads from.  A wave waits there for its own loads of step
// g + 1, that is until at most the D - 2 batches after them are in flight.
//
// What bounds it: a tile reads (BM + BN) KS bytes a step through the CU's vector
// memory pipe for 2 BM BN KS operations, and the waves of a SIMD do not hide all of
// that, nor the barrier, under each other's products (16384x6912x5120: 2.53 POP/s in 256
// x 192, 2.25 in 256 x 128, 1.9 in 128 x 128; without loads 2.7, without loads and LDS
// reads 3.2, at which the card's power limit lowers the clock); and the tile ends, whose
// stores all CUs make at once while no products run (226 MB of bfloat16 take some 50 us
// of 16384x6912x1280's 154).  256 x 192 is the largest tile whose sums (96 registers) and
// two sets of fragments (80) leave room: 256 x 256 spills.  Tried and left out: the tile
// before written during the next one's first steps, its sums set aside (33 to 49
// registers spill, 126 -> 166 us); a wave's priority raised for its products (+4%);
// lines touched steps ahead for the L2s (+30%: a touch costs the pipe as much as a
// load); steps of 64 (half lines, +10%); starts of the CUs apart (no change).
// ---------------------------------------------------------------------------
namespace mm {
template <int BM_, int BN_, int WM_, int WN_, int KS_, int D_, int PERCU_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KS = KS_, D = D_, PERCU = PERCU_;
  static constexpr int NW = WM * WN, NT = 64 * NW, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int U = KS / 64, CH = KS / 16, RPL = 64 / CH;   // substeps, chunks a row, rows a wave's load
  static constexpr int kAStage = BM * KS, kStage = (BM + BN) * KS, kLds = D * kStage;
  static constexpr int kALoads = kAStage / 1024 / NW, kWLoads = BN * KS / 1024 / NW, kBatch = kALoads + kWLoads;
  static constexpr int kWait = (D - 2) * kBatch;
  static_assert(kALoads * 1024 * NW == kAStage && kWLoads * 1024 * NW == BN * KS, "whole loads");
  // scales and biases of a tile's rows and columns, in 64-lane loads
  static constexpr int kAux = BM / 64 + 2 * (BN / 64), kAuxLoads = (kAux + NW - 1) / NW, kAuxBytes = 256 * kAux;
  static_assert(FM * 16 * WM == BM && FN * 16 * WN == BN && BM % 64 == 0 && BN % 64 == 0 && D >= 2, "tile");
  static_assert((kLds + kAuxBytes) * PERCU <= 160 * 1024, "LDS");
  __host__ __device__ static constexpr int at(int r, int c) { return r * KS + 16 * (c ^ ((r >> 1) & (CH - 1))); }
};
}  // namespace mm

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

struct MArgs {
  const int8_t *A, *W;   // rows of the output, rows of its columns
  Out o;
  int64_t R, Cc, K;      // rows, columns, row length in bytes (a multiple of 16)
  int32_t tiles_r, tiles_c, tiles, band_cols, xcds;
  int32_t nk;     // steps
  int32_t tail;   // 16-byte chunks of the last step
};

// ---------------------------------------------------------------------------
// A tile's output.  Scales and biases come from LDS, where the tile's loads have
// put them: a global load here would wait for the stores before it, since a
// wave's memory operations complete in order (1782x3456x1280 bf16 took 19.1 us with
// such loads and 16.4 without).  For the same reason a residual is read a fragment row
// ahead, before the stores of the row in hand.
//   aux: BM row scales, then BN column scales (COLS) or nothing, then BN biases
// A fragment row goes out as in epi_run: bfloat16 fragments in pairs, 16 bytes a
// lane, four lanes 64 bytes of a row; float32 16 bytes a lane, 64 a row.
// ---------------------------------------------------------------------------
template <class C, int E, bool BF, bool GUARD>
struct PlainOut {
  static constexpr int FM = C::FM, FN = C::FN, kKind = BF ? OUT_BF16 : OUT_F32;
  static_assert(FN % 2 == 0, "pairs of fragments");
  const Out &o;
  const float *aux;        // LDS
  int64_t R, N, r0, c0;    // the output, the wave's first row and column
  int rl, cl;              // the same in the tile
  int lane;

  __device__ __forceinline__ int col_of(int jj) const {   // of the wave's columns: the first of register set jj
    const int p = lane & 3;
    return BF ? 32 * (jj / 2) + 8 * p + 4 * (jj & 1) : 16 * jj + 4 * p;
  }
  __device__ __forceinline__ void load_res(float (&x)[FN][4], int i) const {
    int64_t row = r0 + (lane >> 2) + 16 * i;
    if (GUARD && row >= R) row = R - 1;
#pragma unroll
    for (int jj = 0; jj < FN; ++jj) {
      const int64_t col = c0 + col_of(jj), at = row * N + col;
      if (!GUARD || col + 3 < N) {
        if constexpr (BF) {
          const v2u_u v = *reinterpret_cast<const v2u_u *>(static_cast<const uint16_t *>(o.res) + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[jj][e] = __uint_as_float(e & 1 ? v[e / 2] & 0xFFFF0000u : v[e / 2] << 16);
        } else {
          const v4f_u v = *reinterpret_cast<const v4f_u *>(static_cast<const float *>(o.res) + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[jj][e] = v[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t in = row * N + (col + e < N ? col + e : N - 1);   // past the row its last element, never stored
          x[jj][e] = BF ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(o.res)[in] << 16)
                        : static_cast<const float *>(o.res)[in];
        }
      }
    }
  }
  __device__ __forceinline__ void store(void *base, const float (&y)[FN][4], int i) const {
    const int64_t row = r0 + (lane >> 2) + 16 * i;
    if (GUARD && row >= R) return;
#pragma unroll
    for (int jj = 0; jj < FN; ++jj) {
      const int64_t col = c0 + col_of(jj), at = row * N + col;
      if (BF && !(jj & 1) && (!GUARD || col + 7 < N)) {
        *reinterpret_cast<v4u_u *>(static_cast<uint16_t *>(base) + at) =
            v4u_u{bf16_pack(y[jj][0], y[jj][1]), bf16_pack(y[jj][2], y[jj][3]), bf16_pack(y[jj | 1][0], y[jj | 1][1]),
                  bf16_pack(y[jj | 1][2], y[jj | 1][3])};
      } else if (BF && (jj & 1) && (!GUARD || col + 3 < N)) {
        // went with the set before it
      } else if (!GUARD || col + 3 < N) {
        store4(base, kKind, at, y[jj]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < N) store1(base, kKind, at + e, y[jj][e]);
      }
    }
  }
  __device__ __forceinline__ void run(const v4i (&acc)[FM][FN]) const {
#pragma clang fp contract(off)   // every kernel rounds alike
    const int p = lane & 3, src = 4 * ((lane >> 2) + 16 * p);
    const float *cs = aux + C::BM + cl, *bias = cs + C::BN;
    float res[2][FN][4];
    if (o.res) load_res(res[0], 0);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (o.res && i + 1 < FM) load_res(res[(i + 1) & 1], i + 1);
      const float rs = aux[rl + (lane >> 2) + 16 * i];
      float y[FN][4];
      {
        v4i v[FN];
#pragma unroll
        for (int jj = 0; jj < FN; ++jj) v[jj] = acc[i][jj];
        if constexpr (BF) {
#pragma unroll
          for (int k = 0; k < FN; k += 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const auto h = __builtin_amdgcn_permlane32_swap(v[k][e], v[k + 1][e], false, false);
              const auto q = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
              v[k][e] = q[0];
              v[k + 1][e] = q[1];
            }
        }
#pragma unroll
        for (int jj = 0; jj < FN; ++jj)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[jj][e] = __fmul_rn((float)__builtin_amdgcn_ds_bpermute(src, v[jj][e]), rs);
      }
      if (o.cs) {
#pragma unroll
        for (int jj = 0; jj < FN; ++jj) {
          const float4 c = *reinterpret_cast<const float4 *>(cs + col_of(jj));
          y[jj][0] *= c.x;
          y[jj][1] *= c.y;
          y[jj][2] *= c.z;
          y[jj][3] *= c.w;
        }
      }
      if (o.bias) {
#pragma unroll
        for (int jj = 0; jj < FN; ++jj) {
          const float4 b = *reinterpret_cast<const float4 *>(bias + col_of(jj));
          y[jj][0] += b.x;
          y[jj][1] += b.y;
          y[jj][2] += b.z;
          y[jj][3] += b.w;
        }
      }
      if (o.z) store(o.z, y, i);
      if ((E & kEpiAct) != EPI_POLY || o.act != TGEMM_ACT_NONE) {
#pragma unroll
        for (int jj = 0; jj < FN; ++jj)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[jj][e] = epi_act<E>(y[jj][e], o.act);
      }
      if (o.res) {
#pragma unroll
        for (int jj = 0; jj < FN; ++jj)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[jj][e] += res[i & 1][jj][e];
      }
      store(o.ptr, y, i);
      __builtin_amdgcn_sched_barrier(0);   // the next row's registers do not mix with this one's
    }
  }
};

// The same for column pairs (gated): lane groups and registers are exchanged
// (permlane swaps) until group p of 16 lanes holds 4 FN neighbouring columns, and
// ds_bpermute then gives four neighbouring lanes a row: a lane has 2 FN
// neighbouring outputs, and a row's four lanes 8 FN.
//   aux: BM row scales, BN of nothing, BN / 2 biases of the gate, BN / 2 of the up projection
template <class C, int E, bool BF, bool GUARD>
struct GatedOut {
  static constexpr int FM = C::FM, FN = C::FN, kKind = BF ? OUT_BF16 : OUT_F32;
  static_assert(FN % 2 == 0, "pairs of fragments");
  const Out &o;
  const float *aux;
  int64_t R, N, r0, c0;    // N, c0 and cl count outputs
  int rl, cl;
  int lane;

  template <int OUT>
  __device__ __forceinline__ void store(void *base, int64_t at, int64_t col, const float (&y)[OUT]) const {
    if (!GUARD || col + OUT <= N) {
      if constexpr (BF && OUT == 8) {
        *reinterpret_cast<v4u_u *>(static_cast<uint16_t *>(base) + at) =
            v4u_u{bf16_pack(y[0], y[1]), bf16_pack(y[2], y[3]), bf16_pack(y[4], y[5]), bf16_pack(y[6], y[7])};
      } else {
#pragma unroll
        for (int k = 0; k < OUT; k += 4) store4(base, kKind, at + k, {y[k], y[k + 1], y[k + 2], y[k + 3]});
      }
    } else {
#pragma unroll
      for (int k = 0; k < OUT; ++k)
        if (col + k < N) store1(base, kKind, at + k, y[k]);
    }
  }
  // fragments F0 .. F0 + F - 1 (F 2 or 4) of fragment row i
  template <int F0, int F>
  __device__ __forceinline__ void part(const v4i (&acc)[FM][FN], int i) const {
#pragma clang fp contract(off)   // every kernel rounds alike
    constexpr int kOut = 2 * F;
    const int p = lane & 3, src = 4 * ((lane >> 2) + 16 * p), at = 8 * F0 + kOut * p;
    const int64_t row = r0 + (lane >> 2) + 16 * i, col = c0 + at;
    const float rs = aux[rl + (lane >> 2) + 16 * i];
    float g[kOut], u[kOut];
    {
      v4i v[F];
#pragma unroll
      for (int j = 0; j < F; ++j) v[j] = acc[i][F0 + j];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (F == 4) {
          const auto a = __builtin_amdgcn_permlane32_swap(v[0][e], v[2][e], false, false);
          const auto b = __builtin_amdgcn_permlane32_swap(v[1][e], v[3][e], false, false);
          const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
          const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
          v[0][e] = c[0];
          v[1][e] = c[1];
          v[2][e] = d[0];
          v[3][e] = d[1];
        } else {
          const auto a = __builtin_amdgcn_permlane32_swap(v[0][e], v[1][e], false, false);
          const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[1], false, false);
          v[0][e] = b[0];
          v[1][e] = b[1];
        }
      }
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          g[2 * j + e] = scaled(__builtin_amdgcn_ds_bpermute(src, v[j][2 * e]), rs, o.cscal);
          u[2 * j + e] = scaled(__builtin_amdgcn_ds_bpermute(src, v[j][2 * e + 1]), rs, o.cscal2);
        }
    }
    if (o.bias) {
      const float *bias = aux + C::BM + C::BN + cl + at;
#pragma unroll
      for (int k = 0; k < kOut; k += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(bias + k), b = *reinterpret_cast<const float4 *>(bias + C::BN / 2 + k);
        g[k] += a.x;
        g[k + 1] += a.y;
        g[k + 2] += a.z;
        g[k + 3] += a.w;
        u[k] += b.x;
        u[k + 1] += b.y;
        u[k + 2] += b.z;
        u[k + 3] += b.w;
      }
    }
    const bool in = !GUARD || row < R;
    if (o.z && in) {
      store<kOut>(o.z, 2 * row * N + col, col, g);
      store<kOut>(o.z, (2 * row + 1) * N + col, col, u);
    }
    if ((E & kEpiAct) != EPI_POLY || o.act != TGEMM_ACT_NONE) {
#pragma unroll
      for (int k = 0; k < kOut; ++k) g[k] = epi_act<E>(g[k], o.act);
    }
#pragma unroll
    for (int k = 0; k < kOut; ++k) g[k] *= u[k];
    if (in) store<kOut>(o.ptr, row * N + col, col, g);
    __builtin_amdgcn_sched_barrier(0);   // as above
  }
  template <int F0>
  __device__ __forceinline__ void row_out(const v4i (&acc)[FM][FN], int i) const {
    constexpr int F = FN - F0 >= 4 ? 4 : 2;
    part<F0, F>(acc, i);
    if constexpr (F0 + F < FN) row_out<F0 + F>(acc, i);
  }
  __device__ __forceinline__ void run(const v4i (&acc)[FM][FN]) const {
#pragma unroll
    for (int i = 0; i < FM; ++i) row_out<0>(acc, i);
  }
  static constexpr int kStores = FM * (BF ? (FN + 2) / 4 : FN / 2);   // of a whole tile, without Z's
};

template <class C, int E, bool BF>
__global__ __attribute__((amdgpu_flat_work_group_size(C::NT, C::NT), amdgpu_waves_per_eu(2)))
void tgemm_int8(MArgs a) {
  constexpr int FM = C::FM, FN = C::FN, D = C::D, U = C::U;
  __shared__ __attribute__((aligned(1024))) int8_t smem[C::kLds];
  __shared__ __attribute__((aligned(256))) float aux[C::kAuxBytes / 4];
  const uint32_t lbase = (uint32_t)(uintptr_t)smem;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;

  const int32_t nx = (int32_t)gridDim.x / a.xcds, xcd = (int32_t)blockIdx.x % a.xcds, j0 = (int32_t)blockIdx.x / a.xcds;
  const int32_t q8 = a.tiles / a.xcds, r8 = a.tiles % a.xcds;
  const int32_t start = xcd * q8 + (xcd < r8 ? xcd : r8) + j0, cnt = q8 + (xcd < r8 ? 1 : 0);
  const int32_t ntile = cnt > j0 ? (cnt - j0 + nx - 1) / nx : 0;
  if (ntile == 0) return;
  auto tile_at = [&](int32_t it, int64_t &m0, int64_t &n0) {
    int32_t tr, tc;
    tile_rc(start + it * nx, a.tiles_r, a.tiles_c, a.band_cols, &tr, &tc);
    m0 = (int64_t)tr * C::BM;
    n0 = (int64_t)tc * C::BN;
  };

  // A wave's load i fills the RPL rows from RPL (kALoads wave + i) on, lane l slot
  // l % CH of row l / CH; offsets are from the tile's first row, 255 rows of 16 MB at
  // most.  Rows past the output load the last one again (computed, never stored).
  uint32_t offA[C::kALoads], offW[C::kWLoads];
  const int8_t *ab, *wb;
  const int lrow = lane / C::CH, lslot = lane % C::CH;
  auto set_loads = [&](int32_t it) {
    int64_t m0, n0;
    tile_at(it, m0, n0);
    ab = a.A + m0 * a.K;
    wb = a.W + n0 * a.K;
    const int32_t mr = (int32_t)(a.R - m0 < C::BM ? a.R - m0 : C::BM) - 1, nr = (int32_t)(a.Cc - n0 < C::BN ? a.Cc - n0 : C::BN) - 1;
#pragma unroll
    for (int i = 0; i < C::kALoads; ++i) {
      const int r = C::RPL * (C::kALoads * wave + i) + lrow;
      offA[i] = (uint32_t)(r < mr ? r : mr) * (uint32_t)a.K + 16 * (uint32_t)(lslot ^ ((r >> 1) & (C::CH - 1)));
    }
#pragma unroll
    for (int i = 0; i < C::kWLoads; ++i) {
      const int r = C::RPL * (C::kWLoads * wave + i) + lrow;
      offW[i] = (uint32_t)(r < nr ? r : nr) * (uint32_t)a.K + 16 * (uint32_t)(lslot ^ ((r >> 1) & (C::CH - 1)));
    }
  };
  // the last step's chunks past the contraction load its last one again
  auto clip_loads = [&]() {
#pragma unroll
    for (int i = 0; i < C::kALoads; ++i) {
      const int c = lslot ^ (((C::RPL * (C::kALoads * wave + i) + lrow) >> 1) & (C::CH - 1));
      if (c >= a.tail) offA[i] -= 16 * (uint32_t)(c - (a.tail - 1));
    }
#pragma unroll
    for (int i = 0; i < C::kWLoads; ++i) {
      const int c = lslot ^ (((C::RPL * (C::kWLoads * wave + i) + lrow) >> 1) & (C::CH - 1));
      if (c >= a.tail) offW[i] -= 16 * (uint32_t)(c - (a.tail - 1));
    }
  };
  auto load = [&](int i, int st, int32_t s) {
    if (i < C::kALoads)
      dma16(__builtin_amdgcn_readfirstlane(lbase + st * C::kStage + 1024 * (C::kALoads * wave + i)),
            offA[i < C::kALoads ? i : 0], ab + C::KS * s);
    else
      dma16(__builtin_amdgcn_readfirstlane(lbase + st * C::kStage + C::kAStage + 1024 * (C::kWLoads * wave + i - C::kALoads)),
            offW[i >= C::kALoads ? i - C::kALoads : 0], wb + C::KS * s);
  };
  // the scales and biases of tile it, 64 a load: row scales, then the columns'
  // scales, then their biases (gated: the gate's, then the up projection's)
  auto load_aux = [&](int32_t it) {
    int64_t m0, n0;
    tile_at(it, m0, n0);
#pragma unroll
    for (int i = 0; i < C::kAuxLoads; ++i) {
      const int x = wave + C::NW * i;
      const float *src = a.o.rs + m0;
      int64_t left = a.R - m0;
      int at = 64 * x + lane;
      uint32_t half = 0;   // elements from the gate's biases to the up projection's
      if (x >= C::BM / 64) {
        at = 64 * ((x - C::BM / 64) % (C::BN / 64)) + lane;
        src = x >= C::BM / 64 + C::BN / 64 ? a.o.bias : a.o.cs;
        left = a.Cc - n0;
        if constexpr (E & EPI_GATED) {
          left /= 2;
          if (src) src += n0 / 2;
          if (at >= C::BN / 2) {
            at -= C::BN / 2;
            half = (uint32_t)(a.Cc / 2);
          }
        } else if (src) {
          src += n0;
        }
      }
      if (x < C::kAux && src)
        dma4(__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)aux + 256 * x),
             4 * ((uint32_t)(at < left ? at : left - 1) + half), src);
    }
  };
  // load cursor: the next step whose loads go out; past the end it stays on the last
  int32_t it_ld = 0, s_ld = 0;
  auto next_load = [&]() {
    if (s_ld + 1 < a.nk) {
      ++s_ld;
    } else if (it_ld + 1 < ntile) {
      ++it_ld;
      s_ld = 0;
      set_loads(it_ld);
    } else {
      return;
    }
    if (s_ld == a.nk - 1 && a.tail != C::CH) clip_loads();
  };
  set_loads(0);
  if (a.nk == 1 && a.tail != C::CH) clip_loads();
#pragma unroll
  for (int s = 0; s < D; ++s) {
#pragma unroll
    for (int i = 0; i < C::kBatch; ++i) load(i, s, s_ld);
    next_load();
  }
  v4i acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int jj = 0; jj < FN; ++jj) acc[i][jj] = v4i{0, 0, 0, 0};

  int qoff[U], poff[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    qoff[u] = wm * C::TM * C::KS + C::at(lane & 15, 4 * u + (lane >> 4));
    poff[u] = C::kAStage + wn * C::TN * C::KS + C::at(lane & 15, 4 * u + (lane >> 4));
  }
  v4i q[2][FM], p[2][FN];
  auto frag_q = [&](int st, int u, int i) { return *reinterpret_cast<const v4i *>(smem + st * C::kStage + qoff[u] + i * 16 * C::KS); };
  auto frag_p = [&](int st, int u, int j) { return *reinterpret_cast<const v4i *>(smem + st * C::kStage + poff[u] + j * 16 * C::KS); };
  wait_barrier<(D - 1) * C::kBatch>();
  // stores of a whole tile: without Z, and with it.  They are younger than the
  // loads that the next tile's first barrier waits for, which therefore counts them.
  constexpr int kStores = E & EPI_GATED ? GatedOut<C, E, BF, false>::kStores : FM * (BF ? FN / 2 : FN);
  constexpr int kStoresZ = (E & EPI_GATED ? 3 : 2) * kStores;
  static_assert(C::kWait + kStoresZ <= 63, "vmcnt field");
  int st = 0, after = 0;   // after: 1 or 2, a tile without or with Z was stored right before this step
  // One step: its products, the loads of step g + D into the stage that it frees,
  // and, but for a tile's last step, the first fragments of the step after it.
  auto step = [&](int32_t it, int32_t s, auto last) __attribute__((always_inline)) {
    constexpr bool kLast = decltype(last)::value;
    const int st1 = st + 1 == D ? 0 : st + 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int cur = u & 1, nxt = U == 1 ? 0 : cur ^ 1;
      const bool reads = u + 1 < U || !kLast;
      v4i qn[FM], pn[FN];
      // chunks past the contraction: A's count as zeros
      if (kLast && a.tail != C::CH && 4 * u + (lane >> 4) >= a.tail) {
#pragma unroll
        for (int i = 0; i < FM; ++i) q[cur][i] = v4i{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if (u == U - 1 && i == 0) {
          if (after == 2)
            wait_barrier<C::kWait + kStoresZ>();
          else if (after)
            wait_barrier<C::kWait + kStores>();
          else
            wait_barrier<C::kWait>();
          after = 0;
          if (s == 0) load_aux(it);   // every wave has written the tile before
        }
        const int sn = u + 1 < U ? st : st1, un = u + 1 < U ? u + 1 : 0;
        // fragments of the next substep, the columns' first
        if (reads) {
#pragma unroll
          for (int x = i * (FM + FN) / FM; x < (i + 1) * (FM + FN) / FM; ++x) {
            if (x < FN)
              pn[x < FN ? x : 0] = frag_p(sn, un, x);
            else
              qn[x >= FN ? x - FN : 0] = frag_q(sn, un, x - FN);
          }
        }
        if (u == U - 1) {
#pragma unroll
          for (int x = i * C::kBatch / FM; x < (i + 1) * C::kBatch / FM; ++x) load(x, st, s_ld);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(p[cur][j], q[cur][i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (reads) {
#pragma unroll
        for (int i = 0; i < FM; ++i) q[nxt][i] = qn[i];
#pragma unroll
        for (int j = 0; j < FN; ++j) p[nxt][j] = pn[j];
      }
    }
    next_load();
    st = st1;
  };
  for (int32_t it = 0; it < ntile; ++it) {
    // a tile's first fragments (its first stage was published with the last one
    // of the tile before, whose end needs the registers)
#pragma unroll
    for (int i = 0; i < FM; ++i) q[0][i] = frag_q(st, 0, i);
#pragma unroll
    for (int j = 0; j < FN; ++j) p[0][j] = frag_p(st, 0, j);
    for (int32_t s = 0; s + 1 < a.nk; ++s) step(it, s, Flag<false>());
    step(it, a.nk - 1, Flag<true>());
    int64_t m0, n0;
    tile_at(it, m0, n0);
    // the scales have landed once D - 2 whole batches were waited for after them
    if (a.nk < D) wait_barrier<0>();
    const bool inside = m0 + C::BM <= a.R && n0 + C::BN <= a.Cc;
    const int64_t r0 = m0 + wm * C::TM, c0 = n0 + wn * C::TN;
    if constexpr (E & EPI_GATED) {
      if (inside)
        GatedOut<C, E, BF, false>{a.o, aux, a.R, a.Cc / 2, r0, c0 / 2, wm * C::TM, wn * C::TN / 2, lane}.run(acc);
      else
        GatedOut<C, E, BF, true>{a.o, aux, a.R, a.Cc / 2, r0, c0 / 2, wm * C::TM, wn * C::TN / 2, lane}.run(acc);
    } else {
      if (inside)
        PlainOut<C, E, BF, false>{a.o, aux, a.R, a.Cc, r0, c0, wm * C::TM, wn * C::TN, lane}.run(acc);
      else
        PlainOut<C, E, BF, true>{a.o, aux, a.R, a.Cc, r0, c0, wm * C::TM, wn * C::TN, lane}.run(acc);
    }
    after = !inside ? 0 : a.o.z ? 2 : 1;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int jj = 0; jj < FN; ++jj) acc[i][jj] = v4i{0, 0, 0, 0};
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ---------------------------------------------------------------------------
// Few rows (s8s8): the weights are nearly all of the bytes, and a workgroup of 8
// or 16 waves owns 16 NB columns and 16 MF rows.  Its waves split the contraction
// into super-steps of 256 (wave w takes w, w + 8, ... or w, w + 16, ...), operands straight into
// registers a super-step ahead, and their sums meet in LDS, in wave order.
// Lane l loads 16 bytes of row l % 16 at 64 q + 16 (l / 16), so that load q
// takes 64 bytes of 16 rows, and q = 0 .. 3 are the four MFMA steps of the
// super-step.  Any contraction and any alignment: loads are byte-aligned
// vectors, and the last, partial super-step reads the bytes inside one by one.
// Bound by reading the weights and, where they are few, by one round trip to memory:
// 1x16384x1280 6.2 us in a graph (21 MB), 1x4096x4096 5.6 us, 1x16384x4096 16.0 us (4.2 TB/s),
// 27 rows of it 19.9 us, A coming from the L2s for every column block.
// ---------------------------------------------------------------------------
constexpr int kFewStep = 256;
typedef int32_t v4i_u __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32_u __attribute__((aligned(1)));

struct FewArgs {
  const int8_t *A, *W;
  Out o;
  int64_t M, N, K;
  int32_t rblocks;   // blocks of 16 MF rows
  int32_t xcds;
};

// bytes 0 .. n - 1 of p, zeros past them
__device__ __forceinline__ v4i load_part(const int8_t *p, int64_t n) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int b = 0; b < 16; ++b)
    if (b < n) w[b >> 2] |= (uint32_t)(uint8_t)p[b] << (8 * (b & 3));
  return v4i{(int32_t)w[0], (int32_t)w[1], (int32_t)w[2], (int32_t)w[3]};
}

template <int MF, int NB, int WAVES, int E>
__global__ __attribute__((amdgpu_flat_work_group_size(64 * WAVES, 64 * WAVES), amdgpu_waves_per_eu(WAVES / 4)))
void int8_few(FewArgs a) {
  constexpr int kWaves = WAVES, kNT = 64 * WAVES, kStep = kFewStep;
  constexpr int kPitch = 4 * NB + 1, kWave = 16 * MF * kPitch;
  __shared__ v4i red[kWaves * kWave];
  const int tid = threadIdx.x, lane = tid & 63;
  const int32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  // an XCD's workgroups take neighbouring column blocks, the row blocks of one together
  const int32_t pos = xcd_tile((int32_t)blockIdx.x, (int32_t)gridDim.x, a.xcds);
  const int64_t n0 = (int64_t)(pos / a.rblocks) * 16 * NB, m0 = (int64_t)(pos % a.rblocks) * 16 * MF;
  const int8_t *wr[NB], *ar[MF];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int64_t n = n0 + 16 * nb + r;
    wr[nb] = a.W + (n < a.N ? n : a.N - 1) * a.K + 16 * g;
  }
#pragma unroll
  for (int mf = 0; mf < MF; ++mf) {
    const int64_t m = m0 + 16 * mf + r;
    ar[mf] = a.A + (m < a.M ? m : a.M - 1) * a.K + 16 * g;
  }
  v4i acc[MF][NB];
#pragma unroll
  for (int mf = 0; mf < MF; ++mf)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mf][nb] = v4i{0, 0, 0, 0};
  typedef v4i W4[NB][4];
  typedef v4i A4[MF][4];
  auto load = [&](W4 &w, A4 &x, int64_t k) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) w[nb][q] = *reinterpret_cast<const v4i_u *>(wr[nb] + k + 64 * q);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int mf = 0; mf < MF; ++mf) x[mf][q] = *reinterpret_cast<const v4i_u *>(ar[mf] + k + 64 * q);
  };
  auto step = [&](const W4 &w, const A4 &x) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mf = 0; mf < MF; ++mf)
          acc[mf][nb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[nb][q], x[mf][q], acc[mf][nb], 0, 0, 0);
  };
  const int32_t nfull = (int32_t)(a.K / kStep), cnt = nfull > wave ? (nfull - wave + kWaves - 1) / kWaves : 0;
  if (cnt > 0) {
    W4 w0, w1;
    A4 x0, x1;
    const int32_t last = wave + kWaves * (cnt - 1);   // past it the loads repeat it: in range, never used
    load(w0, x0, (int64_t)kStep * wave);
    int32_t s = wave;
    for (int32_t i = 0; i + 2 <= cnt; i += 2) {
      const int32_t s1 = s + kWaves, s2 = s1 + kWaves < last ? s1 + kWaves : last;
      load(w1, x1, (int64_t)kStep * s1);
      __builtin_amdgcn_sched_barrier(0);   // the loads ahead of the products
      step(w0, x0);
      load(w0, x0, (int64_t)kStep * s2);
      __builtin_amdgcn_sched_barrier(0);
      step(w1, x1);
      s += 2 * kWaves;
    }
    if (cnt & 1) step(w0, x0);
  }
  if (a.K % kStep != 0 && wave == nfull % kWaves) {
    const int64_t k = (int64_t)kStep * nfull;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const int64_t at = k + 64 * q, n = a.K - at - 16 * g;   // bytes of this lane's chunk inside
      if (at >= a.K) break;
      v4i w[NB], x[MF];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) w[nb] = n >= 16 ? v4i(*reinterpret_cast<const v4i_u *>(wr[nb] + at)) : load_part(wr[nb] + at, n);
#pragma unroll
      for (int mf = 0; mf < MF; ++mf) x[mf] = n >= 16 ? v4i(*reinterpret_cast<const v4i_u *>(ar[mf] + at)) : load_part(ar[mf] + at, n);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mf = 0; mf < MF; ++mf)
          acc[mf][nb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[nb], x[mf], acc[mf][nb], 0, 0, 0);
    }
  }
  v4i *mine = red + wave * kWave;
#pragma unroll
  for (int mf = 0; mf < MF; ++mf)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) mine[(16 * mf + r) * kPitch + 4 * nb + g] = acc[mf][nb];
  __syncthreads();
  constexpr int kQuads = 4 * NB, kOut = 16 * MF * kQuads;
  static_assert(kOut <= kNT, "a quad a thread");
  if (tid >= kOut) return;
  const int m = tid / kQuads, cq = tid % kQuads;
  v4i sum = red[m * kPitch + cq];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += red[w * kWave + m * kPitch + cq];
  const int64_t row = m0 + m, col = n0 + 4 * cq;
  if (row >= a.M) return;
  const float rs = a.o.rs[row];
  if (col + 3 < a.N) {
    epi_put4<E>(a.o, a.N, row, col, sum, rs);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < a.N) epi_put1<E>(a.o, a.N, row, col + e, sum[e], rs);
  }
}

// ---------------------------------------------------------------------------
// Rows laid out for tgemm_int8: as they are, with a length that is whole 16-byte
// chunks (zeros past the contraction), or decoded from stored codes, a gate's row
// and an up projection's in turn.  A workgroup takes eight rows, a thread 16 bytes
// at a time, four loads ahead of their stores; past 2^20 groups it takes more of them
// (a launch has fewer than 2^32 threads).  The gated weights of 3456x1280 (11.1 MB read and
// written) take 7 to 8.6 us and of 4096x4096 (42 MB) 12: some 7 TB/s and 6.5 us that do not
// depend on the size, of a launch and of one chain of a load, a decode and a store.
// ---------------------------------------------------------------------------
constexpr int kLayT = 256, kLayRows = 8;
constexpr int64_t kLayGrid = 1 << 20;
template <class Load>
__device__ __forceinline__ void lay_out(int8_t *dst, int64_t R, int32_t chunks, Load load) {
  for (int64_t row0 = (int64_t)blockIdx.x * kLayRows; row0 < R; row0 += (int64_t)gridDim.x * kLayRows) {
    const uint32_t rows = (uint32_t)(R - row0 < kLayRows ? R - row0 : kLayRows), n = rows * (uint32_t)chunks;
    v4i *q = reinterpret_cast<v4i *>(dst) + row0 * chunks;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += 4 * kLayT) {
      v4i v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t i = i0 + k * kLayT;
        if (i < n) v[k] = load(row0 + i / (uint32_t)chunks, i % (uint32_t)chunks);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i0 + k * kLayT < n) q[i0 + k * kLayT] = v[k];
    }
  }
}
__global__ __launch_bounds__(kLayT) void lay_rows(const int8_t *__restrict__ src, int8_t *__restrict__ dst, int64_t R,
                                                  int64_t K, int32_t chunks) {
  lay_out(dst, R, chunks, [&](int64_t row, uint32_t c) {
    const int8_t *p = src + row * K + 16 * c;
    const int64_t n = K - 16 * (int64_t)c;
    return n >= 16 ? v4i(*reinterpret_cast<const v4i_u *>(p)) : load_part(p, n);
  });
}
__global__ __launch_bounds__(kLayT) void lay_gated(const uint8_t *__restrict__ src, int8_t *__restrict__ dst, int64_t N,
                                                   int64_t K, int32_t chunks) {
  lay_out(dst, 2 * N, chunks, [&](int64_t row, uint32_t c) {
    const uint8_t *p = src + ((row & 1) * N + (row >> 1)) * (K / 4) + 4 * c;
    const int64_t n = K / 4 - 4 * (int64_t)c;
    uint32_t x = 0;
    if (n >= 4) {
      x = *reinterpret_cast<const u32_u *>(p);
    } else {
#pragma unroll
      for (int b = 0; b < 3; ++b)
        if (b < n) x |= (uint32_t)p[b] << (8 * b);
    }
    return decode16(x);   // code 0 is weight 0
  });
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct Machine {
  int32_t cus, xcds;
};

int64_t align_of(const void *p) {
  const uintptr_t v = (uintptr_t)p;
  return v ? (int64_t)(v & (~v + 1)) : 1 << 20;
}
int64_t min_align(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t round_up(int64_t v, int64_t n) { return ceil_div(v, n) * n; }

bool mul_ok(int64_t a, int64_t b, int64_t *out) {
  if (b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}
// few rows: 16 threads a column at most, fewer than 2^32 a launch; the tiles' loads of
// biases reach 8 N bytes in 32 bits
constexpr int64_t kMaxCols = (int64_t)1 << 27;
int check_sizes(int64_t M, int64_t N, int64_t K) {
  int64_t t;
  if (M < 1 || N < 1 || K < 1) return TGEMM_ERR_DIM;
  // every byte count (two float32 matrices side by side at most) fits, and so do the tiles
  if (!mul_ok(M, K, &t) || !mul_ok(t, 8, &t) || !mul_ok(N, K, &t) || !mul_ok(t, 8, &t) || !mul_ok(M, N, &t) ||
      !mul_ok(t, 8, &t))
    return TGEMM_ERR_DIM;
  if (N > kMaxCols || ceil_div(M, 16) * ceil_div(2 * N, 16) > INT32_MAX) return TGEMM_ERR_DIM;
  return TGEMM_OK;
}

typedef mm::Cfg<256, 192, 4, 2, 128, 2, 1> T256x192;
typedef mm::Cfg<256, 128, 4, 2, 128, 3, 1> T256x128;
typedef mm::Cfg<128, 192, 4, 2, 128, 3, 1> T128x192;
typedef mm::Cfg<128, 128, 2, 4, 128, 4, 1> T128x128;
typedef mm::Cfg<64, 128, 2, 2, 128, 3, 2> T64x128;
typedef mm::Cfg<64, 64, 2, 2, 128, 4, 2> T64x64;
constexpr int kStep = 128;   // of each of them
static_assert(T256x192::KS == kStep && T256x128::KS == kStep && T128x192::KS == kStep && T128x128::KS == kStep &&
                  T64x128::KS == kStep && T64x64::KS == kStep,
              "time_of");

int64_t mm_grid(int64_t tiles, int64_t percu, const Machine &mc) {
  return tiles < mc.cus * percu ? round_up(tiles, mc.xcds) : mc.cus * percu;
}
// an XCD's tiles in flight, 8 columns wide: 16384x6912x1280 141 us, 16 wide 147, 4 144, 2 150
int32_t mm_band(int32_t tiles_c) { return tiles_c < 8 ? tiles_c : 8; }
template <class C, int E>
int launch_mm(MArgs a, const Machine &mc, hipStream_t stream) {
  a.tiles_r = (int32_t)ceil_div(a.R, C::BM);
  a.tiles_c = (int32_t)ceil_div(a.Cc, C::BN);
  a.tiles = a.tiles_r * a.tiles_c;
  a.xcds = mc.xcds;
  a.band_cols = mm_band(a.tiles_c);
  a.nk = (int32_t)ceil_div(a.K, C::KS);
  a.tail = (int32_t)((a.K - (int64_t)(a.nk - 1) * C::KS) / 16);
  const int64_t grid = mm_grid(a.tiles, C::PERCU, mc);
  if (a.o.kind == OUT_BF16)
    hipLaunchKernelGGL((tgemm_int8<C, E, true>), dim3((unsigned)grid), dim3(C::NT), 0, stream, a);
  else
    hipLaunchKernelGGL((tgemm_int8<C, E, false>), dim3((unsigned)grid), dim3(C::NT), 0, stream, a);
  return hipGetLastError() == hipSuccess ? TGEMM_OK : TGEMM_ERR_HIP;
}
// The tile with the least estimated time: rounds of tiles over the CUs, each of
// `step` us a step and at its end `end` us, `out` for each 2 bytes that it moves
// an output column of the product, and `act` if it takes a sigmoid of each.  A last
// round that leaves CUs idle has up to 20% faster steps and, since its stores do
// not meet all the other CUs', down to a quarter of `out`; of the two kernels with two
// workgroups a CU, a last round of one a CU has its own figures.  Fitted to 578 calls
// of 65 to 16384 rows, bfloat16 and float32, with and without Z, a residual and a
// sigmoid: the choice is the fastest of the six or within 2% of it on 516 of them,
// past 10% on 7 (18% at most, float32 with Z and more than one round), and 0.6% slower
// in the mean.  (Few tiles are best small: 128x4096x4096 takes 11.4 us in 64x64 and 17.6
// in 128x128, 200x1280x1280 float32 with residual and Z 7.4 and 12.3; large outputs best
// large: 16384x6912x1280 takes 141 us in 256x192, 152 in 256x128, 158 in 128x192.)
struct TileTime {
  int32_t bm, bn, percu;
  double step, end, out, act, step1, end1, out1, act1;
};
template <class C>
constexpr TileTime tile_time(double step, double end, double out, double act, double step1 = 0, double end1 = 0,
                             double out1 = 0, double act1 = 0) {
  return {C::BM, C::BN, C::PERCU, step, end, out, act, step1, end1, out1, act1};
}
constexpr TileTime kTiles[] = {
    tile_time<T256x192>(1.14, 4.17, 4.44, 0.71),
    tile_time<T256x128>(0.79, 2.71, 2.95, 0.35),
    tile_time<T128x192>(0.64, 2.5, 2.12, 0.84),
    tile_time<T128x128>(0.51, 1.9, 1.4, 0.2),
    tile_time<T64x128>(0.67, 0.92, 1.51, 0.0, 0.38, 1.38, 0.67, 0.42),
    tile_time<T64x64>(0.4, 0.8, 0.71, 0.0, 0.26, 1.09, 0.35, 0.13)};
constexpr int kNumTiles = sizeof(kTiles) / sizeof(kTiles[0]);
// out: 2-byte units written and read at a tile's end for each column of the product,
// act: sigmoids for each
double time_of(const TileTime &t, int64_t R, int64_t Cc, int64_t K, double out, double act, int64_t cus) {
  const int64_t tiles = ceil_div(R, t.bm) * ceil_div(Cc, t.bn), slots = cus * t.percu, rem = tiles % slots;
  const double steps = (double)ceil_div(K, kStep), full = (double)(tiles / slots);
  const double us = full * (t.step * steps + t.end + t.out * out + t.act * act);
  if (rem == 0) return us;
  const bool one = t.percu == 2 && rem <= cus;
  const double fill = (double)rem / (double)(one ? cus : slots), fs = 0.8 + 0.2 * fill, fo = 0.25 + 0.75 * fill;
  return us + (one ? t.step1 * fs * steps + t.end1 + t.out1 * fo * out + t.act1 * act
                   : t.step * fs * steps + t.end + t.out * fo * out + t.act * act);
}
int best_tile(int64_t R, int64_t Cc, int64_t K, bool gated, int kind, int act, bool z, bool res, int64_t cus) {
  const double out = (kind == OUT_BF16 ? 1.0 : 2.0) * (gated ? 0.5 + z : 1.0 + z + res);
  const double sg = epi_of(act) == EPI_SIGM ? (gated ? 0.5 : 1.0) : 0.0;
  int best = 0;
  double least = time_of(kTiles[0], R, Cc, K, out, sg, cus);
  for (int i = 1; i < kNumTiles; ++i) {
    const double us = time_of(kTiles[i], R, Cc, K, out, sg, cus);
    if (us < least) {
      best = i;
      least = us;
    }
  }
  return best;
}
template <int E>
int pick_mm(const MArgs &a, const Machine &mc, hipStream_t stream) {
  switch (best_tile(a.R, a.Cc, a.K, E & EPI_GATED, a.o.kind, a.o.act, a.o.z, a.o.res, mc.cus)) {
    case 0: return launch_mm<T256x192, E>(a, mc, stream);
    case 1: return launch_mm<T256x128, E>(a, mc, stream);
    case 2: return launch_mm<T128x192, E>(a, mc, stream);
    case 3: return launch_mm<T128x128, E>(a, mc, stream);
    case 4: return launch_mm<T64x128, E>(a, mc, stream);
    default: return launch_mm<T64x64, E>(a, mc, stream);
  }
}
template <int FLAG>
int pick_mm_act(const MArgs &a, const Machine &mc, hipStream_t stream) {
  return epi_of(a.o.act) == EPI_POLY ? pick_mm<EPI_POLY | FLAG>(a, mc, stream) : pick_mm<EPI_SIGM | FLAG>(a, mc, stream);
}

dim3 lay_grid(int64_t R) {
  const int64_t n = ceil_div(R, kLayRows);
  return dim3((unsigned)(n < kLayGrid ? n : kLayGrid));
}
void lay(const int8_t *src, int8_t *dst, int64_t R, int64_t K, int64_t Kp, hipStream_t stream) {
  hipLaunchKernelGGL(lay_rows, lay_grid(R), dim3(kLayT), 0, stream, src, dst, R, K, (int32_t)(Kp / 16));
}

// Few rows go to int8_few, which needs no layout: 32, and up to 64 where the
// weights are small, or would have to be copied first (48 rows, int8_few against
// the tiles: 3456x1280 6.0 and 6.4 us, 1280x3456 8.8 and 10.0, but 4096x4096 13.2 and
// 11.1, 16384x1280 12.7 and 8.7).
bool few_rows(int64_t M, int64_t N, int64_t K, bool copy) { return M <= 32 || (M <= 64 && (copy || N * K <= 6000000)); }

// the workspace of a call: the rows of either operand laid out anew where they
// are not whole, aligned 16-byte chunks, those of the gated product's weights always
struct Layout {
  int64_t kp, a_bytes, w_bytes;
};
Layout layout_of(int64_t M, int64_t rows, int64_t K, bool lay_a, bool lay_w) {
  Layout l;
  l.kp = round_up(K, 16);
  l.a_bytes = lay_a ? round_up(M * l.kp, 256) : 0;
  l.w_bytes = lay_w ? rows * l.kp : 0;
  return l;
}
Layout s8s8_layout(int64_t M, int64_t N, int64_t K, int64_t a_align, int64_t w_align) {
  const bool lay_a = K % 16 != 0 || a_align % 16 != 0, lay_w = K % 16 != 0 || w_align % 16 != 0;
  const bool few = few_rows(M, N, K, lay_a || lay_w);
  return layout_of(M, N, K, !few && lay_a, !few && lay_w);
}
Layout gated_layout(int64_t M, int64_t N, int64_t K, int64_t a_align, int64_t w_align) {
  const bool few = gated_few_ok(M, N, K, min_align(a_align, w_align));
  return layout_of(M, 2 * N, K, !few && (K % 16 != 0 || a_align % 16 != 0), !few);
}

template <int MF, int NB, int WAVES>
int launch_few(FewArgs a, hipStream_t stream) {
  a.rblocks = (int32_t)ceil_div(a.M, 16 * MF);
  const dim3 grid((unsigned)(ceil_div(a.N, 16 * NB) * a.rblocks)), block(64 * WAVES);
  if (epi_of(a.o.act) == EPI_POLY)
    hipLaunchKernelGGL((int8_few<MF, NB, WAVES, EPI_POLY | EPI_COLS>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((int8_few<MF, NB, WAVES, EPI_SIGM | EPI_COLS>), grid, block, 0, stream, a);
  return hipGetLastError() == hipSuccess ? TGEMM_OK : TGEMM_ERR_HIP;
}
// 16 or 32 rows, column blocks as wide as leaves every CU one, and sixteen waves where a
// block of 16 has more super-steps than eight
struct FewPlan {
  int32_t mf, nb, waves;
};
FewPlan few_plan(int64_t M, int64_t N, int64_t K, int64_t cus) {
  const int32_t nb = N >= 64 * cus ? 4 : N >= 32 * cus ? 2 : 1;
  return {M <= 16 ? 1 : 2, nb, nb == 1 && K > 8 * kFewStep ? 16 : 8};
}
template <int MF>
int pick_few(const FewArgs &a, const FewPlan &p, hipStream_t stream) {
  if (p.nb == 4) return launch_few<MF, 4, 8>(a, stream);
  if (p.nb == 2) return launch_few<MF, 2, 8>(a, stream);
  return p.waves == 16 ? launch_few<MF, 1, 16>(a, stream) : launch_few<MF, 1, 8>(a, stream);
}

// The plans' common part, and those of tgemm_int8
int start_plan(int64_t M, int64_t Cc, int64_t K, int act, int out_kind, int32_t cus, int32_t xcds, tgemm_plan *plan) {
  if (cus < 1 || xcds < 1 || cus % xcds != 0) return TGEMM_ERR_DIM;
  if (out_kind != TGEMM_OUT_F32 && out_kind != TGEMM_OUT_BF16) return TGEMM_ERR_KIND;
  if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_VALUE;
  *plan = {};
  plan->out_rows = M;
  plan->out_cols = Cc;
  plan->contraction = K;
  plan->xcds = xcds;
  return TGEMM_OK;
}
void tile_plan(int tile, int64_t R, int64_t Cc, const Machine &mc, tgemm_plan *plan) {
  static constexpr int kThreads[] = {T256x192::NT, T256x128::NT, T128x192::NT, T128x128::NT, T64x128::NT, T64x64::NT};
  static constexpr int kBytes[] = {T256x192::kLds + T256x192::kAuxBytes, T256x128::kLds + T256x128::kAuxBytes,
                                   T128x192::kLds + T128x192::kAuxBytes, T128x128::kLds + T128x128::kAuxBytes,
                                   T64x128::kLds + T64x128::kAuxBytes,   T64x64::kLds + T64x64::kAuxBytes};
  static_assert(sizeof(kThreads) / sizeof(int) == kNumTiles && sizeof(kBytes) / sizeof(int) == kNumTiles, "tiles");
  const TileTime &t = kTiles[tile];
  plan->kernel = TGEMM_KERNEL_INT8;
  plan->tile_rows = t.bm;
  plan->tile_cols = t.bn;
  plan->tiles = ceil_div(R, t.bm) * ceil_div(Cc, t.bn);
  plan->workgroups = mm_grid(plan->tiles, t.percu, mc);
  plan->tiles_per_workgroup = ceil_div(ceil_div(plan->tiles, mc.xcds), plan->workgroups / mc.xcds);
  plan->band_cols = mm_band((int32_t)ceil_div(Cc, t.bn));
  plan->threads_per_workgroup = kThreads[tile];
  plan->lds_bytes = kBytes[tile];
}

}  // namespace

extern "C" {

int ternary_gemm_s8s8_workspace(int64_t M, int64_t N, int64_t K, int64_t align, int64_t *bytes) {
  if (!bytes) return TGEMM_ERR_NULL;
  const int st = check_sizes(M, N, K);
  if (st != TGEMM_OK) return st;
  if (K > TGEMM_INT8_MAX_CONTRACTION) return TGEMM_ERR_BOUND;
  const Layout l = s8s8_layout(M, N, K, align > 0 ? align : 1, align > 0 ? align : 1);
  *bytes = l.a_bytes + l.w_bytes;
  return TGEMM_OK;
}

int ternary_gemm_s8s8_epilogue(const int8_t *A, const int8_t *W, const float *a_row_scale, const float *w_col_scale,
                               const float *bias, int act, const void *residual, void *Y, void *Z, int out_kind,
                               int64_t M, int64_t N, int64_t K, void *workspace, int64_t workspace_bytes,
                               hipStream_t stream) {
  if (!A || !W || !a_row_scale || !Y) return TGEMM_ERR_NULL;
  if (out_kind != TGEMM_OUT_F32 && out_kind != TGEMM_OUT_BF16) return TGEMM_ERR_KIND;
  if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_VALUE;
  const int st = check_sizes(M, N, K);
  if (st != TGEMM_OK) return st;
  if (K > TGEMM_INT8_MAX_CONTRACTION) return TGEMM_ERR_BOUND;
  const Layout l = s8s8_layout(M, N, K, align_of(A), align_of(W));
  if (!workspace_ok(workspace, workspace_bytes, l.a_bytes + l.w_bytes)) return TGEMM_ERR_WORKSPACE;
  const int64_t ob = M * N * (out_kind == TGEMM_OUT_F32 ? 4 : 2);
  const Buf outs[] = {{Y, ob}, {Z, ob}, {workspace, workspace_bytes > 0 ? workspace_bytes : 0}};
  const Buf ins[] = {{A, M * K}, {W, N * K}, {a_row_scale, 4 * M}, {w_col_scale, 4 * N}, {bias, 4 * N}, {residual, ob}};
  const void *const same[3][2] = {{residual, residual}};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  Machine mc;
  if (ternary_gemm_machine(&mc.cus, &mc.xcds) != TGEMM_OK) return TGEMM_ERR_HIP;
  Out o{};
  o.ptr = Y;
  o.rs = a_row_scale;
  o.cs = w_col_scale;
  o.cscal = 1.f;
  o.kind = out_kind;
  o.bias = bias;
  o.res = residual;
  o.z = Z;
  o.act = act;
  const bool copy = K % 16 != 0 || align_of(A) % 16 != 0 || align_of(W) % 16 != 0;
  if (few_rows(M, N, K, copy)) {
    const FewArgs a = {A, W, o, M, N, K, 0, mc.xcds};
    const FewPlan p = few_plan(M, N, K, mc.cus);
    return p.mf == 1 ? pick_few<1>(a, p, stream) : pick_few<2>(a, p, stream);
  }
  int8_t *la = static_cast<int8_t *>(workspace), *lw = la + l.a_bytes;
  if (l.a_bytes) lay(A, la, M, K, l.kp, stream);
  if (l.w_bytes) lay(W, lw, N, K, l.kp, stream);
  const MArgs a = {l.a_bytes ? la : A, l.w_bytes ? lw : W, o, M, N, l.kp, 0, 0, 0, 0, 0, 0, 0};
  return pick_mm_act<EPI_COLS>(a, mc, stream);
}

int ternary_gemm_s8s8_plan(int64_t M, int64_t N, int64_t K, int64_t align, int act, int residual, int save, int out_kind,
                           int32_t cus, int32_t xcds, tgemm_plan *plan) {
  if (!plan) return TGEMM_ERR_NULL;
  int st = check_sizes(M, N, K);
  if (st != TGEMM_OK) return st;
  if (K > TGEMM_INT8_MAX_CONTRACTION) return TGEMM_ERR_BOUND;
  st = start_plan(M, N, K, act, out_kind, cus, xcds, plan);
  if (st != TGEMM_OK) return st;
  const bool copy = K % 16 != 0 || align < 1 || align % 16 != 0;
  plan->fast_path = copy ? 0 : 1;
  if (few_rows(M, N, K, copy)) {
    const FewPlan p = few_plan(M, N, K, cus);
    plan->kernel = TGEMM_KERNEL_INT8_FEW;
    plan->tile_rows = 16 * p.mf;
    plan->tile_cols = 16 * p.nb;
    plan->band_cols = (int32_t)ceil_div(N, 16 * p.nb);
    plan->tiles = plan->workgroups = plan->band_cols * ceil_div(M, 16 * p.mf);
    plan->tiles_per_workgroup = 1;
    plan->threads_per_workgroup = 64 * p.waves;
    plan->lds_bytes = 16 * p.waves * 16 * p.mf * (4 * p.nb + 1);
  } else {
    tile_plan(best_tile(M, N, round_up(K, 16), false, out_kind, act, save != 0, residual != 0, cus), M, N, {cus, xcds}, plan);
  }
  return TGEMM_OK;
}

int ternary_gemm_s8_gated_plan(int64_t M, int64_t N, int64_t K, int64_t align, int act, int save, int out_kind, int32_t cus,
                               int32_t xcds, tgemm_plan *plan) {
  if (!plan) return TGEMM_ERR_NULL;
  int st = check_sizes(M, N, K);
  if (st != TGEMM_OK) return st;
  if (K % 4 != 0) return TGEMM_ERR_PACK;
  if (K > TGEMM_TERNARY_MAX_CONTRACTION) return TGEMM_ERR_BOUND;
  st = start_plan(M, 2 * N, K, act, out_kind, cus, xcds, plan);
  if (st != TGEMM_OK) return st;
  if (align < 1) align = 1;
  if (gated_few_ok(M, N, K, align)) {
    plan->fast_path = 1;
    gated_few_plan(M, N, K, cus, xcds, plan);
  } else {
    plan->fast_path = K % 16 == 0 && align % 16 == 0;
    tile_plan(best_tile(M, 2 * N, round_up(K, 16), true, out_kind, act, save != 0, false, cus), M, 2 * N, {cus, xcds}, plan);
  }
  return TGEMM_OK;
}

int ternary_gemm_s8_gated_workspace(int64_t M, int64_t N, int64_t K, int64_t align, int64_t *bytes) {
  if (!bytes) return TGEMM_ERR_NULL;
  const int st = check_sizes(M, N, K);
  if (st != TGEMM_OK) return st;
  if (K % 4 != 0) return TGEMM_ERR_PACK;
  if (K > TGEMM_TERNARY_MAX_CONTRACTION) return TGEMM_ERR_BOUND;
  const Layout l = gated_layout(M, N, K, align > 0 ? align : 1, align > 0 ? align : 1);
  *bytes = l.a_bytes + l.w_bytes;
  return TGEMM_OK;
}

int ternary_gemm_s8_gated(const int8_t *A, const uint8_t *Wpacked, const float *a_row_scale, float gate_scale,
                          float up_scale, const float *bias, int act, void *Y, void *Z, int out_kind, int64_t M, int64_t N,
                          int64_t K, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!A || !Wpacked || !a_row_scale || !Y) return TGEMM_ERR_NULL;
  if (out_kind != TGEMM_OUT_F32 && out_kind != TGEMM_OUT_BF16) return TGEMM_ERR_KIND;
  if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_VALUE;
  const int st = check_sizes(M, N, K);
  if (st != TGEMM_OK) return st;
  if (K % 4 != 0) return TGEMM_ERR_PACK;
  if (K > TGEMM_TERNARY_MAX_CONTRACTION) return TGEMM_ERR_BOUND;
  const Layout l = gated_layout(M, N, K, align_of(A), align_of(Wpacked));
  if (!workspace_ok(workspace, workspace_bytes, l.a_bytes + l.w_bytes)) return TGEMM_ERR_WORKSPACE;
  const int64_t ob = M * N * (out_kind == TGEMM_OUT_F32 ? 4 : 2);
  const Buf outs[] = {{Y, ob}, {Z, 2 * ob}, {workspace, workspace_bytes > 0 ? workspace_bytes : 0}};
  const Buf ins[] = {{A, M * K}, {Wpacked, 2 * N * (K / 4)}, {a_row_scale, 4 * M}, {bias, 8 * N}};
  const void *const same[3][2] = {};
  if (alias(outs, ins, same)) return TGEMM_ERR_ALIAS;
  Machine mc;
  if (ternary_gemm_machine(&mc.cus, &mc.xcds) != TGEMM_OK) return TGEMM_ERR_HIP;
  if (!l.w_bytes)
    return gated_few({A, Wpacked, a_row_scale, bias, gate_scale, up_scale, Y, Z, out_kind, act, M, N, K}, mc.cus, mc.xcds,
                     stream);
  int8_t *la = static_cast<int8_t *>(workspace), *lw = la + l.a_bytes;
  if (l.a_bytes) lay(A, la, M, K, l.kp, stream);
  hipLaunchKernelGGL(lay_gated, lay_grid(2 * N), dim3(kLayT), 0, stream, Wpacked, lw, N, K, (int32_t)(l.kp / 16));
  Out o{};
  o.ptr = Y;
  o.rs = a_row_scale;
  o.cscal = gate_scale;
  o.cscal2 = up_scale;
  o.kind = out_kind;
  o.bias = bias;
  o.z = Z;
  o.act = act;
  const MArgs a = {l.a_bytes ? la : A, lw, o, M, 2 * N, l.kp, 0, 0, 0, 0, 0, 0, 0};
  return pick_mm_act<EPI_GATED>(a, mc, stream);
}

}  // extern "C"
