// Grouped linear forward for few rows a group (decode steps): every group's
// weights are streamed from HBM once and meet at most 32 rows, so the launch
// is bound by reading W.
//
//   z[r] = x[src(r)] W_e^T + b_e,  y[r] = act(z[r]) + residual[r]
//
// A workgroup owns a 32-row tile of a group and 128 rows of its W (SwiGLU:
// 64 gate rows and the 64 up rows of the same columns).  Its wavefronts are 4
// column slices x KS slices of K.  A wavefront holds 32 rows of W: it loads
// their MFMA fragments straight into registers, whole 128-byte lines of each
// row, four steps of 128 bytes of x at a time with every load of the four in
// flight; W passes through no LDS, which nothing but this wavefront would
// read.  The rows of x come through the caches the same way (all wavefronts
// and all workgroups of a group read the same few).  The KS partial products
// meet in LDS, added in slice order, and go through the common epilogue.
//
// Few workgroups (one token's down projection, a dense product of a few rows)
// leave compute units without weights to read.  The grid then has `parts`
// layers, each a contiguous share of K; they write fp32 partial rows, and a
// second launch adds them in order and runs the epilogue.  Mixtral-shaped down
// projection of one token (2 experts, 14336 -> 4096, bf16): 121 us in one
// launch, 60 with 8 parts, 55 with 16, 59 with 32.
//
// FP8 weights: 64 codes for each 128 bytes of x; a lane's 16 codes are 16
// consecutive elements of K, so its two fragments of x are neighbouring
// chunks.  The codes are widened to bf16 right before their MFMAs.
#include <algorithm>
#include <type_traits>

#include "linear.h"
#include "lds_ring.h"

namespace moe {
namespace {

constexpr int kBM = 32, kBZ = 128;   // rows of x and rows of W of a workgroup
constexpr int kPitch = kBZ + 4;      // floats of a staged result row

template <typename T, typename TW, bool GATED, int KS>
__global__ __launch_bounds__(256 * KS) void linear_rows_kernel(LinearArgs g,
                                                               float* __restrict__ partial) {
  constexpr bool FP8W = sizeof(TW) != sizeof(T);
  constexpr int COLS = GATED ? kBZ / 2 : kBZ;       // output columns of a workgroup
  constexpr int WSTEP = 128 * sizeof(TW) / sizeof(T);  // bytes of a W row per step
  constexpr int WLD = FP8W ? 1 : 2;                 // 16-byte loads of a W row per step
  __shared__ __attribute__((aligned(16))) float stg[KS * kBM * kPitch];

  const int nt = (g.out_dim + COLS - 1) / COLS;
  TileAt at;
  int col;
  if (!find_item(g.offsets, g.groups, g.rows, kBM, nt, at, col)) return;
  const int e = at.e, n0 = col * COLS, row0 = at.begin + at.m * kBM;
  const int valid = min(kBM, at.end - row0);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cw = wave & 3, kw = wave >> 2;
  const int fr = lane & 15, fq = lane >> 4;

  // lane: row fr (+ 16) of x, row fr of each of two 16-row blocks of W
  const size_t xrow = static_cast<size_t>(g.in_dim) * sizeof(T);
  const size_t wrow = static_cast<size_t>(g.in_dim) * sizeof(TW);
  const char* xp[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + min(i * 16 + fr, valid - 1);
    const int src = g.row_index != nullptr ? min(max(g.row_index[r], 0), g.x_rows - 1) : r;
    xp[i] = static_cast<const char*>(g.x) + src * xrow + (FP8W ? 2 * fq : fq) * 16;
  }
  const char* wp[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    // block j of the slice: gate and up of the same 16 columns, or 16 + 16 columns
    const int n = min(n0 + (GATED ? cw * 16 : cw * 32 + j * 16) + fr, g.out_dim - 1) +
                  (GATED && j == 1 ? g.out_dim : 0);
    wp[j] = static_cast<const char*>(g.w) +
            (static_cast<size_t>(e) * g.z_dim + n) * wrow + fq * 16;
  }
  // this wavefront's steps: slice kw of the share of K that layer blockIdx.y has
  const int steps = static_cast<int>(xrow / 128), parts = gridDim.y * KS;
  const int per = (steps + parts - 1) / parts, slice = blockIdx.y * KS + kw;
  const int s0 = min(slice * per, steps), s1 = min(s0 + per, steps);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    xp[i] += static_cast<size_t>(s0) * 128;
    wp[i] += static_cast<size_t>(s0) * WSTEP;
  }

  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // N steps at the pointers, then past them; RB 16-row blocks of x
  auto run = [&](auto n_, auto rb_) {
    constexpr int N = decltype(n_)::value, RB = decltype(rb_)::value;
    u32x4 w[N][2][WLD], x[N][RB][2];
#pragma unroll
    for (int s = 0; s < N; ++s) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < WLD; ++h)
          w[s][j][h] = *reinterpret_cast<const u32x4*>(wp[j] + s * WSTEP + h * 64);
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[s][i][h] = *reinterpret_cast<const u32x4*>(xp[i] + s * 128 + h * (FP8W ? 16 : 64));
    }
    // all of them are issued before the first is waited for
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      xp[i] += N * 128;
      wp[i] += N * WSTEP;
    }
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          u32x4 b;
          if constexpr (FP8W)
            b = e4m3x8_to_bf16(make_uint2(w[s][j][0][2 * h], w[s][j][0][2 * h + 1]));
          else
            b = w[s][j][h];
#pragma unroll
          for (int i = 0; i < RB; ++i) acc[i][j] = Mfma<T>::step(x[s][i][h], b, acc[i][j]);
        }
  };
  auto loop = [&](auto n_, auto rb_) {
    constexpr int N = decltype(n_)::value;
    int s = s0;
    for (; s + N <= s1; s += N) run(n_, rb_);
    for (; s < s1; ++s) run(std::integral_constant<int, 1>{}, rb_);
  };
  using std::integral_constant;
  if (valid > 16) loop(integral_constant<int, FP8W ? 4 : 2>{}, integral_constant<int, 2>{});
  else loop(integral_constant<int, 4>{}, integral_constant<int, 1>{});

  // partial products [kw][row][W row of the workgroup]; SwiGLU: gate columns
  // 0 .. 63, up columns 64 .. 127
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        stg[(kw * kBM + i * 16 + 4 * fq + r) * kPitch +
            (GATED ? j * 64 + cw * 16 : cw * 32 + j * 16) + fr] = acc[i][j][r];
  if constexpr (KS == 1) {
    if (partial != nullptr) {
      lds_barrier();
      float* const p = partial + (static_cast<size_t>(blockIdx.y) * g.rows + row0) * g.z_dim;
      const int c = tid % (kBZ / 8) * 8;
      const int n = n0 + (GATED ? c % 64 : c), z = GATED && c >= 64 ? g.out_dim + n : n;
      for (int row = tid / (kBZ / 8); row < valid; row += 256 / (kBZ / 8)) {
        float v[8];
        load8<float>(stg + row * kPitch + c, v);
        if (n < g.out_dim) store8<float>(p + static_cast<size_t>(row) * g.z_dim + z, v);
      }
      return;
    }
  }
  const int c = tid % (COLS / 8) * 8, n = n0 + c;
  const bool in = n < g.out_dim;
  float sv[8], su[8], bv[8], bu[8];
  const size_t eo = static_cast<size_t>(e) * g.z_dim + n;
  load_cols8(g.w_scale, eo, in, 1.f, sv);
  load_cols8(g.bias, eo, in, 0.f, bv);
  if (GATED) {
    load_cols8(g.w_scale, eo + g.out_dim, in, 1.f, su);
    load_cols8(g.bias, eo + g.out_dim, in, 0.f, bu);
  }
  lds_barrier();
  for (int row = tid / (COLS / 8); row < kBM; row += 256 * KS / (COLS / 8)) {
    const bool ok = row < valid && in;
    Raw8<T> res;
    load_residual<T>(g, row0 + row, n, ok, res);
    float v[8], u[8];
    load8<float>(stg + row * kPitch + c, v);
    if (GATED) load8<float>(stg + row * kPitch + 64 + c, u);
#pragma unroll
    for (int q = 1; q < KS; ++q) {
      float t[8];
      load8<float>(stg + (q * kBM + row) * kPitch + c, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += t[i];
      if (GATED) {
        load8<float>(stg + (q * kBM + row) * kPitch + 64 + c, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] += t[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = v[i] * sv[i] + bv[i];
      if (GATED) u[i] = u[i] * su[i] + bu[i];
    }
    linear_epilogue8<T, GATED>(g, row0 + row, n, ok, v, u, res);
  }
}

// The epilogue of a forward split over K: adds the parts of a row in order.
// One workgroup per row and 2048 columns of y.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void join_rows_kernel(LinearArgs g,
                                                        const float* __restrict__ partial,
                                                        int parts) {
  const int row = blockIdx.x, lane = threadIdx.x & 63;
  // the row's group: the groups before it end at or before it
  int e = 0;
  for (int i0 = 0; i0 < g.groups; i0 += 64) {
    const int i = i0 + lane;
    const int2 r = group_range(g.offsets, min(i, g.groups - 1), g.rows);
    e += __popcll(__ballot(i < g.groups && r.y <= row));
  }
  if (e >= g.groups || group_range(g.offsets, e, g.rows).x > row) return;
  const int n = (blockIdx.y * 256 + threadIdx.x) * 8;
  const bool in = n < g.out_dim;
  Raw8<T> res;
  load_residual<T>(g, row, n, in, res);
  float v[8], u[8], s[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
  const float* p = partial + static_cast<size_t>(row) * g.z_dim + n;
  for (int q = 0; q < parts && in; ++q, p += static_cast<size_t>(g.rows) * g.z_dim) {
    float t[8];
    load8<float>(p, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
    if (GATED) {
      load8<float>(p + g.out_dim, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += t[i];
    }
  }
  const size_t eo = static_cast<size_t>(e) * g.z_dim + n;
  load_cols8(g.w_scale, eo, in, 1.f, s);
  load_cols8(g.bias, eo, in, 0.f, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * s[i] + b[i];
  if (GATED) {
    load_cols8(g.w_scale, eo + g.out_dim, in, 1.f, s);
    load_cols8(g.bias, eo + g.out_dim, in, 0.f, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = u[i] * s[i] + b[i];
  }
  linear_epilogue8<T, GATED>(g, row, n, in, v, u, res);
}

// Workgroups of one layer of the grid (all tiles there can be).
long rows_blocks(const LinearArgs& g) {
  const int cols = g.act == kActSwiglu ? kBZ / 2 : kBZ;
  const long tiles = g.rows / kBM + std::min(g.groups, g.rows);
  return tiles * ((g.out_dim + cols - 1) / cols);
}

template <typename T, typename TW, bool GATED, int KS>
hipError_t launch_ks(const LinearArgs& g, int parts, float* partial, hipStream_t s) {
  constexpr int COLS = GATED ? kBZ / 2 : kBZ;
  const long nt = (g.out_dim + COLS - 1) / COLS;
  hipLaunchKernelGGL((linear_rows_kernel<T, TW, GATED, KS>),
                     dim3(static_cast<unsigned>(item_grid(g.rows, g.groups, kBM, nt)), parts),
                     dim3(256 * KS), 0, s, g, partial);
  return hipGetLastError();
}

template <typename T, typename TW, bool GATED>
hipError_t launch_t(const LinearArgs& g, int cus, float* partial, hipStream_t s) {
  const int parts = linear_rows_parts(static_cast<int>(sizeof(T)), g, cus);
  if (parts > 1) {
    const hipError_t err = launch_ks<T, TW, GATED, 1>(g, parts, partial, s);
    if (err != hipSuccess) return err;
    return launch_join_rows(sizeof(T) == 2 ? 1 : 0, g, partial, parts, s);
  }
  // Two slices of K in a workgroup where one would give a compute unit fewer
  // than 6 wavefronts.  One / two slices: 448 workgroups (one FP8 token's gate
  // and up projection) 46.5 / 51.7 us, 224 (8 rows, 4096 -> 2 x 14336) 54 / 49,
  // 170 (2 rows, 8192 -> 2 x 10880) 92 / 76; four measured as two.
  if (rows_blocks(g) * 4 >= 6L * cus) return launch_ks<T, TW, GATED, 1>(g, 1, nullptr, s);
  return launch_ks<T, TW, GATED, 2>(g, 1, nullptr, s);
}

template <typename T>
hipError_t launch_join_t(const LinearArgs& g, const float* partial, int parts, hipStream_t s) {
  const dim3 grid(g.rows, (g.out_dim + 2047) / 2048);
  if (g.act == kActSwiglu)
    hipLaunchKernelGGL((join_rows_kernel<T, true>), grid, dim3(256), 0, s, g, partial, parts);
  else
    hipLaunchKernelGGL((join_rows_kernel<T, false>), grid, dim3(256), 0, s, g, partial, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_join_rows(int dtype, const LinearArgs& g, const float* partial, int parts,
                            hipStream_t s) {
  return dtype == 1 ? launch_join_t<bf16_t>(g, partial, parts, s)
                    : launch_join_t<float>(g, partial, parts, s);
}

bool linear_rows_fits(const LinearArgs& g) {
  return rows_blocks(g) < (1L << 23);  // 2^32 threads, the XCDs' shares rounded up
}

// Fewer workgroups than half the compute units: as many parts as make four for
// each, none shorter than 8 steps.
int linear_rows_parts(int elem_bytes, const LinearArgs& g, int cus) {
  const long blocks = rows_blocks(g), steps = static_cast<long>(g.in_dim) * elem_bytes / 128;
  if (blocks <= 0 || blocks >= cus / 2) return 1;
  const long parts = std::min((4L * cus + blocks - 1) / blocks, steps / 8);
  return parts < 2 ? 1 : static_cast<int>(std::min(parts, 64L));
}

hipError_t launch_linear_rows(int dtype, bool wfp8, const LinearArgs& g, int cus, float* partial,
                              hipStream_t s) {
  const bool gated = g.act == kActSwiglu;
  if (wfp8)
    return gated ? launch_t<bf16_t, uint8_t, true>(g, cus, partial, s)
                 : launch_t<bf16_t, uint8_t, false>(g, cus, partial, s);
  if (dtype == 1)
    return gated ? launch_t<bf16_t, bf16_t, true>(g, cus, partial, s)
                 : launch_t<bf16_t, bf16_t, false>(g, cus, partial, s);
  return gated ? launch_t<float, float, true>(g, cus, partial, s)
               : launch_t<float, float, false>(g, cus, partial, s);
}

}  // namespace moe
