// Grouped linear maps on register-staged 128 x 128 or 64 x 64 tiles: every
// type and direction in one kernel.
//
//   forward  z[r] = x[src(r)] W_e^T + b_e,  y[r] = act(z[r]) + residual[r]
//   dX       dX[r] = dz[r] W_e
//   dW       dW_e = sum_r dz[r]^T x[src(r)]
//
// All three are C = A B^T over K, where an operand lies in memory either by
// its rows (K contiguous: x, dz and W of the forward, dz of dX) or by its
// K-rows (the rows of C's side contiguous: W of dX, dz and x of dW).  A
// K-row operand is turned while it is stored to LDS, so both kinds feed the
// same 16-byte MFMA fragments.
//
// One workgroup owns a B x B tile of one group (B = 128, or 64 where the
// larger tiles would leave compute units without work: launch_t), its 4
// wavefronts a quarter each; a K step is 128 bytes of every row, fetched into
// registers one or two steps before it is multiplied out of one of two LDS
// buffers.  Rows past a group's end repeat its last row (results not written);
// K-rows past it are zeros in both operands, so that no NaN of a neighbouring
// group enters.  A forward of few tiles is split over K: the layers of the grid
// write fp32 partial tiles, and a second launch adds them in order and runs the
// epilogue (linear_tile_parts).
// fp32 reaches 130 of the 153 TFLOP/s of a large library product (8192 rows,
// 4096 -> 4096), 105 with 8 groups of 256 rows.
#include <algorithm>
#include <type_traits>

#include "linear.h"
#include "lds_ring.h"

namespace moe {
namespace {

constexpr int kFwd = 0, kDx = 1, kDw = 2;

// One operand tile: L x 32 rows of 128 bytes, L 16-byte chunks a thread, held
// for two K steps (slots P).
template <typename T, typename TW, bool KROW, int L>
struct Operand;

// K contiguous: chunk c = tid + 256 i is 16 bytes (8 codes of an FP8 weight)
// ch = c % 8 of tile row c / 8.
template <typename T, typename TW, int L>
struct Operand<T, TW, false, L> {
  static constexpr int CB = 16 * static_cast<int>(sizeof(TW)) / static_cast<int>(sizeof(T));
  static constexpr bool FP8 = sizeof(TW) != sizeof(T);
  const char* p[L];
  int steps;  // K steps there are (a load past them repeats the last)
  u32x4 v[2][FP8 ? 1 : L];
  uint2 c8[2][FP8 ? L : 1];  // codes, widened on their way into LDS
  template <int P> __device__ __forceinline__ void load(int step) {
    const size_t off = static_cast<size_t>(min(step, steps - 1)) * 8 * CB;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if constexpr (FP8) c8[P][i] = *reinterpret_cast<const uint2*>(p[i] + off);
      else v[P][i] = *reinterpret_cast<const u32x4*>(p[i] + off);
    }
  }
  template <int P> __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int c = threadIdx.x + 256 * i;
      u32x4* const d = reinterpret_cast<u32x4*>(lds + lds_swz(c >> 3, c & 7));
      if constexpr (FP8) *d = e4m3x8_to_bf16(c8[P][i]);
      else *d = v[P][i];
    }
  }
};

// K-rows: chunk c is 16 bytes (V columns) of K-row c % KE of the step.
template <typename T, int L>
struct Operand<T, T, true, L> {
  static constexpr int V = 16 / static_cast<int>(sizeof(T)), KE = 128 / static_cast<int>(sizeof(T));
  const T* base;              // K-row 0 of the tile's first column
  size_t ld;                  // elements of a K-row
  int cols, krows;            // columns of the operand from the tile's first; K-rows there are
  const int32_t* index;       // source row of K-row j, or null
  int index_rows;             // rows the index may name
  u32x4 v[2][L];
  template <int P> __device__ __forceinline__ void load(int step) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int c = threadIdx.x + 256 * i;
      const int kk = step * KE + c % KE, col = c / KE * V;
      v[P][i] = u32x4{0u, 0u, 0u, 0u};
      if (kk < krows && col < cols) {
        const int src = index != nullptr ? min(max(index[kk], 0), index_rows - 1) : kk;
        v[P][i] = *reinterpret_cast<const u32x4*>(base + static_cast<size_t>(src) * ld + col);
      }
    }
  }
  template <int P> __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int c = threadIdx.x + 256 * i;
      const int kb = c % KE * static_cast<int>(sizeof(T)), col = c / KE * V;
      const T* e = reinterpret_cast<const T*>(&v[P][i]);
#pragma unroll
      for (int q = 0; q < V; ++q)
        *reinterpret_cast<T*>(lds + lds_swz(col + q, kb >> 4) + (kb & 15)) = e[q];
    }
  }
};

template <typename T, typename TW, int MODE, bool GATED, int B>
__global__ __launch_bounds__(256, 2) void linear_tile_kernel(LinearArgs g, const T* __restrict__ dz,
                                                             T* __restrict__ out,
                                                             float* __restrict__ partial) {
  constexpr int TILE = B * 128;
  constexpr int NB = B / 32;           // 16-row and 16-column blocks of a wavefront
  constexpr int L = B / 32;            // 16-byte chunks of an operand tile a thread
  constexpr int PITCH = B + 4;         // floats of a staged result row
  constexpr int STG = B * PITCH * 4;
  __shared__ __attribute__((aligned(1024))) char smem[4 * TILE > STG ? 4 * TILE : STG];
  constexpr int COLS = GATED ? B / 2 : B;  // output columns of a tile

  const int n_dim = MODE == kFwd ? g.out_dim : g.in_dim;  // columns of C
  const int nt = (n_dim + COLS - 1) / COLS;
  int e, m0, n0, valid, seg, count;
  if constexpr (MODE == kDw) {
    const int mt = (g.z_dim + B - 1) / B;
    const int per = mt * nt;
    e = blockIdx.x / per;
    const int r = blockIdx.x - e * per;
    m0 = (r % mt) * B;
    n0 = (r / mt) * COLS;
    const int2 range = group_range(g.offsets, e, g.rows);
    seg = range.x;
    count = range.y - range.x;
    valid = min(B, g.z_dim - m0);
  } else {
    TileAt at;
    int col;
    if (!find_item(g.offsets, g.groups, g.rows, B, nt, at, col)) return;
    e = at.e;
    m0 = at.m * B;
    n0 = col * COLS;
    seg = at.begin;
    count = at.end - at.begin;
    valid = min(B, count - m0);
  }

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // wavefront (wm, wn): 16-row blocks wm, wm + 2, ..., columns B / 2 wn ..; taking
  // turns, the two share the rows of a partly filled tile, and run the MFMAs
  // of the `live` blocks that hold rows
  const int wm = wave >> 1, wn = wave & 1;
  const int live = __builtin_amdgcn_readfirstlane(min(max((valid - wm * 16 + 31) / 32, 0), NB));
  const size_t wmat = static_cast<size_t>(g.z_dim) * g.in_dim;

  Operand<T, T, MODE == kDw, L> opa;
  Operand<T, TW, MODE != kFwd, L> opb;
  int nsteps;
  if constexpr (MODE == kDw) {
    opa.base = dz + static_cast<size_t>(seg) * g.z_dim + m0;
    opa.ld = g.z_dim;
    opa.cols = g.z_dim - m0;
    opa.krows = count;
    opa.index = nullptr;
    opa.index_rows = 0;
    const bool gather = g.row_index != nullptr;
    opb.base = static_cast<const T*>(g.x) + (gather ? 0 : static_cast<size_t>(seg) * g.in_dim) + n0;
    opb.ld = g.in_dim;
    opb.cols = g.in_dim - n0;
    opb.krows = count;
    opb.index = gather ? g.row_index + seg : nullptr;
    opb.index_rows = g.x_rows;
    nsteps = (count + opb.KE - 1) / opb.KE;
  } else {
    const int k_dim = MODE == kFwd ? g.in_dim : g.z_dim;
    const char* src = MODE == kFwd ? static_cast<const char*>(g.x)
                                   : reinterpret_cast<const char*>(dz);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int c = tid + 256 * i;
      const int row = seg + m0 + min(c >> 3, valid - 1);
      int srow = row;
      if (MODE == kFwd && g.row_index != nullptr)
        srow = min(max(g.row_index[row], 0), g.x_rows - 1);
      opa.p[i] = src + static_cast<size_t>(srow) * k_dim * sizeof(T) + (c & 7) * 16;
    }
    nsteps = static_cast<int>(static_cast<size_t>(k_dim) * sizeof(T) / 128);
    int s0 = 0;  // first step of this layer's share
    if (MODE == kFwd && B == 64 && partial != nullptr) {
      const int per = (nsteps + gridDim.y - 1) / gridDim.y;
      s0 = min(static_cast<int>(blockIdx.y) * per, nsteps);
      nsteps = min(per, nsteps - s0);
#pragma unroll
      for (int i = 0; i < L; ++i) opa.p[i] += static_cast<size_t>(s0) * 128;
    }
    opa.steps = nsteps;
    if constexpr (MODE == kFwd) {
      opb.steps = nsteps;
      const char* w = static_cast<const char*>(g.w) + e * wmat * sizeof(TW);
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int c = tid + 256 * i, r = c >> 3;
        // SwiGLU: the tile's gate rows, then the up rows of the same columns
        const bool up = GATED && r >= COLS;
        const int n = min(n0 + (up ? r - COLS : r), g.out_dim - 1) + (up ? g.out_dim : 0);
        opb.p[i] = w + (static_cast<size_t>(n) * g.in_dim) * sizeof(TW) + (c & 7) * opb.CB +
                   static_cast<size_t>(s0) * 8 * opb.CB;
      }
    } else {
      opb.base = static_cast<const T*>(g.w) + e * wmat + n0;
      opb.ld = g.in_dim;
      opb.cols = g.in_dim - n0;
      opb.krows = g.z_dim;
      opb.index = nullptr;
      opb.index_rows = 0;
    }
  }

  f32x4 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto stage = [&](int q) -> char* { return smem + q * 2 * TILE; };
  auto compute = [&](const char* st, auto full_) {
#pragma unroll
    for (int kc = 0; kc < 2; ++kc) {
      const int ch = kc * 4 + (lane >> 4);
      u32x4 af[NB], bf[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        af[i] = *reinterpret_cast<const u32x4*>(st + lds_swz(i * 32 + wm * 16 + (lane & 15), ch));
        bf[i] = *reinterpret_cast<const u32x4*>(st + TILE +
                                                lds_swz(wn * (B / 2) + i * 16 + (lane & 15), ch));
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (decltype(full_)::value || i < live) {
#pragma unroll
          for (int j = 0; j < NB; ++j) acc[i][j] = Mfma<T>::step(af[i], bf[j], acc[i][j]);
        }
    }
  };
  // The forward leaves out the MFMAs of blocks without rows.  In dX and dW the
  // branches cost more than they save (7 % of the fp32 backward).
  auto multiply = [&](const char* st) {
    if (MODE != kFwd || live == NB) compute(st, std::true_type{});
    else if (live > 0) compute(st, std::false_type{});
  };
  // Two steps of loads in flight, but for the 128 x 128 tiles of dX and dW,
  // whose turned operand takes the registers (fp32 backward of 2048 rows, 4096
  // -> 2 x 2048: 1728 us with one step, 1807 with two; forward 950 / 896, 1000
  // bf16 rows of 4096 -> 1024 on 64 x 64 tiles 41 / 26).
  constexpr bool DEEP = MODE == kFwd || B == 64;
  if (!DEEP && nsteps > 0) {
    opa.template load<0>(0);
    opb.template load<0>(0);
    opa.template store<0>(stage(0));
    opb.template store<0>(stage(0) + TILE);
    lds_barrier();
    for (int s = 0; s < nsteps; ++s) {
      const bool more = s + 1 < nsteps;
      if (more) {
        opa.template load<0>(s + 1);
        opb.template load<0>(s + 1);
      }
      multiply(stage(s & 1));
      if (more) {
        opa.template store<0>(stage((s + 1) & 1));
        opb.template store<0>(stage((s + 1) & 1) + TILE);
      }
      lds_barrier();
    }
  } else if (nsteps > 0) {
    opa.template load<0>(0);
    opb.template load<0>(0);
    opa.template load<1>(1);
    opb.template load<1>(1);
    opa.template store<0>(stage(0));
    opb.template store<0>(stage(0) + TILE);
    lds_barrier();
    // two steps of loads in flight: step s + 2 is asked for while step s is
    // multiplied out of one buffer and step s + 1 waits to go into the other
    for (int s = 0;; s += 2) {
      opa.template load<0>(s + 2);
      opb.template load<0>(s + 2);
      multiply(stage(0));
      if (s + 1 >= nsteps) break;
      opa.template store<1>(stage(1));
      opb.template store<1>(stage(1) + TILE);
      lds_barrier();
      opa.template load<1>(s + 3);
      opb.template load<1>(s + 3);
      multiply(stage(1));
      if (s + 2 >= nsteps) break;
      opa.template store<0>(stage(0));
      opb.template store<0>(stage(0) + TILE);
      lds_barrier();
    }
    lds_barrier();
  }

  // the tile as fp32 rows in LDS, then 8 columns of a row per lane
  float* const stg = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        stg[(i * 32 + wm * 16 + 4 * (lane >> 4) + r) * PITCH + wn * (B / 2) + j * 16 +
            (lane & 15)] = acc[i][j][r];
  lds_barrier();
  // a lane keeps its columns: 256 is a multiple of COLS / 8
  const int c = tid % (COLS / 8) * 8, n = n0 + c;
  float sv[8], su[8], bv[8], bu[8];
  if constexpr (MODE == kFwd) {
    const size_t eo = static_cast<size_t>(e) * g.z_dim + n;
    load_cols8(g.w_scale, eo, n < n_dim, 1.f, sv);
    load_cols8(g.bias, eo, n < n_dim, 0.f, bv);
    if (GATED) {
      load_cols8(g.w_scale, eo + g.out_dim, n < n_dim, 1.f, su);
      load_cols8(g.bias, eo + g.out_dim, n < n_dim, 0.f, bu);
    }
  }
  for (int row = tid / (COLS / 8); row < B; row += 256 * 8 / COLS) {
    const bool ok = row < valid && n < n_dim;
    float v[8], u[8];
    load8<float>(stg + row * PITCH + c, v);
    if (MODE == kFwd && B == 64 && partial != nullptr) {
      if (ok) {
        float* const p = partial +
                         (static_cast<size_t>(blockIdx.y) * g.rows + seg + m0 + row) * g.z_dim + n;
        store8<float>(p, v);
        if (GATED) {
          load8<float>(stg + row * PITCH + COLS + c, u);
          store8<float>(p + g.out_dim, u);
        }
      }
    } else if constexpr (MODE == kFwd) {
      Raw8<T> res;
      load_residual<T>(g, seg + m0 + row, n, ok, res);
      if (GATED) load8<float>(stg + row * PITCH + COLS + c, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = v[i] * sv[i] + bv[i];
        if (GATED) u[i] = u[i] * su[i] + bu[i];
      }
      linear_epilogue8<T, GATED>(g, seg + m0 + row, n, ok, v, u, res);
    } else if (ok) {
      const size_t row0 = MODE == kDx ? static_cast<size_t>(seg) + m0 + row
                                      : static_cast<size_t>(e) * g.z_dim + m0 + row;
      store8<T>(out + row0 * g.in_dim + n0 + c, v);
    }
  }
}

template <typename T, typename TW, int MODE, int B>
hipError_t launch_b(const LinearArgs& g, const void* dz, void* out, hipStream_t s, int parts = 1,
                    float* partial = nullptr) {
  const bool gated = MODE == kFwd && g.act == kActSwiglu;
  const int cols = gated ? B / 2 : B;
  const long nt = ((MODE == kFwd ? g.out_dim : g.in_dim) + cols - 1) / cols;
  const long blocks = MODE == kDw ? static_cast<long>(g.groups) * ((g.z_dim + B - 1) / B) * nt
                                  : item_grid(g.rows, g.groups, B, nt);
  if (blocks > 0x7fffffffL) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks), parts);
  if constexpr (MODE == kFwd) {
    if (gated) {
      hipLaunchKernelGGL((linear_tile_kernel<T, TW, MODE, true, B>), grid, dim3(256), 0, s, g,
                         static_cast<const T*>(dz), static_cast<T*>(out), partial);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((linear_tile_kernel<T, TW, MODE, false, B>), grid, dim3(256), 0, s, g,
                     static_cast<const T*>(dz), static_cast<T*>(out), partial);
  return hipGetLastError();
}

// Tiles of b rows that a product of the mode has; a group's last row tile
// counts half, for its rows are not known here.
template <int MODE> long tiles_of(const LinearArgs& g, long b) {
  const long cols = MODE == kFwd && g.act == kActSwiglu ? b / 2 : b;
  const long nt = ((MODE == kFwd ? g.out_dim : g.in_dim) + cols - 1) / cols;
  if (MODE == kDw) return g.groups * ((g.z_dim + b - 1) / b) * nt;
  if (g.groups == 1) return (g.rows + b - 1) / b * nt;
  return (2 * g.rows / b + std::min(g.groups, g.rows)) * nt / 2;
}

// 64 x 64 tiles where the 128 x 128 ones are fewer than the compute units (a
// small product is bound by one tile's chain of steps, and theirs is a quarter
// as long), and for fp32, which is bound by its MFMAs with either, where the
// larger tiles would not fill their rounds of two on each compute unit: tile
// for tile they are 12 % faster.  fp32 us on large / small tiles:
//   8 groups of 256 rows, 4096 -> 2 x 2048: forward 897 / 657, dX 887 / 775, dW
//   (8192 tiles) 884 / 934; 2048 -> 2048 of 3000 rows (384) 275 / 249, of 4096
//   (512) 268 / 295, of 5000 (640) 525 / 402, of 12000 (1504) 807 / 877
template <typename T, typename TW, int MODE>
hipError_t launch_t(const LinearArgs& g, const void* dz, void* out, int cus, hipStream_t s,
                    float* partial = nullptr) {
  if constexpr (MODE == kFwd) {
    const int parts = linear_tile_parts(static_cast<int>(sizeof(T)), g, cus);
    if (parts > 1) {
      const hipError_t err = launch_b<T, TW, MODE, 64>(g, dz, out, s, parts, partial);
      return err != hipSuccess ? err
                               : launch_join_rows(sizeof(T) == 2 ? 1 : 0, g, partial, parts, s);
    }
  }
  const bool gated = MODE == kFwd && g.act == kActSwiglu;
  const long large = tiles_of<MODE>(g, 128), round = 2L * cus;
  const bool small =
      large < cus || (std::is_same_v<T, float> &&
                      tiles_of<MODE>(g, 64) * 28 < (large + round - 1) / round * round * 100);
  // (half of 64 columns is no checkpoint block)
  if (small && !(gated && g.z_codes != nullptr)) return launch_b<T, TW, MODE, 64>(g, dz, out, s);
  return launch_b<T, TW, MODE, 128>(g, dz, out, s);
}

}  // namespace

// Fewer 64 x 64 tiles than compute units: as many parts as leave two workgroups
// or less for each, none shorter than 16 steps.  bf16 us whole / split: 64 rows
// of 14336 -> 4096 108 / 50, of 4096 -> 4096 25 / 15 (19 with 8 parts of 8
// steps), of 4096 -> 14336 (224 tiles) 37.4 / 34.5; with more tiles than units
// (1200 rows of 4 groups 4096 -> 2 x 704, 456) 32 / 34.
int linear_tile_parts(int elem_bytes, const LinearArgs& g, int cus) {
  const long tiles = tiles_of<kFwd>(g, 64), steps = static_cast<long>(g.in_dim) * elem_bytes / 128;
  if (tiles <= 0 || tiles > cus) return 1;
  const long parts = std::min(2L * cus / tiles, steps / 16);
  return parts < 2 ? 1 : static_cast<int>(std::min(parts, 16L));
}

hipError_t launch_linear_tile(int dtype, bool wfp8, const LinearArgs& g, int cus, float* partial,
                              hipStream_t s) {
  if (wfp8) return launch_t<bf16_t, uint8_t, kFwd>(g, nullptr, nullptr, cus, s, partial);
  if (dtype == 1) return launch_t<bf16_t, bf16_t, kFwd>(g, nullptr, nullptr, cus, s, partial);
  return launch_t<float, float, kFwd>(g, nullptr, nullptr, cus, s, partial);
}

hipError_t launch_linear_dx_tile(int dtype, const LinearArgs& g, const void* dz, void* dx, int cus,
                                 hipStream_t s) {
  if (dtype == 1) return launch_t<bf16_t, bf16_t, kDx>(g, dz, dx, cus, s);
  return launch_t<float, float, kDx>(g, dz, dx, cus, s);
}

hipError_t launch_linear_dw_tile(int dtype, const LinearArgs& g, const void* dz, void* dw, int cus,
                                 hipStream_t s) {
  if (dtype == 1) return launch_t<bf16_t, bf16_t, kDw>(g, dz, dw, cus, s);
  return launch_t<float, float, kDw>(g, dz, dw, cus, s);
}

}  // namespace moe
