// Packing for the 8-bit products: rows (as they are, activated, or a gradient
// through an activation), turned rows and weights as E4M3 codes with one power
// of two for each block of 128.
//
//   e = the smallest power of two with max |v| / 2^e <= 448 over the block
//   code = E4M3(v / 2^e), to nearest even
//
// v / 2^e is exact, so a code has one rounding (at most 2^-4 of the value), and
// turned codes and row codes are made from the same fp32 values.  Every call is
// one pass: bound by HBM.
#include "block.h"

namespace moe {
namespace {

// Group of turned block b and its rows [begin, end) of the whole; end <= begin:
// the block belongs to no group.  The groups' first blocks rise by one at
// least, so the last one that starts at or before b owns it.
struct RowBlock {
  int begin, end;
};
__device__ __forceinline__ RowBlock find_block(const int32_t* offsets, int groups, int rows,
                                               int b) {
  if (offsets == nullptr) return RowBlock{b * kBlk, min(rows, (b + 1) * kBlk)};
  int lo = 0, hi = groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (turned_first(min(max(offsets[mid], 0), rows), mid) <= b) lo = mid;
    else hi = mid - 1;
  }
  const int2 r = group_range(offsets, lo, rows);
  const long at = static_cast<long>(r.x) + static_cast<long>(b - turned_first(r.x, lo)) * kBlk;
  if (at < r.x || at >= r.y) return RowBlock{0, 0};
  return RowBlock{static_cast<int>(at), min(r.y, static_cast<int>(at) + kBlk)};
}

// 8 packed values of a row at column c (a multiple of 8).
template <typename T, int ACT, bool BACK>
__device__ __forceinline__ void values8(const PackArgs& g, int row, int c, float* v) {
  int src = row;
  if (g.row_index != nullptr) src = min(max(g.row_index[row], 0), g.x_rows - 1);
  const T* const x = static_cast<const T*>(g.x);
  if constexpr (ACT == kActSwiglu) {
    const int half = BACK ? g.cols / 2 : g.cols;
    const int at = BACK && c >= half ? c - half : c;
    const T* const z = x + static_cast<size_t>(src) * 2 * half + at;
    float a[8], b[8];
    load8<T>(z, a);
    load8<T>(z + half, b);
    if constexpr (!BACK) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a[i] * sigmoid_close(a[i]) * b[i];
    } else {
      float d[8];
      load8<T>(static_cast<const T*>(g.dy) + static_cast<size_t>(row) * half + at, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = sigmoid_close(a[i]);
        v[i] = c >= half ? d[i] * a[i] * p : d[i] * b[i] * p * (1.0f + a[i] * (1.0f - p));
      }
    }
  } else {
    load8<T>(x + static_cast<size_t>(src) * g.cols + c, v);
    if constexpr (!BACK) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = ACT == kActSilu ? v[i] * sigmoid_close(v[i]) : activate<float>(ACT, v[i]);
    } else {
      float d[8];
      load8<T>(static_cast<const T*>(g.dy) + static_cast<size_t>(row) * g.cols + c, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (ACT == kActSilu) {
          const float p = sigmoid_close(v[i]);
          v[i] = d[i] * p * (1.0f + v[i] * (1.0f - p));
        } else {
          v[i] = d[i] * activate_slope<float>(ACT, v[i]);
        }
      }
    }
  }
}

// The largest of the 16 lanes that hold a row's block.
__device__ __forceinline__ float max16(float m) {
  m = fmaxf(m, __shfl_xor(m, 1, 64));
  m = fmaxf(m, __shfl_xor(m, 2, 64));
  m = fmaxf(m, __shfl_xor(m, 4, 64));
  return fmaxf(m, __shfl_xor(m, 8, 64));
}

constexpr int kRowsWg = 16;

// Rows only: a workgroup packs 16 rows, 16 lanes to a block of 128 columns.
template <typename T, int ACT, bool BACK>
__global__ __launch_bounds__(256) void pack_rows_kernel(PackArgs g, int blocks_wg) {
  const int tid = threadIdx.x, l16 = tid & 15;
  const int row = blockIdx.x * kRowsWg + (tid >> 4);
  int first = 0, last = g.rows;
  if (g.offsets != nullptr) {
    first = min(max(g.offsets[0], 0), g.rows);
    last = min(max(g.offsets[g.groups], 0), g.rows);
  }
  const bool live = row >= first && row < last;
  const int blocks = (g.cols + kBlk - 1) / kBlk;
  const int b0 = blockIdx.y * blocks_wg, b1 = min(blocks, b0 + blocks_wg);
  for (int b = b0; b < b1; ++b) {
    const int c = b * kBlk + l16 * 8;
    const bool in = live && c < g.cols;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) values8<T, ACT, BACK>(g, row, c, v);
    bool bad = false;
    const int e = e8m0_of(max16(finite_max8(v, bad)));
    if (in)
      *reinterpret_cast<uint2*>(g.codes + static_cast<size_t>(row) * g.cols + c) =
          encode8_finite(v, e8m0_inverse(e), bad);
    if (live && l16 == 0) g.scale[b * g.line + row] = static_cast<uint8_t>(e);
  }
}

// Both forms: a workgroup packs 128 rows of a group by 128 columns; a thread
// holds 8 columns of 8 consecutive rows.  Column sums of maxima go through LDS,
// and so do the turned codes: 8-byte pieces (8 rows of a column), piece p of
// column c at place p ^ (c / 8 mod 16), so that the 16 lanes of a row's columns
// write to different banks.
struct TileShared {
  __attribute__((aligned(16))) uint8_t t[kBlk * kBlk];
  float top[4][kBlk];
};
__device__ __forceinline__ void turn_codes(TileShared& sh, const uint32_t (*q)[8], int l16,
                                           int slot) {
  // q[r]: 8 codes of row r as two words, [0]: columns 0-3, [1]: 4-7
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      lo |= ((q[j >> 2][r] >> (8 * (j & 3))) & 0xffu) << (8 * r);
      hi |= ((q[j >> 2][r + 4] >> (8 * (j & 3))) & 0xffu) << (8 * r);
    }
    const int col = l16 * 8 + j;
    *reinterpret_cast<uint2*>(sh.t + col * kBlk + ((slot ^ l16) << 3)) = make_uint2(lo, hi);
  }
}
// 16 codes of a column, rows 16 h .. + 15.
__device__ __forceinline__ uint4 turned16(const TileShared& sh, int col, int h) {
  const int key = (col >> 3) & 15;
  const uint2 a = *reinterpret_cast<const uint2*>(sh.t + col * kBlk + (((2 * h) ^ key) << 3));
  const uint2 b = *reinterpret_cast<const uint2*>(sh.t + col * kBlk + (((2 * h + 1) ^ key) << 3));
  return make_uint4(a.x, a.y, b.x, b.y);
}

template <typename T, int ACT, bool BACK>
__global__ __launch_bounds__(256) void pack_both_kernel(PackArgs g) {
  __shared__ TileShared sh;
  const int tid = threadIdx.x, l16 = tid & 15, slot = tid >> 4;
  const int blocks = (g.cols + kBlk - 1) / kBlk;
  const int tb = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const RowBlock rb = find_block(g.offsets, g.groups, g.rows, tb);
  if (rb.end <= rb.begin) return;
  const int c = cb * kBlk + l16 * 8;
  const bool cin = c < g.cols;
  float v[8][8];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = rb.begin + slot * 8 + r;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[r][i] = 0.f;
    if (cin && row < rb.end) values8<T, ACT, BACK>(g, row, c, v[r]);
  }
  float col[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = rb.begin + slot * 8 + r;
    const float m = finite_max8(v[r], bad);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(v[r][i]);
      col[i] = fmaxf(col[i], a < INFINITY ? a : 0.f);
    }
    if (g.codes != nullptr) {
      const int e = e8m0_of(max16(m));
      if (cin && row < rb.end)
        *reinterpret_cast<uint2*>(g.codes + static_cast<size_t>(row) * g.cols + c) =
            encode8_finite(v[r], e8m0_inverse(e), bad);
      if (l16 == 0 && row < rb.end) g.scale[cb * g.line + row] = static_cast<uint8_t>(e);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    col[i] = fmaxf(col[i], __shfl_xor(col[i], 16, 64));
    col[i] = fmaxf(col[i], __shfl_xor(col[i], 32, 64));
    if ((tid & 63) < 16) sh.top[tid >> 6][l16 * 8 + i] = col[i];
  }
  __syncthreads();
  float inv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = l16 * 8 + i;
    const int e = e8m0_of(fmaxf(fmaxf(sh.top[0][k], sh.top[1][k]), fmaxf(sh.top[2][k], sh.top[3][k])));
    inv[i] = e8m0_inverse(e);
    if (slot == 0 && cin) g.scale_t[static_cast<size_t>(tb) * g.cols + c + i] = static_cast<uint8_t>(e);
  }
  uint32_t q[2][8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[r][i] *= inv[i];
    const uint2 u = encode8_finite(v[r], 1.0f, bad);
    q[0][r] = u.x;
    q[1][r] = u.y;
  }
  turn_codes(sh, q, l16, slot);
  __syncthreads();
  uint8_t* const out = g.codes_t + (static_cast<size_t>(tb) * g.cols + cb * kBlk) * kBlk;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int p = k * 256 + tid;  // 16-byte pieces of the tile, column after column
    if (cb * kBlk + (p >> 3) < g.cols)
      *reinterpret_cast<uint4*>(out + static_cast<size_t>(p) * 16) = turned16(sh, p >> 3, p & 7);
  }
}

// A block of 128 x 128 weights, both ways round.
template <typename T>
__global__ __launch_bounds__(256) void pack_weights_kernel(PackWeightArgs g) {
  __shared__ TileShared sh;
  const int tid = threadIdx.x, l16 = tid & 15, slot = tid >> 4;
  const int ib = (g.in + kBlk - 1) / kBlk, ob = (g.out + kBlk - 1) / kBlk;
  const int cb = blockIdx.x % ib, q0 = blockIdx.x / ib;
  const int rbk = q0 % ob, e = q0 / ob;
  const int c = cb * kBlk + l16 * 8;
  const bool cin = c < g.in;
  const size_t mat = static_cast<size_t>(e) * g.out * g.in;
  const T* const w = static_cast<const T*>(g.w) + mat;
  float v[8][8];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = rbk * kBlk + slot * 8 + r;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[r][i] = 0.f;
    if (cin && row < g.out) load8<T>(w + static_cast<size_t>(row) * g.in + c, v[r]);
  }
  float m = 0.f;
#pragma unroll
  for (int r = 0; r < 8; ++r) m = fmaxf(m, finite_max8(v[r], bad));
  m = max16(m);
  m = fmaxf(m, __shfl_xor(m, 16, 64));
  m = fmaxf(m, __shfl_xor(m, 32, 64));
  if ((tid & 63) == 0) sh.top[tid >> 6][0] = m;
  __syncthreads();
  const int s = e8m0_of(fmaxf(fmaxf(sh.top[0][0], sh.top[1][0]), fmaxf(sh.top[2][0], sh.top[3][0])));
  const float inv = e8m0_inverse(s);
  if (tid == 0) {
    if (g.codes != nullptr)
      g.scale[(static_cast<size_t>(e) * ob + rbk) * ib + cb] = static_cast<uint8_t>(s);
    if (g.codes_t != nullptr)
      g.scale_t[(static_cast<size_t>(e) * ib + cb) * ob + rbk] = static_cast<uint8_t>(s);
  }
  uint32_t q[2][8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = rbk * kBlk + slot * 8 + r;
    const uint2 u = encode8_finite(v[r], inv, bad);
    q[0][r] = u.x;
    q[1][r] = u.y;
    if (g.codes != nullptr && cin && row < g.out)
      *reinterpret_cast<uint2*>(g.codes + mat + static_cast<size_t>(row) * g.in + c) = u;
  }
  if (g.codes_t == nullptr) return;
  turn_codes(sh, q, l16, slot);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int p = k * 256 + tid, col = cb * kBlk + (p >> 3), row = rbk * kBlk + (p & 7) * 16;
    if (col < g.in && row < g.out)
      *reinterpret_cast<uint4*>(g.codes_t + mat + static_cast<size_t>(col) * g.out + row) =
          turned16(sh, p >> 3, p & 7);
  }
}

template <typename T, int ACT, bool BACK>
hipError_t pack_t(const PackArgs& g, hipStream_t s) {
  const int blocks = (g.cols + kBlk - 1) / kBlk;
  if (g.codes_t != nullptr) {
    const long n = (g.rows / kBlk + static_cast<long>(g.groups)) * blocks;
    hipLaunchKernelGGL((pack_both_kernel<T, ACT, BACK>), dim3(static_cast<unsigned>(n)), dim3(256),
                       0, s, g);
    return hipGetLastError();
  }
  const int rows_wg = (g.rows + kRowsWg - 1) / kRowsWg;
  const int per = 1;
  hipLaunchKernelGGL((pack_rows_kernel<T, ACT, BACK>),
                     dim3(static_cast<unsigned>(rows_wg), (blocks + per - 1) / per), dim3(256), 0,
                     s, g, per);
  return hipGetLastError();
}
template <typename T>
hipError_t pack_act(const PackArgs& g, hipStream_t s) {
  const bool b = g.dy != nullptr;
  switch (g.act) {
    case kActNone: return pack_t<T, kActNone, false>(g, s);
    case kActRelu: return b ? pack_t<T, kActRelu, true>(g, s) : pack_t<T, kActRelu, false>(g, s);
    case kActGelu: return b ? pack_t<T, kActGelu, true>(g, s) : pack_t<T, kActGelu, false>(g, s);
    case kActSilu: return b ? pack_t<T, kActSilu, true>(g, s) : pack_t<T, kActSilu, false>(g, s);
    default: return b ? pack_t<T, kActSwiglu, true>(g, s) : pack_t<T, kActSwiglu, false>(g, s);
  }
}

}  // namespace

hipError_t launch_block_pack(int dtype, const PackArgs& g, hipStream_t s) {
  return dtype == 1 ? pack_act<bf16_t>(g, s) : pack_act<float>(g, s);
}

hipError_t launch_block_pack_weights(int dtype, const PackWeightArgs& g, hipStream_t s) {
  const long n = static_cast<long>(g.groups) * ((g.out + kBlk - 1) / kBlk) *
                 ((g.in + kBlk - 1) / kBlk);
  if (dtype == 1)
    hipLaunchKernelGGL(pack_weights_kernel<bf16_t>, dim3(static_cast<unsigned>(n)), dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL(pack_weights_kernel<float>, dim3(static_cast<unsigned>(n)), dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace moe
