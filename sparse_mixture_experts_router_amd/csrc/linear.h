// Internal declarations of the grouped linear maps (products grouped by
// expert, with their epilogue and gradients), the 8-bit checkpoints, the
// row grouping and the combine.
//
// Row r of y belongs to group e when offsets[e] <= r < offsets[e + 1]; rows
// at or past offsets[groups] belong to none and are neither read nor written.
// The kernels take offsets as they find them on the device, but clamp each
// group's range into [0, rows], so that no offset can send an access out of
// bounds.
#pragma once

#include "mfma.h"
#include "vec.h"

namespace moe {

// moe_activation (include/moe.h)
enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };

constexpr int kCkptBlock = 64;       // columns of a row that share one scale
constexpr float kCkptMax = 448.0f;   // largest finite E4M3 value
constexpr float kCkptTiny = 1e-30f;  // smallest block maximum a scale is made from

struct LinearArgs {
  const void* x;             // forward: [x_rows or rows, in]; see launchers
  const int32_t* row_index;  // source row of x for every row, or null
  const int32_t* offsets;    // [groups + 1]
  const void* w;             // [groups, z_dim, in]
  const float* w_scale;      // [groups, z_dim] (FP8 weights) or null
  const float* bias;         // [groups, z_dim] or null
  const void* residual;      // [rows, out] or null
  void* y;                   // [rows, out]
  uint8_t* z_codes;          // [rows, z_dim] or null
  float* z_scale;            // [rows, z_dim / 64] or null
  int rows, groups;
  int in_dim;                // columns of x
  int out_dim;               // columns of y
  int z_dim;                 // rows of a group's W: out_dim, or 2 out_dim (SwiGLU)
  int x_rows;                // rows of x
  int act;
};

// ---------------------------------------------------------------- launchers
// Forward: y = act(x W^T + b) + residual; wfp8: E4M3 weights; cus: compute
// units of the device.
// linear_tile_parts: shares of K that the launch is split into; more than one
// takes partial [parts, rows, z_dim].
int linear_tile_parts(int elem_bytes, const LinearArgs& g, int cus);
hipError_t launch_linear_tile(int dtype, bool wfp8, const LinearArgs& g, int cus, float* partial,
                              hipStream_t s);
// dX[r] = dz[r] W_e.  dz [rows, z_dim], dx [rows, in].
hipError_t launch_linear_dx_tile(int dtype, const LinearArgs& g, const void* dz, void* dx, int cus,
                                 hipStream_t s);
// dW_e = sum_r dz[r]^T x[src(r)]; groups without rows get zeros.
hipError_t launch_linear_dw_tile(int dtype, const LinearArgs& g, const void* dz, void* dw, int cus,
                                 hipStream_t s);

// The epilogue of a forward split over K: y from partial [parts, rows, z_dim].
hipError_t launch_join_rows(int dtype, const LinearArgs& g, const float* partial, int parts,
                            hipStream_t s);

// Forward for few rows a group: 32-row tiles, W streamed through registers.
// linear_rows_parts: shares of K that the launch is split into; more than one
// takes partial [parts, rows, z_dim].
bool linear_rows_fits(const LinearArgs& g);
int linear_rows_parts(int elem_bytes, const LinearArgs& g, int cus);
hipError_t launch_linear_rows(int dtype, bool wfp8, const LinearArgs& g, int cus, float* partial,
                              hipStream_t s);
// The same three on 256 x 256 tiles (bf16; forward: weights in bf16 or FP8):
// dW takes x's rows in order, without row_index.
// (gather: x is read through row_index.)
bool linear_mfma_fits(bool wfp8, bool gather, const LinearArgs& g);
hipError_t launch_linear_mfma(bool wfp8, const LinearArgs& g, hipStream_t s);
hipError_t launch_linear_mfma_dx(const LinearArgs& g, const void* dz, void* dx, hipStream_t s);
hipError_t launch_linear_mfma_dw(const LinearArgs& g, const void* dz, void* dw, hipStream_t s);
// xg[r] = x[row_index[r]] for the rows that belong to a group (bf16).
hipError_t launch_gather_rows(const LinearArgs& g, void* xg, hipStream_t s);

// Row tiles of kActRows rows that the activation's backward works in; the
// most there can be for `rows` rows in `groups` groups.
constexpr int kActRows = 16;
inline long act_tiles(long rows, long groups) {
  return rows / kActRows + (groups < rows ? groups : rows);
}
// dz = dy act'(z) from the checkpoint of z (dz null: dy itself is dz), and,
// when partial is not null, the sum of every tile's unrounded dz rows:
// partial [act_tiles, z_dim].
hipError_t launch_act_backward(int dtype, const LinearArgs& g, const void* dy, void* dz,
                               float* partial, hipStream_t s);
// dbias[e] = the sum of group e's tiles of partial, in a fixed order.
hipError_t launch_bias_grad(const LinearArgs& g, const float* partial, float* dbias,
                            hipStream_t s);

hipError_t launch_checkpoint_pack(int dtype, const void* x, long rows, int cols, uint8_t* codes,
                                  float* scale, hipStream_t s);
hipError_t launch_checkpoint_unpack(int dtype, const uint8_t* codes, const float* scale,
                                    long rows, int cols, void* x, hipStream_t s);

// Workgroups (and rows of the count table) that the grouping of n (token,
// slot) pairs runs on.
int group_blocks(long n);
hipError_t launch_group_rows(const int32_t* topk_idx, int T, int N, int k, int capacity,
                             int32_t* table, int32_t* offsets, int32_t* row_token,
                             int32_t* slot_row, hipStream_t s);
hipError_t launch_combine_rows(int dtype, const void* rows, const int32_t* slot_row,
                               const float* gate, int n_rows, int T, int k, int d, void* y,
                               hipStream_t s);
hipError_t launch_combine_rows_backward(int dtype, const void* rows, const int32_t* slot_row,
                                        const float* gate, const void* dy, int n_rows, int T,
                                        int k, int d, void* drows, float* dgate, hipStream_t s);

// ---------------------------------------------------------------- device helpers
// Rows [begin, end) of group e, whatever the offsets hold.
__device__ __forceinline__ int2 group_range(const int32_t* offsets, int e, int rows) {
  const int b = min(max(offsets[e], 0), rows);
  return make_int2(b, min(max(offsets[e + 1], b), rows));
}

// Row tiles of BM rows, group after group, found by every wavefront on its
// own: lane l adds up the tiles of groups l per .. (l + 1) per - 1, one
// wavefront scan gives the first tile of each lane's groups.
struct TileScan {
  int per;    // groups per lane
  int first;  // tiles before this lane's groups
  int mine;   // tiles of this lane's groups
  int total;  // tiles in all
};
__device__ __forceinline__ TileScan scan_tiles(const int32_t* offsets, int groups, int rows,
                                               int bm) {
  TileScan t;
  const int lane = threadIdx.x & 63;
  t.per = (groups + 63) >> 6;
  t.mine = 0;
  for (int i = 0; i < t.per; ++i) {
    const int e = lane * t.per + i;
    if (e < groups) {
      const int2 r = group_range(offsets, e, rows);
      t.mine += (r.y - r.x + bm - 1) / bm;
    }
  }
  int incl = t.mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(incl, off, 64);
    if (lane >= off) incl += o;
  }
  t.first = incl - t.mine;
  t.total = __shfl(incl, 63, 64);
  return t;
}
// Group e and the index of tile `tile` (0 <= tile < t.total) inside it;
// `tiles`: the group's tiles, `before`: tiles of the groups before it.
struct TileAt {
  int e, m, tiles, before, begin, end;
};
__device__ __forceinline__ TileAt find_tile(const TileScan& t, const int32_t* offsets, int groups,
                                            int rows, int bm, int tile) {
  const unsigned long long hit = __ballot(t.first <= tile && tile < t.first + t.mine);
  const int l = hit != 0 ? __ffsll(hit) - 1 : 0;
  int before = __shfl(t.first, l, 64);
  TileAt a{};
  for (int i = 0; i < t.per; ++i) {
    const int e = l * t.per + i;
    if (e >= groups) break;
    const int2 r = group_range(offsets, e, rows);
    const int n = (r.y - r.x + bm - 1) / bm;
    a = TileAt{e, tile - before, n, before, r.x, r.y};
    if (tile < before + n) break;
    before += n;
  }
  return a;
}

// Work item (group, row tile, column tile) of workgroup blockIdx.x on a grid
// of 8 equal shares: workgroups take the 8 XCDs in turn, and each XCD walks a
// contiguous share of the list, so the tiles it runs at once share rows of x
// and of W in its L2.  Inside a group the tiles go in bands of 8 row tiles,
// column by column.  False: nothing to do.
__device__ __forceinline__ bool find_item(const int32_t* offsets, int groups, int rows, int bm,
                                          int nt, TileAt& at, int& col) {
  const TileScan t = scan_tiles(offsets, groups, rows, bm);
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const long items = static_cast<long>(t.total) * nt;
  const long lo = items * xcd / 8, hi = items * (xcd + 1) / 8;
  if (lo + idx >= hi) return false;
  const long w = lo + idx;
  at = find_tile(t, offsets, groups, rows, bm, static_cast<int>(w / nt));
  const int q = static_cast<int>(w - static_cast<long>(at.before) * nt);
  const int band = q / (8 * nt), tw = min(8, at.tiles - band * 8), r = q - band * 8 * nt;
  col = r / tw;
  at.m = band * 8 + r % tw;
  return true;
}
inline long item_grid(long rows, long groups, int bm, long nt) {
  const long tiles = rows / bm + (groups < rows ? groups : rows);
  return 8 * ((tiles * nt + 7) / 8 + 1);
}

template <typename T> __device__ __forceinline__ void load8(const T* p, float* v);
template <> __device__ __forceinline__ void load8<bf16_t>(const bf16_t* p, float* v) {
  Vec<bf16_t>::load(p, v);
}
template <> __device__ __forceinline__ void load8<float>(const float* p, float* v) {
  Vec<float>::load(p, v);
  Vec<float>::load(p + 4, v + 4);
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float* v);
template <> __device__ __forceinline__ void store8<bf16_t>(bf16_t* p, const float* v) {
  Vec<bf16_t>::store(p, v);
}
template <> __device__ __forceinline__ void store8<float>(float* p, const float* v) {
  Vec<float>::store(p, v);
  Vec<float>::store(p + 4, v + 4);
}

// 1 / (1 + e^-z).  fp32 layers take the exact exponential and division,
// bf16 layers the hardware's (relative error below 2^-18 for |z| < 40, far
// inside a bf16 rounding).  At z = -inf both give 0.
template <typename T> __device__ __forceinline__ float sigmoid(float z);
template <> __device__ __forceinline__ float sigmoid<float>(float z) {
  return 1.0f / (1.0f + expf(-z));
}
template <> __device__ __forceinline__ float sigmoid<bf16_t>(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}
// The normal distribution's CDF at z, and e = exp(-z^2 / 2).
//
// fp32 layers: erfc(-z / sqrt 2) / 2, which keeps its relative accuracy in the
// lower tail, where (1 + erf(z / sqrt 2)) / 2 cancels (4 % off at z = -5, 0
// below -5.6).  2000 rows of 256 -> 8192 98.6 us, 94.0 with erff.
//
// bf16 layers: Abramowitz and Stegun's 7.1.26,
//   erfc(x) = (a1 t + ... + a5 t^5) e^-x^2,  t = 1 / (1 + p x),  x >= 0,
// which shares its exponential with the density.  Evaluated in fp32 for the
// tail it is within 3e-7 of the CDF, and z times it within 2^-9 of GELU for
// z > -5, where GELU is -1.4e-6, and 2^-8 (half a bf16 step) for z > -6; below
// it is off by 1 % at -8, 2 % at -10, of values under 6e-9.  4096 tokens' gate
// and up rows (8192 x 28672 values) cost a forward 210 us with erff, 105 this way.
template <typename T> __device__ __forceinline__ float normal_cdf(float z, float& e);
template <> __device__ __forceinline__ float normal_cdf<float>(float z, float& e) {
  e = expf(-0.5f * z * z);
  return 0.5f * erfcf(z * -0.70710678118654752f);
}
template <> __device__ __forceinline__ float normal_cdf<bf16_t>(float z, float& e) {
  e = __expf(-0.5f * z * z);
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * 0.70710678f * fabsf(z));
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  const float tail = 0.5f * t * p * e;
  return z < 0.f ? tail : 1.0f - tail;
}

template <typename T> __device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;  // keeps NaN
    case kActGelu: {
      float e;
      return z * normal_cdf<T>(z, e);
    }
    case kActSilu: return z * sigmoid<T>(z);
    default: return z;
  }
}
// d act / dz.  ReLU: 0 at z = 0.
template <typename T> __device__ __forceinline__ float activate_slope(int act, float z) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
    case kActGelu: {
      float e;
      const float c = normal_cdf<T>(z, e);
      return fmaf(z * 0.39894228040143268f, e, c);
    }
    case kActSilu: {
      const float p = sigmoid<T>(z);
      return p + z * p * (1.f - p);
    }
    default: return 1.f;
  }
}

template <typename T>
__device__ __forceinline__ void activate_slope8(int act, const float* z, float* o) {
  // one uniform branch for the 8 values
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = activate_slope<T>(kActRelu, z[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = activate_slope<T>(kActGelu, z[i]);
      break;
    default:
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = activate_slope<T>(kActSilu, z[i]);
  }
}

// 8 values as E4M3 codes of v * inv, round to nearest even.  |v| is at most
// the block's maximum, so |v inv| is 448 and a rounding at most, which goes to
// 448; NaN becomes the NaN code.
__device__ __forceinline__ uint2 encode8(const float* v, float inv) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = v[i] * inv;
  uint2 r;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
  r.x = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], lo, true));
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[4], s[5], 0, false);
  r.y = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(s[6], s[7], hi, true));
  return r;
}
__device__ __forceinline__ void decode8(uint2 c, float scale, float* v) {
  typedef __attribute__((ext_vector_type(2))) float f32x2;
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.x), false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.x), true);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.y), false);
  const f32x2 e = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.y), true);
  v[0] = a[0] * scale; v[1] = a[1] * scale; v[2] = b[0] * scale; v[3] = b[1] * scale;
  v[4] = d[0] * scale; v[5] = d[1] * scale; v[6] = e[0] * scale; v[7] = e[1] * scale;
}
// One 64-column block of a row, 8 columns in each of 8 neighbouring lanes
// (lane mod 8 in column order): its codes, and its scale from the first of
// them.  `ok` is the same for the 8 lanes.
__device__ __forceinline__ void pack_block(const float* v, bool ok, uint8_t* codes, float* scale) {
  auto block_max = [](const float* x) {  // NaN does not count
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    m = fmaxf(m, __shfl_xor(m, 1, 64));
    m = fmaxf(m, __shfl_xor(m, 2, 64));
    return fmaxf(m, __shfl_xor(m, 4, 64));
  };
  float m = block_max(v);
  uint2 c;
  if (__builtin_expect(__any(m == INFINITY), 0)) {
    // infinities neither count, and E4M3 has none: as NaN
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fabsf(v[i]) < INFINITY ? v[i] : __builtin_nanf("");
    m = fmaxf(block_max(f), kCkptTiny);
    c = encode8(f, kCkptMax / m);
  } else {
    m = fmaxf(m, kCkptTiny);
    c = encode8(v, kCkptMax / m);
  }
  if (!ok) return;
  *reinterpret_cast<uint2*>(codes) = c;
  if ((threadIdx.x & 7) == 0) *scale = m / kCkptMax;
}

// 8 floats at p (fill where p is null or the columns lie past the end): the
// bias or the FP8 scales of a lane's columns.
__device__ __forceinline__ void load_cols8(const float* p, size_t at, bool ok, float fill,
                                           float* v) {
  if (p != nullptr && ok) {
    load8<float>(p + at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fill;
  }
}
// 8 values as they lie in memory, widened when they are used, so that a caller
// can have many in flight.  Read once: bf16 past the caches.
template <typename T> struct Raw8;
template <> struct Raw8<bf16_t> {
  u32x4 r;
  __device__ __forceinline__ void load(const bf16_t* p) {
    r = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  }
  __device__ __forceinline__ void zero() { r = u32x4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
  }
};
template <> struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};
template <typename T>
__device__ __forceinline__ void load_residual(const LinearArgs& g, long row, int n, bool ok,
                                              Raw8<T>& r) {
  if (g.residual != nullptr && ok)
    r.load(static_cast<const T*>(g.residual) + static_cast<size_t>(row) * g.out_dim + n);
  else
    r.zero();
}
// y is not read again by the launch that writes it: bf16 goes past the caches,
// where the rows of x and W that other tiles use stay longer.
template <typename T> __device__ __forceinline__ void store_once8(T* p, const float* v);
template <> __device__ __forceinline__ void store_once8<bf16_t>(bf16_t* p, const float* v) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(f32_to_bf16(v[2 * i])) |
           (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
}
template <> __device__ __forceinline__ void store_once8<float>(float* p, const float* v) {
  store8<float>(p, v);
}

// The epilogue of the forward on 8 columns of one row: columns n .. n + 7 of
// y, n a multiple of 8, 8 neighbouring lanes holding a whole 64-column block.
// v: z's columns (SwiGLU: v the gate's, u the up projection's), bias included.
template <typename T, bool GATED>
__device__ __forceinline__ void linear_epilogue8(const LinearArgs& g, long row, int n, bool ok,
                                                 const float* v, const float* u,
                                                 const Raw8<T>& res) {
  if (g.z_codes != nullptr) {
    const size_t zo = static_cast<size_t>(row) * g.z_dim;
    uint8_t* c = g.z_codes + zo;
    float* sc = g.z_scale + zo / kCkptBlock;
    pack_block(v, ok, c + n, sc + n / kCkptBlock);
    if (GATED) pack_block(u, ok, c + g.out_dim + n, sc + (g.out_dim + n) / kCkptBlock);
  }
  if (!ok) return;
  float h[8];
  if (GATED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = v[i] * sigmoid<T>(v[i]) * u[i];
  } else {
    // one uniform branch for the 8 values
    switch (g.act) {
      case kActRelu:
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = activate<T>(kActRelu, v[i]);
        break;
      case kActGelu:
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = activate<T>(kActGelu, v[i]);
        break;
      case kActSilu:
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = activate<T>(kActSilu, v[i]);
        break;
      default:
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] += res.get(i);
  store_once8<T>(static_cast<T*>(g.y) + static_cast<size_t>(row) * g.out_dim + n, h);
}

}  // namespace moe
