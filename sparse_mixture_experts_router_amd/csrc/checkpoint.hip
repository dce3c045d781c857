// Activation checkpoints in 8 bits, and the backward of an activation from
// one.
//
// A checkpoint of a [rows, cols] array holds an E4M3 code for each element
// and one fp32 scale for each block of 64 columns of a row: with m the
// block's largest magnitude (at least 1e-30),
//   scale = m / 448,  code = E4M3(v (448 / m)),  v' = code scale,
// so |v' - v| <= max(2^-4 |v|, 2^-10 scale).  It takes 1.0625 bytes an element against 2 of bf16.
//
// Every kernel here moves each byte once and computes a few operations per
// element: all are bound by HBM.
#include "linear.h"

namespace moe {
namespace {

// 8-column chunks of one thread, loaded before the first is used.  Packing 2 /
// 4 / 8: 4096 x 4096 bf16 12.0 / 11.0 / 12.6 us; unpacking 8192 x 28672 112.6 /
// 115.2 / 115.4.
constexpr int kPackUnroll = 4, kUnpackUnroll = 2;

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(const T* __restrict__ x, long chunks,
                                                   uint8_t* __restrict__ codes,
                                                   float* __restrict__ scale) {
  const long c0 = static_cast<long>(blockIdx.x) * (256 * kPackUnroll) + threadIdx.x;
  float v[kPackUnroll][8];
#pragma unroll
  for (int i = 0; i < kPackUnroll; ++i) {
    const long c = c0 + 256 * i;
    load8<T>(x + (c < chunks ? c : 0) * 8, v[i]);
  }
#pragma unroll
  for (int i = 0; i < kPackUnroll; ++i) {
    const long c = c0 + 256 * i;  // chunks is a multiple of 8: a block is whole or absent
    pack_block(v[i], c < chunks, codes + c * 8, scale + c / 8);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void unpack_kernel(const uint8_t* __restrict__ codes,
                                                     const float* __restrict__ scale, long chunks,
                                                     T* __restrict__ x) {
  const long c0 = static_cast<long>(blockIdx.x) * (256 * kUnpackUnroll) + threadIdx.x;
  uint2 q[kUnpackUnroll];
  float s[kUnpackUnroll];
#pragma unroll
  for (int i = 0; i < kUnpackUnroll; ++i) {
    const long c = c0 + 256 * i < chunks ? c0 + 256 * i : 0;
    q[i] = *reinterpret_cast<const uint2*>(codes + c * 8);
    s[i] = scale[c / 8];
  }
#pragma unroll
  for (int i = 0; i < kUnpackUnroll; ++i) {
    const long c = c0 + 256 * i;
    float v[8];
    decode8(q[i], s[i], v);
    if (c < chunks) store_once8<T>(x + c * 8, v);
  }
}

// dz = dy act'(z) for one row tile of kActRows rows of a group and up to 512
// columns of y; z is decoded from its checkpoint.  `lpr` lanes (a power of
// two) hold one row's columns, 8 each, so the workgroup takes 256 / lpr rows
// at a time, kActUnroll of them with their loads in flight together.  A lane
// keeps its columns through the tile and adds up its unrounded dz; the
// workgroup's sums, in a fixed order, are the tile's row of partial.
constexpr int kActUnroll = 4;
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void act_backward_kernel(LinearArgs g, const T* __restrict__ dy,
                                                           T* __restrict__ dz,
                                                           float* __restrict__ partial, int lpr) {
  constexpr int NS = GATED ? 16 : 8;
  __shared__ float s_sum[256][NS + 1];
  const TileScan t = scan_tiles(g.offsets, g.groups, g.rows, kActRows);
  const int tile = blockIdx.x;
  if (tile >= t.total) return;
  const TileAt at = find_tile(t, g.offsets, g.groups, g.rows, kActRows, tile);
  const int row0 = at.begin + at.m * kActRows, row1 = min(row0 + kActRows, at.end);
  const int tid = threadIdx.x, rpp = 256 / lpr;  // rows of a pass
  const int c = (blockIdx.y * lpr + tid % lpr) * 8;
  const bool in = c < g.out_dim;
  float sum[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) sum[i] = 0.f;
  if (in) {
    for (int r0 = row0 + tid / lpr; r0 < row1; r0 += kActUnroll * rpp) {
      Raw8<T> d[kActUnroll];
      uint2 qz[kActUnroll], qu[kActUnroll];
      float sz[kActUnroll], su[kActUnroll];
#pragma unroll
      for (int k = 0; k < kActUnroll; ++k) {
        const int r = min(r0 + k * rpp, row1 - 1);
        const size_t zo = static_cast<size_t>(r) * g.z_dim + c;
        d[k].load(dy + static_cast<size_t>(r) * g.out_dim + c);
        if (g.act != kActNone) {
          qz[k] = *reinterpret_cast<const uint2*>(g.z_codes + zo);
          sz[k] = g.z_scale[zo / kCkptBlock];
          if (GATED) {
            qu[k] = *reinterpret_cast<const uint2*>(g.z_codes + zo + g.out_dim);
            su[k] = g.z_scale[(zo + g.out_dim) / kCkptBlock];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kActUnroll; ++k) {
        const int r = r0 + k * rpp;
        if (r >= row1) break;
        const size_t zo = static_cast<size_t>(r) * g.z_dim + c;
        float o[NS];
        if (g.act == kActNone) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = d[k].get(i);
        } else {
          float z[8];
          decode8(qz[k], sz[k], z);
          if constexpr (GATED) {
            float u[8];
            decode8(qu[k], su[k], u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float p = sigmoid<T>(z[i]), dh = d[k].get(i);
              o[i] = dh * u[i] * (p + z[i] * p * (1.f - p));
              o[8 + i] = dh * z[i] * p;
            }
          } else {
            activate_slope8<T>(g.act, z, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= d[k].get(i);
          }
        }
        if (dz != nullptr) {
          store8<T>(dz + zo, o);
          if (GATED) store8<T>(dz + zo + g.out_dim, o + 8);
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) sum[i] += o[i];
      }
    }
  }
  if (partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < NS; ++i) s_sum[tid][i] = sum[i];
  __syncthreads();
  if (tid >= lpr || !in) return;
  for (int q = tid + lpr; q < 256; q += lpr)
#pragma unroll
    for (int i = 0; i < NS; ++i) sum[i] += s_sum[q][i];
  float* p = partial + static_cast<size_t>(tile) * g.z_dim + c;
  store8<float>(p, sum);
  if (GATED) store8<float>(p + g.out_dim, sum + 8);
}

// A running fp32 sum and what its additions rounded off (Knuth's two-sum): a
// group of a million equal rows would otherwise round the same way every time
// (2^20 rows of 0.1 in one chain: off by 6e-4).
struct LongSum {
  float s = 0.f, low = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = s + v, w = t - s;
    low += (s - (t - w)) + (v - w);
    s = t;
  }
  // (past the largest float, or with a NaN, `low` is NaN)
  __device__ __forceinline__ float value() const { return fabsf(s) < INFINITY ? s + low : s; }
};

// dbias of one group and 64 columns: its tiles' partial sums, 8 tiles in turn
// for each wavefront, the wavefronts' sums added in order.  Backward of 16384
// bf16 rows of 64 -> 1024 248 us (306 with one chain a column), of 128 fp32
// rows of 4 groups 128 -> 256 23.7 (23.4).
// cap: rows of partial (offsets that overlap could name more tiles).
constexpr int kBiasWaves = 8;
__global__ __launch_bounds__(64 * kBiasWaves) void bias_grad_kernel(
    LinearArgs g, const float* __restrict__ partial, int cap, float* __restrict__ dbias) {
  __shared__ float s_sum[kBiasWaves][64], s_low[kBiasWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x, n = blockIdx.y * 64 + lane;
  // tiles of the groups before e
  int before = 0;
  for (int i = lane; i < e; i += 64) {
    const int2 r = group_range(g.offsets, i, g.rows);
    before += (r.y - r.x + kActRows - 1) / kActRows;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) before += __shfl_xor(before, off, 64);
  const int2 r = group_range(g.offsets, e, g.rows);
  const int tiles = min((r.y - r.x + kActRows - 1) / kActRows, cap - before);
  const float* p = partial + static_cast<size_t>(before) * g.z_dim + n;
  LongSum acc;
  for (int t0 = wave * 8; t0 < tiles; t0 += 8 * kBiasWaves) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = t0 + i < tiles ? p[static_cast<size_t>(t0 + i) * g.z_dim] : 0.f;
    acc.add(((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7])));
  }
  s_sum[wave][lane] = acc.s;
  s_low[wave][lane] = acc.low;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < kBiasWaves; ++w) {
    acc.add(s_sum[w][lane]);
    acc.low += s_low[w][lane];
  }
  dbias[static_cast<size_t>(e) * g.z_dim + n] = acc.value();
}

constexpr long kMaxBlocks = (1L << 24) - 1;  // below 2^32 threads of 256-thread workgroups

}  // namespace

hipError_t launch_checkpoint_pack(int dtype, const void* x, long rows, int cols, uint8_t* codes,
                                  float* scale, hipStream_t s) {
  const long chunks = rows * (cols / 8);
  const long blocks = (chunks + 256 * kPackUnroll - 1) / (256 * kPackUnroll);
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (dtype == 1)
    hipLaunchKernelGGL(pack_kernel<bf16_t>, grid, dim3(256), 0, s, static_cast<const bf16_t*>(x),
                       chunks, codes, scale);
  else
    hipLaunchKernelGGL(pack_kernel<float>, grid, dim3(256), 0, s, static_cast<const float*>(x),
                       chunks, codes, scale);
  return hipGetLastError();
}

hipError_t launch_checkpoint_unpack(int dtype, const uint8_t* codes, const float* scale,
                                    long rows, int cols, void* x, hipStream_t s) {
  const long chunks = rows * (cols / 8);
  const long blocks = (chunks + 256 * kUnpackUnroll - 1) / (256 * kUnpackUnroll);
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (dtype == 1)
    hipLaunchKernelGGL(unpack_kernel<bf16_t>, grid, dim3(256), 0, s, codes, scale, chunks,
                       static_cast<bf16_t*>(x));
  else
    hipLaunchKernelGGL(unpack_kernel<float>, grid, dim3(256), 0, s, codes, scale, chunks,
                       static_cast<float*>(x));
  return hipGetLastError();
}

template <typename T>
static hipError_t act_backward_t(const LinearArgs& g, const void* dy, void* dz, float* partial,
                                 hipStream_t s) {
  int lpr = 8;  // a row's columns over 8 .. 64 lanes
  while (lpr < 64 && lpr * 8 < g.out_dim) lpr *= 2;
  const long tiles = act_tiles(g.rows, g.groups);
  if (tiles > kMaxBlocks) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles), (g.out_dim + lpr * 8 - 1) / (lpr * 8));
  if (g.act == kActSwiglu)
    hipLaunchKernelGGL((act_backward_kernel<T, true>), grid, dim3(256), 0, s, g,
                       static_cast<const T*>(dy), static_cast<T*>(dz), partial, lpr);
  else
    hipLaunchKernelGGL((act_backward_kernel<T, false>), grid, dim3(256), 0, s, g,
                       static_cast<const T*>(dy), static_cast<T*>(dz), partial, lpr);
  return hipGetLastError();
}

hipError_t launch_act_backward(int dtype, const LinearArgs& g, const void* dy, void* dz,
                               float* partial, hipStream_t s) {
  return dtype == 1 ? act_backward_t<bf16_t>(g, dy, dz, partial, s)
                    : act_backward_t<float>(g, dy, dz, partial, s);
}

hipError_t launch_bias_grad(const LinearArgs& g, const float* partial, float* dbias,
                            hipStream_t s) {
  const dim3 grid(g.groups, g.z_dim / 64);
  hipLaunchKernelGGL(bias_grad_kernel, grid, dim3(64 * kBiasWaves), 0, s, g, partial,
                     static_cast<int>(act_tiles(g.rows, g.groups)), dbias);
  return hipGetLastError();
}

}  // namespace moe
