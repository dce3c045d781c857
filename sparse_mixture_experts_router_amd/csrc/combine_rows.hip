// Combine of the experts' rows into tokens, and its gradient.
//
//   y[t]    = sum_s gate[t, s] rows[slot_row[t, s]]       (gate null: 1)
//   drows[slot_row[t, s]] = gate[t, s] dy[t]
//   dgate[t, s] = <dy[t], rows[slot_row[t, s]]>
//
// over the slots that have a row (slot_row inside [0, n_rows); a dropped slot
// adds nothing and its dgate is 0).  Sums in fp32, slot after slot, rounded
// once.  One workgroup per token and 16 bytes of a row per lane: every row is
// read (and written) once, so HBM bounds both.  With gate null the combine is
// also the gradient of reading x rows through row_token.
#include "linear.h"

namespace moe {
namespace {

// Threads of a token's workgroup: each takes 8 columns at a time, in as few
// passes as 512 threads need, with no wavefront idle in the last one.
inline int token_threads(int d) {
  const int chunks = d / 8, passes = (chunks + 511) / 512;
  return ((chunks + passes - 1) / passes + 63) / 64 * 64;
}

// KS: slots whose rows are asked for together.  Rows are read once and results
// written once, in bf16 past the caches (fp32 by plain accesses): 8192 tokens x
// 8 rows of 7168 219 us with plain loads and stores, 4 slots; 204 with 8 slots
// and non-temporal loads, 188 with non-temporal stores too (5.6 TB/s).  Columns
// are unsigned: the step past the last may pass 2^31.
template <typename T, int KS>
__global__ __launch_bounds__(512) void combine_rows_kernel(const T* __restrict__ rows,
                                                           const int32_t* __restrict__ slot_row,
                                                           const float* __restrict__ gate,
                                                           int n_rows, int k, unsigned d,
                                                           T* __restrict__ y) {
  const size_t t = blockIdx.x;
  const int32_t* sr = slot_row + t * k;
  const float* gt = gate != nullptr ? gate + t * k : nullptr;
  for (unsigned c = threadIdx.x * 8; c < d; c += blockDim.x * 8) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int s0 = 0; s0 < k; s0 += KS) {
      Raw8<T> v[KS];
      float w[KS];
      bool on[KS];
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        const int r = s0 + q < k ? sr[s0 + q] : -1;
        on[q] = r >= 0 && r < n_rows;  // uniform over the workgroup
        w[q] = 1.f;
        if (!on[q]) continue;
        if (gt != nullptr) w[q] = gt[s0 + q];
        v[q].load(rows + static_cast<size_t>(r) * d + c);
      }
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        if (!on[q]) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[q], v[q].get(i), acc[i]);
      }
    }
    store_once8<T>(y + t * d + c, acc);
  }
}

template <typename T, int KS>
__global__ __launch_bounds__(512) void combine_rows_backward_kernel(
    const T* __restrict__ rows, const int32_t* __restrict__ slot_row,
    const float* __restrict__ gate, const T* __restrict__ dy, int n_rows, int k, unsigned d,
    T* __restrict__ drows, float* __restrict__ dgate) {
  __shared__ float s_dot[KS][8];
  const size_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int32_t* sr = slot_row + t * k;
  for (int s0 = 0; s0 < k; s0 += KS) {
    int row[KS];
    float w[KS], dot[KS];
#pragma unroll
    for (int q = 0; q < KS; ++q) {
      const int r = s0 + q < k ? sr[s0 + q] : -1;
      row[q] = r < n_rows ? r : -1;
      w[q] = gate != nullptr && row[q] >= 0 ? gate[t * k + s0 + q] : 1.f;
      dot[q] = 0.f;
    }
    for (unsigned c = threadIdx.x * 8; c < d; c += blockDim.x * 8) {
      float g[8];
      Raw8<T> v[KS];
      if (dgate != nullptr) {
#pragma unroll
        for (int q = 0; q < KS; ++q)
          if (row[q] >= 0) v[q].load(rows + static_cast<size_t>(row[q]) * d + c);
      }
      load8<T>(dy + t * d + c, g);
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        if (row[q] < 0) continue;  // uniform over the workgroup
        if (dgate != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[q] = fmaf(g[i], v[q].get(i), dot[q]);
        }
        if (drows != nullptr) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = w[q] * g[i];
          store_once8<T>(drows + static_cast<size_t>(row[q]) * d + c, o);
        }
      }
    }
    if (dgate == nullptr) continue;
#pragma unroll
    for (int q = 0; q < KS; ++q) {
      float v = dot[q];
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
      if (lane == 0) s_dot[q][wave] = v;
    }
    __syncthreads();
    if (threadIdx.x < KS && s0 + static_cast<int>(threadIdx.x) < k) {
      float v = 0.f;
      for (int i = 0; i < waves; ++i) v += s_dot[threadIdx.x][i];
      dgate[t * k + s0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

// A wavefront copies kGatherRows rows, one chunk of each in flight together.
constexpr int kGatherRows = 4;
__global__ __launch_bounds__(256) void gather_rows_kernel(LinearArgs g, bf16_t* __restrict__ xg) {
  const int r0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * kGatherRows, lane = threadIdx.x & 63;
  const int n = min(max(g.offsets[g.groups], 0), g.rows) - r0;  // rows of x left
  if (n <= 0) return;
  const bf16_t* x[kGatherRows];
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    const size_t src = min(max(g.row_index[r0 + min(i, n - 1)], 0), g.x_rows - 1);
    x[i] = static_cast<const bf16_t*>(g.x) + src * g.in_dim;
  }
  bf16_t* const o = xg + static_cast<size_t>(r0) * g.in_dim;
  for (int c = lane * 8; c < g.in_dim; c += 512) {
    u32x4 v[kGatherRows];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) v[i] = *reinterpret_cast<const u32x4*>(x[i] + c);
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i)
      if (i < n) *reinterpret_cast<u32x4*>(o + static_cast<size_t>(i) * g.in_dim + c) = v[i];
  }
}

}  // namespace

hipError_t launch_gather_rows(const LinearArgs& g, void* xg, hipStream_t s) {
  hipLaunchKernelGGL(gather_rows_kernel, dim3((g.rows + 4 * kGatherRows - 1) / (4 * kGatherRows)),
                     dim3(256), 0, s, g,
                     static_cast<bf16_t*>(xg));
  return hipGetLastError();
}

template <typename T>
static hipError_t combine_t(const void* rows, const int32_t* slot_row, const float* gate,
                            int n_rows, int T_, int k, int d, void* y, hipStream_t s) {
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(T_), dim3(token_threads(d)), 0, s,
                       static_cast<const T*>(rows), slot_row, gate, n_rows, k, d,
                       static_cast<T*>(y));
    return hipGetLastError();
  };
  if (k <= 2) return run(combine_rows_kernel<T, 2>);
  if (k <= 4) return run(combine_rows_kernel<T, 4>);
  return run(combine_rows_kernel<T, 8>);
}

hipError_t launch_combine_rows(int dtype, const void* rows, const int32_t* slot_row,
                               const float* gate, int n_rows, int T_, int k, int d, void* y,
                               hipStream_t s) {
  return dtype == 1 ? combine_t<bf16_t>(rows, slot_row, gate, n_rows, T_, k, d, y, s)
                    : combine_t<float>(rows, slot_row, gate, n_rows, T_, k, d, y, s);
}

template <typename T>
static hipError_t combine_backward_t(const void* rows, const int32_t* slot_row, const float* gate,
                                     const void* dy, int n_rows, int T_, int k, int d, void* drows,
                                     float* dgate, hipStream_t s) {
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(T_), dim3(token_threads(d)), 0, s,
                       static_cast<const T*>(rows), slot_row, gate, static_cast<const T*>(dy),
                       n_rows, k, d, static_cast<T*>(drows), dgate);
    return hipGetLastError();
  };
  if (k <= 2) return run(combine_rows_backward_kernel<T, 2>);
  if (k <= 4) return run(combine_rows_backward_kernel<T, 4>);
  return run(combine_rows_backward_kernel<T, 8>);
}

hipError_t launch_combine_rows_backward(int dtype, const void* rows, const int32_t* slot_row,
                                        const float* gate, const void* dy, int n_rows, int T_,
                                        int k, int d, void* drows, float* dgate, hipStream_t s) {
  return dtype == 1 ? combine_backward_t<bf16_t>(rows, slot_row, gate, dy, n_rows, T_, k, d, drows,
                                                 dgate, s)
                    : combine_backward_t<float>(rows, slot_row, gate, dy, n_rows, T_, k, d, drows,
                                                dgate, s);
}

}  // namespace moe
