// Grouping of (token, slot) pairs by expert, from the router's indices alone.
//
// With the pairs in flat order i = t k + s and e_i their experts:
//   count[e]    = pairs of expert e (at most `capacity` when that is set)
//   offsets[e]  = exclusive prefix sum of count
//   rank(i)     = pairs of e_i before i
//   slot_row[i] = offsets[e_i] + rank(i), or -1 when rank(i) >= capacity or
//                 e_i is no expert (a padded token's -1)
//   row_token[slot_row[i]] = t
// a stable counting sort, so each expert's rows are in token order and the
// result does not depend on how the work is split.
//
// Each of `blocks` workgroups takes one contiguous range of pairs.  The first
// launch writes every range's counts to a table [blocks, N]; in the second
// every workgroup adds up the table's columns for itself (at most 256 x 512
// ints from L2, cheaper than a launch between the two) and ranks its pairs
// again.  One workgroup does it all in one launch when there is one range.
// A wavefront ranks 64 pairs at once: lanes with the same expert find each
// other by a ballot for each bit of the index.
//
// Bound by the chain of loads and barriers, not by bytes: the first indices
// are asked for before the table, and a pair's counts of the 16 wavefronts are
// read together.  2048 pairs in one launch take 7.0 us, 16384 x 8 pairs of 128
// experts 2.8 and 6.8.
#include "linear.h"

namespace moe {
namespace {

constexpr int kGThreads = 1024, kGWaves = kGThreads / 64;
constexpr int kMaxBlocks = 256;

// Lanes of the wavefront that hold the same key (0 <= key < 1024).
__device__ __forceinline__ unsigned long long same_key(int key, int bits) {
  unsigned long long m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const unsigned long long ones = __ballot((key >> b) & 1);
    m &= ((key >> b) & 1) ? ones : ~ones;
  }
  return m;
}

// Range of workgroup b: whole chunks of kGThreads pairs, equally many in every range
// but the last.
__device__ __forceinline__ void block_range(long n, int blocks, int b, long& lo, long& hi) {
  const long chunks = (n + kGThreads - 1) / kGThreads;
  const long per = (chunks + blocks - 1) / blocks;
  lo = min(n, b * per * kGThreads);
  hi = min(n, lo + per * kGThreads);
}

// Counts of this workgroup's range into s_cnt [N] (LDS).
__device__ __forceinline__ void count_range(const int32_t* __restrict__ idx, long lo, long hi,
                                            int N, int* s_cnt) {
  for (int e = threadIdx.x; e < N; e += kGThreads) s_cnt[e] = 0;
  __syncthreads();
  for (long i = lo + threadIdx.x; i < hi; i += kGThreads) {
    const int e = idx[i];
    if (e >= 0 && e < N) atomicAdd(&s_cnt[e], 1);  // integers: any order, one sum
  }
  __syncthreads();
}

__global__ __launch_bounds__(kGThreads) void group_count_kernel(const int32_t* __restrict__ idx,
                                                                long n, int N,
                                                                int32_t* __restrict__ table) {
  __shared__ int s_cnt[kMaxExperts];
  long lo, hi;
  block_range(n, gridDim.x, blockIdx.x, lo, hi);
  count_range(idx, lo, hi, N, s_cnt);
  for (int e = threadIdx.x; e < N; e += kGThreads)
    table[static_cast<size_t>(blockIdx.x) * N + e] = s_cnt[e];
}

// TABLE false: one workgroup, no table.
template <bool TABLE>
__global__ __launch_bounds__(kGThreads) void group_rows_kernel(
    const int32_t* __restrict__ idx, long n, int N, int k, int capacity,
    const int32_t* __restrict__ table, int32_t* __restrict__ offsets,
    int32_t* __restrict__ row_token, int32_t* __restrict__ slot_row) {
  __shared__ int s_run[kMaxExperts];   // rank of the next pair of every expert
  __shared__ int s_off[kMaxExperts];   // offsets
  __shared__ int s_wave[kGWaves][kMaxExperts];  // counts of a chunk by wavefront
  __shared__ int s_part[kGWaves];
  __shared__ int s_tot[kGThreads], s_bef[kGThreads];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  long lo, hi;
  block_range(n, gridDim.x, blockIdx.x, lo, hi);

  // The first chunk's indices, asked for before the table.
  auto load_key = [&](long i) {
    const int v = i < hi ? idx[i] : -1;
    return v >= 0 && v < N ? v : N;
  };
  int e = load_key(lo + tid);

  // Totals, and the counts of the ranges before this one (N <= 512 < threads):
  // kGThreads / N threads share an expert's column of the table, 8 loads of
  // each in flight.
  int total = 0, before = 0;
  if (TABLE) {
    const int parts = kGThreads / N, nb = gridDim.x, me = blockIdx.x;
    const int col = tid % N, part = tid / N;
    const int per = (nb + parts - 1) / parts;
    if (part < parts) {
      const int b1 = min(nb, (part + 1) * per);
      for (int b0 = part * per; b0 < b1; b0 += 8) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = b0 + i < b1 ? table[static_cast<size_t>(b0 + i) * N + col] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          total += v[i];
          if (b0 + i < me) before += v[i];
        }
      }
    }
    s_tot[tid] = total;
    s_bef[tid] = before;
    __syncthreads();
    if (tid < N)
      for (int p = 1; p < parts; ++p) {
        total += s_tot[p * N + tid];
        before += s_bef[p * N + tid];
      }
  } else {
    count_range(idx, lo, hi, N, s_run);
    if (tid < N) total = s_run[tid];
    __syncthreads();
  }
  const int kept = capacity > 0 ? min(total, capacity) : total;
  int incl = tid < N ? kept : 0;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(incl, off, 64);
    if (lane >= off) incl += o;
  }
  if (lane == 63) s_part[wave] = incl;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kGWaves; ++w) {  // all read together
    const int v = s_part[w];
    incl += w < wave ? v : 0;
  }
  if (tid < N) {
    s_run[tid] = before;
    s_off[tid] = incl - kept;
    if (blockIdx.x == 0) {
      offsets[tid + 1] = incl;
      if (tid == 0) offsets[0] = 0;
    }
  }
  int bits = 0;
  while ((1 << bits) <= N) ++bits;  // keys 0 .. N, N: no expert

  for (long c0 = lo; c0 < hi; c0 += kGThreads) {
    for (int x = lane; x < N; x += 64) s_wave[wave][x] = 0;  // its own: no barrier
    const long i = c0 + tid;
    if (c0 != lo) e = load_key(i);
    const unsigned long long same = same_key(e, bits);
    const int in_wave = __popcll(same & ((1ull << lane) - 1));
    if (e < N && in_wave == 0) s_wave[wave][e] = __popcll(same);
    __syncthreads();
    if (i < hi) {
      int row = -1;
      if (e < N) {
        int rank = s_run[e] + in_wave;
#pragma unroll
        for (int w = 0; w < kGWaves; ++w) {
          const int v = s_wave[w][e];
          rank += w < wave ? v : 0;
        }
        // (the second bound only matters if idx changed since it was counted)
        if ((capacity <= 0 || rank < capacity) && s_off[e] + rank < n) {
          row = s_off[e] + rank;
          row_token[row] = static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(k));
        }
      }
      slot_row[i] = row;
    }
    if (c0 + kGThreads >= hi) break;
    __syncthreads();
    for (int x = tid; x < N; x += kGThreads) {
      int a = 0;
#pragma unroll
      for (int w = 0; w < kGWaves; ++w) a += s_wave[w][x];
      s_run[x] += a;
    }
    __syncthreads();
  }
}

}  // namespace

// One range up to 2048 pairs, then about 1024 pairs a range, at most 256 ranges.
int group_blocks(long n) {
  if (n <= 2048) return 1;
  const long b = (n + 1023) / 1024;
  return static_cast<int>(b < kMaxBlocks ? b : kMaxBlocks);
}

hipError_t launch_group_rows(const int32_t* topk_idx, int T, int N, int k, int capacity,
                             int32_t* table, int32_t* offsets, int32_t* row_token,
                             int32_t* slot_row, hipStream_t s) {
  const long n = static_cast<long>(T) * k;
  const int blocks = group_blocks(n);
  if (blocks == 1) {
    hipLaunchKernelGGL(group_rows_kernel<false>, dim3(1), dim3(kGThreads), 0, s, topk_idx, n, N, k,
                       capacity, nullptr, offsets, row_token, slot_row);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(group_count_kernel, dim3(blocks), dim3(kGThreads), 0, s, topk_idx, n, N,
                     table);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(group_rows_kernel<true>, dim3(blocks), dim3(kGThreads), 0, s, topk_idx, n, N,
                     k, capacity, table, offsets, row_token, slot_row);
  return hipGetLastError();
}

}  // namespace moe
