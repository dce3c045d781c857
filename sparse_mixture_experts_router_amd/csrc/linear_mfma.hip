// Grouped linear maps in bf16 on 256 x 256 tiles: the shapes with many rows a
// group.  Same products as linear_tile.hip,
//
//   forward  z[r] = x[src(r)] W_e^T + b_e,  y[r] = act(z[r]) + residual[r]
//   dX       dX[r] = dz[r] W_e
//   dW       dW_e = sum_r dz[r]^T x[src(r)]
//
// bound by the matrix cores and by L2 -> LDS bytes: a tile does 128 operations
// for each byte that it stages.  One workgroup of 8 wavefronts, two on each SIMD, owns a tile and
// the whole LDS; a wavefront accumulates a quarter of the rows and half of the
// columns in AGPRs.  A stage is 64 elements of K.  The wavefronts of a SIMD
// take turns: while one runs its 64 MFMAs of a stage from registers, the other
// issues its loads (global -> LDS, no registers) and reads its 24 fragments of
// the next stage; a barrier ends every phase.  Wavefronts 0-3 load the A operand one stage ahead (2
// buffers), wavefronts 4-7 the B operand two stages ahead (3 buffers, for W
// comes from HBM while the rows of x are mostly in L2).
//
// Operands staged from their rows (K contiguous): 128 bytes of each of 256
// rows, 16-byte chunks XOR-swizzled by row (swz128).  Operands staged from
// their K-rows (W of dX; dz and x of dW): 512 contiguous bytes of each of 64
// K-rows, and the fragments are turned on the way out of LDS by
// ds_read_b64_tr_b16, so nothing is ever transposed in memory.
//
// FP8 weights (forward): a buffer of the B operand holds 128 codes of each row,
// two stages, and is loaded every other stage.  One 16-byte read gives a lane
// the codes of both K steps of a stage, 16 consecutive elements, so the rows of
// x are read in that order too; a fragment is widened to bf16 right before its
// MFMAs, and the scales multiply the sums in the epilogue.
#include "linear.h"
#include "lds_ring.h"

namespace moe {
namespace {

constexpr int kFwd = 0, kDx = 1, kDw = 2;
constexpr int kT = 256;                 // rows and (effective) columns of a tile
constexpr int kBuf = kT * kLineBytes;   // bytes of a staged operand
constexpr int kABufs = 2, kBBufs = 3;
constexpr int kLds = (kABufs + kBBufs) * kBuf;  // 160 KB
constexpr int kMB = 4, kWN = 128, kNB = kWN / 16;  // a wavefront's 16-row and 16-column blocks
constexpr int kStgPitch = 64 * 4 + 16;  // bytes of a staged result row of 64 columns
static_assert(8 * 2 * 32 * kStgPitch <= kLds, "staging space");

template <int N> struct CInt { static constexpr int value = N; };

// What K-rows past the end of a group read.
__device__ __align__(16) const uint32_t zero_chunk[4] = {0u, 0u, 0u, 0u};

// 16-byte chunk c of staged K-row kk lies at chunk c ^ krow_key(kk): the 16
// K-rows that one transposing read touches (8 g + 4 h + r with g, r < 4) get
// 16 distinct keys, which spreads them over the banks.
__device__ __forceinline__ int krow_key(int kk) { return 2 * ((kk & 3) + 4 * ((kk >> 3) & 3)); }

// The fragments of N 16-column blocks of a K-row operand, for the stage's two
// K steps (32 K-rows = 16384 bytes apart).  A transposing read takes 4 columns
// of each of 4 K-rows for every 16 lanes: lane j points at 4 columns of K-row
// j / 4, lane i receives column i of the four rows; two reads make a fragment.
// One block of asm with its wait: the reads' results are there when it ends.
// (Through the builtin the compiler waits for every global -> LDS load in
// flight before each of them, for they share LDS.)  Outputs are early-clobber:
// data that returns must not overwrite an address.
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
#define MOE_TR4(d0, d1, d2, d3, a)                  \
  "ds_read_b64_tr_b16 " d0 ", " a "\n\t"            \
  "ds_read_b64_tr_b16 " d1 ", " a " offset:2048\n\t"  \
  "ds_read_b64_tr_b16 " d2 ", " a " offset:16384\n\t" \
  "ds_read_b64_tr_b16 " d3 ", " a " offset:18432\n\t"
template <int N>
__device__ __forceinline__ void read_krow_blocks(u32x4* s0, u32x4* s1, const uint32_t* addr) {
  static_assert(N == 1 || N == 2 || N == 4, "blocks");
  u32x2 r[N][4];
  if constexpr (N == 4) {
    asm volatile(MOE_TR4("%0", "%1", "%2", "%3", "%16") MOE_TR4("%4", "%5", "%6", "%7", "%17")
                     MOE_TR4("%8", "%9", "%10", "%11", "%18")
                         MOE_TR4("%12", "%13", "%14", "%15", "%19") "s_waitcnt lgkmcnt(0)"
                 : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3]), "=&v"(r[1][0]),
                   "=&v"(r[1][1]), "=&v"(r[1][2]), "=&v"(r[1][3]), "=&v"(r[2][0]), "=&v"(r[2][1]),
                   "=&v"(r[2][2]), "=&v"(r[2][3]), "=&v"(r[3][0]), "=&v"(r[3][1]), "=&v"(r[3][2]),
                   "=&v"(r[3][3])
                 : "v"(addr[0]), "v"(addr[1]), "v"(addr[2]), "v"(addr[3])
                 : "memory");
  } else if constexpr (N == 2) {
    asm volatile(MOE_TR4("%0", "%1", "%2", "%3", "%8") MOE_TR4("%4", "%5", "%6", "%7", "%9")
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3]), "=&v"(r[1][0]),
                   "=&v"(r[1][1]), "=&v"(r[1][2]), "=&v"(r[1][3])
                 : "v"(addr[0]), "v"(addr[1])
                 : "memory");
  } else {
    asm volatile(MOE_TR4("%0", "%1", "%2", "%3", "%4") "s_waitcnt lgkmcnt(0)"
                 : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3])
                 : "v"(addr[0])
                 : "memory");
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s0[i] = u32x4{r[i][0][0], r[i][0][1], r[i][1][0], r[i][1][1]};
    s1[i] = u32x4{r[i][2][0], r[i][2][1], r[i][3][0], r[i][3][1]};
  }
}
#undef MOE_TR4

// Source of one wavefront's 8 loads of a stage: a base that moves with the
// stage, and each lane's offset from it.
struct Feed {
  const char* base;
  size_t step;      // bytes from one stage to the next
  uint32_t off[8];
  int krow;         // K-row operand: this lane's K-row of load 0 (load j: + 2 j)
  int kcount;       // K-rows there are (those past it read zeros)
};

template <int MODE, bool GATED, bool FP8W>
__global__ __launch_bounds__(512, 1) void linear_mfma_kernel(LinearArgs g,
                                                             const bf16_t* __restrict__ dz,
                                                             bf16_t* __restrict__ out) {
  static_assert(!FP8W || MODE == kFwd, "FP8 weights: forward");
  constexpr bool AK = MODE == kDw, BK = MODE != kFwd;
  constexpr int COLS = GATED ? kT / 2 : kT;
  __shared__ __attribute__((aligned(1024))) char smem[kLds];
  auto abuf = [&](int i) -> char* { return smem + i * kBuf; };
  auto bbuf = [&](int i) -> char* { return smem + (kABufs + i) * kBuf; };

  // ------------------------------------------------------- work of this block
  const int n_dim = MODE == kFwd ? g.out_dim : g.in_dim;
  const int nt = (n_dim + COLS - 1) / COLS;
  int e, m0, n0, valid, seg, count;
  if constexpr (MODE == kDw) {
    // Tiles of a group in bands of 4 row tiles, column by column, and the
    // list dealt to the XCDs in chunks of 16 (4 x 4 tiles): a chunk fetches
    // 4 + 4 operand tiles into one L2 for its 16 tiles, and a group with many
    // rows spreads over all XCDs.
    constexpr int BAND = 4, CHUNK = 16;
    const int mt = (g.z_dim + kT - 1) / kT;
    const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
    const long per = static_cast<long>(mt) * nt;
    const long w = (static_cast<long>(idx / CHUNK) * 8 + xcd) * CHUNK + idx % CHUNK;
    if (w >= per * g.groups) return;
    e = static_cast<int>(w / per);
    const int q = static_cast<int>(w - e * per);
    const int band = q / (BAND * nt), h = min(BAND, mt - band * BAND), r = q - band * BAND * nt;
    m0 = (band * BAND + r % h) * kT;
    n0 = r / h * COLS;
    const int2 range = group_range(g.offsets, e, g.rows);
    seg = __builtin_amdgcn_readfirstlane(range.x);
    count = __builtin_amdgcn_readfirstlane(range.y) - seg;
    valid = min(kT, g.z_dim - m0);
  } else {
    TileAt at;
    int col;
    if (!find_item(g.offsets, g.groups, g.rows, kT, nt, at, col)) return;
    e = __builtin_amdgcn_readfirstlane(at.e);
    m0 = __builtin_amdgcn_readfirstlane(at.m) * kT;
    n0 = __builtin_amdgcn_readfirstlane(col) * COLS;
    seg = __builtin_amdgcn_readfirstlane(at.begin);
    count = __builtin_amdgcn_readfirstlane(at.end) - seg;
    valid = min(kT, count - m0);
  }

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Wavefront (grp, q) computes the 16-row blocks q, q + 4, q + 8, q + 12 of
  // the tile, effective columns 128 grp ...  Taking turns, the four share the
  // rows of a partly filled tile: its phases run the MFMAs of `mlive` blocks.
  const int grp = wave >> 2, q = wave & 3;
  const int mlive = __builtin_amdgcn_readfirstlane(min(max((valid - q * 16 + 63) / 64, 0), kMB));
  const size_t wmat = static_cast<size_t>(g.z_dim) * g.in_dim;
  const char* const w = static_cast<const char*>(g.w) + e * wmat * (FP8W ? 1 : 2);

  // --------------------------------------------------- this lane's sources
  // Row operand: load j of wavefront q stages rows 64 q + 8 j .. + 7, lane l
  // the chunk of row l / 8 that the swizzle puts at its place.  K-row operand:
  // K-rows 16 q + 2 j and + 1, 32 lanes each.  Rows and columns past the end
  // repeat the last one; what they give is not written.
  Feed f;
  const int chunk = line_lane_chunk(lane, 0) * 16;
  f.krow = 2 * 8 * q + (lane >> 5);
  f.kcount = MODE == kDw ? count : g.z_dim;
  auto krow_feed = [&](const bf16_t* p, int ld, int c0) {
    f.base = reinterpret_cast<const char*>(p + c0);
    f.step = static_cast<size_t>(64) * ld * 2;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int kk = f.krow + 2 * j;
      const int c = min(c0 + 8 * ((lane & 31) ^ krow_key(kk)), ld - 8);
      f.off[j] = (static_cast<uint32_t>(kk) * ld + (c - c0)) * 2;
    }
  };
  if (grp == 0) {
    if constexpr (AK) {
      krow_feed(dz + static_cast<size_t>(seg) * g.z_dim, g.z_dim, m0);
    } else {
      const uint32_t row_bytes = static_cast<uint32_t>(MODE == kFwd ? g.in_dim : g.z_dim) * 2;
      const bool gather = MODE == kFwd && g.row_index != nullptr;
      f.base = MODE == kFwd ? static_cast<const char*>(g.x) : reinterpret_cast<const char*>(dz);
      if (!gather) f.base += static_cast<size_t>(seg + m0) * row_bytes;
      f.step = kLineBytes;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = min(q * 64 + j * 8 + (lane >> 3), valid - 1);
        const int src = gather ? min(max(g.row_index[seg + m0 + r], 0), g.x_rows - 1) : r;
        f.off[j] = static_cast<uint32_t>(src) * row_bytes + chunk;
      }
    }
  } else if constexpr (MODE == kDw) {
    krow_feed(static_cast<const bf16_t*>(g.x) + static_cast<size_t>(seg) * g.in_dim, g.in_dim, n0);
  } else if constexpr (MODE == kDx) {
    krow_feed(reinterpret_cast<const bf16_t*>(w), g.in_dim, n0);
  } else {
    // SwiGLU: staged rows 0 .. 127 are gate rows, 128 .. 255 the up rows of
    // the same columns
    const uint32_t row_bytes = static_cast<uint32_t>(g.in_dim) * (FP8W ? 1 : 2);
    const bool up = GATED && q >= 2;
    f.base = w + (static_cast<size_t>(n0) + (up ? g.out_dim : 0)) * row_bytes;
    f.step = kLineBytes;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = q * 64 + j * 8 + (lane >> 3) - (up ? COLS : 0);
      f.off[j] = static_cast<uint32_t>(min(r, n_dim - 1 - n0)) * row_bytes + chunk;
    }
  }
  {  // the same in every lane: keep it in scalar registers
    const uint64_t b = reinterpret_cast<uint64_t>(f.base);
    const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(b)));
    const uint64_t hi =
        static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(b >> 32)));
    f.base = reinterpret_cast<const char*>(lo | (hi << 32));
  }
  const int nst = MODE == kDw ? (count + 63) / 64
                              : (MODE == kFwd ? g.in_dim : g.z_dim) / 64;  // stages
  const int last = (FP8W && grp == 1 ? nst / 2 : nst) - 1;  // last buffer of this operand
  // The loads of buffer p into `ring`; past the end the last one again, into
  // a buffer that nobody reads any more.  nt_: with the non-temporal policy.
  auto issue = [&](int p, char* ring, auto nt_) {
    const int pc = min(p, last);
    const char* const src = f.base + pc * f.step;
    char* const dst = ring + q * 8192;
    if (MODE == kDw && pc * 64 + 64 > f.kcount) {  // the group's last, partial stage
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = pc * 64 + f.krow + 2 * j < f.kcount;
        load_lds16(in ? src + f.off[j] : reinterpret_cast<const char*>(zero_chunk), dst + j * 1024);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // opaque, so that it is widened here and the load takes the scalar base
      // and a 32-bit offset; hoisted, each would hold a 64-bit address
      uint32_t o = f.off[j];
      asm volatile("" : "+v"(o));
      if constexpr (decltype(nt_)::value != 0) load_lds16_nt(src + o, dst + j * 1024);
      else load_lds16(src + o, dst + j * 1024);
    }
  };

  // ------------------------------------------------------- fragment addresses
  const int frow = lane & 15, fkey = swz128_key(frow);
  // a row's chunk of K step 0 and 1 of a stage; of codes: of the first and the
  // second stage of a buffer
  const int ch0 = FP8W ? 2 * (lane >> 4) : lane >> 4, ch1 = FP8W ? ch0 + 1 : ch0 + 4;
  const int fl0 = frow * kLineBytes + ((ch0 ^ fkey) << 4);
  const int fl1 = frow * kLineBytes + ((ch1 ^ fkey) << 4);
  const int f8l0 = frow * kLineBytes + (((lane >> 4) ^ fkey) << 4);
  const int f8l1 = frow * kLineBytes + (((4 + (lane >> 4)) ^ fkey) << 4);
  const int krow = 8 * (lane >> 4) + ((lane & 15) >> 2);
  const int klane = krow * 512 + ((lane & 3) >> 1) * 16 + (lane & 1) * 8;
  const int kkey = krow_key(krow);
  auto b_row = [&](int j) {  // first staged row (column of the tile) of block j
    if (GATED) return (j < kNB / 2 ? 0 : COLS) + grp * 64 + (j % (kNB / 2)) * 16;
    return grp * kWN + j * 16;
  };
  // K-row operand: N blocks from tile column c0 + i dc into fr[0 .. 1][first + i].
  // The addresses are made anew from an opaque key, so that none lives in a
  // register through the loop.
  u32x4 fr[2][kMB + kNB];
  auto read_krows = [&](const char* buf, auto n_, int first, int c0, int dc) {
    constexpr int N = decltype(n_)::value;
    uint32_t kx = static_cast<uint32_t>(kkey) << 4;
    uint32_t la = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
                      (const __attribute__((address_space(3))) char*)(buf))) +
                  klane;
    asm volatile("" : "+v"(kx), "+v"(la));
    uint32_t addr[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      addr[i] = la + ((static_cast<uint32_t>((c0 + i * dc) >> 3) << 4) ^ kx);
    read_krow_blocks<N>(&fr[0][first], &fr[1][first], addr);
  };

  f32x4 acc[kMB][kNB];
#pragma unroll
  for (int i = 0; i < kMB; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (nst > 0) {  // the same for the whole workgroup
    // W of a group whose rows fit one tile is read by this tile alone: past
    // L2, where the rows of x stay longer
    const bool once = MODE == kFwd && count <= kT;
    if (grp == 0) {
      issue(0, abuf(0), CInt<0>{});
      wait_vmem<0>();
    } else {
      if (once) {
        issue(0, bbuf(0), CInt<1>{});
        issue(1, bbuf(1), CInt<1>{});
      } else {
        issue(0, bbuf(0), CInt<0>{});
        issue(1, bbuf(1), CInt<0>{});
      }
      wait_vmem<8>();
    }
    stage_barrier();

    // A straight loop for each of the two halves: a shared one that branches
    // every phase makes the compiler move the accumulators out of the AGPRs.
    // Phases h = 0 .. 2 nst: half 0 reads in h = 2p and computes in 2p + 1,
    // half 1 reads in 2p + 1 and computes in 2p + 2.
    auto run = [&](auto live_, auto grp_, auto nt_) {
      constexpr int LIVE = decltype(live_)::value, G = decltype(grp_)::value;
      auto read = [&](int p) {
        const char* const a = abuf(p & 1);
        const char* const b = bbuf(FP8W ? (p >> 1) % 3 : p % 3);
        if (G == 0) issue(p + 1, abuf((p + 1) & 1), nt_);
        else if (!FP8W) issue(p + 2, bbuf((p + 2) % 3), nt_);
        else if ((p & 1) == 0) issue((p >> 1) + 2, bbuf(((p >> 1) + 2) % 3), nt_);
        if constexpr (LIVE > 0) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int fl = t ? fl1 : fl0;
            if constexpr (!AK) {
#pragma unroll
              for (int i = 0; i < LIVE; ++i)
                fr[t][i] =
                    *reinterpret_cast<const u32x4*>(a + (i * 64 + q * 16) * kLineBytes + fl);
            }
            if constexpr (!BK) {
              if (!FP8W || t == 0) {
#pragma unroll
                for (int j = 0; j < kNB; ++j)
                  fr[t][kMB + j] = *reinterpret_cast<const u32x4*>(
                      b + b_row(j) * kLineBytes + (FP8W ? ((p & 1) ? f8l1 : f8l0) : fl));
              }
            }
          }
          if constexpr (AK) read_krows(a, live_, 0, q * 16, 64);
          if constexpr (BK) {
            read_krows(b, CInt<4>{}, kMB, grp * kWN, 16);
            read_krows(b, CInt<4>{}, kMB + 4, grp * kWN + 64, 16);
          }
        }
        // fragments are in registers; half 0 leaves A(p + 1) in flight, half 1
        // waits for B(p + 1) and leaves B(p + 2) (codes: the next two stages'
        // buffer after an odd stage; after an even one it is there already)
        if (G == 0 || (FP8W && (p & 1) == 0)) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        else wait_vmem<8>();
      };
      auto compute = [&]() {
        __builtin_amdgcn_s_setprio(2);
        if constexpr (FP8W && LIVE > 0) {
          // the first MFMA of a widened fragment waits out the VALU's write;
          // the fragment before stays allocated until this one's MFMAs are
          // issued, so no widening writes what an MFMA just issued still reads
          u32x4 before = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < kNB; ++j) {
              const u32x4 c = fr[0][kMB + j];
              const u32x4 v = e4m3x8_to_bf16(t ? make_uint2(c[2], c[3]) : make_uint2(c[0], c[1]));
              mfma_bf16_agpr_after_valu(acc[0][j], fr[t][0], v);
#pragma unroll
              for (int i = 1; i < LIVE; ++i) mfma_bf16_agpr(acc[i][j], fr[t][i], v);
              asm volatile("" ::"v"(before));
              before = v;
            }
        } else {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < kNB; ++j)
#pragma unroll
              for (int i = 0; i < LIVE; ++i) mfma_bf16_agpr(acc[i][j], fr[t][i], fr[t][kMB + j]);
        }
        __builtin_amdgcn_s_setprio(0);
      };
      if (G == 0) {
        for (int p = 0; p < nst; ++p) {
          read(p);
          stage_barrier();
          compute();
          wait_vmem<0>();  // A(p + 1) has landed before anyone reads it
          stage_barrier();
        }
        stage_barrier();
      } else {
        stage_barrier();
        for (int p = 0; p < nst; ++p) {
          read(p);
          stage_barrier();
          compute();
          stage_barrier();
        }
        wait_vmem<0>();  // the loads past the last stage
      }
      stage_barrier();  // nothing is in flight, nobody reads the buffers
    };
    auto run_live = [&](auto grp_, auto nt_) {
      if (mlive == 4 || (AK && mlive == 3)) run(CInt<4>{}, grp_, nt_);
      else if (mlive == 3) run(CInt<AK ? 4 : 3>{}, grp_, nt_);
      else if (mlive == 2) run(CInt<2>{}, grp_, nt_);
      else if (mlive == 1) run(CInt<1>{}, grp_, nt_);
      else run(CInt<0>{}, grp_, nt_);
    };
    if (grp == 0) run_live(CInt<0>{}, CInt<0>{});
    else if (once) run_live(CInt<1>{}, CInt<1>{});
    else run_live(CInt<1>{}, CInt<0>{});
  }

  // -------------------------------------------------------------- epilogue
  // 32 rows of the wavefront's block at a time through LDS, as two fp32
  // arrays of 64 columns (SwiGLU: gate and up of the same columns), then 8
  // columns of a row per lane: whole 128-byte lines of y, and the 8 lanes of
  // a 64-column block agree on its checkpoint scale.  A lane's columns are the
  // same throughout, so the bias is read once; the residual's rows are asked
  // for before the staging.
  mfma_drain();
  char* const stg = smem + wave * 2 * 32 * kStgPitch;
  const int c = (lane & 7) * 8;
  const int n = n0 + (GATED ? grp * 64 : grp * kWN) + c;
  const bool in0 = n < n_dim, in1 = !GATED && n + 64 < n_dim;
  float b0[8], b1[8], s0[8], s1[8];
  if constexpr (MODE == kFwd) {
    const size_t eo = static_cast<size_t>(e) * g.z_dim + n;
    if constexpr (FP8W) {
      load_cols8(g.w_scale, eo, in0, 1.f, s0);
      load_cols8(g.w_scale, eo + (GATED ? g.out_dim : 64), GATED ? in0 : in1, 1.f, s1);
    }
    load_cols8(g.bias, eo, in0, 0.f, b0);
    load_cols8(g.bias, eo + (GATED ? g.out_dim : 64), GATED ? in0 : in1, 0.f, b1);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    auto tile_row = [&](int k) {
      const int lr = k * 8 + (lane >> 3);
      return (2 * h + (lr >> 4)) * 64 + q * 16 + (lr & 15);
    };
    Raw8<bf16_t> r0[4], r1[4];
    if constexpr (MODE == kFwd) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = tile_row(k);
        load_residual<bf16_t>(g, seg + m0 + row, n, row < valid && in0, r0[k]);
        if (!GATED) load_residual<bf16_t>(g, seg + m0 + row, n + 64, row < valid && in1, r1[k]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<float*>(stg + (j / 4 * 32 + i * 16 + 4 * (lane >> 4) + r) * kStgPitch +
                                    ((j % 4) * 16 + (lane & 15)) * 4) = acc[2 * h + i][j][r];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // own rows only: no barrier
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int lr = k * 8 + (lane >> 3), row = tile_row(k);
      float v[8], u[8];
      load8<float>(reinterpret_cast<const float*>(stg + lr * kStgPitch) + c, v);
      load8<float>(reinterpret_cast<const float*>(stg + (32 + lr) * kStgPitch) + c, u);
      if constexpr (MODE == kFwd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = (FP8W ? v[i] * s0[i] : v[i]) + b0[i];
          u[i] = (FP8W ? u[i] * s1[i] : u[i]) + b1[i];
        }
        const long r = static_cast<long>(seg) + m0 + row;
        if constexpr (GATED) {
          linear_epilogue8<bf16_t, true>(g, r, n, row < valid && in0, v, u, r0[k]);
        } else {
          linear_epilogue8<bf16_t, false>(g, r, n, row < valid && in0, v, nullptr, r0[k]);
          linear_epilogue8<bf16_t, false>(g, r, n + 64, row < valid && in1, u, nullptr, r1[k]);
        }
      } else {
        const size_t r = MODE == kDx ? static_cast<size_t>(seg) + m0 + row
                                     : static_cast<size_t>(e) * g.z_dim + m0 + row;
        bf16_t* const o = out + r * g.in_dim + n;
        if (row < valid && in0) store_once8<bf16_t>(o, v);
        if (row < valid && in1) store_once8<bf16_t>(o + 64, u);
      }
    }
    asm volatile("" ::: "memory");
  }
}

template <int MODE, bool GATED, bool FP8W = false>
hipError_t launch_t(const LinearArgs& g, const void* dz, void* out, hipStream_t s) {
  constexpr int COLS = GATED ? kT / 2 : kT;
  const long nt = ((MODE == kFwd ? g.out_dim : g.in_dim) + COLS - 1) / COLS;
  long blocks;
  if (MODE == kDw) {
    const long chunks = (static_cast<long>(g.groups) * ((g.z_dim + kT - 1) / kT) * nt + 15) / 16;
    blocks = 8 * ((chunks + 7) / 8) * 16;
  } else {
    blocks = item_grid(g.rows, g.groups, kT, nt);
  }
  hipLaunchKernelGGL((linear_mfma_kernel<MODE, GATED, FP8W>), dim3(static_cast<unsigned>(blocks)),
                     dim3(512), 0, s, g, static_cast<const bf16_t*>(dz),
                     static_cast<bf16_t*>(out));
  return hipGetLastError();
}

}  // namespace

bool linear_mfma_fits(bool wfp8, bool gather, const LinearArgs& g) {
  // 32-bit offsets into x when its rows are gathered; whole buffers of codes
  return (!gather || static_cast<size_t>(g.x_rows) * g.in_dim * 2 < (size_t{1} << 32)) &&
         (!wfp8 || g.in_dim % 128 == 0);
}

hipError_t launch_linear_mfma(bool wfp8, const LinearArgs& g, hipStream_t s) {
  if (!linear_mfma_fits(wfp8, g.row_index != nullptr, g)) return hipErrorInvalidValue;
  if (wfp8)
    return g.act == kActSwiglu ? launch_t<kFwd, true, true>(g, nullptr, nullptr, s)
                               : launch_t<kFwd, false, true>(g, nullptr, nullptr, s);
  return g.act == kActSwiglu ? launch_t<kFwd, true>(g, nullptr, nullptr, s)
                             : launch_t<kFwd, false>(g, nullptr, nullptr, s);
}

hipError_t launch_linear_mfma_dx(const LinearArgs& g, const void* dz, void* dx, hipStream_t s) {
  return launch_t<kDx, false>(g, dz, dx, s);
}

hipError_t launch_linear_mfma_dw(const LinearArgs& g, const void* dz, void* dw, hipStream_t s) {
  if (g.row_index != nullptr) return hipErrorInvalidValue;
  return launch_t<kDw, false>(g, dz, dw, s);
}

}  // namespace moe
