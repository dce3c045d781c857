// Host side of the calls for experts of one's own (include/moe.h): argument
// checks, workspace layout and launch sequences.  Nothing here allocates,
// frees or waits on the device.
#include "moe.h"
#include "api_error.h"
#include "linear.h"

#include <algorithm>

namespace moe {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int z_dim(const moe_linear_config& c) {
  return c.activation == MOE_ACT_SWIGLU ? 2 * c.out_dim : c.out_dim;
}

long weights(const moe_linear_config& c) {
  return static_cast<long>(c.groups) * z_dim(c) * c.in_dim;
}

moe_status check_dtype(int dtype) {
  return dtype == MOE_F32 || dtype == MOE_BF16 ? MOE_OK : fail(MOE_ERR_INVALID_ARG, "bad dtype");
}

moe_status check_linear(const moe_linear_config* c) {
  if (c == nullptr) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
  if (c->rows < 0 || c->x_rows < 0 || c->groups <= 0 || c->in_dim <= 0 || c->out_dim <= 0)
    return fail(MOE_ERR_INVALID_ARG, "sizes must be positive (rows, x_rows >= 0)");
  if (check_dtype(c->dtype) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (c->weight_format != MOE_WEIGHTS_DTYPE && c->weight_format != MOE_WEIGHTS_FP8_E4M3)
    return fail(MOE_ERR_INVALID_ARG, "bad weight_format");
  if (c->activation < MOE_ACT_NONE || c->activation > MOE_ACT_SWIGLU)
    return fail(MOE_ERR_INVALID_ARG, "bad activation");
  if (c->weight_format == MOE_WEIGHTS_FP8_E4M3 && c->dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "FP8 weights need dtype MOE_BF16");
  if (c->groups > kMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "groups > 512");
  if (c->in_dim % 64 != 0 || c->out_dim % 64 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "in_dim and out_dim must be multiples of 64");
  if (c->in_dim > (1 << 20) || c->out_dim > (1 << 20))
    return fail(MOE_ERR_UNSUPPORTED, "in_dim or out_dim > 2^20");
  if (c->rows >= (1 << 27) || c->x_rows >= (1 << 30))
    return fail(MOE_ERR_UNSUPPORTED, "too many rows");
  // Grids stay below 2^32 threads: at most 2^23 tiles of 128 rows by 64 columns,
  // forward and dX.  There are twice as many tiles of 64 x 64, but launch_t
  // takes them only for few tiles, or where fewer than 3.6 of them make one of
  // 128 x 128: for 7 columns of them at most, times 2^21 rows of tiles.
  const long wide = std::max(c->in_dim, z_dim(*c));
  if ((c->rows / 128 + c->groups) * (wide / 64) > (1L << 23))
    return fail(MOE_ERR_UNSUPPORTED, "too many tiles");
  if (weights(*c) > (1L << 39)) return fail(MOE_ERR_UNSUPPORTED, "more than 2^39 weights");
  return MOE_OK;
}

moe_status check_rows_of_x(const moe_linear_config& c, const int32_t* row_index) {
  if ((c.x_rows > 0) != (row_index != nullptr) && c.rows > 0)
    return fail(MOE_ERR_INVALID_ARG, "row_index and x_rows go together");
  return MOE_OK;
}

moe_status check_space(const void* ws, size_t have, size_t need) {
  if (ws == nullptr) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0)
    return fail(MOE_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (have < need) return fail(MOE_ERR_WORKSPACE, "workspace smaller than its size function says");
  return MOE_OK;
}

LinearArgs linear_args(const moe_linear_config& c) {
  LinearArgs g{};
  g.rows = c.rows;
  g.groups = c.groups;
  g.in_dim = c.in_dim;
  g.out_dim = c.out_dim;
  g.z_dim = z_dim(c);
  g.x_rows = c.x_rows > 0 ? c.x_rows : c.rows;
  g.act = c.activation;
  return g;
}

// Whether the forward streams W through registers (linear_rows.hip) instead of
// taking tiles: few rows a group on average.  Mixtral-shaped gate and up
// projection (8 experts, 4096 -> 14336, SwiGLU), us with few-row / with the
// other kernels:
//   bf16  8 rows a group 327 / 339, 12: 341 / 334, 16: 376 / 346, 32: 620 / 330
//   FP8   8 rows 193 / 244, 12: 227 / 239, 16: 255 / 239, 32: 448 / 239
//   fp32  1 row 656 / 649, 8: 649 / 624, 16: 695 / 634, 32: 1032 / 810; one
//         expert 1 row 100 / 109, 8: 103 / 109, 24: 144 / 114; 1024 -> 2048 of
//         one expert 1 row 12.3 / 15.7, 8: 13.5 / 16.3, 32: 16.6 / 16.7
// Only the average is known here, so few rows in all as well: 256 experts of
// 2048 -> 2 x 2048 with 2048 rows, spread evenly / all in one of them,
//   bf16  693 / 237 against 703 / 45 (256 rows: 683 / 41 against 694 / 44)
//   FP8   411 / 183 against 530 / 51
//   fp32  1513 / 532 against 1546 / 314 (256 rows: 1409 / 77 against 1534 / 57)
bool streams_rows(const moe_linear_config& c, const LinearArgs& g) {
  const long G = c.groups;
  const long most = c.weight_format == MOE_WEIGHTS_FP8_E4M3 ? std::min(12 * G, 2048L)
                                                            : std::min(8 * G, 256L);
  return c.rows <= most && linear_rows_fits(g);
}

// Whether a bf16 product has enough 256 x 256 tiles for the large-tile kernel
// (linear_mfma.hip): with at most a quarter of the compute units, the tiles of
// linear_tile.hip spread it over more of them.  us with large / with small
// tiles: forward of 1000 rows 2048 -> 4096 (64 tiles) 41 / 33, 3000 rows 4096
// -> 2048 (96) 70 / 76; backward of 600 rows of 4 experts 512 -> 1024 (12 and
// 32) 45 / 30, of 2000 rows of one expert 1024 -> 2 x 4096 201 / 205, and 151
// with dX (32) on small and dW (128) on large ones.
bool large_tiles(long row_tiles, int cols) {
  return row_tiles * ((cols + 255) / 256) > device_cus() / 4;
}
// Row tiles of 256 rows that the rows of all groups can need.
long row_tiles(const moe_linear_config& c) { return c.rows / 256 + std::min(c.groups, c.rows); }
// The same for the forward.  Small tiles also where few rows a group leave the
// large ones mostly empty and too few for the compute units: the forward with
// large / with small tiles of 500 rows of 16 groups 2048 -> 2048 (at most 136
// tiles, 16 by its rows) 41.8 / 34.5, of 200 rows of 4 groups 1024 -> 2 x 4096
// (128, 25) 24.2 / 13.8, of 512 rows of 8 groups 4096 -> 4096 (160, 32) 76.7 /
// 66.7; but 1000 rows of 16 groups 2048 -> 4096 in FP8 (304, 63) 39.5 / 46.0,
// 4000 rows of 8 groups 1024 -> 2048 (184, 125) 27.1 / 39.5.  (dX: 500 rows of
// 16 groups 2048 -> 2048, backward in all, 86.6 / 92.7.)
bool forward_large(const moe_linear_config& c, const LinearArgs& g) {
  const long nt = (g.z_dim + 255) / 256, cus = device_cus();
  return c.dtype == MOE_BF16 && large_tiles(row_tiles(c), g.z_dim) &&
         (c.rows * nt / 256 > cus / 4 || row_tiles(c) * nt > cus) &&
         linear_mfma_fits(c.weight_format == MOE_WEIGHTS_FP8_E4M3, c.x_rows > 0, g);
}
// Shares of K that the forward is split into.
int forward_parts(const moe_linear_config& c, const LinearArgs& g) {
  const int eb = c.dtype == MOE_BF16 ? 2 : 4;
  if (streams_rows(c, g)) return linear_rows_parts(eb, g, device_cus());
  return forward_large(c, g) ? 1 : linear_tile_parts(eb, g, device_cus());
}

// Workspace of the backward.
struct BackSpace {
  size_t dz, partial, xg, total;
};
BackSpace back_space(const moe_linear_config& c) {
  const size_t eb = c.dtype == MOE_BF16 ? 2 : 4, z = z_dim(c);
  BackSpace b{};
  size_t o = 0;
  b.dz = o;
  if (c.activation != MOE_ACT_NONE) o += align_up(static_cast<size_t>(c.rows) * z * eb);
  b.partial = o;
  o += align_up(static_cast<size_t>(act_tiles(c.rows, c.groups)) * z * 4);
  b.xg = o;
  if (c.dtype == MOE_BF16 && c.x_rows > 0)
    o += align_up(static_cast<size_t>(c.rows) * c.in_dim * eb);
  b.total = o > 0 ? o : kAlign;
  return b;
}

constexpr long kMaxGroupPairs = 1L << 30;

moe_status check_group(int32_t T, int32_t N, int32_t k) {
  if (T < 0 || N <= 0 || k <= 0) return fail(MOE_ERR_INVALID_ARG, "bad T, N or k");
  if (N > kMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "n_experts > 512");
  if (k > kMaxTopK) return fail(MOE_ERR_UNSUPPORTED, "top_k > 16");
  if (static_cast<long>(T) * k >= kMaxGroupPairs)
    return fail(MOE_ERR_UNSUPPORTED, "T * k too large");
  return MOE_OK;
}

moe_status check_combine(int32_t T, int32_t k, int32_t n_rows, int32_t d, int32_t dtype) {
  if (T < 0 || k <= 0 || n_rows < 0 || d <= 0)
    return fail(MOE_ERR_INVALID_ARG, "bad T, k, n_rows or d");
  if (check_dtype(dtype) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (k > kMaxTopK) return fail(MOE_ERR_UNSUPPORTED, "top_k > 16");
  if (d % 64 != 0) return fail(MOE_ERR_UNSUPPORTED, "d must be a multiple of 64");
  if (T >= (1 << 23)) return fail(MOE_ERR_UNSUPPORTED, "T >= 2^23");
  return MOE_OK;
}

moe_status check_checkpoint(int64_t rows, int32_t cols, int32_t dtype, const void* x,
                            const void* codes, const void* scale) {
  if (rows < 0 || cols <= 0) return fail(MOE_ERR_INVALID_ARG, "bad rows or cols");
  if (check_dtype(dtype) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (cols % kCkptBlock != 0) return fail(MOE_ERR_UNSUPPORTED, "cols must be a multiple of 64");
  if (rows > (int64_t{1} << 35) / cols) return fail(MOE_ERR_UNSUPPORTED, "rows * cols too large");
  if (rows == 0) return MOE_OK;
  if (x == nullptr || codes == nullptr || scale == nullptr)
    return fail(MOE_ERR_INVALID_ARG, "x, codes or scale is NULL");
  if (!aligned16(x) || !aligned16(codes))
    return fail(MOE_ERR_INVALID_ARG, "x or codes not 16-byte aligned");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_group_workspace_size(int32_t T, int32_t N, int32_t k) {
  if (check_group(T, N, k) != MOE_OK) return 0;
  return align_up(static_cast<size_t>(group_blocks(static_cast<long>(T) * k)) * N * 4);
}

moe_status moe_group_rows(int32_t T, int32_t N, int32_t k, int32_t capacity,
                          const int32_t* topk_idx, int32_t* offsets, int32_t* row_token,
                          int32_t* slot_row, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  moe_status st = check_group(T, N, k);
  if (st != MOE_OK) return st;
  if (capacity < 0) return fail(MOE_ERR_INVALID_ARG, "capacity < 0");
  if (offsets == nullptr) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if (T > 0 && (topk_idx == nullptr || row_token == nullptr || slot_row == nullptr))
    return fail(MOE_ERR_INVALID_ARG, "topk_idx, row_token or slot_row is NULL");
  if ((st = check_space(workspace, ws_bytes, moe_group_workspace_size(T, N, k))) != MOE_OK)
    return st;
  const hipError_t err =
      launch_group_rows(topk_idx, T, N, k, capacity, static_cast<int32_t*>(workspace), offsets,
                        row_token, slot_row, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_OK : hip_fail(err, "grouping kernel");
}

size_t moe_linear_workspace_size(const moe_linear_config* cfg) {
  if (check_linear(cfg) != MOE_OK) return 0;
  const LinearArgs g = linear_args(*cfg);
  const int parts = forward_parts(*cfg, g);
  return parts > 1 ? align_up(static_cast<size_t>(parts) * g.rows * g.z_dim * 4) : kAlign;
}

moe_status moe_grouped_linear(const moe_linear_config* cfg, const moe_linear_args* a,
                              void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  moe_status st = check_linear(cfg);
  if (st != MOE_OK) return st;
  const moe_linear_config& c = *cfg;
  if (a == nullptr) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
  if (c.rows == 0) return MOE_OK;
  const bool fp8 = c.weight_format == MOE_WEIGHTS_FP8_E4M3;
  if (a->x == nullptr || a->offsets == nullptr || a->w == nullptr || a->y == nullptr)
    return fail(MOE_ERR_INVALID_ARG, "x, offsets, w or y is NULL");
  if (fp8 != (a->w_scale != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "w_scale goes with FP8 weights");
  if ((a->z_codes != nullptr) != (a->z_scale != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "z_codes and z_scale go together");
  if (!aligned16(a->x) || !aligned16(a->w) || !aligned16(a->y) || !aligned16(a->residual) ||
      !aligned16(a->bias) || !aligned16(a->w_scale) || !aligned16(a->z_codes))
    return fail(MOE_ERR_INVALID_ARG, "a tensor is not 16-byte aligned");
  if ((st = check_rows_of_x(c, a->row_index)) != MOE_OK) return st;
  if ((st = check_space(workspace, ws_bytes, moe_linear_workspace_size(cfg))) != MOE_OK) return st;
  LinearArgs g = linear_args(c);
  g.x = a->x;
  g.row_index = a->row_index;
  g.offsets = a->offsets;
  g.w = a->w;
  g.w_scale = a->w_scale;
  g.bias = a->bias;
  g.residual = a->residual;
  g.y = a->y;
  g.z_codes = a->z_codes;
  g.z_scale = a->z_scale;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t err;
  if (streams_rows(c, g))
    err = launch_linear_rows(c.dtype, fp8, g, device_cus(), static_cast<float*>(workspace), s);
  else if (forward_large(c, g))
    err = launch_linear_mfma(fp8, g, s);
  else
    err = launch_linear_tile(c.dtype, fp8, g, device_cus(), static_cast<float*>(workspace), s);
  return err == hipSuccess ? MOE_OK : hip_fail(err, "grouped linear kernel");
}

size_t moe_linear_backward_workspace_size(const moe_linear_config* cfg) {
  if (check_linear(cfg) != MOE_OK) return 0;
  return back_space(*cfg).total;
}

moe_status moe_grouped_linear_backward(const moe_linear_config* cfg,
                                       const moe_linear_grad_args* a, void* workspace,
                                       size_t ws_bytes, void* stream) {
  clear_error();
  moe_status st = check_linear(cfg);
  if (st != MOE_OK) return st;
  const moe_linear_config& c = *cfg;
  if (c.weight_format != MOE_WEIGHTS_DTYPE)
    return fail(MOE_ERR_UNSUPPORTED, "the backward needs weights in dtype");
  if (a == nullptr) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
  // (without rows the only gradients there can be are those of w and bias)
  if (a->dw == nullptr && a->dbias == nullptr && c.rows == 0) return MOE_OK;
  if (a->dx == nullptr && a->dw == nullptr && a->dbias == nullptr)
    return fail(MOE_ERR_INVALID_ARG, "no gradient asked for");
  // dW's grid: below 2^24 tiles of 64 x 64
  if (a->dw != nullptr && weights(c) >= (1L << 36))
    return fail(MOE_ERR_UNSUPPORTED, "dw of 2^36 weights or more");
  if (a->offsets == nullptr) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  const bool act = c.activation != MOE_ACT_NONE;
  if (c.rows > 0) {
    if (a->dy == nullptr || (a->dx != nullptr && a->w == nullptr) ||
        (a->dw != nullptr && a->x == nullptr))
      return fail(MOE_ERR_INVALID_ARG, "dy, w or x is NULL");
    if (act && (a->z_codes == nullptr || a->z_scale == nullptr))
      return fail(MOE_ERR_INVALID_ARG, "the activation's backward needs z_codes and z_scale");
    if (a->dw != nullptr && (st = check_rows_of_x(c, a->row_index)) != MOE_OK) return st;
  }
  if (!aligned16(a->x) || !aligned16(a->w) || !aligned16(a->dy) || !aligned16(a->dx) ||
      !aligned16(a->dw) || !aligned16(a->dbias) || !aligned16(a->z_codes))
    return fail(MOE_ERR_INVALID_ARG, "a tensor is not 16-byte aligned");
  const BackSpace b = back_space(c);
  if ((st = check_space(workspace, ws_bytes, b.total)) != MOE_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  LinearArgs g = linear_args(c);
  g.x = a->x;
  g.row_index = a->row_index;
  g.offsets = a->offsets;
  g.w = a->w;
  g.z_codes = const_cast<uint8_t*>(a->z_codes);
  g.z_scale = const_cast<float*>(a->z_scale);
  char* base = static_cast<char*>(workspace);
  float* partial = a->dbias != nullptr ? reinterpret_cast<float*>(base + b.partial) : nullptr;
  const bool products = a->dx != nullptr || a->dw != nullptr;
  const void* dz = act ? base + b.dz : a->dy;
  hipError_t err;
  if (c.rows > 0 && ((act && products) || partial != nullptr)) {
    err = launch_act_backward(c.dtype, g, a->dy, act && products ? base + b.dz : nullptr, partial,
                              s);
    if (err != hipSuccess) return hip_fail(err, "activation backward");
  }
  if (a->dbias != nullptr && (err = launch_bias_grad(g, partial, a->dbias, s)) != hipSuccess)
    return hip_fail(err, "bias gradient");
  const bool bf16 = c.dtype == MOE_BF16;
  if (c.rows > 0 && a->dx != nullptr) {
    const bool large = bf16 && large_tiles(row_tiles(c), c.in_dim);
    err = large ? launch_linear_mfma_dx(g, dz, a->dx, s)
                : launch_linear_dx_tile(c.dtype, g, dz, a->dx, device_cus(), s);
    if (err != hipSuccess) return hip_fail(err, "dx");
  }
  if (a->dw != nullptr) {
    const bool large = bf16 && large_tiles(c.groups * ((g.z_dim + 255L) / 256), c.in_dim);
    if (large && g.row_index != nullptr && c.rows > 0) {
      // the large tiles stage x by its rows in order
      if ((err = launch_gather_rows(g, base + b.xg, s)) != hipSuccess)
        return hip_fail(err, "gather of x");
      g.x = base + b.xg;
    }
    if (large) g.row_index = nullptr;
    err = large ? launch_linear_mfma_dw(g, dz, a->dw, s)
                : launch_linear_dw_tile(c.dtype, g, dz, a->dw, device_cus(), s);
    if (err != hipSuccess) return hip_fail(err, "dw");
  }
  return MOE_OK;
}

moe_status moe_checkpoint_pack(int64_t rows, int32_t cols, int32_t dtype, const void* x,
                               uint8_t* codes, float* scale, void* stream) {
  clear_error();
  const moe_status st = check_checkpoint(rows, cols, dtype, x, codes, scale);
  if (st != MOE_OK || rows == 0) return st;
  const hipError_t err =
      launch_checkpoint_pack(dtype, x, rows, cols, codes, scale, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_OK : hip_fail(err, "checkpoint kernel");
}

moe_status moe_checkpoint_unpack(int64_t rows, int32_t cols, int32_t dtype, const uint8_t* codes,
                                 const float* scale, void* x, void* stream) {
  clear_error();
  const moe_status st = check_checkpoint(rows, cols, dtype, x, codes, scale);
  if (st != MOE_OK || rows == 0) return st;
  const hipError_t err = launch_checkpoint_unpack(dtype, codes, scale, rows, cols, x,
                                                  static_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_OK : hip_fail(err, "checkpoint kernel");
}

moe_status moe_combine(int32_t T, int32_t k, int32_t n_rows, int32_t d, int32_t dtype,
                       const void* rows, const int32_t* slot_row, const float* gate, void* y,
                       void* stream) {
  clear_error();
  const moe_status st = check_combine(T, k, n_rows, d, dtype);
  if (st != MOE_OK || T == 0) return st;
  if ((rows == nullptr && n_rows > 0) || slot_row == nullptr || y == nullptr)
    return fail(MOE_ERR_INVALID_ARG, "rows, slot_row or y is NULL");
  if (!aligned16(rows) || !aligned16(y))
    return fail(MOE_ERR_INVALID_ARG, "rows or y not 16-byte aligned");
  const hipError_t err = launch_combine_rows(dtype, rows, slot_row, gate, n_rows, T, k, d, y,
                                             static_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_OK : hip_fail(err, "combine kernel");
}

moe_status moe_combine_backward(int32_t T, int32_t k, int32_t n_rows, int32_t d, int32_t dtype,
                                const void* rows, const int32_t* slot_row, const float* gate,
                                const void* dy, void* drows, float* dgate, void* stream) {
  clear_error();
  const moe_status st = check_combine(T, k, n_rows, d, dtype);
  if (st != MOE_OK || T == 0) return st;
  if (drows == nullptr && dgate == nullptr)
    return fail(MOE_ERR_INVALID_ARG, "no gradient asked for");
  if (slot_row == nullptr || dy == nullptr || (dgate != nullptr && rows == nullptr && n_rows > 0))
    return fail(MOE_ERR_INVALID_ARG, "slot_row, dy or rows is NULL");
  if (!aligned16(rows) || !aligned16(dy) || !aligned16(drows))
    return fail(MOE_ERR_INVALID_ARG, "rows, dy or drows not 16-byte aligned");
  const hipError_t err =
      launch_combine_rows_backward(dtype, rows, slot_row, gate, dy, n_rows, T, k, d, drows, dgate,
                                   static_cast<hipStream_t>(stream));
  return err == hipSuccess ? MOE_OK : hip_fail(err, "combine backward kernel");
}

}  // extern "C"
