// C ABI of the dense operators: argument checks and launches.  The operations
// are documented in include/moe_capi.h.
#include "dense_internal.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char* p = static_cast<const char*>(a);
  const char* q = static_cast<const char*>(b);
  return p < q + nb && q < p + na;
}

size_t type_size(int type) { return type == MOE_FP32 ? 4 : 2; }

// The packed product's arguments; rows already counts gate and up rows.
int check_linear(const LinearCall& c, const moe_config* cfg, int out_cols) {
  if (!cfg || c.rows <= 0 || c.cols <= 0 || c.T < 0) return MOE_ERR_INVALID_ARG;
  if (c.x_type != MOE_BF16 && c.x_type != MOE_FP16) return MOE_ERR_INVALID_ARG;
  if (c.y_type != MOE_BF16 && c.y_type != MOE_FP16 && c.y_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (cfg->bits != 4 || (cfg->block != 32 && cfg->block != 128)) return MOE_ERR_UNSUPPORTED;
  if (cfg->half_levels != 0 && cfg->half_levels != 1) return MOE_ERR_UNSUPPORTED;
  if (cfg->scale_fmt != 0 && cfg->scale_fmt != 1) return MOE_ERR_UNSUPPORTED;
  if (cfg->scale_fmt == 1 && (cfg->block == 128 || cfg->half_levels)) return MOE_ERR_UNSUPPORTED;
  if (c.cols % cfg->block != 0 || c.cols > kLinearMaxCols || c.rows > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (c.T == 0) return MOE_OK;
  if (!c.codes || !c.scales || !c.x || !c.y) return MOE_ERR_INVALID_ARG;
  if (!aligned(c.codes, 16) || !aligned(c.scales, 16) || !aligned(c.x, 16) || !aligned(c.y, 16))
    return MOE_ERR_INVALID_ARG;
  if (cfg->scale_fmt == 1 ? (!c.row_scales || !aligned(c.row_scales, 16)) : c.row_scales != nullptr)
    return MOE_ERR_INVALID_ARG;
  if (c.bias && !aligned(c.bias, 4)) return MOE_ERR_INVALID_ARG;
  if (overlap(c.x, size_t(c.T) * c.cols * 2, c.y, size_t(c.T) * out_cols * type_size(c.y_type)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int run_linear(LinearCall& c, const moe_config* cfg, int out_cols, void* stream) {
  const int st = check_linear(c, cfg, out_cols);
  if (st != MOE_OK || c.T == 0) return st;
  c.block = cfg->block;
  c.half_levels = cfg->half_levels;
  c.scale_fmt = cfg->scale_fmt;
  return status_of_cuda(launch_linear(c, num_sms_of_current_device(), static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int moe_linear_forward(const moe_config* cfg, const uint8_t* codes, const void* scales, const float* row_scales,
                       int32_t rows, int32_t cols, const float* bias, const void* x, int32_t x_type, int32_t T,
                       void* y, int32_t y_type, void* stream) {
  LinearCall c{};
  c.codes = codes; c.scales = scales; c.row_scales = row_scales; c.bias = bias; c.x = x; c.y = y;
  c.rows = rows; c.cols = cols; c.T = T; c.x_type = x_type; c.y_type = y_type;
  return run_linear(c, cfg, rows, stream);
}

int moe_linear_gated_forward(const moe_config* cfg, const uint8_t* codes, const void* scales,
                             const float* row_scales, int32_t inter, int32_t cols, const void* x, int32_t x_type,
                             int32_t T, void* h, int32_t h_type, void* stream) {
  if (inter <= 0) return MOE_ERR_INVALID_ARG;
  if (inter > (1 << 29)) return MOE_ERR_UNSUPPORTED;
  LinearCall c{};
  c.codes = codes; c.scales = scales; c.row_scales = row_scales; c.x = x; c.y = h;
  c.rows = 2 * inter; c.cols = cols; c.T = T; c.x_type = x_type; c.y_type = h_type; c.gated = 1;
  return run_linear(c, cfg, inter, stream);
}

}  // extern "C"
