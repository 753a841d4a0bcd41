// Selective state-space scan: gam_selective_scan, and its calls in fp32.
#include "selective_scan.cuh"

namespace gam {
namespace ops {

gam_status scan_f16(const gam_scan_args& p, int sms, cudaStream_t s);
gam_status scan_bf16(const gam_scan_args& p, int sms, cudaStream_t s);

}  // namespace ops
}  // namespace gam

using namespace gam::ops;

extern "C" gam_status gam_selective_scan(const gam_scan_args* args, void* stream) {
  return guarded([&] {
    if (!args) return op_fail(GAM_ERR_INVALID_ARG, "null args");
    const gam_scan_args p = *args;
    if (!is_float_dtype(p.dtype)) return op_fail(GAM_ERR_INVALID_ARG, "dtype must be f32, f16 or bf16");
    if (p.batch < 0 || p.t_max < 0 || p.d < 1) return op_fail(GAM_ERR_INVALID_ARG, "batch >= 0, t_max >= 0 and d >= 1");
    if (p.n < 1 || p.n > 64) return op_fail(GAM_ERR_SHAPE, "n must be 1 .. 64");
    if (p.t_max > kMaxDim || p.d > kMaxDim) return op_fail(GAM_ERR_CAPACITY, "t_max and d up to 2^30");
    if (p.batch == 0) return GAM_OK;
    if (!p.a || (p.t_max > 0 && (!p.x || !p.dt || !p.b || !p.c || !p.y)))
      return op_fail(GAM_ERR_INVALID_ARG, "null pointer");
    const int es = dtype_size(p.dtype);
    if (!aligned(p.x, es) || !aligned(p.dt, es) || !aligned(p.b, es) || !aligned(p.c, es) || !aligned(p.z, es) ||
        !aligned(p.y, es) || !aligned(p.a, 4) || !aligned(p.d_skip, 4) || !aligned(p.dt_bias, 4) ||
        !aligned(p.lengths, 4) || !aligned(p.state_in, 4) || !aligned(p.state_out, 4))
      return op_fail(GAM_ERR_INVALID_ARG, "a buffer is not aligned to its element type");
    if (p.t_max > 0 && (p.y == p.x || p.y == p.dt || p.y == p.b || p.y == p.c || p.y == p.z))
      return op_fail(GAM_ERR_INVALID_ARG, "y must not be an input");
    if (!rows_apart(p.batch, p.t_max, p.d, p.y_batch_stride, p.y_row_stride))
      return op_fail(GAM_ERR_SHAPE, "rows of y overlap");
    int sms = 0;
    if (gam_status st = check_device(&sms)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.dtype == GAM_DTYPE_F32) return launch<float>(p, sms, s);
    if (p.dtype == GAM_DTYPE_F16) return scan_f16(p, sms, s);
    return scan_bf16(p, sms, s);
  });
}
