// Selective state-space scan: calls in bf16.
#include "selective_scan.cuh"

namespace gam {
namespace ops {

gam_status scan_bf16(const gam_scan_args& p, int sms, cudaStream_t s) { return launch<bf16>(p, sms, s); }

}  // namespace ops
}  // namespace gam
