// Selective state-space scan: calls in f16.
#include "selective_scan.cuh"

namespace gam {
namespace ops {

gam_status scan_f16(const gam_scan_args& p, int sms, cudaStream_t s) { return launch<__half>(p, sms, s); }

}  // namespace ops
}  // namespace gam
