// The selective scan's passes for bfloat16 storage.
#include "pn_ssm_scan.hpp"

namespace pn {
template hipError_t launch_ssm_pass<bf16>(const pn_ssm_args&, const SsmPlan&, SsmPass, hipStream_t);
}  // namespace pn
