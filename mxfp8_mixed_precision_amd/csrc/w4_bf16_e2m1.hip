#include "w4_core.h"

namespace temx {

te_status launch_w4_bf16_e2m1(const W4Params& p, hipStream_t stream) { return w4_run<bf16_t, TE_W4_E2M1>(p, stream); }

}  // namespace temx
