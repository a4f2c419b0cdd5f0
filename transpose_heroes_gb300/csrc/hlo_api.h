// Host-side helpers of the C-ABI entry points, shared by hlo_api.cu (which defines them) and
// layer_api.cu: the thread's last error, fault injection and the checks of quantization parameters.
#pragma once
#include "hlo_fusion.h"
#include "hlo_internal.h"

namespace hlo {

hlo_status api_fail(hlo_status s, const char* fmt, ...);
hlo_status api_ok();
hlo_status api_cuda_status(cudaError_t e, const char* what);
bool api_injected(const char* site);
hlo_status api_check_quant(const hlo_quant* q, const hlo_array& a, const char* what, QuantParams* out);

}  // namespace hlo
