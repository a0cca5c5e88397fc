// linear_tc.cu -- the linear-attention scan on tensor cores: no shape is served yet.
#include "../linear.h"
namespace ssd {
bool scan_tc_supported(const ScanRole&, const ScanPlan&, bool) { return false; }
cudaError_t launch_scan_tc(const ScanLaunch&, bool, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace ssd
