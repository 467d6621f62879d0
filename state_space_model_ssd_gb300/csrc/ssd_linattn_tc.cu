#include "linattn.cuh"
namespace ssd {
namespace linattn {
bool tc_fits(const Pass&) { return false; }
cudaError_t tc_sums(const WalkArgs&, Launch&) { return cudaErrorNotSupported; }
cudaError_t tc_walk(const WalkArgs&, Launch&) { return cudaErrorNotSupported; }
}  // namespace linattn
}  // namespace ssd
