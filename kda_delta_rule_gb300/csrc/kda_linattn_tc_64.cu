// Linear attention on the tensor cores, heads of 64 key channels.
#include "kda_linattn_tc.cuh"

namespace kda {

cudaError_t launch_linattn_tc_64(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s) {
  return a.dv == 32 ? run_tc<64, 32>(a, sched, s) : a.dv == 64 ? run_tc<64, 64>(a, sched, s) : run_tc<64, 128>(a, sched, s);
}
int read_and_clear_linattn_tc_64_errors(int* flags) { return read_and_clear_errors_here(flags); }

}  // namespace kda
