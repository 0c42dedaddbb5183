// Linear attention on the tensor cores, heads of 32 key channels.
#include "kda_linattn_tc.cuh"

namespace kda {

cudaError_t launch_linattn_tc_32(const LinPrefillArgs& a, const LinSched& sched, cudaStream_t s) {
  return a.dv == 32 ? run_tc<32, 32>(a, sched, s) : a.dv == 64 ? run_tc<32, 64>(a, sched, s) : run_tc<32, 128>(a, sched, s);
}
int read_and_clear_linattn_tc_32_errors(int* flags) { return read_and_clear_errors_here(flags); }

}  // namespace kda
