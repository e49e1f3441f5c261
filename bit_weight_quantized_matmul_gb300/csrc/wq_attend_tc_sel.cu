// wq_attend_tc_sel.cu -- the same (wq_attend_tc.cuh) for sinks and trees of drafted tokens.
//
// Measured on GB300: 2 x 1024 over 16384 behind a window of 2048 and 16 sinks, 32/8 heads of 128 (q4_0), 121 us (572 TFLOP/s of the
// visible pairs; 256 blocks of 18 or 19 tiles on 152 SMs); 32 trees of 20 .. 64 nodes over 2000 .. 16000 (NVFP4) 272 us, 822
// TFLOP/s, with their mask; one of 26 nodes over 60001 48 us and the join.
#include "wq_attend_tc.cuh"

namespace wq {

int attend_tc_sel(const AttendArgs& a, const AttendTcPlan& pl, cudaStream_t s) { return launch_tc<true>(a, pl, s); }

int take_status_attend_tc_sel() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
