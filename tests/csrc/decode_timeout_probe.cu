// decode_timeout_probe.cu -- test-only library: the decode-side calls with a limit, set by the test, on the tries that a
// helper warp of single-token attention makes before it gives up. A run of ordinary length exceeds a small one. The launch
// then ends early, by the same way as after a wait that ran out: status word, abort flag, copies in flight awaited. Nothing
// faults or hangs: every other wait sees the flag.
#include <cuda_runtime.h>

__device__ int idle_tries = 1 << 24;
#define SEGPAGED_DECODE_IDLE_TRIES idle_tries
#define SEGPAGED_DECODE_IDLE_CHECK 4
#include "../../head_sparse_paged_b200/csrc/segpaged_decode.cu"

extern "C" int segpaged_test_set_idle_tries(int n) {
  return cudaMemcpyToSymbol(idle_tries, &n, sizeof(n)) == cudaSuccess ? 0 : -1;
}
