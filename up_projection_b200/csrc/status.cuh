// status.cuh -- a kernel file's device status word, read by the host.
#pragma once

#include <cuda_runtime.h>

namespace swiglu {

// The word, once the stream's earlier work is done; cleared if it is set.  (A
// clear word is not written: 11 words take swiglu_sync_status 136 us, with a
// write and its wait for each 188.)
template <typename Word>
cudaError_t fetch_and_clear(const Word &word, unsigned int *host_out, cudaStream_t stream) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(host_out, word, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess || *host_out == 0) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbolAsync(word, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(stream);
}

}  // namespace swiglu
