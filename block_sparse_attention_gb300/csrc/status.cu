// status.cu -- clearing bits of a device status word while other calls may set some, sm_103a.
#include "bsattn.h"
#include "host_internal.h"

namespace bsattn {
namespace {

__global__ void clear_bits_kernel(int* word, int bits) { atomicAnd(word, ~bits); }

}  // namespace

// Only the bits that the caller has read: one that a kernel on another stream has set since stays.  Where
// the stream is another device's than the word's a kernel on it may not reach the word; that word is set to
// 0 as a whole.
int clear_status_bits(void* word, int bits, cudaStream_t st) {
    cudaPointerAttributes at{};
    int current = 0, stream_device = 0;
    if (cudaGetDevice(&current) != cudaSuccess || cudaStreamGetDevice(st, &stream_device) != cudaSuccess ||
        cudaPointerGetAttributes(&at, word) != cudaSuccess)
        return BSATTN_ERR_CUDA;
    const bool device_memory = at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
    cudaError_t rc;
    if (!device_memory || at.device != stream_device) {
        rc = cudaMemsetAsync(word, 0, sizeof(int), st);
    } else {
        if (stream_device != current && cudaSetDevice(stream_device) != cudaSuccess) return BSATTN_ERR_CUDA;
        clear_bits_kernel<<<1, 1, 0, st>>>(static_cast<int*>(word), bits);
        rc = cudaGetLastError();
        if (stream_device != current) cudaSetDevice(current);
    }
    return rc == cudaSuccess && cudaStreamSynchronize(st) == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace bsattn
