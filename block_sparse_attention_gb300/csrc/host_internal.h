// host_internal.h -- helpers shared by the launchers (not part of the C ABI).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace bsattn {

// Budget of every bounded device wait, set by bsattn_set_wait_budget_ns.
unsigned long long wait_budget_ns();

// Where a paged-serving call records what its kernel finds: the word that this thread has set with
// bsattn_set_status_word, else the one at the start of the call's workspace.
int* status_word(void* workspace);

// Encodes a 3-D tiled TMA descriptor over 16-bit elements (bf16 if `bf16`, else fp16):
// dims {dim0 (innermost), dim1, dim2}, byte strides of dims 1 and 2, box {box0, box1, box2},
// optional 128-byte swizzle, zero fill out of bounds.  Returns a bsattn_status.
int encode_3d(CUtensorMap* map, const void* base, int bf16, uint64_t dim0, uint64_t dim1,
              uint64_t dim2, uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box0,
              uint32_t box1, uint32_t box2, bool swizzle128);

// The same with four dimensions, byte strides of dims 1-3, and the 128-byte swizzle.
int encode_4d(CUtensorMap* map, const void* base, int bf16, const uint64_t (&dims)[4],
              const uint64_t (&stride_bytes)[3], const uint32_t (&box)[4]);

// Clears `bits` of a device status word and synchronises the stream (status.cu).  Returns a bsattn_status.
int clear_status_bits(void* word, int bits, cudaStream_t st);

// SM count of the current device (0 if it cannot be queried).
int num_sms_of_current_device();

// Raises a kernel's dynamic shared memory limit to `bytes` on the current device, once for each device
// (`done` is the kernel's own record: a bit a device).  Returns a bsattn_status.
int raise_smem_limit(const void* kernel, int bytes, std::atomic<unsigned long long>& done);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether na bytes at a and nb bytes at b share any.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// The 128-row prefill for a 128-token block mask (prefill128.cu).  Arguments are checked by the
// caller; returns BSATTN_ERR_UNSUPPORTED when the mask rows do not fit its shared memory.
int prefill128_launch(const void* q, const void* k, const void* v, const uint8_t* block_mask,
                      int is_causal, void* out, int B, int H, int Sq, int Sk, int d, bool bf16,
                      void* workspace, cudaStream_t stream);

}  // namespace bsattn
