// Host-side helpers shared by the C-ABI sources (h2o_api.cpp, pool_api.cpp):
// error reporting, the current stream, scratch memory and the error word.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

namespace h2o {
namespace host {

// Records the calling thread's error message and returns `code`.
int fail(int code, const std::string& msg);
int cuda_fail(cudaError_t e, const char* what);

// The calling thread's current PyTorch stream.
cudaStream_t current_stream();

// Memory from PyTorch's caching allocator; throws when there is none (or when
// h2o_test_fail_allocations asked for it).
void* device_alloc(size_t bytes, cudaStream_t s);
void device_free(void* p);

// One device allocation, freed on scope exit.
struct Scratch {
  void* p = nullptr;
  explicit Scratch(size_t bytes, cudaStream_t s) {
    if (bytes) p = device_alloc(bytes, s);
  }
  ~Scratch() {
    if (p) device_free(p);
  }
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Reads, then clears, a device error word on `s` after the stream's work so
// far; H2O_EDEVICE if it was set. Allocates nothing.
int check_error_word(int32_t* word_dev, cudaStream_t s);

}  // namespace host
}  // namespace h2o
