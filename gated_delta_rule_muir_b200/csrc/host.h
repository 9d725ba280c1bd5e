// Host-side services that the translation units of libmuir.so share: the calling
// thread's error message and the launch accounting live in muir.cu; each unit has
// its own copy of the device status word, and muir_device_status() joins them.
#pragma once

#include <cuda_runtime.h>

namespace muir_host {

void clear_error();
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int check_launch(const char* what);  // cudaGetLastError() -> MUIR_OK or MUIR_ERR_CUDA
void* launch_begin(const char* name, cudaStream_t s);
void launch_end(void* event, cudaStream_t s);

// Brackets one kernel launch on stream s (construct right before the launch).
struct LaunchScope {
  cudaStream_t s;
  void* e;
  LaunchScope(const char* name, cudaStream_t st) : s(st), e(launch_begin(name, st)) {}
  ~LaunchScope() { launch_end(e, s); }
};

// Reads and clears layer.cu's device status word; false if a copy failed.
bool take_layer_status(unsigned int* word);

}  // namespace muir_host
