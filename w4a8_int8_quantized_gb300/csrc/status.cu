// Device-side error words.  Word 0 is shared by the kernels that contain bounded
// waits: a kernel whose wait gives up stores a nonzero code (which wait) there and
// returns.  Word 1 is where the cache kernels report an index out of its range:
// apart from the first, since it says less (the rest of that call is right) and must
// not hide a wait that gave up after it.  w8a8_check_status() reads and clears both.
#include <atomic>
#include <mutex>

#include "common.cuh"

namespace w8a8 {
namespace {
__device__ unsigned int g_device_error[2] = {0, 0};
std::atomic<long long> g_wait_limit{kTimeoutCycles};
std::atomic<int> g_skip_first_copy{0};
}

long long role_wait_limit() { return g_wait_limit.load(); }
bool skip_first_copy() { return g_skip_first_copy.load() != 0; }

unsigned int *device_error_word() {
  static unsigned int *cache[64] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == nullptr) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    cache[dev] = static_cast<unsigned int *>(p);
  }
  return cache[dev];
}

int read_and_clear_device_error(unsigned int *code) {
  *code = 0;
  unsigned int words[2] = {0, 0};
  if (cudaMemcpyFromSymbol(words, g_device_error, sizeof(words)) != cudaSuccess)
    return W8A8_ERR_CUDA;
  if (words[0] != 0 || words[1] != 0) {
    const unsigned int zero[2] = {0, 0};
    if (cudaMemcpyToSymbol(g_device_error, zero, sizeof(zero)) != cudaSuccess)
      return W8A8_ERR_CUDA;
  }
  *code = words[0] != 0 ? words[0] : words[1];
  return W8A8_OK;
}

}  // namespace w8a8

extern "C" int w8a8_test_set_fault(long long wait_limit_cycles, int skip_first_copy) {
  if (wait_limit_cycles < 0 || (skip_first_copy != 0 && skip_first_copy != 1))
    return W8A8_ERR_INVALID_ARG;
  w8a8::g_wait_limit.store(wait_limit_cycles == 0 ? w8a8::kTimeoutCycles : wait_limit_cycles);
  w8a8::g_skip_first_copy.store(skip_first_copy);
  return W8A8_OK;
}
