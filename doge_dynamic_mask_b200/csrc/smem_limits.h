// Dynamic shared-memory limits that kernels were granted, per (kernel, device).
#pragma once

#include <map>
#include <mutex>
#include <utility>

namespace dma {

// A kernel's limit only grows: a launch that was promised its bytes must find them,
// whatever smaller launch another thread prepares in between.
class SmemLimits {
 public:
  // Makes sure that `func` may use `bytes` on device `dev`: calls set(), whose 0 means
  // success, unless as much or more was granted before.  Returns what set() returned.
  template <class Set>
  int raise(const void* func, int dev, int bytes, Set&& set) {
    std::lock_guard<std::mutex> lock(mu_);
    int& have = granted_[{func, dev}];
    if (have >= bytes) return 0;
    const int e = set();
    if (e == 0) have = bytes;
    return e;
  }

 private:
  std::mutex mu_;
  std::map<std::pair<const void*, int>, int> granted_;
};

}  // namespace dma
