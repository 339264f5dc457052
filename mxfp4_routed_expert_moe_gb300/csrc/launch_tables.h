// launch_tables.h — what launch code asks the driver once per kernel and keeps.
// Host code without CUDA types: calls may come from several threads.
#pragma once

#include <stddef.h>

#include <mutex>

namespace moe {

// The dynamic shared memory that a kernel may use.  A smaller size never
// replaces a larger one: a kernel whose size goes with its arguments (sampling)
// is asked for both at the same time by two threads, and the attribute is what
// was set last.
class SmemTable {
 public:
  // set(kernel, bytes) -> 0 or an error, which is returned.
  template <typename Set>
  int ensure(const void* kernel, size_t bytes, Set set) {
    std::lock_guard<std::mutex> lock(mutex_);
    Entry* e = nullptr;
    for (int i = 0; i < n_ && !e; ++i)
      if (entry_[i].kernel == kernel) e = &entry_[i];
    if (e && e->bytes >= bytes) return 0;
    const int err = set(kernel, bytes);
    if (err) return err;
    if (!e && n_ < kMost) {
      e = &entry_[n_++];
      e->kernel = kernel;
    }
    if (e) e->bytes = bytes;
    return 0;
  }

 private:
  static constexpr int kMost = 64;  // more than the library has kernels
  struct Entry {
    const void* kernel;
    size_t bytes;
  };
  std::mutex mutex_;
  Entry entry_[kMost];
  int n_ = 0;
};

// CTAs of a kernel that fit an SM, by threads and dynamic shared memory.
class OccupancyTable {
 public:
  // ask(kernel, threads, smem, &ctas) -> 0 or an error, which is returned.
  template <typename Ask>
  int get(const void* kernel, int threads, size_t smem, int* out, Ask ask) {
    std::lock_guard<std::mutex> lock(mutex_);
    for (int i = 0; i < n_; ++i)
      if (entry_[i].kernel == kernel && entry_[i].threads == threads && entry_[i].smem == smem) {
        *out = entry_[i].ctas;
        return 0;
      }
    int ctas = 0;
    const int err = ask(kernel, threads, smem, &ctas);
    if (err) return err;
    if (ctas < 1) ctas = 1;
    if (n_ < kMost) entry_[n_++] = {kernel, threads, smem, ctas};
    *out = ctas;
    return 0;
  }

 private:
  static constexpr int kMost = 64;
  struct Entry {
    const void* kernel;
    int threads;
    size_t smem;
    int ctas;
  };
  std::mutex mutex_;
  Entry entry_[kMost];
  int n_ = 0;
};

}  // namespace moe
