// A limit that is raised when a call needs more and never lowered, by any number
// of threads.
#pragma once

#include <atomic>
#include <mutex>

namespace qz {

class GrowLimit {
 public:
  // Makes the limit at least `want`: set(value) sets it and answers 0, or an error,
  // after which the limit counts as what it was.  The look, the set and the note are one
  // step: a smaller value set beside a larger one would stay behind the larger one's note.
  template <class Set>
  int ensure(int want, Set &&set) {
    if (now_.load(std::memory_order_acquire) >= want) return 0;
    const std::lock_guard<std::mutex> one(m_);
    if (now_.load(std::memory_order_relaxed) >= want) return 0;
    const int e = set(want);
    if (e == 0) now_.store(want, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<int> now_{0};
  std::mutex m_;
};

}  // namespace qz
