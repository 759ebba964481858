// What a process asks each GPU once.
#pragma once
#include <atomic>
#include <mutex>

namespace gb300 {

// A value for each device, found by the first call that needs it and can find it.
template <typename T>
class PerDevice {
 public:
  // `ask` fills in a value and says whether it could; false: nothing is kept, the next call
  // asks again.
  template <typename Ask>
  bool get(int device, T* value, Ask ask) {
    Entry& e = entries_[device];
    if (!e.known.load(std::memory_order_acquire)) {
      const std::lock_guard<std::mutex> lock(mutex_);
      if (!e.known.load(std::memory_order_relaxed)) {
        T found{};
        if (!ask(&found)) return false;
        e.value = found;
        e.known.store(true, std::memory_order_release);
      }
    }
    *value = e.value;
    return true;
  }

 private:
  struct Entry {
    std::atomic<bool> known{false};
    T value{};
  };
  Entry entries_[64];  // as many devices as the library knows
  std::mutex mutex_;
};

}  // namespace gb300
