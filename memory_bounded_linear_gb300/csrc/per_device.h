// A number that is asked of each device once per process (host code).
#pragma once

#include <atomic>

namespace lce {

// Threads may ask at the same time; where two find no answer yet, both ask and keep the same one.  A
// query that fails is not kept: it is reported, and the next call asks again.
template <int DEVICES>
class PerDevice {
 public:
  // *value of device dev (0 .. DEVICES - 1), by query(value), which returns 0 or an error code.
  template <typename Query>
  auto get(int dev, Query&& query, int* value) -> decltype(query(value)) {
    if (known_[dev].load(std::memory_order_acquire)) {
      *value = value_[dev].load(std::memory_order_relaxed);
      return {};
    }
    const auto error = query(value);
    if (error == decltype(query(value)){}) {
      value_[dev].store(*value, std::memory_order_relaxed);
      known_[dev].store(true, std::memory_order_release);
    }
    return error;
  }

 private:
  std::atomic<int> value_[DEVICES] = {};
  std::atomic<bool> known_[DEVICES] = {};
};

}  // namespace lce
