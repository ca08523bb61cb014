// What a launcher has asked of a device and need not ask again, by device ordinal: the
// devices of one process may hold different numbers of a kernel's clusters.
#pragma once

#include <atomic>

namespace kda {

template <int SIZES>
class DeviceCounts {
 public:
  // The count for `size` (below SIZES) on `device`; ask(&count) finds it, returning 0, the
  // first time. Ordinals past the table are asked every time, and errors are not kept.
  template <typename Ask>
  int get(int device, int size, int* count, Ask ask) {
    std::atomic<int>* slot = device >= 0 && device < kDevices ? &known_[device][size] : nullptr;
    if (slot != nullptr) {
      const int known = slot->load(std::memory_order_relaxed);
      if (known != 0) {
        *count = known - 1;
        return 0;
      }
    }
    const int error = ask(count);
    if (error == 0 && slot != nullptr) slot->store(*count + 1, std::memory_order_relaxed);
    return error;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices][SIZES] = {};  // the count + 1; 0: not asked
};

}  // namespace kda
