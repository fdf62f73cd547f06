// Which dynamic shared memory limits have been raised, per kernel and device: remembering it saves most of
// a microsecond per launch. (Only a cache of what the driver holds: an entry that another kernel has taken
// is looked up there.) A limit never sinks: between one thread's call and its launch another may ask for
// less of the same kernel. Host code without CUDA, so that it is tested without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

namespace lla {

class SmemLimits {
 public:
  static constexpr int kEntries = 256;
  static int slot(const void* kern, int dev) { return (int)((reinterpret_cast<uintptr_t>(kern) / 16 * 31 + dev) % kEntries); }
  // held(&bytes) reads the driver's limit, raise(bytes) sets it; both return 0 or an error.
  template <typename Held, typename Raise>
  auto ensure(const void* kern, int dev, size_t bytes, Held held, Raise raise) -> decltype(raise(bytes)) {
    Entry& e = table_[slot(kern, dev)];
    std::lock_guard<std::mutex> lk(mu_);
    if (e.kern == kern && e.dev == dev && e.bytes >= bytes) return {};
    size_t now = 0;
    auto err = held(&now);
    if (err) return err;
    if (now < bytes) {
      err = raise(bytes);
      if (err) return err;
      now = bytes;
    }
    e = {kern, dev, now};
    return {};
  }

 private:
  struct Entry {
    const void* kern;
    int dev;
    size_t bytes;
  };
  std::mutex mu_;
  Entry table_[kEntries] = {};
};

}  // namespace lla
