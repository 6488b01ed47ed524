// Workspaces prepared for the single pass (host only, no HIP): start address
// and size of each, under a lock. The single pass trusts the control words at
// the start of such a workspace, so nothing else of the library may write them.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <mutex>
#include <unordered_map>

namespace gla {

class Prepared {
 public:
  explicit Prepared(size_t ctrl_bytes) : ctrl_(ctrl_bytes) {}
  void add(const void* ws, size_t bytes) {
    std::lock_guard<std::mutex> lk(mu_);
    bytes_[addr(ws)] = bytes;
  }
  void remove(const void* ws) {
    std::lock_guard<std::mutex> lk(mu_);
    bytes_.erase(addr(ws));
  }
  // ws is the start of a prepared workspace.
  bool contains(const void* ws) const {
    std::lock_guard<std::mutex> lk(mu_);
    const auto it = bytes_.find(addr(ws));
    return it != bytes_.end() && it->second >= ctrl_;
  }
  // Some control word of a prepared workspace lies in [p, p + n).
  bool control_words_in(const void* p, size_t n) const {
    std::lock_guard<std::mutex> lk(mu_);
    for (const auto& e : bytes_)
      if (e.first < addr(p) + n && addr(p) < e.first + ctrl_) return true;
    return false;
  }

 private:
  static uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
  const size_t ctrl_;
  mutable std::mutex mu_;
  std::unordered_map<uintptr_t, size_t> bytes_;
};

}  // namespace gla
