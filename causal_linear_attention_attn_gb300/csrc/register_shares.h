// Whether a kernel's register shares by role (setmaxnreg) fit what it is launched with.
//
// A warpgroup that raises its share draws on the registers the block was launched with.  The compiler
// decides how many those are, so a kernel whose shares add up to `share` a thread may run only where the
// compiled code is given that many: with fewer, the raise would wait forever.  Plain C++: no CUDA headers,
// so that the rule can be unit-tested on a machine without a GPU.
#pragma once

#include <mutex>
#include <utility>
#include <vector>

namespace la {

// Registers are given out to a warp in units of 256, eight a thread.
constexpr int allocated_registers(int used) { return (used + 7) / 8 * 8; }

// The answer per device.  query() gives the compiled kernel's registers a thread, or a negative number when
// it could not be found out; that answer is no, and is not kept.
class RegisterShares {
 public:
  template <typename Query>
  bool fit(int dev, int share, Query &&query) {
    std::lock_guard<std::mutex> lk(mu_);
    for (const std::pair<int, bool> &e : known_)
      if (e.first == dev) return e.second;
    const int used = query();
    if (used < 0) return false;
    known_.emplace_back(dev, allocated_registers(used) >= share);
    return known_.back().second;
  }

 private:
  std::mutex mu_;
  std::vector<std::pair<int, bool>> known_;
};

}  // namespace la
