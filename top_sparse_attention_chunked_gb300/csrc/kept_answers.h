// What a query of the device answered, kept for the life of the process (host code only).
#pragma once

#include <mutex>

namespace dsa {

// A slot's answer (>= 0) is asked for until the query succeeds, and then kept. One that fails
// answers 0 for this call alone: what made it fail may be gone by the next.
template <int SLOTS>
class KeptAnswers {
 public:
  // ask(int* answer): whether the query succeeded
  template <class F>
  int get(int slot, F&& ask) {
    std::lock_guard<std::mutex> lock(mu_);
    if (kept_[slot]) return kept_[slot] - 1;
    int n = 0;
    if (!ask(&n)) return 0;
    kept_[slot] = n + 1;
    return n;
  }

 private:
  std::mutex mu_;
  int kept_[SLOTS] = {};   // and 1; 0: none yet
};

}  // namespace dsa
