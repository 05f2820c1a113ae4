// A bounded wait: looks that remain, and whether this one was the last.
#pragma once

#include <stdint.h>

namespace rl {

// One more look found what it waits for (`done`) or not.  True ends the wait,
// with `done` telling how; every caller acts on this one answer, so that a wait
// that ends has its result written.
constexpr bool wait_over(bool done, uint32_t& left) {
  if (done || left == 0) return true;
  --left;
  return false;
}

}  // namespace rl
