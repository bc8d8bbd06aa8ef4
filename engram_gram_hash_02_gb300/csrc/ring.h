// Phases of a ring of barriers whose places are requested in turn. Plain C++ (host and device), so that a host program can
// check it.
#pragma once

#include "fastdiv.h"

namespace engram {

// The parity of place s's last request, where place `at` is requested next, in a round of parity `phase` (0 in the first one).
// For a place that was never requested it is that of the phase before a barrier's first, which counts as complete.
ENGRAM_HD uint32_t last_request(int s, int at, uint32_t phase) { return s < at ? phase : phase ^ 1u; }

}  // namespace engram
