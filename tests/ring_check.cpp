// Host check of the phases of a ring of barriers (csrc/ring.h): after any number of requests, a wait for a place's last one ends
// when that one is complete, not before, and at once for a place that was never requested.
#include <stdio.h>

#include "ring.h"

// A barrier's phases, told apart by parity: complete(p) is whether the phase of parity p is over, phase 0 being the first
struct Barrier {
  int phases = 0;
  bool over(uint32_t parity) const { return ((uint32_t)phases & 1u) != parity; }
};

int main() {
  for (int places = 1; places <= 5; ++places)
    for (int requests = 0; requests <= 4 * places + 1; ++requests)
      for (int pending = 0; pending <= requests && pending <= places; ++pending) {
        Barrier b[5];
        int at = 0;
        uint32_t phase = 0;
        for (int r = 0; r < requests; ++r) {
          if (r < requests - pending) ++b[at].phases;      // complete: the place may be requested again
          if (++at == places) { at = 0; phase ^= 1u; }
        }
        for (int s = 0; s < places; ++s) {
          bool open = false;                              // place s has a request under way
          for (int r = requests - pending; r < requests; ++r) open |= r % places == s;
          if (b[s].over(engram::last_request(s, at, phase)) == open) {
            printf("%d places, %d requests, %d under way: place %d\n", places, requests, pending, s);
            return 1;
          }
        }
      }
  printf("ok\n");
  return 0;
}
