// Host-side check of the drain of a ring of copies after an abort: the barriers
// are modelled as counts of completed phases, a wait on parity P passes when the
// current phase's parity differs from P (the mbarrier rule), and one that has
// nothing in flight to wait for would run out.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "ring_drain.cuh"

struct Ring {
  int slots, owners, period;                 // fill f belongs to owner (f % period) * owners / period
  std::vector<int> next;                     // next fill of each owner
  std::vector<int64_t> done;                 // completed phases a slot
  std::vector<int> flight;                   // the fill in flight in a slot, or -1
  int used = 0;                              // fills consumed, in order
  int owner(int f) const { return f % period * owners / period; }
  int after(int f) const {                   // the owner's fill behind f
    int g = f + 1;
    while (owner(g) != owner(f)) ++g;
    return g;
  }
};

static int waits, late;

// `lands`: percentage of steps in which a copy lands
static void run(int slots, int owners, int period, int steps, int lands) {
  Ring r{slots, owners, period};
  r.done.assign(slots, 0);
  r.flight.assign(slots, -1);
  for (int o = 0; o < owners; ++o) {
    int f = 0;
    while (r.owner(f) != o) ++f;
    r.next.push_back(f);
  }
  for (int s = 0; s < steps; ++s) {
    const int x = rand() % 3;
    if (x == 0) {                            // an owner issues its next fill, if its slot is free
      int& f = r.next[rand() % owners];
      if (f < r.used + slots) {
        r.flight[f % slots] = f;
        f = r.after(f);
      }
    } else if (x == 1) {                     // a copy lands
      const int slot = rand() % slots;
      if (rand() % 100 < lands && r.flight[slot] >= 0) { r.flight[slot] = -1; ++r.done[slot]; }
    } else {                                 // the consumer uses the next fill, if it has landed
      if (r.done[r.used % slots] > r.used / slots) ++r.used;
    }
  }
  // the abort: every owner knows the position behind its last fill
  std::vector<int> ends(owners, 0);
  int end = 0;
  for (int o = 0; o < owners; ++o) {
    for (int f = 0; f < r.next[o]; ++f)
      if (r.owner(f) == o) ends[o] = f + 1;
    end = std::max(end, ends[o]);
  }
  mla::drain_ring(end, slots, [&](int f) { return f < ends[r.owner(f)]; },
                  [&](int slot, uint32_t parity) {
                    ++waits;
                    if ((uint32_t)(r.done[slot] & 1) != parity) return;       // passed already
                    if (r.flight[slot] < 0) { ++late; return; }               // would run out
                    r.flight[slot] = -1;
                    ++r.done[slot];
                  });
  for (int slot = 0; slot < slots; ++slot)
    if (r.flight[slot] >= 0) {
      printf("slots %d owners %d: fill %d still in flight\n", slots, owners, r.flight[slot]);
      exit(1);
    }
}

int main() {
  srand(1);
  const int shapes[][3] = {{8, 2, 4}, {11, 2, 4}, {2, 1, 1}, {1, 1, 1}, {10, 1, 1}, {5, 2, 4}};
  for (const auto& s : shapes)
    for (int i = 0; i < 4000; ++i) run(s[0], s[1], s[2], rand() % 400, i % 3 * 50);
  if (late) { printf("%d waits without a copy\n", late); return 1; }
  printf("ok %d waits\n", waits);
  return 0;
}
