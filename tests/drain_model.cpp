// A model of barriers whose copies land late, for the counting in csrc/drain.cuh: random runs that stop at a
// wait which ran out, after which the drain has to wait for every copy in flight and for nothing else.
#include <cstdio>
#include <cstdlib>
#include <deque>

#include "drain.cuh"

// An mbarrier of one arrival a phase: a wait for parity P is over when the current phase's parity is not P.
struct Barrier {
  unsigned landed = 0, started = 0;
  bool done(unsigned parity) const { return (landed & 1u) != parity; }
};

static int failures = 0;
static void expect(bool ok, const char* what) {
  if (!ok && failures++ < 5) std::printf("%s\n", what);
}

// What the bounded wait on the abort path does: lets copies land until the phase is over. A phase that nothing
// in flight completes would run into the time limit.
static void drain_wait(Barrier& b, unsigned parity) {
  while (!b.done(parity)) {
    expect(b.landed < b.started, "drain waits for a phase that no copy completes");
    if (b.landed >= b.started) return;
    ++b.landed;
  }
}

// One barrier, a copy at a time.
static void lone(unsigned seed) {
  std::srand(seed);
  Barrier b;
  hbl::LoneCopies c;
  for (int left = std::rand() % 5; left > 0; --left) {
    ++b.started;
    c.start();
    bool gave_up = false;
    while (!b.done(c.parity()) && !gave_up) {
      if (std::rand() % 2) ++b.landed;
      else gave_up = std::rand() % 4 == 0;
    }
    if (gave_up) break;
    expect(b.landed == b.started, "a wait is over before its copy has landed");
  }
  c.drain([&](unsigned parity) { drain_wait(b, parity); });
  expect(b.landed == b.started, "a copy is in flight after the drain");
}

template <int N>
static void ring(unsigned seed) {
  std::srand(seed);
  Barrier bars[N];
  hbl::RingCopies<N> c;
  int next = 0;                       // stage of the next copy
  const int blocks = std::rand() % 40;  // copies in all
  int started = 0, used = 0;
  std::deque<int> flight;
  auto start = [&] {
    if (started == blocks) return;
    expect(bars[next].started == bars[next].landed, "a stage is filled while a copy lands in it");
    ++bars[next].started;
    flight.push_back(next);
    next = (next + 1) % N;
    ++started;
    c.start();
  };
  for (int i = 0; i < N; ++i) start();
  while (used < started) {
    if (std::rand() % 3 && !flight.empty()) {  // copies may land in any order
      const int i = std::rand() % (int)flight.size();
      ++bars[flight[i]].landed;
      flight.erase(flight.begin() + i);
    }
    if (!bars[c.stage].done(c.parity)) {
      if (std::rand() % 20 == 0) break;  // the wait runs out
      continue;
    }
    c.use();
    ++used;
    start();
  }
  c.drain([&](int s, unsigned parity) { drain_wait(bars[s], parity); });
  for (const Barrier& b : bars) expect(b.landed == b.started, "a copy is in flight after the drain");
  expect(c.ahead == 0, "copies left over");
}

int main() {
  for (unsigned seed = 0; seed < 20000; ++seed) {
    lone(seed);
    ring<1>(seed);
    ring<2>(seed);
    ring<3>(seed);
  }
  std::printf(failures ? "%d failures\n" : "ok\n", failures);
  return failures != 0;
}
