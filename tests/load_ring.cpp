// A loader and a consumer over LoadRing with barriers that are modelled: an arrival
// count, outstanding bytes, phases; copies land when the random numbers say so.  From
// some step on waits may give up, the loader's and the consumer's, as they do after a
// timeout anywhere in a launch.  Exit status: 0 = every copy was armed on a phase of
// its own and had landed when the loader left, 1 = not, 2 = the model itself is off.
// With CARRY_ON the loader copies on after a wait that gave up.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "load_ring.cuh"

namespace {

struct Bar {                   // as an mbarrier of one arrival a phase
  int pending = 1, tx = 0;
  uint32_t phase = 0;
  bool bad = false;
  void turn() {
    if (pending == 0 && tx == 0) {
      pending = 1;
      phase ^= 1u;
    }
  }
  void arrive_expect(int bytes) {
    if (pending == 0) bad = true;              // the count underflows
    tx += bytes;
    --pending;
    turn();
  }
  void arrive() {
    if (pending == 0) bad = true;
    --pending;
    turn();
  }
  void land(int bytes) {
    tx -= bytes;
    turn();
  }
  bool done(uint32_t parity) const { return phase != parity; }
};

template <int N>
int run(unsigned seed, int items, int fails_at) {
  std::mt19937 rng(seed);
  auto chance = [&](int of) { return (int)(rng() % (unsigned)of) == 0; };
  Bar full[N], empty[N];
  struct Flight {
    int stage, bytes;
  };
  std::vector<Flight> flight;
  int used = 0, clock = 0;     // the consumer's: stages used
  bool timeout = false;
  auto tick = [&] {            // a little time passes
    ++clock;
    if (!flight.empty() && chance(3)) {
      const size_t i = rng() % flight.size();
      full[flight[i].stage].land(flight[i].bytes);
      flight.erase(flight.begin() + i);
    }
    // the consumer, unless it hangs: waits for the next stage and frees it
    const bool gone = fails_at >= 0 && clock >= fails_at;
    if (gone && clock >= fails_at + 50) timeout = true;          // its own wait gave up
    const int s = used % N;
    if (!gone && chance(2) && full[s].done((uint32_t)(used / N) & 1u)) {
      empty[s].arrive();
      ++used;
    }
  };
  auto wait = [&](Bar& b, uint32_t parity) {
    for (int i = 0; i < (timeout ? 3 : 400); ++i) {
      if (b.done(parity)) return true;
      tick();
    }
    timeout = true;
    return false;
  };
  msa::LoadRing<N> lr;
  int issued = 0;
  for (int k = 0; k < items; ++k) {
    const bool ok = lr.free([&](int s, uint32_t par) { return wait(empty[s], par); });
#ifdef CARRY_ON
    lr.going = true;
#else
    if (!ok) break;
#endif
    (void)ok;
    const int bytes = 16 * (1 + (int)(rng() % 8));
    if (chance(9)) {                           // a page that is not there
      full[lr.stage].arrive();
    } else {
      full[lr.stage].arrive_expect(bytes);
      flight.push_back({lr.stage, bytes});
    }
    lr.armed();
    ++issued;
  }
  if (!timeout && issued != items) return 2;
  // without a timeout the consumer waits for what was issued; with one the loader does
  while (!timeout && used < issued) tick();
  if (timeout)
    lr.drain([&](int s, uint32_t par) {
      for (int i = 0; i < 100000 && !full[s].done(par); ++i) tick();
    });
  for (const Bar& b : full)
    if (b.bad) return 1;
  return flight.empty() ? 0 : 1;
}

template <int N>
int all() {
  for (unsigned seed = 0; seed < 3000; ++seed) {
    const int items = (int)(seed % 41);
    for (int fails : {-1, (int)(seed % 97), 300}) {
      const int st = run<N>(seed, items, fails);
      if (st) {
        std::printf("N %d seed %u items %d fails at %d: %d\n", N, seed, items, fails, st);
        return st;
      }
    }
  }
  return 0;
}

}  // namespace

int main() {
  int st;
  if ((st = all<1>()) || (st = all<2>()) || (st = all<3>()) || (st = all<8>())) return st;
  return 0;
}
