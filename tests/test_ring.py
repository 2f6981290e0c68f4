"""The ring of the product's copies (csrc/ring.h) on the host: where copies go, and what is waited for at its end."""
import subprocess
from pathlib import Path

CSRC = Path(__file__).resolve().parent.parent / "streaming_selection_primitive_gb300" / "csrc"

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "ring.h"

using profk::RingPlace;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s, %d stages, %d copies, %d used\n", __LINE__, #x, stages, copies, used); std::exit(1); } } while (0)

// A barrier of one arrival a phase: a wait for a parity is over once the phase of that parity is.
struct Barrier {
  int phases = 0;
  bool over(unsigned parity) const { return (phases & 1) != static_cast<int>(parity); }
};

int main() {
  for (int stages = 1; stages <= 6; ++stages)
    for (int copies = 0; copies <= 3 * stages + 1; ++copies)
      for (int used = copies > stages ? copies - stages : 0; used <= copies; ++used) {
        // `copies` have been issued, the products of the first `used` of them are done.
        std::vector<Barrier> full(stages), empty(stages);
        RingPlace at;
        std::vector<RingPlace> places;
        int issued = 0;
        for (int i = 0; i < copies; ++i) {
          CHECK(at.stage == i % stages && at.full() == static_cast<unsigned>(i / stages % 2));
          if (i - stages >= 0) {
            if (i - stages < used) ++empty[at.stage].phases;
            full[at.stage].phases = i / stages;  // (the copy before has arrived)
          }
          CHECK(i < stages || empty[at.stage].over(at.empty()));
          places.push_back(at);
          issued = issued < stages ? issued + 1 : stages;
          at.next(stages);
        }
        for (int i = copies > stages ? copies - stages : 0; i < copies; ++i)
          if (i < used) ++empty[i % stages].phases;
        std::vector<RingPlace> waited;
        bool gave_up = false;
        profk::leave_ring(
            at, issued, stages,
            [&](RingPlace p) {
              const bool over = empty[p.stage].over(p.empty());
              gave_up |= !over;
              return over;
            },
            [&](RingPlace p) { waited.push_back(p); });
        CHECK(gave_up == (used < copies));
        // All used: no copy is on its way.  Else the last one to each stage is waited for, by its own phase.
        CHECK(static_cast<int>(waited.size()) == (used < copies ? issued : 0));
        for (size_t i = 0; i < waited.size(); ++i) {
          const RingPlace want = places[copies - 1 - i];
          CHECK(waited[i].stage == want.stage && waited[i].full() == want.full());
          Barrier& b = full[want.stage];
          b.phases = (copies - 1 - static_cast<int>(i)) / stages;
          CHECK(!b.over(waited[i].full()));  // while the copy is on its way
          ++b.phases;
          CHECK(b.over(waited[i].full()));
        }
      }
  return 0;
}
"""


def test_places_and_the_end_of_the_ring(tmp_path):
    (tmp_path / "ring.cpp").write_text(PROGRAM)
    built = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", str(CSRC), str(tmp_path / "ring.cpp"), "-o", str(tmp_path / "ring")],
                           capture_output=True, text=True)
    assert built.returncode == 0, built.stderr
    ran = subprocess.run([str(tmp_path / "ring")], capture_output=True, text=True)
    assert ran.returncode == 0, ran.stdout
