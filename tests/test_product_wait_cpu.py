"""The products' bounded wait, run on the CPU with a clock of the test's own: it gives up when no
stage has been copied for the limit's time, however long it has lasted, and only then."""
import subprocess

from hyper_connection_mix_gb300 import build as hbuild

PROGRAM = r"""
#include <cstdio>
#include "hcmix_product.cuh"
using namespace hcmix::sublayer;

// What is waited for comes at `done`; a stage is copied every `every` cycles up to `until`; somebody
// gives up at `aborted`.  A look takes 1000 cycles.
static int64_t now, ended;
static int wait(int64_t done, int64_t every, int64_t until, int64_t aborted) {
  int abort = 0;
  uint32_t copied = 0;
  now = 0;
  const bool got = wait_while_moving(
      [&] {
        now += 1000;
        copied = (uint32_t)((now < until ? now : until) / every);
        abort = now >= aborted;
        return now >= done;
      },
      [&] { return now; }, &abort, &copied, kProductWait);
  ended = now;
  return got;
}

#define CHECK(what) \
  if (!(what)) return std::printf("%s: ended at %lld\n", #what, (long long)ended), 1

int main() {
  const int64_t most = kProductWait, never = 1000 * most;
  CHECK(wait(500, never, 0, never));
  CHECK(wait(most / 2, never, 0, never));
  // nothing moves: given up after the limit
  CHECK(!wait(never, never, 0, never) && ended > most && ended < most + most / 100);
  // a tile that takes fifty times the limit, copied a stage after the other
  CHECK(wait(50 * most, 4000, 50 * most, never));
  CHECK(wait(50 * most, most / 2, 50 * most, never));
  // stages that stop coming: given up after at most twice the limit from there
  CHECK(!wait(never, 4000, 10 * most, never) && ended >= 11 * most && ended <= 12 * most + most / 100);
  // another role's giving up ends it at once
  CHECK(!wait(never, 4000, never, 3 * most) && ended < 3 * most + most / 100);
  return 0;
}
"""


def test_a_wait_is_given_up_only_when_nothing_moves(tmp_path):
    source, program = tmp_path / "wait.cu", tmp_path / "wait"
    source.write_text(PROGRAM)
    subprocess.run([hbuild.nvcc(), *hbuild.ARCH, "-O2", "-std=c++17", "-I", hbuild.INCLUDE, "-I", hbuild.CSRC,
                    "-o", str(program), str(source)], check=True)
    run = subprocess.run([str(program)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
