"""The waits in front of a kernel's end cover every copy in flight, whatever the order in which the
copies land: csrc/ring.h compiled for the host, against a model of the loading warp."""
import os
import subprocess

import block_sparse_long_branch_b200 as msa

PROGRAM = r"""
#include "ring.h"
#include <cstdio>
#include <cstdlib>
#include <vector>

// One warp fills a ring of `slots` tiles.  Each tile is of one of two kinds, each with its own
// `slots` barriers, used in turn.  A tile's slot is filled again only when its copy has landed and
// been read, so any of the last `slots` copies may be in flight when the warp stops.
struct Copy { int kind; uint32_t use; };

static long last_use(uint32_t uses, uint32_t bars, uint32_t bar) {  // by counting; -1: none
  long last = -1;
  for (uint32_t n = 0; n < uses; ++n)
    if (n % bars == bar) last = n;
  return last;
}

static int check(uint32_t slots, const std::vector<int>& kinds) {
  std::vector<Copy> copies;
  uint32_t uses[2] = {0, 0};
  for (int k : kinds) copies.push_back({k, uses[k]++});
  std::vector<long> waited[2] = {std::vector<long>(slots, -1), std::vector<long>(slots, -1)};
  for (int k = 0; k < 2; ++k)
    for (uint32_t i = 0; i < slots; ++i) {
      const uint32_t r = uses[k] + slots - 1 - i;
      if (r < slots) continue;
      const uint32_t bar = r % slots;
      const long last = last_use(uses[k], slots, bar);
      // a wait for another phase's parity would pass early, or never
      if (last < 0 || ((last / slots) & 1) != msa::ring_parity(r, slots) || waited[k][bar] >= 0) return 1;
      waited[k][bar] = last;
    }
  const size_t n = copies.size();
  for (size_t i = n > slots ? n - slots : 0; i < n; ++i) {
    const Copy& c = copies[i];
    if (waited[c.kind][c.use % slots] < (long)c.use) return 2;
  }
  // a ring of one kind, walked by slot and phase
  uint32_t slot = 0, phase = 0;
  for (size_t i = 0; i < n; ++i)
    if (++slot == slots) slot = 0, phase ^= 1;
  for (uint32_t i = 0; i < slots; ++i) {
    const long last = last_use(n, slots, i);
    if (msa::ring_last_parity(i, slot, phase) != (last < 0 ? 1 : ((last / slots) & 1))) return 3;
  }
  return 0;
}

int main() {
  srand(1);
  for (uint32_t slots = 1; slots <= 6; ++slots)
    for (int run = 0; run < 3000; ++run) {
      std::vector<int> kinds(rand() % 40);
      const int mostly = rand() % 4;
      for (int& k : kinds) k = mostly == 0 ? 0 : mostly == 1 ? rand() % 2 : mostly == 2 ? rand() % 8 == 0 : 1;
      if (int e = check(slots, kinds)) {
        printf("slots %u, %zu copies: %d\n", slots, kinds.size(), e);
        return 1;
      }
    }
  puts("ok");
}
"""


def test_every_copy_in_flight_is_waited_for(tmp_path):
    csrc = os.path.join(os.path.dirname(os.path.abspath(msa.__file__)), "csrc")
    src = tmp_path / "ring.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "ring"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout
