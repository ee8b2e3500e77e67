"""Which copy a leaving CTA waits for on each slot of the K/V ring (host build
of the kernels' own function).  Waiting for an earlier item of a slot than the
last one issued would either miss a copy in flight or, two phases on, wait for
a phase that never comes."""

import subprocess

import numpy as np
import pytest

from paged_kv_cache_222_gb300 import build as B

HARNESS = r"""
#include <cstdio>
#include "pkv_internal.h"
int main() {
  int slots, next_k, next_v;
  while (std::scanf("%d %d %d", &slots, &next_k, &next_v) == 3) {
    for (int s = 0; s < slots; ++s) std::printf("%d ", pkv::ring_last_item(s, slots, next_k, next_v));
    std::printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def last_items(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cu").write_text(HARNESS)
    subprocess.run([B.nvcc(), "-std=c++17", "-I", B.CSRC, "-I", B.INCLUDE, str(d / "ring.cu"), "-o", str(d / "ring")],
                   check=True, capture_output=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "ring")], input=text, check=True, capture_output=True, text=True).stdout
        return [[int(x) for x in line.split()] for line in out.splitlines()]
    return ask


def test_last_item_of_every_slot(last_items):
    # two loaders that issue items 0, 2, 4, ... and 1, 3, 5, ... in any order
    # the ring allows: item i once item i - slots has been issued (and read)
    rng = np.random.default_rng(1)
    cases, want = [], []
    for slots in (3, 4, 6, 8):
        for _ in range(40):
            issued, nxt = [-1] * slots, [0, 1]
            done = set()
            for _ in range(int(rng.integers(0, 60))):
                v = int(rng.integers(0, 2))
                i = nxt[v]
                if i >= slots and i - slots not in done:
                    continue
                done.add(i)
                issued[i % slots] = i
                nxt[v] += 2
                cases.append((slots, *nxt))
                want.append(list(issued))
            cases.append((slots, *nxt))
            want.append(list(issued))
    assert last_items(cases) == want
