"""The cross attention's ring of key and value tiles, from the header that the
kernel takes it from: a wait for a fill is told by its parity alone, so the
slot's fill before it has to be one that the waiter has itself waited for."""
import os
import shutil
import subprocess

import pytest

from bit_diffusion_transformer_nvfp4_b200 import build

# per form: slots and rings as cross_attention.cuh has them
FORMS = {"split, 64 columns": (12, 2), "split, 128 columns": (6, 2), "persistent, 64 columns": (8, 1),
         "persistent, 128 columns": (4, 1)}

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "xattn_ring.h"
int main(int argc, char** argv) {
  const unsigned slots = std::atoi(argv[1]), rings = std::atoi(argv[2]);
  for (unsigned t = 0; t < rings; ++t) {
    const w4a4::XRing r = w4a4::xattn_ring(slots, rings, t);
    for (unsigned k = 0; k < 100; ++k)
      for (unsigned fill : {w4a4::xattn_fill_k(k), w4a4::xattn_fill_v(k)})
        std::printf("%u %u %u %u\\n", t, fill, r.slot(fill), r.parity(fill));
  }
}
"""


def unsure_waits(waits):
    """(sequence, fill) of the waits whose slot's fill before was not waited
    for by the same sequence.  waits: per sequence, (fill, slot, parity) in
    the order in which it waits; fills of a slot are numbered over all."""
    by_slot = {}
    for t, w in waits.items():
        for fill, slot, parity in w:
            by_slot.setdefault(slot, []).append((fill, t, parity))
    bad = []
    for users in by_slot.values():
        users.sort()
        for i, (fill, t, parity) in enumerate(users):
            assert parity == i & 1, (fill, t)       # the barrier's own phase
            if i > 0 and users[i - 1][1] != t:
                bad.append((t, fill))
    return bad


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a C++ compiler")
@pytest.mark.parametrize("form", FORMS)
def test_every_wait_knows_the_fill_before(tmp_path, form):
    src, exe = tmp_path / "ring.cc", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    slots, rings = FORMS[form]
    out = subprocess.run([str(exe), str(slots), str(rings)], check=True, capture_output=True, text=True).stdout
    waits = {}
    for line in out.splitlines():
        t, fill, slot, parity = map(int, line.split())
        assert 0 <= slot < slots
        waits.setdefault(t, []).append((fill, slot, parity))
    assert len(waits) == rings and unsure_waits(waits) == []
    for w in waits.values():
        assert [fill for fill, _, _ in w] == list(range(200))  # each fill once, in turn
    # every slot is used
    assert len({slot for w in waits.values() for _, slot, _ in w}) == slots


def test_one_ring_for_two_streams_would_not_do():
    """Fills K0 K1 V0 K2 V1 K3 ... of six slots, every second tile a stream's:
    values wait behind the other stream's."""
    waits = {0: [], 1: []}
    for i in range(50):
        for fill in ((0 if i == 0 else 2 * i - 1), 2 * i + 2):
            waits[i & 1].append((fill, fill % 6, fill // 6 & 1))
    assert (1, 8) in unsure_waits(waits)


def test_the_kernel_has_these_rings():
    with open(os.path.join(build.CSRC, "cross_attention.cuh")) as f:
        text = f.read()
    assert "SLOTS = (SPLIT ? 12 : 8) / DB;" in text and "RINGS = SPLIT ? 2 : 1;" in text
