"""How the expert kernels walk a row of weights (chunk_of and stretch_of in csrc/moe.hpp, compiled
for the host; the loops are those of Products::run in csrc/moe_impl.hpp): every slot is taken once,
and every round of loads starts at an even slot, since its scales are one load of whole words."""
import ctypes
import itertools
import subprocess

import pytest

from bit_affine_quantized_qmv_amd import build

ENTRIES = 40 * 1024 // 16            # 16-byte words of the staged activations

SOURCE = """
#include "moe.hpp"
extern "C" int chunk_of(int slot_entries, int xrl, int round) { return qmm::moe::chunk_of(slot_entries, xrl, round); }
extern "C" int stretch_of(int n, int parts) { return qmm::moe::stretch_of(n, parts); }
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("walk")
    (d / "walk.hip").write_text(SOURCE)
    cmd = [build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", build.CSRC,
           str(d / "walk.hip"), "-o", str(d / "walk.so")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return ctypes.CDLL(str(d / "walk.so"))


def geometry(bits, group):
    """Span of a slot in K, slots of the ring, 16-byte entries of a slot per row (Slot, Stream)."""
    span = 64 if bits == 8 and group == 64 else 128
    words = 4 * (1 if bits == 4 else span // 64) if bits in (4, 8) else 2 * (span // 32)
    depth = 4 if words <= 4 and span // group < 4 else 2
    return span, depth, span // 32 * 4


@pytest.mark.parametrize("bits,group", itertools.product((2, 3, 4, 5, 6, 8), (32, 64, 128)))
@pytest.mark.parametrize("planes", [1, 2])
def test_rounds_start_even_and_take_every_slot_once(walk, bits, group, planes):
    span, depth, entries = geometry(bits, group)
    for k, splits, xrl, parts in itertools.product((64, 128, 640, 1024, 2048, 2176, 6208, 14336), (1, 2, 3), range(5),
                                                   (1, 2, 4)):
        if k % group or (splits > 1 and k < 6144):
            continue
        slots = -(-k // span)
        share = walk.stretch_of(slots, splits)
        chunk = walk.chunk_of(entries * planes, xrl, parts * depth)
        assert chunk >= 2 and (chunk * entries * planes << xrl) <= ENTRIES
        taken = [0] * slots
        for z, part in itertools.product(range(splits), range(parts)):
            k0, k1 = min(slots, z * share), min(slots, (z + 1) * share)
            for c in range(k0, k1, chunk):
                c1 = min(k1, c + chunk)
                per = walk.stretch_of(c1 - c, parts)
                s0 = c + part * per
                for base in range(s0, s0 + -(-per // depth) * depth, depth):
                    assert base % 2 == 0, (k, splits, xrl, parts, base)
                    for slot in range(base, base + depth):
                        if slot < min(c1, s0 + per):
                            taken[slot] += 1
        assert taken == [1] * slots, (k, splits, xrl, parts)
