"""The attention kernels' page lookup (block_of_tile and page_recip in csrc/kv_cache.hpp), compiled
for the host: the block of a token is its quotient by the page size, up to the longest sequence."""
import ctypes
import subprocess

import numpy as np
import pytest

from bit_affine_quantized_qmv_amd import build

TOKENS = 2 ** 30             # the most tokens of a sequence

SOURCE = """
#include "kv_cache.hpp"
// the number of tiles (16 tokens each) whose block is not tile / (page_size / 16)
extern "C" long wrong_blocks(int page_size, const unsigned* tiles, long n) {
  const uint64_t recip = qmm::kv::page_recip(page_size);
  long wrong = 0;
  for (long i = 0; i < n; ++i)
    wrong += qmm::kv::block_of_tile(tiles[i], recip) != (int)(tiles[i] / (unsigned)(page_size / 16));
  return wrong;
}
"""


@pytest.fixture(scope="module")
def wrong_blocks(tmp_path_factory):
    d = tmp_path_factory.mktemp("lookup")
    (d / "lookup.hip").write_text(SOURCE)
    cmd = [build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", build.CSRC,
           str(d / "lookup.hip"), "-o", str(d / "lookup.so")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    f = ctypes.CDLL(str(d / "lookup.so")).wrong_blocks
    f.restype = ctypes.c_long
    f.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_long]

    def call(page_size, tiles):
        tiles = np.ascontiguousarray(tiles, dtype=np.uint32)
        return f(page_size, tiles.ctypes.data, tiles.size)

    return call


def test_every_page_size_at_the_edges_of_its_blocks(wrong_blocks):
    """A quotient is wrong first at a block's first or last tile: all blocks' of the short range,
    a thousand over the whole range, and the last ones."""
    last = TOKENS // 16 - 1
    for page_size in range(16, 65536 + 1, 16):
        d = page_size // 16
        blocks = np.unique(np.concatenate([np.arange(64), np.linspace(0, last // d, 1000).astype(np.int64),
                                           last // d - np.arange(8)]).clip(0, last // d))
        tiles = np.concatenate([blocks * d, blocks * d + d - 1, [last]])
        assert wrong_blocks(page_size, tiles[tiles <= last]) == 0, page_size


@pytest.mark.parametrize("page_size", [16, 32, 48, 64, 256, 65520])
def test_every_tile_of_some_page_sizes(wrong_blocks, page_size):
    for start in range(0, TOKENS // 16, 2 ** 23):
        assert wrong_blocks(page_size, np.arange(start, start + 2 ** 23, dtype=np.uint32)) == 0, start
