"""CPU tests of the largest calls of the cache's entry points: refused on the host, with a message,
where one launch would have more threads than HIP allows."""
import ctypes

import pytest

import bit_affine_quantized_qmv_amd as q
from test_abi_decode_ops import P, cache, expect


@pytest.mark.parametrize("heads,head_dim", [(1, 64), (8, 128), (4096, 256), (3, 256)])
def test_append_and_read_refuse_more_threads_than_a_launch_has(heads, head_dim):
    lib, c = q.load(), cache(heads=heads, head_dim=head_dim, pages=2 ** 26)
    rows = 2048 // head_dim                                  # of a workgroup of 256 threads
    most = (2 ** 24 - 1) // (2 * heads) * rows               # 2^24 - 1 workgroups: fewer than 2^32 threads
    for tokens in (most + 1, 2 ** 31 - 1):
        if tokens < 2 ** 31:
            expect(lib.qmm_kv_append(ctypes.byref(c), P, 256, 128, P, 256, 128, P, tokens, None), "SHAPE", "2^34")
            expect(lib.qmm_kv_read(ctypes.byref(c), P, tokens, P, P, None), "SHAPE", "2^34")
