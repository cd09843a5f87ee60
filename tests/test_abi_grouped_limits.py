"""CPU tests of the largest calls of the grouped products and the expert layer: refused on the host, with a
message, where one launch would have 2^32 threads or more."""
import ctypes

import pytest

import bit_affine_quantized_qmv_amd as q
from test_abi_decode_ops import P, expect
from test_abi_tree_ops import experts, layer

R = ctypes.byref
SIZE = 1 << 60


def stack(count, n, k, group=32, bits=4):
    return experts(count=count, n=n, k=k, w_row_stride=k * bits // 32, sb_row_stride=k // group, group_size=group, bits=bits)


@pytest.mark.parametrize("rows,k,group", [
    (2 ** 20, 2 ** 15, 32),                  # 2^24 blocks of 256 threads
    (2 ** 20, 2 ** 15, 128),
    (2 ** 20, 2 ** 20, 64),                  # every limit
    (2 ** 16, 2 ** 19, 64),
    (2 ** 20, 31 * 1024 + 128, 128),         # sums of 256 groups: padded to 32768 columns
])
def test_grouped_refuses_rows_whose_staging_is_more_than_a_launch(rows, k, group):
    lib = q.load()
    expect(lib.qmm_grouped(P, k, rows, R(stack(1, 8, k, group)), P, P, 8, P, SIZE, None), "SHAPE", "rows * K")


@pytest.mark.parametrize("rows,n,count", [
    (64 * 4096, 4095 * 256, 1),              # 4097 tiles of 4095 blocks: 2^24 - 1 workgroups, launched as 2^24
    (64 * 4096, 4096 * 256, 1),
    (64 * 12290, 1365 * 256, 1),
])
def test_grouped_refuses_more_workgroups_than_a_launch(rows, n, count):
    lib = q.load()
    expect(lib.qmm_grouped(P, 32, rows, R(stack(count, n, 32)), P, P, n, P, SIZE, None), "SHAPE", "rows * N")


@pytest.mark.parametrize("tokens,top_k,count,inter", [
    (24518, 32, 32, 1365 * 128),             # 12291 tiles of 1365 blocks: 2^24 - 1
    (32768, 32, 32, 1365 * 128),
])
def test_layer_refuses_more_workgroups_than_a_launch(tokens, top_k, count, inter):
    lib = q.load()
    gate, up, down = stack(count, inter, 32), stack(count, inter, 32), stack(count, 32, inter)
    call = layer(tokens=tokens, top_k=top_k, x_stride=32, y_stride=32, router_stride=count, gate=gate, up=up, down=down)
    expect(lib.qmm_moe_prompt(R(call), P, P, SIZE, None), "SHAPE", "too large")
