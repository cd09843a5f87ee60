"""CPU tests of the argument checks of the tree, move, page and fork entry points: every refusal
happens on the host, with a code and a message, before anything is enqueued (no GPU is needed)."""
import ctypes

import pytest
import torch

import bit_affine_quantized_qmv_amd as q
from bit_affine_quantized_qmv_amd import _lib
from test_abi_decode_ops import BAD_ATTENDS, BAD_CACHES, CODE, P, attend, cache, expect

R = ctypes.byref


def accept(**kw):
    d = dict(parents=P, tokens=P, sampled=P, parents_stride=8, tokens_stride=8, sampled_stride=8, batch=2, nodes=8)
    return _lib.TreeAcceptDesc(**{**d, **kw})


def move(**kw):
    d = dict(block_table=P, table_stride=10, blocks=10, to_table=P, to_stride=10, to_blocks=10, index=P, index_stride=5,
             batch=3, count=5, origin=P, start=P)
    return _lib.KVMoveDesc(**{**d, **kw})


def fork(**kw):
    d = dict(refs=P, pages=100, page_size=16, block_table=P, table_stride=10, blocks=10, lengths=P, batch=3, parents=P,
             want=P, rows=4, new_table=P, new_stride=12, new_blocks=12)
    return _lib.KVForkDesc(**{**d, **kw})


@pytest.mark.parametrize("change,error", BAD_CACHES)
def test_caches(change, error):
    lib, c = q.load(), cache(**change)
    expect(lib.qmm_kv_attend_tree(R(c), R(attend()), P, P, P, P, 1 << 40, None), error, "kv")
    expect(lib.qmm_kv_move(R(c), R(move()), None), error, "kv")
    expect(lib.qmm_kv_copy_pages(R(c), P, P, 4, None), error, "kv")


@pytest.mark.parametrize("change,error", BAD_ATTENDS)
def test_attend_descriptions(change, error):
    lib, c, a = q.load(), cache(), attend(**change)
    expect(lib.qmm_kv_attend_tree(R(c), R(a), P, P, P, P, 1 << 40, None), error, "kv_attend")
    assert lib.qmm_kv_attend_tree_workspace_bytes(R(c), R(a)) == CODE["QMM_ERR_" + error]


def test_attend_tree():
    lib, c = q.load(), cache()

    def call(mask=P, depth=P, out=P, ws=P, size=1 << 40, **kw):
        return lib.qmm_kv_attend_tree(R(c), R(attend(**kw)), mask, depth, out, ws, size, None)

    expect(lib.qmm_kv_attend_tree(R(c), None, P, P, P, P, 0, None), "NULL", "args")
    expect(call(causal=0), "UNSUPPORTED", "causal")
    expect(call(q_len=1025), "SHAPE", "1024")
    expect(call(mask=None), "NULL", "mask")
    expect(call(depth=None, window=4), "NULL", "depth")
    expect(call(mask=P + 2), "ALIGN")
    expect(call(depth=P + 2), "ALIGN")
    for name in ("q", "lengths", "block_table"):
        expect(call(**{name: None}), "NULL")
    expect(call(out=None), "NULL")
    expect(call(out=P + 8), "ALIGN")
    expect(call(size=0, q_len=8), "SHAPE", "workspace")
    expect(call(ws=None, size=0, q_len=8), "NULL", "workspace")
    assert call(mask=None, depth=None, batch=0) == 0 and call(mask=None, q_len=0) == 0


def test_tree_mask_and_accept():
    lib = q.load()
    expect(lib.qmm_tree_mask(None, 8, 2, 8, 0, P, P, None), "NULL")
    expect(lib.qmm_tree_mask(P, 8, 2, 8, 0, None, P, None), "NULL")
    expect(lib.qmm_tree_mask(P, 7, 2, 8, 0, P, P, None), "SHAPE")
    expect(lib.qmm_tree_mask(P, 2000, 2, 1025, 0, P, P, None), "SHAPE")
    expect(lib.qmm_tree_mask(P, 8, 65536, 8, 0, P, P, None), "SHAPE")
    expect(lib.qmm_tree_mask(P, 8, -1, 8, 0, P, P, None), "SHAPE")
    expect(lib.qmm_tree_mask(P, 8, 2, 8, -1, P, P, None), "UNSUPPORTED", "window")
    expect(lib.qmm_tree_mask(P + 1, 8, 2, 8, 0, P, P, None), "ALIGN")
    expect(lib.qmm_tree_mask(P, 8, 2, 8, 0, P, P + 2, None), "ALIGN")
    assert lib.qmm_tree_mask(None, 8, 0, 8, 0, None, None, None) == 0
    assert lib.qmm_tree_mask(None, 0, 2, 0, 0, None, None, None) == 0
    expect(lib.qmm_tree_accept(None, P, P, P, None), "NULL")
    for name in ("parents", "tokens", "sampled"):
        expect(lib.qmm_tree_accept(R(accept(**{name: None})), P, P, P, None), "NULL")
        expect(lib.qmm_tree_accept(R(accept(**{name: P + 2})), P, P, P, None), "ALIGN")
        expect(lib.qmm_tree_accept(R(accept(**{name + "_stride": 7})), P, P, P, None), "SHAPE")
    for i in range(3):
        out = [P, P, P]
        out[i] = None
        expect(lib.qmm_tree_accept(R(accept()), *out, None), "NULL")
    expect(lib.qmm_tree_accept(R(accept(nodes=0)), P, P, P, None), "SHAPE")
    expect(lib.qmm_tree_accept(R(accept(batch=65536)), P, P, P, None), "SHAPE")
    assert lib.qmm_tree_accept(R(accept(batch=0, parents=None)), None, None, None, None) == 0


def test_move_and_copy_pages():
    lib, c = q.load(), cache()

    def call(**kw):
        return lib.qmm_kv_move(R(c), R(move(**kw)), None)

    expect(lib.qmm_kv_move(R(c), None, None), "NULL")
    for name in ("block_table", "index", "start"):
        expect(call(**{name: None}), "NULL")
    for name in ("block_table", "to_table", "index", "origin", "start"):
        expect(call(**{name: P + 2}), "ALIGN")
    for bad in (dict(batch=-1), dict(batch=65536), dict(count=-1), dict(count=2 ** 30 + 1, index_stride=2 ** 31),
                dict(blocks=-1), dict(blocks=11), dict(to_blocks=11), dict(to_blocks=-1), dict(index_stride=4)):
        expect(call(**bad), "SHAPE", "kv_move")
    expect(lib.qmm_kv_move(R(cache(heads=4096)), R(move(batch=4096)), None), "SHAPE", "heads")
    assert call(batch=0, index=None) == 0 and call(count=0, start=None) == 0
    expect(lib.qmm_kv_copy_pages(R(c), None, P, 4, None), "NULL")
    expect(lib.qmm_kv_copy_pages(R(c), P, None, 4, None), "NULL")
    expect(lib.qmm_kv_copy_pages(R(c), P, P + 2, 4, None), "ALIGN")
    expect(lib.qmm_kv_copy_pages(R(c), P, P, -1, None), "SHAPE")
    expect(lib.qmm_kv_copy_pages(R(c), P, P, 2 ** 31, None), "SHAPE")
    assert lib.qmm_kv_copy_pages(R(c), None, None, 0, None) == 0


def test_fork():
    lib = q.load()

    def call(src=P, dst=P, short=P, ws=P, size=1 << 40, **kw):
        return lib.qmm_kv_fork(R(fork(**kw)), src, dst, short, ws, size, None)

    expect(lib.qmm_kv_fork(None, P, P, P, P, 1 << 40, None), "NULL")
    for name in ("refs", "block_table", "lengths", "parents", "new_table"):
        expect(call(**{name: None}), "NULL")
    for name in ("refs", "block_table", "lengths", "parents", "new_table", "want"):
        expect(call(**{name: P + 2}), "ALIGN")
    for name in ("src", "dst", "short", "ws"):
        expect(call(**{name: None}), "NULL")
        expect(call(**{name: P + 2}), "ALIGN")
    for bad in (dict(page_size=24), dict(page_size=0), dict(page_size=65552), dict(pages=0), dict(pages=2 ** 27),
                dict(batch=-1), dict(batch=65536), dict(rows=65536), dict(rows=-1), dict(blocks=-1), dict(blocks=11),
                dict(new_blocks=13), dict(new_blocks=-1), dict(rows=65535, new_blocks=2 ** 15, new_stride=2 ** 15)):
        expect(call(**bad), "SHAPE", "kv_fork")
        assert lib.qmm_kv_fork_workspace_bytes(R(fork(**bad))) == CODE["QMM_ERR_SHAPE"]
    need = lib.qmm_kv_fork_workspace_bytes(R(fork(refs=None)))
    assert need >= 4 * (4 + 4 + 1 + 48)
    expect(call(size=need - 1), "SHAPE", "workspace")


def test_python_arguments():
    i = torch.zeros(2, 4, dtype=torch.int32)
    c = q.kv_cache(2, 16, 2, 64, 32, "bf16", device="cpu")
    with pytest.raises(ValueError, match="parents"):
        q.tree_mask(i)                                     # not on a GPU
    with pytest.raises(ValueError, match="index"):
        q.kv_move(c, i, i.long(), i[:, 0])
    with pytest.raises(ValueError, match="src"):
        q.kv_copy_pages(c, i, i)
    with pytest.raises(ValueError, match="refs"):
        q.kv_fork(i, i, i[:, 0], i[0], 16)
    with pytest.raises(ValueError, match="parents"):
        q.tree_accept(i, i, i)
    with pytest.raises(ValueError, match="q"):
        q.kv_attend_tree(torch.zeros(2, 4, 2), c, i, i[:, 0], i)
