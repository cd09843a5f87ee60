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


# ---------------------------------------------------------------- grouped products and the layer

def weight(n=96, k=128, **kw):
    d = dict(w_packed=P, w_row_stride=16, scales=P, biases=P, sb_row_stride=2, N=n, K=k, group_size=64, bits=4, dtype=1)
    return _lib.WeightDesc(*[{**d, **kw}[f] for f, _ in _lib.WeightDesc._fields_])


def experts(count=4, expert=None, **kw):
    w = weight(**kw)
    return _lib.ExpertStack(w, count, w.N * w.w_row_stride if expert is None else expert, w.N * w.sb_row_stride)


def test_grouped():
    lib = q.load()

    def call(x=P, stride=128, rows=50, offsets=P, y=P, ys=96, ws=P, size=1 << 40, w=None):
        return lib.qmm_grouped(x, stride, rows, R(experts() if w is None else w), offsets, y, ys, ws, size, None)

    expect(lib.qmm_grouped(P, 128, 50, None, P, P, 96, P, 1 << 40, None), "NULL", "weights")
    for name in ("x", "offsets", "y", "ws"):
        expect(call(**{name: None}), "NULL")
    for name, at in (("x", P + 8), ("ws", P + 8), ("offsets", P + 2), ("y", P + 1)):
        expect(call(**{name: at}), "ALIGN")
    expect(call(rows=-1), "SHAPE")
    expect(call(rows=2 ** 20 + 1), "SHAPE")
    expect(call(stride=-128), "LAYOUT")
    expect(call(stride=132), "ALIGN")
    expect(call(ys=95), "SHAPE")
    expect(call(w=experts(count=513)), "SHAPE", "experts")
    expect(call(w=experts(count=0)), "SHAPE")
    expect(call(w=experts(bits=7)), "UNSUPPORTED")
    expect(call(w=experts(group_size=16)), "UNSUPPORTED")
    expect(call(w=experts(k=96)), "SHAPE")                          # not a multiple of the group
    expect(call(w=experts(w_row_stride=15)), "SHAPE")
    expect(call(w=experts(w_row_stride=18)), "ALIGN")
    expect(call(w=experts(expert=96 * 16 - 4)), "SHAPE", "expert")
    expect(call(w=experts(w_packed=P + 8)), "ALIGN")
    expect(call(w=experts(scales=P + 1)), "ALIGN")
    expect(call(w=experts(biases=None)), "NULL")
    expect(call(w=experts(n=2 ** 20, w_row_stride=512)), "SHAPE", "1 GiB")
    need = lib.qmm_grouped_workspace_bytes(50, R(experts(w_packed=None, scales=None, biases=None)))
    assert need > 0
    expect(call(size=need - 1), "SHAPE", "workspace")
    assert lib.qmm_grouped_workspace_bytes(2 ** 20 + 1, R(experts())) == CODE["QMM_ERR_SHAPE"]
    assert lib.qmm_grouped_workspace_bytes(5, None) == CODE["QMM_ERR_NULL"]
    assert lib.qmm_grouped_workspace_bytes(2 ** 20, R(experts())) >= 2 ** 20 // 64 * 16
    assert call(rows=0, x=None, offsets=None, y=None, ws=None, size=0) == 0


def layer(**kw):
    gate, up, down = (kw.pop(n, d) for n, d in (("gate", experts()), ("up", experts()),
                                                ("down", experts(n=128, k=96, w_row_stride=12, sb_row_stride=3,
                                                                 group_size=32))))
    d = dict(x=P, x_stride=128, router_logits=P, router_stride=4, tokens=40, top_k=2, renormalize=1, dtype=1,
             gate=ctypes.pointer(gate), up=ctypes.pointer(up), down=ctypes.pointer(down), y_stride=128)
    return _lib.MoeDesc(**{**d, **kw})


def test_moe_prompt():
    lib = q.load()

    def call(y=P, ws=P, size=1 << 50, **kw):
        return lib.qmm_moe_prompt(R(layer(**kw)), y, ws, size, None)

    expect(lib.qmm_moe_prompt(None, P, P, 0, None), "NULL")
    for name in ("x", "router_logits"):
        expect(call(**{name: None}), "NULL")
    expect(call(y=None), "NULL")
    expect(call(ws=None), "NULL")
    expect(call(x=P + 8), "ALIGN")
    expect(call(ws=P + 8), "ALIGN")
    expect(call(y=P + 1), "ALIGN")
    expect(call(dtype=3), "UNSUPPORTED")
    expect(call(dtype=2), "UNSUPPORTED", "dtype")
    expect(call(tokens=-1), "SHAPE")
    expect(call(tokens=65536), "SHAPE")
    expect(call(top_k=0), "SHAPE")
    expect(call(top_k=5), "SHAPE")
    expect(call(x_stride=132), "ALIGN")
    expect(call(x_stride=-8), "LAYOUT")
    expect(call(y_stride=120), "SHAPE")
    wide = dict(gate=experts(k=16384, w_row_stride=2048, sb_row_stride=256), up=experts(k=16384, w_row_stride=2048, sb_row_stride=256),
                down=experts(n=16384, k=96, w_row_stride=12, sb_row_stride=3, group_size=32))
    expect(call(x_stride=16384, y_stride=16384, tokens=65535, top_k=1, **wide), "SHAPE", "2^29")
    expect(call(up=experts(group_size=32, sb_row_stride=4)), "UNSUPPORTED", "share")
    expect(call(up=experts(count=5)), "SHAPE", "experts")
    expect(call(down=experts()), "SHAPE", "down")
    need = lib.qmm_moe_prompt_workspace_bytes(40, 4, 2, 128, 96)
    expect(call(size=need - 1), "SHAPE", "workspace")
    sizes = [40, 4, 2, 128, 96]
    for i in range(5):
        more = list(sizes)
        more[i] += 64 if i != 2 else 1
        assert lib.qmm_moe_prompt_workspace_bytes(*more) >= need
    for bad in ([65536, 4, 2, 128, 96], [40, 513, 2, 128, 96], [40, 4, 5, 128, 96], [40, 4, 2, 0, 96],
                [40, 4, 2, 128, 2 ** 20 + 1], [65535, 64, 32, 128, 96]):
        assert lib.qmm_moe_prompt_workspace_bytes(*bad) == CODE["QMM_ERR_SHAPE"]
    assert call(tokens=0, x=None, router_logits=None, y=None, ws=None, size=0) == 0


def test_moe_prompt_workspace_grows_with_every_size():
    lib = q.load()
    base = dict(tokens=3, experts=8, top_k=2, hidden=512, inter=2048)
    sizes = dict(tokens=[1, 2, 3, 8, 9, 31, 32, 33, 100, 640, 1000, 4000, 20000], experts=[2, 3, 8, 40, 300, 512],
                 top_k=[1, 2, 5, 8], hidden=[32, 256, 288, 4096, 16384], inter=[32, 1024, 1056, 2080, 14336, 2 ** 17])
    for big in (1, 60, 1000):
        for name, values in sizes.items():
            last = 0
            for v in values:
                at = dict(base, tokens=base["tokens"] * big)
                at[name] = v
                n = lib.qmm_moe_prompt_workspace_bytes(at["tokens"], at["experts"], at["top_k"], at["hidden"], at["inter"])
                assert n > 0 and n >= last, (name, v, n, last)
                last = n
