"""CPU tests of the decode-step entry points' argument checks: every refusal happens on the
host, with a code and a message, before anything is enqueued (no GPU is needed)."""
import ctypes

import pytest

import bit_affine_quantized_qmv_amd as q
from bit_affine_quantized_qmv_amd import _lib

CODE = {name: code for code, name in _lib.ERRORS.items()}
P = 1 << 20                      # an aligned address that no refused call touches


def expect(rc, name, word=None):
    assert rc == CODE["QMM_ERR_" + name], (rc, name, _lib.load().qmm_last_error())
    message = _lib.load().qmm_last_error().decode()
    assert message and (word is None or word in message), message


def cache(**kw):
    d = dict(data=P, pages=10, page_size=16, heads=2, head_dim=128, group_size=64, dtype=1)
    d.update(kw)
    return _lib.KVCacheDesc(**d)


BAD_CACHES = [
    (dict(dtype=3), "UNSUPPORTED"), (dict(head_dim=96), "UNSUPPORTED"), (dict(group_size=16), "UNSUPPORTED"),
    (dict(head_dim=64, group_size=128), "UNSUPPORTED"), (dict(page_size=24), "SHAPE"), (dict(page_size=0), "SHAPE"),
    (dict(page_size=65552), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(pages=0), "SHAPE"),
    (dict(pages=2 ** 27, page_size=16), "SHAPE"), (dict(data=None), "NULL"), (dict(data=P + 8), "ALIGN"),
]


@pytest.mark.parametrize("change,error", BAD_CACHES)
def test_cache_descriptions_are_checked_by_every_entry(change, error):
    lib, c = q.load(), cache(**change)
    expect(lib.qmm_kv_append(ctypes.byref(c), P, 256, 128, P, 256, 128, P, 4, None), error, "kv")
    expect(lib.qmm_kv_read(ctypes.byref(c), P, 4, P, P, None), error, "kv")
    a = attend()
    expect(lib.qmm_kv_attend(ctypes.byref(c), ctypes.byref(a), P, P, 1 << 40, None), error, "kv")
    if error not in ("NULL", "ALIGN"):
        assert lib.qmm_kv_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(a)) == CODE["QMM_ERR_" + error]


def test_append_and_read_refusals():
    lib, c = q.load(), cache()
    r = ctypes.byref(c)
    expect(lib.qmm_kv_append(None, P, 256, 128, P, 256, 128, P, 4, None), "NULL", "cache")
    for i in (1, 4, 7):
        args = [r, P, 256, 128, P, 256, 128, P, 4, None]
        args[i] = None
        expect(lib.qmm_kv_append(*args), "NULL")
    for i in (2, 3, 5, 6):
        args = [r, P, 256, 128, P, 256, 128, P, 4, None]
        args[i] = -256
        expect(lib.qmm_kv_append(*args), "LAYOUT")
        args[i] = 132
        expect(lib.qmm_kv_append(*args), "ALIGN")
    expect(lib.qmm_kv_append(r, P + 2, 256, 128, P, 256, 128, P, 4, None), "ALIGN")
    expect(lib.qmm_kv_append(r, P, 256, 128, P, 256, 128, P + 2, 4, None), "ALIGN")
    expect(lib.qmm_kv_append(r, P, 256, 128, P, 256, 128, P, -1, None), "SHAPE")
    expect(lib.qmm_kv_read(r, None, 4, P, P, None), "NULL")
    expect(lib.qmm_kv_read(r, P, 4, None, P, None), "NULL")
    expect(lib.qmm_kv_read(r, P, 4, P, P + 8, None), "ALIGN")
    expect(lib.qmm_kv_read(r, P, 2 ** 31, P, P, None), "SHAPE")
    # nothing to do is no error, whatever the pointers
    assert lib.qmm_kv_append(r, None, 256, 128, None, 256, 128, None, 0, None) == 0
    assert lib.qmm_kv_read(r, None, 0, None, None, None) == 0
    assert lib.qmm_last_error() == b""


def attend(**kw):
    d = dict(q=P, q_batch_stride=1024, q_token_stride=1024, q_head_stride=128, batch=3, q_len=1, q_heads=8, causal=1,
             window=0, scale=0.1, block_table=P, table_stride=10, max_blocks=10, lengths=P, max_length=160)
    d.update(kw)
    return _lib.KVAttendDesc(**d)


BAD_ATTENDS = [
    (dict(batch=-1), "SHAPE"), (dict(batch=65536), "SHAPE"), (dict(q_len=-1), "SHAPE"), (dict(q_len=40000), "SHAPE"),
    (dict(q_heads=0), "SHAPE"), (dict(q_heads=7), "SHAPE"), (dict(window=-1), "UNSUPPORTED"),
    (dict(window=5, causal=0), "UNSUPPORTED"), (dict(max_blocks=11), "SHAPE"), (dict(max_blocks=-1), "SHAPE"),
    (dict(max_length=161), "SHAPE"), (dict(max_length=-1), "SHAPE"),
    (dict(table_stride=2 ** 27, max_blocks=2 ** 27, max_length=2 ** 30 + 1), "SHAPE"),
    (dict(q_token_stride=-8), "LAYOUT"), (dict(q_head_stride=4), "ALIGN"),
]


@pytest.mark.parametrize("change,error", BAD_ATTENDS)
def test_attend_descriptions_are_checked(change, error):
    lib, c, a = q.load(), cache(), attend(**change)
    expect(lib.qmm_kv_attend(ctypes.byref(c), ctypes.byref(a), P, P, 1 << 40, None), error, "kv_attend")
    assert lib.qmm_kv_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(a)) == CODE["QMM_ERR_" + error]


def test_attend_pointers_and_workspace():
    lib, c = q.load(), cache()
    r = ctypes.byref(c)

    def call(out=P, ws=P, size=1 << 40, **kw):
        return lib.qmm_kv_attend(r, ctypes.byref(attend(**kw)), out, ws, size, None)

    expect(lib.qmm_kv_attend(r, None, P, P, 0, None), "NULL", "args")
    expect(call(q=None), "NULL")
    expect(call(out=None), "NULL")
    expect(call(lengths=None), "NULL")
    expect(call(block_table=None), "NULL")
    expect(call(q=P + 2), "ALIGN")
    expect(call(out=P + 8), "ALIGN")
    expect(call(ws=P + 8), "ALIGN")
    expect(call(block_table=P + 2), "ALIGN")
    # a call that splits its tokens needs the workspace it asks for
    need = lib.qmm_kv_attend_workspace_bytes(r, ctypes.byref(attend()))
    assert need > 0
    expect(call(ws=None), "NULL", "workspace")
    expect(call(size=need - 4), "SHAPE", "workspace")
    assert call(batch=0, q=None, lengths=None, block_table=None, out=None, ws=None, size=0) == 0
    assert call(q_len=0, q=None, lengths=None, block_table=None, out=None, ws=None, size=0) == 0


def test_attend_workspace_grows_with_the_length_and_serves_windows():
    lib, c = q.load(), cache(pages=2 ** 20)
    last = 0
    for length in (0, 1, 100, 129, 1000, 5000, 10 ** 5, 10 ** 6, 2 ** 24):
        a = attend(max_blocks=2 ** 20, table_stride=2 ** 20, max_length=length)
        n = lib.qmm_kv_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(a))
        assert n >= last
        last = n
        for window in (1, 77, 1000, 10 ** 5):
            a.window = window
            assert lib.qmm_kv_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(a)) == n


def stack(n, k, bits=4, gs=64, dtype=1, experts=8, **kw):
    row = k * bits // 32
    w = dict(w_packed=P, w_row_stride=row, scales=P, biases=P, sb_row_stride=k // gs, N=n, K=k, group_size=gs, bits=bits,
             dtype=dtype)
    s = dict(num_experts=experts, w_expert_stride=n * row, sb_expert_stride=n * (k // gs))
    for key, value in kw.items():
        (w if key in w else s)[key] = value
    return _lib.ExpertStack(w=_lib.WeightDesc(**w), **s)


def moe(gate=None, up=None, down=None, y=P, ws=P, size=1 << 40, **kw):
    lib = q.load()
    gate, up, down = gate or stack(128, 256), up or stack(128, 256), down or stack(256, 128)
    d = dict(x=P, x_stride=256, router_logits=P, router_stride=8, tokens=4, top_k=2, renormalize=1, dtype=1,
             gate=ctypes.pointer(gate), up=ctypes.pointer(up), down=ctypes.pointer(down), y_stride=256)
    d.update(kw)
    return lib.qmm_moe(ctypes.byref(_lib.MoeDesc(**d)), y, ws, size, None)


def test_moe_refusals():
    lib = q.load()
    expect(lib.qmm_moe(None, P, P, 0, None), "NULL")
    for name in ("x", "router_logits"):
        expect(moe(**{name: None}), "NULL")
    expect(moe(y=None), "NULL")
    expect(moe(ws=None), "NULL")
    expect(moe(gate=stack(128, 256, w_packed=None)), "NULL", "gate")
    expect(moe(tokens=33), "SHAPE", "tokens")
    expect(moe(tokens=-1), "SHAPE")
    expect(moe(top_k=0), "SHAPE", "top_k")
    expect(moe(top_k=9), "SHAPE", "top_k")
    expect(moe(y_stride=255), "SHAPE", "y_stride")
    expect(moe(x_stride=-256), "LAYOUT")
    expect(moe(dtype=3), "UNSUPPORTED")
    expect(moe(x_stride=260), "ALIGN")
    expect(moe(x=P + 8), "ALIGN")
    expect(moe(ws=P + 8), "ALIGN")
    expect(moe(up=stack(128, 320)), "SHAPE", "up")
    expect(moe(down=stack(128, 256)), "SHAPE", "down")
    expect(moe(up=stack(128, 256, experts=7)), "SHAPE", "experts")
    expect(moe(up=stack(128, 256, bits=8)), "UNSUPPORTED", "bits")
    expect(moe(up=stack(128, 256, gs=32)), "UNSUPPORTED", "group_size")
    expect(moe(down=stack(256, 128, bits=7)), "UNSUPPORTED", "down")
    expect(moe(down=stack(256, 128, dtype=2)), "UNSUPPORTED", "dtype")
    expect(moe(gate=stack(128, 256, w_row_stride=31)), "SHAPE", "row")
    expect(moe(gate=stack(128, 256, w_row_stride=34, w_expert_stride=128 * 34)), "ALIGN", "multiples of 4")
    expect(moe(gate=stack(128, 256, w_expert_stride=128 * 32 - 4)), "SHAPE", "expert")
    expect(moe(gate=stack(128, 256, w_packed=P + 4)), "ALIGN")
    expect(moe(gate=stack(128, 256, scales=P + 1)), "ALIGN")
    big = 2 ** 20
    expect(moe(gate=stack(big, 2048, experts=2, w_row_stride=2048, w_expert_stride=big * 2048),
               up=stack(big, 2048, experts=2), down=stack(2048, big, experts=2), x_stride=2048, y_stride=2048),
           "SHAPE", "1 GiB")
    need = lib.qmm_moe_workspace_bytes(4, 8, 2, 256, 128)
    expect(moe(size=need - 1), "SHAPE", "workspace")
    for args, name in (((33, 8, 2, 256, 128), "SHAPE"), ((4, 513, 2, 256, 128), "SHAPE"), ((4, 8, 33, 256, 128), "SHAPE")):
        assert lib.qmm_moe_workspace_bytes(*args) == CODE["QMM_ERR_" + name]
    assert moe(tokens=0, x=None, router_logits=None, y=None, ws=None, size=0) == 0


def test_sample_refusals():
    lib = q.load()
    p = _lib.SampleParams(None, None, None, None, 1.0, 0, 1.0, 0.0)

    def call(logits=P, dtype=1, rows=2, n=100, stride=100, params=p, u=P, index=P, prob=P, ws=P):
        return lib.qmm_sample(logits, dtype, rows, n, stride, ctypes.byref(params) if params else None, u, index, prob,
                              ws, None)

    expect(call(dtype=3), "UNSUPPORTED")
    for kw in (dict(rows=-1), dict(rows=65536), dict(n=0, stride=0), dict(n=(1 << 22) + 1, stride=1 << 23),
               dict(stride=99)):
        expect(call(**kw), "SHAPE")
    for name in ("logits", "params", "u", "index", "ws"):
        expect(call(**{name: None}), "NULL")
    for kw in (dict(logits=P + 1), dict(u=P + 2), dict(index=P + 2), dict(prob=P + 2), dict(ws=P + 4)):
        expect(call(**kw), "ALIGN")
    for i in range(4):
        arrays = [None] * 4
        arrays[i] = P + 2
        expect(call(params=_lib.SampleParams(*arrays, 1.0, 0, 1.0, 0.0)), "ALIGN")
    assert call(rows=0, logits=None, u=None, index=None, prob=None, ws=None) == 0
    assert lib.qmm_last_error() == b""
