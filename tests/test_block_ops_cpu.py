"""The attention half's operators without a GPU: argument checks, sizes, and the cache layout's formulas."""
import ctypes

import numpy as np
import pytest
import torch

from tests import block_ref as R
from gguf_block_quant_gb300 import zdmmv as Z

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    return Z.lib()


class _RmsnormArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "residual", "weight", "out", "xq", "y")] + [
        (n, ctypes.c_int64) for n in ("rows", "cols", "x_stride", "residual_stride")] + [("eps", ctypes.c_float)]


class _KvCache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ("n_seq", "max_pages", "page_tokens", "n_kv_heads", "head_dim")]


class _KvAppendArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "q", "seq", "pos", "rope", "q_out", "k_val", "v_val",
                                               "status_dev")] + [
        (n, ctypes.c_int64) for n in ("k_stride", "v_stride", "q_stride", "rope_rows")] + [
        (n, ctypes.c_int32) for n in ("n_tok", "n_q_heads", "rot_dim", "rope_style")]


class _AttnArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "q_start", "kv_len", "out", "workspace", "status_dev")] + [
        ("workspace_bytes", ctypes.c_size_t), ("q_stride", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ("n_tok", "n_q_heads", "max_q_len", "max_kv_len", "window")] + [
        ("scale", ctypes.c_float)]


def _header_fields(name):
    """[(C type, field)] of a struct of include/zdmmv.h, in order."""
    import os
    import re
    from gguf_block_quant_gb300 import _build
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(_build.INCLUDE, "zdmmv.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
    out = []
    for line in body.split(";"):
        line = " ".join(line.split())
        if line:
            kind = re.match(r"(const )?(\w+)", line).group(2)
            for f in line[line.index(kind) + len(kind):].split(","):
                out.append(("ptr" if "*" in f else kind, f.replace("*", "").strip()))
    return out


@pytest.mark.parametrize("name, c, packed", [
    ("zdmmv_rmsnorm_args", _RmsnormArgs, Z._RMSNORM_ARGS), ("zdmmv_kv_cache", _KvCache, Z._KV_CACHE),
    ("zdmmv_kv_append_args", _KvAppendArgs, Z._KV_APPEND_ARGS), ("zdmmv_attn_args", _AttnArgs, Z._ATTN_ARGS)])
def test_packed_structs_match_the_header(name, c, packed):
    kinds = {"ptr": ctypes.c_void_p, "int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float,
             "size_t": ctypes.c_size_t}
    want = _header_fields(name)
    # pointers that share a line ("const float *k, *v") keep their star each
    assert [(f, t) for f, t in c._fields_] == [(f, kinds[k]) for k, f in want]
    assert packed.size == ctypes.sizeof(c)
    values = [1000 + i for i in range(len(want))]
    s = c.from_buffer_copy(packed.pack(*values))
    assert [getattr(s, f) for _, f in want] == values


def _cache(**k):
    d = dict(pages=FAKE, page_table=FAKE, n_pages=9, n_seq=2, max_pages=4, page_tokens=32, n_kv_heads=2, head_dim=128)
    return _KvCache(**{**d, **k})


def _norm(**k):
    d = dict(x=FAKE, residual=FAKE, weight=FAKE, out=FAKE, xq=FAKE, y=FAKE, rows=3, cols=64, x_stride=64,
             residual_stride=64, eps=1e-6)
    return _RmsnormArgs(**{**d, **k})


def _append(**k):
    d = dict(k=FAKE, v=FAKE, q=FAKE, seq=FAKE, pos=FAKE, rope=FAKE, q_out=FAKE, k_val=FAKE, v_val=FAKE,
             status_dev=FAKE, k_stride=256, v_stride=256, q_stride=1024, rope_rows=100, n_tok=3, n_q_heads=8,
             rot_dim=128, rope_style=0)
    return _KvAppendArgs(**{**d, **k})


def _attn(**k):
    d = dict(q=FAKE, q_start=FAKE, kv_len=FAKE, out=FAKE, workspace=FAKE, status_dev=FAKE, workspace_bytes=1 << 40,
             q_stride=1024, n_tok=3, n_q_heads=8, max_q_len=2, max_kv_len=100, window=0, scale=0.1)
    return _AttnArgs(**{**d, **k})


@pytest.mark.parametrize("code, change", [
    (2, dict(rows=-1)), (2, dict(cols=48)), (2, dict(cols=0)), (2, dict(cols=32800)), (2, dict(eps=0.0)),
    (2, dict(eps=float("nan"))), (2, dict(eps=float("inf"))), (2, dict(x_stride=60)), (2, dict(residual_stride=32)),
    (2, dict(x_stride=68)), (2, dict(residual_stride=68, x=FAKE * 2)),            # out in place of a strided input
    (1, dict(x=None)), (1, dict(out=None, xq=None, y=None)),
    (3, dict(x=FAKE + 4, out=None)), (3, dict(residual=FAKE + 8)), (3, dict(weight=FAKE + 4)), (3, dict(xq=FAKE + 2)),
    (3, dict(y=FAKE + 4)), (3, dict(out=FAKE + 4)), (3, dict(x_stride=66, out=None)),
    (0, dict(rows=0, x=None)),
])
def test_norm_checks(L, code, change):
    assert L.zdmmv_add_rmsnorm_q8_0(ctypes.byref(_norm(**change)), None) == code


@pytest.mark.parametrize("code, change", [
    (2, dict(page_tokens=24)), (2, dict(page_tokens=0)), (2, dict(page_tokens=1040)), (2, dict(n_kv_heads=0)),
    (2, dict(head_dim=80)), (2, dict(head_dim=512)), (2, dict(n_pages=0)), (2, dict(n_seq=0)), (2, dict(max_pages=0)),
    (1, dict(pages=None)), (1, dict(page_table=None)), (3, dict(pages=FAKE + 8)), (3, dict(page_table=FAKE + 2)),
])
def test_cache_checks(L, code, change):
    c = _cache(**change)
    assert L.zdmmv_kv_append_q4_0(ctypes.byref(c), ctypes.byref(_append()), None) == code
    assert L.zdmmv_attn_q4_0(ctypes.byref(c), ctypes.byref(_attn()), None) == code


@pytest.mark.parametrize("code, change", [
    (2, dict(n_tok=-1)), (2, dict(rot_dim=3)), (2, dict(rot_dim=130)), (2, dict(rot_dim=-2)), (2, dict(rope_style=2)),
    (2, dict(rope_rows=0)), (2, dict(n_q_heads=0)), (2, dict(q=None)), (2, dict(n_q_heads=65536)),
    (2, dict(k_stride=252)), (2, dict(v_stride=128)), (2, dict(q_stride=1020)), (2, dict(q_stride=1028)),
    (1, dict(k=None)), (1, dict(v=None)), (1, dict(seq=None)), (1, dict(pos=None)), (1, dict(rope=None)),
    (1, dict(q_out=None)),
    (3, dict(k=FAKE + 4)), (3, dict(v=FAKE + 8)), (3, dict(q=FAKE + 4)), (3, dict(q_out=FAKE + 8)),
    (3, dict(rope=FAKE + 4)), (3, dict(k_val=FAKE + 4)), (3, dict(v_val=FAKE + 2)), (3, dict(seq=FAKE + 2)),
    (3, dict(status_dev=FAKE + 1)), (3, dict(k_stride=258)),
    (0, dict(n_tok=0, k=None)), (0, dict(n_tok=0, q=None, n_q_heads=0)),
])
def test_append_checks(L, code, change):
    assert L.zdmmv_kv_append_q4_0(ctypes.byref(_cache()), ctypes.byref(_append(**change)), None) == code


@pytest.mark.parametrize("code, change", [
    (2, dict(n_tok=-1)), (2, dict(n_q_heads=7)), (2, dict(n_q_heads=0)), (2, dict(n_q_heads=65536)),
    (2, dict(max_q_len=0)), (2, dict(max_kv_len=-1)), (2, dict(window=-1)), (2, dict(scale=float("inf"))),
    (2, dict(scale=float("nan"))), (2, dict(q_stride=1000)),
    (1, dict(q=None)), (1, dict(q_start=None)), (1, dict(kv_len=None)), (1, dict(out=None)),
    (3, dict(q=FAKE + 4)), (3, dict(out=FAKE + 8)), (3, dict(q_start=FAKE + 1)), (3, dict(kv_len=FAKE + 2)),
    (3, dict(workspace=FAKE + 8)), (3, dict(status_dev=FAKE + 2)), (3, dict(q_stride=1026)),
    (1, dict(workspace=None, max_kv_len=100000)), (6, dict(workspace_bytes=8192, max_kv_len=100000)),
    (0, dict(n_tok=0, q=None)),
])
def test_attention_checks(L, code, change):
    assert L.zdmmv_attn_q4_0(ctypes.byref(_cache()), ctypes.byref(_attn(**change)), None) == code


def test_attention_workspace_grows_with_the_bounds(L):
    c = _cache(max_pages=1 << 16)
    size = lambda heads, new, most: L.zdmmv_attn_q4_0_workspace_bytes(ctypes.byref(c), heads, new, most)  # noqa: E731
    assert size(8, 1, 16) == 0                                   # one split: none needed
    last = 0
    for most in (1000, 1001, 5000, 20000, 20016, 65536, 1 << 20):
        assert size(8, 1, most) >= last >= 0
        last = size(8, 1, most)
    assert last > 8192
    assert size(7, 1, 1000) == 0 and size(8, 0, 1000) == 0       # refused shapes


def test_null_structs(L):
    c = _cache()
    assert L.zdmmv_add_rmsnorm_q8_0(None, None) == 1
    assert L.zdmmv_kv_append_q4_0(ctypes.byref(c), None, None) == 1
    assert L.zdmmv_kv_append_q4_0(None, ctypes.byref(_append()), None) == 1
    assert L.zdmmv_attn_q4_0(ctypes.byref(c), None, None) == 1
    assert L.zdmmv_attn_q4_0(None, ctypes.byref(_attn()), None) == 1


def test_page_bytes(L):
    assert Z.kv_page_bytes(16, 1, 128) == 16 * 2 * 128 * 18 // 32
    assert Z.kv_page_bytes(1024, 3, 96) == 1024 * 3 * 2 * 96 * 18 // 32
    for bad in ((8, 1, 128), (16, 0, 128), (16, 1, 32), (2048, 1, 128)):
        assert Z.kv_page_bytes(*bad) == 0


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_layout_is_a_permutation_that_keeps_tokens_apart(dim):
    k, v, s = R.tile_index(dim)
    for i, n in ((k, 16 * dim), (v, 16 * dim), (s, 16 * dim // 32)):
        assert np.array_equal(np.sort(i.ravel()), np.arange(n))
    # no byte of codes holds values of two tokens
    for i in (k, v):
        owner = np.full(8 * dim, -1)
        for r in range(16):
            b = i[r] // 2
            assert np.all((owner[b] == -1) | (owner[b] == r))
            owner[b] = r


def test_layout_round_trip():
    rng = np.random.default_rng(1)
    pages = np.zeros(2 * Z.kv_page_bytes(32, 2, 96), np.uint8)
    x = rng.standard_normal(96).astype(np.float32)
    q, d = R.quantize_q4(x)
    R.put(pages, 32, 2, 96, 1, 21, 1, 1, q, d)
    k, v = R.values(pages, 32, 2, 96)
    want = (q - 8) * np.repeat(d.astype(np.float64), 32)
    assert np.array_equal(v[1, 1, 21], want) and not k.any() and np.count_nonzero(v) <= 96
    # a block's value of the largest magnitude is code 0 (-8), every value within half a step (a whole one at the top)
    step = np.abs(np.repeat(d.astype(np.float64), 32))
    assert np.all(np.abs(want - x) <= step * 1.01) and q.reshape(-1, 32).min(1).tolist() == [0, 0, 0]


def test_q4_by_hand():
    x = np.zeros(64, np.float32)
    x[3], x[7], x[9] = 4.0, -4.0, 1.0       # the first of the largest magnitude sets the sign: d = -0.5
    q, d = R.quantize_q4(x)
    assert d[0] == np.float16(-0.5) and d[1] == 0
    assert q[3] == 0 and q[7] == 15 and q[9] == 6 and q[0] == 8 and np.all(q[32:] == 8)


def test_binding_refusals():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        Z.add_rmsnorm_q8_0(x, None, 1e-6)                        # a host tensor
    with pytest.raises(ValueError):
        Z.KVCache(torch.zeros(9, dtype=torch.uint8), 20, 1, 128, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        Z.KVCache(torch.zeros(9, dtype=torch.uint8), 16, 1, 128, torch.zeros(1, 1, dtype=torch.int64))
