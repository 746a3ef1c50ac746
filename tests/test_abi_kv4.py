"""The attention block's entry points reject bad arguments before touching HIP
(no GPU needed), their structs match the header, and the host helpers."""
import ctypes
import math
import re

import pytest

from w8a8_online_quantized_amd import cider

INV = cider.CIDER_ERROR_INVALID_VALUE
NULL = None
PTR = 1 << 20


@pytest.fixture(scope="module")
def L():
    return cider.lib()


def cache(**kw):
    a = dict(k_codes=PTR, k_scale=PTR * 2, v_codes=PTR * 3, v_scale=PTR * 4, n_pages=8, page_size=16, kv_heads=2,
             head_dim=128, group_size=0)
    a.update(kw)
    return cider.Kv4CacheArrays(**a)


BAD_CACHES = [dict(head_dim=96), dict(head_dim=0), dict(head_dim=512), dict(group_size=16), dict(group_size=48),
              dict(group_size=256), dict(group_size=-1), dict(head_dim=256, group_size=32), dict(head_dim=64, group_size=16),
              dict(page_size=8), dict(page_size=24), dict(page_size=2048), dict(page_size=0), dict(kv_heads=0),
              dict(kv_heads=1025), dict(n_pages=0), dict(n_pages=-1), dict(n_pages=1 << 27)]
NO_ARRAYS = [dict(k_codes=None), dict(k_scale=None), dict(v_codes=None), dict(v_scale=None), dict(k_codes=PTR + 8),
             dict(k_scale=PTR + 8), dict(v_codes=PTR + 4), dict(v_scale=PTR + 2)]


def rope_args(**kw):
    a = dict(x=PTR, positions=PTR, inv_freq=PTR, y=PTR * 2, T=4, x_row_stride=256, x_head_stride=64, y_row_stride=256,
             y_head_stride=64, dtype=0, heads=4, head_dim=64, rotary_dim=64, interleaved=0, scale=1.0)
    a.update(kw)
    return cider.Rope(**a)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 23), dict(heads=-1), dict(heads=65537), dict(head_dim=0), dict(head_dim=1),
    dict(head_dim=1025, rotary_dim=64, y_head_stride=1025, y_row_stride=5000), dict(rotary_dim=0), dict(rotary_dim=63),
    dict(rotary_dim=66), dict(head_dim=1024, rotary_dim=514, y_head_stride=1024, y_row_stride=4096), dict(dtype=2),
    dict(interleaved=2), dict(interleaved=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(x=None), dict(y=None),
    dict(positions=None), dict(inv_freq=None), dict(x=PTR + 2), dict(y=PTR * 2 + 8), dict(positions=PTR + 4),
    dict(inv_freq=PTR + 8), dict(x_row_stride=-1), dict(x_head_stride=-64), dict(y_head_stride=63), dict(y_row_stride=255),
    dict(y_head_stride=0), dict(y=PTR, y_row_stride=512),                     # in place, but elsewhere
    dict(T=(1 << 23) - 1, heads=65536, head_dim=1024, rotary_dim=64, y_head_stride=1024, y_row_stride=1 << 26)])
def test_rope_rejects(L, bad):
    assert L.cider_rope(ctypes.byref(rope_args(**bad)), NULL) == INV


def test_rope_empty_and_null(L):
    assert L.cider_rope(NULL, NULL) == INV
    none = dict(x=None, y=None, positions=None, inv_freq=None)
    assert L.cider_rope(ctypes.byref(rope_args(T=0, **none)), NULL) == 0
    assert L.cider_rope(ctypes.byref(rope_args(heads=0, **none)), NULL) == 0


def append_args(cache_kw=None, **kw):
    a = dict(cache=cache(**(cache_kw or {})), q=PTR, k=PTR, v=PTR, q_norm=PTR, k_norm=PTR, positions=PTR, inv_freq=PTR,
             slots=PTR, q_out=PTR * 2, T=4, q_row_stride=512, q_head_stride=128, k_row_stride=256, k_head_stride=128,
             v_row_stride=256, v_head_stride=128, out_row_stride=512, out_head_stride=128, dtype=0, q_heads=4, rotary_dim=128,
             interleaved=0, rope_scale=1.0, eps=1e-6)
    a.update(kw)
    return cider.Kv4Append(**a)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 23), dict(q_heads=0), dict(q_heads=-1), dict(q_heads=16385), dict(dtype=2), dict(q=None),
    dict(q_out=None), dict(q=None, q_out=None), dict(k=None), dict(v=None), dict(slots=None), dict(positions=None),
    dict(inv_freq=None), dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=-16),
    dict(interleaved=2), dict(rope_scale=float("nan")), dict(eps=0.0), dict(eps=1e-40), dict(eps=float("inf")), dict(eps=float("nan")),
    dict(q=PTR + 8), dict(k=PTR + 8), dict(v=PTR + 2), dict(q_norm=PTR + 8), dict(k_norm=PTR + 8), dict(positions=PTR + 4),
    dict(inv_freq=PTR + 8), dict(slots=PTR + 4), dict(q_out=PTR + 8), dict(k_row_stride=252), dict(v_head_stride=-128),
    dict(q_row_stride=516), dict(out_row_stride=504), dict(out_head_stride=64), dict(q_out=PTR, out_row_stride=1024)])
def test_append_rejects(L, bad):
    assert L.cider_kv4_append(ctypes.byref(append_args(**bad)), NULL) == INV


@pytest.mark.parametrize("bad", BAD_CACHES + NO_ARRAYS)
def test_append_rejects_caches(L, bad):
    assert L.cider_kv4_append(ctypes.byref(append_args(bad)), NULL) == INV


def test_append_empty_and_null(L):
    assert L.cider_kv4_append(NULL, NULL) == INV
    none = dict(q=None, k=None, v=None, q_norm=None, k_norm=None, positions=None, inv_freq=None, slots=None, q_out=None)
    empty = dict(k_codes=None, k_scale=None, v_codes=None, v_scale=None)
    assert L.cider_kv4_append(ctypes.byref(append_args(empty, T=0, **none)), NULL) == 0
    assert L.cider_kv4_append(ctypes.byref(append_args(dict(page_size=17), T=0, **none)), NULL) == INV


def test_read_rejects(L):
    def read(c=None, slots=PTR, n=4, k=PTR, v=PTR, dt=0):
        return L.cider_kv4_read(ctypes.byref(cache(**(c or {}))), slots, n, k, v, dt, NULL)
    for bad in BAD_CACHES + NO_ARRAYS:
        assert read(bad) == INV, bad
    assert L.cider_kv4_read(NULL, PTR, 4, PTR, PTR, 0, NULL) == INV
    assert read(n=-1) == INV and read(n=1 << 31) == INV and read(dt=2) == INV
    for bad in (dict(slots=NULL), dict(k=NULL), dict(v=NULL), dict(slots=PTR + 4), dict(k=PTR + 8), dict(v=PTR + 8)):
        assert read(**bad) == INV, bad
    assert read(NO_ARRAYS[0], slots=NULL, n=0, k=NULL, v=NULL) == 0


def attend_args(cache_kw=None, **kw):
    a = dict(cache=cache(**(cache_kw or {})), q=PTR, page_table=PTR, lengths=PTR, query_offsets=None, y=PTR * 2,
             workspace=PTR * 8, workspace_bytes=1 << 40, T=4, B=4, max_pages=64, q_row_stride=512, q_head_stride=128,
             dtype=0, q_heads=4, causal=1, window=0, softmax_scale=0.1)
    a.update(kw)
    return cider.Kv4Attention(**a)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 31), dict(B=0), dict(B=-1), dict(B=3), dict(B=1 << 31), dict(max_pages=-1), dict(max_pages=1 << 27),
    dict(q_heads=0), dict(q_heads=3), dict(q_heads=16386), dict(dtype=2), dict(causal=2), dict(causal=-1), dict(window=-1),
    dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf")), dict(q=None), dict(y=None), dict(lengths=None),
    dict(page_table=None), dict(q=PTR + 8), dict(y=PTR + 8), dict(lengths=PTR + 4), dict(page_table=PTR + 4),
    dict(query_offsets=PTR + 4), dict(workspace=PTR + 4), dict(workspace=None), dict(workspace_bytes=16),
    dict(q_row_stride=-8), dict(q_row_stride=516), dict(q_head_stride=100), dict(T=1 << 30, B=1 << 30),
    dict(max_pages=(1 << 26) + 1)])
def test_attention_rejects(L, bad):
    assert L.cider_kv4_attention(ctypes.byref(attend_args(**bad)), NULL) == INV


@pytest.mark.parametrize("bad", BAD_CACHES + NO_ARRAYS)
def test_attention_rejects_caches(L, bad):
    assert L.cider_kv4_attention(ctypes.byref(attend_args(bad)), NULL) == INV


def test_attention_empty_and_null(L):
    assert L.cider_kv4_attention(NULL, NULL) == INV
    none = dict(q=None, page_table=None, lengths=None, y=None, workspace=None, workspace_bytes=0)
    assert L.cider_kv4_attention(ctypes.byref(attend_args(NO_ARRAYS[0], T=0, **none)), NULL) == 0


def test_attention_workspace_query(L):
    q = L.cider_kv4_attention_workspace_size
    assert q(0, 4, 16, 8, 128, 4096) == 0
    assert q(1, 1, 16, 8, 128, 0) == 0 and q(1, 1, 16, 8, 128, 128) == 0      # one part: no partial results
    one = q(1, 1, 16, 8, 128, 4096)
    assert one > 0 and one % 16 == 0
    assert q(1, 1, 16, 8, 128, 1 << 20) >= one                                # more tokens, more parts
    many = q(512, 1, 16, 8, 128, 1 << 16)                                     # partial rows of 128 averages, m and l
    assert many > 0 and many % (512 * 16 * 130 * 4) == 0
    for bad in ((-1, 1, 16, 8, 128, 64), (1, 0, 16, 8, 128, 64), (1, 1, 15, 8, 128, 64), (1, 1, 16, 0, 128, 64),
                (1, 1, 16, 8, 96, 64), (1, 1, 16, 8, 128, -1), (1, 1, 16, 8, 128, 1 << 31), (1 << 31, 1, 16, 8, 128, 64),
                (1 << 28, 1, 16, 8, 128, 64), (1, 1, 16, 8, 128, (1 << 30) + 16), ((1 << 26) + 1, 1 << 26, 16, 8, 128, 64)):
        assert q(*bad) == -1, bad
    with pytest.raises(ValueError):
        cider.cider_kv4_attention_workspace_size(1, 1, 16, (1 << 32) + 8, 128, 64)


@pytest.mark.parametrize("name,struct", [("cider_rope_t", cider.Rope), ("cider_kv4_cache_t", cider.Kv4CacheArrays),
                                         ("cider_kv4_append_t", cider.Kv4Append),
                                         ("cider_kv4_attention_t", cider.Kv4Attention)])
def test_structs_match_the_header(name, struct):
    with open(cider.HEADER_PATH) as f:
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, f.read()).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields, sizes = [], {"int64_t": 8, "int32_t": 4, "float": 4, "cider_kv4_cache_t": 56}
    for decl in body.split(";"):
        if decl.strip():
            words = re.match(r"\s*(?:const )?(\w+)(.*)", decl, re.S)
            for one in words.group(2).split(","):
                fields.append((one.strip(" *\n"), 8 if "*" in one else sizes[words.group(1)]))
    assert [n for n, _ in fields] == [f[0] for f in struct._fields_]
    assert [s for _, s in fields] == [ctypes.sizeof(f[1]) for f in struct._fields_]


def test_frequencies():
    pytest.importorskip("torch")
    f, s = cider.rope_frequencies(64, base=10000.0, device="cpu")
    assert s == 1.0 and f.numel() == 32 and f[0] == 1.0 and math.isclose(f[31], 10000.0 ** (-62 / 64), rel_tol=1e-15)
    lin, s = cider.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert s == 1.0 and bool((lin * 4 == f).all())
    # the slowest pair turns factor times slower, the fastest as before
    b, s = cider.rope_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert s == 1.0 and b[0] == 1.0 and math.isclose(b[31], float(f[31]) / 4, rel_tol=1e-12)
    p, s = cider.rope_frequencies(64, scaling="parts", factor=16.0, trained=4096, device="cpu")
    assert math.isclose(s, 0.1 * math.log(16) + 1)
    turns = f * 4096 / (2 * math.pi)
    assert bool((p[turns > 34] == f[turns > 34]).all())
    slow = turns < 0.7
    assert bool(slow.any()) and bool(((p[slow] * 16 - f[slow]).abs() <= 1e-12 * f[slow]).all())
    assert bool((p <= f).all()) and bool((p >= f / 16 * (1 - 1e-12)).all()) and bool((p[1:] < p[:-1]).all())
    assert cider.rope_frequencies(2, scaling="base", factor=4.0, device="cpu")[0].tolist() == [1.0]
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, factor=0.5),
                dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, scaling="parts", fast=1.0, slow=2.0),
                dict(rotary_dim=8, factor=float("nan"))):
        with pytest.raises(ValueError):
            cider.rope_frequencies(device="cpu", **bad)
