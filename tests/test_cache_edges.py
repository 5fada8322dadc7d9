"""Cached attention without a GPU: sizes at the edge of what the calls take."""

import os
import re
import sys

import pytest
import torch

import precision_attention_video_b200 as pav
from precision_attention_video_b200 import build as build_module
from precision_attention_video_b200 import cache as C


def params(**kw):
    base = dict(n_pages=10, page_size=16, H=32, Hkv=8, d=128, S=2, T=2000, max_pages=400, n_select=16)
    base.update(kw)
    return pav.make_cache_params(**base)


def test_workspace_has_no_logits_where_the_choice_refuses_the_sizes():
    # what sparse attention and append need is there; 2000 rows of 65536 pages
    # would have taken 33 GB of logits that no call can use
    lists = pav.cache_workspace_bytes(params(n_select=16, max_pages=16385))
    for kw in (dict(max_pages=65536), dict(max_pages=1 << 26), dict(max_pages=16384, H=8 * 129)):
        n = pav.cache_workspace_bytes(params(**kw))
        assert 0 < n < 1 << 29, kw
    assert lists < pav.cache_workspace_bytes(params(max_pages=16384))


def test_workspace_of_a_long_prompt_is_bounded():
    # logits for 4 GiB of rows at a time; beside them what grows with the rows
    # is some ten bytes a (row, head), and with the table the split means
    short, long = params(T=2000, max_pages=512), params(T=100000, max_pages=512)
    assert pav.cache_workspace_bytes(short) < 1 << 29
    assert pav.cache_workspace_bytes(long) < (1 << 32) + 100000 * (32 * 4 + 8 * 8 + 8) + (1 << 26)
    wide = params(T=4000, max_pages=16384)
    assert pav.cache_workspace_bytes(wide) < (1 << 32) + 2 * 8 * 16384 * 520 + (1 << 26)
    # a token a sequence: no split means
    assert pav.cache_workspace_bytes(params(T=3000, S=3000, max_pages=16384)) < (1 << 32) + (1 << 26)


# ---- without the C++ entry ----
def without_entry(monkeypatch):
    monkeypatch.setitem(sys.modules, "precision_attention_video_b200._cache_call", None)
    monkeypatch.delattr(pav, "_cache_call", raising=False)
    monkeypatch.setattr(C, "_call", None)


def test_the_library_is_built_where_the_entry_is_not(monkeypatch, tmp_path, capfd):
    # torch's C++ headers or Python's are missing: the library needs neither
    def fails():
        raise RuntimeError("compiler failed on ta_cache_py.cpp")

    old = tmp_path / "_cache_call.so"
    old.write_bytes(b"of another library")
    os.utime(old, (1, 1))
    monkeypatch.setattr(build_module, "CALL", str(old))
    monkeypatch.setattr(build_module, "_build_call", fails)
    assert build_module.build() == build_module.LIB and os.path.exists(build_module.LIB)
    assert not old.exists() and "_cache_call.so is not built" in capfd.readouterr().err


def test_calls_without_the_entry_are_checked_in_python(monkeypatch):
    without_entry(monkeypatch)
    p = params(T=2, max_pages=4)
    c = pav.make_cache(p, "cpu")
    Q, ws = torch.zeros(2, 32, 128, dtype=torch.bfloat16), torch.zeros(16, dtype=torch.uint8)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="through ctypes"):
        with pytest.raises(ValueError, match="expected CUDA tensors"):
            pav.cache_decode(p, c, Q, table, lens, ws, Q)
    with pytest.raises(ValueError, match="expected CUDA tensors"):    # (and once only)
        pav.cache_select(p, c, Q, table, lens, ws, table)


# ---- a cache's tensors ----
def test_the_tensors_of_a_cache_cannot_be_exchanged():
    # calls would go on reading the old ones, which nothing holds any more
    c = pav.make_cache(params(), "cpu")
    for name in ("k", "v", "k_scale", "v_scale", "k_mean"):
        with pytest.raises(AttributeError, match="make a new PagedCache"):
            setattr(c, name, torch.zeros(1))
    c.k[0] = 1.0                                     # (their values may)
    c.k *= 2
    assert c.k[0, 0, 0, 0] == 2 and pav.PagedCache(None, None, k_mean=c.k_mean).k is None


# ---- constants of the page choice ----
CSRC = os.path.join(os.path.dirname(os.path.abspath(build_module.__file__)), "csrc")


def test_the_bound_of_the_fast_logits_covers_its_parts():
    # f16 parts of the means and the queries, fp32 sums of 64 products, the join
    # of two sums and two scales (d = 128, the larger of the two)
    with open(os.path.join(CSRC, "ta_cache.cu")) as f:
        err = float(re.search(r"kLogitErr = ([0-9.e-]+)f;", f.read()).group(1))
    u = 2.0 ** -24
    parts = 2.0 ** -22 + 2 * 128 ** 0.5 * 2.0 ** -25 + 4 * 17 * u + 3 * u
    assert parts <= err <= 1.05 * parts
