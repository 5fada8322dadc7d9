"""Cached attention without a GPU: sizes at the edge of what the calls take."""

import functools
import math
import os
import random
import re
import sys
from decimal import Decimal, getcontext
from fractions import Fraction

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


@functools.cache
def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def exp_down(x):
    """The fp64 exponential of the page choice, step by step, its constants read
    from the source.  fma as the product's and the sum's exact value, rounded
    once."""
    body = source("ta_cache.cu")
    body = body[body.index("double exp_down("):]
    body = re.sub(r"//[^\n]*", "", body[:body.index("\n}\n")])
    magic, low, inv = (float(re.search(p, body).group(1)) for p in (
        r"magic = ([0-9.]+);", r"fmax\(x, (-[0-9.]+)\)", r"fma\(y, ([0-9.]+), magic\)"))
    ln2 = [float.fromhex(h) for h in re.findall(r"fma\(n, (-0x[0-9a-f.]+p-?[0-9]+), \w\)", body)]
    tail = [float(a) / float(b) for a, b in re.findall(r"([0-9.]+) / ([0-9.]+)", body)]
    assert len(ln2) == 2 and tail == [1 / 720, 1 / 120, 1 / 24, 1 / 6]
    fma = lambda a, b, c: float(Fraction(a) * Fraction(b) + Fraction(c))  # noqa: E731
    y = max(x, low)
    z = fma(y, inv, magic)
    n = z - magic
    k, e = int(n) & 31, int(n) >> 5
    r = fma(n, ln2[1], fma(n, ln2[0], y))
    p = fma(r, tail[0], tail[1])
    for c in (*tail[2:], 0.5, 1.0):
        p = fma(r, p, c)
    t = math.exp2(k / 32)
    v = fma(t * r, p, t)
    return v * 2.0 ** (e >> 1) * 2.0 ** (e - (e >> 1))


def test_the_fp64_exponential_is_right_to_about_a_unit():
    # against e^x in 50 digits; below 2^-1022 half a subnormal step comes on top
    getcontext().prec = 50
    rng = random.Random(0)
    xs = [-rng.uniform(0, 1) for _ in range(500)] + [-rng.uniform(0, 708) for _ in range(1500)] + \
        [-j * math.log(2) / 32 for j in range(0, 2000, 7)] + [-2.0 ** -k for k in range(60)]
    worst = 0.0
    for x in xs:
        want = Decimal(x).exp()
        unit = Decimal(math.ulp(float(want)))
        worst = max(worst, float(abs(Decimal(exp_down(x)) - want) / unit))
    assert worst <= 1.25, worst
    assert exp_down(0.0) == 1.0 and exp_down(-745.5) == exp_down(-900.0) == exp_down(-1e30) == 0.0
    for x in (-710.0, -730.3, -744.0):
        assert abs(exp_down(x) - math.exp(x)) <= 2 * 5e-324
