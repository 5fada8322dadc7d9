"""Cached attention without a GPU: the C ABI's validation, the layout of its
structures, the binding's refusals, and the oracle on cases worked by hand."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import precision_attention_video_b200 as pav
from oracle import cache as OC
from precision_attention_video_b200 import binding as B
from precision_attention_video_b200 import cache as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def params(**kw):
    base = dict(n_pages=10, page_size=64, H=8, Hkv=2, d=128, S=2, T=2, max_pages=4, n_select=3,
                rot_dim=128)
    base.update(kw)
    return pav.make_cache_params(**base)


def test_workspace_bytes_and_what_is_refused():
    n = pav.cache_workspace_bytes(params())
    assert n > 0 and n % 256 == 0
    # the fixed part does not depend on the parameters; page choice adds its logits
    assert pav.cache_workspace_bytes(params(n_select=0)) == \
        pav.cache_workspace_bytes(params(n_select=0, T=700, S=700, max_pages=900))
    assert pav.cache_workspace_bytes(params(T=1000)) >= n + 998 * 8 * 4 * 8
    bad = [dict(n_pages=0), dict(page_size=48), dict(page_size=8), dict(H=7), dict(Hkv=0),
           dict(d=96), dict(d=256), dict(format=2), dict(S=0), dict(T=0), dict(max_pages=0),
           dict(n_select=-1), dict(n_select=2, n_first=2, n_recent=1), dict(n_recent=0),
           dict(n_select=1025), dict(rot_dim=24), dict(rot_dim=144), dict(rot_interleaved=2),
           dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")), dict(max_pages=1 << 26),
           dict(n_first=-1)]
    for kw in bad:
        assert pav.cache_workspace_bytes(params(**kw)) == 0, kw


def call(name, p, *args):
    return C._fn(name)(p, *args)


def test_c_abi_refuses_on_the_host():
    # no pointer here is read: every call returns before any launch
    A = 1 << 20
    p = params()
    for k in ("stride_page", "stride_head", "stride_slot", "stride_k_t", "stride_k_h", "stride_v_t",
              "stride_v_h", "stride_q_t", "stride_q_h", "stride_o_t", "stride_o_h"):
        setattr(p, k, 1024)
    p.stride_table, p.rot_rows = 4, 10
    cache = C.ta_cache(A, A, None, None, A)
    n = pav.cache_workspace_bytes(p)
    INV, UNS, WS = B.TA_ERR_INVALID_ARG, B.TA_ERR_UNSUPPORTED, B.TA_ERR_WORKSPACE

    def append(p=p, cache=cache, k=A, v=A, q=None, qo=None, cos=A, sin=A, lens=A, table=A, ws=A, n=n):
        return call("tiered_attn_cache_append", p, cache, k, v, q, qo, cos, sin, None, None, lens,
                    table, ws, n, None)

    def decode(p=p, cache=cache, q=A, lens=A, table=A, o=A, ws=A, n=n):
        return call("tiered_attn_cache_decode", p, cache, q, lens, table, o, None, ws, n, None)

    def select(p=p, cache=cache, q=A, lens=A, table=A, sel=A, ws=A, n=n):
        return call("tiered_attn_cache_select", p, cache, q, None, lens, table, sel, ws, n, None)

    def sparse(p=p, cache=cache, q=A, sel=A, lens=A, table=A, o=A, ws=A, n=n):
        return call("tiered_attn_cache_sparse", p, cache, q, sel, None, lens, table, o, None, ws, n, None)

    def other(**kw):
        r = C.ta_cache_params.from_buffer_copy(p)
        for k, v in kw.items():
            setattr(r, k, v)
        return r

    for f in (append, decode, select, sparse):
        assert f(p=other(d=80)) == UNS
        assert f(p=other(H=9)) == INV
        assert f(lens=None) == INV and f(table=A + 2) == INV
        assert f(ws=None) == INV and f(ws=A + 16) == INV and f(n=100) == WS
        assert f(p=other(T=3)) == INV                      # cu = NULL: one row a sequence
        assert f(p=other(stride_table=3)) == INV
    for f in (append, decode, sparse):
        assert f(cache=C.ta_cache(None, A, None, None, A)) == INV
        assert f(cache=C.ta_cache(A, A + 8, None, None, A)) == INV
        assert f(p=other(format=1)) == INV                 # no scales
        assert f(p=other(stride_slot=120)) == INV and f(p=other(stride_slot=132)) == INV
        assert f(p=other(stride_head=1028)) == INV and f(p=other(stride_page=4)) == INV
    for f in (decode, select, sparse):
        assert f(q=None) == INV and f(q=A + 4) == INV and f(p=other(stride_q_t=1028)) == INV
    for f in (decode, sparse):
        assert f(o=None) == INV and f(p=other(stride_o_h=4)) == INV
    assert append(k=None) == INV and append(v=A + 2) == INV and append(cos=None) == INV
    assert append(sin=A + 4) == INV and append(q=A) == INV and append(q=A, qo=A + 2) == INV
    assert append(cache=C.ta_cache(A, A, None, None, A + 4)) == INV
    assert select(cache=C.ta_cache(None, None, None, None, None)) == INV
    assert select(sel=None) == INV and select(n=n - 256) == WS
    assert select(p=other(n_select=0)) == INV and sparse(p=other(n_select=0)) == INV
    assert select(p=other(max_pages=16385, stride_table=16385), n=1 << 40) == UNS
    assert select(p=other(S=70000, T=70000), n=1 << 50) == UNS
    assert select(p=other(H=258, Hkv=2), n=1 << 50) == UNS
    assert decode(p=other(S=5000, T=5000)) == UNS
    assert sparse(sel=None) == INV
    assert C._fn("tiered_attn_cache_init")(None, 1 << 30, None) == INV
    assert C._fn("tiered_attn_cache_init")(A, 256, None) == WS


def test_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    lines = ['#include <stdio.h>', '#include "tiered_attn_cache.h"', 'int main(void) {']
    for struct, cls in (("ta_cache_params", C.ta_cache_params), ("ta_cache", C.ta_cache)):
        lines.append(f'  printf("{struct} %zu\\n", sizeof({struct}));')
        for name, _ in cls._fields_:
            lines.append(f'  printf("{struct}.{name} %zu\\n", offsetof({struct}, {name}));')
    for c in ("TA_CACHE_BF16", "TA_CACHE_FP8", "TA_ERR_BAD_INDEX"):
        lines.append(f'  printf("{c} %d\\n", (int){c});')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\n  return 0;\n}\n")
    for comp, std, ext in ((cc, "-std=c99", "c"), (shutil.which("g++") or cc, "-std=c++17", "cpp")):
        f = tmp_path / f"layout.{ext}"
        f.write_text(src.read_text())
        subprocess.run([comp, std, "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(ROOT, "include"), str(f), "-o", str(tmp_path / "layout")],
                       check=True, capture_output=True)
        out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True)
        got = dict(line.split() for line in out.stdout.splitlines())
        for struct, cls in (("ta_cache_params", C.ta_cache_params), ("ta_cache", C.ta_cache)):
            assert int(got[struct]) == ctypes.sizeof(cls)
            for name, _ in cls._fields_:
                assert int(got[f"{struct}.{name}"]) == getattr(cls, name).offset, name
        for c in ("TA_CACHE_BF16", "TA_CACHE_FP8", "TA_ERR_BAD_INDEX"):
            assert int(got[c]) == getattr(C, c)
    assert "out of range" in pav.status_string(C.TA_ERR_BAD_INDEX)


def test_the_binding_refuses_host_and_mis_shaped_caches():
    p = params()
    c = pav.make_cache(p, "cpu")
    assert c.k.shape == (10, 2, 64, 128) and c.k_mean.shape == (10, 2, 128)
    n = pav.make_cache(params(format=1), "cpu", "nhd")
    assert n.k.dtype == torch.float8_e4m3fn and n.k.stride() == (64 * 2 * 128, 128, 2 * 128, 1)
    assert n.k_scale.shape == (10, 2, 64)
    with pytest.raises(ValueError, match="layout"):
        pav.make_cache(p, "cpu", "dhn")
    z = torch.zeros
    ws, Q = z(16, dtype=torch.uint8), z(2, 8, 128, dtype=torch.bfloat16)
    table, lens = z(2, 4, dtype=torch.int32), z(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="expected CUDA tensors"):
        pav.cache_decode(p, c, Q, table, lens, ws, Q)
    with pytest.raises(ValueError, match="neither keys nor means"):
        pav.PagedCache(None, None)
    with pytest.raises(TypeError, match="k: expected torch.bfloat16"):
        pav.PagedCache(c.k.float(), c.v.float())
    with pytest.raises(ValueError, match="equal strides"):
        pav.PagedCache(c.k, pav.make_cache(p, "cpu", "nhd").v)
    with pytest.raises(TypeError, match="v: expected a tensor of k's type"):
        pav.PagedCache(c.k, None)
    with pytest.raises(TypeError, match="k_scale: expected a torch.Tensor"):
        pav.PagedCache(n.k, n.v)
    with pytest.raises(ValueError, match="k_mean: expected a contiguous tensor of shape"):
        pav.PagedCache(c.k, c.v, k_mean=z(10, 2, 64))
    with pytest.raises(TypeError, match="k_mean: expected torch.float32"):
        pav.PagedCache(c.k, c.v, k_mean=z(10, 2, 128, dtype=torch.float64))
    with pytest.raises(pav.TieredAttnError):
        pav.alloc_cache_workspace(params(d=96), "cpu")
    with pytest.raises(ValueError, match="ws: expected a CUDA tensor"):
        pav.init_cache_workspace(ws)


def test_the_native_entry_refuses_without_work():
    # host tensors, wrong kinds of arguments, the wrong number of them: None
    # (the module's own checks then raise), never an exception or a call
    m = C._native()
    p, c = params(), pav.make_cache(params(), "cpu")
    z = torch.zeros
    Q, K = z(2, 8, 128, dtype=torch.bfloat16), z(2, 2, 128, dtype=torch.bfloat16)
    table, lens = z(2, 4, dtype=torch.int32), z(2, dtype=torch.int32)
    ws, sel = z(1 << 20, dtype=torch.uint8), z(2, 2, 3, dtype=torch.int32)
    for args in ((p, c._view, Q, table, lens, ws, Q, None, None), (p, c._view, Q, table), (),
                 (p, c, Q, table, lens, ws, Q, None, None), (b"x", b"y", 1, 2, 3, 4, 5, 6, 7),
                 (p, c._view, None, None, None, None, None, None, "stream")):
        assert m.decode(*args) is None and m.select(*args) is None
    assert m.append(p, c._view, K, K, table, lens, ws, None, None, None, None, None, None, None) is None
    assert m.sparse(p, c._view, Q, sel, table, lens, ws, Q, None, None, None) is None


def test_the_bindings_tensor_checks():
    z = torch.zeros
    with pytest.raises(ValueError, match="lens: expected a tensor on device 0"):
        C._plain("lens", z(2, dtype=torch.int32), torch.int32, (2,), 0)
    with pytest.raises(TypeError, match="lens: expected torch.int32"):
        C._plain("lens", z(2), torch.int32, (2,), -1)
    with pytest.raises(ValueError, match="contiguous tensor of shape"):
        C._plain("lens", z(4, dtype=torch.int32)[::2], torch.int32, (2,), -1)
    with pytest.raises(TypeError, match="Q: expected torch.bfloat16"):
        C._rows("Q", z(2, 8, 128), (2, 8, 128), -1)
    with pytest.raises(ValueError, match="last dimension contiguous"):
        C._rows("Q", z(2, 128, 8, dtype=torch.bfloat16).transpose(1, 2), (2, 8, 128), -1)
    with pytest.raises(ValueError, match="expected shape"):
        C._rows("Q", z(3, 8, 128, dtype=torch.bfloat16), (2, 8, 128), -1)


# ---------------------------------------------------------------------------
# the oracle, by hand
# ---------------------------------------------------------------------------
def test_oracle_rows():
    assert OC.rows_of([5, 0, 3], [0, 2, 2, 5], 3) == [(0, 0, 3), (1, 0, 4), (2, 2, 0), (3, 2, 1), (4, 2, 2)]
    assert OC.rows_of([5, 0], None, 2) == [(0, 0, 4), (1, 1, None)]
    assert OC.rows_of([1], [0, 2], 1) == [(0, 0, None), (1, 0, 0)]


def test_oracle_rotation_quarter_turns():
    x = np.arange(8, dtype=np.float64)
    c, s = np.zeros(2), np.ones(2)                       # 90 degrees, first 4 elements
    for f in (OC.rotate32, OC.rotate64):
        np.testing.assert_array_equal(f(x, c, s, True), [-1, 0, -3, 2, 4, 5, 6, 7])
        np.testing.assert_array_equal(f(x, c, s, False), [-2, -3, 0, 1, 4, 5, 6, 7])


def test_oracle_token_scale():
    assert [OC.token_scale(a) for a in (0.0, 448.0, 449.0, 224.0, 1.0)] == [1, 1, 2, 0.5, 2.0 ** -8]
    assert np.isnan(OC.token_scale(np.inf)) and OC.token_scale(1e-44) == 2.0 ** -126


def test_oracle_append_and_mean():
    k, v = np.zeros((2, 1, 2, 4)), np.zeros((2, 1, 2, 4))
    mean = np.full((2, 1, 4), -1.0)
    K = np.arange(12, dtype=np.float64).reshape(3, 1, 4)
    OC.append(k, v, None, None, mean, K, -K, [4], [0, 3], [[1, 0]])
    np.testing.assert_array_equal(k[1, 0], [[0, 0, 0, 0], [0, 1, 2, 3]])
    np.testing.assert_array_equal(k[0, 0], [[4, 5, 6, 7], [8, 9, 10, 11]])
    np.testing.assert_array_equal(v, -k)
    np.testing.assert_array_equal(mean[0, 0], [6, 7, 8, 9])
    np.testing.assert_array_equal(mean[1, 0], [0, .5, 1, 1.5])


def test_oracle_attention():
    rng = np.random.default_rng(0)
    q, K, V = rng.normal(size=(1, 16)), rng.normal(size=(9, 16)), rng.normal(size=(9, 16))
    o, lse, A, big = OC.attend(q[0], K, V, 0.25)
    s = K @ q[0] * 0.25
    np.testing.assert_allclose(o, np.exp(s) / np.exp(s).sum() @ V, rtol=1e-13)
    assert abs(lse - np.log(np.exp(s).sum())) < 1e-13 and (A >= np.abs(o)).all() and big >= np.abs(s).max()
    o, lse, _, _ = OC.attend(q[0], K[:0], V[:0], 0.25)
    assert not o.any() and lse == -np.inf


def test_oracle_choice_follows_the_mass_routers_order():
    # one query row a block: the pages chosen are the heads of the (-M, j)
    # order of the router's pooled masses
    rng = np.random.default_rng(3)
    n, d = 12, 16
    mean, q = rng.normal(size=(n, 1, d)), rng.normal(size=(1, 1, d))
    mean[7] = mean[3]                                    # a tie
    sel = OC.select(q, mean, [n * 16 + 1], None, [list(range(n)) + [n]], 1, 16, 6, 0, 1, 0.25)
    lg = mean[:, 0] @ q[0, 0] * 0.25
    M = np.exp(lg - lg.max()) / np.exp(lg - lg.max()).sum()
    order = sorted(range(n), key=lambda j: (-M[j], j))[:5]
    assert sel[0, 0].tolist() == sorted(order) + [n]
