"""Cached attention where its numbers leave the ordinary range: page choices
whose border masses no float holds, queries whose squares underflow, more
rows than have their logits in the workspace at a time; calls without the C++
entry; keys and queries of very different magnitudes; rotated keys that no
float holds; results over the queries; positions and lengths out
of range; sizes at the ends of their ranges; frames whose tokens see each other."""

import numpy as np
import pytest
import torch

from oracle import cache as OC
from test_gpu_cache import BF, DEV, Step, check_some, np64, pav

pytestmark = pytest.mark.gpu


def same_choice(st):
    """The lists of `st` are fp64's."""
    want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps,
                     st.p.n_select, st.p.n_first, st.p.n_recent, st.scale)
    np.testing.assert_array_equal(st.select().cpu().numpy(), want)
    assert st.status() == 0


def set_logits(st, logits):
    """Page j's logit for query head g of each key head is logits[j][g] (nats),
    for a query of ones: head g reads element g alone."""
    mean = torch.zeros(st.P, st.Hkv, st.d, dtype=torch.float64)
    for j, row in enumerate(logits):
        mean[st.table[0][j], :, :st.G] = torch.as_tensor(row, dtype=torch.float64) / st.scale
    st.cache.k_mean.copy_(mean)
    st.Q.zero_()
    for h in range(st.H):
        st.Q[:, h, h % st.G] = 1.0


# ---- masses at the border that a float holds as 0, or in few bits ----
@pytest.mark.parametrize("d", [64, 128])
def test_select_masses_that_no_float_holds(cuda_ok, d):
    # in log2: page 3's two terms lie below the smallest normal float and their
    # sum above page 2's one term, which does not
    st = Step([(4 + 12) * 16], [800], H=4, Hkv=2, d=d, ps=16, n_select=5, n_first=1, n_recent=1)
    rows = [(-300.0, -300.0)] * (st.W + 1)
    rows[1:5] = (0.0, 0.0), (-100.0, -100.0), (-125.8, -400.0), (-126.2, -126.2)
    set_logits(st, np.array(rows[:st.W]) * np.log(2.0))
    same_choice(st)


@pytest.mark.parametrize("pages", [60, 900, 3000])
@pytest.mark.parametrize("G", [2, 8])
def test_select_borders_far_below_the_greatest_page(cuda_ok, G, pages):
    # one page far above all others, whose heads' logits differ by nats around
    # where a float's terms vanish, and rows whose queries differ in length
    st = Step([pages * 16], [300], H=8 * G, Hkv=8, d=64, ps=16, n_select=12, seed=pages + G)
    logits = -75.0 - 20.0 * torch.rand(st.W, G, generator=st.g, dtype=torch.float64)
    logits[7] = 0.0
    set_logits(st, logits)
    st.Q *= (1.0 + torch.randint(-16, 17, (st.T, 1, 1), generator=st.g) / 128.0).to(BF).to(st.Q.device)
    same_choice(st)


# ---- queries whose squares underflow ----
@pytest.mark.parametrize("ek,eq", [(90, -90), (100, -100)])
@pytest.mark.parametrize("near", [1e-6, 1e-5])
def test_select_near_ties_of_tiny_queries(cuda_ok, near, ek, eq):
    # logits of hundreds as the product of tiny queries and huge means, with
    # pages that differ by no more than the fast sums' error
    st = Step([3000], [800], H=8, Hkv=4, ps=16, n_select=12, seed=19)
    base = torch.randn(3, 1, st.Hkv, st.d, generator=st.g)
    mean = base[torch.randint(0, 3, (st.P,), generator=st.g), 0]
    mean = mean + near * torch.randn(st.P, st.Hkv, st.d, generator=st.g)
    st.cache.k_mean.copy_(8 * mean * 2.0 ** ek)
    st.Q *= 8 * 2.0 ** eq
    same_choice(st)


# ---- more rows than have their logits in the workspace at a time ----
@pytest.mark.parametrize("old,new,kw", [
    # the fast choice: 256 rows at a time, tiles of 8 rows
    ([900, 0, 40, 3, 500], [130, 300, 0, 1, 270], dict(H=128, Hkv=8, d=64, n_select=5)),
    # fp64, two rows a tile, single rows among them
    ([150] * 400, [2] * 200 + [1] * 200, dict(H=128, Hkv=32, d=64, n_select=6, pad=2)),
    # fp64, a row a sequence
    (list(range(300)), [1] * 300, dict(H=128, Hkv=32, d=64, n_select=4)),
])
def test_select_in_parts(cuda_ok, old, new, kw):
    st = Step(old, new, ps=16, spare=16384 - 100, seed=23, **kw)
    assert 16256 < st.W <= 16384 and st.T * st.H * 16384 * 8 > 1 << 32
    mean = torch.randn(st.P, st.Hkv, st.d, generator=st.g)
    st.cache.k_mean.copy_(mean)
    n = pav().cache_workspace_bytes(st.p)
    assert n < 5 << 30
    same_choice(st)
    # and a captured call of them, other lengths in the same buffers
    sel = torch.full((st.T, st.Hkv, st.p.n_select), -2, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pav().cache_select(st.p, st.cache, st.Q, st.t_table, st.t_lens, st.ws, sel, cu=st.t_cu)
    st.lens = [max(n, a - 7) for a, n in zip(st.lens, st.new)]
    st.t_lens.copy_(torch.tensor(st.lens, dtype=torch.int32))
    sel.fill_(-2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(sel, st.select())
    same_choice(st)


# ---- without the C++ entry ----
@pytest.mark.filterwarnings("ignore:_cache_call.so is missing")
def test_calls_through_ctypes_give_the_same_bits(cuda_ok, monkeypatch):
    from test_cache_edges import without_entry

    def step():
        st = Step([70, 0, 300], [30, 9, 1], rot=64, inter=True, fp8=True, seed=5, pad=2)
        cos, sin = st.tables(400)
        Qr = torch.full_like(st.Q, 7.0)
        st.append(cos, sin, pos=torch.arange(st.T, dtype=torch.int32, device=DEV), Q_out=Qr)
        sel = st.select()
        one = Step([900, 0], [0, 0], seed=6, cu=False)
        return (Qr, st.cache.k.view(torch.uint8), st.cache.k_scale, st.cache.k_mean, sel, *st.sparse(sel),
                *one.decode())

    with_entry = step()
    without_entry(monkeypatch)
    for a, b in zip(with_entry, step()):
        assert torch.equal(a.nan_to_num(9) if a.is_floating_point() else a,
                           b.nan_to_num(9) if b.is_floating_point() else b)


# ---- keys and queries of very different magnitudes ----
@pytest.mark.parametrize("up", [-100, 100, 116])
@pytest.mark.parametrize("fp8", [False, True])
def test_scores_of_huge_keys_and_tiny_queries(cuda_ok, fp8, up):
    # the scores are ordinary; neither factor of theirs is
    def scaled(st):
        if fp8:
            st.cache.k_scale *= 2.0 ** up
        else:
            st.cache.k *= 2.0 ** up
        st.Q *= 2.0 ** -up
        return st

    st = scaled(Step([700, 65, 3000], [0, 0, 0], fp8=fp8, seed=81, cu=False))
    st.check(*st.decode())
    st = Step([100, 40], [300, 333], H=16, Hkv=4, fp8=fp8, n_select=5, seed=82)
    st.append()
    scaled(st)
    lists = torch.randint(-1, 8, (st.T, 4, 5), generator=st.g, dtype=torch.int32)
    O, lse = st.sparse(lists.to(DEV))
    check_some(st, O, lse, lists.tolist(), every=7)
    assert st.status() == 0


# ---- rotated keys that fp32 does not hold ----
@pytest.mark.parametrize("inter", [False, True])
def test_append_fp8_keys_beyond_floats(cuda_ok, inter):
    # bf16 holds 3e38, and a pair of them turned by 45 degrees is 4.2e38: a
    # token that is not finite (its scale is NaN); 2.2e38 still is
    st = Step([0], [6], fp8=True, H=2, Hkv=1, d=64, ps=16, rot=64, inter=inter, seed=12)
    st.K[1], st.K[2], st.K[3] = 3e38, 2.2e38, -3e38
    cos = torch.full((8, 32), 0.5 ** 0.5, device=DEV)
    k, v, ks, vs = st.arrays()
    OC.append(k, v, ks, vs, None, np64(st.K), np64(st.V), st.lens, st.cu, st.table, np64(cos), np64(cos),
              inter, fp8=True)
    st.append(cos, cos)
    k2, v2, ks2, vs2 = st.arrays()
    pg = st.table[0][0]
    assert np.isnan(ks[pg, 0, [1, 3]]).all() and np.isfinite(ks[pg, 0, [0, 2, 4, 5]]).all()
    np.testing.assert_array_equal(ks2, ks)
    np.testing.assert_array_equal(vs2, vs)
    np.testing.assert_array_equal(v2, v)
    for r in (0, 2, 4, 5):
        np.testing.assert_array_equal(k2[pg, 0, r], k[pg, 0, r])


# ---- results over the queries ----
def test_sparse_does_not_write_over_its_queries(cuda_ok):
    # rows with a hidden value that is not finite are done again from their
    # queries: O on top of them is refused
    st = Step([0], [800], H=8, Hkv=8, d=64, ps=16, n_select=3, seed=7)
    st.append()
    lists = torch.randint(0, 50, (800, 8, 3), generator=st.g, dtype=torch.int32)
    with pytest.raises(pav().TieredAttnError, match="invalid argument"):
        pav().cache_sparse(st.p, st.cache, st.Q, lists.to(DEV), st.t_table, st.t_lens, st.ws, st.Q, cu=st.t_cu)


# ---- the fast choice at every width of the table ----
@pytest.mark.parametrize("W", [240, 700, 3000, 9000])
@pytest.mark.parametrize("near", [1e-4, 1e-6])
def test_select_near_ties_at_every_width(cuda_ok, near, W):
    st = Step([3000, 500], [400, 100], ps=16, n_select=12, H=12, Hkv=3, seed=29, spare=W - 213)
    assert st.W == W
    base = torch.randn(3, 1, st.Hkv, st.d, generator=st.g)
    mean = base[torch.randint(0, 3, (st.P,), generator=st.g), 0]
    st.cache.k_mean.copy_(mean + near * torch.randn(st.P, st.Hkv, st.d, generator=st.g))
    same_choice(st)


def test_select_many_rows_of_more_than_8192_pages(cuda_ok):
    st = Step([9000 * 16], [100], H=32, Hkv=8, d=64, ps=16, n_select=24, seed=30)
    st.cache.k_mean.copy_(torch.randn(st.P, st.Hkv, st.d, generator=st.g))
    same_choice(st)


# ---- positions and lengths out of range ----
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_append_positions_outside_the_angles(cuda_ok, fp8, given):
    # rows 3 and 20: their slots stay as they were, and their pages' means count that
    st = Step([10], [60], ps=16, d=64, rot=64, fp8=fp8, seed=31)
    cos, sin = st.tables(70)
    pos = torch.arange(10, 70, dtype=torch.int32)
    bad = [3, 20] if given else [58, 59]
    if given:
        pos[3], pos[20] = -1, 70
    else:
        cos, sin = cos[:68].contiguous(), sin[:68].contiguous()
    if fp8:                                          # (something to count)
        st.cache.k.view(torch.uint8).fill_(0x38)
        st.cache.k_scale.fill_(0.25)
    else:
        st.cache.k.fill_(0.25)
    k, v, ks, vs = st.arrays()
    mean = np64(st.cache.k_mean)
    before = [None if x is None else x.copy() for x in (k, v, ks, vs)]
    clipped = [min(max(int(p), 0), len(cos) - 1) for p in pos]

    def put_back():
        for t in bad:
            pg, slot = st.table[0][(10 + t) // 16], (10 + t) % 16
            for x, b in zip((k, v, ks, vs), before):
                if x is not None:
                    x[pg, :, slot] = b[pg, :, slot]

    OC.append(k, v, ks, vs, None, np64(st.K), np64(st.V), st.lens, st.cu, st.table, np64(cos), np64(sin),
              fp8=fp8, pos=clipped)
    put_back()
    for j in range(4):                               # means of the pages as they now stand
        pg, acc = st.table[0][j], np.zeros((st.Hkv, st.d), np.float32)
        x = OC.decoded(k, ks, fp8)[pg].astype(np.float32)
        for r in range(16):
            acc = acc + x[:, r]
        mean[pg] = acc * np.float32(1 / 16)
    Qr = torch.full_like(st.Q, 7.0)
    st.append(cos, sin, pos=pos.to(DEV) if given else None, Q_out=Qr)
    torch.cuda.synchronize()
    assert st.status() == pav().TA_ERR_BAD_INDEX
    for a, b in zip(st.arrays(), (k, v, ks, vs)):
        if a is not None:
            np.testing.assert_array_equal(a, b)
    np.testing.assert_array_equal(np64(st.cache.k_mean), mean)
    for t in range(60):
        want = OC.rotate32(np64(st.Q)[t], np64(cos)[clipped[t]], np64(sin)[clipped[t]], False)
        np.testing.assert_array_equal(np64(Qr)[t], 7.0 if t in bad else OC.bf16_rne(np.float64(want)))


@pytest.mark.parametrize("fp8", [False, True])
def test_lengths_are_clamped_to_the_table(cuda_ok, fp8):
    # 10^9 tokens are the 256 of the table's four pages, -3 are none
    st = Step([256, 0], [0, 0], seed=51, cu=False, H=4, Hkv=2, fp8=fp8)
    assert st.W == 4
    want, want_lse = st.decode()
    st.check(want, want_lse)
    st.t_lens.copy_(torch.tensor([10 ** 9, -3], dtype=torch.int32))
    O, lse = st.decode()
    torch.cuda.synchronize()
    assert st.status() == pav().TA_ERR_BAD_INDEX
    assert torch.equal(O, want) and torch.equal(lse, want_lse)
    assert (O[1] == 0).all() and (lse[1] == -float("inf")).all()


# ---- sizes at the ends of their ranges ----
@pytest.mark.parametrize("G", [33, 48, 64, 65, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_large_groups(cuda_ok, fp8, G):
    # up to 128 query heads of a key head: decode, choice of few and many rows,
    # sparse attention of few and many
    kw = dict(H=2 * G, Hkv=2, d=64, ps=16, fp8=fp8, n_select=5)
    st = Step([300, 0, 17], [0, 0, 0], seed=G, cu=False, **kw)
    st.check(*st.decode())
    for old, new in (([200, 90], [1, 2]), ([100, 30], [330, 290])):
        st = Step(old, new, seed=G + 1, **kw)
        st.append()
        same_choice(st)
        lists = torch.randint(-1, st.W + 1, (st.T, 2, 5), generator=st.g, dtype=torch.int32)
        O, lse = st.sparse(lists.to(DEV))
        check_some(st, O, lse, lists.tolist(), every=37)
        assert st.status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_as_many_sequences_as_a_decode_takes(cuda_ok, fp8):
    lens = [(7 * i) % 97 for i in range(2048)]
    st = Step(lens, [0] * 2048, H=2, Hkv=1, d=64, ps=32, fp8=fp8, seed=91, cu=False)
    O, lse = st.decode()
    check_some(st, O, lse, None, every=11)
    assert st.status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_one_page_one_head_one_slot(cuda_ok, fp8):
    # a cache of one page (whose strides say nothing), and its first token
    st = Step([0], [1], H=1, Hkv=1, d=64, ps=16, fp8=fp8, n_select=2, seed=92)
    m = pav()
    c = m.make_cache(m.make_cache_params(n_pages=1, page_size=16, H=1, Hkv=1, d=64, S=1, T=1, max_pages=1,
                                         format=int(fp8)), DEV)
    p = m.make_cache_params(n_pages=1, page_size=16, H=1, Hkv=1, d=64, S=1, T=1, max_pages=1,
                            format=int(fp8), n_select=2)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    ws = m.alloc_cache_workspace(p, DEV)
    O, lse = st.out()
    sel = torch.full((1, 1, 2), -2, dtype=torch.int32, device=DEV)
    m.cache_append(p, c, st.K, st.V, table, st.t_lens, ws)
    m.cache_select(p, c, st.Q, table, st.t_lens, ws, sel)
    m.cache_decode(p, c, st.Q, table, st.t_lens, ws, O, lse=lse)
    assert sel.tolist() == [[[0, -1]]] and m.get_status(ws) == 0
    st.cache, st.table = c, [[0]]
    st.check(O, lse)
    m.cache_sparse(p, c, st.Q, sel, table, st.t_lens, ws, O, lse=lse)
    st.check(O, lse)


def test_steps_without_rows_and_rows_without_pages(cuda_ok):
    # every sequence empty and only padding; then a prompt of which no row lists a page
    st = Step([40, 0], [0, 0], cu=True, pad=700, H=8, Hkv=4, seed=93)
    k = [None if x is None else x.copy() for x in st.arrays()]
    st.append()
    lists = torch.zeros((700, 4, 4), dtype=torch.int32, device=DEV)
    O, lse = st.sparse(lists)
    assert (st.select() == -2).all() and (O == 7).all() and (lse == 7).all()
    for a, b in zip(k, st.arrays()):
        np.testing.assert_array_equal(a, b) if a is not None else None
    st = Step([100, 0], [400, 350], H=16, Hkv=4, seed=94)
    st.append()
    O, lse = st.sparse(torch.full((750, 4, 4), -1, dtype=torch.int32, device=DEV))
    assert (O == 0).all() and (lse == -float("inf")).all() and st.status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_fused_projections_and_a_fused_cache(cuda_ok, fp8):
    # Q, K, V as parts of one row, rotated in place; keys and values of a page
    # next to each other in one tensor
    m = pav()
    st = Step([50, 3], [300, 280], H=16, Hkv=4, d=64, ps=32, rot=64, fp8=fp8, n_select=6, seed=95)
    cos, sin = st.tables(400)
    qkv = torch.cat([x.flatten(1) for x in (st.Q, st.K, st.V)], 1)
    q, k, v = (x.unflatten(1, (-1, 64)) for x in qkv.split([16 * 64, 4 * 64, 4 * 64], 1))
    both = torch.empty((st.P, 2, *st.cache.k.shape[1:]), dtype=torch.uint8 if fp8 else BF, device=DEV)
    both = both.view(st.cache.k.dtype)
    raw = (lambda x: x.view(torch.uint8)) if fp8 else (lambda x: x)
    raw(both)[:, 0], raw(both)[:, 1] = raw(st.cache.k), raw(st.cache.v)
    c = m.PagedCache(both[:, 0], both[:, 1], st.cache.k_scale, st.cache.v_scale, st.cache.k_mean)
    means = st.cache.k_mean.clone()
    m.cache_append(st.p, c, k, v, st.t_table, st.t_lens, st.ws, cu=st.t_cu, cos=cos, sin=sin, Q=q, Q_out=q)
    sel = torch.full((st.T, 4, 6), -2, dtype=torch.int32, device=DEV)
    m.cache_select(st.p, c, q, st.t_table, st.t_lens, st.ws, sel, cu=st.t_cu)
    O, lse = st.out()
    m.cache_sparse(st.p, c, q, sel, st.t_table, st.t_lens, st.ws, O, cu=st.t_cu, lse=lse)
    got = [raw(both[:, 0]).clone(), raw(both[:, 1]).clone(), c.k_mean.clone(), sel, O, lse, q.contiguous()]
    # the same with tensors of their own
    c.k_mean.copy_(means)
    Qr = torch.empty_like(st.Q)
    st.append(cos, sin, Q_out=Qr)
    st.Q = Qr
    want = [raw(st.cache.k), raw(st.cache.v), st.cache.k_mean, st.select()]
    want += [*st.sparse(want[3]), Qr]
    for a, b in zip(got, want):
        a, b = (x.nan_to_num(9) if x.is_floating_point() else x for x in (a, b))
        assert torch.equal(a, b)
    check_some(st, O, lse, sel.tolist(), every=17)


# ---- a frame whose tokens see each other ----
@pytest.mark.parametrize("fp8", [False, True])
def test_a_frame_whose_tokens_see_each_other(cuda_ok, fp8):
    # appended as rows of its sequence, then a sequence for each row
    m = pav()
    st = Step([300], [90], H=8, Hkv=4, ps=32, rot=128, fp8=fp8, n_select=6, seed=96)
    cos, sin = st.tables(400)
    st.append(cos, sin, Q_out=st.Q)
    st.p = m.make_cache_params(n_pages=st.P, page_size=32, H=8, Hkv=4, d=128, S=90, T=90, max_pages=st.W,
                               format=int(fp8), n_select=6)
    st.S, st.cu, st.t_cu = 90, None, None
    st.lens, st.t_lens = st.lens * 90, st.t_lens.repeat(90)
    st.table, st.t_table = st.table * 90, st.t_table.repeat(90, 1)
    st.ws = m.alloc_cache_workspace(st.p, DEV)
    st.check(*st.decode())
    same_choice(st)
    sel = st.select()
    O, lse = st.sparse(sel)
    st.check(O, lse, sel.tolist())
    assert st.status() == 0
