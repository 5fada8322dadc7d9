"""Cached attention on the GPU against the plain fp64 oracle: append, decode,
page choice and sparse attention, at the sizes, masks, layouts and lengths
where they can go wrong.  Slots that hold no key, pages of nobody and table
entries behind a sequence's end are poisoned."""

import math

import numpy as np
import pytest
import torch

from oracle import cache as OC

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


def pav():
    import precision_attention_video_b200 as m
    return m


def np64(x):
    if x.dtype == torch.float8_e4m3fn:
        return x.contiguous().view(torch.uint8).cpu().numpy()
    return x.detach().to("cpu", torch.float64).numpy()


class Step:
    """A cache with `old` tokens of each sequence, about to take `new` more."""

    def __init__(self, old, new, H=8, Hkv=2, d=128, ps=64, fp8=False, layout="hnd", seed=0,
                 cu=None, n_select=4, n_first=1, n_recent=1, rot=0, inter=False, pad=0,
                 scale=0.0, spare=0):
        m = pav()
        g = torch.Generator().manual_seed(seed)
        S = len(old)
        self.old, self.new = list(old), list(new)
        self.lens = [a + b for a, b in zip(old, new)]
        use_cu = cu if cu is not None else any(n != 1 for n in new)
        self.cu = [sum(new[:i]) for i in range(S + 1)] if use_cu else None
        T = sum(new) + pad if use_cu else S
        W = max(1, max(-(-n // ps) for n in self.lens)) + spare
        need = [-(-n // ps) for n in self.lens]
        P = sum(need) + 2
        perm = torch.randperm(P, generator=g).tolist()
        self.table = [[2 ** 31 - 1 if j % 2 else -1 for j in range(W)] for _ in range(S)]
        at = 0
        for s in range(S):
            for j in range(need[s]):
                self.table[s][j] = perm[at]
                at += 1
        self.p = m.make_cache_params(n_pages=P, page_size=ps, H=H, Hkv=Hkv, d=d, S=S, T=T,
                                     max_pages=W, format=1 if fp8 else 0, n_select=n_select,
                                     n_first=n_first, n_recent=n_recent, rot_dim=rot,
                                     rot_interleaved=int(inter), softmax_scale=scale)
        self.scale = scale or d ** -0.5
        self.H, self.Hkv, self.G, self.d, self.ps, self.fp8 = H, Hkv, H // Hkv, d, ps, fp8
        self.S, self.T, self.W, self.P, self.rot, self.inter = S, T, W, P, rot, inter
        c = m.make_cache(self.p, DEV, layout)
        # poison, then the old tokens
        nan = 0x7F
        if fp8:
            c.k.view(torch.uint8).fill_(nan)
            c.v.view(torch.uint8).fill_(nan)
            c.k_scale.fill_(float("nan"))
            c.v_scale.fill_(float("nan"))
        else:
            c.k.fill_(float("nan"))
            c.v.fill_(float("nan"))
        c.k_mean.fill_(float("nan"))
        for s in range(S):
            for j in range(-(-self.old[s] // ps)):
                n = min(ps, self.old[s] - j * ps)
                pg = self.table[s][j]
                if fp8:
                    for x, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
                        codes = torch.randint(0, 256, (Hkv, n, d), generator=g, dtype=torch.int32)
                        codes = torch.where((codes & 0x7F) == 0x7F, codes - 8, codes).to(torch.uint8)
                        x.view(torch.uint8)[pg, :, :n] = codes.to(DEV)
                        e = torch.randint(-10, -6, (Hkv, n), generator=g).float()
                        sc[pg, :, :n] = torch.exp2(e).to(DEV)
                else:
                    c.k[pg, :, :n] = torch.randn(Hkv, n, d, generator=g).to(BF).to(DEV)
                    c.v[pg, :, :n] = torch.randn(Hkv, n, d, generator=g).to(BF).to(DEV)
        self.cache = c
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        self.t_table, self.t_lens = i32(self.table), i32(self.lens)
        self.t_cu = i32(self.cu) if self.cu is not None else None
        self.ws = m.alloc_cache_workspace(self.p, DEV)
        self.Q = (2 * torch.randn(T, H, d, generator=g)).to(BF).to(DEV)
        self.K = torch.randn(T, Hkv, d, generator=g).to(BF).to(DEV)
        self.V = torch.randn(T, Hkv, d, generator=g).to(BF).to(DEV)
        self.g = g

    def tables(self, rows):
        inv = 100.0 ** (-np.arange(0, self.rot, 2) / self.rot)
        ang = np.arange(rows)[:, None] * inv
        return (torch.tensor(np.cos(ang), dtype=torch.float32, device=DEV),
                torch.tensor(np.sin(ang), dtype=torch.float32, device=DEV))

    def arrays(self):
        c = self.cache
        ks = np64(c.k_scale) if self.fp8 else None
        vs = np64(c.v_scale) if self.fp8 else None
        return np64(c.k), np64(c.v), ks, vs

    def status(self):
        return pav().get_status(self.ws)

    def out(self):
        rows = torch.full((self.T, self.H, self.d), 7.0, dtype=BF, device=DEV)
        return rows, torch.full((self.T, self.H), 7.0, device=DEV)

    def check(self, O, lse, lists=None):
        """O and lse against the oracle within the bound of the arithmetic:
        O's rounding (2^-8 relative), P's rounding (2^-8 of sum p |v|), the
        scores' errors (d products in fp32 and the scaling, doubled through
        exp), and the fp32 sums over n keys.  FP8: the weights are f16 with
        2^15 for weight 1 at the largest V scale seen (of the sequence at
        most), so half a subnormal step, 2^-25, is 2^-40 of that scale times
        the key's code (448 at most); the sum of weights is 1 or more, since
        the greatest weight is 1: n 2^-40 448 max(scale) on O."""
        kd, vd = self.decoded()
        vs = np64(self.cache.v_scale) if self.fp8 else None
        O, lse, Q = np64(O), np64(lse), np64(self.Q)
        used = set()
        for t, s, pos in OC.rows_of(self.lens, self.cu, self.S):
            used.add(t)
            n = 0 if pos is None else pos + 1
            for h in range(self.H):
                hk = h // self.G
                K, V = OC.keys_of(kd, self.table[s], n, hk), OC.keys_of(vd, self.table[s], n, hk)
                if lists is not None:
                    idx = [i for e in lists[t][hk] if e >= 0
                           for i in range(e * self.ps, min(n, (e + 1) * self.ps))]
                    K, V = K[idx], V[idx]
                o, z, A, big = OC.attend(Q[t, h], K, V, self.scale)
                u = 2.0 ** -24
                ds = (self.d + 8) * big * u
                rest = 2 * ds + (K.shape[0] + 64) * u + 2.0 ** -20
                tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + rest) * A * (1 + 2.0 ** -7)
                if self.fp8 and self.lens[s] > 0:
                    top = OC.keys_of(vs[..., None], self.table[s], self.lens[s], hk).max()
                    tol = tol + K.shape[0] * 2.0 ** -40 * 448 * top
                assert (np.abs(O[t, h] - o) <= tol).all(), (t, h, np.abs(O[t, h] - o).max())
                if math.isinf(z):
                    assert lse[t, h] == z
                else:
                    assert abs(lse[t, h] - z) <= rest + abs(z) * 2.0 ** -22, (t, h, lse[t, h], z)
        for t in range(self.T):
            if t not in used:
                assert (O[t] == 7).all() and (lse[t] == 7).all()

    def decoded(self):
        k, v, ks, vs = self.arrays()
        with np.errstate(invalid="ignore"):
            return OC.decoded(k, ks, self.fp8), OC.decoded(v, vs, self.fp8)

    def append(self, cos=None, sin=None, pos=None, Q_out=None):
        pav().cache_append(self.p, self.cache, self.K, self.V, self.t_table, self.t_lens, self.ws,
                           cu=self.t_cu, cos=cos, sin=sin, pos=pos,
                           Q=None if Q_out is None else self.Q, Q_out=Q_out)

    def decode(self):
        O, lse = self.out()
        pav().cache_decode(self.p, self.cache, self.Q, self.t_table, self.t_lens, self.ws, O, lse=lse)
        return O, lse

    def select(self):
        sel = torch.full((self.T, self.Hkv, self.p.n_select), -2, dtype=torch.int32, device=DEV)
        pav().cache_select(self.p, self.cache, self.Q, self.t_table, self.t_lens, self.ws, sel,
                           cu=self.t_cu)
        return sel

    def sparse(self, sel):
        O, lse = self.out()
        pav().cache_sparse(self.p, self.cache, self.Q, sel, self.t_table, self.t_lens, self.ws, O,
                           cu=self.t_cu, lse=lse)
        return O, lse


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
APPEND = [
    # old, new, kwargs
    ([0], [1], dict()),
    ([63, 64, 0, 5], [1, 1, 1, 1], dict(rot=128)),
    ([0, 10, 130], [200, 0, 7], dict(rot=64, inter=True, pad=3)),
    ([15, 0], [34, 16], dict(ps=16, d=64, rot=64, H=6, Hkv=3, layout="nhd")),
    ([100, 3], [29, 125], dict(ps=128, rot=32, H=4, Hkv=1)),
    ([31, 0, 1], [1, 65, 0], dict(ps=32, d=64, rot=16, inter=True, H=24, Hkv=12)),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_bit_for_bit(cuda_ok, case, fp8):
    old, new, kw = APPEND[case]
    st = Step(old, new, fp8=fp8, seed=case, **kw)
    cos = sin = None
    if st.rot:
        cos, sin = st.tables(max(st.lens) + 1)
    k, v, ks, vs = st.arrays()
    mean = np64(st.cache.k_mean)
    cn, sn = (np64(cos), np64(sin)) if st.rot else (None, None)
    with np.errstate(invalid="ignore"):
        OC.append(k, v, ks, vs, mean, np64(st.K), np64(st.V), st.lens, st.cu, st.table, cn, sn,
                  st.inter, fp8=fp8)
    Qr = torch.full_like(st.Q, 7.0)
    st.append(cos, sin, Q_out=Qr)
    torch.cuda.synchronize()
    assert st.status() == 0
    k2, v2, ks2, vs2 = st.arrays()
    np.testing.assert_array_equal(k2, k)
    np.testing.assert_array_equal(v2, v)
    if fp8:
        np.testing.assert_array_equal(ks2, ks)
        np.testing.assert_array_equal(vs2, vs)
    np.testing.assert_array_equal(np64(st.cache.k_mean), mean)
    q, qr = np64(st.Q), np64(Qr)
    used = set()
    for t, s, p in OC.rows_of(st.lens, st.cu, st.S):
        used.add(t)
        want = OC.rotate32(q[t], cn[p], sn[p], st.inter) if st.rot else q[t]
        np.testing.assert_array_equal(qr[t], OC.bf16_rne(np.float64(want)))
    for t in range(st.T):
        if t not in used:
            assert (qr[t] == 7).all()


def test_append_in_parts_and_after_a_rollback(cuda_ok):
    # the mean of a page depends on its keys alone
    whole = Step([5, 0], [150, 70], rot=128, seed=3)
    cos, sin = whole.tables(200)
    whole.append(cos, sin)
    want = whole.arrays() + (np64(whole.cache.k_mean),)
    parts = Step([5, 0], [150, 70], rot=128, seed=3)
    m = pav()
    first = [0, 150]
    junk = torch.full_like(parts.K[:1], 3.0)
    for lo, hi in ((0, 1), (1, 40), (30, 59), (59, 60), (60, 150)):   # 30..39: taken back, again
        n = [hi - lo, max(0, min(hi, 70) - min(lo, 70))]
        rows = list(range(lo, hi)) + list(range(150 + min(lo, 70), 150 + min(lo, 70) + n[1]))
        K, V = parts.K[rows].clone(), parts.V[rows].clone()
        if (lo, hi) == (1, 40):
            K[29:39] = junk
        p = m.make_cache_params(n_pages=parts.P, page_size=64, H=8, Hkv=2, d=128, S=2,
                                T=len(rows), max_pages=parts.W, n_select=4, rot_dim=128)
        lens = torch.tensor([5 + hi, min(hi, 70)], dtype=torch.int32, device=DEV)
        cu = torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32, device=DEV)
        m.cache_append(p, parts.cache, K, V, parts.t_table, lens, parts.ws, cu=cu, cos=cos, sin=sin)
    assert first and parts.status() == 0
    for a, b in zip(want, parts.arrays() + (np64(parts.cache.k_mean),)):
        if a is not None:
            np.testing.assert_array_equal(a, b)


def test_append_given_positions_and_in_place_queries(cuda_ok):
    for inter in (False, True):
        st = Step([3, 0], [4, 9], rot=128, inter=inter, seed=5, pad=2)
        cos, sin = st.tables(40)
        pos = torch.randint(0, 40, (st.T,), generator=st.g, dtype=torch.int32)
        k, v, _, _ = st.arrays()
        OC.append(k, v, None, None, None, np64(st.K), np64(st.V), st.lens, st.cu, st.table, np64(cos),
                  np64(sin), inter, pos=pos.tolist())
        q = np64(st.Q)
        st.append(cos, sin, pos=pos.to(DEV), Q_out=st.Q)
        assert st.status() == 0
        np.testing.assert_array_equal(st.arrays()[0], k)
        for t in range(13):
            want = OC.rotate32(q[t], np64(cos)[pos[t]], np64(sin)[pos[t]], inter)
            np.testing.assert_array_equal(np64(st.Q)[t], OC.bf16_rne(np.float64(want)))
        np.testing.assert_array_equal(np64(st.Q)[13:], q[13:])


def test_append_fp8_extreme_tokens(cuda_ok):
    # a zero token, the borders of the scale, tiny and huge values, and
    # tokens that are not finite (NaN scale; the next slot is untouched by it)
    st = Step([0], [8], fp8=True, H=2, Hkv=1, d=64, ps=16)
    for x in (st.K, st.V):
        x[0] = 0.0
        x[1, 0, 5] = 448.0
        x[2, 0, 5] = 450.0
        x[3] *= 2.0 ** -130
        x[4] *= 2.0 ** 120
        x[5, 0, 7] = float("inf")
        x[6, 0, 63] = float("nan")
    k, v, ks, vs = st.arrays()
    OC.append(k, v, ks, vs, None, np64(st.K), np64(st.V), st.lens, st.cu, st.table, fp8=True)
    st.append()
    k2, v2, ks2, vs2 = st.arrays()
    np.testing.assert_array_equal(ks2, ks)
    np.testing.assert_array_equal(vs2, vs)
    pg = st.table[0][0]
    for r in (0, 1, 2, 3, 4, 7):
        np.testing.assert_array_equal(k2[pg, 0, r], k[pg, 0, r])
        np.testing.assert_array_equal(v2[pg, 0, r], v[pg, 0, r])


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
DECODE = [
    ([1], dict()),
    ([5, 0, 64, 65], dict()),
    ([300, 1, 0, 129, 128, 127], dict(H=6, Hkv=6, d=64, ps=32, layout="nhd")),
    ([1000, 17], dict(H=10, Hkv=2, ps=16)),
    ([257, 700], dict(H=16, Hkv=1, ps=128)),
    ([400], dict(H=24, Hkv=1, d=64, ps=64)),
    ([90, 2000, 33], dict(H=40, Hkv=2, ps=64, scale=0.3)),
    ([0, 0], dict()),
    ([513] * 20, dict(H=8, Hkv=8, d=64, ps=16)),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(cuda_ok, case, fp8):
    lens, kw = DECODE[case]
    st = Step(lens, [0] * len(lens), fp8=fp8, seed=100 + case, cu=False, spare=case % 3, **kw)
    O, lse = st.decode()
    torch.cuda.synchronize()
    assert st.status() == 0
    st.check(O, lse)
    # once more on the same workspace, and into strided rows
    big = torch.full((st.T, 2, st.H, st.d), 5.0, dtype=BF, device=DEV)
    q2 = torch.empty_like(big)
    q2[:, 1] = st.Q
    m = pav()
    m.cache_decode(st.p, st.cache, q2[:, 1], st.t_table, st.t_lens, st.ws, big[:, 1])
    assert torch.equal(big[:, 1], O) and (big[:, 0] == 5).all()


# groups of more than 8 query heads where the cache may be long (its table is)
WIDE = [
    ([400, 90, 700], dict(H=16, Hkv=1, ps=128)),
    ([1000, 17, 3], dict(H=40, Hkv=2, ps=128)),
    ([700, 65, 0, 300], dict(H=24, Hkv=1, d=64, ps=128)),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_decode_wide_groups(cuda_ok, case, fp8):
    lens, kw = WIDE[case]
    st = Step(lens, [0] * len(lens), fp8=fp8, seed=150 + case, cu=False, spare=5000, **kw)
    O, lse = st.decode()
    assert st.status() == 0
    st.check(O, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_sparse_wide_groups(cuda_ok, case, fp8):
    lens, kw = WIDE[case]
    lens = [n + 37 * i for i in range(4) for n in lens]
    st = Step(lens, [1] * len(lens), fp8=fp8, seed=160 + case, spare=1000, n_select=1000, **kw)
    st.append()
    lists = torch.full((st.T, st.Hkv, 1000), -1, dtype=torch.int32)
    lists[..., 3:12] = torch.randint(-1, 10, (st.T, st.Hkv, 9), generator=st.g, dtype=torch.int32)
    O, lse = st.sparse(lists.to(DEV))
    assert st.status() == 0
    st.check(O, lse, lists.tolist())


def test_decode_long_and_split_over_the_gpu(cuda_ok):
    st = Step([20000, 3, 7777], [0] * 3, H=4, Hkv=1, seed=9, cu=False)
    a, la = st.decode()
    st.check(a, la)
    for _ in range(5):
        b, lb = st.decode()
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_decode_infinite_and_nan_values(cuda_ok):
    # a NaN key or value that the row sees is NaN in its head alone; slots
    # behind the end never matter (they are NaN in every test here)
    st = Step([100, 100], [0, 0], H=4, Hkv=2, seed=2, cu=False)
    st.cache.k[st.table[0][1], 1, 3, 5] = float("nan")
    st.cache.v[st.table[1][0], 0, 7, 9] = float("inf")
    O, lse = st.decode()
    O, lse = O.float(), lse
    assert O[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert O[0, :2].isfinite().all() and O[1, 2:].isfinite().all()
    assert (O[1, :2, 9] == math.inf).all()
    assert O[1, :2, :9].isfinite().all() and lse[1].isfinite().all()


def test_decode_large_scores_and_far_apart(cuda_ok):
    # scores of several hundred: the running maximum must carry the sums
    st = Step([500], [0], H=8, Hkv=1, seed=4, cu=False, scale=4.0)
    O, lse = st.decode()
    st.check(O, lse)


# ---------------------------------------------------------------------------
# choice of pages
# ---------------------------------------------------------------------------
SELECT = [
    ([600, 64, 0, 1], [1, 1, 1, 1], dict()),
    ([100, 700, 0], [80, 1, 30], dict(ps=16, n_select=9, n_first=2, n_recent=3, pad=2)),
    ([2000], [5], dict(ps=16, H=10, Hkv=2, d=64, n_select=40)),
    ([300, 900], [70, 0], dict(ps=32, H=3, Hkv=3, n_select=3, n_first=0, n_recent=3)),
    ([5000, 4000], [1, 1], dict(ps=16, H=32, Hkv=2, n_select=100, n_first=0, n_recent=1)),
    # few rows a sequence, given by cu
    ([600, 300, 10], [1, 1, 2], dict(ps=16, H=6, Hkv=3, n_select=5, pad=1)),
    ([900, 40, 0, 2000], [2, 0, 1, 3], dict(ps=32, d=64, H=20, Hkv=1, n_select=8)),
]


def means_of(st, tie=False):
    mean = torch.randn(st.P, st.Hkv, st.d, generator=st.g)
    if tie:
        mean[:] = mean[:1]
    # what must never be read: pages that are not full, and pages of nobody
    used = {st.table[s][j] for s in range(st.S) for j in range(st.lens[s] // st.ps)}
    for pg in range(st.P):
        if pg not in used:
            mean[pg] = float("nan")
    st.cache.k_mean.copy_(mean)


@pytest.mark.parametrize("tie", [False, True])
@pytest.mark.parametrize("case", range(len(SELECT)))
def test_select(cuda_ok, case, tie):
    old, new, kw = SELECT[case]
    st = Step(old, new, seed=200 + case, **kw)
    means_of(st, tie)
    sel = st.select()
    assert st.status() == 0
    want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps,
                     st.p.n_select, st.p.n_first, st.p.n_recent, st.scale)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("near", [1e-2, 1e-4, 1e-6, 3e-8])
@pytest.mark.parametrize("span", [0.0, 12.0])
def test_select_near_ties(cuda_ok, near, span):
    # pages that differ by little, means of very different sizes and queries
    # of very different elements: fp64's choice, whatever the fast sums say
    for old, new, kw in (([3000, 500], [60, 3], dict(ps=16, n_select=12, H=12, Hkv=3)),
                         ([40000], [1], dict(ps=16, n_select=64, H=4, Hkv=1, d=64)),
                         ([12000, 9000], [700, 1], dict(ps=16, n_select=7, H=8, Hkv=4))):
        st = Step(old, new, seed=17, **kw)
        base = torch.randn(3, 1, st.Hkv, st.d, generator=st.g)
        mean = base[torch.randint(0, 3, (st.P,), generator=st.g), 0]
        mean = mean + near * torch.randn(st.P, st.Hkv, st.d, generator=st.g)
        mean *= torch.exp2(span * (torch.rand(st.Hkv, st.d, generator=st.g) - 0.5))
        st.cache.k_mean.copy_(mean)
        st.Q *= torch.exp2(span * (torch.rand(st.H, st.d, generator=st.g) - 0.7)).to(BF).to(DEV)
        sel = st.select()
        want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps,
                         st.p.n_select, 1, 1, st.scale)
        np.testing.assert_array_equal(sel.cpu().numpy(), want)
    assert st.status() == 0


def test_select_many_pages(cuda_ok):
    for W, new in ((16384, [1]), (5000, [2]), (700, [300])):
        st = Step([W * 16 - new[0]], new, H=2, Hkv=1, d=64, ps=16, n_select=20, seed=W)
        means_of(st)
        want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps, 20, 1,
                         1, st.scale)
        np.testing.assert_array_equal(st.select().cpu().numpy(), want)


def test_select_extreme_magnitudes(cuda_ok):
    # means and queries outside f16's range, denormal and huge
    for ek, eq in ((30, -20), (-40, 30), (-140, 0), (100, -90), (0, -135), (60, 60)):
        st = Step([900], [4], H=4, Hkv=2, n_select=5, ps=32, seed=3)
        means_of(st)
        st.cache.k_mean *= 2.0 ** ek if ek > -126 else 2.0 ** (ek + 40) * 2.0 ** -40
        st.Q *= 2.0 ** eq if eq > -126 else 2.0 ** (eq + 40)
        if eq <= -126:
            st.Q *= 2.0 ** -40
        want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps, 5, 1, 1,
                         st.scale)
        np.testing.assert_array_equal(st.select().cpu().numpy(), want, err_msg=str((ek, eq)))


def test_select_values_that_are_not_finite(cuda_ok):
    st = Step([700], [1], H=4, Hkv=2, n_select=5, seed=1)
    means_of(st)
    st.cache.k_mean[st.table[0][3], 0, 5] = float("nan")
    st.cache.k_mean[st.table[0][4], 1, :] = float("inf")
    want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps, 5, 1, 1,
                     st.scale)
    np.testing.assert_array_equal(st.select().cpu().numpy(), want)


# rows enough for the logits in f16 parts
SELECT_MANY = [
    ([600, 64, 0, 10], [90, 200, 1, 300], dict()),
    ([100, 700], [400, 150], dict(ps=16, n_select=9, n_first=2, n_recent=3, pad=2)),
    ([2000], [700], dict(ps=16, H=10, Hkv=2, d=64, n_select=40)),
    ([300, 900], [700, 0], dict(ps=32, H=3, Hkv=3, n_select=3, n_first=0, n_recent=3)),
    ([900, 40, 0, 2000], [200, 0, 1, 300], dict(ps=32, d=64, H=20, Hkv=1, n_select=8)),
    ([30000], [200], dict(ps=16, H=16, Hkv=2, n_select=64)),
]


@pytest.mark.parametrize("tie", [False, True])
@pytest.mark.parametrize("case", range(len(SELECT_MANY)))
def test_select_many_rows(cuda_ok, case, tie):
    old, new, kw = SELECT_MANY[case]
    st = Step(old, new, seed=500 + case, **kw)
    means_of(st, tie)
    sel = st.select()
    assert st.status() == 0
    want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps,
                     st.p.n_select, st.p.n_first, st.p.n_recent, st.scale)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


def test_select_many_rows_extreme_magnitudes(cuda_ok):
    for ek, eq in ((30, -20), (-40, 30), (-140, 0), (100, -90), (0, -135), (60, 60)):
        st = Step([900], [800], H=4, Hkv=2, n_select=5, ps=32, seed=3)
        means_of(st)
        st.cache.k_mean *= 2.0 ** ek if ek > -126 else 2.0 ** (ek + 40) * 2.0 ** -40
        st.Q *= 2.0 ** eq if eq > -126 else 2.0 ** (eq + 40)
        if eq <= -126:
            st.Q *= 2.0 ** -40
        want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps, 5, 1, 1,
                         st.scale)
        np.testing.assert_array_equal(st.select().cpu().numpy(), want, err_msg=str((ek, eq)))


def test_select_many_rows_values_that_are_not_finite(cuda_ok):
    st = Step([700], [800], H=4, Hkv=2, n_select=5, seed=1)
    means_of(st)
    st.cache.k_mean[st.table[0][3], 0, 5] = float("nan")
    st.cache.k_mean[st.table[0][4], 1, :] = float("inf")
    want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps, 5, 1, 1,
                     st.scale)
    np.testing.assert_array_equal(st.select().cpu().numpy(), want)


@pytest.mark.parametrize("rows", [1, 800])
def test_select_masses_of_every_size(cuda_ok, rows):
    # logits 18 apart, down to exp(-724), which only a subnormal holds: the
    # order of the masses is theirs to the last
    st = Step([640 + 16], [rows], H=4, Hkv=4, d=64, ps=16, n_select=38, seed=2)
    mean = torch.zeros(st.P, st.Hkv, st.d)
    order = torch.randperm(40, generator=st.g)
    for j in range(40):
        mean[st.table[0][j], :, 0] = -18.1 * float(order[j]) / st.scale
    st.cache.k_mean.copy_(mean)
    st.Q.zero_()
    st.Q[..., 0] = 1.0
    want = OC.select(np64(st.Q), np64(st.cache.k_mean), st.lens, st.cu, st.table, st.G, st.ps, 38, 1, 1,
                     st.scale)
    np.testing.assert_array_equal(st.select().cpu().numpy(), want)


# ---------------------------------------------------------------------------
# sparse attention
# ---------------------------------------------------------------------------
SPARSE = [
    ([600, 64, 0, 1], [1, 1, 1, 1], dict()),
    ([100, 700, 0], [20, 1, 30], dict(ps=16, n_select=9, pad=2)),
    ([500], [6], dict(ps=32, H=10, Hkv=2, d=64, n_select=7, layout="nhd")),
    ([300, 900], [17, 0], dict(ps=128, H=3, Hkv=3, n_select=3)),
    ([1000], [2], dict(ps=16, H=32, Hkv=2, n_select=33)),
    ([700, 30], [3, 3], dict(H=20, Hkv=1, n_select=6)),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(SPARSE)))
def test_sparse(cuda_ok, case, fp8):
    old, new, kw = SPARSE[case]
    st = Step(old, new, fp8=fp8, seed=300 + case, **kw)
    st.append()
    lists = torch.randint(-1, st.W + 2, (st.T, st.Hkv, st.p.n_select), generator=st.g, dtype=torch.int32)
    lists[0] = -1                                  # a row that reads nothing
    if st.T > 1:
        lists[1, 0, -2:] = 0                       # a page twice
    O, lse = st.sparse(lists.to(DEV))
    assert st.status() == 0
    st.check(O, lse, lists.tolist())


# enough rows for tiles that share their pages' loads
MANY = [
    ([300, 40], [400, 333], dict(H=16, Hkv=4, pad=5)),
    ([0, 500, 3], [510, 0, 300], dict(H=40, Hkv=8, d=64, ps=16, n_select=7, layout="nhd")),
    ([2000], [640], dict(H=32, Hkv=2, ps=128, n_select=5)),
    ([10, 70], [2400, 100], dict(H=2, Hkv=2, d=64, ps=32, n_select=3)),
    # and tiles of 128 (row, query head) pairs
    ([100, 0], [900, 401], dict(H=32, Hkv=8, n_select=6, pad=3)),
    ([700], [430], dict(H=64, Hkv=4, ps=128, n_select=3)),
    ([64, 3, 90], [310, 0, 333], dict(H=64, Hkv=8, ps=16, n_select=9, layout="nhd")),
    ([5000], [600], dict(H=24, Hkv=8, ps=32, n_select=40, scale=1.0)),
    # tiles of one head; whole tiles and cut ones; every tile cut
    ([0], [700], dict(H=40, Hkv=40, d=64, ps=16, n_select=4)),
    ([2000, 9], [1300, 25], dict(H=32, Hkv=8, n_select=12)),
    ([900], [40], dict(H=64, Hkv=8, ps=16, n_select=30)),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_sparse_many_rows(cuda_ok, case, fp8):
    old, new, kw = MANY[case]
    st = Step(old, new, fp8=fp8, seed=400 + case, **kw)
    st.append()
    # neighbours agree on most pages
    K, W = st.p.n_select, st.W
    base = torch.randint(-1, W + 1, (st.T // 16 + 1, st.Hkv, K), generator=st.g, dtype=torch.int32)
    lists = base.repeat_interleave(16, 0)[:st.T].clone()
    own = torch.randint(-1, W + 1, (st.T, st.Hkv, K), generator=st.g, dtype=torch.int32)
    lists = torch.where(torch.rand(st.T, st.Hkv, K, generator=st.g) < 0.3, own, lists)
    lists[5] = -1
    O, lse = st.sparse(lists.to(DEV))
    assert st.status() == 0
    assert torch.equal(O, st.sparse(lists.to(DEV))[0])
    check_some(st, O, lse, lists.tolist(), every=7)


def check_some(st, O, lse, lists, every):
    """`check` for every `every`-th row, and the padding."""
    rows = [x for x in OC.rows_of(st.lens, st.cu, st.S)]
    keep = {t for t, _, _ in rows if t % every == 0 or t in (5, rows[-1][0])}
    real = OC.rows_of
    try:
        OC.rows_of = lambda *a: [x for x in rows if x[0] in keep]
        T = st.T
        used = {t for t, _, _ in rows}
        for t in range(T):
            if t not in used:
                assert (O[t] == 7).all() and (lse[t] == 7).all()
        st.T = 0
        st.check(O, lse, lists)
    finally:
        OC.rows_of, st.T = real, T


@pytest.mark.parametrize("Hkv,d", [(4, 64), (8, 128)])
@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_many_rows_hidden_values_that_are_not_finite(cuda_ok, fp8, Hkv, d):
    # a page with a NaN in V (a NaN scale, FP8): rows that do not list it, and
    # rows before that key, must not see it
    st = Step([0], [800], H=4 * Hkv, Hkv=Hkv, d=d, ps=16, fp8=fp8, n_select=3, seed=7)
    st.append()
    bad_pos = 411
    pg, slot = st.table[0][bad_pos // 16], bad_pos % 16
    if fp8:
        st.cache.v_scale[pg, 2, slot] = float("nan")
    else:
        st.cache.v[pg, 2, slot, 9] = float("nan")
        st.cache.v[pg, 1, slot, 3] = float("inf")
    lists = torch.randint(0, 50, (800, Hkv, 3), generator=st.g, dtype=torch.int32)
    lists[400:500, :, 0] = 25                        # page 25 holds key 411
    lists[:, :, 1] = torch.where(lists[:, :, 1] == 25, 26, lists[:, :, 1])
    O, lse = st.sparse(lists.to(DEV))
    L = lists.tolist()
    sees = [t >= bad_pos and 25 in L[t][2] for t in range(800)]
    got = O[:, 8:12].isnan().any(-1).any(-1).tolist()
    assert got == sees
    if not fp8:
        sees1 = [t >= bad_pos and 25 in L[t][1] for t in range(800)]
        assert O[:, 4:8].isinf().any(-1).any(-1).tolist() == sees1
        assert O[:, 4:8].isnan().sum() == 0
    clean = [t for t in range(800) if not any(t >= bad_pos and 25 in L[t][h] for h in range(Hkv))]
    for x in (st.cache.v,) if not fp8 else ():
        x[pg, 2, slot, 9] = 0.0
        x[pg, 1, slot, 3] = 0.0
    if fp8:
        st.cache.v_scale[pg, 2, slot] = 1.0
    real = OC.rows_of
    try:
        OC.rows_of = lambda *a: [(t, 0, t) for t in clean[::9]]
        st.T = 0
        st.check(O, lse, L)
    finally:
        OC.rows_of = real


def test_sparse_many_rows_a_page_twice(cuda_ok):
    st = Step([100], [700], H=8, Hkv=8, d=64, ps=32, n_select=4, seed=8)
    st.append()
    lists = torch.randint(0, 20, (700, 8, 4), generator=st.g, dtype=torch.int32)
    lists[100:130, 3, 2] = lists[100:130, 3, 0]
    O, lse = st.sparse(lists.to(DEV))
    check_some(st, O, lse, lists.tolist(), every=10)


def test_sparse_over_every_page_is_dense_causal(cuda_ok):
    st = Step([70, 0], [50, 90], n_select=4, seed=11)
    st.append()
    every = torch.arange(4, dtype=torch.int32).expand(st.T, st.Hkv, 4).contiguous().to(DEV)
    O, lse = st.sparse(every)
    st.check(O, lse, every.tolist())
    # and equals decode at the sequences' ends up to the split of the keys
    last = Step([70, 0], [50, 90], n_select=4, seed=11)
    rows = [st.cu[1] - 1, st.cu[2] - 1]
    m = pav()
    p = m.make_cache_params(n_pages=st.P, page_size=64, H=8, Hkv=2, d=128, S=2, T=2, max_pages=st.W)
    O2 = torch.empty(2, 8, 128, dtype=BF, device=DEV)
    m.cache_decode(p, st.cache, st.Q[rows].contiguous(), st.t_table, st.t_lens, last.ws, O2)
    assert (O2.float() - O[rows].float()).abs().max() <= 2 ** -6 * O[rows].float().abs().max()


# ---------------------------------------------------------------------------
# together, replayed, and refused on the device
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fp8", [False, True])
def test_generation_prompt_then_tokens(cuda_ok, fp8):
    # prompts in one call, then tokens one by one: append (queries rotated in
    # place), choose, attend, and the dense decode beside it
    m = pav()
    H, Hkv, d, ps, S = 8, 2, 128, 16, 3
    total = [150, 40, 97]
    prompt = [140, 1, 90]
    st = Step([0] * S, total, H=H, Hkv=Hkv, d=d, ps=ps, fp8=fp8, rot=128, seed=21, n_select=4)
    cos, sin = st.tables(200)
    q_all, k_all, v_all = st.Q.clone(), st.K, st.V
    off = st.cu
    done = [0] * S
    steps = [prompt] + [[min(1, total[s] - prompt[s] - i) if i < total[s] - prompt[s] else 0
                         for s in range(S)] for i in range(4)]
    for new in steps:
        rows = [off[s] + done[s] + i for s in range(S) for i in range(new[s])]
        done = [a + b for a, b in zip(done, new)]
        T = len(rows)
        view = Step.__new__(Step)
        view.__dict__.update(st.__dict__)
        view.lens, view.T = list(done), T
        view.cu = [sum(new[:i]) for i in range(S + 1)]
        view.p = m.make_cache_params(n_pages=st.P, page_size=ps, H=H, Hkv=Hkv, d=d, S=S, T=T,
                                     max_pages=st.W, format=int(fp8), n_select=4, rot_dim=128)
        view.t_lens = torch.tensor(done, dtype=torch.int32, device=DEV)
        view.t_cu = torch.tensor(view.cu, dtype=torch.int32, device=DEV)
        view.ws = m.alloc_cache_workspace(view.p, DEV)
        view.Q, view.K, view.V = q_all[rows].clone(), k_all[rows], v_all[rows]
        view.append(cos, sin, Q_out=view.Q)
        sel = view.select()
        want = OC.select(np64(view.Q), np64(st.cache.k_mean), done, view.cu, st.table, st.G, ps, 4, 1,
                         1, st.scale)
        np.testing.assert_array_equal(sel.cpu().numpy(), want)
        O, lse = view.sparse(sel)
        view.check(O, lse, want.tolist())
        if new == [1, 1, 1]:
            view.cu = view.t_cu = None
            view.check(*view.decode())
        assert view.status() == 0


def test_captured_steps_share_a_workspace(cuda_ok):
    # two graphs (dense and sparse decode) on one workspace, replayed in turn
    # with other lengths in the same buffers
    st = Step([3000, 50], [0, 0], H=8, Hkv=1, seed=31, cu=False, n_select=6, ps=16)
    means_of(st)
    O1, lse1 = st.out()
    O2, lse2 = st.out()
    sel = torch.zeros((2, 1, 6), dtype=torch.int32, device=DEV)
    m = pav()

    def dense():
        m.cache_decode(st.p, st.cache, st.Q, st.t_table, st.t_lens, st.ws, O1, lse=lse1)

    def sparse():
        m.cache_select(st.p, st.cache, st.Q, st.t_table, st.t_lens, st.ws, sel)
        m.cache_sparse(st.p, st.cache, st.Q, sel, st.t_table, st.t_lens, st.ws, O2, lse=lse2)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for f in (dense, sparse):
            f()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                f()
            graphs.append(g)
        for lens in ([3000, 50], [17, 0], [2999, 1], [1600, 49]):
            st.lens = lens
            st.t_lens.copy_(torch.tensor(lens, dtype=torch.int32))
            O1.fill_(7), O2.fill_(7)
            for g in graphs + graphs:
                g.replay()
            s.synchronize()
            st.check(O1, lse1)
            st.check(O2, lse2, sel.tolist())
    assert st.status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_captured_and_replayed_between_other_calls(cuda_ok, fp8):
    # the fast choice and cut tiles in a graph, other calls of other sizes on
    # the same workspace between its replays: the same bits every time
    st = Step([900, 300], [500, 330], H=16, Hkv=4, fp8=fp8, n_select=6, seed=45)
    st.append()
    O, lse = st.out()
    sel = torch.zeros((st.T, st.Hkv, 6), dtype=torch.int32, device=DEV)
    m = pav()
    p1 = m.make_cache_params(n_pages=st.P, page_size=st.ps, H=16, Hkv=4, d=128, S=2, T=2, max_pages=st.W,
                             format=int(fp8), n_select=6, n_recent=1)
    O1 = torch.empty(2, 16, 128, dtype=BF, device=DEV)
    sel1 = torch.zeros((2, 4, 6), dtype=torch.int32, device=DEV)

    def prompt():
        m.cache_select(st.p, st.cache, st.Q, st.t_table, st.t_lens, st.ws, sel, cu=st.t_cu)
        m.cache_sparse(st.p, st.cache, st.Q, sel, st.t_table, st.t_lens, st.ws, O, cu=st.t_cu, lse=lse)

    def token():
        m.cache_decode(p1, st.cache, st.Q[:2], st.t_table, st.t_lens, st.ws, O1)
        m.cache_select(p1, st.cache, st.Q[:2], st.t_table, st.t_lens, st.ws, sel1)
        m.cache_sparse(p1, st.cache, st.Q[:2], sel1, st.t_table, st.t_lens, st.ws, O1)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        prompt()
        s.synchronize()
        first = [x.clone() for x in (O, lse, sel)]
        check_some(st, O, lse, sel.tolist(), every=23)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            prompt()
        for _ in range(3):
            token()
            O.fill_(7), lse.fill_(7), sel.fill_(0)
            g.replay()
            s.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(first, (O, lse, sel)))
    assert st.status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_with_a_page_outside_the_cache(cuda_ok, fp8):
    # reported, and its keys are nobody's
    st = Step([0, 100], [700, 300], H=16, Hkv=4, fp8=fp8, n_select=5, seed=46)
    st.append()
    st.t_table[0, 3] = st.P
    st.t_table[1, 1] = -7
    lists = torch.randint(-1, 11, (st.T, 4, 5), generator=st.g, dtype=torch.int32)
    O, lse = st.sparse(lists.to(DEV))
    torch.cuda.synchronize()
    assert st.status() == pav().TA_ERR_BAD_INDEX
    lists[:700][lists[:700] == 3] = -1
    lists[700:][lists[700:] == 1] = -1
    check_some(st, O, lse, lists.tolist(), every=13)


def test_another_stream_and_two_workspaces_at_once(cuda_ok):
    a = Step([4000], [0], H=8, Hkv=1, seed=41, cu=False)
    b = Step([3000], [0], H=8, Hkv=1, seed=42, cu=False)
    m = pav()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [x.out() for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s, (O, lse) in ((a, s1, outs[0]), (b, s2, outs[1])):
            m.cache_decode(x.p, x.cache, x.Q, x.t_table, x.t_lens, x.ws, O, lse=lse, stream=s)
    torch.cuda.synchronize()
    a.check(*outs[0])
    b.check(*outs[1])


def test_bad_pages_and_lengths_are_reported_and_harmless(cuda_ok):
    BAD = pav().TA_ERR_BAD_INDEX
    # a page number outside the cache: its keys are skipped
    st = Step([200, 200], [0, 0], seed=51, cu=False, H=4, Hkv=2)
    good = [list(r) for r in st.table]
    st.t_table[0, 1] = st.P
    st.t_table[1, 0] = -5
    O, lse = st.decode()
    torch.cuda.synchronize()
    assert st.status() == BAD
    lists = [[[0, 2, 3]] * 2, [[1, 2, 3]] * 2]
    st.table = good
    st.check(O, lse, lists)
    pav().init_cache_workspace(st.ws)
    assert st.status() == 0
    # lengths outside the table are clamped
    st.t_table.copy_(torch.tensor(good, dtype=torch.int32))
    st.t_lens.copy_(torch.tensor([10 ** 9, -3], dtype=torch.int32))
    st2 = Step([256, 0], [0, 0], seed=51, cu=False, H=4, Hkv=2)
    O, lse = st.decode()
    torch.cuda.synchronize()
    assert st.status() == BAD and (O[1] == 0).all() and st2 is not None
    # append: nothing is written through a bad table, or before position 0
    st = Step([0, 0], [70, 5], seed=52)
    before = st.arrays()
    st.t_table.fill_(st.P + 7)
    st.append()
    torch.cuda.synchronize()
    assert st.status() == BAD
    for x, y in zip(before, st.arrays()):
        if x is not None:
            np.testing.assert_array_equal(x, y)
    st = Step([0], [70], seed=53)
    st.t_lens.fill_(6)                              # 70 new tokens, 6 in all
    want = [x.copy() if x is not None else None for x in st.arrays()]
    pg = st.table[0][0]
    for i in range(6):
        want[0][pg, :, i] = np64(st.K)[64 + i]
        want[1][pg, :, i] = np64(st.V)[64 + i]
    st.append()
    torch.cuda.synchronize()
    assert st.status() == BAD
    np.testing.assert_array_equal(st.arrays()[0], want[0])
    np.testing.assert_array_equal(st.arrays()[1], want[1])


def test_the_native_entry_takes_ordinary_calls(cuda_ok):
    # 0, not None: the checks in C++ read the structures as Python wrote them
    from precision_attention_video_b200 import cache as C
    m = C._native()
    st = Step([70, 200], [30, 1], rot=128, seed=71)
    cos, sin = st.tables(300)
    sel = torch.zeros((st.T, st.Hkv, 4), dtype=torch.int32, device=DEV)
    O, lse = st.out()
    a = (st.p, st.cache._view)
    assert m.append(*a, st.K, st.V, st.t_table, st.t_lens, st.ws, st.t_cu, cos, sin, None, st.Q, O, None) == 0
    assert m.select(*a, st.Q, st.t_table, st.t_lens, st.ws, sel, st.t_cu, None) == 0
    assert m.sparse(*a, st.Q, sel, st.t_table, st.t_lens, st.ws, O, st.t_cu, lse, None) == 0
    # refused: other devices' or shapes' tensors; then the reason
    assert m.sparse(*a, st.Q, sel.cpu(), st.t_table, st.t_lens, st.ws, O, st.t_cu, lse, None) is None
    assert m.sparse(*a, st.Q[1:], sel, st.t_table, st.t_lens, st.ws, O, st.t_cu, lse, None) is None
    for bad, why in ((dict(sel=sel.cpu()), "sel: expected a tensor on device 0"),
                     (dict(sel=sel[:, :, :3]), "sel: expected a contiguous tensor"),
                     (dict(Q=st.Q.float()), "Q: expected torch.bfloat16"),
                     (dict(table=st.t_table[:1]), "table: expected"),
                     (dict(ws=st.ws.view(-1, 2)), "ws: expected"),
                     (dict(lens=st.t_lens.long()), "lens: expected torch.int32")):
        kw = {**dict(Q=st.Q, sel=sel, table=st.t_table, lens=st.t_lens, ws=st.ws, O=O), **bad}
        with pytest.raises((ValueError, TypeError), match=why):
            pav().cache_sparse(st.p, st.cache, **kw, cu=st.t_cu)
    one = Step([100], [0], seed=72, cu=False)
    O, lse = one.out()
    assert m.decode(one.p, one.cache._view, one.Q, one.t_table, one.t_lens, one.ws, O, lse,
                    torch.cuda.current_stream().cuda_stream) == 0
    one.check(O, lse)
    with pytest.raises(pav().TieredAttnError, match="workspace too small"):
        pav().cache_decode(one.p, one.cache, one.Q, one.t_table, one.t_lens, one.ws[:4096], O)


def test_far_pages_pass_32_bits(cuda_ok):
    # a cache of more than 2^31 elements: its last pages
    m = pav()
    ps, Hkv, d = 128, 8, 128
    P = 2 ** 31 // (ps * Hkv * d) + 40
    p = m.make_cache_params(n_pages=P, page_size=ps, H=8, Hkv=Hkv, d=d, S=1, T=1, max_pages=3,
                            n_select=2, rot_dim=0)
    k = torch.empty((P, Hkv, ps, d), dtype=BF, device=DEV)
    v = torch.empty_like(k)
    mean = torch.empty((P, Hkv, d), device=DEV)
    st = Step([257], [1], H=8, Hkv=Hkv, d=d, ps=ps, seed=61)
    pages = [P - 1, P - 17, P - 30]
    for j in range(3):
        k[pages[j]], v[pages[j]] = st.cache.k[st.table[0][j]], st.cache.v[st.table[0][j]]
    cache = m.PagedCache(k, v, k_mean=mean)
    table = torch.tensor([pages], dtype=torch.int32, device=DEV)
    ws = m.alloc_cache_workspace(p, DEV)
    O, lse = st.out()
    m.cache_append(p, cache, st.K, st.V, table, st.t_lens, ws)
    m.cache_decode(p, cache, st.Q, table, st.t_lens, ws, O, lse=lse)
    st.append()
    O2, lse2 = st.decode()
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    assert m.get_status(ws) == 0
