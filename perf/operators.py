"""Cases of the cached-attention operators: a paged key-value cache that is
appended to with the position rotation, attention of one new token over the
whole cache, the choice of pages by their mean key, and attention over the
chosen pages only.

``run`` computes an operator in plain torch where ``own`` is false, and calls
the library where it is true.  Lengths depend on the case alone, values on the
seed.  All lengths, tables and offsets live on the GPU, as in a serving loop.
"""

import math
import random

import torch

own = False

DEV = "cuda"
BF, F32, F64, E4 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn

BASE = dict(S=1, n=1, len=1000, H=32, Hkv=8, d=128, ps=64, fp8=False, nhd=False,
            K=16, first=1, recent=2, rot=128, inter=False, base=10000.0)


def _case(name, op, **kw):
    return {"name": name, "op": op, **{**BASE, **kw}}


def listed():
    return [
        # one token for each of a few sequences: the append of a decoding step
        _case("append-token", "append", S=16, len=4096),
        # a batch of prompts of uneven length into an FP8 cache, half of each
        # head rotated, neighbouring elements paired
        _case("append-prompt-fp8", "append", S=4, n=4096, len=8192, fp8=True, rot=64, inter=True),
        # a causal video model: one latent frame of 30 x 52 tokens for each of
        # two clips, a key head for every query head, token-major pages
        _case("append-frame", "append", S=2, n=1560, len=12480, H=40, Hkv=40, nhd=True, inter=True),
        # one short sequence, small pages: latency alone
        _case("decode-one", "decode", S=1, len=1000, ps=16),
        # an ordinary serving batch of uneven lengths
        _case("decode-batch", "decode", S=64, len=16384),
        # few long sequences in FP8, split over their length
        _case("decode-long-fp8", "decode", S=4, len=131072, H=64, fp8=True),
        # a key head for every query head, 64-wide, token-major pages
        _case("decode-heads", "decode", S=16, len=4095, H=12, Hkv=12, d=64, ps=32, nhd=True, rot=64),
        # choosing pages for one new token of long sequences
        _case("select-token", "select", S=32, len=131072, K=32),
        # choosing pages for every token of new prompts or frames
        _case("select-prompt", "select", S=3, n=1560, len=32760, K=16),
        # attention over chosen pages: one sequence
        _case("sparse-one", "sparse", S=1, len=16000, K=16),
        # a serving batch on an FP8 cache
        _case("sparse-batch-fp8", "sparse", S=64, len=16384, K=32, fp8=True),
        # every token of two prompts, each with its own pages
        _case("sparse-prompt", "sparse", S=2, n=1000, len=16384, K=16),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))  # noqa: E731
    op = rng.choice(["append", "decode", "select", "sparse"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 12])
    G = min(rng.choice([1, 2, 4, 5, 8, 16]), 64 // Hkv)
    ps = rng.choice([16, 32, 64, 64, 128])
    c = dict(BASE, op=op, d=d, Hkv=Hkv, H=Hkv * G, ps=ps, fp8=rng.random() < 0.4,
             nhd=rng.random() < 0.4, inter=rng.random() < 0.5, rot=rng.choice([d, d, d // 2]),
             first=rng.choice([0, 1, 2]), recent=rng.choice([1, 2, 4]))
    c["K"] = c["first"] + c["recent"] + rng.choice([1, 4, 9, 13, 26])
    if op == "append":
        c["S"] = log(1, 64)
        c["n"] = 1 if rng.random() < 0.4 else log(2, max(2, 8000 // c["S"]))
        c["len"] = c["n"] + log(1, 4000)
    elif op == "decode":
        c["S"] = log(1, 64)
        c["len"] = log(1, max(2, min(100000, 600000 // c["S"])))
    elif op == "select":
        c["S"] = log(1, 24)
        c["n"] = 1 if rng.random() < 0.5 else log(2, max(2, 2500 // c["S"]))
        c["H"] = Hkv * min(G, 4) if c["n"] > 1 else c["H"]
        # pages enough that there is a choice to make
        c["len"] = c["n"] + log(ps * (c["K"] + 4) * 4, 20000 if c["n"] > 1 else 80000)
    else:
        c["S"] = log(1, 48)
        c["n"] = 1 if rng.random() < 0.5 else log(2, max(2, 1200 // c["S"]))
        c["K"] = min(c["K"], c["first"] + c["recent"] + 1024 // ps)
        c["len"] = c["n"] + log(1, max(2, min(30000, 400000 // c["S"])))
    return c


# ---------------------------------------------------------------------------
# Lengths: of the case alone
# ---------------------------------------------------------------------------
def _lens(c):
    """(new tokens, total length after them) of each sequence."""
    r = random.Random("%d %d %d" % (c["S"], c["n"], c["len"]))
    new, tot = [], []
    for s in range(c["S"]):
        n = c["n"] if c["n"] == 1 or c["n"] == 1560 else r.randint((c["n"] + 1) // 2, c["n"])
        new.append(n)
        tot.append(c["len"] if s == 0 else max(n, r.randint(c["len"] // 4, c["len"])))
    return new, tot


def _pages(tot, ps):
    return [-(-t // ps) for t in tot]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _fp8_scale(amax):
    """The smallest power of two s with amax <= 448 s; 1 for 0."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8))
    return torch.where(amax == 0, torch.ones_like(s), s)


def _codes(x):
    """x [..., d] as e4m3 values, rounded once from x's own type, and one scale per row."""
    s = _fp8_scale(x.abs().amax(-1))
    y = x / s.unsqueeze(-1)
    step = torch.ldexp(torch.ones_like(y), torch.frexp(y).exponent.clamp(min=-5) - 4)
    return (torch.round(y / step) * step).float().to(E4), s.float()


def prepare(case, seed):
    c = dict(BASE, **case)
    g = torch.Generator(DEV).manual_seed(seed)
    rand = lambda *shape, dtype=F32: torch.randn(*shape, generator=g, device=DEV, dtype=dtype)  # noqa: E731
    new, tot = _lens(c)
    S, T, H, Hkv, d, ps = c["S"], sum(new), c["H"], c["Hkv"], c["d"], c["ps"]
    width = max(_pages(tot, ps))
    P = sum(_pages(tot, ps)) + 3                     # a few pages belong to nobody
    order = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, k in enumerate(_pages(tot, ps)):
        table[s, :k] = order[at:at + k]
        at += k
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    st = dict(c=c, table=table, lens=i32(tot), q=(2 * rand(T, H, d)).to(BF))
    st["cu"] = i32([sum(new[:i]) for i in range(S + 1)]) if c["n"] > 1 else None

    # the cache: pages of [head][slot][d], or of [slot][head][d] (token-major)
    shape = (P, ps, Hkv, d) if c["nhd"] else (P, Hkv, ps, d)
    view = (lambda x: x.transpose(1, 2)) if c["nhd"] else (lambda x: x)
    st["ks"] = st["vs"] = None
    if c["op"] != "select":
        if c["fp8"]:
            (k, ks), (v, vs) = _codes(rand(*shape, dtype=BF).float()), _codes(rand(*shape, dtype=BF).float())
            st["ks"], st["vs"] = view(ks).contiguous(), view(vs).contiguous()
        else:
            k, v = rand(*shape, dtype=BF), rand(*shape, dtype=BF)
        st["k"], st["v"] = view(k), view(v)
    if c["op"] in ("append", "select"):
        st["km"] = 0.5 * rand(P, Hkv, d)
    if c["op"] == "append":
        st["kn"], st["vn"] = rand(T, Hkv, d, dtype=BF), rand(T, Hkv, d, dtype=BF)
        inv = c["base"] ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=F64) / c["rot"])
        ang = torch.arange(c["len"] + 1, device=DEV, dtype=F64)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["qr"] = torch.empty_like(st["q"])
    else:
        st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty(T, H, device=DEV)
        st["sel"] = torch.full((T, Hkv, c["K"]), -1, dtype=torch.int32, device=DEV)
    if c["op"] == "sparse":
        # rows of a sequence mostly agree on what matters: one taste for each
        # sequence and head, and some of its own for each row
        seq, length = _rows(st["lens"], st["cu"], T)
        npg = -(-length // ps)
        j = torch.arange(width, device=DEV)
        taste = rand(S, Hkv, width)[seq] + 0.3 * rand(T, Hkv, width)
        forced = (j < c["first"]) | (j >= npg[:, None] - c["recent"])
        taste = torch.where(forced[:, None], math.inf, taste)
        taste = taste.masked_fill((j >= npg[:, None])[:, None], -math.inf)
        top = taste.topk(min(c["K"], width), -1)
        ids = torch.where(top.values > -math.inf, top.indices, width).sort(-1).values
        st["sel"][..., :ids.shape[-1]] = torch.where(ids < width, ids, -1).to(torch.int32)
    if own:
        # the handles that a serving program keeps: parameters and workspace
        import precision_attention_video_b200 as pav
        st["p"] = pav.make_cache_params(
            n_pages=P, page_size=ps, H=H, Hkv=Hkv, d=d, S=S, T=T, max_pages=width,
            format=pav.TA_CACHE_FP8 if c["fp8"] else pav.TA_CACHE_BF16,
            n_select=c["K"], n_first=c["first"], n_recent=c["recent"],
            rot_dim=c["rot"], rot_interleaved=int(c["inter"]))
        st["ws"] = pav.alloc_cache_workspace(st["p"], DEV)
        st["cache"] = pav.PagedCache(k=st.get("k"), v=st.get("v"), k_scale=st["ks"],
                                     v_scale=st["vs"], k_mean=st.get("km"))
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _rows(lens, cu, T):
    """Sequence and visible length (its own key included) of every row."""
    t = torch.arange(T, device=lens.device)
    if cu is None:
        return t, lens.long()
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(cu.dtype), right=True)
    return seq, (lens[seq] - cu[seq + 1] + t + 1).long()


def _rotate(x, cos, sin, inter):
    r2 = cos.shape[-1]
    if inter:
        a, b = x[..., 0:2 * r2:2], x[..., 1:2 * r2:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r2], x[..., r2:2 * r2]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * r2:]), -1)


def _plain_append(st):
    c = st["c"]
    ps = c["ps"]
    seq, length = _rows(st["lens"], st["cu"], st["q"].shape[0])
    pos = length - 1
    page, slot = st["table"][seq, pos // ps].long(), pos % ps
    cos, sin = st["cos"][pos].unsqueeze(1), st["sin"][pos].unsqueeze(1)
    # FP8 keys are turned in 64 bits: a key next to a border of that coarse
    # grid would else fall to either side of it
    w = F64 if c["fp8"] else F32
    k, v = _rotate(st["kn"].to(w), cos.to(w), sin.to(w), c["inter"]), st["vn"].float()
    st["qr"].copy_(_rotate(st["q"].float(), cos, sin, c["inter"]))
    h = torch.arange(c["Hkv"], device=DEV)
    where = (page[:, None], h, slot[:, None])
    if c["fp8"]:
        for x, name in ((k, "k"), (v, "v")):
            codes, s = _codes(x)
            st[name].view(torch.uint8)[where] = codes.view(torch.uint8)
            st[name + "s"][where] = s
    else:
        st["k"][where] = k.to(BF)
        st["v"][where] = v.to(BF)
    full = page[slot == ps - 1]                      # pages that this call filled
    keys = st["k"].view(torch.uint8)[full].view(E4) if c["fp8"] else st["k"][full]
    keys = keys.float()
    if c["fp8"]:
        keys = keys * st["ks"][full].unsqueeze(-1)
    st["km"][full] = keys.mean(2)
    return _outputs(st)


def _outputs(st):
    out = {"k": st["k"], "v": st["v"], "k_mean": st["km"], "q": st["qr"]}
    if st["c"]["fp8"]:
        out.update(k_scale=st["ks"], v_scale=st["vs"])
    return out


def _gather(st, name, pages):
    """Pages [...] of head h as [..., ps, d] floats; pages is [R, Hkv, n]."""
    h = torch.arange(st["c"]["Hkv"], device=DEV)[:, None]
    if st["c"]["fp8"]:
        x = st[name].view(torch.uint8)[pages, h].view(E4).float()
        return x.mul_(st[name + "s"][pages, h].unsqueeze(-1))
    return st[name][pages, h].float()


def _plain_attend(st, ids, rows, length):
    """Attention of each row over the pages `ids` [R, Hkv, n] of its sequence
    (-1: none), keys at and past `length` hidden."""
    c = st["c"]
    R, Hkv, n = ids.shape
    ps, d, G = c["ps"], c["d"], c["H"] // c["Hkv"]
    at = ids.long().clamp(min=0)
    pages = st["table"][rows[:, None, None], at].long().clamp(min=0)
    key = (at.unsqueeze(-1) * ps + torch.arange(ps, device=DEV)).flatten(2)
    seen = (key < length[:, None, None]) & (ids >= 0).repeat_interleave(ps, 2)
    q = st["q"].float().view(R, Hkv, G, d)
    k = _gather(st, "k", pages).view(R, Hkv, n * ps, d)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5)
    del k
    s = s.masked_fill_(~seen.unsqueeze(2), -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    e = s.sub_(m).exp_()
    z = e.sum(-1, keepdim=True)
    v = _gather(st, "v", pages).view(R, Hkv, n * ps, d)
    o = torch.matmul(e, v) / z.clamp(min=1e-38)
    st["o"].copy_(o.view(R, c["H"], d))
    st["lse"].copy_((m + z.log()).view(R, c["H"]))
    return {"o": st["o"], "lse": st["lse"]}


def _plain_decode(st):
    c = st["c"]
    R = st["q"].shape[0]
    rows, length = _rows(st["lens"], None, R)
    ids = torch.arange(st["table"].shape[1], device=DEV).expand(R, c["Hkv"], -1)
    ids = ids.masked_fill(ids * c["ps"] >= length[:, None, None], -1)
    return _plain_attend(st, ids, rows, length)


def _plain_sparse(st):
    rows, length = _rows(st["lens"], st["cu"], st["q"].shape[0])
    return _plain_attend(st, st["sel"], rows, length)


def _plain_select(st):
    """The pages of greatest pooled mass, in 64 bits: borders are close."""
    c = st["c"]
    T, S, H, Hkv, d, ps, K = st["q"].shape[0], c["S"], c["H"], c["Hkv"], c["d"], c["ps"], c["K"]
    G, n, W = H // Hkv, c["n"], st["table"].shape[1]
    rows, length = _rows(st["lens"], st["cu"], T)
    npg = -(-length // ps)
    km = st["km"][st["table"].long().clamp(min=0)].double()          # [S, W, Hkv, d]
    if c["n"] == 1:
        q = st["q"].view(S, 1, Hkv, G, d).double()
        local = torch.zeros_like(rows)
    else:
        local = torch.arange(T, device=DEV) - st["cu"][rows]
        q = torch.zeros(S, n, Hkv, G, d, dtype=F64, device=DEV)
        q[rows, local] = st["q"].view(T, Hkv, G, d).double()
    lg = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * G, d), km.permute(0, 2, 3, 1))
    lg = lg.mul_(d ** -0.5).view(S, Hkv, n, G, W)
    lg = lg.permute(0, 2, 1, 3, 4)[rows, local]                      # [T, Hkv, G, W]
    j = torch.arange(W, device=DEV)
    forced = ((j < c["first"]) | (j >= npg[:, None] - c["recent"])) & (j < npg[:, None])
    cand = ((j < npg[:, None]) & ~forced)[:, None, None]
    lg = lg.masked_fill_(~cand | ~lg.isfinite(), -math.inf)
    e = lg.sub_(lg.amax(-1, keepdim=True).clamp(min=-1e300)).exp_()
    mass = (e / e.sum(-1, keepdim=True).clamp(min=1e-300)).sum(2)     # [T, Hkv, W]
    mass = mass.masked_fill_(~cand[:, :, 0], -1.0)
    mass = mass.masked_fill_(forced[:, None], math.inf)
    top = mass.sort(dim=-1, descending=True, stable=True)
    ids = torch.where(top.values[..., :K] >= 0, top.indices[..., :K], W).sort(-1).values
    st["sel"].fill_(-1)
    st["sel"][..., :ids.shape[-1]] = torch.where(ids < W, ids, -1)
    return {"sel": st["sel"]}


def _own(st):
    import precision_attention_video_b200 as pav
    c, p, ws, cache = st["c"], st["p"], st["ws"], st["cache"]
    table, lens, cu = st["table"], st["lens"], st["cu"]
    if c["op"] == "append":
        pav.cache_append(p, cache, st["kn"], st["vn"], table, lens, ws, cu=cu, cos=st["cos"],
                         sin=st["sin"], Q=st["q"], Q_out=st["qr"])
        return _outputs(st)
    if c["op"] == "decode":
        pav.cache_decode(p, cache, st["q"], table, lens, ws, st["o"], lse=st["lse"])
        return {"o": st["o"], "lse": st["lse"]}
    if c["op"] == "select":
        pav.cache_select(p, cache, st["q"], table, lens, ws, st["sel"], cu=cu)
        return {"sel": st["sel"]}
    pav.cache_sparse(p, cache, st["q"], st["sel"], table, lens, ws, st["o"], cu=cu, lse=st["lse"])
    return {"o": st["o"], "lse": st["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode, "select": _plain_select,
            "sparse": _plain_sparse}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------
# Work, and the values in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    c = dict(BASE, **case)
    new, tot = _lens(c)
    T, H, Hkv, d, ps, K = sum(new), c["H"], c["Hkv"], c["d"], c["ps"], c["K"]
    row = d + 4 if c["fp8"] else 2 * d               # bytes of one cached key or value
    if c["op"] == "append":
        filled = sum(t // ps - (t - n) // ps for n, t in zip(new, tot))
        # keys of a page that an earlier call began are read back for its mean
        back = sum((t - n) % ps for n, t in zip(new, tot) if t // ps > (t - n) // ps)
        nbytes = (T * Hkv * (4 * d + 2 * row) + 4 * T * H * d + T * c["rot"] * 4
                  + filled * Hkv * d * 4 + back * Hkv * row)
        return {"bytes": nbytes, "flops": 3 * T * (H + Hkv) * c["rot"]}
    io = T * H * (4 * d + 4)
    if c["op"] == "decode":
        return {"bytes": io + 2 * sum(tot) * Hkv * row, "flops": 4 * sum(tot) * H * d}
    # visible pages of every row
    seen = [-(-(t - n + i + 1) // ps) for n, t in zip(new, tot) for i in range(n)]
    cand = [max(0, x - c["first"] - c["recent"]) for x in seen]
    if c["op"] == "select":
        means = sum(max(0, x - c["first"] - c["recent"]) for x in _pages(tot, ps))
        return {"bytes": T * H * d * 2 + means * Hkv * d * 4 + T * Hkv * K * 4,
                "flops": 2 * sum(cand) * H * d}
    kept = sum(min(K, x) for x in seen)
    pages = sum(min(x, n * K) for x, n in zip(_pages(tot, ps), new))
    return {"bytes": io + T * Hkv * K * 4 + 2 * pages * ps * Hkv * row,
            "flops": 4 * kept * ps * H * d}


def exact(case, seed):
    """The definitions, sequence by sequence (and row by row) in 64 bits."""
    st = prepare(case, seed)
    c, new, tot = st["c"], *_lens(dict(BASE, **case))
    ps, d, Hkv, G, K = c["ps"], c["d"], c["Hkv"], c["H"] // c["Hkv"], c["K"]
    table = st["table"].tolist()
    starts = [sum(new[:i]) for i in range(len(new))]
    if c["op"] == "append":
        return _exact_append(st, c, new, tot, table, starts)
    if c["op"] == "select":
        return None                                   # whole numbers only
    o = torch.zeros(sum(new), c["H"], d, dtype=F64, device=DEV)
    lse = torch.full((sum(new), c["H"]), -math.inf, dtype=F64, device=DEV)

    def whole(name, s, h):
        """All keys or values of sequence s and head h, in 64 bits."""
        idx = st["table"][s, :-(-tot[s] // ps)].long()
        x = st[name][:, h]
        x = (x.view(torch.uint8)[idx].view(E4) if c["fp8"] else x[idx]).double()
        if c["fp8"]:
            x = x * st[name + "s"][idx, h].double().unsqueeze(-1)
        return x.reshape(-1, d)

    for s in range(len(new)):
        rows = slice(starts[s], starts[s] + new[s])
        length = torch.arange(tot[s] - new[s] + 1, tot[s] + 1, device=DEV)
        for h in range(Hkv):
            k, v = whole("k", s, h), whole("v", s, h)
            key = torch.arange(k.shape[0], device=DEV)
            hide = key >= length[:, None]
            if c["op"] == "sparse":
                kept = torch.zeros(new[s], k.shape[0] // ps + 1, dtype=torch.bool, device=DEV)
                ids = st["sel"][rows, h].long()
                kept.scatter_(1, torch.where(ids < 0, kept.shape[1] - 1, ids), True)
                hide = hide | ~kept[:, :-1].repeat_interleave(ps, 1)
            x = torch.einsum("rgd,kd->rgk", st["q"][rows, h * G:(h + 1) * G].double(), k) / math.sqrt(d)
            x.masked_fill_(hide[:, None], -math.inf)
            lse[rows, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            o[rows, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return {"o": o, "lse": lse}


def _exact_append(st, c, new, tot, table, starts):
    ps, r2, inter = c["ps"], c["rot"] // 2, c["inter"]
    # e4m3 is not a type to index or to assign by parts
    full = lambda x: x.float().double()  # noqa: E731
    k, v, km = full(st["k"]), full(st["v"]), st["km"].double()
    ks, vs = (st["ks"].double(), st["vs"].double()) if c["fp8"] else (None, None)
    first = torch.arange(0, 2 * r2, 2, device=DEV) if inter else torch.arange(r2, device=DEV)
    second = first + 1 if inter else first + r2

    def turned(x, pos):
        x = x.double()
        y = x.clone()
        cos, sin = st["cos"].double()[pos][:, None], st["sin"].double()[pos][:, None]
        y[..., first] = x[..., first] * cos - x[..., second] * sin
        y[..., second] = x[..., second] * cos + x[..., first] * sin
        return y

    def stored(x):
        """Values as the cache holds them, and their scales."""
        if not c["fp8"]:
            return x, None
        amax = x.abs().amax(-1)
        s = torch.exp2(torch.ceil(torch.log2(torch.where(amax > 0, amax, 448.0) / 448)))
        y = x / s[..., None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(y / step) * step, s

    q = torch.empty_like(st["q"], dtype=F64)
    for s, n in enumerate(new):
        rows = slice(starts[s], starts[s] + n)
        pos = torch.arange(tot[s] - n, tot[s], device=DEV)
        q[rows] = turned(st["q"][rows], pos)
        page = torch.tensor(table[s], device=DEV)[pos // ps]
        (kk, s1), (vv, s2) = stored(turned(st["kn"][rows], pos)), stored(st["vn"][rows].double())
        k[page, :, pos % ps], v[page, :, pos % ps] = kk, vv
        if c["fp8"]:
            ks[page, :, pos % ps], vs[page, :, pos % ps] = s1, s2
        for j in range((tot[s] - n) // ps, tot[s] // ps):
            x = k[table[s][j]]
            x = x * ks[table[s][j]][..., None] if c["fp8"] else x.to(BF).double()
            km[table[s][j]] = x.mean(1)
    out = {"k": k, "v": v, "k_mean": km, "q": q}
    if c["fp8"]:
        out.update(k_scale=ks, v_scale=vs)
    return out
