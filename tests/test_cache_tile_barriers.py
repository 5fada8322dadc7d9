"""The barriers of cache_tile_kernel (ta_cache_attn.cu), every interleaving of
its roles on the CPU: the waits, arrivals, commits and loads of each role are
read from the source, in its order, and a state search over four units runs
them with the semantics of an mbarrier.  A wait tests a phase's parity only, so
it is passed too early, or never, when the barrier is a phase away from where
the waiter thinks it is: both fail here, and so does any state in which nobody
can go on.  Where a wait may run out instead (any one, at any time: all roles
then leave), no load and no product may still be on its way at the end."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "precision_attention_video_b200", "csrc", "ta_cache_attn.cu")
UNITS, WARPS = 4, 2                    # (two softmax warps stand for eight)
LEFT = 1000                            # added to a softmax warp's position: a wait of its has run out

OP = re.compile(r"mbar_wait\((\w+), (\(i - 1\) & 1|i & 1|\(units - 1\) & 1), |mbar_arrive_expect_tx\((\w+), "
                r"|(if \(ok\) )?mbar_arrive\((\w+)\)|tc_commit\((\w+)\)")


def roles(fp8, waits_for_v):
    """Per role the operations of unit i, [(kind, barrier, offset of the phase)],
    and of the softmax what follows its loop."""
    src = open(SRC).read()
    src = src[src.index("cache_tile_kernel("):]
    src = re.sub(r"//[^\n]*", "", src[:src.index("\n}\n")].replace("// ---- ", "@@ "))
    text = {}
    for part in src.split("@@ ")[1:]:
        text[re.match(r"\w+", part).group()] = part
    out = {}
    for role, part in text.items():
        ops = []
        for m in OP.finditer(part):
            wait, phase, armed, fine, arrived, commit = m.groups()
            name = wait or armed or arrived or commit
            if (name == "seen" and fp8) or (arrived == "k_ready" and not fp8):
                continue
            if name == "k_ready" and not fp8:
                name = "full_k"
            kind = "wait" if wait else "load" if armed else "commit" if commit else "arrive_if" if fine else "arrive"
            off = {"i & 1": 0, "(i - 1) & 1": -1, "(units - 1) & 1": "last"}.get(phase, 0)
            ops.append((kind, name, off))
        out[role] = ops
    loads, products, softmax = out["loads"], out["products"], out["softmax"]
    # of the softmax's two waits for V, FP8 has the first, slots without a key
    # the second, and whole bf16 pages none
    v = [k for k, o in enumerate(softmax) if o[1] == "full_v"]
    assert len(v) == 2
    softmax = [o for k, o in enumerate(softmax) if k not in v or (k == v[0] and (fp8 or waits_for_v))]
    # what a role waits for behind its loop: the last phase that it gave out
    drains = [re.findall(r"if \((n\w)\) mbar_wait_drain\((\w+), \(\1 - 1\) & 1\);", text[r])
              for r in ("loads", "products")]
    return loads, products, softmax, [[b for _, b in d] for d in drains]


def run(fp8, waits_for_v, gives_up=False):
    loads, products, softmax, drains = roles(fp8, waits_for_v)
    assert [o[:2] for o in loads if o[0] == "load"] == [("load", "full_k"), ("load", "full_v")]
    assert [o[1] for o in products if o[0] == "commit"] == ["s_ready", "o_done"]
    body = [o for o in softmax if o[2] != "last"]
    progs = [
        [(k, b, i + d) for i in range(UNITS) for k, b, d in loads if i + d >= 0],
        [(k, b, i + d) for i in range(UNITS) for k, b, d in products],
    ] + [[(k, b, i + d) for i in range(UNITS) for k, b, d in body] + [("wait", "o_done", UNITS - 1)]] * WARPS
    bars = sorted({b for p in progs for _, b, _ in p})
    # arrivals of a phase: the softmax's warps, or one commit, or one load's end
    need = {b: WARPS if any(k.startswith("arrive") and c == b for k, c, _ in progs[2]) else 1 for b in bars}
    at = {b: k for k, b in enumerate(bars)}

    def given(r, pc, b):
        """Phases of b that role r has given out before its step pc."""
        return sum(k in ("load", "commit") and c == b for k, c, _ in progs[r][:pc])

    # state: a position in each program (a pair where the role has left its loop:
    # drains done and where it left), (phases done, arrivals) of each barrier,
    # loads on their way (a set), commits on their way (in order), whether a
    # wait has run out
    start = ((0,) * len(progs), ((0, 0),) * len(bars), (), (), False)
    seen, todo = {start}, [start]

    def arrive(state, b):
        done, n = state[at[b]]
        n += 1
        done, n = (done + 1, 0) if n == need[b] else (done, n)
        return state[:at[b]] + ((done, n),) + state[at[b] + 1:]

    while todo:
        pcs, barriers, flying, commits, out = todo.pop()
        nexts = []
        for k, b in enumerate(flying):           # a load lands
            nexts.append((pcs, arrive(barriers, b), flying[:k] + flying[k + 1:], commits, out))
        if commits:                              # the oldest products end
            nexts.append((pcs, arrive(barriers, commits[0]), flying, commits[1:], out))
        where = []
        for r, prog in enumerate(progs):
            def to(pc):
                return pcs[:r] + (pc,) + pcs[r + 1:]
            if r < 2 and (isinstance(pcs[r], tuple) or pcs[r] == len(prog)):
                n, left = pcs[r] if isinstance(pcs[r], tuple) else (0, len(prog))
                if n < len(drains[r]):
                    b = drains[r][n]
                    last = given(r, left, b) - 1
                    where.append(("drain", b, last))
                    if last < 0 or barriers[at[b]][0] & 1 != last & 1:
                        assert last < 0 or barriers[at[b]][0] == last + 1
                        nexts.append((to((n + 1, left)), barriers, flying, commits, out))
                continue
            pc = pcs[r] % LEFT
            if pc == len(prog):
                continue
            kind, b, phase = prog[pc]
            where.append(prog[pc])
            on = to(pcs[r] + 1)
            if pcs[r] >= LEFT and kind in ("wait", "arrive_if"):
                nexts.append((on, barriers, flying, commits, out))
            elif kind == "wait":
                done = barriers[at[b]][0]
                if gives_up:                     # loads and products leave, the softmax goes on without waits
                    nexts.append((to((0, pc) if r < 2 else LEFT + pc + 1), barriers, flying, commits, True))
                if done & 1 == phase & 1:
                    continue                     # the parity says: not yet
                assert out or done == phase + 1, f"role {r} passes {b} for phase {phase} with {done} done"
                nexts.append((on, barriers, flying, commits, out))
            elif kind == "load":
                assert out or b not in flying, f"{b} armed twice"
                nexts.append((on, barriers, tuple(sorted(flying + (b,))), commits, out))
            elif kind == "commit":
                nexts.append((on, barriers, flying, commits + (b,), out))
            else:
                nexts.append((on, arrive(barriers, b), flying, commits, out))
        assert nexts or not where, f"nobody can go on: {where}"
        if not where:
            assert not flying and not commits, f"still on their way at the end: {flying + commits}"
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return len(seen)


@pytest.mark.parametrize("fp8,waits_for_v", [(False, False), (False, True), (True, True)])
def test_every_interleaving_ends(fp8, waits_for_v):
    assert run(fp8, waits_for_v) > 500


@pytest.mark.parametrize("fp8,waits_for_v", [(False, False), (True, True)])
def test_nothing_is_on_its_way_when_a_wait_has_run_out(fp8, waits_for_v):
    assert run(fp8, waits_for_v, gives_up=True) > 500
