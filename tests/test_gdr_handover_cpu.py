"""The hand-overs of the tensor-memory state pass (csrc/kda_gdr_state_tc.cu), on the CPU: every order in
which its warps, its products and its copies may run ends, and no buffer is written while it is read.

A wait on an mbarrier names a parity: it passes when the current phase's parity is another one.  A warp
that has not looked by the time the next phase completes too therefore waits for a third one, which
may never come.  The model has the kernel's roles as lists of steps (two chain warps, of which the
first issues the chain's products, and two read-out warps, of which the first loads and issues P U;
the other warps of a role do what its second one does) and follows every order of the steps.
`test_the_model_follows_the_kernel` holds the source's waits and arrivals against the list that the
model was made from.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_prologue_b200", "csrc")
OUT, KEEP, MAP = "read-out", "kept for the backward", "map"

# What the source does with its barriers, in its order (arrivals of a commit or a copy included).
KERNEL = """
chain: arrive s_ready, wait full, wait s_ready, commit d_s, wait d_s, wait u_ready, arrive r_ready, wait r_ready,
  commit d_u, wait d_u, arrive w_ready, wait w_ready, wait q_read, commit d_acc, wait d_acc, arrive empty,
read-out: load, load, wait empty, load, wait full, wait s_ready, wait out_done, wait empty, load, wait d_s,
  arrive q_read, wait r_ready, wait d_u, arrive u_ready, arrive u_ready, wait u_ready, commit d_pu, wait d_pu,
  arrive out_done
"""


# A step: (kind, name, chunk).  wait: for the chunk's phase of a barrier; arrive; commit and load: an
# arrival at any later time; use: a buffer's contents of this chunk are read; give: they are written, which
# asks that all readers of what was there before (`depth` chunks earlier) are done.
DEPTH = dict(stage=2, s_scale=2, r_scale=2, U=1, QS=1, PU=1)


def full(c):
    return f"full{c & 1}"


def empty(c):
    return f"empty{c & 1}"


def chain(role, chunks, issuer, old):
    s = []
    for c in range(chunks):
        s += [("give", "s_scale", c), ("arrive", "s_ready", c), ("wait", full(c), c // 2)]
        if issuer:
            s += [("wait", "s_ready", c), ("give", "QS", c), ("commit", "d_s", c)]
        s += [("wait", "d_s", c), ("give", "r_scale", c)]
        freed = issuer and role != MAP and c > 0
        if freed and not old:
            s += [("wait", "u_ready", c - 1)]
        s += [("arrive", "r_ready", c)]
        if issuer:
            s += [("wait", "r_ready", c)]
            if freed and old:
                s += [("wait", "u_ready", c - 1)]
            s += [("give", "U", c), ("commit", "d_u", c)]
        s += [("wait", "d_u", c), ("arrive", "w_ready", c)]
        if issuer:
            s += [("wait", "w_ready", c)]
            if role == OUT:
                s += [("wait", "q_read", c)]
            s += [("over", "QS", c), ("commit", "d_acc", c)]
        s += [("wait", "d_acc", c), ("use", "stage", c)]
        if not old:
            s += [("arrive", empty(c), c // 2)]
    return s


def reader(role, chunks, issuer, old):
    s = [("load", full(c), c) for c in range(min(2, chunks))] if issuer else []
    for c in range(chunks):
        more = c > 0 and c + 1 < chunks
        if role == MAP:
            if not issuer:
                return s
            if old:
                s += [("wait", "s_ready", c)]
            elif more:
                s += [("wait", empty(c - 1), (c - 1) // 2)]
            if more:
                s += [("load", full(c + 1), c + 1)]
            continue
        s += [("wait", full(c), c // 2)]
        if role == OUT or old:
            s += [("wait", "s_ready", c)]
        if issuer and c > 0:
            s += [("wait", "out_done", c - 1)]
            if more:
                s += [] if old else [("wait", empty(c - 1), (c - 1) // 2)]
                s += [("load", full(c + 1), c + 1)]
        if role == OUT:
            s += [("use", "s_scale", c), ("wait", "d_s", c), ("use", "QS", c), ("arrive", "q_read", c)]
        s += [("wait", "r_ready", c), ("use", "r_scale", c), ("wait", "d_u", c), ("use", "U", c),
              ("arrive", "u_ready", c)]
        if role == OUT:
            if issuer:
                s += [("wait", "u_ready", c), ("give", "PU", c), ("commit", "d_pu", c)]
            s += [("wait", "d_pu", c), ("use", "PU", c)]
        s += [("use", "stage", c), ("arrive", "out_done", c)]
    return s


def explore(role, chunks, old=False):
    """None, or what went wrong: a warp that waits for good, or a buffer written too early."""
    agents = [chain(role, chunks, True, old), chain(role, chunks, False, old),
              reader(role, chunks, True, old), reader(role, chunks, False, old)]
    count = dict(s_ready=2, r_ready=2, w_ready=2, empty0=2, empty1=2, q_read=2, u_ready=2, out_done=2)
    names = sorted({x[1] for a in agents for x in a if x[0] in ("wait", "arrive", "commit", "load")})
    place = {n: i for i, n in enumerate(names)}

    def readers_done(pcs, name, c):
        want = ("use", name, c)
        return all(want not in a[pc:] for a, pc in zip(agents, pcs))

    # pcs, arrivals per barrier so far, and those still on their way (commits and copies)
    start = (tuple(0 for _ in agents), (0,) * len(names), (0,) * len(names))
    seen, todo = {start}, [start]

    def add(state):
        if state not in seen:
            seen.add(state)
            todo.append(state)

    def bump(t, i, d):
        return t[:i] + (t[i] + d,) + t[i + 1:]

    while todo:
        pcs, done, coming = todo.pop()
        moved = False
        for i, n in enumerate(coming):
            if n:
                moved = True
                add((pcs, bump(done, i, 1), bump(coming, i, -1)))
        for k, (a, pc) in enumerate(zip(agents, pcs)):
            if pc == len(a):
                continue
            kind, name, c = a[pc]
            nxt = bump(pcs, k, 1)
            if kind == "wait":
                phases = done[place[name]] // count.get(name, 1)
                if phases % 2 == c % 2:  # the current phase has the parity that is waited for
                    continue
                add((nxt, done, coming))
            elif kind == "arrive":
                add((nxt, bump(done, place[name], 1), coming))
            elif kind in ("commit", "load"):
                if kind == "load" and not readers_done(nxt, "stage", c - DEPTH["stage"]):
                    return f"chunk {c} is loaded over a stage in use"
                add((nxt, done, bump(coming, place[name], 1)))
            else:
                before = c if kind == "over" else c - DEPTH[name]
                if kind != "use" and not readers_done(nxt, name, before):
                    return f"{name} of chunk {c} is written while it is read"
                add((nxt, done, coming))
            moved = True
        if not moved and any(pc < len(a) for a, pc in zip(agents, pcs)):
            return "waits for good: " + ", ".join(str(a[pc]) for a, pc in zip(agents, pcs) if pc < len(a))
    return None


@pytest.mark.parametrize("role", [OUT, KEEP, MAP])
@pytest.mark.parametrize("chunks", [1, 2, 3, 6])
def test_every_order_ends(role, chunks):
    assert explore(role, chunks) is None


@pytest.mark.parametrize("role", [OUT, KEEP, MAP])
def test_the_model_sees_overtaken_waits(role):
    """The read-out warps' waits for s_ready (kept, map) and r_ready (all) without anything that holds
    the chain until they have looked: some order never ends."""
    assert "waits for good" in explore(role, 4, old=True)


def test_the_model_follows_the_kernel():
    with open(os.path.join(CSRC, "kda_gdr_state_tc.cu")) as f:
        src = f.read()
    body = src[src.index("if (warp < kChainWarps) {"):src.index("tmem_dealloc(tm")]
    chain_src, reader_src = body.split("  } else {\n    auto load = ", 1)
    chain_src = chain_src[chain_src.index("for (int c = 0; c < chunks; ++c)"):]
    call = re.compile(r"\bwait\(&sm\.(\w+)|\bwarp_arrive\(&sm\.(\w+)|\bcommit\(leader, &sm\.(\w+)"
                      r"|(\bload\()(?:0|1|c \+ 1)\)")

    def calls(text):
        out = []
        for w, a, m, ld in call.findall(text):
            out.append(f"wait {w}" if w else f"arrive {a}" if a else f"commit {m}" if m else "load")
        return out

    want = KERNEL.replace("\n", " ").split("read-out:")
    for text, listed in ((chain_src, want[0].replace("chain:", "")), (reader_src, want[1])):
        listed = [x.strip() for x in listed.split(",") if x.strip()]
        assert calls(text) == listed, (calls(text), listed)
