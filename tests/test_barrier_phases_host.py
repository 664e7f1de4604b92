"""The barrier protocols of kernels whose roles run ahead of one another, over every order in which
the roles can take their steps.

An mbarrier wait names a phase by its parity only.  A wait for phase k is right while k or k + 1
phases are complete; with k + 2 it blocks for good, with k - 1 it passes too early, and an arrival
that comes while another phase is open counts for that one.  Which barriers are arrays by parity is
read from the kernels' sources; the roles' steps are restated here."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mla_latent_kv_attn_b200", "csrc")


def declared(source, start, name):
    """The extents of barrier array `name`, declared behind `start` (empty for a single barrier)."""
    body = open(os.path.join(CSRC, source)).read().split(start, 1)[1]
    m = re.search(rf"uint64_t (?:[^;]*, )?{name}((?:\[[^\]]+\])*)[,;]", body)
    return re.findall(r"\[([^\]]+)\]", m.group(1))


class Roles:
    """Roles are lists of steps: ("wait", barrier, phase), ("arrive", barrier, phase),
    ("post", queue) and ("take", queue).  counts[barrier] arrivals end a phase."""

    def __init__(self, counts):
        self.counts, self.steps = counts, {}

    def role(self, name):
        return self.steps.setdefault(name, [])

    def explore(self):
        """Visits every reachable state; returns the first fault, or None."""
        names = list(self.steps)
        start = (0,) * len(names)
        seen, todo = {start}, [start]
        # arrivals and posts of a role up to each of its steps
        so_far = []
        for n in names:
            at, rows = {}, [{}]
            for kind, what, *_ in self.steps[n]:
                if kind != "wait":
                    at = {**at, (kind, what): at.get((kind, what), 0) + 1}
                rows.append(at)
            so_far.append(rows)
        while todo:
            state = todo.pop()
            total = lambda key: sum(so_far[i][pc].get(key, 0) for i, pc in enumerate(state))
            moved = False
            for i, n in enumerate(names):
                if state[i] == len(self.steps[n]):
                    continue
                kind, what, *phase = self.steps[n][state[i]]
                if kind == "take":
                    if total(("post", what)) <= total(("take", what)):
                        continue
                elif kind != "post":
                    done = total(("arrive", what)) // self.counts.get(what, 1)
                    if kind == "arrive" and done != phase[0]:
                        return f"{n}: arrival for phase {phase[0]} of {what} in phase {done}"
                    if kind == "wait" and not phase[0] <= done <= phase[0] + 1:
                        return f"{n}: waits for phase {phase[0]} of {what} with {done} complete"
                    if kind == "wait" and done == phase[0]:
                        continue
                moved = True
                after = state[:i] + (state[i] + 1,) + state[i + 1:]
                if after not in seen:
                    seen.add(after)
                    todo.append(after)
            if not moved and any(pc < len(self.steps[n]) for n, pc in zip(names, state)):
                return f"stuck at {dict(zip(names, state))}"
        return None


def by_parity(name, arrays):
    """(barrier, phase) of use u of a barrier that is or is not an array of two."""
    return lambda u: (f"{name}[{u & 1}]", u >> 1) if arrays else (name, u)


def dq_roles(tiles, ds_arrays):
    """cross_dq_tc_kernel: items of `tiles` tiles of states each, two softmax threads."""
    r = Roles({})
    a, b, threads = r.role("issuer S"), r.role("issuer dP, dQ"), [r.role("x0"), r.role("x1")]
    ta, tb = r.role("tensor S"), r.role("tensor dP, dQ")        # what the issuers' products complete
    dp_full, dq_done = by_parity("dp_full", True), by_parity("dq_done", True)
    ds_full = by_parity("ds_full", ds_arrays)
    for i in range(2):
        r.counts.update({"s_free": 2, "acc_free": 2, "ds_full": 2, f"ds_full[{i}]": 2})

    def issue_dp(u):
        if u >= 2:
            b.append(("wait", *dq_done(u - 2)))
        b.append(("post", "dP, dQ"))
        tb.extend([("take", "dP, dQ"), ("arrive", *dp_full(u))])

    t = 0
    for n, nt in enumerate(tiles):
        issue_dp(t)
        for j in range(nt):
            if t > 0:
                a.append(("wait", "s_free", t - 1))
            a.append(("post", "S"))
            ta.extend([("take", "S"), ("arrive", "s_full", t)])
            if j + 1 < nt:
                issue_dp(t + 1)
            b.append(("wait", *ds_full(t)))
            if j == 0 and n > 0:
                b.append(("wait", "acc_free", n - 1))
            b.append(("post", "dP, dQ"))
            tb.extend([("take", "dP, dQ"), ("arrive", *dq_done(t))])
            for x in threads:
                x.extend([("wait", "s_full", t), ("arrive", "s_free", t), ("wait", *dp_full(t)),
                          ("arrive", *ds_full(t))])
            t += 1
        for x in threads:
            x.extend([("wait", *dq_done(t - 1)), ("arrive", "acc_free", n)])
    return r


@pytest.mark.parametrize("tiles", [[5], [1, 1, 1, 1], [3, 2], [2, 1, 3]], ids=str)
def test_gradient_of_the_queries(tiles):
    arrays = declared("cross_bwd_sm100.cu", "struct DqShared {", "ds_full") == ["2"]
    assert dq_roles(tiles, arrays).explore() is None


def store_roles(items, arrays):
    """cross_fwd_tc_kernel's hand-over of O to the warp that stores it: items of one or two streams,
    two softmax threads each.  K and V of an item are loaded behind its Q tiles."""
    r = Roles({})
    producer, store = r.role("producer"), r.role("store")
    count = [0, 0]
    for n, streams in enumerate(items):
        for i in range(streams):
            c = count[i]
            buf = f"[{i}][{c & 1}]"
            if c >= 2:
                producer.append(("wait", "q_empty" + buf, (c >> 1) - 1))
            staged = (f"o_staged{buf}", c >> 1) if arrays else (f"o_staged[{i}]", c)
            r.counts.update({staged[0]: 2, f"o_free[{i}]": 2})
            store.extend([("wait", *staged), ("arrive", "q_empty" + buf, c >> 1)])
            issuer = r.role(f"issuer {i}")
            issuer.append(("take", f"loads {i}"))
            if c > 0:
                issuer.append(("wait", f"o_free[{i}]", c - 1))
            issuer.append(("arrive", f"pv_done[{i}]", c))
            for x in range(2):
                r.role(f"x{i}{x}").extend([("wait", f"pv_done[{i}]", c),
                                           ("arrive", f"o_free[{i}]", c), ("arrive", *staged)])
            count[i] += 1
        for i in range(streams):
            producer.append(("post", f"loads {i}"))
    return r


@pytest.mark.parametrize("items", [[2, 2, 2, 2], [1, 1, 1, 1, 1], [2, 2, 1, 1]], ids=str)
def test_stores_of_the_forward(items):
    arrays = declared("cross_sm100.cu", "struct FwdShared {", "o_staged") == ["2", "2"]
    assert store_roles(items, arrays).explore() is None


def aliased_p_roles(nt, arrays, rescale):
    """attention_tc_kernel with P in the S buffers (256 content latents): two softmax warps, of which
    those in `rescale` wait for the product before each tile's."""
    r = Roles({f"p_full[{i}]": 2 for i in range(2)} | {"p_full": 2})
    qk, pv = r.role("issuer QK"), r.role("issuer PV")
    tqk, tpv = r.role("tensor QK"), r.role("tensor PV")
    s_full, buf_done = by_parity("s_full", True), by_parity("pv_buf_done", True)
    p_full = by_parity("p_full", arrays)
    for j in range(nt):
        if j >= 2:
            qk.append(("wait", *buf_done(j - 2)))
        qk.append(("post", "QK"))
        tqk.extend([("take", "QK"), ("arrive", *s_full(j))])
        pv.extend([("wait", *p_full(j)), ("post", "PV")])
        tpv.extend([("take", "PV"), ("arrive", "pv_done", j), ("arrive", *buf_done(j))])
    for x in range(2):
        steps = r.role(f"x{x}")
        for j in range(nt):
            steps.append(("wait", *s_full(j)))
            if x in rescale and j > 0:
                steps.append(("wait", "pv_done", j - 1))
            steps.append(("arrive", *p_full(j)))
        steps.append(("wait", *(buf_done(nt - 1) if arrays else ("pv_done", nt - 1))))
    return r


@pytest.mark.parametrize("rescale", [(), (0,), (0, 1)], ids=str)
@pytest.mark.parametrize("nt", [1, 2, 3, 6])
def test_probabilities_in_the_score_buffers(nt, rescale):
    arrays = declared("attention_sm100.cu", "attention_tc_kernel(", "p_full") == ["kAliasP ? 2 : 1"]
    assert aliased_p_roles(nt, arrays, rescale).explore() is None


def test_a_single_barrier_misses_a_phase():
    """The explorer finds what it is for: with one barrier for every use, arrivals for a phase come
    while the one before it is open."""
    assert dq_roles([3], False).explore() is not None
    assert store_roles([2, 2, 2], False).explore() is not None
    assert aliased_p_roles(3, False, ()).explore() is not None
