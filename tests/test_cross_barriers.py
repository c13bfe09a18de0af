"""The barriers of the cross attention kernels, as a model on the CPU: every order in which the roles of a
CTA can run ends, whatever the time that each of them takes.

A role is the list of its waits and arrivals in program order, several items long; the tensor core is a
queue that works in order and arrives for each commit.  A wait for a parity passes when the phase before
the barrier's current one had that parity, which is the rule of the hardware's barriers: a role that
looks after two phases have passed does not see the first.  All states that any interleaving reaches are
searched; one in which nothing can move and not all roles are done is a stall.  Tile loads and the
scrubber keep ring order with the rest and are left out.
"""
import pytest

WARPS = 2                                                      # elementwise warps of the model (8 in the kernels)


def search(arrivals, roles):
    """Number of states reached, or the state of a stall."""
    names = list(arrivals)
    at = {b: i for i, b in enumerate(names)}
    need = [arrivals[b] for b in names]
    start = (tuple(0 for _ in roles), tuple((0, n) for n in need), ())
    seen, todo = {start}, [start]

    def arrive(bars, b):
        phase, left = bars[at[b]]
        out = list(bars)
        out[at[b]] = (phase ^ 1, need[at[b]]) if left == 1 else (phase, left - 1)
        return tuple(out)
    while todo:
        pcs, bars, queue = todo.pop()
        nexts = []
        if queue:                                              # the tensor core reaches the oldest commit
            nexts.append((pcs, arrive(bars, queue[0]), queue[1:]))
        for r, prog in enumerate(roles):
            if pcs[r] == len(prog):
                continue
            op, b, *parity = prog[pcs[r]]
            pc = pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:]
            if op == "wait" and bars[at[b]][0] != parity[0]:
                nexts.append((pc, bars, queue))
            elif op == "arrive":
                nexts.append((pc, arrive(bars, b), queue))
            elif op == "commit":
                nexts.append((pc, bars, queue + (b,)))
        if not nexts and any(pc < len(p) for pc, p in zip(pcs, roles)):
            return dict(stall={r: prog[pcs[r]] for r, prog in enumerate(roles) if pcs[r] < len(prog)})
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return len(seen)


def dq(items, ds_barriers):
    """Roles of the dQ kernel for items of so many key tiles: products, elementwise warps, store."""
    arrivals = dict(QF=1, QE=1, SF=1, SR=WARPS, PF0=1, PF1=1, AF=1, AE=1)
    arrivals |= {"DS%d" % i: WARPS for i in range(ds_barriers)}

    def ds(g):
        return "DS%d" % (g % ds_barriers), (g // ds_barriers) & 1
    mma, elem, store, load = [], [], [], []
    g = 0
    pending = None
    for n, tiles in enumerate(items + [None]):
        if tiles is not None:
            load += [("wait", "QE", (n & 1) ^ 1), ("arrive", "QF")]
            store += [("wait", "AF", n & 1), ("arrive", "AE")]
        for j in range(tiles or 1):
            if tiles is not None:
                if j == 0:
                    mma.append(("wait", "QF", n & 1))
                if g > 0:
                    mma.append(("wait", "SR", (g - 1) & 1))
                mma.append(("commit", "SF"))
                if j == tiles - 1:
                    mma.append(("commit", "QE"))
                mma.append(("commit", "PF%d" % (g & 1)))
                elem += [("wait", "SF", g & 1), ("arrive", "SR"), ("wait", "PF%d" % (g & 1), (g >> 1) & 1), ("arrive", ds(g)[0])]
            if pending:
                mma.append(("wait", *ds(g - 1)))
                if pending["first"] and pending["item"] > 0:
                    mma.append(("wait", "AE", (pending["item"] - 1) & 1))
                if pending["last"]:
                    mma.append(("commit", "AF"))
            if tiles is not None:
                pending = dict(first=j == 0, last=j == tiles - 1, item=n)
                g += 1
    return arrivals, [mma, store, load] + [elem] * WARPS


def dkv(items):
    """Roles of the dK/dV kernel for items of so many query tiles: products, elementwise warps."""
    arrivals = dict(SF=1, SR=WARPS, PF=1, DS=WARPS, AF=1, AE=WARPS)
    mma, elem = [], []
    g = 0
    pending = None
    for n, tiles in enumerate(items + [None]):
        for i in range(tiles or 1):
            if tiles is not None:
                if g > 0:
                    mma.append(("wait", "SR", (g - 1) & 1))
                mma.append(("commit", "SF"))
                elem += [("wait", "SF", g & 1), ("arrive", "SR"), ("wait", "PF", g & 1), ("arrive", "DS")]
            if i == 0 and n > 0:
                elem += [("wait", "AF", (n - 1) & 1), ("arrive", "AE")]
            if pending:
                mma.append(("wait", "DS", (g - 1) & 1))
                if pending["first"] and pending["item"] > 0:
                    mma.append(("wait", "AE", (pending["item"] - 1) & 1))
                if pending["last"]:
                    mma.append(("commit", "AF"))
            if tiles is None:
                break
            mma.append(("commit", "PF"))
            pending = dict(first=i == 0, last=i == tiles - 1, item=n)
            g += 1
    return arrivals, [mma] + [elem] * WARPS


def forward(items):
    """Roles of the forward kernel for items of (query tiles, key tiles): products, each query tile's
    softmax warps, output, Q's loads."""
    arrivals = dict(QF=1, QE=1)
    for t in (0, 1):
        arrivals |= {"SF%d" % t: 1, "PF%d" % t: WARPS, "OF%d" % t: 1, "OE%d" % t: 1}
    steps = [dict(item=n, ntile=nt, first=j == 0, last=j == nk - 1) for n, (nt, nk) in enumerate(items) for j in range(nk)]
    mma, soft, out, load = [], [[], []], [], []
    pc, oc, sc, done, q = [0, 0], [0, 0], [0, 0], [0, 0], 0
    for prev, cur in zip([None] + steps, steps + [None]):
        for t in (0, 1):
            if prev and t < prev["ntile"]:
                mma.append(("wait", "PF%d" % t, pc[t] & 1))
                pc[t] += 1
                if prev["first"]:
                    if oc[t] > 0:
                        mma.append(("wait", "OE%d" % t, (oc[t] - 1) & 1))
                    oc[t] += 1
                if prev["last"]:
                    mma.append(("commit", "OF%d" % t))
            if cur and t < cur["ntile"]:
                if t == 0 and cur["first"]:
                    mma.append(("wait", "QF", q & 1))
                mma.append(("commit", "SF%d" % t))
                soft[t] += [("wait", "SF%d" % t, sc[t] & 1), ("arrive", "PF%d" % t)]
                sc[t] += 1
        if cur and cur["last"]:
            mma.append(("commit", "QE"))
            q += 1
    for n, (nt, _) in enumerate(items):
        load += [("wait", "QE", (n & 1) ^ 1), ("arrive", "QF")]
        for t in range(nt):
            out += [("wait", "OF%d" % t, done[t] & 1), ("arrive", "OE%d" % t)]
            done[t] += 1
    return arrivals, [mma, out, load] + [soft[0]] * WARPS + [soft[1]] * WARPS


@pytest.mark.parametrize("items", [[1, 1, 1], [1, 3, 2], [2, 1, 1, 2], [5]])
def test_dq_never_stalls(items):
    assert isinstance(search(*dq(items, ds_barriers=2)), int)


def test_dq_with_one_barrier_for_dS_would_stall():
    """Step g's dS may be stored before the products' warp looks for step g - 1's."""
    got = search(*dq([3], ds_barriers=1))
    assert isinstance(got, dict) and got["stall"][0][:2] == ("wait", "DS0")


@pytest.mark.parametrize("items", [[1, 1, 1], [1, 3, 2], [2, 1, 1, 2], [5]])
def test_dkv_never_stalls(items):
    assert isinstance(search(*dkv(items)), int)


@pytest.mark.parametrize("items", [[(2, 1), (2, 1), (2, 1)], [(2, 2), (1, 1), (2, 3)], [(1, 3), (1, 1), (2, 1)], [(2, 4)]])
def test_forward_never_stalls(items):
    assert isinstance(search(*forward(items)), int)
