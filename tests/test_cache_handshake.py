"""How the roles of the fp32 kernel for many rows (csrc/cache_tc32.cu) hand units and queries to
one another, as a model whose every order of steps is tried on the host.

A barrier counts its arrivals; a wait names a parity, as the kernel's waits do, and passes while
the phase under way has the other one.  A role that is two phases behind
therefore waits for good: such an order must not exist.
"""
from collections import deque

SLOTS = 3                # unit records in flight (kRecSlots)


def decoder(units):
    """Publishes a record per unit, and one that ends every role."""
    for k in range(len(units) + 1):
        yield ("wait", f"empty{k % SLOTS}", (k // SLOTS & 1) ^ 1)
        yield ("arrive", f"full{k % SLOTS}")


def product(units, skips):
    count = issued = added = 0
    for k, tiles in enumerate(units):
        yield ("wait", f"full{k % SLOTS}", k // SLOTS & 1)
        yield ("arrive", f"empty{k % SLOTS}")
        if skips and tiles == 0:
            continue
        yield ("wait", "queries", count & 1)
        count += 1
        for j in range(tiles):                   # scores of a tile ahead, then a tile's output
            for _ in range((j == 0) + (j + 1 < tiles)):
                yield ("arrive", f"scores{issued & 1}")
                issued += 1
            yield ("wait", f"weights{added & 1}", added >> 1 & 1)
            added += 1
    yield ("wait", f"full{len(units) % SLOTS}", len(units) // SLOTS & 1)


def softmax(units, skips):
    it = 0
    for k, tiles in enumerate(units):
        yield ("wait", f"full{k % SLOTS}", k // SLOTS & 1)
        if tiles or not skips:
            yield ("arrive", "queries")
        for _ in range(tiles):
            yield ("wait", f"scores{it & 1}", it >> 1 & 1)
            yield ("arrive", f"weights{it & 1}")
            it += 1
        yield ("arrive", f"empty{k % SLOTS}")
    yield ("wait", f"full{len(units) % SLOTS}", len(units) // SLOTS & 1)


def stuck_orders(units, skips):
    """Whether some order of the roles' steps ends with a role waiting for good."""
    roles = [list(decoder(units)), list(product(units, skips)), list(softmax(units, skips))]
    names = sorted({s[1] for r in roles for s in r})
    need = {n: 2 if n.startswith("empty") else 1 for n in names}     # arrivals of a phase
    start = ((0,) * len(roles), (0,) * len(names))                   # steps done, arrivals
    seen, todo = {start}, deque([start])
    while todo:
        at, arrived = todo.popleft()
        moved = False
        for r, steps in enumerate(roles):
            if at[r] == len(steps):
                continue
            step = steps[at[r]]
            b = names.index(step[1])
            now = arrived
            if step[0] == "wait":
                if (arrived[b] // need[step[1]] & 1) == step[2]:     # that phase is under way
                    continue
            else:
                now = arrived[:b] + (arrived[b] + 1,) + arrived[b + 1:]
            moved = True
            nxt = (at[:r] + (at[r] + 1,) + at[r + 1:], now)
            if nxt not in seen:
                seen.add(nxt)
                todo.append(nxt)
        if not moved and any(a < len(s) for a, s in zip(at, roles)):
            return True
    return False


RUNS = [[], [0], [2], [0, 0, 0, 0, 0], [1, 0, 0, 2], [0, 0, 1, 0, 0, 0, 1], [2, 1, 0, 0, 0, 0, 2], [1, 1, 1, 1]]


def test_queries_of_units_without_tiles_could_pass_unseen():
    """A barrier for every unit's queries, nothing back from the products: the softmax warps pass
    units without a tile as fast as the records come, and the products miss a phase."""
    assert stuck_orders([0, 0, 0, 0, 0], skips=False)
    assert not stuck_orders([1, 1, 1, 1], skips=False)


def test_no_order_of_the_roles_waits_for_good():
    for units in RUNS:
        assert not stuck_orders(units, skips=True), units
