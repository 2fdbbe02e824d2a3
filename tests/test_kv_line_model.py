"""CPU model of how the attention kernels cut their work (kv_attention.cu,
kv_prefill.cu): items laid end to end on a line, each `overhead` units and then its
steps, the line cut evenly among workers.  Every step must be done exactly once, an item
done by one worker written by it, and an item shared by several joined exactly once from
parts that are where the joining looks for them.  The rules are those of the kernels,
restated."""
import random

import pytest


def _cut(items, workers, overhead):
    start = [0]
    for steps in items:
        start.append(start[-1] + overhead + steps)
    total = start[-1]
    begins = [w * total // workers for w in range(workers + 1)]
    holder = lambda unit: ((unit + 1) * workers - 1) // total  # largest w with begins[w] <= unit
    whole, parts = set(), {}
    for w in range(workers):
        at, i = begins[w], 0
        while at < begins[w + 1]:
            while start[i + 1] <= at:
                i += 1
            first, end = start[i], start[i + 1]
            step0 = max(0, at - first - overhead)
            step1 = min(begins[w + 1], end) - first - overhead
            if step1 <= step0:
                break
            if step0 == 0 and step1 == items[i]:
                assert i not in whole
                whole.add(i)
            else:
                key = (w, 0 if at == begins[w] else 1)
                assert key not in parts
                g0 = holder(first + overhead)
                parts[key] = dict(item=i, steps=(step0, step1), g0=g0, last=holder(end - 1),
                                  head_slot=0 if begins[g0] >= first else 1,
                                  joins=step0 > 0 and at == begins[g0 + 1])
            at = first + overhead + step1
    return whole, parts


@pytest.mark.parametrize("workers", [1, 2, 3, 7, 148, 592])
@pytest.mark.parametrize("overhead", [0, 1, 2, 3, 5])
def test_every_item_is_finished_once(workers, overhead):
    rng = random.Random(workers * 10 + overhead)
    for _ in range(60):
        items = [rng.choice([1, 1, 2, 3, 40, rng.randint(1, 1500)]) for _ in range(rng.randint(1, 60))]
        whole, parts = _cut(items, workers, overhead)
        joined = set()
        for k in range(1, workers):
            p = parts.get((k, 0))
            if p is None or not p["joins"]:
                continue
            assert p["item"] not in joined
            joined.add(p["item"])
            covered = []
            for w in range(p["g0"], p["last"] + 1):
                q = parts.get((w, p["head_slot"] if w == p["g0"] else 0))
                if q is None:
                    continue  # a worker without steps of it
                assert q["item"] == p["item"]
                covered.append(q["steps"])
            assert covered[0][0] == 0 and covered[-1][1] == items[p["item"]]
            assert all(a[1] == b[0] for a, b in zip(covered, covered[1:]))
        assert not joined & whole
        assert joined | whole == set(range(len(items)))
