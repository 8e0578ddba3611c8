"""CPU-only checks of what the operator classes refuse before they call the library."""
import itertools
import random

import grouped_gemm_device_gb300 as g


def test_written_tensors_that_share_memory_are_found():
    """Against every pair of spans: two that overlap, at least one of them written."""
    r = random.Random(0)
    seen = set()
    for _ in range(3000):
        def span():
            return r.randrange(1, 60), r.choice([0, 1, 2, 5, 12])
        grads = [span() for _ in range(r.randrange(1, 5))]
        outs = [s if r.random() < 0.5 else span() for s in grads]
        items = [(o, True) for o in outs] + [(a, False) for a, o in zip(grads, outs) if a != o]
        want = any((wa or wb) and max(a[0], b[0]) < min(a[0] + a[1], b[0] + b[1])
                   for (a, wa), (b, wb) in itertools.combinations(items, 2))
        assert g._collide(grads, outs) == want
        seen.add(want)
    assert seen == {True, False}
