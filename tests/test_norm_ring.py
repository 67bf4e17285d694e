"""The ring of layer norm's kernels (tg_norm.cu): what it rests on and no result shows, in a model of
its arithmetic and in its source."""

import os
import random
import re

from fp16_gemm_relu_gb300 import build


def source():
    with open(os.path.join(build.CSRC, "tg_norm.cu")) as f:
        return f.read()


def ring_kernels():
    found = [m.group(0) for m in re.finditer(r"__global__.*?\n}\n", source(), re.S)
             if "fetch_blocks" in m.group(0)]
    assert len(found) == 2
    return found


def edges(base, ld, rows, n, row):
    """Bytes of a row that fetch_edges writes, as (first, last), from span_of and plan_fetch."""
    lo, hi = (base + 15) & ~15, (base + 2 * ((rows - 1) * ld + n)) & ~15
    a = base + 2 * row * ld
    z = a + 2 * n
    start, end = a & ~15, (z + 15) & ~15
    begin, to = max(start, lo), min(end, hi)
    to = max(to, begin)
    return max(min(z, begin) - a, 0), max(z - max(to, a), 0)


def test_only_the_first_and_last_row_have_edges():
    """So a slot's generic writes come before a later copy into it only among the first fetches."""
    rng = random.Random(1)
    for _ in range(3000):
        n, rows = rng.randint(513, 16384), rng.randint(1, 40)
        ld, base = n + rng.randint(0, 40), 256 + 2 * rng.randint(0, 7)
        for r in range(rows):
            first, last = edges(base, ld, rows, n, r)
            assert (first == 0 or r == 0) and (last == 0 or r == rows - 1)


def test_generic_writes_of_a_slot_come_before_later_copies():
    for text in ring_kernels():
        assert re.search(r"s < S && s < count; \+\+s\) fetch\(s, s\);\s*//[^\n]*\s*"
                         r"if constexpr \(!VEC\) tg::fence_async_smem\(\);", text)


def test_the_drain_waits_for_the_last_fetch_of_each_slot():
    # fetch k goes to slot k mod S and is that slot's phase k / S, whose parity is waited for
    for S in (2, 3):
        for fetched in range(1, 40):
            for s in range(min(S, fetched)):
                last = max(k for k in range(fetched) if k % S == s)
                assert last // S & 1 == (fetched - 1 - s) // S & 1


def test_after_a_timeout_nothing_more_is_fetched_and_copies_are_waited_for():
    assert "(fetched - 1 - s) / S) & 1u" in source()
    for text in ring_kernels():
        assert "if (fetcher && k + S < count) fetch(k + S, s);" in text
        assert text.count("fetch(") == 2  # the first fetches, and that one
        waits = re.findall(r"if \(!slot_wait\([^;]*fetcher\) \{\s*slots_drain<S>\([^;]*;\s*"
                           r"fetcher = false;", text)
        assert len(waits) == 1 == text.count("slot_wait(")
