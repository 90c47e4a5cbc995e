"""The ring of bucket tiles of the attention over the 8-bit cache, as a small model on the host (no GPU): one warp copies
the tiles in order and copies land in any order, two groups of softmax threads take alternate tiles, and products are
issued in order, scores two tiles ahead.  Every order of these steps is gone through."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_graph_spmv_gb300", "csrc")


def passes(completed, parity):
    """A barrier's wait for a phase of this parity, after so many completed phases: it does not tell a phase from the next but one."""
    return completed % 2 != parity


def read_too_early(buffers, tiles=9):
    """A tile whose group gets past its wait while its buffer holds something else, or None if no order of steps has one."""
    # copied tiles, copies under way, buffers' tiles, phases of full and empty; of both groups: tile and step; finished tiles
    start = (0, (), (None,) * buffers, (0,) * buffers, (0,) * buffers, ((0, 0), (1, 0)), ())
    seen, todo = {start}, [start]

    def put(t, i, x):
        return t[:i] + (x,) + t[i + 1:]

    while todo:
        copied, flying, holds, full, empty, groups, finished = todo.pop()
        after = []
        if copied < tiles and (copied < buffers or passes(empty[copied % buffers], (copied // buffers - 1) & 1)):
            after.append((copied + 1, tuple(sorted(flying + (copied,))), holds, full, empty, groups, finished))
        for t in flying:
            b = t % buffers
            after.append((copied, tuple(x for x in flying if x != t), put(holds, b, t), put(full, b, full[b] + 1), empty, groups, finished))
        products = 0                                     # issued in order, as weights are there
        while products in finished:
            products += 1
        for w, (i, step) in enumerate(groups):
            if i >= tiles:
                continue
            b = i % buffers
            if step == 0 and passes(full[b], (i // buffers) & 1):        # bucket bytes; first biases
                if holds[b] != i:
                    return i
                after.append((copied, flying, holds, full, empty, put(groups, w, (i, 1)), finished))
            elif step == 1 and (i < 2 or products > i - 2):              # scores; the other biases, weights
                if holds[b] != i:
                    return i
                after.append((copied, flying, holds, full, put(empty, b, empty[b] + 1), put(groups, w, (i + 2, 0)), tuple(sorted(finished + (i,)))))
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


def buffers_of(kernel):
    with open(os.path.join(CSRC, kernel)) as f:
        found = re.findall(r"constexpr int kBufs = (\d+);", f.read())
    assert len(found) == 1
    return int(found[0])


def test_three_buffers_can_be_read_too_early():
    """A buffer's uses take turns between the groups: at tile i a group has waited for no copy of tile i - 3, and nothing it
    waited for has."""
    assert read_too_early(3) is not None


@pytest.mark.parametrize("buffers", [2, 4])
def test_a_buffer_of_one_group_is_not(buffers):
    assert read_too_early(buffers) is None


def test_the_kernels_ring_is_not_read_too_early():
    assert read_too_early(buffers_of("k2t_attn_cached.cuh")) is None


def test_bytes_are_not_looked_up_after_a_wait_that_ran_out():
    """What lies in a buffer whose wait ran out may be any byte, and byte 255 of 16 heads is 16320 bytes into a table of at most
    4224 that ends less than that before the block's shared memory does.  Between such a wait and the lookups the
    bytes are dropped, and every lookup asks whether there are any."""
    with open(os.path.join(CSRC, "k2t_attn_cached.cuh")) as f:
        loop = f.read().split("for (uint32_t i = w; i < tiles; i += 2, ++mine)")[1].split("sum.add(tile_sum)")[0]
    early, rest = loop.split("ok = __all_sync(~0u, ok);")
    first = early.split("hop_full[buf]")[1]
    assert first.index("bytes = bytes && ok;") < first.index("look_up(")
    assert rest.index("bytes = bytes && ok;") < min(rest.index(x) for x in ("look_up(", "bias_scores("))
    for part in (early, rest):
        for at in re.finditer(r"look_up\(", part):
            assert re.search(r"if \([^\n]*bytes\)[^;]*$", part[:at.start()])
    assert "bias_scores(s, sc, !bytes," in rest
