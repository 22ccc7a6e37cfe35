"""The barriers of pa_attn_tc_kernel (pa_attn_tc.cu) in a model, without a GPU: whatever the warps' timing, no wait misses
its phase.  A segment's entries are its blocks, then one without a block for each of the two softmax groups; a request
without keys (a padded batch) is a segment of no block."""

import itertools

import pytest

from tests.barrier_order import Order

SEGMENTS = [*itertools.product((0, 1, 2), repeat=3), (3, 0, 0, 0, 1), (1, 0, 1, 0, 2, 1), (0, 0, 0, 0, 0, 1), (2, 3, 0, 0, 3, 1, 1)]


def kernel(segments, stages, without=()):
    """The roles' programs for segments of that many blocks; without: waits that are left out."""
    o = Order()

    def wait(agent, bar, phase, name=None):
        if (name or bar) not in without:
            o.wait(agent, bar, phase)
    entries = [(seg, i < n, i == n) for seg, n in enumerate(segments) for i in range(n + 2)]  # segment, a block, the first end
    for j, (seg, block, _) in enumerate(entries):  # the copies
        wait("copies", f"empty{j % stages}", j // stages - 1)
        o.touch("copies", "w", f"info{j % 16}", j)
        if block:
            o.touch("copies", "w", f"stage{j % stages}", j)
        o.arrive("copies", f"full{j % stages}", j // stages, 1)
    for i in range(4):  # keys and queries
        k = f"keys{i}"

        def lay_out(seg):
            o.touch(k, "w", f"q tile {i}", seg)
            o.touch(k, "w", f"row_scale{seg & 1} {i}", seg)
            o.arrive(k, "item_full", seg, 8)
        lay_out(0)
        for j, (seg, block, end) in enumerate(entries):
            wait(k, f"full{j % stages}", j // stages)
            wait(k, "k_empty", j - 1)
            o.touch(k, "r", f"info{j % 16}", j)
            if block:
                o.touch(k, "r", f"stage{j % stages}", j)
                o.touch(k, "w", f"k tile {i}", j)
                o.touch(k, "w", f"scales{j & 3} {i}", j)
            o.arrive(k, "k_full", j, 4)
            o.arrive(k, f"empty{j % stages}", j // stages, 8)
            if end and seg + 1 < len(segments):
                wait(k, "item_seen", seg)
                lay_out(seg + 1)
    for i in range(4):  # values
        v, nv = f"values{i}", 0
        last = None
        for j, (seg, block, _) in enumerate(entries):
            if seg != last:
                last = seg
                wait(v, "item_seen", seg - 1, "softmax in the segment before")
                o.touch(v, "w", f"notes{(seg + 1) & 3} {i}", seg + 1)
                o.arrive(v, "item_full", seg, 8)
            wait(v, f"full{j % stages}", j // stages)
            o.touch(v, "r", f"info{j % 16}", j)
            if block:
                wait(v, "v_empty", nv - 1)
                o.touch(v, "r", f"stage{j % stages}", j)
                o.touch(v, "w", f"v tile {i}", nv)
                for part in range(4):
                    o.touch(v, "a", f"notes{seg & 3} {part}", seg)
                o.arrive(v, "v_full", nv, 4)
                nv += 1
            o.arrive(v, f"empty{j % stages}", j // stages, 8)
    # the thread that issues the products, and the tensor core, which takes them in order
    nb, had, pc, ns, pending, last = 0, [0, 0], [0, 0], [0, 0], None, None
    for j, (seg, block, _) in enumerate(entries):
        g = j & 1
        if seg != last:
            last, any_yet = seg, False
            wait("mma", "meet", seg - 1, "ends taken")
        wait("mma", "k_full", j)
        o.touch("mma", "r", f"info{j % 16}", j)
        if block:
            wait("mma", f"pv_done{g}", had[g] - 1)
            at = o.op("mma", "issues S")
            for i in range(4):
                o.touch("tensor", "r", f"q tile {i}", seg, (at,))
                o.touch("tensor", "r", f"k tile {i}", j)
                o.touch("tensor", "w", f"S{g} {i}", ("S", j))
            o.arrive("tensor", f"s_full{g}", ns[g], 1, (at,))
            o.arrive("tensor", "k_empty", j, 1, (at,))
            had[g] += 1
            ns[g] += 1
        if pending is not None:
            h = g ^ 1
            wait("mma", f"p_full{h}", pc[h])
            wait("mma", "v_full", nb)
            if not any_yet:
                wait("mma", "seg_done", seg - 1)
            any_yet = True
            at = o.op("mma", "issues PV")
            for i in range(4):
                o.touch("tensor", "r", f"S{h} {i}", ("P", pending), (at,))
                o.touch("tensor", "r", f"v tile {i}", nb)
                o.touch("tensor", "w", f"O{h} {i}", (seg, pending))
            o.arrive("tensor", f"pv_done{h}", pc[h], 1, (at,))
            o.arrive("tensor", "v_empty", nb, 1, (at,))
            pc[h] += 1
            nb += 1
        pending = j if block else None
        if not block:
            o.arrive("tensor", f"s_full{g}", ns[g], 1, (o.op("mma", "issues an end"),))
            ns[g] += 1
            o.arrive("mma", "k_empty", j, 1)
    for g, i in itertools.product(range(2), range(4)):  # softmax
        s, n, blocks = f"softmax{g}{i}", 0, 0
        for seg in range(len(segments)):
            wait(s, "item_full", seg)
            o.arrive(s, "item_seen", seg, 8)
            for part in range(4):
                o.touch(s, "r", f"row_scale{seg & 1} {part}", seg)
            mine = [j for j, e in enumerate(entries) if e[0] == seg and j & 1 == g]
            for j in mine:
                wait(s, f"s_full{g}", n)
                n += 1
                o.touch(s, "r", f"info{j % 16}", j)
                if entries[j][1]:
                    o.touch(s, "r", f"S{g} {i}", ("S", j))
                    for part in range(4):
                        o.touch(s, "r", f"scales{j & 3} {part}", j)
                    if j != mine[0]:  # the references move
                        o.touch(s, "r", f"O{g} {i}", (seg, j - 2))
                        o.touch(s, "w", f"O{g} {i}", (seg, j - 2))
                    o.touch(s, "w", f"S{g} {i}", ("P", j))
                    o.arrive(s, f"p_full{g}", blocks, 4)
                    blocks += 1
            o.touch(s, "w", f"sums{g} {i}", seg)
            o.arrive(s, "meet", seg, 8)
            wait(s, "meet", seg)
            for h in range(2):
                o.touch(s, "r", f"sums{h} {i}", seg)
                of_h = [j for j, e in enumerate(entries) if e[0] == seg and e[1] and j & 1 == h]
                if of_h:
                    o.touch(s, "r", f"O{h} {i}", (seg, of_h[-1]))
            for part in range(4):
                o.touch(s, "r", f"notes{seg & 3} {part}", seg)
            o.arrive(s, "seg_done", seg, 8)
            wait(s, "seg_done", seg)
    return o


@pytest.mark.parametrize("stages", [3, 4, 5])
def test_no_phase_is_missed_and_nothing_is_read_too_early(stages):
    for segments in SEGMENTS:
        assert kernel(segments, stages).faults() == [], segments


@pytest.mark.parametrize("missing,segments,of", [
    ("ends taken", (1, 0, 1), "s_full"), ("ends taken", (0, 0, 0), "s_full"),  # the products' thread runs ahead of the softmax
    ("item_seen", (1, 1, 1), "item_full"), ("softmax in the segment before", (0, 0, 0, 1), "notes"), ("k_full", (1, 1), "k tile"),
    ("v_empty", (2,), "v tile"), ("meet", (1, 1), "sums"), ("full1", (2,), "stage1")])
def test_a_missing_wait_is_found(missing, segments, of):
    assert any(of in str(f) for f in kernel(segments, 3, [missing]).faults())
