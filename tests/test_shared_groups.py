"""The groups of a step that shares prefixes: cut where that saves the most
reading (no GPU)."""
import itertools

import numpy as np
import pytest

from paged_kv_cache_139_gb300 import engine

B = 4


def tables_of(common, width):
    """Block tables whose neighbours e and e + 1 begin with common[e] equal blocks."""
    t = np.zeros((len(common) + 1, width), np.int32)
    fresh = 0
    for s in range(len(common) + 1):
        k = int(common[s - 1]) if s else 0
        t[s, :k] = t[s - 1, :k]
        t[s, k:] = np.arange(fresh, fresh + width - k)
        fresh += width - k
    return t


def find(common, width=None):
    width = width or max([1, *common]) + 1
    return engine.SharedGroups.find(tables_of(common, width), np.full(len(common) + 1, width * B), B)


def saved(g):
    """Blocks that a step with these groups does not read again."""
    first = g.start[:-1]
    return int((g.prefix[first] // B * (np.diff(g.start) - 1)).sum())


def most(common):
    """The most that any cuts save, and the fewest groups that save it, by trying all."""
    best = (-1, 0)
    for cuts in itertools.product((False, True), repeat=len(common)):
        total, part = 0, []
        for e, c in enumerate([*cuts, True]):
            if c:
                total, part = total + len(part) * min(part, default=0), []
            else:
                part.append(common[e])
        # (neighbours that share nothing are always parted: a group without a prefix is none)
        if all(c or v for c, v in zip(cuts, common)):
            best = max(best, (total, -1 - sum(cuts)))
    return best[0], -best[1]


def test_a_stranger_before_forks_keeps_its_hands_off_their_prefix():
    """One request that shares the first block with the 64 forks of a long prompt after it."""
    g = find([1] + [125] * 63)
    assert g.start.tolist() == [0, 1, 65] and g.prefix.tolist() == [0] + [500] * 64


def test_two_prompts_after_one_instruction():
    g = find([9, 9, 9, 2, 30, 30, 30])
    assert g.start.tolist() == [0, 4, 8] and g.prefix.tolist() == [36] * 4 + [120] * 4


def test_the_best_part_in_the_middle():
    assert find([1, 1, 9, 1, 1]).start.tolist() == [0, 2, 4, 6]


def test_of_equal_savings_the_fewest_groups():
    assert find([2, 1, 1, 1]).start.tolist() == [0, 5]


@pytest.mark.parametrize("seed", range(6))
def test_no_cuts_save_more(seed):
    rng = np.random.default_rng(seed)
    for _ in range(60):
        n = int(rng.integers(0, 10))
        common = rng.integers(0, (2, 3, 4, 12, 40, 5)[seed], n).tolist()
        if seed == 5:                                    # longer stretches of one value
            common = np.repeat(common, 2)[:9].tolist()
        g = find(common)
        assert g.start[0] == 0 and g.start[-1] == len(common) + 1 and (np.diff(g.start) > 0).all()
        assert (saved(g), len(g.start) - 1) == most(common), common
        for a, b in zip(g.start[:-1], g.start[1:]):
            shares = min(common[a:b - 1], default=0)
            assert (g.prefix[a:b] == shares * B).all()


def test_full_blocks_bound_what_neighbours_share():
    t = tables_of([5, 5], 6)
    g = engine.SharedGroups.find(t, np.array([24, 13, 24]), B)
    assert g.start.tolist() == [0, 3] and g.prefix.tolist() == [12] * 3
    g = engine.SharedGroups.find(t, np.array([24, 3, 24]), B)
    assert g.start.tolist() == [0, 1, 2, 3] and not g.prefix.any()


def test_prefixes_of_many_lengths():
    """Neighbours part before, at and behind every stretch of blocks that is compared at once."""
    common = [0, 1, 2, 8, 9, 10, 72, 73, 74, 512, 583, 584, 585, 586, 1096, 1097, 1098, 1300, 0, 1300, 585, 1]
    t = tables_of(common, 1301)
    for full in (1300, 1301):
        ctx = np.full(len(t), full * B)
        g = engine.SharedGroups.find(t, ctx, B)
        assert saved(g) == saved(find(common, 1301))
        for a, b in zip(g.start[:-1], g.start[1:]):
            assert (g.prefix[a:b] == min(common[a:b - 1], default=0) * B).all()
    pair = engine.SharedGroups.find(t[[0, 0]], np.array([1301 * B, 1301 * B]), B)
    assert pair.prefix.tolist() == [1301 * B] * 2
