"""What the header says of assignments that cannot be refused, and of who may write where, by the 64-bit form."""
import numpy as np

from oracle import paged as ref


def test_as_many_free_pages_as_the_worst_case_are_enough_and_rows_end_in_pages_of_their_own():
    """Over random steps: with sum of ceil((L % page + grow) / page) pages free a call is carried out, and afterwards no
    slot's pages from the one in which its rows end on are another's."""
    rng = np.random.default_rng(7)
    B, P, page, N = 6, 7, 16, 22
    table, held, refs, lens = [[-1] * P] * B, [0] * B, [0] * N, [0] * B
    refused = 0
    for step in range(400):
        src = None if step % 4 == 0 else [int(x) for x in rng.integers(-1, B, B)]
        now = [lens[b] if src is None else (lens[src[b]] if src[b] >= 0 else 0) for b in range(B)]
        grow = [int(rng.integers(0, min(50, P * page - x) + 1)) for x in now]
        free, worst = refs.count(0), sum(-(-(x % page + g) // page) for x, g in zip(now, grow))
        got = ref.pages_assign(table, held, refs, lens, grow, src, page)
        if got is None:
            assert free < worst
            refused += 1
            grow, src = [0] * B, [-1 if rng.random() < 0.6 else b for b in range(B)]
            now = [0 if s < 0 else lens[b] for b, s in enumerate(src)]
            got = ref.pages_assign(table, held, refs, lens, grow, src, page)
            if got is None:                                # (their last pages are shared and no page is free)
                got = ref.pages_assign(table, held, refs, lens, [0] * B, [-1] * B, page)
                now = [0] * B
        table, held, refs, lens, _ = got
        for b in range(B):
            for t in range(lens[b] // page, held[b]):
                assert refs[table[b][t]] == 1
        # rows are committed; sometimes lengths are cut back
        lens = [min(held[b] * page, x + int(rng.integers(0, 40))) for b, x in enumerate(now)]
        if rng.random() < 0.3:
            lens = [int(rng.integers(0, x + 1)) for x in lens]
    assert refused > 5
