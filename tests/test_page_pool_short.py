"""The plain model of the page pool where pages run out, without a GPU."""
import random

from oracle import pool as OP


def test_whoever_the_pages_left_cover_is_served():
    m = OP.Pool(5, 5, 8)
    _, short = m.reserve([6 * 64, 64, 1, 65, 64])
    assert short == [0] and m.held == [[], [0], [1], [2, 3], [4]]


def test_who_sits_out_keeps_its_pages_and_is_marked():
    """Random demands on few pages: a sequence is marked exactly if the last call with demands by sequence gave it no
    slots, and what it holds covers its length and no more."""
    for seed in range(40):
        r = random.Random(seed)
        B, N, P = r.randint(1, 8), r.randint(2, 20), r.randint(1, 6)
        m = OP.Pool(B, N, P)
        for _ in range(30):
            n = [r.choice([0, 1, 5, 64, 130]) for _ in range(B)]
            before = [list(x) for x in m.held]
            _, short = m.reserve(n)
            fits = [x + k <= P * 64 for x, k in zip(m.len, n)]
            free = m.ref().count(0)
            for b in range(B):
                out = n[b] == 0 or b in short or not fits[b]
                last = m.table()[b][OP.pages_for(m.len[b]) - 1]
                assert (last <= -2 - OP.OUT) == (out and m.len[b] > 0), (seed, b)
                need = OP.pages_for(m.len[b] + n[b]) - OP.pages_for(m.len[b])
                assert b not in short or (need + 1 > free and m.held[b] == before[b][:OP.pages_for(m.len[b])])
                if not out:
                    m.len[b] += n[b]
            if r.random() < 0.3:
                m.free([r.randrange(B)])
            if r.random() < 0.3:
                m.fork([r.randrange(B)], [r.randrange(B)])
