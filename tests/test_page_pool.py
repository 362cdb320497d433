"""The device page pool without a GPU: the plain model pinned by the contents it
keeps, and the refusals of the entry points."""
import ctypes
import random

import pytest

from oracle import pool as OP


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decoding_verification_pass_gb300 import binding
    return binding


def test_model_keeps_every_sequence_its_own_rows():
    """Random calls, with rows written as a pass writes them: what a sequence reads is always what it wrote itself or
    what its source had written when it was forked."""
    for seed in range(30):
        r = random.Random(seed)
        B, N, P = r.randint(1, 6), r.randint(2, 30), r.randint(1, 8)
        m = OP.Pool(B, N, P)
        cells, text, stamp = {}, [[] for _ in range(B)], 0
        for _ in range(60):
            op = r.choice(["pass", "pass", "fork", "free", "back", "compact", "trim"])
            if op == "pass":
                n = [r.choice([0, 1, 5, 70]) for _ in range(B)]
                moves, short = m.reserve(n)
                new = dict(cells)
                for a, b, s in moves:
                    for t in range(s):
                        new[b, t] = cells[a, t]
                cells = new
                for b in range(B):
                    if b in short or m.len[b] + n[b] > P * 64:
                        continue
                    for t in range(m.len[b], m.len[b] + n[b]):
                        stamp += 1
                        cells[m.held[b][t // 64], t % 64] = stamp
                        text[b].append(stamp)
                    m.len[b] += n[b]
            elif op == "fork":
                a, b = r.randrange(B), r.randrange(B)
                if not m.fork([a], [b]):
                    text[b] = list(text[a])
            elif op == "free":
                b = r.randrange(B)
                m.free([b])
                text[b] = []
            elif op == "back":
                b = r.randrange(B)
                k = r.randint(0, m.len[b])
                if m.guard[b] and k % 64 == 0:
                    continue
                if OP.pages_for(k) == OP.pages_for(m.len[b]) or not m.guard[b]:
                    m.len[b], text[b] = k, text[b][:k]
            elif op == "compact":
                cells.update({(b, t): v for a, b in m.compact() for t in range(64)
                              for v in [cells.get((a, t))]})
            else:
                m.reserve(0)
            for b in range(B):
                assert [cells[m.held[b][t // 64], t % 64] for t in range(m.len[b])] == text[b], (seed, op, b)
            ref = m.ref()
            assert sum(ref) == sum(len(x) for x in m.held)


def test_refusals(lib):
    L = lib.lib()
    f = 4096
    cfg = ctypes.byref(lib.ModelConfig(2, 256, 4, 2, 256, 1000).c())
    ws = lib.spec_pages_workspace_bytes(2, 10, 4)
    assert ws > 256 and lib.spec_pages_workspace_bytes(-1, 10, 4) == 0 == lib.spec_pages_workspace_bytes(2, 0, 4)

    def pages(table=f, ln=f, mapped=f, ref=f, n_free=f, batch=2, n=10, per=4):
        return ctypes.byref(lib.spec_pages(table, ln, mapped, ref, n_free, batch, n, per))

    def data(k=f, v=f, ks=None, vs=None, n=10):
        return ctypes.byref(lib.spec_page_data(k, v, ks, vs, n))

    def reserve(c=cfg, p=pages(), d=data(), n=1, dn=None, w=f, wb=ws):
        return L.spec_pages_reserve(c, p, d, n, dn, w, wb, None)

    def fork(p=pages(), n=1, a=f, b=f, w=f, wb=ws):
        return L.spec_pages_fork(p, n, a, b, w, wb, None)

    def free(p=pages(), n=1, a=f, w=f, wb=ws):
        return L.spec_pages_free(p, n, a, w, wb, None)

    def compact(c=cfg, p=pages(), d=data(), w=f, wb=ws):
        return L.spec_pages_compact(c, p, d, w, wb, None)

    def copy(c=cfg, d=data(), t=data(), n=1, a=f, b=f, w=f):
        return L.spec_pages_copy(c, d, t, n, a, b, w, None)

    books = [dict(p=x) for x in (None, pages(table=None), pages(ln=None), pages(mapped=None), pages(ref=None),
                                 pages(n_free=None), pages(batch=-1), pages(n=0), pages(per=0), pages(table=4098),
                                 pages(ref=4097))]
    for g in (reserve, fork, free, compact):
        for bad in books + [dict(w=None), dict(w=4098)]:
            assert g(**bad) == lib.SPEC_EINVAL, bad
        assert g(wb=ws - 1) == lib.SPEC_ESIZE
        assert g(p=pages(batch=65536), wb=1 << 30) == lib.SPEC_ESIZE
        assert g(p=pages(per=16385), wb=1 << 30) == lib.SPEC_ESIZE
    for bad in books:
        assert L.spec_pages_init(bad["p"], None) == lib.SPEC_EINVAL
    datas = [dict(d=x) for x in (None, data(k=None), data(v=None), data(k=4104), data(ks=f), data(vs=f), data(n=0),
                                 data(ks=4098, vs=f))] + [dict(c=None)]
    for g in (reserve, compact, copy):
        for bad in datas:
            assert g(**bad) == lib.SPEC_EINVAL, bad
    for g in (reserve, compact):
        assert g(d=data(n=9)) == lib.SPEC_EINVAL  # another pool's data
    assert reserve(n=-1) == lib.SPEC_EINVAL == reserve(dn=4098)
    assert reserve(p=pages(batch=0)) == lib.SPEC_OK
    big = 1 << 26
    assert copy(d=data(n=big), n=1) == lib.SPEC_ESIZE
    for bad in (dict(n=-1), dict(a=None), dict(b=None), dict(a=4098), dict(b=4098)):
        assert fork(**bad) == lib.SPEC_EINVAL == copy(**bad), bad
    assert fork(n=0) == free(n=0) == copy(n=0) == lib.SPEC_OK
    assert fork(n=65536) == free(n=65536) == copy(n=11) == lib.SPEC_ESIZE
    assert free(a=None) == free(n=-1) == free(a=4098) == lib.SPEC_EINVAL
    assert copy(d=data(ks=f, vs=f)) == lib.SPEC_EINVAL == copy(w=None)  # 8-bit pages to a bf16 cache
