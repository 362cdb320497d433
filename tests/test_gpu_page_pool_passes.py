"""The device page pool around passes, on a GPU: passes right behind the calls
that write the tables, pools that run short in the middle of a round, and
sequences that sit one out.
"""
import numpy as np
import pytest
import torch

from oracle import pool as OP
from speculative_decoding_verification_pass_gb300 import binding as sb
from speculative_decoding_verification_pass_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

CFG = sb.ModelConfig(2, 256, 4, 2, 256, 1000)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _held(e):
    return e if e >= -1 else -2 - e if e > -2 - sb.PAGES_OUT else -2 - sb.PAGES_OUT - e


class Round:
    """A cache with its device pool, a model, and the passes on them."""

    def __init__(self, kv8, B, n_pages, max_pages, cfg=CFG, seed=3):
        self.cfg, self.kv8, self.B = cfg, kv8, B
        self.kv = (sb.KV8Cache if kv8 else sb.PagedKVCache)(cfg, B, n_pages, max_pages)
        self.pages = sb.Pages(self.kv)
        most = min(128, 512 // B)
        self.ws = sb.workspace(max(sb.spec_workspace_bytes(cfg, B, most - 1, max_pages * 64),
                                   sb.spec_kv8_workspace_bytes(cfg, B, most),
                                   sb.spec_pages_workspace_bytes(B, n_pages, max_pages)))
        self.model = sb.Model(cfg, seed)

    def reserve(self, n):
        sb.spec_pages_reserve(self.pages, n if isinstance(n, int) else _ints(n), self.ws)

    def forward(self, tokens):
        n = tokens.shape[1]
        z = torch.empty(self.B, n, self.cfg.vocab, device="cuda")
        if self.kv8:
            sb.spec_verify_forward_kv8(self.model.handle, tokens, self.B, n, self.kv, z, self.ws)
        else:
            sb.spec_verify_forward_paged(self.model.handle, tokens, self.B, n - 1, self.kv, z, self.ws)
        return z

    def truncate(self, accepted, gamma):
        f = sb.spec_kv8_truncate if self.kv8 else sb.spec_paged_kv_truncate
        f(self.kv, _ints(accepted), gamma, self.ws)

    def status(self):
        return sb.spec_device_status(self.ws)[1]

    def bytes_of(self, b, slots):
        """What sequence b's first `slots` slots hold, k and v (and the scales of their blocks)."""
        row = [_held(e) for e in self.kv.table[b].tolist()]
        page = torch.tensor([row[t // 64] for t in range(slots)], dtype=torch.long, device="cuda")
        at = torch.arange(slots, device="cuda") % 64
        out = [t.view(torch.uint8)[:, page, :, at].cpu() for t in (self.kv.k, self.kv.v)]
        if self.kv8:
            blocks = torch.arange(0, slots, 16, device="cuda")
            out += [t[:, page[blocks], :, at[blocks] // 16].cpu() for t in (self.kv.k_scale, self.kv.v_scale)]
        return out

    def close(self):
        self.model.close()


def _tokens(seed, B, n, cfg=CFG):
    return _ints(wl.tokens(seed, B, n, cfg.vocab).tolist())


@pytest.mark.parametrize("schedule", ["persistent", "per_step"])
@pytest.mark.parametrize("kv8", [False, True])
def test_a_pass_right_behind_a_compaction(kv8, schedule, monkeypatch):
    """Pages reserved, moved, and read by the pass that is launched next: the logits of a pool that moves none."""
    if schedule == "per_step":
        monkeypatch.setenv("SPEC_FORWARD_PERSISTENT", "0")
    B, P = 24, 6
    runs = []
    for compact in (False, True):
        r = Round(kv8, B, 2 * B * P, P)
        log = []
        for i in range(4):
            n = (70, 9, 5, 21)[i]
            r.reserve(n)
            if compact:
                sb.spec_pages_compact(r.pages, r.ws)
            for c in range(0, n, 21):
                log.append(r.forward(_tokens(10 * i + c, B, min(21, n - c))))
            gone = _ints([b for b in range(B) if (b + i) % 3 == 0])
            sb.spec_pages_free(r.pages, gone, r.ws)
            sb.spec_pages_fork(r.pages, (gone + 1) % B, gone, r.ws)
        assert r.status() == 0
        runs.append(log + [r.kv.len.clone()])
        r.close()
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def _same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("schedule", ["persistent", "per_step"])
@pytest.mark.parametrize("kv8", [False, True])
def test_a_short_pool_loses_no_tokens(kv8, schedule, monkeypatch):
    """Reserve, pass and rollback with pages for one of three: the others keep lengths and rows, and their next pass is
    that of a pool that never ran short."""
    if schedule == "per_step":
        monkeypatch.setenv("SPEC_FORWARD_PERSISTENT", "0")
    prompt, first, second = _tokens(1, 3, 60), _tokens(2, 3, 5), _tokens(3, 3, 5)
    last = []
    for pages in (4, 12):
        r = Round(kv8, 3, pages, 4)
        r.reserve(60)
        r.forward(prompt)
        if pages == 4:
            held = [r.bytes_of(b, 60) for b in (1, 2)]
            r.reserve(5)
            assert r.status() == sb.DEV_NO_PAGES and r.pages.waiting().tolist() == [False, True, True]
            r.forward(first)
            assert r.status() == sb.DEV_BAD_PAGE
            r.truncate([2, 1, 0], 4)
            assert r.status() == sb.DEV_BAD_PAGE and r.kv.len.tolist() == [63, 60, 60]
            if kv8:  # the same of a tree's commit: the root and three accepted nodes
                sb.spec_kv8_tree_commit(CFG, r.kv, _ints([[1, 2, 4, -1, -1]] * 3), _ints([0, 3, 3]), 5, r.ws)
                assert r.status() == sb.DEV_BAD_PAGE and r.kv.len.tolist() == [59, 60, 60]
            r.reserve(0)  # pages returned alone: it changes nothing for those that wait
            assert r.status() == 0 and r.pages.waiting().tolist() == [False, True, True]
            assert all(_same(x, r.bytes_of(b, 60)) for x, b in zip(held, (1, 2)))
        sb.spec_pages_free(r.pages, _ints([0]), r.ws)
        r.reserve([0, 5, 5])
        assert r.status() == 0 and r.pages.waiting().tolist() == [True, False, False]
        z = r.forward(second)
        assert r.kv.len.tolist() == [0, 65, 65]
        last.append(z[1:].clone())
        r.close()
    assert torch.equal(*last)


@pytest.mark.parametrize("kv8", [False, True])
def test_sequences_without_slots_sit_the_pass_out(kv8):
    """No slots asked for, with room in the last page and without, a last page that is full, one that a longer sequence
    holds too after a rollback, and a sequence at its capacity: nothing is written for them, nothing dropped."""
    r = Round(kv8, 6, 40, 3)
    lens = [70, 10, 61, 128, 70, 190]
    r.reserve(lens)
    r.kv.k.view(torch.uint8).random_(0, 120)
    r.kv.v.view(torch.uint8).random_(0, 120)
    r.kv.len.copy_(_ints(lens))
    sb.spec_pages_fork(r.pages, _ints([0]), _ints([4]), r.ws)
    r.kv.len[4] = 60
    held = [r.bytes_of(b, x) for b, x in enumerate([0, 10, 61, 128, 60, 190])]
    r.reserve([5, 0, 0, 0, 0, 5])
    assert r.status() == sb.DEV_KV_OVERFLOW and r.pages.waiting().tolist() == [False] + [True] * 5
    r.forward(_tokens(4, 6, 5))
    assert r.status() & ~sb.DEV_KV_OVERFLOW == sb.DEV_BAD_PAGE
    r.truncate([1, 0, 0, 0, 0, 0], 4)
    assert r.status() == sb.DEV_BAD_PAGE
    assert r.kv.len.tolist() == [72, 10, 61, 128, 60, 190]
    r.reserve([0, 5, 5, 5, 5, 2])  # a copy of what sequence 4 shares, and pages of their own for the others
    assert r.status() == 0 and r.pages.waiting().tolist() == [True] + [False] * 5
    for b, x in enumerate([0, 10, 61, 128, 60, 190]):
        assert b == 0 or _same(held[b], r.bytes_of(b, x)), b
    r.forward(_tokens(5, 6, 2))
    assert r.status() == sb.DEV_BAD_PAGE and r.kv.len.tolist() == [72, 12, 63, 130, 62, 192]
    r.close()


@pytest.mark.parametrize("kv8", [False, True])
def test_forks_and_compaction_keep_who_sits_out(kv8):
    r = Round(kv8, 4, 6, 3)
    r.reserve([64, 0, 60, 100])
    r.kv.len.copy_(_ints([64, 0, 60, 100]))
    sb.spec_pages_free(r.pages, _ints([2]), r.ws)
    r.reserve([65, 0, 0, 5])
    r.reserve([0, 0, 0, 0])
    assert r.status() == 0 and r.pages.waiting().all()
    sb.spec_pages_fork(r.pages, _ints([0, 3]), _ints([1, 2]), r.ws)
    out = [[-2 - sb.PAGES_OUT - 0, -1, -1]] * 2
    assert r.kv.table.tolist() == out + [[2, -2 - sb.PAGES_OUT - 3, -1]] * 2
    sb.spec_pages_compact(r.pages, r.ws)
    t = r.kv.table.tolist()
    assert t[:2] == out and t[2] == t[3] == [2, -2 - sb.PAGES_OUT - 1, -1] and r.status() == 0
    r.truncate([0, 0, 0, 0], 4)
    assert r.status() == sb.DEV_BAD_PAGE and r.kv.len.tolist() == [64, 64, 100, 100]
    r.reserve(1)  # both of a pair write: a page each past a full one, the first keeps the other, the last copies
    assert r.status() == 0 and r.pages.waiting().tolist() == [False] * 4
    assert r.kv.table.tolist() == [[0, 3, -1], [0, 4, -1], [2, 1, -1], [2, 5, -1]]
    r.close()


@pytest.mark.parametrize("kv8", [False, True])
def test_a_fork_can_still_be_rolled_back(kv8):
    """The mark of a shared page forbids writes alone."""
    r = Round(kv8, 2, 6, 3)
    r.reserve([75, 0])
    r.kv.len.copy_(_ints([75, 0]))
    sb.spec_pages_fork(r.pages, _ints([0]), _ints([1]), r.ws)
    r.truncate([1, 3], 4)
    assert r.status() == 0 and r.kv.len.tolist() == [72, 74]
    r.close()


def test_pools_of_more_pages_than_marks_tell_apart_are_refused():
    kv = sb.PagedKVCache(CFG, 1, 1, 1)
    p = sb.Pages(kv).c()
    p.n_pages = sb.PAGES_OUT // 2
    with pytest.raises(sb.SpecError):
        sb._check(sb.lib().spec_pages_fork(p, 0, None, None, sb.workspace(256).data_ptr(), 1 << 40, None), "fork")


def test_a_demand_that_is_not_met_leaves_the_pages_to_the_others():
    r = Round(False, 5, 5, 8)
    r.reserve([6 * 64, 64, 1, 65, 64])
    assert r.status() == sb.DEV_NO_PAGES and r.pages.waiting().tolist() == [True] + [False] * 4
    assert [x[:3] for x in r.kv.table.tolist()] == [[-1, -1, -1], [0, -1, -1], [1, -1, -1], [2, 3, -1], [4, -1, -1]]
    assert r.pages.mapped.tolist() == [0, 1, 1, 2, 1] and r.pages.n_free.item() == 0
    r.close()


@pytest.mark.parametrize("B,N,P", [(40, 60, 9), (300, 170, 6), (2100, 3000, 5)])
def test_short_pools_against_the_model(B, N, P):
    """Demands of all sizes on too few pages, copies among them, more sequences than threads."""
    g = wl.rng(B, 50)
    kv = sb.PagedKVCache(sb.ModelConfig(1, 128, 2, 1, 128, 100), B, N, P)
    pages, ws = sb.Pages(kv), sb.workspace(sb.spec_pages_workspace_bytes(B, N, P))
    m = OP.Pool(B, N, P)
    served = refused = 0
    for i in range(12):
        n = [int(x) for x in g.choice([0, 1, 5, 63, 64, 65, 130, 200], size=B)]
        sb.spec_pages_reserve(pages, _ints(n), ws)
        _, short = m.reserve(n)
        over = any(x + k > P * 64 for x, k in zip(m.len, n))
        want = (sb.DEV_NO_PAGES if short else 0) | (sb.DEV_KV_OVERFLOW if over else 0)
        assert sb.spec_device_status(ws)[1] == want
        m.len = [x + k if b not in short and x + k <= P * 64 else x for b, (x, k) in enumerate(zip(m.len, n))]
        served, refused = served + B - len(short), refused + len(short)
        kv.len.copy_(_ints(m.len))
        gone = [int(b) for b in g.permutation(B)[:B // 3]]
        left = [b for b in range(B) if b not in gone]
        src = [int(g.choice(left)) for _ in gone[::2]]
        sb.spec_pages_free(pages, _ints(gone), ws)
        sb.spec_pages_fork(pages, _ints(src), _ints(gone[::2]), ws)
        m.free(gone)
        assert m.fork(src, gone[::2]) == []
        assert kv.table.tolist() == m.table() and kv.len.tolist() == m.len
        assert pages.ref.tolist() == m.ref() and pages.n_free.item() == m.ref().count(0)
    assert served > B and refused > B


def _shared_and_short(kv8, slots):
    """A prompt in two sequences that share a partly filled page, a third that fills the pool, and a reservation that has
    no page for the second's copy."""
    full = -(-slots // 64)
    r = Round(kv8, 3, full + 1, 4)
    r.reserve([slots, 0, 64])
    r.forward(_tokens(6, 3, slots))  # (sequences 1 and 2 have no room for it)
    r.status()
    assert r.kv.len.tolist() == [slots, 0, 0]
    sb.spec_pages_fork(r.pages, _ints([0]), _ints([1]), r.ws)
    r.kv.len[2] = 59
    r.reserve(5)
    assert r.status() == sb.DEV_NO_PAGES
    return r


def _layer(r, scale, n=5):
    """Rows of one layer put in by hand: their queries' output is of no account."""
    d, kvd = CFG.d_model, CFG.d_model // CFG.n_heads * CFG.n_kv_heads
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (scale * torch.randn(3 * n, w, device="cuda", generator=g) for w in (d, kvd, kvd))
    q_out = torch.empty(3 * n, d, dtype=torch.bfloat16, device="cuda")
    rope = sb.RopeTable(CFG.head_dim, CFG.rope_theta)
    for layer in range(CFG.n_layers):
        sb.spec_kv8_append(CFG, r.kv, layer, n, q, k, v, rope, q_out, r.ws)


@pytest.mark.parametrize("by_hand", [False, True])
@pytest.mark.parametrize("slots", [100, 70, 79])
def test_8_bit_rows_of_a_waiting_sequence_are_not_rounded_again(slots, by_hand):
    """The first of two forks keeps the page they share; the other waits for a copy.  Larger values behind its rows
    would change their block's scale: neither a pass nor appends by hand touch them, and the first waits too."""
    r = _shared_and_short(True, slots)
    assert r.pages.waiting().tolist() == [True, True, False]
    before = r.bytes_of(1, slots)
    if by_hand:
        _layer(r, 1e-3)  # (values that need no larger scale change nothing)
        assert r.status() == sb.DEV_BAD_PAGE and r.kv.table[0].min() == -1
        assert _same(before, r.bytes_of(1, slots))
        _layer(r, 1e6)
        sb.spec_kv8_advance(r.kv, 1, r.ws)
    else:
        r.forward(_tokens(7, 3, 5))
    assert r.status() == sb.DEV_BAD_PAGE
    lens = [slots, slots, 60 if by_hand else 64]
    assert r.kv.len.tolist() == lens and r.pages.waiting().tolist() == [True, True, False]
    r.truncate([0, 0, 4], 4)
    assert r.status() == sb.DEV_BAD_PAGE and r.kv.len.tolist() == lens
    sb.spec_kv8_tree_commit(CFG, r.kv, _ints([[1, 3, -1, -1, -1]] * 3), _ints([2, 2, 0]), 5, r.ws)
    assert r.status() == sb.DEV_BAD_PAGE and r.kv.len.tolist() == [slots, slots, lens[2] - 4]
    assert _same(before, r.bytes_of(1, slots)) and _same(before, r.bytes_of(0, slots))
    r.reserve([5, 5, 0])  # as short as before: tried again, the first keeps the page
    assert r.status() == sb.DEV_NO_PAGES and r.kv.table[0].min() == -1
    r.forward(_tokens(7, 3, 5))
    assert r.status() == sb.DEV_BAD_PAGE and r.kv.len.tolist()[:2] == [slots, slots]
    assert _same(before, r.bytes_of(1, slots)) and _same(before, r.bytes_of(0, slots))
    # pages for both
    sb.spec_pages_free(r.pages, _ints([2]), r.ws)
    r.reserve([5, 5, 0])
    assert r.status() == 0 and r.pages.waiting().tolist() == [False, False, True]
    assert _same(before, r.bytes_of(0, slots)) and _same(before, r.bytes_of(1, slots))
    z = r.forward(_tokens(8, 3, 5))
    assert r.kv.len.tolist() == [slots + 5, slots + 5, 0]
    # the same in a pool that was never short
    a = Round(True, 3, 12, 4)
    a.reserve([slots, slots, 0])
    a.forward(_ints([_tokens(6, 3, slots)[0].tolist()] * 3))
    a.reserve([5, 5, 0])
    assert torch.equal(a.forward(_tokens(8, 3, 5))[:2], z[:2])
    r.close()
    a.close()


@pytest.mark.parametrize("kv8,slots", [(True, 96), (True, 80), (False, 100), (False, 79)])
def test_rows_of_a_waiting_sequence_in_blocks_of_their_own(kv8, slots):
    """Where no scale is shared (a new block, or bf16) the keeper of the page goes on."""
    r = _shared_and_short(kv8, slots)
    assert r.pages.waiting().tolist() == [False, True, False]
    before = r.bytes_of(1, slots)
    for accepted in (3, 1):
        r.forward(_tokens(9, 3, 5))
        assert r.status() == sb.DEV_BAD_PAGE
        r.truncate([accepted, 0, 0], 4)
        assert r.status() == sb.DEV_BAD_PAGE
        r.reserve([5, 5, 0])
        assert r.status() == sb.DEV_NO_PAGES
        assert _same(before, r.bytes_of(1, slots))
    assert r.kv.len.tolist()[:2] == [slots + 6, slots]
    r.close()
