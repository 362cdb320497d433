"""The device page pool on a GPU against its plain model: tables, counts and
what every sequence reads, through random calls; and rounds of parallel
continuations on shared pages against the same rounds without sharing.
"""
import random

import numpy as np
import pytest
import torch

from oracle import pool as OP
from speculative_decoding_verification_pass_gb300 import binding as sb
from speculative_decoding_verification_pass_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

CFGS = [sb.ModelConfig(2, 256, 4, 2, 256, 1000),        # hd 64
        sb.ModelConfig(3, 512, 4, 1, 384, 1003)]        # hd 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(cfg, kv8, B, n_pages, max_pages):
    return (sb.KV8Cache if kv8 else sb.PagedKVCache)(cfg, B, n_pages, max_pages)


class Twin:
    """A pool on the device and its model; every row of every layer, head, k and v holds a stamp of its own."""

    def __init__(self, cfg, kv8, B, n_pages, max_pages):
        self.kv = _cache(cfg, kv8, B, n_pages, max_pages)
        self.kv8, self.n_pages = kv8, n_pages
        self.kv.table.fill_(7)
        self.kv.len.fill_(9)
        self.pages = sb.Pages(self.kv)
        self.ws = sb.workspace(sb.spec_pages_workspace_bytes(B, n_pages, max_pages))
        self.m = OP.Pool(B, n_pages, max_pages)
        g = torch.Generator(device="cuda").manual_seed(1)
        for t in self._data():  # anything
            raw = t.view(torch.uint8)
            raw.copy_(torch.randint(0, 256, raw.shape, dtype=torch.uint8, device="cuda", generator=g))
        self.want = [t.view(torch.uint8).cpu().clone() for t in self._data()]

    def _data(self):
        kv = self.kv
        return [kv.k, kv.v] + ([kv.k_scale, kv.v_scale] if self.kv8 else [])

    def move(self, moves):
        for t in self.want:
            new = t.clone()
            for a, b, slots in moves:
                if t.dim() == 5:
                    new[:, b, :, :slots] = t[:, a, :, :slots]
                else:
                    new[:, b] = t[:, a]
            t.copy_(new)

    def status(self):
        return sb.spec_device_status(self.ws)[1]

    def reserve(self, n):
        sb.spec_pages_reserve(self.pages, n if isinstance(n, int) else _ints(n), self.ws)
        moves, short = self.m.reserve(n)
        self.move(moves)
        over = [b for b in range(self.m.batch)
                if self.m.len[b] + (n if isinstance(n, int) else n[b]) > self.m.max_pages * 64]
        assert self.status() == (sb.DEV_NO_PAGES if short else 0) | (sb.DEV_KV_OVERFLOW if over else 0)
        return short

    def fork(self, src, dst):
        sb.spec_pages_fork(self.pages, _ints(src), _ints(dst), self.ws)
        bad = self.m.fork(src, dst)
        assert self.status() == (sb.DEV_BAD_SEQ if bad else 0)

    def free(self, seqs):
        sb.spec_pages_free(self.pages, _ints(seqs), self.ws)
        self.m.free(seqs)
        assert self.status() == (sb.DEV_BAD_SEQ if any(not 0 <= b < self.m.batch for b in seqs) else 0)

    def compact(self):
        sb.spec_pages_compact(self.pages, self.ws)
        self.move([(a, b, 64) for a, b in self.m.compact()])
        assert self.status() == 0

    def set_len(self, lens):
        self.m.len = list(lens)
        self.kv.len.copy_(_ints(lens))

    def check(self, data=True):
        ref = self.m.ref()
        assert self.kv.table.tolist() == self.m.table()
        assert self.kv.len.tolist() == self.m.len
        assert self.pages.mapped.tolist() == [len(x) for x in self.m.held]
        assert self.pages.ref.tolist() == ref
        assert self.pages.n_free.item() == ref.count(0)
        if data:
            for t, w in zip(self._data(), self.want):
                assert torch.equal(t.view(torch.uint8).cpu(), w)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("ci", [0, 1])
@pytest.mark.parametrize("seed", range(4))
def test_random_calls(kv8, ci, seed):
    r = random.Random(seed * 4 + ci * 2 + kv8)
    B, N, P = r.choice([(1, 5, 3), (3, 9, 4), (6, 40, 8), (40, 130, 5)])
    t = Twin(CFGS[ci], kv8, B, N, P)
    t.check()
    for i in range(40):
        op = r.choice(["pass", "pass", "pass", "fork", "fork", "free", "back", "compact", "trim"])
        if op == "pass":
            n = r.choice([1, 5, 64, [r.choice([0, 1, 5, 63, 64, 65, 200]) for _ in range(B)]])
            short = t.reserve(n)
            n = [n] * B if isinstance(n, int) else n
            t.set_len([L + k if b not in short and L + k <= P * 64 else L
                       for b, (L, k) in enumerate(zip(t.m.len, n))])
        elif op == "fork":
            k = r.randint(1, max(1, B // 2))
            t.fork([r.randint(-1, B) if r.random() < 0.1 else r.randrange(B) for _ in range(k)],
                   [r.randrange(B) for _ in range(k)])
        elif op == "free":
            t.free([r.randrange(B) for _ in range(r.randint(1, 3))] + ([B] if r.random() < 0.1 else []))
        elif op == "back":  # a rollback that leaves a marked page the last one
            t.set_len([L if t.m.guard[b] else r.randint(max(0, L - 70), L) for b, L in enumerate(t.m.len)])
        elif op == "compact":
            t.compact()
        else:
            t.reserve(0)
        t.check(data=i % 4 == 3)
    t.check()


def test_many_sequences_and_pages():
    """More sequences and pages than threads; long tables."""
    cfg = sb.ModelConfig(1, 128, 2, 1, 128, 100)
    B, N, P = 2500, 9001, 300
    t = Twin(cfg, True, B, N, P)
    r = random.Random(3)
    lens = [0] * B
    lens[7], lens[2400] = 300 * 64 - 3, 111 * 64
    t.set_len(lens)
    t.m.len = [0] * B
    t.kv.len.copy_(_ints([0] * B))
    t.reserve([r.choice([0, 1, 100]) if b not in (7, 2400) else lens[b] for b in range(B)])
    t.set_len([min(len(t.m.held[b]) * 64, lens[b] or r.randint(0, len(t.m.held[b]) * 64)) for b in range(B)])
    t.fork([7] * 5 + [2400] * 20, list(range(100, 105)) + list(range(1500, 1520)))
    t.check()
    t.reserve(2)
    t.check()
    t.free(list(range(0, B, 2)))
    t.compact()
    t.check()


def test_short_pool_serves_in_order_and_guards_the_rest():
    cfg = CFGS[0]
    t = Twin(cfg, True, 4, 4, 4)
    assert t.reserve([100, 0, 0, 0]) == []
    t.set_len([100, 0, 0, 0])
    t.fork([0, 0], [1, 2])
    # two copies are needed and a page each for the third and fourth: two pages are there
    assert t.reserve([5, 5, 5, 5]) == [3]
    t.check()
    t.fork([0], [3])
    assert t.reserve([5, 0, 0, 5]) == [3]  # the first takes none from the pool? it keeps the page it shares last
    t.check()


def test_guarded_pages_refuse_a_pass():
    """A forked sequence that was not reserved for is refused by the passes, and what it shares stays."""
    cfg = CFGS[0]
    for kv8 in (False, True):
        B = 2
        kv = _cache(cfg, kv8, B, 8, 3)
        pages = sb.Pages(kv)
        ws = sb.workspace(max(sb.spec_workspace_bytes(cfg, B, 4, 192), sb.spec_kv8_workspace_bytes(cfg, B, 5),
                              sb.spec_pages_workspace_bytes(B, 8, 3)))
        m = sb.Model(cfg, 3)
        tok = _ints(wl.tokens(1, B, 5, cfg.vocab).tolist())
        z = torch.empty(B, 5, cfg.vocab, device="cuda")
        sb.spec_pages_reserve(pages, _ints([5, 0]), ws)
        kv.len.copy_(_ints([5, 0]))
        sb.spec_pages_fork(pages, _ints([0]), _ints([1]), ws)
        before = kv.k.view(torch.uint8).clone()
        if kv8:
            sb.spec_verify_forward_kv8(m.handle, tok, B, 5, kv, z, ws)
        else:
            sb.spec_verify_forward_paged(m.handle, tok, B, 4, kv, z, ws)
        assert sb.spec_device_status(ws)[1] & sb.DEV_BAD_PAGE
        assert torch.equal(kv.k.view(torch.uint8), before) and kv.len.tolist() == [5, 5]
        m.close()


def test_books_that_do_not_fit_are_left_alone():
    """Lengths, counts and ids that no call of the pool makes: flagged, nothing outside the arrays touched."""
    cfg = CFGS[0]
    B, N, P = 4, 14, 3
    cases = [("len", 0, -1, sb.DEV_KV_OVERFLOW), ("len", 1, 2 ** 31 - 1, sb.DEV_KV_OVERFLOW),
             ("len", 0, 64 * 3, sb.DEV_KV_OVERFLOW), ("mapped", 1, -5, sb.DEV_BAD_PAGE),
             ("mapped", 2, 2 ** 30, sb.DEV_BAD_PAGE), ("mapped", 0, 0, sb.DEV_BAD_PAGE)]
    for name, b, v, bit in cases:
        kv = _cache(cfg, False, B, N, P)
        pages = sb.Pages(kv)
        ws = sb.workspace(sb.spec_pages_workspace_bytes(B, N, P))
        sb.spec_pages_reserve(pages, 70, ws)
        kv.len.fill_(70)
        assert sb.spec_device_status(ws)[1] == 0
        (kv.len if name == "len" else pages.mapped)[b] = v
        row = kv.table[b].clone()
        sb.spec_pages_reserve(pages, 1, ws)
        assert sb.spec_device_status(ws)[1] == bit, (name, v)
        assert torch.equal(kv.table[b], row)
        sb.spec_pages_fork(pages, _ints([b]), _ints([3]), ws)
        assert sb.spec_device_status(ws)[1] == sb.DEV_BAD_PAGE, (name, v)
    for e in (-1, N, 2 ** 31 - 1, -2 - N, -2 ** 31):
        kv = _cache(cfg, False, B, N, P)
        pages = sb.Pages(kv)
        sb.spec_pages_reserve(pages, 70, ws)
        kv.len.fill_(70)
        kv.table[1, 1] = e
        sb.spec_pages_reserve(pages, 64, ws)
        assert sb.spec_device_status(ws)[1] == sb.DEV_BAD_PAGE
        for a, b in ((1, 2), (0, 1)):
            sb.spec_pages_fork(pages, _ints([a]), _ints([b]), ws)
            assert sb.spec_device_status(ws)[1] == sb.DEV_BAD_PAGE
        sb.spec_pages_free(pages, _ints([1]), ws)
        assert sb.spec_device_status(ws)[1] == sb.DEV_BAD_PAGE
        sb.spec_pages_compact(pages, ws)
        sb.spec_device_status(ws)


@pytest.mark.parametrize("kv8", [False, True])
def test_copy_between_pools(kv8):
    cfg = CFGS[1]
    a, b = _cache(cfg, kv8, 1, 9, 1), _cache(cfg, kv8, 2, 6, 1)
    ws = sb.workspace(256)
    bufs = lambda kv: [kv.k, kv.v] + ([kv.k_scale, kv.v_scale] if kv8 else [])
    for kv in (a, b):
        for t in bufs(kv):
            raw = t.view(torch.uint8)
            raw.copy_(torch.randint(0, 256, raw.shape, dtype=torch.uint8, device="cuda"))
    want = [t.view(torch.uint8).clone() for t in bufs(b)]
    for w, t in zip(want, bufs(a)):
        w[:, [4, 0, 5]] = t.view(torch.uint8)[:, [8, 2, 2]]
    sb.spec_pages_copy(a, b, _ints([8, 2, 2]), _ints([4, 0, 5]), ws)
    assert sb.spec_device_status(ws)[1] == 0
    assert all(torch.equal(t.view(torch.uint8), w) for t, w in zip(bufs(b), want))
    sb.spec_pages_copy(a, b, _ints([9, 1, -1]), _ints([1, 6, 2]), ws)  # none within both
    assert sb.spec_device_status(ws)[1] == sb.DEV_BAD_PAGE
    assert all(torch.equal(t.view(torch.uint8), w) for t, w in zip(bufs(b), want))
    # within one cache
    want = [t.view(torch.uint8).clone() for t in bufs(a)]
    for w in want:
        w[:, [0, 1]] = w[:, [7, 3]]
    sb.spec_pages_copy(a, a, _ints([7, 3]), _ints([0, 1]), ws)
    assert all(torch.equal(t.view(torch.uint8), w) for t, w in zip(bufs(a), want))
    with pytest.raises(ValueError):
        sb.spec_pages_copy(a, _cache(CFGS[0], kv8, 1, 9, 1), _ints([0]), _ints([1]), ws)
    with pytest.raises(ValueError):
        sb.spec_pages_copy(a, _cache(cfg, not kv8, 1, 9, 1), _ints([0]), _ints([1]), ws)


def test_offsets_past_32_bits():
    """Pools of more than 2^32 bytes: the last pages of the last layer."""
    cfg = sb.ModelConfig(8, 2048, 16, 16, 128, 100)  # a page: 256 KB a layer, k
    N = 2200
    kv = sb.PagedKVCache(cfg, 1, N, 1)
    assert kv.k.numel() * 2 > 2 ** 32
    kv.k[:, N - 1] = 3.0
    kv.v[:, N - 1] = -2.0
    sb.spec_pages_copy(kv, kv, _ints([N - 1]), _ints([N - 2]), sb.workspace(256))
    assert (kv.k[:, N - 2] == 3.0).all() and (kv.v[:, N - 2] == -2.0).all() and (kv.k[:, N - 3] == 0).all()


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("ci", [0, 1])
def test_rounds_of_parallel_continuations(kv8, ci):
    """A prompt forked into four, each drawing its own tokens, verified, filtered, accepted and rolled back for some
    rounds; then the losers freed, a winner forked, the pool compacted, and on.  The same rounds on a cache whose
    sequences share nothing give the same logits and tokens bit for bit."""
    cfg = CFGS[ci]
    B, n, P, seed = 4, 5, 4, 5 + ci
    N = B * P + 2
    V = cfg.vocab
    model = sb.Model(cfg, seed)
    s = sb.Sampling(0.9, 40, 0.95, 0.01)
    ws = sb.workspace(max(sb.spec_workspace_bytes(cfg, B, 127, P * 64), sb.spec_kv8_workspace_bytes(cfg, B, 128),
                          sb.spec_pages_workspace_bytes(B, N, P), sb.spec_accept_workspace_bytes(B, n, V)))
    prompt = wl.tokens(seed, 1, 100, V)

    def rounds(share):
        kv = _cache(cfg, kv8, B, N, P)
        log = []
        pages = sb.Pages(kv)

        def forward(tok):
            k = tok.shape[1]
            z = torch.empty(B, k, V, device="cuda")
            if kv8:
                sb.spec_verify_forward_kv8(model.handle, tok, B, k, kv, z, ws)
            else:
                sb.spec_verify_forward_paged(model.handle, tok, B, k - 1, kv, z, ws)
            return z

        def spread(src, dst):
            if share:
                sb.spec_pages_free(pages, _ints(dst), ws)
                sb.spec_pages_fork(pages, _ints(src), _ints(dst), ws)
                return
            rows = kv.table.clone()  # pages of its own, copied whole
            for a, b in zip(src, dst):
                m = int(pages.mapped[a])
                sb.spec_pages_copy(kv, kv, rows[a, :m].contiguous(), rows[b, :m].contiguous(), ws)
                kv.len[b] = kv.len[a]

        if share:  # the prompt in one sequence; the others hold nothing and repeat it into pages given back
            sb.spec_pages_reserve(pages, 100, ws)
            tok = _ints(np.repeat(prompt, B, 0).tolist())
            z = forward(tok)
            sb.spec_pages_free(pages, _ints([1, 2, 3]), ws)
            sb.spec_pages_fork(pages, _ints([0, 0, 0]), _ints([1, 2, 3]), ws)
        else:
            sb.spec_pages_reserve(pages, P * 64, ws)
            z = forward(_ints(np.repeat(prompt, B, 0).tolist()))
        last = torch.empty(1, B, dtype=torch.int32, device="cuda")  # four draws of one row
        sb.spec_sample(z[0, -1:].contiguous(), s, torch.from_numpy(wl.uniforms(seed, 1, B)).cuda(), last, ws)
        last = last.view(B, 1)
        for r in range(6):
            if share:
                sb.spec_pages_reserve(pages, n, ws)
            q = torch.empty(B * (n - 1), V, device="cuda")
            x = torch.empty(B * (n - 1), 1, dtype=torch.int32, device="cuda")
            g = torch.Generator(device="cuda").manual_seed(r)
            noise = torch.randn(B * (n - 1), V, device="cuda", generator=g) * 0.3
            base = z.view(-1, V)[-1:].clone()
            base[base == -float("inf")] = -20.0
            sb.spec_sample(base + noise, s, torch.from_numpy(wl.uniforms(seed + r, B * (n - 1), 1)).cuda(), x, ws,
                           probs=q)
            z = forward(torch.cat([last, x.view(B, n - 1)], 1).contiguous())
            log.append(z.clone())
            flat = z.view(B * n, V)
            sb.spec_filter_logits(flat, s, flat, ws)
            out = torch.empty(B, n, dtype=torch.int32, device="cuda")
            acc = torch.empty(B, dtype=torch.int32, device="cuda")
            sb.spec_accept(flat, q, x, torch.from_numpy(wl.uniforms(90 + r, B, n)).cuda(), B, n - 1, V, 0.9, 1.0, out,
                           acc, ws)
            (sb.spec_kv8_truncate if kv8 else sb.spec_paged_kv_truncate)(kv, acc, n - 1, ws)
            last = out.gather(1, acc.long().view(B, 1))
            log += [out, acc, kv.len.clone()]
            if r == 2:
                spread([2, 2], [0, 3])
                last = last[[2, 1, 2, 2]].contiguous()
            if r == 3 and share:
                sb.spec_pages_reserve(pages, 0, ws)
                sb.spec_pages_compact(pages, ws)
                used = N - pages.n_free.item()
                assert (pages.ref[:used] > 0).all() and (pages.ref[used:] == 0).all()
        assert sb.spec_device_status(ws)[1] == 0
        if share:
            assert (N - pages.n_free.item()) < sum(-(-int(x) // 64) for x in kv.len)  # the prompt's first page once
        return log

    for a, b in zip(rounds(True), rounds(False)):
        assert torch.equal(a, b)
    model.close()


def test_captured_round():
    """reserve, fork and free captured and replayed from other books."""
    cfg = CFGS[0]
    t = Twin(cfg, True, 4, 12, 4)
    t.reserve([130, 0, 10, 0])
    t.set_len([130, 0, 10, 0])
    free, src, dst = _ints([1, 3]), _ints([0, 2]), _ints([1, 3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sb.spec_pages_free(t.pages, free, t.ws)
        sb.spec_pages_fork(t.pages, src, dst, t.ws)
        sb.spec_pages_reserve(t.pages, 5, t.ws)
        sb.spec_pages_compact(t.pages, t.ws)
    for a, b in (([0, 2], [1, 3]), ([3, 1], [0, 2]), ([0, 2], [3, 1])):
        src.copy_(_ints(a))
        dst.copy_(_ints(b))
        free.copy_(_ints(b))
        g.replay()
        t.m.free(b)
        t.m.fork(a, b)
        t.move(t.m.reserve(5)[0])
        t.move([(x, y, 64) for x, y in t.m.compact()])
        torch.cuda.synchronize()
        t.check()
        assert t.status() == 0
        t.set_len([x + 5 for x in t.m.len])


def test_python_checks():
    cfg = CFGS[0]
    kv = _cache(cfg, False, 2, 4, 2)
    pages, ws = sb.Pages(kv), sb.workspace(sb.spec_pages_workspace_bytes(2, 4, 2))
    for f in (lambda: sb.Pages(kv, mapped=_ints([0, 0])),
              lambda: sb.Pages(kv, mapped=_ints([0, 0]), ref=_ints([0] * 3), n_free=_ints([4])),
              lambda: sb.spec_pages_fork(pages, _ints([0]), _ints([1, 0]), ws),
              lambda: sb.spec_pages_fork(pages, _ints([0]).long(), _ints([1]), ws),
              lambda: sb.spec_pages_free(pages, torch.tensor([0], dtype=torch.int32), ws),
              lambda: sb.spec_pages_reserve(pages, _ints([1, 1, 1]), ws),
              lambda: sb.PagedKVCache(cfg, 2, 4, 2, k=kv.k[:, :3]),
              lambda: sb.PagedKVCache(cfg, 2, 4, 2, k=kv.k, v=kv.v.half())):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(sb.SpecError):
        sb.spec_pages_reserve(pages, 1, sb.workspace(256)[:256])
    with pytest.raises(sb.SpecError):
        sb.spec_pages_reserve(pages, -1, ws)
