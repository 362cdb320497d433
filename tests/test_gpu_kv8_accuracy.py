"""Accuracy of the 8-bit cache's attention: limits that a wrong output does not pass.

Every limit is made per row and dimension from the fp64 weights, so it shrinks with the outputs as contexts grow;
each case shows that an output of zeros lies beyond it, and those of long contexts an output without one tile of keys.
With P_j = p_j vs_j, in units of the row's sum of weights:

* o is bf16: half a step, 2^-8 |o|;
* a weight is rounded to 11 bits, half a step 2^-11 of itself: 2^-11 sum p |v|;
* a small weight is rounded up or down by one step of its last piece or, with many query rows, by half of fp16's
  smallest: where the row's largest P is 2^2 (2^4) or more, a step is 2^-17 (2^-24).  With few rows the slot number
  decides which way, so that n of them add up like n independent errors of half a step: 6 deviations,
  6 2^-20 max P sqrt(sum code^2).  With many rows each may go the same way: 2^-29 max P sum |code|.  (The largest P
  of a weight's own run over the keys is what counts; it is at most the row's.);
* a score s is off by d: q's elements below 2^-13 of the row's largest by 2^-21 of it, its fp32 sum by
  2^-20 of sum |q k|, its exponent by 2^-21 |s|; that moves a weight and the normaliser by that much each:
  2 d sum p |v|, and to second order nothing that counts;
* sums in fp32: an addition may cut off 2^-23 of its sum, one per 32 keys: T / 32 2^-23 sum p |v|.

The older limits of test_gpu_kv8.py add 2^-18 T max|v| to this, which at thousands of slots is more than the outputs.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv8 as O8
from speculative_decoding_verification_pass_gb300 import binding as sb
from speculative_decoding_verification_pass_gb300 import workloads as wl
from test_gpu_kv8 import _close_code

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Cache:
    """A cache of given rows: k, v [pages][Hkv][64][hd] doubles that e4m3 holds, scales [pages][Hkv][4], and each
    sequence's pages in order (a page may serve several places: attention only reads)."""

    def __init__(self, hd, H, k, v, ks, vs, pages, lens, n, columns=0):
        P, Hkv = k.shape[:2]
        self.cfg = sb.ModelConfig(1, hd * H, H, Hkv, 128, 1000)
        self.k, self.v, self.ks, self.vs = (x.double().cuda() for x in (k, v, ks, vs))
        self.pages, self.lens, self.n = [torch.as_tensor(p).long().cuda() for p in pages], list(lens), n
        kv = self.kv = sb.KV8Cache(self.cfg, len(lens), P, max(columns, max(len(p) for p in pages)))
        for dst, x in ((kv.k, self.k), (kv.v, self.v)):
            dst[0] = x.float().to(E4M3)
            assert torch.equal(dst[0].double(), x)
        kv.k_scale[0], kv.v_scale[0] = self.ks.float(), self.vs.float()
        for b, p in enumerate(self.pages):
            kv.table[b, :len(p)] = p.int()
        kv.len.copy_(torch.tensor(lens, dtype=torch.int32))
        self.ws = sb.workspace(256)

    def run(self, q, scale=0.0, anc=None):
        out = torch.full_like(q, 7.0)
        sb.spec_kv8_attention(self.cfg, self.kv, 0, self.n, q, out, self.ws, anc=anc, scale=scale)
        assert sb.spec_device_status(self.ws) == (sb.SPEC_OK, 0)
        return out

    def rows(self, b, h):
        """Keys, values, codes of values and their scales of the sequence's slots: [T][hd], ..., [T]."""
        T, pg = self.lens[b] + self.n, self.pages[b]
        ks, vs = (s[pg, h].repeat_interleave(16, dim=1).reshape(-1)[:T] for s in (self.ks, self.vs))
        k, v = (x[pg, h].reshape(-1, x.shape[-1])[:T] for x in (self.k, self.v))
        return k * ks[:, None], v * vs[:, None], v, vs


def _softmax(s, hide):
    """Weights of the slots that are not hidden; none where all are."""
    p = torch.softmax(s.masked_fill(hide, -math.inf), dim=1)
    return p.masked_fill(hide.all(dim=1, keepdim=True), 0.0)


def _limit(q, K, V, code, vs, hide, scale, q_err):
    """(o, limit) [rows][hd] of q's rows, which do not see the slots of `hide` [rows][T]."""
    T = len(K)
    s = (q @ K.T) * scale
    p = _softmax(s, hide)
    o, a = p @ V, p @ V.abs()
    d = scale * (2.0 ** -20 * (q.abs() @ K.abs().T).amax(1) + q_err * q.abs().amax(1) * K.abs().sum(1).max())
    d += 2.0 ** -21 * s.masked_fill(hide, 0.0).abs().amax(1)
    lim = 2.0 ** -8 * o.abs() + a * (2.0 ** -11 + 2 * d[:, None] + T / 32 * 2.0 ** -23)
    top = (p * vs).amax(1, keepdim=True)
    return o, lim + top * (6 * 2.0 ** -20 * code.norm(dim=0) + 2.0 ** -29 * code.abs().sum(0))


def _check(cache, q, out, scale=0.0, q_err=2.0 ** -21, lost=(), see=None):
    """out against the definition in 64 bits; beyond the limits lie zeros and, for each tile of `lost` (of 128 slots,
    counted among those before the new ones), the output without it.  see [B][n][n]: the new slots that each token
    sees (its own and earlier ones)."""
    cfg, n = cache.cfg, cache.n
    hd, H, Hkv = cfg.head_dim, cfg.n_heads, cfg.n_kv_heads
    G, scale = H // Hkv, scale or hd ** -0.5
    worst = 0.0
    for b, L in list(enumerate(cache.lens))[::3 if len(cache.lens) > 9 else 1]:
        for h in range(Hkv):
            at = (slice(b * n, (b + 1) * n), slice(h * G, (h + 1) * G))
            qq, got = (x.view(-1, H, hd)[at].reshape(n * G, hd).double() for x in (q, out))
            hide = torch.zeros(n, L + n, dtype=torch.bool, device="cuda")
            hide[:, L:] = ~(torch.ones(n, n, device="cuda").tril().bool() if see is None else see[b].cuda())
            hide = hide.repeat_interleave(G, dim=0)
            K, V, code, vs = cache.rows(b, h)
            o, lim = _limit(qq, K, V, code, vs, hide, scale, q_err)
            assert torch.isfinite(got).all()
            over = ((got - o).abs() / lim.clamp_min(1e-200)).max().item()
            worst = max(worst, over)
            assert over <= 1.0, (b, h, L, over)
            assert ((o.abs() > lim).any(dim=1) | hide.all(dim=1)).all(), (b, h, "zeros would pass")
            if b > 1 or h not in (0, Hkv - 1):
                continue
            for t in lost:
                t %= max(1, L // 128)
                if L < 128:
                    continue
                without = hide.clone()
                without[:, 128 * t:128 * t + 128] = True
                p = _softmax((qq @ K.T) * scale, without)
                assert ((p @ V - o).abs() > lim).any(), (b, h, t, "an output without this tile would pass")
    return worst


# ------------------------------------------------------- small weights that count
def _tail(hd, H, Hkv, T, B, where, nats, n, columns=0):
    """One key `nats` above all others, which are alike: of B sequences each has it elsewhere.  By dimension (mod 8)
    the others' values are 1, 1, 0, -1 / 16, 1 in every second slot, 2 in every 16th, 1 and -1 in turn, 0.5 in every
    third, and its own 0 and then 1."""
    t = torch.arange(64)
    by = [1 + 0 * t, 1 + 0 * t, 0 * t, 0 * t - 1 / 16, t % 2, 2 * (t % 16 == 3), 1 - t % 2 * 2, 0.5 * (t % 3 == 1)]
    k, v = torch.zeros(2, Hkv, 64, hd), torch.stack([x.double() for x in by], dim=1).repeat(2, Hkv, 1, hd // 8)
    k[1, :, 17, 0] = 1.0
    v[1, :, 17] = 1.0
    v[1, :, 17, ::8] = 0.0
    ones = torch.ones(2, Hkv, 4)
    pages = []
    for b in range(B):
        p = np.zeros((T + n + 63) // 64, np.int64)
        p[int(where[b % len(where)] * (T // 64 - 1))] = 1
        pages.append(p)
    c = Cache(hd, H, k, v, ones, ones, pages, [T - b for b in range(B)], n, columns)
    q = torch.zeros(B * n, H, hd)
    for m in range(B * n):
        for h in range(H):
            q[m, h, 0] = nats[(m + h) % len(nats)]
    return c, q.to(torch.bfloat16).view(B * n, H * hd).cuda()


@pytest.mark.parametrize("hd,H,Hkv,T,B,n,columns", [
    (128, 8, 8, 131071, 20, 1, 0),     # a run of a whole context
    (128, 8, 8, 131000, 1, 1, 0),      # runs of a cluster's CTAs, two groups each
    (128, 4, 1, (1 << 20) - 2, 1, 2, 0),
    (64, 16, 2, 33000, 80, 1, 0),
    (128, 16, 1, 17000, 170, 2, 0),    # 32 rows
    (128, 12, 1, 9000, 200, 2, 0),     # 24 rows
    (128, 4, 1, 700, 2, 3, 0),
    (64, 4, 1, 5000, 3, 2, 0),
    (128, 8, 8, 16000, 20, 128, 0),    # many query rows
])
def test_one_strong_key_over_a_long_tail(hd, H, Hkv, T, B, n, columns):
    """A tail whose weights are 2^-17 to 2^-23 of the strongest's, but half of the sum by their number."""
    c, q = _tail(hd, H, Hkv, T, B, (0.0, 0.31, 0.77, 1.0), [8.0, 10.0, 12.0, 13.0, 13.5, 14.0, 16.0], n, columns)
    out = c.run(q, scale=1.0)
    _check(c, q, out, scale=1.0)


def test_a_strong_key_after_a_long_weak_run():
    """The strongest key at the end of runs of growing weights, and of falling ones."""
    hd, H, Hkv, T, n = 128, 8, 8, 40000, 1
    for order in (1, -1):
        steps = 40
        k, v = torch.zeros(steps, Hkv, 64, hd), torch.zeros(steps, Hkv, 64, hd)
        for i in range(steps):
            k[i, :, :, i % 8] = 1.0
            k[i, :, :, 8 + i // 8] = 1.0
            v[i, :, :, i] = 1.0
            v[i, :, :, 127] = 1.0
        ones = torch.ones(steps, Hkv, 4)
        per = T // 64 // steps
        pages = np.repeat(np.arange(steps)[::order], per)
        pages = [np.concatenate([pages, np.full((T + n + 63) // 64 - len(pages), pages[-1])])] * 20
        c = Cache(hd, H, k, v, ones, ones, pages, [T] * 20, n)
        q = torch.zeros(20 * n, H, hd)
        q[:, :, :8] = torch.arange(8) * 1.5  # score 1.5 i, over 58 nats
        q[:, :, 8:13] = torch.arange(5) * 12.0
        for b in range(20):
            q[b] *= (b % 5 + 1) / 8
        q = q.to(torch.bfloat16).view(20 * n, H * hd).cuda()
        _check(c, q, c.run(q, scale=1.0), scale=1.0)


# ------------------------------------------------------- queries with a strong channel
@pytest.mark.parametrize("deep", [13, 22])
@pytest.mark.parametrize("hd,H,Hkv,n,columns", [(128, 8, 8, 1, 0), (128, 4, 1, 5, 0), (64, 16, 2, 4, 0), (128, 8, 8, 2, 500),
                                                (128, 4, 1, 40, 1400), (64, 16, 2, 30, 1400)])
def test_small_query_elements_beside_a_large_one(hd, H, Hkv, n, columns, deep):
    """One channel of q is the strongest and another of k: dimension d of q lies 2^-(d mod 14) below the row's
    largest (every element from there on is exact), or as far as 2^-22, and the keys make up for it."""
    g = torch.Generator().manual_seed(61)
    lens, P = (30, 7, 200, 64), 6
    fall = torch.arange(hd) % (deep + 1)
    rise = 2.0 ** (fall * 14.0 / (deep + 1) - 6)
    k = (torch.randn(P, Hkv, 64, hd, generator=g) * rise).clamp(-448, 448).to(E4M3).double()
    v = (torch.randn(P, Hkv, 64, hd, generator=g) * 40).clamp(-448, 448).to(E4M3).double()
    ks, vs = (2.0 ** torch.randint(-8, -5, (P, Hkv, 4), generator=g).double() for _ in "kv")
    pages = [[(b + i) % P for i in range(5)] for b in range(len(lens))]
    c = Cache(hd, H, k, v, ks, vs, pages, lens, n, columns)
    M = len(lens) * n
    q = 1 + torch.randint(0, 128, (M, H, hd), generator=g) / 128
    q = q * 2.0 ** (10 - fall) * (1 - 2 * torch.randint(0, 2, (M, H, hd), generator=g))
    q = q.to(torch.bfloat16).view(M, H * hd).cuda()
    exact = deep <= 13
    _check(c, q, c.run(q, scale=0.7), scale=0.7, q_err=0.0 if exact else 2.0 ** -21)


# ------------------------------------------------------------------ long contexts
def _marked(hd, H, Hkv, lens, n, columns, seed):
    """Random rows; both pages of a tile of 128 slots carry a large value in a dimension that it shares with few
    other tiles.  The sequences take the tiles in orders of their own."""
    g = torch.Generator().manual_seed(seed)
    tiles = (max(lens) + n + 127) // 128
    P = 2 * tiles
    k = torch.randn(P, Hkv, 64, hd, generator=g).mul_(8).to(E4M3)
    v = torch.randn(P, Hkv, 64, hd, generator=g)
    v[torch.arange(P), :, :, torch.arange(P) // 2 % hd] = 64.0
    ks, vs = (2.0 ** torch.randint(a, a + 2, (P, Hkv, 4), generator=g).double() for a in (-4, -7))
    pages = []
    for L in lens:
        order = torch.randperm(tiles, generator=g)[:(L + n + 127) // 128]
        pages.append(torch.stack([2 * order, 2 * order + 1], dim=1).view(-1)[:(L + n + 63) // 64])
    c = Cache(hd, H, k, v.to(E4M3), ks, vs, pages, lens, n, columns)
    q = torch.randn(len(lens) * n, H * hd, generator=g).to(torch.bfloat16).cuda()
    return c, q


@pytest.mark.parametrize("hd,H,Hkv,lens,n,columns", [
    (128, 4, 1, (40000,), 5, 0),                     # 24 query rows a tile, two groups a CTA
    (128, 8, 8, (60000,), 5, 0),                     # 8
    (128, 12, 1, (20000, 9000), 1, 0),               # 16
    (64, 4, 1, (30000,), 7, 0),                      # 32
    (128, 8, 8, (131000,), 1, 0),
    (128, 8, 2, (400000,), 1, 0),
    (128, 8, 2, (1000000,), 1, 0),                   # (a tile is less than the sums' own rounding here)
    (128, 6, 2, (3000, 7000), 9, 1400),              # 27 rows
    (64, 16, 2, (5000, 126, 0), 4, 1400),
    (128, 8, 8, (12000, 300, 7000) * 10, 3, 0),      # one group a CTA, a batch
    (64, 16, 2, (9000, 2000, 6000, 100) * 30, 2, 0),
    (128, 12, 2, (8000, 5000) * 90, 4, 0),
    (64, 8, 2, (4000, 8000) * 60, 8, 0),
    (128, 4, 1, (5000,), 40, 0),                     # many query rows
    (128, 8, 8, (12000, 3000, 100, 7000), 70, 1400),
    (64, 16, 2, (30000, 2000), 100, 0),
    (128, 8, 8, (16000,) * 20, 128, 0),
])
def test_long_contexts(hd, H, Hkv, lens, n, columns):
    """Every tile of a long context counts: runs long enough that the rings turn over many times."""
    c, q = _marked(hd, H, Hkv, lens, n, columns, 71)
    tiles = (0, 1, 2, max(lens) // 300, max(lens) // 150, -2, -1)
    _check(c, q, c.run(q), lost=tiles if max(lens) < 2 ** 19 else ())


@pytest.mark.parametrize("hd,H,Hkv,lens,n,columns", [
    (128, 4, 1, (0, 700, 2500), 13, 0),
    (64, 16, 2, (3000, 1), 15, 0),                   # two row tiles
    (64, 4, 2, (1250, 0), 30, 1400),                 # two groups a CTA
    (128, 12, 1, (2000, 900) * 60, 3, 0),            # one
    (128, 4, 1, (100, 4000), 64, 1400),              # many query rows
    (64, 16, 2, (0, 6000, 77), 21, 1400),
])
def test_trees_in_long_contexts(hd, H, Hkv, lens, n, columns):
    """Draft trees: some nodes do not see themselves, and the first of an empty cache sees nothing."""
    c, q = _marked(hd, H, Hkv, lens, n, columns, 72)
    see, anc = [], []
    for b in range(len(lens)):
        masks, _ = sb.spec_tree_masks(wl.random_tree(80 + b, n))
        masks[0], masks[-1] = 0, masks[-1] & ~(1 << (n - 1))
        see.append(torch.tensor([[m >> i & 1 for i in range(n)] for m in masks]).bool())
        anc.append(masks)
    out = c.run(q, anc=torch.from_numpy(np.array(anc, np.uint64).astype(np.int64)).cuda())
    _check(c, q, out, lost=(0, 3, -1), see=see)
    for b, L in enumerate(lens):
        assert L or (out[b * n] == 0).all()


# ------------------------------------------------------------ rows held while scales grow
def test_rows_held_while_a_scale_grows():
    """Rows of one block appended one by one, each larger: codes and scales are the oracle's, and a row is off by
    its own rounding and at most half of each later scale's smallest step."""
    hd, H, Hkv = 64, 4, 2
    cfg = sb.ModelConfig(1, hd * H, H, Hkv, 128, 1000)
    kv, ws = sb.KV8Cache(cfg, 1, 1, 1), sb.workspace(256)
    kv.table.zero_()
    R = sb.RopeTable(hd, 1e4)
    g = torch.Generator().manual_seed(81)
    want, slack, rows = O8.Rows(Hkv, 64, hd), np.zeros((Hkv, 64, 1)), []
    for t in range(20):
        x = torch.randn(1, Hkv * hd, generator=g) * 2.0 ** (1.5 * (t % 16))
        q = torch.zeros(1, H * hd)
        sb.spec_kv8_append(cfg, kv, 0, 1, q.cuda(), torch.zeros(1, Hkv * hd).cuda(), x.cuda(), R,
                           torch.empty(1, H * hd, dtype=torch.bfloat16, device="cuda"), ws)
        sb.spec_kv8_advance(kv, 1, ws)
        rows.append(x.double().numpy().reshape(Hkv, hd))
        old = want.scale[:, t // 16].copy()
        want.append(t, rows[-1][None])
        grown = want.scale[:, t // 16] > old
        slack[:, t // 16 * 16:t] += np.where(grown, want.scale[:, t // 16] / 1024, 0.0)[:, None, None]
        code = O8.e4m3_of_byte(kv.v.view(torch.uint8)[0, 0].cpu().numpy())
        scale = kv.v_scale[0, 0].double().cpu().numpy()
        blocks = t // 16 + 1
        np.testing.assert_array_equal(scale[:, :blocks], want.scale[:, :blocks])
        np.testing.assert_array_equal(code[:, :t + 1], want.code[:, :t + 1])
        _close_code(code[:, :t + 1], scale, np.stack(rows, axis=1), slack[:, :t + 1])
    assert sb.spec_device_status(ws) == (sb.SPEC_OK, 0)


# ------------------------------------------------------------- scores past fp32's range
@pytest.mark.parametrize("hd,H,Hkv,n,columns", [(128, 8, 1, 2, 0), (64, 4, 2, 1, 600), (128, 4, 1, 40, 1400)])
def test_scores_past_the_range(hd, H, Hkv, n, columns):
    """A score above fp32's range makes the rows that see it NaN; one below it is a key of no weight."""
    for sign in (1, -1):
        g = torch.Generator().manual_seed(91)
        k, v = torch.zeros(4, Hkv, 64, hd), torch.randn(4, Hkv, 64, hd, generator=g).to(E4M3)
        k[2, :, 21] = 448.0 * sign
        ks, vs = torch.full((4, Hkv, 4), 2.0 ** 30), torch.ones(4, Hkv, 4)
        c = Cache(hd, H, k, v, ks, vs, [[0, 1, 2, 3], [3, 0, 1, 1]], [150, 30], n, columns)
        q = torch.full((2 * n, H * hd), 2.0 ** 90, dtype=torch.bfloat16, device="cuda")
        out = c.run(q).view(2, n, H, hd).double()
        if sign > 0:
            assert torch.isnan(out[0]).all()
        for b in range(2):
            if b == 0 and sign > 0:
                continue
            for h in range(H):
                _, V, _, _ = c.rows(b, h // (H // Hkv))
                for j in range(n):
                    seen = torch.arange(c.lens[b] + j + 1, device="cuda")
                    o = V[seen[seen != 2 * 64 + 21] if b == 0 else seen].mean(0)
                    lim = 2.0 ** -8 * o.abs() + 2.0 ** -10 * V.abs().mean(0)
                    assert ((out[b, j, h] - o).abs() <= lim).all()
