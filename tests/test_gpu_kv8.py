"""GPU parity of the 8-bit paged KV cache with the fp64 oracle (oracle/kv8.py).

Tolerances, from the formats:

* a code is the nearest e4m3 value of x / s: |code s - x| <= max(2^-4 |x|,
  2^-10 s) (half a step; the subnormal step is 2^-9), and where x needs no
  rotation (values, unrotated dimensions) the code is the oracle's exactly.
  A rotated x is formed in fp32 from a sine and cosine within 2^-21 of theirs:
  another 2^-20 of the pair's size;
* q_out and o are bf16: half a step, 2^-8 of the value;
* attention: a softmax weight is off by 2^-11 of itself, and by 2^-18 of its
  row's largest (its last piece's subnormal step); a score by 2^-17 of
  sum |q| |k|, which moves a weight and the normaliser by that much each.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv8 as O8
from oracle import model as OM
from oracle import weights as OW
from speculative_decoding_verification_pass_gb300 import binding as sb
from speculative_decoding_verification_pass_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
THETA = 500000.0
HEADS = {"64x4/2": (64, 4, 2), "128x4/1": (128, 4, 1), "128x8/8": (128, 8, 8), "64x16/2": (64, 16, 2),
         "128x6/2": (128, 6, 2)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _cfg(heads, layers=1):
    hd, H, Hkv = HEADS[heads]
    if (hd * H) % 128:
        raise ValueError(heads)
    return sb.ModelConfig(layers, hd * H, H, Hkv, 128, 1000)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Pair:
    """A device cache with shuffled pages and the oracle's rows of the same contents."""

    def __init__(self, cfg, lens, room, seed, layers=1, columns=0):
        self.cfg, self.lens, self.B = cfg, list(lens), len(lens)
        rng = np.random.default_rng(seed)
        need = [(x + room + 63) // 64 for x in lens]
        self.kv = sb.KV8Cache(cfg, self.B, sum(need) + 2, max(max(need) + 1, columns))
        ids = rng.permutation(sum(need) + 2)
        table = np.full((self.B, self.kv.max_pages), -1, np.int32)
        at = 0
        for b in range(self.B):
            table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.table = table
        self.kv.table.copy_(_dev(table))
        self.kv.len.copy_(_dev(np.array(lens, np.int32)))
        hd, Hkv = cfg.head_dim, cfg.n_kv_heads
        shape = tuple(self.kv.k.shape)
        self.bits = {}
        self.scales = {}
        for name in "kv":  # any codes that are numbers; scales near those of unit rows
            self.bits[name] = rng.integers(0, 256, shape).astype(np.uint8)
            self.bits[name][(self.bits[name] & 0x7F) == 0x7F] = 0x30
            self.scales[name] = 2.0 ** rng.integers(-9, -6, shape[:3] + (4,)).astype(np.float64)
        self.rows = {(l, b, name): self._oracle_rows(l, b, name, Hkv, hd) for l in range(layers)
                     for b in range(self.B) for name in "kv"}
        for name in "kv":
            self.put_bits(name)

    def put_bits(self, name):
        getattr(self.kv, name).view(torch.uint8).copy_(_dev(self.bits[name]))
        getattr(self.kv, name + "_scale").copy_(_dev(self.scales[name].astype(np.float32)))

    def _oracle_rows(self, l, b, name, Hkv, hd):
        pages = self.table[b][self.table[b] >= 0]
        r = O8.Rows(Hkv, 64 * len(pages), hd)
        for i, pg in enumerate(pages):
            r.code[:, 64 * i:64 * i + 64] = O8.e4m3_of_byte(self.bits[name][l, pg])
            r.scale[:, 4 * i:4 * i + 4] = self.scales[name][l, pg]
        return r

    def got(self, l, b, name):
        """(codes as values [Hkv][slots][hd], scales [Hkv][blocks]) on the device now."""
        pages = self.table[b][self.table[b] >= 0]
        c = O8.e4m3_of_byte(getattr(self.kv, name).view(torch.uint8)[l].cpu().numpy()[pages])
        s = getattr(self.kv, name + "_scale")[l].cpu().numpy()[pages].astype(np.float64)
        return (np.concatenate(list(c), axis=1), np.concatenate(list(s), axis=1))


def _status(ws):
    return sb.spec_device_status(ws)


# ------------------------------------------------------------------- append
def _close_code(got, scale, x, slack):
    s = np.repeat(scale, 16, axis=1)[:, :got.shape[1], None]
    lim = np.maximum(np.abs(x) / 16, s / 1024) + slack
    err = np.abs(got * s - x)
    assert (err <= lim).all(), (err - lim).max()


ROPES = {"half": dict(inter=False), "inter": dict(inter=True), "part": dict(inter=False, part=True),
         "inter-part-scaled": dict(inter=True, part=True, factor=4.0),
         "by-wavelength": dict(inter=False, factor=8.0, orig=64)}


@pytest.mark.parametrize("heads,rope,dtype,lens,n", [
    ("128x4/1", "half", "bf16", (0, 1, 15, 16, 63, 64, 130), 5),
    ("64x4/2", "half", "f32", (0, 1, 15, 16, 63, 64, 130), 5),
    ("64x4/2", "inter", "bf16", (3, 48), 1),
    ("128x8/8", "inter-part-scaled", "f32", (0, 47), 17),
    ("64x16/2", "part", "bf16", (1000, 5), 33),
    ("128x6/2", "by-wavelength", "f32", (777, 0, 8), 128),
])
def test_append(heads, rope, dtype, lens, n):
    cfg = _cfg(heads)
    hd, H, Hkv = HEADS[heads]
    P = Pair(cfg, lens, n, 11)
    how = ROPES[rope]
    rd = hd // 2 if how.get("part") else hd
    R = sb.RopeTable(rd, THETA, how["inter"], how.get("factor", 1.0), orig_len=how.get("orig", 0))
    freq = O8.frequencies(rd, THETA, how.get("factor", 1.0), orig_len=how.get("orig", 0))
    g = torch.Generator().manual_seed(5)
    M = len(lens) * n
    qkv = torch.randn(M, (H + 2 * Hkv) * hd, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    qkv = qkv.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    qkv[0, H * hd:] = 0  # a token of zeros
    dev = qkv.cuda()
    q, k, v = dev.split([H * hd, Hkv * hd, Hkv * hd], dim=1)  # rows of one wider tensor
    before = {name: P.kv.__dict__[name].view(torch.uint8).clone() for name in "kv"}
    ws = sb.workspace(256)
    q_out = torch.empty(M, H * hd, dtype=torch.bfloat16, device="cuda")
    sb.spec_kv8_append(cfg, P.kv, 0, n, q, k, v, R, q_out, ws)
    assert _status(ws) == (sb.SPEC_OK, 0)
    assert P.kv.len.cpu().tolist() == list(lens)
    x = qkv.double().numpy()
    qx, kx, vx = np.split(x, [H * hd, (H + Hkv) * hd], axis=1)
    got_q = q_out.double().cpu().numpy().reshape(M, H, hd)
    touched = {name: np.zeros(tuple(P.kv.k.shape[1:4]), bool) for name in "kv"}
    for b, L in enumerate(lens):
        new_k = np.zeros((n, Hkv, hd))
        for j in range(n):
            m = b * n + j
            want = O8.rotate(qx[m].reshape(H, hd), L + j, freq, how["inter"])
            slack = 2.0 ** -20 * 2 * np.abs(qx[m]).max()
            assert (np.abs(got_q[m] - want) <= 2.0 ** -8 * np.abs(want) + slack).all()
            new_k[j] = O8.rotate(kx[m].reshape(Hkv, hd), L + j, freq, how["inter"])
        slots = np.arange(L // 16 * 16, L + n)
        for name in "kv":
            pg, r = P.table[b][slots // 64], slots % 64
            touched[name][pg, :, r] = True
        new_v = vx[b * n:(b + 1) * n].reshape(n, Hkv, hd)
        for name, new in (("k", new_k), ("v", new_v)):
            want = P.rows[0, b, name]
            want.append(L, new)
            code, scale = P.got(0, b, name)
            blocks = np.arange(L // 16, (L + n - 1) // 16 + 1)
            np.testing.assert_array_equal(scale[:, blocks], want.scale[:, blocks])
            np.testing.assert_array_equal(code[:, :L], want.code[:, :L])
            if name == "v" or rd < hd:
                np.testing.assert_array_equal(code[:, L:L + n, (0 if name == "v" else rd):],
                                              want.code[:, L:L + n, (0 if name == "v" else rd):])
            s = np.repeat(want.scale, 16, axis=1)[:, L:L + n, None]
            xx = new.transpose(1, 0, 2)
            slack = 2.0 ** -20 * 2 * np.abs(new).max()
            err = np.abs(code[:, L:L + n] * s - xx)
            assert (err <= np.maximum(np.abs(xx) / 16, s / 1024) + slack).all()
    for name in "kv":  # rows and pages that the call has no business with
        now = P.kv.__dict__[name].view(torch.uint8)
        same = (now == before[name])[0].all(-1).cpu().numpy()
        assert same[~touched[name]].all()


def test_append_far_position_and_depths():
    """Positions near the last slot of a 2^20-slot table, and a tree's depths."""
    cfg = _cfg("64x4/2")
    hd, H, Hkv = HEADS["64x4/2"]
    pages = (1 << 20) // 64
    kv = sb.KV8Cache(cfg, 1, 2, pages)
    kv.table[0, -2:] = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    L, n = (1 << 20) - 70, 4
    kv.len.fill_(L)
    depth = np.array([[0, 1, 1, 2]], np.int32)
    R = sb.RopeTable(hd, THETA)
    freq = O8.frequencies(hd, THETA)
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(n, h * hd, generator=g) for h in (H, Hkv, Hkv))
    q_out = torch.empty(n, H * hd, dtype=torch.bfloat16, device="cuda")
    ws = sb.workspace(256)
    sb.spec_kv8_append(cfg, kv, 0, n, q.cuda(), k.cuda(), v.cuda(), R, q_out, ws, depth=_dev(depth))
    assert _status(ws) == (sb.SPEC_OK, 0)
    got = q_out.double().cpu().numpy().reshape(n, H, hd)
    for j in range(n):
        want = O8.rotate(q[j].double().numpy().reshape(H, hd), L + int(depth[0, j]), freq, False)
        assert (np.abs(got[j] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18).all()
    code = O8.e4m3_of_byte(kv.v.view(torch.uint8)[0].cpu().numpy())  # [pages][Hkv][64][hd]
    scale = kv.v_scale[0].cpu().numpy().astype(np.float64)
    rows = O8.Rows(Hkv, 128, hd)
    rows.scale[:] = 1.0  # a new cache's scales: the block holds ten rows from before
    rows.append(58, v.double().numpy().reshape(n, Hkv, hd))
    np.testing.assert_array_equal(code[1, :, 58:62], rows.code[:, 58:62])
    np.testing.assert_array_equal(scale[1, :, 3], rows.scale[:, 3])


def test_append_not_numbers():
    """Infinities saturate and set no scale; NaN stays NaN; neither touches other rows."""
    cfg = _cfg("128x4/1")
    hd, H, Hkv = HEADS["128x4/1"]
    n = 3
    kv = sb.KV8Cache(cfg, 1, 1, 1)
    kv.table.zero_()
    v = torch.randn(n, hd, generator=torch.Generator().manual_seed(3))
    v[1, 5], v[1, 6], v[2, 7] = float("inf"), -float("inf"), float("nan")
    q_out = torch.empty(n, H * hd, dtype=torch.bfloat16, device="cuda")
    ws = sb.workspace(256)
    q = torch.zeros(n, H * hd)
    sb.spec_kv8_append(cfg, kv, 0, n, q.cuda(), torch.zeros(n, hd).cuda(), v.cuda(), sb.RopeTable(hd, THETA), q_out, ws)
    rows = O8.Rows(1, 64, hd)
    rows.append(0, v.double().numpy().reshape(n, 1, hd))
    code = O8.e4m3_of_byte(kv.v.view(torch.uint8)[0, 0].cpu().numpy())
    np.testing.assert_array_equal(code[:, :n], rows.code[:, :n])
    assert code[0, 1, 5] == 448 and code[0, 1, 6] == -448 and np.isnan(code[0, 2, 7])
    assert kv.v_scale[0, 0, 0, 0].item() == rows.scale[0, 0]
    assert kv.k_scale[0, 0, 0, 0].item() == 2.0 ** -40  # a block of zeros


# ---------------------------------------------------------------- attention
def _chain(n):
    return np.tril(np.ones((n, n), bool))


def _check_attention(cfg, P, n, q, out, see, scale):
    hd, H, Hkv = cfg.head_dim, cfg.n_heads, cfg.n_kv_heads
    worst = 0.0
    for b, L in enumerate(P.lens):
        K, V = (P.rows[0, b, name].value(L + n) for name in "kv")
        qb = q[b * n:(b + 1) * n].double().cpu().numpy().reshape(n, H, hd)
        o, a = O8.attention(qb, K, V, L, see[b], scale)
        # the largest score size a row sees: sum |q| |k| over its KV head's slots
        size = np.zeros((n, H, 1))
        for h in range(H):
            size[:, h, 0] = (np.abs(qb[:, h]) @ np.abs(K[h // (H // Hkv)]).T).max(axis=1) * scale
        lim = 2.0 ** -8 * np.abs(o) + (2 * 2.0 ** -11 + 4 * 2.0 ** -17 * size) * a
        lim += 2.0 ** -18 * (L + n) * np.abs(V).max() / max(1, 1)
        got = out[b * n:(b + 1) * n].double().cpu().numpy().reshape(n, H, hd)
        assert np.isfinite(got).all()
        err = np.abs(got - o)
        worst = max(worst, (err / lim).max())
        assert (err <= lim).all(), (b, L, (err / lim).max())
    return worst


def _run_attention(cfg, P, n, q, anc=None, scale=0.0, ws=None):
    out = torch.full_like(q, 7.0)
    ws = sb.workspace(256) if ws is None else ws
    sb.spec_kv8_attention(cfg, P.kv, 0, n, q, out, ws, anc=anc, scale=scale)
    return out, ws


def _q(rows, width, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(rows, width, generator=g)).to(torch.bfloat16).cuda()


def _stale(P, n):
    """Codes that are not numbers, and useless scales, in every slot past the new ones."""
    for b, L in enumerate(P.lens):
        for i, pg in enumerate(P.table[b]):
            if pg < 0:
                continue
            first = min(64, max(0, L + n - 64 * i))
            for name in "kv":
                P.bits[name][0, pg, :, first:] = 0x7F
                P.scales[name][0, pg, :, (first + 15) // 16:] = np.nan
    for name in "kv":
        P.put_bits(name)


@pytest.mark.parametrize("heads,lens,n", [
    ("128x4/1", (0, 1, 63, 64, 127, 128, 129, 400), 1),
    ("128x4/1", (0, 3, 59, 123, 124, 250, 700), 5),
    ("64x4/2", (0, 3, 59, 123, 124, 250, 700), 5),
    ("64x16/2", (2000, 17), 3),
    ("128x6/2", (300, 1), 7),
    ("128x8/8", (130, 0), 9),
    ("64x4/2", (5, 190), 33),
    ("128x4/1", (0, 77, 300), 128),
    ("128x4/1", (5000,), 4),
])
def test_attention_chain(heads, lens, n):
    cfg = _cfg(heads)
    P = Pair(cfg, lens, n + 40, 21)
    _stale(P, n)
    q = _q(len(lens) * n, cfg.n_heads * cfg.head_dim, 31)
    out, ws = _run_attention(cfg, P, n, q)
    assert _status(ws) == (sb.SPEC_OK, 0)
    _check_attention(cfg, P, n, q, out, [_chain(n)] * len(lens), cfg.head_dim ** -0.5)


@pytest.mark.parametrize("heads,lens,n", [("128x4/1", (0, 100, 250), 13), ("64x4/2", (0, 125), 64),
                                          ("64x16/2", (60, 1), 15)])
def test_attention_tree(heads, lens, n):
    """Draft trees; some nodes lack their own bit (and with an empty cache see nothing: zero rows)."""
    cfg = _cfg(heads)
    P = Pair(cfg, lens, n + 40, 22)
    _stale(P, n)
    q = _q(len(lens) * n, cfg.n_heads * cfg.head_dim, 32)
    see, anc = [], []
    for b in range(len(lens)):
        masks, _ = sb.spec_tree_masks(wl.random_tree(40 + b, n))
        masks[0] = 0  # the root's row sees no new slot
        masks[n - 1] &= ~(1 << (n - 1))
        see.append(np.array([[(m >> i) & 1 for i in range(n)] for m in masks], bool))
        # a bit past the last node is ignored
        anc.append([m | (1 << n) if n < 63 else m for m in masks])
    t = _dev(np.array(anc, np.uint64).astype(np.int64))
    out, ws = _run_attention(cfg, P, n, q, anc=t)
    assert _status(ws) == (sb.SPEC_OK, 0)
    _check_attention(cfg, P, n, q, out, see, cfg.head_dim ** -0.5)
    empty = [b for b, L in enumerate(lens) if L == 0]
    for b in empty:
        assert (out[b * n] == 0).all()


def test_attention_scale_strides_and_sharp_rows():
    """A given scale, rows of wider tensors, scores far apart (one key takes all)."""
    cfg, n, lens = _cfg("128x4/1"), 3, (200, 70)
    P = Pair(cfg, lens, n, 23)
    width = cfg.n_heads * cfg.head_dim
    wide = _q(len(lens) * n, width + 64, 33, size=8.0)
    q = wide[:, 64:]
    ow = torch.full((len(lens) * n, width + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = sb.workspace(256)
    sb.spec_kv8_attention(cfg, P.kv, 0, n, q, ow[:, :width], ws, scale=0.5)
    assert (ow[:, width:] == 3.0).all()
    _check_attention(cfg, P, n, q, ow[:, :width], [_chain(n)] * 2, 0.5)


@pytest.mark.parametrize("name,top", [("v", 2.0 ** 30), ("v", 0.0), ("k", 0.0)])
def test_attention_uneven_scales(name, top):
    """Blocks whose scales are far apart, and blocks of zeros at the smallest scale."""
    cfg, n, lens = _cfg("128x4/1"), 5, (300, 40)
    P = Pair(cfg, lens, n, 24)
    pg = P.table[0, 2]
    if top:
        P.scales[name][0, pg] *= top
    else:
        P.bits[name][0, pg] = 0
        P.scales[name][0, pg] = 2.0 ** -40
    P.put_bits(name)
    for b in range(2):
        for nm in "kv":
            P.rows[0, b, nm] = P._oracle_rows(0, b, nm, cfg.n_kv_heads, cfg.head_dim)
    q = _q(len(lens) * n, cfg.n_heads * cfg.head_dim, 34)
    out, _ = _run_attention(cfg, P, n, q)
    _check_attention(cfg, P, n, q, out, [_chain(n)] * 2, cfg.head_dim ** -0.5)


@pytest.mark.parametrize("heads", ["128x4/1", "64x4/2"])
def test_attention_not_numbers(heads):
    """NaN codes reach exactly the rows that see them, and there exactly their dimension (values) or
    the whole row (keys); so do infinities and NaN in q."""
    cfg, n, lens = _cfg(heads), 6, (70, 200)
    H, hd, Hkv = cfg.n_heads, cfg.head_dim, cfg.n_kv_heads
    G = H // Hkv
    q = _q(len(lens) * n, H * hd, 35)
    ref, _ = _run_attention(cfg, Pair(cfg, lens, n + 30, 25), n, q)

    def put(name, b, slot, dim):
        P = Pair(cfg, lens, n + 30, 25)
        P.bits[name][0, P.table[b, slot // 64], Hkv - 1, slot % 64, dim] = 0xFF
        P.put_bits(name)
        out, _ = _run_attention(cfg, P, n, q)
        return out.view(len(lens), n, H, hd)

    want = ref.view(len(lens), n, H, hd)
    last = slice((Hkv - 1) * G, H)
    for name, b, slot, dim in (("v", 0, 70 + 3, 9), ("v", 1, 200 + 3, hd - 1), ("k", 0, 70 + 3, 1), ("v", 1, 20, 3),
                               ("k", 1, 199, 0)):
        out = put(name, b, slot, dim)
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        j0 = max(0, slot - lens[b])
        if name == "v":
            hit[b, j0:, last, dim] = True
        else:
            hit[b, j0:, last, :] = True
        assert torch.equal(torch.isnan(out), hit), (name, b, slot)
        assert torch.equal(out[~hit], want[~hit])
    for bad in (float("inf"), -float("inf"), float("nan")):
        q2 = q.clone()
        q2[n + 2, hd + 5] = bad  # sequence 1, token 2, head 1
        out, _ = _run_attention(cfg, Pair(cfg, lens, n + 30, 25), n, q2)
        out = out.view(len(lens), n, H, hd)
        assert torch.isnan(out[1, 2, 1]).all()
        keep = torch.ones(out.shape[:3], dtype=torch.bool)
        keep[1, 2, 1] = False
        assert torch.equal(out[keep.cuda()], want[keep.cuda()])


# ------------------------------------------------------------------- commit
@pytest.mark.parametrize("heads,lens,n,paths", [
    ("128x4/1", (0, 14, 15, 16, 60, 200), 9, ([], [1], [2, 3, 8], [1, 2, 3], [4, 6], [1, 2, 3, 4, 5, 6, 7, 8])),
    ("64x4/2", (7, 63, 0), 64, (list(range(1, 64)), list(range(30, 64)), [63])),
    ("64x4/2", (5, 130), 1, ([], [])),
])
def test_tree_commit(heads, lens, n, paths):
    layers = 3
    cfg = _cfg(heads, layers)
    P = Pair(cfg, lens, n, 26, layers)
    P.kv.len.add_(n)
    path = np.full((len(lens), n), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    ws = sb.workspace(256)
    sb.spec_kv8_tree_commit(cfg, P.kv, _dev(path), _dev(np.array([len(p) for p in paths], np.int32)), n, ws)
    assert _status(ws) == (sb.SPEC_OK, 0)
    assert P.kv.len.cpu().tolist() == [L + 1 + len(p) for L, p in zip(lens, paths)]
    for (l, b, name), want in P.rows.items():
        want.commit(lens[b], paths[b])
        code, scale = P.got(l, b, name)
        np.testing.assert_array_equal(scale, want.scale)
        np.testing.assert_array_equal(code, want.code)


# ------------------------------------------------- refusals seen by the device
def test_sequences_that_do_not_fit():
    cfg = _cfg("64x4/2")
    hd, H, Hkv = HEADS["64x4/2"]
    n, lens = 3, (4, 126, 10, 2)
    kv = sb.KV8Cache(cfg, 4, 4, 2)
    kv.table.copy_(torch.tensor([[0, -1], [1, 2], [9, -1], [3, -1]], dtype=torch.int32))
    kv.len.copy_(torch.tensor([4, 126, 10, -1], dtype=torch.int32))
    for name in "kv":
        getattr(kv, name).view(torch.uint8).random_(0, 0x70)
    before = [kv.k.view(torch.uint8).clone(), kv.v.view(torch.uint8).clone(), kv.k_scale.clone(), kv.v_scale.clone()]
    M = 4 * n
    q, k, v = (torch.randn(M, h * hd, device="cuda") for h in (H, Hkv, Hkv))
    q_out = torch.empty(M, H * hd, dtype=torch.bfloat16, device="cuda")
    ws = sb.workspace(256)
    sb.spec_kv8_append(cfg, kv, 0, n, q, k, v, sb.RopeTable(hd, THETA), q_out, ws)
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_KV_OVERFLOW | sb.DEV_BAD_PAGE)
    for pg in (1, 2, 3):  # sequence 0 alone was written to
        assert torch.equal(kv.k.view(torch.uint8)[0, pg], before[0][0, pg])
        assert torch.equal(kv.v.view(torch.uint8)[0, pg], before[1][0, pg])
        assert torch.equal(kv.k_scale[0, pg], before[2][0, pg])
    assert not torch.equal(kv.k.view(torch.uint8)[0, 0], before[0][0, 0])
    out = torch.full((M, H * hd), 5.0, dtype=torch.bfloat16, device="cuda")
    sb.spec_kv8_attention(cfg, kv, 0, n, torch.ones_like(out), out, ws)
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_KV_OVERFLOW | sb.DEV_BAD_PAGE)
    assert (out[:n] != 5.0).any(dim=1).all() and (out[n:] == 0).all()  # 5 is a value that a row can hold
    sb.spec_kv8_advance(kv, n, ws)
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_KV_OVERFLOW | sb.DEV_BAD_PAGE)
    assert kv.len.cpu().tolist() == [7, 126, 10, -1]
    # commit: a path out of order, a root below zero, a page outside the pool, and one that is fine
    snap = kv.k.view(torch.uint8).clone()
    path = torch.tensor([[2, 1, -1], [1, -1, -1], [1, -1, -1], [1, 2, -1]], dtype=torch.int32, device="cuda")
    kv.len.copy_(torch.tensor([7, 2, 10, 5], dtype=torch.int32))
    sb.spec_kv8_tree_commit(cfg, kv, path, torch.tensor([2, 1, 1, 2], dtype=torch.int32, device="cuda"), n, ws)
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_BAD_TREE | sb.DEV_KV_OVERFLOW | sb.DEV_BAD_PAGE)
    assert kv.len.cpu().tolist() == [7, 2, 10, 5]
    assert torch.equal(kv.k.view(torch.uint8), snap)  # the last one's path moves nothing
    sb.spec_kv8_truncate(kv, torch.tensor([0, 2, 1, 3], dtype=torch.int32, device="cuda"), 2, ws)
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_BAD_NACC)
    assert kv.len.cpu().tolist() == [5, 2, 9, 5]


def test_lengths_that_are_none():
    """Lengths below zero and past the capacity, some equal, in a batch that is put in order of length: those
    rows are zero, the other sequences are served."""
    cfg, n = _cfg("128x4/1"), 2
    lens = [5, -7, 1 << 30, 64, -(1 << 31), -7, (1 << 31) - 1, 0, -1, 126]
    kv = sb.KV8Cache(cfg, len(lens), 2 * len(lens), 2)
    for b in range(len(lens)):
        kv.reserve(b, 128)
    kv.sync()
    _fill(kv, 5)
    kv.len.copy_(torch.tensor(lens, dtype=torch.int32))
    q = _q(len(lens) * n, cfg.d_model, 37)
    ws = sb.workspace(256)
    out = torch.full_like(q, 3.0)
    sb.spec_kv8_attention(cfg, kv, 0, n, q, out, ws)
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_KV_OVERFLOW)
    one = sb.KV8Cache(cfg, 1, kv.n_pages, 2)
    one.k, one.v, one.k_scale, one.v_scale = kv.k, kv.v, kv.k_scale, kv.v_scale
    for b, L in enumerate(lens):
        got = out[b * n:(b + 1) * n]
        if not 0 <= L <= 128 - n:
            assert (got == 0).all()
            continue
        one.table.copy_(kv.table[b:b + 1])
        one.len.fill_(L)
        want = torch.empty_like(got)
        sb.spec_kv8_attention(cfg, one, 0, n, q[b * n:(b + 1) * n], want, ws)
        assert torch.equal(got, want)
    assert _status(ws) == (sb.SPEC_OK, 0)
    before = kv.k.view(torch.uint8).clone()
    R, q_out = sb.RopeTable(cfg.head_dim, THETA), torch.empty_like(q)
    k = _q(len(lens) * n, cfg.head_dim, 38)
    sb.spec_kv8_append(cfg, kv, 0, n, q, k, k, R, q_out, ws)
    sb.spec_kv8_advance(kv, n, ws)
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_KV_OVERFLOW)
    fits = [0 <= L <= 128 - n for L in lens]
    assert kv.len.cpu().tolist() == [L + n if f else L for L, f in zip(lens, fits)]
    for b in range(len(lens)):
        same = torch.equal(kv.k.view(torch.uint8)[0, kv.table[b].long()], before[0, kv.table[b].long()])
        assert same != fits[b]


def test_first_calls_inside_a_capture():
    """The set-up that a first call makes (attributes, cluster sizes) is allowed while a stream captures."""
    code = """
import sys
sys.path.insert(0, %r)
import torch
from speculative_decoding_verification_pass_gb300 import binding as sb
cfg = sb.ModelConfig(1, 512, 4, 1, 128, 1000)
kv = sb.KV8Cache(cfg, 1, 40, 40)
kv.reserve(0, 2560)
kv.sync()
kv.len.fill_(2000)
R, ws = sb.RopeTable(128, 1e4), sb.workspace(256)
q = torch.ones(3, 512, device='cuda', dtype=torch.bfloat16)
k = torch.ones(3, 128, device='cuda', dtype=torch.bfloat16)
q_out, o = torch.empty_like(q), torch.zeros_like(q)
path, m = torch.tensor([[1, 2, -1]], dtype=torch.int32, device='cuda'), torch.tensor([2], dtype=torch.int32, device='cuda')
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    sb.spec_kv8_append(cfg, kv, 0, 3, q, k, k, R, q_out, ws)
    sb.spec_kv8_attention(cfg, kv, 0, 3, q_out, o, ws)
    sb.spec_kv8_advance(kv, 3, ws)
    sb.spec_kv8_tree_commit(cfg, kv, path, m, 3, ws)
g.replay()
torch.cuda.synchronize()
assert sb.spec_device_status(ws) == (sb.SPEC_OK, 0) and kv.len.tolist() == [2003] and (o > 0).all()
print("captured")
""" % ROOT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_refused_tensors():
    cfg = _cfg("64x4/2")
    kv = sb.KV8Cache(cfg, 1, 1, 1)
    ws = sb.workspace(256)
    q = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    bad = [dict(q=q.float()), dict(q=q[:1]), dict(q=q.t()), dict(q=q.cpu()), dict(out=q[:, :128]),
           dict(anc=torch.zeros(1, 2, dtype=torch.int32, device="cuda")),
           dict(anc=torch.zeros(1, 3, dtype=torch.int64, device="cuda"))]
    for kw in bad:
        with pytest.raises(ValueError):
            sb.spec_kv8_attention(cfg, kv, 0, 2, **dict(dict(q=q, out=torch.empty_like(q), ws=ws), **kw))
    odd = torch.zeros(2, 260, dtype=torch.bfloat16, device="cuda")[:, 1:257]  # rows off 16 bytes
    for kw in (dict(q=odd), dict(out=odd), dict(scale=-1.0), dict(scale=float("nan"))):
        with pytest.raises(sb.SpecError) as e:
            sb.spec_kv8_attention(cfg, kv, 0, 2, **dict(dict(q=q, out=torch.empty_like(q), ws=ws), **kw))
        assert e.value.status == sb.SPEC_EINVAL
    R = sb.RopeTable(64, THETA)
    k = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):  # k of another type than q
        sb.spec_kv8_append(cfg, kv, 0, 2, q, k.float(), k, R, torch.empty_like(q), ws)
    with pytest.raises(ValueError):
        sb.spec_kv8_append(cfg, kv, 0, 2, q, k, k, R, torch.empty_like(q), ws, depth=torch.zeros(1, 2, device="cuda"))


# ------------------------------------------------------------ run together
def _round_trip(cfg, kv, steps, R, ws, stream=None):
    """Chain rounds on one layer: append, attention, advance, truncate; the outputs."""
    outs = []
    for q, k, v, keep in steps:
        n = q.shape[0] // kv.batch
        q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        o = torch.empty_like(q_out)
        sb.spec_kv8_append(cfg, kv, 0, n, q, k, v, R, q_out, ws, stream=stream)
        sb.spec_kv8_attention(cfg, kv, 0, n, q_out, o, ws, stream=stream)
        sb.spec_kv8_advance(kv, n, ws, stream=stream)
        sb.spec_kv8_truncate(kv, keep, n - 1, ws, stream=stream)
        outs += [q_out, o]
    return outs


def _steps(cfg, B, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    hd, H, Hkv = cfg.head_dim, cfg.n_heads, cfg.n_kv_heads
    steps = []
    for n in (40, 5, 5, 1, 7):
        r = [torch.randn(B * n, h * hd, generator=g).to(dtype).cuda() for h in (H, Hkv, Hkv)]
        keep = torch.randint(0, n, (B,), generator=g, dtype=torch.int32).cuda()
        steps.append((*r, keep))
    return steps


def test_rounds_against_the_oracle():
    """Rounds with rollbacks into the middle of blocks: the cache and the outputs follow the oracle's."""
    cfg, B = _cfg("128x4/1"), 3
    kv = sb.KV8Cache(cfg, B, 2 * B, 2)
    for b in range(B):
        kv.reserve(b, 128)
    kv.sync()
    table = kv.host_table()
    hd, H, Hkv = cfg.head_dim, cfg.n_heads, cfg.n_kv_heads
    R, ws = sb.RopeTable(hd, THETA), sb.workspace(256)
    lens = [0] * B
    for step in _steps(cfg, B, 51):
        q_out, o = _round_trip(cfg, kv, [step], R, ws)
        n = q_out.shape[0] // B
        P = Pair.__new__(Pair)
        P.cfg, P.kv, P.table, P.lens, P.B = cfg, kv, table, list(lens), B
        P.rows = {}
        for b in range(B):
            for name, x in (("k", step[1]), ("v", step[2])):
                code, scale = P.got(0, b, name)
                r = O8.Rows(Hkv, 128, hd)
                r.code, r.scale = code, scale
                P.rows[0, b, name] = r
                s = np.repeat(scale, 16, axis=1)[:, lens[b]:lens[b] + n, None]
                if name == "v":  # the rows just written, at a scale that rollbacks may have left larger
                    want = x[b * n:(b + 1) * n].double().cpu().numpy().reshape(n, Hkv, hd).transpose(1, 0, 2)
                    got = code[:, lens[b]:lens[b] + n] * s
                    assert (np.abs(got - want) <= np.maximum(np.abs(want) / 16, s / 1024)).all()
        _check_attention(cfg, P, n, q_out, o, [_chain(n)] * B, hd ** -0.5)
        lens = [L + 1 + int(k) for L, k in zip(lens, step[3].cpu())]
        assert kv.len.cpu().tolist() == lens
    assert _status(ws) == (sb.SPEC_OK, 0)


def test_other_stream_and_graph():
    """The same rounds on a side stream, and captured in a graph and replayed twice, give the same bits."""
    cfg, B = _cfg("64x4/2"), 2
    R, ws = sb.RopeTable(cfg.head_dim, THETA), sb.workspace(256)
    steps = _steps(cfg, B, 52, torch.bfloat16)

    def cache():
        kv = sb.KV8Cache(cfg, B, 2 * B, 2)
        for b in range(B):
            kv.reserve(b, 128)
        kv.sync()
        return kv

    kv = cache()
    want = _round_trip(cfg, kv, steps, R, ws)
    s = torch.cuda.Stream()
    kv2 = cache()
    s.wait_stream(torch.cuda.current_stream())
    got = _round_trip(cfg, kv2, steps, R, ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    kv3 = cache()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _round_trip(cfg, kv3, steps, R, ws)
    for _ in range(2):
        kv3.len.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
    assert torch.equal(kv.k.view(torch.uint8), kv3.k.view(torch.uint8))
    assert _status(ws) == (sb.SPEC_OK, 0)


def _fill(kv, seed):
    """Codes that are numbers and scales near those of unit rows in every page."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for x, s in ((kv.k, kv.k_scale), (kv.v, kv.v_scale)):
        bits = x.view(torch.uint8)
        bits.random_(0, 256, generator=g)
        bits[(bits & 0x7F) == 0x7F] = 0x31
        s.copy_(torch.exp2(torch.randint(-9, -6, s.shape, generator=g, device="cuda").float()))


@pytest.mark.parametrize("B,top,n", [(100, 300, 2), (40, 1500, 5), (13, 4000, 3), (2, 3000, 5), (96, 40, 1)])
def test_attention_of_many_sequences(B, top, n):
    """Batches on either side of the ordering by length, with lengths far apart: every sequence gets what
    it gets alone, but for the order in which its tiles are summed."""
    cfg = _cfg("64x16/2")
    rng = np.random.default_rng(B)
    lens = rng.integers(0, top, B)
    lens[:: 7] //= 50
    lens[0], lens[-1] = 0, top
    pages = [(int(x) + n + 63) // 64 for x in lens]
    kv = sb.KV8Cache(cfg, B, sum(pages), max(pages))
    for b in rng.permutation(B):
        kv.reserve(int(b), int(lens[b]) + n)
    kv.sync()
    _fill(kv, B)
    kv.len.copy_(_dev(lens.astype(np.int32)))
    q = _q(B * n, cfg.d_model, 61)
    ws = sb.workspace(256)
    out = torch.empty_like(q)
    sb.spec_kv8_attention(cfg, kv, 0, n, q, out, ws)
    one = sb.KV8Cache(cfg, 1, kv.n_pages, kv.max_pages)
    one.k, one.v, one.k_scale, one.v_scale = kv.k, kv.v, kv.k_scale, kv.v_scale
    for b in range(B):
        one.table.copy_(kv.table[b:b + 1])
        one.len.fill_(int(lens[b]))
        want = torch.empty(n, cfg.d_model, dtype=torch.bfloat16, device="cuda")
        sb.spec_kv8_attention(cfg, one, 0, n, q[b * n:(b + 1) * n], want, ws)
        got = out[b * n:(b + 1) * n]
        # each side rounds once (half a step each: a whole one between them), its weights 2^-11 of the values
        lim = 2.0 ** -7 * want.float().abs() + 2.0 ** -9 * want.float().abs().max()
        assert ((got.float() - want.float()).abs() <= lim).all(), (b, int(lens[b]))
    assert _status(ws) == (sb.SPEC_OK, 0)


def test_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of one layer: the same rows there and at the start of a small pool."""
    cfg, n, L = _cfg("128x8/8", 2), 5, 300
    many = 70000  # x 8 heads x 64 x 128 bytes = 4.6 GB a layer and side, the second layer past 2^32 from its start
    H, hd, Hkv = cfg.n_heads, cfg.head_dim, cfg.n_kv_heads
    small = sb.KV8Cache(cfg, 1, 8, 6)
    big = sb.KV8Cache(cfg, 1, many, 6)
    _fill(small, 3)
    ids = torch.tensor([[5, 1, 7, 0, 2, 3]], dtype=torch.int32)
    far = ids + many - 8
    small.table.copy_(ids)
    big.table.copy_(far)
    for name in ("k", "v", "k_scale", "v_scale"):
        x, y = getattr(small, name), getattr(big, name)
        y.view(torch.uint8)[:, many - 8:] = x.view(torch.uint8)
    R, ws = sb.RopeTable(hd, THETA), sb.workspace(256)
    q, k, v = (_q(n, h * hd, 70 + i) for i, h in enumerate((H, Hkv, Hkv)))
    res = []
    for kv in (small, big):
        kv.len.fill_(L)
        for layer in range(2):
            q_out, o = torch.empty_like(q), torch.empty_like(q)
            sb.spec_kv8_append(cfg, kv, layer, n, q, k, v, R, q_out, ws)
            sb.spec_kv8_attention(cfg, kv, layer, n, q_out, o, ws)
            res.append(o)
        sb.spec_kv8_advance(kv, n, ws)
        path = torch.tensor([[2, 4, -1, -1, -1]], dtype=torch.int32, device="cuda")
        sb.spec_kv8_tree_commit(cfg, kv, path, torch.tensor([2], dtype=torch.int32, device="cuda"), n, ws)
    assert _status(ws) == (sb.SPEC_OK, 0)
    assert torch.equal(res[0], res[2]) and torch.equal(res[1], res[3]) and not torch.equal(res[0], res[1])
    for name in ("k", "v", "k_scale", "v_scale"):
        x, y = getattr(small, name).view(torch.uint8), getattr(big, name).view(torch.uint8)
        assert torch.equal(x, y[:, many - 8:])
        assert not y[0, :64].any() if name in "kv" else True


def test_two_streams_at_once():
    """Two caches worked on by two streams at the same time, one workspace each."""
    cfg, B = _cfg("128x4/1"), 3
    R = sb.RopeTable(cfg.head_dim, THETA)

    def cache():
        kv = sb.KV8Cache(cfg, B, 2 * B, 2)
        for b in range(B):
            kv.reserve(b, 128)
        kv.sync()
        return kv

    steps = [_steps(cfg, B, s) for s in (81, 82)]
    want = [_round_trip(cfg, cache(), st, R, sb.workspace(256)) for st in steps]
    kvs, wss = [cache() for _ in range(2)], [sb.workspace(256) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(len(steps[0])):
        for k in range(2):
            got[k] += _round_trip(cfg, kvs[k], [steps[k][i]], R, wss[k], stream=streams[k])
    torch.cuda.synchronize()
    for a, b in zip(want[0] + want[1], got[0] + got[1]):
        assert torch.equal(a, b)
    for ws in wss:
        assert _status(ws) == (sb.SPEC_OK, 0)


def test_tree_round_against_the_oracle():
    """Append of a tree at its depths, its attention, the commit, and the next chain round."""
    cfg, n, lens = _cfg("64x4/2"), 11, (13, 60, 0)
    hd, H, Hkv, B = cfg.head_dim, cfg.n_heads, cfg.n_kv_heads, 3
    P = Pair(cfg, lens, n + 8, 27)
    R, ws = sb.RopeTable(hd, THETA), sb.workspace(256)
    masks, depth = zip(*(sb.spec_tree_masks(wl.random_tree(90 + b, n)) for b in range(B)))
    anc = _dev(np.array(masks, np.uint64).astype(np.int64))
    dep = _dev(np.array(depth, np.int32))
    g = torch.Generator().manual_seed(91)
    q, k, v = (torch.randn(B * n, h * hd, generator=g) for h in (H, Hkv, Hkv))
    q_out = torch.empty(B * n, H * hd, dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(q_out)
    sb.spec_kv8_append(cfg, P.kv, 0, n, q.cuda(), k.cuda(), v.cuda(), R, q_out, ws, depth=dep)
    sb.spec_kv8_attention(cfg, P.kv, 0, n, q_out, o, ws, anc=anc)
    freq = O8.frequencies(hd, THETA)
    for b, L in enumerate(lens):
        for j in range(n):
            m = b * n + j
            want = O8.rotate(q[m].double().numpy().reshape(H, hd), L + depth[b][j], freq, False)
            got = q_out[m].double().cpu().numpy().reshape(H, hd)
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18).all()
        for name, x in (("k", k), ("v", v)):  # from here on the rows that the device holds
            new = x[b * n:(b + 1) * n].double().numpy().reshape(n, Hkv, hd)
            want = P.rows[0, b, name]
            want.append(L, new)
            code, scale = P.got(0, b, name)
            if name == "v":
                np.testing.assert_array_equal(code[:, :L + n], want.code[:, :L + n])
                np.testing.assert_array_equal(scale[:, : (L + n + 15) // 16], want.scale[:, : (L + n + 15) // 16])
            want.code, want.scale = code, scale
    see = [np.array([[(m >> i) & 1 for i in range(n)] for m in masks[b]], bool) for b in range(B)]
    _check_attention(cfg, P, n, q_out, o, see, hd ** -0.5)
    sb.spec_kv8_advance(P.kv, n, ws)
    path = np.full((B, n), -1, np.int32)
    paths = []
    for b in range(B):  # root-to-node path of the last node
        m = masks[b][n - 1]
        paths.append([i for i in range(1, n) if (m >> i) & 1])
        path[b, :len(paths[b])] = paths[b]
    sb.spec_kv8_tree_commit(cfg, P.kv, _dev(path), _dev(np.array([len(p) for p in paths], np.int32)), n, ws)
    for b, L in enumerate(lens):
        for name in "kv":
            P.rows[0, b, name].commit(L, paths[b])
            code, scale = P.got(0, b, name)
            np.testing.assert_array_equal(code, P.rows[0, b, name].code)
            np.testing.assert_array_equal(scale, P.rows[0, b, name].scale)
    P.lens = [L + 1 + len(p) for L, p in zip(lens, paths)]
    assert P.kv.len.cpu().tolist() == P.lens
    q2 = _q(B * 4, H * hd, 92)
    out, _ = _run_attention(cfg, P, 4, q2, ws=ws)
    _check_attention(cfg, P, 4, q2, out, [_chain(4)] * B, hd ** -0.5)
    assert _status(ws) == (sb.SPEC_OK, 0)


def test_refused_caches():
    cfg = _cfg("64x4/2")
    kv = sb.KV8Cache(cfg, 2, 4, 2)
    for name, bad in (("k", kv.k[:, :3]), ("k", kv.k.view(torch.uint8)), ("k_scale", kv.k_scale.double()),
                      ("len", kv.len.long()), ("table", kv.table.t()), ("len", kv.len.cpu())):
        with pytest.raises(ValueError):
            setattr(kv, name, bad)
    ws = sb.workspace(256)
    q = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):  # the cache of another shape
        sb.spec_kv8_attention(_cfg("64x4/2", 2), kv, 0, 2, q, q.clone(), ws)
    with pytest.raises(ValueError):
        sb.spec_kv8_attention(cfg, kv, 0, 2, q, q.clone(), ws[:0])
    with pytest.raises(sb.SpecError) as e:
        sb.spec_kv8_attention(cfg, kv, 1, 2, q, q.clone(), ws)
    assert e.value.status == sb.SPEC_EINVAL


def test_attention_in_place():
    """The output may be the queries' own rows."""
    cfg, n, lens = _cfg("128x4/1"), 9, (700, 3)
    P = Pair(cfg, lens, n, 28)
    q = _q(len(lens) * n, cfg.d_model, 36)
    want, ws = _run_attention(cfg, P, n, q)
    sb.spec_kv8_attention(cfg, P.kv, 0, n, q, q, ws)
    assert torch.equal(q, want)


@pytest.mark.parametrize("rope", ["half", "inter-part-scaled"])
def test_append_in_place(rope):
    """The rotated queries may take the queries' own rows."""
    cfg, n, lens = _cfg("128x4/1"), 9, (700, 3)
    g = torch.Generator().manual_seed(51)
    q, k, v = (torch.randn(len(lens) * n, w, generator=g).to(torch.bfloat16).cuda()
               for w in (cfg.d_model, cfg.head_dim, cfg.head_dim))
    how = ROPES[rope]
    R = sb.RopeTable(64 if how.get("part") else 128, THETA, how["inter"], how.get("factor", 1.0))
    want, ws = torch.empty_like(q), sb.workspace(256)
    a, b = Pair(cfg, lens, n, 52), Pair(cfg, lens, n, 52)
    sb.spec_kv8_append(cfg, a.kv, 0, n, q, k, v, R, want, ws)
    sb.spec_kv8_append(cfg, b.kv, 0, n, q, k, v, R, q, ws)
    assert torch.equal(q, want) and torch.equal(a.kv.k.view(torch.uint8), b.kv.k.view(torch.uint8))
    assert _status(ws) == (sb.SPEC_OK, 0)


def test_advance_looks_at_every_page():
    """Lengths move on by themselves: a page id out of the pool anywhere below the new length, a length that
    does not fit, or none of these, in one batch."""
    cfg = _cfg("64x4/2")
    kv, ws = sb.KV8Cache(cfg, 6, 4, 300), sb.workspace(256)
    lens = [0, 19136, 19195, -1, 6000, 2 ** 31 - 1]  # the third fits to the last slot
    table = torch.zeros(6, 300, dtype=torch.int32)
    table[0, 1:] = -1  # not looked at
    table[4, 70] = 4  # one past the pool, in the third group of pages
    kv.table.copy_(table)
    kv.len.copy_(torch.tensor(lens, dtype=torch.int32))
    sb.spec_kv8_advance(kv, 5, ws)
    assert kv.len.cpu().tolist() == [5, 19141, 19200, -1, 6000, 2 ** 31 - 1]
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_BAD_PAGE | sb.DEV_KV_OVERFLOW)
    kv.len.copy_(torch.tensor([60, 19196, 1, 1, 4475, 1], dtype=torch.int32))
    sb.spec_kv8_advance(kv, 5, ws)  # the first's second page is none now; 4480 slots end before page 70
    assert kv.len.cpu().tolist() == [60, 19196, 6, 6, 4480, 6]


# Large capacities (a table of WIDE columns) take calls of more than 64 rows a KV head to the kernel for many rows.
WIDE = 1400


@pytest.mark.parametrize("heads,lens,n", [
    ("128x4/1", (40000,), 5),
    ("128x4/1", (9000, 11), 2),
    ("64x4/2", (30000,), 7),
    ("128x8/8", (20000,), 1),
    ("64x16/2", (5000, 126, 0), 4),
    ("128x6/2", (3000, 7000), 9),
    ("128x4/1", (0, 1, 63, 127, 128, 250, 700, 2000), 8),
    ("64x4/2", (100, 0, 64), 12),
    ("128x8/8", (60000,), 5),  # runs of 39 tiles
])
def test_attention_long_capacity(heads, lens, n):
    """Few sequences in a large capacity: a CTA has an SM to itself and takes its tiles in two groups; runs of
    one tile and of many."""
    cfg = _cfg(heads)
    P = Pair(cfg, lens, n + 40, 91, columns=WIDE)
    _stale(P, n)
    q = _q(len(lens) * n, cfg.d_model, 92)
    out, ws = _run_attention(cfg, P, n, q)
    assert _status(ws) == (sb.SPEC_OK, 0)
    _check_attention(cfg, P, n, q, out, [_chain(n)] * len(lens), cfg.head_dim ** -0.5)
    for _ in range(10):  # launches that overlap; the same bits
        again = torch.empty_like(out)
        sb.spec_kv8_attention(cfg, P.kv, 0, n, q, again, ws)
        assert torch.equal(again, out)


@pytest.mark.parametrize("heads,lens,n", [("128x4/1", (0, 100, 2500), 13), ("64x4/2", (0, 1250), 30)])
def test_attention_long_capacity_tree(heads, lens, n):
    cfg = _cfg(heads)
    P = Pair(cfg, lens, n + 40, 93, columns=WIDE)
    # later keys larger: what is summed is scaled on the way
    P.scales["k"][0, P.table[-1, 9:][P.table[-1, 9:] >= 0]] *= 8
    P.put_bits("k")
    P.rows[0, len(lens) - 1, "k"] = P._oracle_rows(0, len(lens) - 1, "k", cfg.n_kv_heads, cfg.head_dim)
    _stale(P, n)
    q = _q(len(lens) * n, cfg.d_model, 94, size=4.0)
    see, anc = [], []
    for b in range(len(lens)):
        masks, _ = sb.spec_tree_masks(wl.random_tree(90 + b, n))
        masks[0] = 0
        see.append(np.array([[(m >> i) & 1 for i in range(n)] for m in masks], bool))
        anc.append(masks)
    out, ws = _run_attention(cfg, P, n, q, anc=_dev(np.array(anc, np.uint64).astype(np.int64)))
    assert _status(ws) == (sb.SPEC_OK, 0)
    _check_attention(cfg, P, n, q, out, see, cfg.head_dim ** -0.5)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("heads", ["128x4/1", "64x4/2"])
def test_attention_long_capacity_not_numbers(heads):
    cfg, n, lens = _cfg(heads), 6, (70, 1200)
    H, hd, Hkv = cfg.n_heads, cfg.head_dim, cfg.n_kv_heads
    G = H // Hkv
    q = _q(len(lens) * n, H * hd, 95)
    ref, _ = _run_attention(cfg, Pair(cfg, lens, n + 30, 96, columns=WIDE), n, q)
    want = ref.view(len(lens), n, H, hd)
    last = slice((Hkv - 1) * G, H)
    for name, b, slot, dim in (("v", 0, 70 + 3, 9), ("v", 1, 1200 + 3, hd - 1), ("k", 0, 70 + 3, 1), ("v", 1, 20, 3),
                               ("k", 1, 1199, 0)):
        P = Pair(cfg, lens, n + 30, 96, columns=WIDE)
        P.bits[name][0, P.table[b, slot // 64], Hkv - 1, slot % 64, dim] = 0xFF
        P.put_bits(name)
        out, _ = _run_attention(cfg, P, n, q)
        out = out.view(len(lens), n, H, hd)
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        j0 = max(0, slot - lens[b])
        if name == "v":
            hit[b, j0:, last, dim] = True
        else:
            hit[b, j0:, last, :] = True
        assert torch.equal(torch.isnan(out), hit), (name, b, slot)
        assert torch.equal(out[~hit], want[~hit])
    P = Pair(cfg, lens, n + 30, 96, columns=WIDE)
    for at, bit in ((-1, sb.DEV_KV_OVERFLOW), (64 * WIDE - n + 1, sb.DEV_KV_OVERFLOW), (1400, sb.DEV_BAD_PAGE)):
        P.kv.len[1] = at
        out, ws = _run_attention(cfg, P, n, q)
        assert _status(ws) == (sb.SPEC_EDEVICE, bit)
        assert torch.equal(out[:n], ref[:n]) and (out[n:] == 0).all()


@pytest.mark.parametrize("heads,lens,n", [
    ("128x4/1", (0, 77, 300, 1, 640), 128),
    ("128x4/1", (0, 3, 59, 123, 124, 250, 700), 17),
    ("128x8/8", (130, 0), 65),
    ("64x4/2", (5, 190, 62), 33),
    ("64x16/2", (2000, 17), 9),
    ("64x16/2", (255, 0, 128), 100),
    ("128x6/2", (300, 1), 43),
    ("128x4/1", (5000,), 40),
    ("128x8/8", (12000, 3000, 100, 7000), 70),  # runs of 24 tiles: every ring turns over
])
def test_attention_many_rows(heads, lens, n):
    cfg = _cfg(heads)
    P = Pair(cfg, lens, n + 40, 71, columns=WIDE)
    _stale(P, n)
    q = _q(len(lens) * n, cfg.d_model, 72)
    out, ws = _run_attention(cfg, P, n, q)
    assert _status(ws) == (sb.SPEC_OK, 0)
    _check_attention(cfg, P, n, q, out, [_chain(n)] * len(lens), cfg.head_dim ** -0.5)


@pytest.mark.parametrize("heads,lens,n", [("128x4/1", (0, 100, 250), 17), ("64x4/2", (0, 125, 500), 64),
                                          ("64x16/2", (60, 1), 63), ("128x4/1", (1, 130), 64)])
def test_attention_many_rows_tree(heads, lens, n):
    cfg = _cfg(heads)
    P = Pair(cfg, lens, n + 40, 73, columns=WIDE)
    _stale(P, n)
    q = _q(len(lens) * n, cfg.d_model, 74)
    see, anc = [], []
    for b in range(len(lens)):
        masks, _ = sb.spec_tree_masks(wl.random_tree(80 + b, n))
        masks[0] = 0
        masks[n - 1] &= ~(1 << (n - 1))
        see.append(np.array([[(m >> i) & 1 for i in range(n)] for m in masks], bool))
        anc.append([m | (1 << n) if n < 63 else m for m in masks])
    out, ws = _run_attention(cfg, P, n, q, anc=_dev(np.array(anc, np.uint64).astype(np.int64)))
    assert _status(ws) == (sb.SPEC_OK, 0)
    _check_attention(cfg, P, n, q, out, see, cfg.head_dim ** -0.5)
    for b, L in enumerate(lens):
        if L == 0:
            assert (out[b * n] == 0).all()


def test_attention_many_rows_scale_strides_and_sharp_rows():
    """Also rows that start at scores far below the later ones, so that what is summed is scaled on the way."""
    cfg, n, lens = _cfg("128x4/1"), 30, (900, 70)
    P = Pair(cfg, lens, n, 75, columns=WIDE)
    P.scales["k"][0, P.table[0, 9:]] *= 8  # the later keys are the larger ones
    P.put_bits("k")
    for b in range(2):
        P.rows[0, b, "k"] = P._oracle_rows(0, b, "k", cfg.n_kv_heads, cfg.head_dim)
    wide = _q(len(lens) * n, cfg.d_model + 64, 76, size=8.0)
    q = wide[:, 64:]
    ow = torch.full((len(lens) * n, cfg.d_model + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = sb.workspace(256)
    sb.spec_kv8_attention(cfg, P.kv, 0, n, q, ow[:, :cfg.d_model], ws, scale=0.5)
    assert (ow[:, cfg.d_model:] == 3.0).all()
    _check_attention(cfg, P, n, q, ow[:, :cfg.d_model], [_chain(n)] * 2, 0.5)
    # in place: the output may be the queries' own rows
    q = q.contiguous()
    sb.spec_kv8_attention(cfg, P.kv, 0, n, q, q, ws, scale=0.5)
    assert torch.equal(q, ow[:, :cfg.d_model])


@pytest.mark.parametrize("name,top", [("v", 2.0 ** 30), ("v", 0.0), ("k", 0.0)])
def test_attention_many_rows_uneven_scales(name, top):
    cfg, n, lens = _cfg("128x4/1"), 20, (300, 40)
    P = Pair(cfg, lens, n, 77, columns=WIDE)
    pg = P.table[0, 2]
    if top:
        P.scales[name][0, pg] *= top
    else:
        P.bits[name][0, pg] = 0
        P.scales[name][0, pg] = 2.0 ** -40
    P.put_bits(name)
    for b in range(2):
        for nm in "kv":
            P.rows[0, b, nm] = P._oracle_rows(0, b, nm, cfg.n_kv_heads, cfg.head_dim)
    q = _q(len(lens) * n, cfg.d_model, 78)
    out, _ = _run_attention(cfg, P, n, q)
    _check_attention(cfg, P, n, q, out, [_chain(n)] * 2, cfg.head_dim ** -0.5)


@pytest.mark.parametrize("heads", ["128x4/1", "64x4/2"])
def test_attention_many_rows_not_numbers(heads):
    """As in test_attention_not_numbers; and sequences that do not fit get zero rows."""
    cfg, n, lens = _cfg(heads), 40, (70, 200)
    H, hd, Hkv = cfg.n_heads, cfg.head_dim, cfg.n_kv_heads
    G = H // Hkv
    q = _q(len(lens) * n, H * hd, 79)
    ref, _ = _run_attention(cfg, Pair(cfg, lens, n + 30, 80, columns=WIDE), n, q)
    want = ref.view(len(lens), n, H, hd)
    last = slice((Hkv - 1) * G, H)
    for name, b, slot, dim in (("v", 0, 70 + 3, 9), ("v", 1, 200 + 3, hd - 1), ("k", 0, 70 + 3, 1), ("v", 1, 20, 3),
                               ("k", 1, 199, 0), ("v", 1, 239, 33)):
        P = Pair(cfg, lens, n + 30, 80, columns=WIDE)
        P.bits[name][0, P.table[b, slot // 64], Hkv - 1, slot % 64, dim] = 0xFF
        P.put_bits(name)
        out, _ = _run_attention(cfg, P, n, q)
        out = out.view(len(lens), n, H, hd)
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        j0 = max(0, slot - lens[b])
        if name == "v":
            hit[b, j0:, last, dim] = True
        else:
            hit[b, j0:, last, :] = True
        assert torch.equal(torch.isnan(out), hit), (name, b, slot)
        assert torch.equal(out[~hit], want[~hit])
    for bad in (float("inf"), -float("inf"), float("nan")):
        q2 = q.clone()
        q2[n + 2, hd + 5] = bad
        out, _ = _run_attention(cfg, Pair(cfg, lens, n + 30, 80, columns=WIDE), n, q2)
        out = out.view(len(lens), n, H, hd)
        assert torch.isnan(out[1, 2, 1]).all()
        keep = torch.ones(out.shape[:3], dtype=torch.bool)
        keep[1, 2, 1] = False
        assert torch.equal(out[keep.cuda()], want[keep.cuda()])
    P = Pair(cfg, lens, n + 30, 80, columns=WIDE)
    for at, bit in ((-1, sb.DEV_KV_OVERFLOW), (64 * WIDE - n + 1, sb.DEV_KV_OVERFLOW), (400, sb.DEV_BAD_PAGE)):
        P.kv.len[1] = at  # slots 400 .. 439 lie on no page
        out, ws = _run_attention(cfg, P, n, q)
        assert _status(ws) == (sb.SPEC_EDEVICE, bit)
        assert torch.equal(out[:n], ref[:n]) and (out[n:] == 0).all()


def test_attention_many_rows_streams_and_graph():
    """Two calls at once on two streams, of few and of many rows, and a captured one replayed: the same bits."""
    cfg, lens, n = _cfg("64x4/2"), (900, 300, 1500), 128
    P = Pair(cfg, lens, n, 81, columns=WIDE)
    q = _q(len(lens) * n, cfg.d_model, 82)
    want, ws = _run_attention(cfg, P, n, q)
    few, wsf = _run_attention(cfg, P, 5, q[:15])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(want) for _ in range(2)] + [torch.empty_like(few)]
    for _ in range(20):
        for s, o in zip(streams, outs):
            sb.spec_kv8_attention(cfg, P.kv, 0, o.shape[0] // 3, q[:o.shape[0]], o, wsf, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(outs[2], few)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        for _ in range(3):
            sb.spec_kv8_attention(cfg, P.kv, 0, n, q, out, ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert _status(ws) == (sb.SPEC_OK, 0) and _status(wsf) == (sb.SPEC_OK, 0)


def test_attention_many_rows_of_many_sequences():
    """Batches on either side of the ordering by length: every sequence as alone, but for the order of its sums."""
    cfg, n = _cfg("64x16/2"), 10
    for B, top in ((100, 300), (13, 3000)):
        rng = np.random.default_rng(B)
        lens = rng.integers(0, top, B)
        lens[0], lens[-1] = 0, top
        pages = [(int(x) + n + 63) // 64 for x in lens]
        kv = sb.KV8Cache(cfg, B, sum(pages), WIDE)
        for b in range(B):
            kv.reserve(b, int(lens[b]) + n)
        kv.sync()
        _fill(kv, B)
        kv.len.copy_(_dev(lens.astype(np.int32)))
        q, ws = _q(B * n, cfg.d_model, 83), sb.workspace(256)
        out = torch.empty_like(q)
        sb.spec_kv8_attention(cfg, kv, 0, n, q, out, ws)
        one = sb.KV8Cache(cfg, 1, kv.n_pages, WIDE)
        one.k, one.v, one.k_scale, one.v_scale = kv.k, kv.v, kv.k_scale, kv.v_scale
        for b in range(B):
            one.table.copy_(kv.table[b:b + 1])
            one.len.fill_(int(lens[b]))
            want = torch.empty(n, cfg.d_model, dtype=torch.bfloat16, device="cuda")
            sb.spec_kv8_attention(cfg, one, 0, n, q[b * n:(b + 1) * n], want, ws)
            got = out[b * n:(b + 1) * n]
            # each side rounds once (half a step each: a whole one between them), its weights 2^-11 of the values
            lim = 2.0 ** -7 * want.float().abs() + 2.0 ** -9 * want.float().abs().max()
            assert ((got.float() - want.float()).abs() <= lim).all(), (b, int(lens[b]))
        assert _status(ws) == (sb.SPEC_OK, 0)


# ------------------------------------------------------------------ forward
class Kv8State(OM.KVState):
    """The oracle's cache with rows held in 8 bits (keep() rounds the new rows in place)."""

    def __init__(self, cfg, batch, capacity):
        super().__init__(cfg, batch, capacity)
        self.rows = {(l, b, i): O8.Rows(cfg.n_kv_heads, capacity, cfg.head_dim)
                     for l in range(cfg.n_layers) for b in range(batch) for i in range(2)}

    def keep(self, l, b, K, V, start, n):
        for i, x in enumerate((K, V)):
            r = self.rows[l, b, i]
            r.append(start, x[:, start:start + n].transpose(1, 0, 2))
            x[:, :start + n] = r.value(start + n)


@pytest.mark.parametrize("shape", [(2, 256, 4, 2, 256, 1000), (2, 512, 4, 1, 384, 4099)])
def test_forward_on_the_8_bit_cache(shape):
    """Passes with rollbacks against the oracle's forward on rows rounded alike, |d| <= 1e-2 (1 + |logit|)."""
    cfg = sb.ModelConfig(*shape)
    B, seed, cap = 3, 44, 192
    m = sb.Model(cfg, seed)
    kv = sb.KV8Cache(cfg, B, 3 * B, 3)
    ocfg = OM.Config(*shape, cfg.rms_eps, cfg.rope_theta)
    W = OW.Weights(ocfg, seed)
    okv = Kv8State(ocfg, B, cap)
    ws = sb.workspace(sb.spec_kv8_workspace_bytes(cfg, B, 40))
    lens = np.zeros(B, np.int64)
    for n, keep in ((40, (39, 39, 39)), (7, (3, 0, 6)), (5, (4, 1, 2)), (1, (0, 0, 0))):
        toks = wl.tokens(seed + n, B, n, cfg.vocab)
        for b in range(B):
            kv.reserve(b, int(lens[b]) + n)
        kv.sync()
        z = torch.empty(B, n, cfg.vocab, device="cuda")
        sb.spec_verify_forward_kv8(m.handle, _dev(toks), B, n, kv, z, ws)
        ref = OM.forward(ocfg, W, toks, okv, round_kv=False)
        got = z.double().cpu().numpy()
        err = np.abs(got - ref) / (1 + np.abs(ref))
        assert err.max() <= 1e-2, err.max()
        sb.spec_kv8_truncate(kv, _dev(np.array(keep, np.int32)), n - 1, ws)
        okv.lens -= n - 1 - np.array(keep)
        lens = okv.lens.copy()
        for b in range(B):
            kv.release(b, int(lens[b]))
        assert kv.len.cpu().tolist() == lens.tolist()
    assert _status(ws) == (sb.SPEC_OK, 0)
    m.close()


def test_forward_tree_equals_chain_and_commits():
    """A chain given as a tree gives the chain's bits; a branching tree's accepted path then goes on as
    the chain of the same tokens would (same rows, rounded once more at most)."""
    shape = (2, 256, 4, 2, 256, 1000)
    cfg, B, seed, n = sb.ModelConfig(*shape), 2, 45, 6
    m = sb.Model(cfg, seed)
    ws = sb.workspace(sb.spec_kv8_workspace_bytes(cfg, B, 32))

    def fresh():
        kv = sb.KV8Cache(cfg, B, 2 * B, 2)
        for b in range(B):
            kv.reserve(b, 128)
        kv.sync()
        z = torch.empty(B, 32, cfg.vocab, device="cuda")
        sb.spec_verify_forward_kv8(m.handle, _dev(wl.tokens(seed, B, 32, cfg.vocab)), B, 32, kv, z, ws)
        return kv

    toks = wl.tokens(seed + 1, B, n, cfg.vocab)
    za, zb = (torch.empty(B, n, cfg.vocab, device="cuda") for _ in range(2))
    sb.spec_verify_forward_kv8(m.handle, _dev(toks), B, n, fresh(), za, ws)
    masks, depth = sb.spec_tree_masks([-1] + list(range(n - 1)))
    anc, dep = _dev(np.array([masks] * B, np.int64)), _dev(np.array([depth] * B, np.int32))
    sb.spec_verify_forward_kv8(m.handle, _dev(toks), B, n, fresh(), zb, ws, anc=anc, depth=dep)
    assert torch.equal(za, zb)
    # root, two children, the second child's chain: accept nodes 2, 4, 5
    parents = [-1, 0, 0, 1, 2, 4]
    masks, depth = sb.spec_tree_masks(parents)
    anc, dep = _dev(np.array([masks] * B, np.int64)), _dev(np.array([depth] * B, np.int32))
    kv = fresh()
    sb.spec_verify_forward_kv8(m.handle, _dev(toks), B, n, kv, zb, ws, anc=anc, depth=dep)
    path = _dev(np.array([[2, 4, 5, -1, -1, -1]] * B, np.int32))
    sb.spec_kv8_tree_commit(cfg, kv, path, _dev(np.array([3] * B, np.int32)), n, ws)
    assert kv.len.cpu().tolist() == [36, 36]
    chain = np.ascontiguousarray(toks[:, [0, 2, 4, 5]])
    kvc = fresh()
    zc = torch.empty(B, 4, cfg.vocab, device="cuda")
    sb.spec_verify_forward_kv8(m.handle, _dev(chain), B, 4, kvc, zc, ws)
    close = lambda a, b: ((a - b).abs() <= 1e-2 * (1 + b.abs())).all()
    assert close(zb[:, [0, 2, 4, 5]], zc)
    nxt = _dev(wl.tokens(seed + 2, B, 3, cfg.vocab))
    zt, zd = (torch.empty(B, 3, cfg.vocab, device="cuda") for _ in range(2))
    sb.spec_verify_forward_kv8(m.handle, nxt, B, 3, kv, zt, ws)
    sb.spec_verify_forward_kv8(m.handle, nxt, B, 3, kvc, zd, ws)
    assert close(zt, zd)
    assert _status(ws) == (sb.SPEC_OK, 0)
    m.close()


@pytest.mark.parametrize("n", [5, 64])
def test_forward_in_a_large_capacity(n):
    """A pass on caches of a small and of a large capacity, whose attention takes different kernels: the
    same logits but for rounding (a layer's codes may differ where a value lies on a border)."""
    cfg, B, seed = sb.ModelConfig(2, 256, 4, 2, 256, 1000), 2, 47
    m = sb.Model(cfg, seed)
    ws = sb.workspace(sb.spec_kv8_workspace_bytes(cfg, B, n))
    toks = _dev(wl.tokens(seed, B, n, cfg.vocab))
    out = []
    for pages in (3, WIDE):
        kv = sb.KV8Cache(cfg, B, 3 * B, pages)
        for b in range(B):
            kv.reserve(b, 3 * 64)
        kv.sync()
        z = torch.empty(2, B, n, cfg.vocab, device="cuda")
        for k in range(2):
            sb.spec_verify_forward_kv8(m.handle, toks, B, n, kv, z[k], ws)
        assert _status(ws) == (sb.SPEC_OK, 0) and kv.len.cpu().tolist() == [2 * n] * B
        out.append(z)
    assert ((out[0] - out[1]).abs() <= 1e-2 * (1 + out[0].abs())).all()
    m.close()


def test_forward_of_a_large_batch_and_refusals():
    """More than 128 token rows: each sequence as in a batch of its own; and what the pass refuses."""
    shape = (2, 256, 4, 2, 256, 1000)
    cfg, B, n, seed = sb.ModelConfig(*shape), 40, 5, 46
    m = sb.Model(cfg, seed)
    ws = sb.workspace(sb.spec_kv8_workspace_bytes(cfg, B, 12))
    lens = np.random.default_rng(4).integers(1, 12, B)
    toks = wl.tokens(seed, B, 12, cfg.vocab)
    new = wl.tokens(seed + 1, B, n, cfg.vocab)

    def run(rows):
        kv = sb.KV8Cache(cfg, len(rows), len(rows), 1)
        for i in range(len(rows)):
            kv.reserve(i, 64)
        kv.sync()
        z = torch.empty(len(rows), 12, cfg.vocab, device="cuda")
        sb.spec_verify_forward_kv8(m.handle, _dev(toks[rows]), len(rows), 12, kv, z, ws)
        kv.len.copy_(_dev(lens[rows].astype(np.int32)))  # sequences of different lengths
        z = torch.empty(len(rows), n, cfg.vocab, device="cuda")
        sb.spec_verify_forward_kv8(m.handle, _dev(new[rows]), len(rows), n, kv, z, ws)
        return z, kv

    z, kv = run(np.arange(B))
    assert kv.len.cpu().tolist() == (lens + n).tolist()
    for b in (0, 7, 39):
        want, _ = run(np.array([b]))
        assert ((z[b] - want[0]).abs() <= 1e-2 * (1 + want[0].abs())).all()
    assert _status(ws) == (sb.SPEC_OK, 0)
    # a sequence without room is flagged and keeps its length and rows
    kv.len[3] = 62
    before = kv.k.view(torch.uint8)[:, int(kv.table[3, 0])].clone()
    sb.spec_verify_forward_kv8(m.handle, _dev(new), B, n, kv, z, ws)
    assert _status(ws) == (sb.SPEC_EDEVICE, sb.DEV_KV_OVERFLOW)
    assert int(kv.len[3]) == 62 and torch.equal(kv.k.view(torch.uint8)[:, int(kv.table[3, 0])], before)
    for kw, status in ((dict(ws=ws[:4096]), sb.SPEC_ESIZE), (dict(n=13), sb.SPEC_ESIZE)):
        k = dict(dict(n=n, ws=ws), **kw)
        t = torch.zeros(B, k["n"], dtype=torch.int32, device="cuda")
        with pytest.raises(sb.SpecError) as e:
            sb.spec_verify_forward_kv8(m.handle, t, B, k["n"], kv, torch.empty(B, k["n"], cfg.vocab, device="cuda"), k["ws"])
        assert e.value.status == status
    for bad in (z[:, :4], z.half(), z[:39]):  # logits of another size or type
        with pytest.raises(ValueError):
            sb.spec_verify_forward_kv8(m.handle, _dev(new), B, n, kv, bad, ws)
    with pytest.raises(sb.SpecError) as e:  # a tree's masks without its depths
        sb.spec_verify_forward_kv8(m.handle, _dev(new), B, n, kv, z, ws,
                                   anc=torch.zeros(B, n, dtype=torch.int64, device="cuda"))
    assert e.value.status == sb.SPEC_EINVAL
    m.close()


def test_cache_of_given_buffers():
    """Codes and scales of the caller's own are the cache's, without a second allocation; others are refused."""
    cfg = sb.ModelConfig(2, 256, 4, 2, 256, 1000)
    B, pages = 2, 2000
    whole = torch.zeros(2, 2, pages, 2, 64, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.ones(2, 2, pages, 2, 4, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    given = dict(k=whole[0], v=whole[1], k_scale=scale[0], v_scale=scale[1])
    kv = sb.KV8Cache(cfg, B, pages, 3, **given)
    assert torch.cuda.max_memory_allocated() - before < 1 << 16
    assert all(getattr(kv, name).data_ptr() == t.data_ptr() for name, t in given.items())
    other = sb.KV8Cache(cfg, B, pages, 3, v=whole[1])
    assert other.v.data_ptr() == kv.v.data_ptr() and other.k.data_ptr() != kv.k.data_ptr()
    m = sb.Model(cfg, 48)
    ws = sb.workspace(sb.spec_kv8_workspace_bytes(cfg, B, 5))
    toks = _dev(wl.tokens(48, B, 5, cfg.vocab))
    z = torch.empty(2, B, 5, cfg.vocab, device="cuda")
    for c, out in ((kv, z[0]), (sb.KV8Cache(cfg, B, pages, 3), z[1])):
        for b in range(B):
            c.reserve(b, 64)
        c.sync()
        sb.spec_verify_forward_kv8(m.handle, toks, B, 5, c, out, ws)
    assert _status(ws) == (sb.SPEC_OK, 0) and torch.equal(z[0], z[1])
    assert (whole.view(torch.uint8) != 0).any()
    for bad in (dict(k=whole[0, :1]), dict(k=whole[0].view(torch.uint8)), dict(v=whole[1].cpu()),
                dict(k_scale=scale[0].double()), dict(v_scale=scale[:, 0].transpose(1, 2)), dict(k=whole[:, :, :, 0])):
        with pytest.raises(ValueError):
            sb.KV8Cache(cfg, B, pages, 3, **bad)
    m.close()
