"""Workloads of the 8-bit paged KV cache: append, attention, draft-tree commit.

Each case is one call of one operator as a serving loop makes it: the cache,
its page table and lengths, the rotary table and the workspace are kept
between calls (``prepare``), the call's inputs are device tensors.  ``run``
computes the operator either with the library's kernels (``own``) or in
elementary torch operations; ``exact`` gives the definition in 64 bits.

The cache holds e4m3 values with one power-of-two scale per block of 16 slots
and KV head; a cached row is (value in 8 bits) x (its block's scale).  The
state is returned as those 8-bit floating values and the scales.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
BLOCK = 16
E4M3 = torch.float8_e4m3fn
FMAX = 448.0
LO_EXP, HI_EXP = -40, 40


def listed():
    return [
        # one user's stream, draft depth 4, 8B-shaped heads: the smallest append of a decode step
        dict(name="append b1 n5", op="append", hd=128, H=32, Hkv=8, B=1, n=5, lo=2048, hi=2048, dtype="bf16",
             rd=128, inter=False, factor=1.0, orig=0, tree=False),
        # a full serving batch at draft depth 4, ragged contexts
        dict(name="append b64 n5", op="append", hd=128, H=32, Hkv=8, B=64, n=5, lo=512, hi=4096, dtype="bf16",
             rd=128, inter=False, factor=1.0, orig=0, tree=False),
        # a prefill chunk of four prompts at far positions, fp32 projections, interleaved partial rotary
        # with the frequencies scaled for long contexts, head dim 64
        dict(name="append prefill b4 n128", op="append", hd=64, H=32, Hkv=8, B=4, n=128, lo=9000, hi=30000,
             dtype="f32", rd=32, inter=True, factor=8.0, orig=8192, tree=False),
        # one stream's verify attention, context 2048
        dict(name="attend b1 n5 t2048", op="attend", hd=128, H=32, Hkv=8, B=1, n=5, lo=2048, hi=2048, tree=False),
        # one stream, one token, a very long context
        dict(name="attend b1 n1 t131000", op="attend", hd=128, H=32, Hkv=8, B=1, n=1, lo=131000, hi=131000,
             tree=False),
        # a medium batch with ragged contexts
        dict(name="attend b16 n5", op="attend", hd=128, H=32, Hkv=8, B=16, n=5, lo=512, hi=4096, tree=False),
        # the full batch
        dict(name="attend b64 n5", op="attend", hd=128, H=32, Hkv=8, B=64, n=5, lo=512, hi=4096, tree=False),
        # draft trees of 15 nodes, 1B-shaped heads (head dim 64)
        dict(name="attend tree b4 n15 hd64", op="attend", hd=64, H=32, Hkv=8, B=4, n=15, lo=700, hi=1900, tree=True),
        # a prefill chunk over a cached prefix
        dict(name="attend prefill n128", op="attend", hd=128, H=32, Hkv=8, B=1, n=128, lo=4000, hi=4000,
             tree=False),
        # the commit of an accepted path, one stream, 8B-shaped layers
        dict(name="commit b1 n7 l32", op="commit", hd=128, H=32, Hkv=8, B=1, n=7, lo=2000, hi=2000, layers=32),
        # a batch of large trees
        dict(name="commit b16 n33 l32", op="commit", hd=128, H=32, Hkv=8, B=16, n=33, lo=512, hi=4096, layers=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "commit"])
    hd, H, Hkv = rng.choice([(128, 32, 8), (128, 32, 8), (64, 32, 8), (128, 4, 1), (64, 4, 2), (128, 8, 8)])
    B = _log_int(rng, 1, 64)
    if op == "append":
        rd = rng.choice([hd, hd, hd // 2])
        n = rng.randint(1, 9) if rng.random() < 0.7 else _log_int(rng, 1, max(1, min(128, 512 // B)))
        hi = _log_int(rng, 1, 30000)
        return dict(op=op, hd=hd, H=H, Hkv=Hkv, B=B, n=n, lo=rng.randint(0, hi), hi=hi,
                    dtype=rng.choice(["bf16", "f32"]), rd=rd, inter=rng.random() < 0.5,
                    factor=rng.choice([1.0, 4.0]), orig=rng.choice([0, 8192]),
                    tree=rng.random() < 0.3 and n <= 64)
    if op == "commit":
        layers = _log_int(rng, 1, 32)
        n = rng.randint(2, 33)
        B = min(B, 16)
        hi = _log_int(rng, 1, 4096)
        return dict(op=op, hd=hd, H=H, Hkv=Hkv, B=B, n=n, lo=rng.randint(0, hi), hi=hi, layers=layers)
    n = rng.randint(1, 9) if rng.random() < 0.7 else _log_int(rng, 1, max(1, min(128, 512 // B)))
    hi = _log_int(rng, 1, max(16, min(131000, 140000 // B)))
    if n > 16:
        hi = min(hi, 4096)
    return dict(op=op, hd=hd, H=H, Hkv=Hkv, B=B, n=n, lo=rng.randint(hi // 4, hi), hi=hi,
                tree=rng.random() < 0.3 and n <= 64)


# ------------------------------------------------------------------- inputs
def _lens(case, seed):
    r = random.Random(seed * 7919 + 13)
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _trees(case, seed):
    """(ancestor masks, depths) of one random draft tree per sequence."""
    r = random.Random(seed * 104729 + 7)
    anc, depth = [], []
    for _ in range(case["B"]):
        a, d = [1], [0]
        for i in range(1, case["n"]):
            p = r.randint(max(0, i - 4), i - 1)
            a.append(a[p] | (1 << i))
            d.append(d[p] + 1)
        anc.append([x - (1 << 64) if x >> 63 else x for x in a])
        depth.append(d)
    return torch.tensor(anc, dtype=torch.int64), torch.tensor(depth, dtype=torch.int32)


def _paths(case, seed):
    """Accepted paths [B][n] (-1 padded, strictly increasing) and their lengths."""
    r = random.Random(seed * 31 + 5)
    n = case["n"]
    path, m = [], []
    for _ in range(case["B"]):
        k = min(n - 1, r.choice([0, 1, 2, 2, 3, 4, 5, 6]))
        p = sorted(r.sample(range(1, n), k))
        path.append(p + [-1] * (n - k))
        m.append(k)
    return torch.tensor(path, dtype=torch.int32), torch.tensor(m, dtype=torch.int32)


def _rounded(x):
    """(e4m3 values, scales) of rows [..., 64 slots, hd], a power-of-two scale per 16 slots."""
    b = x.view(*x.shape[:-2], PAGE // BLOCK, BLOCK, x.shape[-1])
    s = _scale_of(b.abs().amax(dim=(-1, -2)))
    c = (b / s[..., None, None]).clamp_(-FMAX, FMAX).to(E4M3)
    return c.view(x.shape), s


def _scale_of(amax):
    m, e = torch.frexp(amax / FMAX)  # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, LO_EXP)).clamp(LO_EXP, HI_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _inputs(case, seed):
    """Everything the call works on, from the seed alone."""
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    B, n, hd, Hkv, H = case["B"], case["n"], case["hd"], case["Hkv"], case["H"]
    L = case.get("layers", 1)
    lens = _lens(case, seed)
    r = random.Random(seed + 17)
    slack = 2 * BLOCK  # pages are reserved a little ahead of the new slots
    need = [(x + n + slack + PAGE - 1) // PAGE for x in lens]
    shared = case["op"] != "attend"  # whole pages before the new slots: one prefix that every sequence shares
    own_from = [x // PAGE if shared else 0 for x in lens]
    if shared:  # pages for any starting slot within a page, so that a pool's size goes by the case alone
        total = B * ((PAGE - 1 + n + slack + PAGE - 1) // PAGE) + 1
    else:
        total = sum(need) + 1
    ids = list(range(1, total))
    r.shuffle(ids)
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    for b in range(B):
        k = need[b] - own_from[b]
        table[b, :own_from[b]] = 0
        table[b, own_from[b]:need[b]] = torch.tensor(ids[:k], dtype=torch.int32)
        ids = ids[k:]
    gain = torch.ones(hd, device=dev)
    gain[:: hd // 4] = 4.0  # a few strong key channels
    k8, v8, ks, vs = [], [], [], []
    for _ in range(L):
        size = torch.exp(0.3 * torch.randn(total, Hkv, PAGE, 1, generator=g, device=dev))
        c, s = _rounded(torch.randn(total, Hkv, PAGE, hd, generator=g, device=dev) * gain * size)
        k8.append(c)
        ks.append(s)
        c, s = _rounded(torch.randn(total, Hkv, PAGE, hd, generator=g, device=dev) * size)
        v8.append(c)
        vs.append(s)
    st = dict(k=torch.stack(k8), v=torch.stack(v8), k_scale=torch.stack(ks), v_scale=torch.stack(vs),
              table=table.to(dev), lens=lens)
    length = [x + n for x in lens] if case["op"] == "commit" else lens
    st["len"] = torch.tensor(length, dtype=torch.int32, device=dev)
    if case["op"] == "attend":  # slots past the new ones hold anything: here codes that are not numbers
        for b in range(B):
            t = lens[b] + n
            p0 = t // PAGE
            if p0 < need[b]:
                pg = int(table[b, p0])
                st["k"].view(torch.uint8)[:, pg, :, t % PAGE:] = 0x7F
                st["v"].view(torch.uint8)[:, pg, :, t % PAGE:] = 0x7F
    M = B * n
    if case["op"] != "commit":
        dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
        st["q"] = torch.randn(M, H * hd, generator=g, device=dev).to(dt)
        if case["op"] == "append":  # one projection's output: rows of q, k and v heads together
            k = (torch.randn(M, Hkv, hd, generator=g, device=dev) * gain).view(M, Hkv * hd).to(dt)
            v = torch.randn(M, Hkv * hd, generator=g, device=dev).to(dt)
            st["q"], st["knew"], st["vnew"] = torch.cat([st["q"], k, v], dim=1).split(
                [H * hd, Hkv * hd, Hkv * hd], dim=1)
        anc, depth = _trees(case, seed) if case["tree"] else (None, None)
        st["anc"] = None if anc is None else anc.to(dev)
        st["depth"] = None if depth is None else depth.to(dev)
    else:
        path, m = _paths(case, seed)
        st["path"], st["m"] = path.to(dev), m.to(dev)
    return st


def _freqs(case):
    """Rotary frequencies in radians per position (numpy, 64 bits)."""
    rd = case["rd"]
    f = 500000.0 ** (-2.0 * np.arange(rd // 2) / rd)
    if case["factor"] == 1.0:
        return f
    if not case["orig"]:
        return f / case["factor"]
    turns = case["orig"] * f / (2 * math.pi)  # turns over the original length: below 1 scaled, above 4 kept
    w = np.clip((turns - 1.0) / 3.0, 0.0, 1.0)
    return f * w + f / case["factor"] * (1 - w)


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if case["op"] == "append":
        st["freq"] = torch.from_numpy(_freqs(case)).to(st["q"].device)
        st["q_out"] = torch.empty(case["B"] * case["n"], case["H"] * case["hd"], dtype=torch.bfloat16,
                                  device=st["q"].device)
    if case["op"] == "attend":
        st["out"] = torch.empty_like(st["q"])
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        L = case.get("layers", 1)
        cfg = sb.ModelConfig(n_layers=L, d_model=case["H"] * case["hd"], n_heads=case["H"],
                             n_kv_heads=case["Hkv"], d_ffn=128, vocab=1000)
        st["cfg"] = cfg
        kv = sb.KV8Cache(cfg, case["B"], st["k"].shape[1], st["table"].shape[1])
        kv.k, kv.v, kv.k_scale, kv.v_scale = st["k"], st["v"], st["k_scale"], st["v_scale"]
        kv.len, kv.table = st["len"], st["table"]
        st["kv"] = kv
        st["ws"] = sb.workspace(256)
        if case["op"] == "append":
            st["rope"] = sb.RopeTable(case["rd"], 500000.0, interleaved=case["inter"], factor=case["factor"],
                                      low_freq=1.0, high_freq=4.0, orig_len=case["orig"])
    if case["op"] == "commit":
        st["len0"] = st["len"].clone()
    return st


def run(st):
    op = st["case"]["op"]
    return _append(st) if op == "append" else _attend(st) if op == "attend" else _commit(st)


def _state(st):
    return dict(k=st["k"], v=st["v"], k_scale=st["k_scale"], v_scale=st["v_scale"])


# ------------------------------------------------------------------- append
def _rotate(x, cos, sin, rd, inter):
    """x [M, heads, hd] fp32, cos / sin [M, 1, rd / 2]."""
    y = x.clone()
    a, b = (slice(0, rd, 2), slice(1, rd, 2)) if inter else (slice(0, rd // 2), slice(rd // 2, rd))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _put(codes, scales, table, length, n, new):
    """Rows `new` [B, n, Hkv, hd] to slots length .. length + n - 1 of one layer's pages."""
    B, _, Hkv, hd = new.shape
    dev = new.device
    nb = (BLOCK - 1 + n + BLOCK - 1) // BLOCK  # blocks that n slots can touch
    ln = length.long()
    blk = ln[:, None] // BLOCK + torch.arange(nb, device=dev)
    per = PAGE // BLOCK
    page = table.long().gather(1, blk // per)
    sub = blk % per
    slot = blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)  # [B, nb, 16]
    j = slot - ln[:, None, None]
    fresh = (j >= 0) & (j < n)
    held = j < 0
    x = torch.take_along_dim(new[:, None].expand(B, nb, n, Hkv, hd),
                             j.clamp(0, n - 1)[..., None, None].expand(-1, -1, -1, Hkv, hd), 2)
    x = torch.where(fresh[..., None, None], x, 0.0).transpose(2, 3)  # [B, nb, Hkv, 16, hd]
    c = codes.view(torch.uint8).view(-1, Hkv, per, BLOCK, hd)
    old_bits = c[page, :, sub]  # [B, nb, Hkv, 16, hd]
    s_old = scales[page, :, sub]  # [B, nb, Hkv]
    s_new = _scale_of(torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=(-1, -2)))
    keeps = held.any(2)[:, :, None]
    touched = fresh.any(2)[:, :, None]
    s = torch.where(keeps, torch.maximum(s_old, s_new), s_new)
    s = torch.where(touched, s, s_old)
    val = torch.where(held[:, :, None, :, None], old_bits.view(E4M3).float() * s_old[..., None, None], x)
    bits = (val / s[..., None, None]).clamp(-FMAX, FMAX).to(E4M3).view(torch.uint8)
    write = ((held & touched) | fresh)[:, :, None, :, None]
    c[page, :, sub] = torch.where(write, bits, old_bits)
    scales[page, :, sub] = s


def _append(st):
    c = st["case"]
    B, n, H, Hkv, hd = c["B"], c["n"], c["H"], c["Hkv"], c["hd"]
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        sb.spec_kv8_append(st["cfg"], st["kv"], 0, n, st["q"], st["knew"], st["vnew"], st["rope"], st["q_out"],
                           st["ws"], depth=st["depth"])
        return dict(_state(st), q=st["q_out"])
    step = st["depth"] if st["depth"] is not None else torch.arange(n, device=st["q"].device)[None]
    pos = (st["len"][:, None] + step).reshape(-1, 1, 1).double()
    ang = pos * st["freq"]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    q = _rotate(st["q"].float().reshape(B * n, H, hd), cos, sin, c["rd"], c["inter"])
    k = _rotate(st["knew"].float().reshape(B * n, Hkv, hd), cos, sin, c["rd"], c["inter"])
    _put(st["k"][0], st["k_scale"][0], st["table"], st["len"], n, k.view(B, n, Hkv, hd))
    _put(st["v"][0], st["v_scale"][0], st["table"], st["len"], n, st["vnew"].float().reshape(B, n, Hkv, hd))
    return dict(_state(st), q=q.view(B * n, H * hd).to(torch.bfloat16))


# ---------------------------------------------------------------- attention
def _attend(st):
    c = st["case"]
    B, n, H, Hkv, hd = c["B"], c["n"], c["H"], c["Hkv"], c["hd"]
    G = H // Hkv
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        sb.spec_kv8_attention(st["cfg"], st["kv"], 0, n, st["q"], st["out"], st["ws"], anc=st["anc"])
        return st["out"]
    dev = st["q"].device
    T = st["table"].shape[1] * PAGE
    page = st["table"].long().clamp_min(0)
    ln = st["len"].long()[:, None]
    t = torch.arange(T, device=dev)[None]
    valid = t < ln + n  # [B, T]

    def rows(codes, scales):
        x = codes.view(torch.uint8)[page].view(E4M3).float()  # [B, pages, Hkv, 64, hd]
        x = x.view(*x.shape[:3], PAGE // BLOCK, BLOCK, hd) * scales[page][..., None, None]
        x = x.view(B, -1, Hkv, PAGE, hd).transpose(1, 2).reshape(B, Hkv, T, hd)
        return torch.where(valid[:, None, :, None], x, 0.0)

    q = st["q"].float().view(B, n, Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, hd)
    s = torch.matmul(q, rows(st["k"][0], st["k_scale"][0]).transpose(2, 3)) / math.sqrt(hd)
    new = (t - ln)[:, None, :]  # [B, 1, T]
    j = torch.arange(n, device=dev)[None, :, None]
    if st["anc"] is not None:
        bit = (st["anc"][:, :, None] >> new.clamp(0, 63)) & 1
        see = (new < 0) | ((bit == 1) & (new < n))
    else:
        see = new <= j
    see = see[:, None, :, None, :].expand(B, 1, n, G, T).reshape(B, 1, n * G, T)
    s = torch.where(see, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    o = torch.matmul(p, rows(st["v"][0], st["v_scale"][0]))
    tot = p.sum(-1, keepdim=True)
    o = torch.where(tot > 0, o / tot, 0.0)
    return o.view(B, Hkv, n, G, hd).permute(0, 2, 1, 3, 4).reshape(B * n, H * hd).to(torch.bfloat16)


# ------------------------------------------------------------------- commit
def _move(codes, scales, table, L0, path, m):
    """Rows L0 + path[d - 1] to L0 + d of every layer: codes [L, pages, Hkv, 64, hd]."""
    L, _, Hkv, _, hd = codes.shape
    B, n = path.shape
    dev = codes.device
    per = PAGE // BLOCK
    d = torch.arange(1, n, device=dev)[None]
    moved = d <= m[:, None]  # [B, n - 1]
    src = L0[:, None] + torch.where(moved, path[:, : n - 1].long(), 0)
    c = codes.view(torch.uint8)
    spage, sslot = table.long().gather(1, src // PAGE), src % PAGE
    src_s = scales[:, spage, :, sslot // BLOCK]  # [B, n - 1, L, Hkv]
    val = c[:, spage, :, sslot].view(E4M3).float() * src_s[..., None]
    nb = (BLOCK - 1 + n + BLOCK - 1) // BLOCK
    blk = L0[:, None] // BLOCK + torch.arange(nb, device=dev)
    page, sub = table.long().gather(1, blk // per), blk % per
    slot = blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)
    off = slot - L0[:, None, None]  # the row's distance from the root
    lands = (off >= 1) & (off <= m[:, None, None])  # [B, nb, 16]
    keeps = off <= 0
    at = (off - 1).clamp(0, n - 2)

    def of(x):  # [B, n - 1, ...] -> the row landing in each slot [B, nb, 16, ...]
        return x[torch.arange(B, device=dev)[:, None, None], at]

    s_old = scales[:, page, :, sub]  # [B, nb, L, Hkv]
    s_in = torch.where(lands[..., None, None], of(src_s), 0.0).amax(2)
    s = torch.where(keeps.any(2)[..., None, None], torch.maximum(s_old, s_in), s_in)
    touched = lands.any(2)[..., None, None]
    s = torch.where(touched, s, s_old)
    c6 = c.view(L, -1, Hkv, per, BLOCK, hd)
    old = c6[:, page, :, sub]  # [B, nb, L, Hkv, 16, hd]
    rows = of(val).permute(0, 1, 3, 4, 2, 5)
    x = torch.where(lands[:, :, None, None, :, None], rows, old.view(E4M3).float() * s_old[..., None, None])
    bits = (x / s[..., None, None]).clamp(-FMAX, FMAX).to(E4M3).view(torch.uint8)
    write = (lands | (keeps & lands.any(2, keepdim=True)))[:, :, None, None, :, None]
    c6[:, page, :, sub] = torch.where(write, bits, old)
    scales[:, page, :, sub] = s


def _commit(st):
    c = st["case"]
    st["len"].copy_(st["len0"])  # the pass that scored the tree has advanced the lengths
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        sb.spec_kv8_tree_commit(st["cfg"], st["kv"], st["path"], st["m"], c["n"], st["ws"])
    else:
        L0 = st["len"].long() - c["n"]
        _move(st["k"], st["k_scale"], st["table"], L0, st["path"], st["m"].long())
        _move(st["v"], st["v_scale"], st["table"], L0, st["path"], st["m"].long())
        st["len"].copy_(L0 + 1 + st["m"])
    return dict(_state(st), len=st["len"])


# --------------------------------------------------------------------- work
def work(case):
    B, n, hd, Hkv, H = case["B"], case["n"], case["hd"], case["Hkv"], case["H"]
    M = B * n
    mean = (case["lo"] + case["hi"]) / 2
    if case["op"] == "append":
        e = 4 if case["dtype"] == "f32" else 2
        rows = M * (H + 2 * Hkv) * hd
        return dict(bytes=rows * e + M * H * hd * 2 + 2 * M * Hkv * (hd + 4 / BLOCK),
                    flops=6.0 * M * (H + Hkv) * case["rd"] / 2 + 2.0 * M * 2 * Hkv * hd)
    if case["op"] == "attend":
        T = B * (mean + n)
        pairs = B * n * (mean + (n + 1) / 2)
        return dict(bytes=2 * T * Hkv * (hd + 4 / BLOCK) + 2 * M * H * hd * 2, flops=4.0 * pairs * H * hd)
    rows = B * min(n - 1, 3)
    return dict(bytes=2 * 2 * rows * case["layers"] * Hkv * (hd + 4 / BLOCK),
                flops=2.0 * 2 * rows * case["layers"] * Hkv * hd)


# -------------------------------------------------------------------- exact
def _round8(x):
    """Nearest e4m3 value of a 64-bit number, ties to even (|x| <= 448), by its steps."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -20))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _power(amax):
    if amax <= 0:
        return 2.0 ** LO_EXP
    e = LO_EXP
    while e < HI_EXP and 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def exact(case, seed):
    st = _inputs(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "commit": _exact_commit}[case["op"]](case, st)


def _exact_append(case, st):
    B, n, H, Hkv, hd, rd = (case[k] for k in ("B", "n", "H", "Hkv", "hd", "rd"))
    f = _freqs(case)
    depth = None if st["depth"] is None else st["depth"].cpu().numpy()
    turn = np.array([[(st["lens"][b] + (j if depth is None else int(depth[b, j]))) * f for j in range(n)]
                     for b in range(B)])
    z = torch.from_numpy(np.exp(1j * turn)).to(st["q"].device).view(B * n, 1, rd // 2)

    def turned(x, heads):
        x = x.double().reshape(B * n, heads, hd).clone()
        r = x[..., :rd]
        w = (torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) if case["inter"] else
             torch.complex(r[..., : rd // 2].contiguous(), r[..., rd // 2:].contiguous())) * z
        if case["inter"]:
            x[..., 0:rd:2], x[..., 1:rd:2] = w.real, w.imag
        else:
            x[..., : rd // 2], x[..., rd // 2: rd] = w.real, w.imag
        return x

    out = {"q": turned(st["q"], H).view(B * n, H * hd)}
    table = st["table"].cpu().numpy()
    for name, x in (("k", turned(st["knew"], Hkv)), ("v", st["vnew"].double().reshape(B * n, Hkv, hd))):
        codes, scales = st[name].double(), st[name + "_scale"].double()
        for b in range(B):
            L, end = st["lens"][b], st["lens"][b] + n
            for blk in range(L // BLOCK, (end - 1) // BLOCK + 1):
                lo, hi = max(blk * BLOCK, L), min((blk + 1) * BLOCK, end)
                pg, sub, r0 = int(table[b, blk * BLOCK // PAGE]), blk % (PAGE // BLOCK), blk * BLOCK % PAGE
                rows = x[b * n + lo - L: b * n + hi - L].transpose(0, 1)  # [Hkv, rows, hd]
                tops = rows.abs().amax(dim=(1, 2)).cpu().tolist()
                s = torch.tensor([_power(a) for a in tops], dtype=torch.float64, device=rows.device)
                kept = lo - blk * BLOCK
                if kept:
                    old = scales[0, pg, :, sub]
                    s = torch.maximum(s, old)
                    held = codes[0, pg, :, r0: r0 + kept]
                    codes[0, pg, :, r0: r0 + kept] = _round8(held * (old / s)[:, None, None])
                a = kept + r0
                codes[0, pg, :, a: a + hi - lo] = _round8((rows / s[:, None, None]).clamp(-448, 448))
                scales[0, pg, :, sub] = s
        out[name], out[name + "_scale"] = codes, scales
    return out


def _exact_attend(case, st):
    B, n, H, Hkv, hd = (case[k] for k in ("B", "n", "H", "Hkv", "hd"))
    G = H // Hkv
    out = torch.zeros(B * n, H * hd, dtype=torch.float64, device=st["q"].device)
    for b in range(B):
        T = st["lens"][b] + n
        pg = st["table"][b, : (T + PAGE - 1) // PAGE].long()
        kv = []
        for name in ("k", "v"):
            s = st[name + "_scale"][0][pg].double().repeat_interleave(BLOCK, dim=2)  # [pages, Hkv, 64]
            x = st[name][0].view(torch.uint8)[pg].view(E4M3).double() * s[..., None]
            kv.append(x.transpose(0, 1).reshape(Hkv, -1, hd)[:, :T])
        q = st["q"][b * n: (b + 1) * n].double().view(n, Hkv, G, hd)
        s = torch.einsum("jhgd,htd->hgjt", q, kv[0]) * hd ** -0.5
        see = torch.ones(n, T, dtype=torch.bool)
        for j in range(n):
            for i in range(n):
                see[j, T - n + i] = i <= j if st["anc"] is None else bool((int(st["anc"][b, j]) >> i) & 1)
        s = s.masked_fill(~see.to(s.device), -math.inf)
        out[b * n: (b + 1) * n] = torch.einsum("hgjt,htd->jhgd", torch.softmax(s, -1), kv[1]).reshape(n, H * hd)
    return out


def _exact_commit(case, st):
    B, n = case["B"], case["n"]
    table, path, m = st["table"].cpu().numpy(), st["path"].cpu().numpy(), st["m"].cpu().numpy()
    out = {"len": torch.tensor([st["lens"][b] + 1 + int(m[b]) for b in range(B)], dtype=torch.int32)}
    for name in ("k", "v"):
        codes, scales = st[name].double(), st[name + "_scale"].double()
        for b in range(B):
            L0, k = st["lens"][b], int(m[b])

            def where(slot):
                return int(table[b, slot // PAGE]), slot % PAGE, slot % PAGE // BLOCK

            came = []
            for d in range(1, k + 1):
                p, r, sub = where(L0 + int(path[b, d - 1]))
                came.append((codes[:, p, :, r].clone(), scales[:, p, :, sub].clone()))
            for blk in range((L0 + 1) // BLOCK, (L0 + k) // BLOCK + 1) if k else []:
                lands = [d for d in range(1, k + 1) if (L0 + d) // BLOCK == blk]
                p, r0, sub = where(blk * BLOCK)
                s = came[lands[0] - 1][1]
                for d in lands[1:]:
                    s = torch.maximum(s, came[d - 1][1])
                kept = L0 + 1 - blk * BLOCK
                if kept > 0:
                    old = scales[:, p, :, sub].clone()
                    s = torch.maximum(s, old)
                    codes[:, p, :, r0: r0 + kept] = _round8(codes[:, p, :, r0: r0 + kept] * (old / s)[..., None, None])
                for d in lands:
                    c0, s0 = came[d - 1]
                    codes[:, p, :, (L0 + d) % PAGE] = _round8(c0 * (s0 / s)[..., None])
                scales[:, p, :, sub] = s
        out[name], out[name + "_scale"] = codes, scales
    return out
