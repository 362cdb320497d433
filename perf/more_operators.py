"""Workloads of truncated sampling and of the device page pool.

* ``sample``: tokens drawn from softmax(z / T) after min-p, top-k and top-p,
  with parameters per row, several draws a row and the distribution itself
  where a verification needs it;
* ``filter``: the same truncation as -inf in the logits (the target's rows
  before an acceptance test);
* ``branch``: one step of parallel continuations on a paged cache: the losing
  sequences are freed, the winners forked into their places, and slots for the
  next tokens reserved, the partly filled last pages copied where they are
  shared;
* ``compact``: the pool's used pages moved to its lowest page numbers;
* ``copy``: pages handed from one pool to another.

``run`` computes an operator either with the library's kernels (``own``) or in
elementary torch operations; ``exact`` gives the definition in 64 bits.

A row's truncation is one threshold on its logits: min-p keeps z >= M + T ln
min_p (M the largest), top-k every logit not below the k-th largest, top-p, on
what those two leave, every logit not below the one where the descending
cumulative mass first reaches top_p of the total.  A draw is the smallest id
whose cumulative weight among the kept exceeds u times their total.

Pages hold 64 slots.  ``ref`` counts the sequences that hold each page; pages
are taken lowest number first, by sequence and then by position.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
BLOCK = 16
E4M3 = torch.float8_e4m3fn

# layers, KV heads and head dim of the two model shapes
SHAPES = {"8b": (32, 8, 128), "1b": (16, 8, 64)}


def listed():
    return [
        # one stream's next token, one user's settings: the smallest call, all latency
        dict(name="sample b1", op="sample", rows=1, V=128256, draws=1, dtype="f32", probs=False, par="chat"),
        # a serving batch's drafts, every request with settings of its own, q rows kept for the acceptance test
        dict(name="sample b64 mixed probs", op="sample", rows=64, V=128256, draws=1, dtype="f32", probs=True,
             par="mixed"),
        # the children of draft-tree nodes: four draws from each row, a small draft model's logits in bf16
        dict(name="sample tree b60 bf16", op="sample", rows=60, V=32000, draws=4, dtype="bf16", probs=True,
             par="mixed"),
        # batch 64 at draft depth 4, top-p alone: the whole row's mass counts
        dict(name="sample b320 top-p", op="sample", rows=320, V=128256, draws=1, dtype="f32", probs=False,
             par="topp"),
        # one stream's verification rows, draft depth 4
        dict(name="filter b5", op="filter", rows=5, V=128256, dtype="f32", par="chat"),
        # a full batch's verification rows, settings per sequence
        dict(name="filter b320 mixed", op="filter", rows=320, V=128256, dtype="f32", par="mixed"),
        # one prompt in four continuations, 8B-shaped bf16 cache
        dict(name="branch 1x4 8b bf16", op="branch", shape="8b", kv8=False, groups=1, ways=4, lo=2005, hi=2005, n=5),
        # sixteen prompts in four continuations each, ragged contexts, 8-bit cache
        dict(name="branch 16x4 8b kv8", op="branch", shape="8b", kv8=True, groups=16, ways=4, lo=512, hi=4096, n=5),
        # a small pool, every second page free
        dict(name="compact 96 1b bf16", op="compact", shape="1b", kv8=False, pages=96, used=0.5),
        # a large fragmented pool of the 8-bit cache
        dict(name="compact 1200 8b kv8", op="compact", shape="8b", kv8=True, pages=1200, used=0.5),
        # a short prefix handed to another pool
        dict(name="copy 4 1b kv8", op="copy", shape="1b", kv8=True, pages=4),
        # a batch of contexts handed to another pool
        dict(name="copy 200 8b bf16", op="copy", shape="8b", kv8=False, pages=200),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "filter", "branch", "compact", "copy"])
    if op in ("sample", "filter"):
        V = rng.choice([128256, 32000, 128256, 50257, 151936, _log_int(rng, 8, 200000)])
        rows = _log_int(rng, 1, max(1, min(512, 40_000_000 // V)))
        c = dict(op=op, rows=rows, V=V, dtype=rng.choice(["f32", "f32", "bf16"]),
                 par=rng.choice(["chat", "mixed", "mixed", "topp", "plain"]))
        if op == "sample":
            c.update(draws=rng.choice([1, 1, 1, rng.randint(2, 16)]), probs=rng.random() < 0.4)
        return c
    shape, kv8 = rng.choice(["8b", "1b"]), rng.random() < 0.5
    if op == "branch":
        hi = _log_int(rng, 64, 4096)
        groups = _log_int(rng, 1, 8)
        return dict(op=op, shape=shape, kv8=kv8, groups=groups, ways=rng.randint(2, 8 if groups < 5 else 4),
                    lo=rng.randint(1, hi), hi=hi, n=rng.randint(1, 70))
    if op == "compact":
        return dict(op=op, shape=shape, kv8=kv8, pages=_log_int(rng, 8, 500 if kv8 else 300),
                    used=round(rng.uniform(0.1, 0.95), 2))
    return dict(op=op, shape=shape, kv8=kv8, pages=_log_int(rng, 1, 150))


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _generator(seed):
    return torch.Generator(device=_device()).manual_seed(seed)


# ------------------------------------------------------------------- inputs
def _params(case, seed):
    """Temperature, top-k, top-p and min-p of each row (lists)."""
    r = random.Random(seed * 7919 + 3)
    out = []
    for _ in range(case["rows"]):
        kind = case["par"]
        if kind == "mixed":
            kind = r.choice(["chat", "chat", "topp", "minp", "k", "plain", "greedy"])
        T = r.choice([0.6, 0.7, 0.8, 1.0, 1.2])
        p = {"chat": (T, 50, 0.95, 0.0), "topp": (T, 0, r.choice([0.9, 0.95]), 0.0),
             "minp": (T, 0, 1.0, r.choice([0.05, 0.1])), "k": (T, r.choice([20, 40, 1000]), 1.0, 0.0),
             "plain": (T, 0, 1.0, 0.0), "greedy": (0.0, 0, 1.0, 0.0)}[kind]
        out.append(p)
    return [list(x) for x in zip(*out)]


def _logit_inputs(case, seed):
    dev, g = _device(), _generator(seed)
    rows, V = case["rows"], case["V"]
    z = 2.0 * torch.randn(rows, V, generator=g, device=dev)
    # a few likely continuations; how far they stand out goes by the row
    m = min(64, V)
    ids = torch.randint(0, V, (rows, m), generator=g, device=dev)
    far = torch.tensor([0.0, 1.5, 3.0, 4.5], device=dev)[torch.arange(rows, device=dev) % 4]
    bump = -torch.log(torch.rand(rows, m, generator=g, device=dev).clamp_min(1e-9)) * far[:, None]
    z.scatter_add_(1, ids, bump)
    if rows > 7:  # rows under a constraint allow few tokens
        allowed = torch.rand(1, V, generator=g, device=dev) < 0.01
        allowed[:, V // 2] = True
        z[7::8] = torch.where(allowed, z[7::8], -math.inf)
    st = dict(z=z.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32))
    T, k, p, mp = _params(case, seed)
    st["T"] = torch.tensor(T, dtype=torch.float32, device=dev)
    st["k"] = torch.tensor(k, dtype=torch.int32, device=dev)
    st["p"] = torch.tensor(p, dtype=torch.float32, device=dev)
    st["mp"] = torch.tensor(mp, dtype=torch.float32, device=dev)
    if case["op"] == "sample":
        st["u"] = torch.rand(rows, case["draws"], generator=g, device=dev)
    return st


def _pool(shape, kv8, pages, g):
    """k, v (and scales) of a pool with anything in it."""
    L, Hkv, hd = SHAPES[shape]
    dev = _device()

    def rows():
        b = torch.randint(0, 256, (L, pages, Hkv, PAGE, hd if kv8 else 2 * hd), dtype=torch.uint8, generator=g,
                          device=dev)
        if kv8:
            return b.bitwise_and_(0xF7).view(E4M3)  # no NaN codes
        return b.view(torch.int16).bitwise_and_(-16449).view(torch.bfloat16)  # 0xBFBF: finite

    st = dict(k=rows(), v=rows())
    if kv8:
        for s in ("k_scale", "v_scale"):
            e = torch.randint(-12, 3, (L, pages, Hkv, PAGE // BLOCK), generator=g, device=dev)
            st[s] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return st


def _page_state(B, n_pages, max_pages, held, lens):
    """table, len, mapped, ref and n_free as views of one buffer, so that a loop restores them in one copy."""
    dev = _device()
    table = np.full((B, max_pages), -1, np.int32)
    ref = np.zeros(n_pages, np.int32)
    for b, ids in enumerate(held):
        table[b, : len(ids)] = ids
        np.add.at(ref, ids, 1)
    flat = np.concatenate([table.ravel(), np.array(lens, np.int32), np.array([len(x) for x in held], np.int32), ref,
                           np.array([(ref == 0).sum()], np.int32)])
    flat = torch.from_numpy(flat).to(dev)
    return dict(first=flat, **_views(flat.clone(), B, n_pages, max_pages))


def _views(flat, B, n_pages, max_pages):
    t, ln, mp, rf, nf = flat.split([B * max_pages, B, B, n_pages, 1])
    return dict(flat=flat, table=t.view(B, max_pages), len=ln, mapped=mp, ref=rf, n_free=nf)


def _page_inputs(case, seed):
    r, g = random.Random(seed * 31 + 5), _generator(seed)
    if case["op"] == "branch":
        G, W, n = case["groups"], case["ways"], case["n"]
        lens = [r.randint(case["lo"], case["hi"]) for _ in range(G)]
        need = [(x + PAGE - 1) // PAGE for x in lens]
        # a pool's size goes by the case alone
        n_pages = G * ((case["hi"] + PAGE - 1) // PAGE) + G * W * ((n + PAGE - 1) // PAGE + 1) + 3
        ids = list(range(n_pages))
        r.shuffle(ids)
        held, all_lens, src, dst = [], [], [], []
        for i in range(G):
            first = len(held)
            held.append(ids[: need[i]])
            ids = ids[need[i]:]
            all_lens.append(lens[i])
            for _ in range(W - 1):
                src.append(first)
                dst.append(len(held))
                held.append([])
                all_lens.append(0)
        max_pages = (case["hi"] + n + PAGE - 1) // PAGE
        st = _page_state(G * W, n_pages, max_pages, held, all_lens)
        st["src"] = torch.tensor(src, dtype=torch.int32, device=_device())
        st["dst"] = torch.tensor(dst, dtype=torch.int32, device=_device())
        st["n_pages"] = n_pages
    elif case["op"] == "compact":
        n_pages = case["pages"]
        used = max(1, min(n_pages - 1, int(case["used"] * n_pages)))
        ids = r.sample(range(n_pages), used)
        B = min(16, used)
        shared = ids[: used // 8] if B > 1 else []  # a prefix that every sequence holds
        rest = ids[len(shared):]
        held = [shared + rest[b::B] for b in range(B)]
        max_pages = max(len(x) for x in held) + 2
        st = _page_state(B, n_pages, max_pages, held, [len(x) * PAGE - b for b, x in enumerate(held)])
        st["n_pages"] = n_pages
    else:
        n_pages = case["pages"] + 5
        a, b = r.sample(range(n_pages), case["pages"]), r.sample(range(n_pages), case["pages"])
        st = dict(src=torch.tensor(a, dtype=torch.int32, device=_device()),
                  dst=torch.tensor(b, dtype=torch.int32, device=_device()), n_pages=n_pages)
        st["to"] = _pool(case["shape"], case["kv8"], n_pages, g)
    st["pool"] = _pool(case["shape"], case["kv8"], n_pages, g)
    return st


def _cache(case, pool, batch, n_pages, max_pages):
    from speculative_decoding_verification_pass_gb300 import binding as sb
    L, Hkv, hd = SHAPES[case["shape"]]
    cfg = sb.ModelConfig(n_layers=L, d_model=32 * hd, n_heads=32, n_kv_heads=Hkv, d_ffn=128, vocab=1000)
    if case["kv8"]:
        return sb.KV8Cache(cfg, batch, n_pages, max_pages, **pool)
    return sb.PagedKVCache(cfg, batch, n_pages, max_pages, **pool)


def prepare(case, seed):
    if case["op"] in ("sample", "filter"):
        st = _logit_inputs(case, seed)
        rows, V = case["rows"], case["V"]
        if case["op"] == "sample":
            st["tokens"] = torch.empty(rows, case["draws"], dtype=torch.int32, device=st["z"].device)
            st["probs"] = torch.empty(rows, V, dtype=torch.float32, device=st["z"].device) if case["probs"] else None
        else:
            st["out"] = torch.empty_like(st["z"])
        if own:
            from speculative_decoding_verification_pass_gb300 import binding as sb
            st["sampling"] = sb.Sampling(temperature=st["T"], top_k=st["k"], top_p=st["p"], min_p=st["mp"])
            st["ws"] = sb.workspace(256)
    else:
        st = _page_inputs(case, seed)
        if own:
            from speculative_decoding_verification_pass_gb300 import binding as sb
            if case["op"] == "copy":
                st["kv"] = _cache(case, st["pool"], 1, st["n_pages"], 1)
                st["kv_to"] = _cache(case, st["to"], 1, st["n_pages"], 1)
                st["ws"] = sb.workspace(256)
            else:
                B, max_pages = st["table"].shape
                kv = _cache(case, st["pool"], B, st["n_pages"], max_pages)
                kv.table, kv.len = st["table"], st["len"]
                st["pages"] = sb.Pages(kv, mapped=st["mapped"], ref=st["ref"], n_free=st["n_free"])
                st["ws"] = sb.workspace(sb.spec_pages_workspace_bytes(B, st["n_pages"], max_pages))
    st["case"] = case
    return st


def run(st):
    return {"sample": _sample, "filter": _filter, "branch": _branch, "compact": _compact, "copy": _copy}[
        st["case"]["op"]](st)


# ----------------------------------------------------------------- sampling
def _truncate(st):
    """(z in 32 bits, weights in 64 bits, kept) of every row."""
    z = st["z"].float()
    z = torch.where(torch.isnan(z), -math.inf, z)
    rows, V = z.shape
    top = z.amax(1, keepdim=True)
    greedy = st["T"][:, None] == 0
    T = torch.where(greedy, 1.0, st["T"][:, None]).double()
    zs = torch.sort(z, dim=1, descending=True).values
    k = torch.where((st["k"] <= 0) | (st["k"] > V), V, st["k"]).long()[:, None]
    bound = torch.maximum(zs.gather(1, k - 1).double(), top.double() + T * torch.log(st["mp"].double())[:, None])
    ws = torch.where(zs.double() >= bound, torch.exp((zs.double() - top.double()) / T), 0.0)
    cum = ws.cumsum(1)
    reach = torch.searchsorted(cum, st["p"].double()[:, None] * cum[:, -1:]).clamp_max(V - 1)
    nucleus = torch.where(st["p"][:, None] < 1, zs.gather(1, reach).double(), -math.inf)
    keep = (z.double() >= torch.maximum(bound, nucleus)) & (z > -math.inf)
    ids = torch.arange(V, device=z.device)
    first = torch.where(z == top, ids, V).amin(1, keepdim=True)
    keep = torch.where(greedy, ids == first, keep)
    w = torch.where(keep, torch.exp((z.double() - top.double()) / T), 0.0)
    return z, w, keep


def _sample(st):
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        sb.spec_sample(st["z"], st["sampling"], st["u"], st["tokens"], st["ws"], probs=st["probs"])
        return dict(tokens=st["tokens"], probs=st["probs"]) if st["case"]["probs"] else dict(tokens=st["tokens"])
    z, w, keep = _truncate(st)
    cum = w.cumsum(1)
    tot = cum[:, -1:].clone()
    t = torch.searchsorted(cum, st["u"].double() * tot, right=True)
    last = torch.where(keep, torch.arange(z.shape[1], device=z.device), 0).amax(1, keepdim=True)
    tokens = torch.minimum(t, last).to(torch.int32)
    if not st["case"]["probs"]:
        return dict(tokens=tokens)
    return dict(tokens=tokens, probs=(w / tot).float())


def _filter(st):
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        sb.spec_filter_logits(st["z"], st["sampling"], st["out"], st["ws"])
        return st["out"]
    _, _, keep = _truncate(st)
    return torch.where(keep, st["z"], -math.inf)


# -------------------------------------------------------------------- pages
def _books(st):
    return dict(st["pool"], table=st["table"], len=st["len"], mapped=st["mapped"], ref=st["ref"],
                n_free=st["n_free"])


def _put_back(st, rows):
    """The pages of these sequences are returned, their lengths 0."""
    ids = st["table"][rows]
    st["ref"].scatter_add_(0, ids.clamp_min(0).flatten().long(), -(ids >= 0).int().flatten())
    st["table"][rows] = -1
    st["mapped"][rows] = 0
    st["len"][rows] = 0


def _branch(st):
    n = st["case"]["n"]
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        pages, ws = st["pages"], st["ws"]
        sb.spec_pages_free(pages, st["dst"], ws)
        sb.spec_pages_fork(pages, st["src"], st["dst"], ws)
        sb.spec_pages_reserve(pages, n, ws)
        return _books(st)
    table, length, ref = st["table"], st["len"], st["ref"]
    B, P = table.shape
    j = torch.arange(P, device=table.device)[None]
    src, dst = st["src"].long(), st["dst"].long()
    _put_back(st, dst)
    # the first pages of each source, shared
    base = (length[src] + PAGE - 1) // PAGE
    rows = torch.where(j < base[:, None], table[src], -1)
    table[dst], st["mapped"][dst], length[dst] = rows, base, length[src]
    ref.scatter_add_(0, rows.clamp_min(0).flatten().long(), (rows >= 0).int().flatten())
    # pages past the lengths are returned, then the new slots' pages taken
    base = (length + PAGE - 1) // PAGE
    past = (j >= base[:, None]) & (table >= 0)
    ref.scatter_add_(0, table.clamp_min(0).flatten().long(), -past.int().flatten())
    table.masked_fill_(past, -1)
    seq = torch.arange(B, device=table.device)
    writes = length % PAGE > 0
    at = (length // PAGE).clamp_max(P - 1).long()
    page = table.gather(1, at[:, None])[:, 0].clamp_min(0).long()
    writers = torch.zeros_like(ref).scatter_add_(0, page, writes.int())
    lowest = torch.full_like(ref, B).scatter_reduce_(0, page, torch.where(writes, seq, B).int(), "amin")
    copies = writes & ~((ref[page] == writers[page]) & (lowest[page] == seq))
    end = (length + n + PAGE - 1) // PAGE
    takes = (j >= base[:, None]) & (j < end[:, None]) | ((j == at[:, None]) & copies[:, None])
    free = torch.argsort((ref > 0).int(), stable=True)  # lowest numbers first
    nth = (takes.flatten().cumsum(0) - 1).clamp_min(0)
    fresh = free[nth].view(B, P).int()
    new = torch.where(takes, fresh, table)
    _move(st["pool"], st["pool"], page, new.gather(1, at[:, None])[:, 0].long(), (length % PAGE) * copies)
    ref.scatter_add_(0, page, -copies.int())
    ref.scatter_add_(0, new.clamp_min(0).flatten().long(), takes.int().flatten())
    table.copy_(new)
    st["mapped"].copy_(end)
    st["n_free"].copy_((ref == 0).sum())
    return _books(st)


def _move(a, b, src, dst, rows):
    """The first `rows` slots of pages src of pool a to pages dst of pool b, with the pages' scales."""
    some = rows > 0
    src, dst, rows = src[some], dst[some], rows[some]
    held = (torch.arange(PAGE, device=src.device)[None] < rows[:, None])[None, :, None, :, None]
    for name in ("k", "v"):
        x, y = a[name], b[name]
        bits = torch.uint8 if x.dtype == E4M3 else torch.int16
        x, y = x.view(bits), y.view(bits)
        y[:, dst] = torch.where(held, x[:, src], y[:, dst])
        if name + "_scale" in a:
            b[name + "_scale"][:, dst] = a[name + "_scale"][:, src]


def _compact(st):
    st["flat"].copy_(st["first"])  # the books of a fragmented pool
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        sb.spec_pages_compact(st["pages"], st["ws"])
        return _books(st)
    ref, table = st["ref"], st["table"]
    used = ref > 0
    total = used.sum()
    ids = torch.arange(ref.numel(), device=ref.device)
    src = ids[used & (ids >= total)]
    dst = ids[~used & (ids < total)]
    for name in st["pool"]:
        x = st["pool"][name]
        x = x.view(torch.uint8) if x.dtype == E4M3 else x
        x[:, dst] = x[:, src]
    to = ids.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp_min(0).long()].int(), table))
    ref[dst] = ref[src]
    ref[src] = 0
    return _books(st)


def _copy(st):
    if own:
        from speculative_decoding_verification_pass_gb300 import binding as sb
        sb.spec_pages_copy(st["kv"], st["kv_to"], st["src"], st["dst"], st["ws"])
        return st["to"]
    src, dst = st["src"].long(), st["dst"].long()
    for name, x in st["pool"].items():
        y = st["to"][name]
        if x.dtype == E4M3:
            x, y = x.view(torch.uint8), y.view(torch.uint8)
        y[:, dst] = x[:, src]
    return st["to"]


# --------------------------------------------------------------------- work
def _page_bytes(case):
    L, Hkv, hd = SHAPES[case["shape"]]
    return 2 * L * Hkv * (PAGE * hd + 4 * PAGE // BLOCK if case["kv8"] else PAGE * hd * 2)


def work(case):
    if case["op"] in ("sample", "filter"):
        n, e = case["rows"] * case["V"], 4 if case["dtype"] == "f32" else 2
        if case["op"] == "filter":
            return dict(bytes=2.0 * n * e, flops=4.0 * n)
        return dict(bytes=n * e + (4.0 * n if case["probs"] else 0.0), flops=4.0 * n)
    if case["op"] == "branch":  # half a page for each sequence but the first of a group
        pages = case["groups"] * (case["ways"] - 1) * 0.5
    elif case["op"] == "compact":  # the used share of the pages past the used ones' number
        used = max(1, min(case["pages"] - 1, int(case["used"] * case["pages"])))
        pages = used * (case["pages"] - used) / case["pages"]
    else:
        pages = case["pages"]
    return dict(bytes=2.0 * pages * _page_bytes(case), flops=0.0)


# -------------------------------------------------------------------- exact
def exact(case, seed):
    if case["op"] in ("sample", "filter"):
        return _exact_rows(case, seed)
    st = _page_inputs(case, seed)
    return {"branch": _exact_branch, "compact": _exact_compact, "copy": _exact_copy}[case["op"]](case, st)


def _exact_rows(case, seed):
    st = _logit_inputs(case, seed)
    z = st["z"].double().cpu().numpy()
    T, K, P, MP = (st[x].double().cpu().numpy() for x in ("T", "k", "p", "mp"))
    tokens, dist, kept = [], [], []
    for r in range(case["rows"]):
        x = z[r]
        best = int(np.argmax(x))
        if T[r] == 0:
            keep = np.zeros(len(x), bool)
            keep[best] = True
        else:
            keep = np.isfinite(x)
            if MP[r] > 0:
                keep &= (x - x[best]) / T[r] >= np.log(MP[r])
            if 0 < K[r] < len(x):
                keep &= x >= np.partition(x, len(x) - int(K[r]))[len(x) - int(K[r])]
            if P[r] < 1:
                left = np.sort(x[keep])  # ascending: what may be dropped is the lowest mass
                mass = np.cumsum(np.exp((left - x[best]) / T[r]))
                total = mass[-1]
                # left[i] stays if the mass of i and above falls short of, or first reaches, the target
                above = total - mass  # strictly above i
                stay = left[above < P[r] * total]
                keep &= x >= stay[0]
        kept.append(keep)
        if case["op"] == "filter":
            continue
        ids = np.flatnonzero(keep)
        w = np.exp((x[ids] - x[best]) / (T[r] if T[r] else 1.0))
        c = np.cumsum(w)
        u = st["u"][r].double().cpu().numpy()
        tokens.append([int(ids[min(int((c <= v * c[-1]).sum()), len(ids) - 1)]) for v in u])
        if case["probs"]:
            q = np.zeros(len(x))
            q[ids] = w / c[-1]
            dist.append(torch.from_numpy(q))
    if case["op"] == "filter":
        return torch.where(torch.from_numpy(np.stack(kept)).to(st["z"].device), st["z"].double(), -math.inf)
    out = dict(tokens=torch.tensor(tokens, dtype=torch.int32))
    if case["probs"]:
        out["probs"] = torch.stack(dist)
    return out


def _exact_pages(pool, moves):
    """moves: (source, destination, slots) one after another."""
    for name, x in pool.items():
        for a, b, slots in moves:
            if name.endswith("scale"):
                x[:, b] = x[:, a]
            else:
                x.view(torch.uint8)[:, b, :, :slots] = x.view(torch.uint8)[:, a, :, :slots]
    return pool


def _held(st):
    table, mapped = st["table"].cpu().tolist(), st["mapped"].cpu().tolist()
    return [row[:m] for row, m in zip(table, mapped)]


def _exact_books(st, held, lens):
    table = torch.full(st["table"].shape, -1, dtype=torch.int32)
    ref = [0] * st["n_pages"]
    for b, row in enumerate(held):
        for i, p in enumerate(row):
            table[b, i] = p
            ref[p] += 1
    ints = lambda x: torch.tensor(x, dtype=torch.int32)
    return dict(st["pool"], table=table, len=ints(lens), mapped=ints([len(x) for x in held]), ref=ints(ref),
                n_free=ints([ref.count(0)]))


def _exact_branch(case, st):
    held, lens = _held(st), st["len"].cpu().tolist()
    for a, b in zip(st["src"].cpu().tolist(), st["dst"].cpu().tolist()):
        held[b], lens[b] = list(held[a][: -(-lens[a] // PAGE)]), lens[a]
    held = [row[: -(-x // PAGE)] for row, x in zip(held, lens)]
    users = {}
    for b, row in enumerate(held):
        for p in row:
            users.setdefault(p, []).append(b)
    writers = {}
    for b, row in enumerate(held):
        if lens[b] % PAGE:
            writers.setdefault(row[-1], []).append(b)
    free = [p for p in range(st["n_pages"]) if p not in users]
    moves = []
    for b, row in enumerate(held):
        if lens[b] % PAGE:
            p = row[-1]
            if users[p] != writers[p] or writers[p][0] != b:
                row[-1] = free.pop(0)
                moves.append((p, row[-1], lens[b] % PAGE))
        while len(row) * PAGE < lens[b] + case["n"]:
            row.append(free.pop(0))
    _exact_pages(st["pool"], moves)
    return _exact_books(st, held, lens)


def _exact_compact(case, st):
    held, lens = _held(st), st["len"].cpu().tolist()
    used = sorted({p for row in held for p in row})
    gaps = sorted(set(range(len(used))) - set(used))
    to = dict(zip([p for p in used if p >= len(used)], gaps))
    _exact_pages(st["pool"], [(a, b, PAGE) for a, b in to.items()])
    return _exact_books(st, [[to.get(p, p) for p in row] for row in held], lens)


def _exact_copy(case, st):
    for a, b in zip(st["src"].cpu().tolist(), st["dst"].cpu().tolist()):
        for name, x in st["pool"].items():
            st["to"][name].view(torch.uint8)[:, b] = x.view(torch.uint8)[:, a]
    return st["to"]
