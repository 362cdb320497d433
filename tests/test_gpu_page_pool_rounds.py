"""The device page pool within rounds, on a GPU: passes right behind the calls
that write the tables, pools that run short in the middle of a round, and
sequences that sit one out.
"""
import numpy as np
import pytest
import torch

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
        row = self.kv.table[b].tolist()
        rows = [row[t // 64] for t in range(slots)]
        page, at = torch.tensor(rows, device="cuda"), torch.arange(slots, device="cuda") % 64
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
