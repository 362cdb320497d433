"""What the page pool's Python calls hand to the library, without a GPU."""
import types

import pytest
import torch

from speculative_decoding_verification_pass_gb300 import binding as sb


class _Buffer:
    """A tensor's address, and nothing else of it."""

    def __init__(self, address):
        self.address = address

    def data_ptr(self):
        return self.address

    def get_device(self):
        return 0


class _Derived8(sb.KV8Cache):
    pass


class _Derived16(sb.PagedKVCache):
    pass


def _bare(cls):
    """A cache object without its buffers' memory."""
    kv = object.__new__(cls)
    names = ("k", "v", "k_scale", "v_scale") if issubclass(cls, sb.KV8Cache) else ("k", "v")
    kv.__dict__.update({x: _Buffer(4096 * (i + 1)) for i, x in enumerate(names)},
                       cfg=sb.ModelConfig(2, 256, 4, 2, 256, 1000), n_pages=9, pool=None)
    return kv


@pytest.mark.parametrize("cls", [sb.KV8Cache, _Derived8])
def test_every_8_bit_cache_goes_with_its_scales(cls):
    """Without them the library takes rows of twice the bytes, and its copies leave the buffers."""
    d = sb._page_data(_bare(cls))
    assert (d.k, d.v, d.k_scale, d.v_scale, d.n_pages) == (4096, 8192, 12288, 16384, 9)


@pytest.mark.parametrize("cls", [sb.PagedKVCache, _Derived16])
def test_a_bf16_cache_goes_without(cls):
    d = sb._page_data(_bare(cls))
    assert (d.k, d.v, d.k_scale, d.v_scale, d.n_pages) == (4096, 8192, None, None, 9)


@pytest.mark.parametrize("a,b", [(sb.KV8Cache, sb.PagedKVCache), (_Derived8, _Derived16), (_Derived16, sb.KV8Cache)])
def test_copies_between_kinds_are_refused(a, b):
    ids = types.SimpleNamespace(numel=lambda: 1)
    with pytest.raises(ValueError, match="one kind"):
        sb.spec_pages_copy(_bare(a), _bare(b), ids, ids, None)


@pytest.mark.parametrize("a,b", [(sb.KV8Cache, _Derived8), (_Derived16, sb.PagedKVCache)])
def test_a_derived_cache_is_of_its_base_kind(a, b):
    """Past the check of kinds: the next one, of the workspace's device, refuses this call."""
    ws = types.SimpleNamespace(get_device=lambda: -1, nbytes=256)
    ids = types.SimpleNamespace(numel=lambda: 1)
    with pytest.raises(ValueError, match="cuda:0"):
        sb.spec_pages_copy(_bare(a), _bare(b), ids, ids, ws)


def _rows(cfg, pages, dtype=torch.bfloat16):
    return torch.zeros(cfg.n_layers, pages, cfg.n_kv_heads, 64, cfg.head_dim, dtype=dtype)


def test_a_cache_is_made_around_v_alone():
    """The other buffers go to the device of the one given."""
    cfg = sb.ModelConfig(2, 256, 4, 2, 256, 1000)
    v = _rows(cfg, 3)
    kv = sb.PagedKVCache(cfg, 2, 3, 4, v=v)
    assert kv.v is v and kv.k.shape == v.shape and kv.k.device == kv.len.device == v.device
    with pytest.raises(ValueError):
        sb.PagedKVCache(cfg, 2, 4, 4, v=v)


def test_buffers_put_in_place_later_are_looked_at():
    """Kernels go by the cache's sizes: a buffer of others is refused when it is put there."""
    cfg = sb.ModelConfig(2, 256, 4, 2, 256, 1000)
    kv = sb.PagedKVCache(cfg, 2, 5, 4, device="cpu")
    k, table, length = kv.k, kv.table, kv.len
    ints = lambda *n: torch.zeros(n, dtype=torch.int32)
    for name, bad in (("k", _rows(cfg, 4)), ("v", _rows(cfg, 5, torch.float16)), ("v", _rows(cfg, 10)[:, ::2]),
                      ("v", torch.empty(kv.v.shape, dtype=torch.bfloat16, device="meta")), ("table", ints(2, 3)),
                      ("table", ints(2, 4).long()), ("table", ints(4, 2).t()), ("len", ints(3)),
                      ("len", ints(2).float())):
        with pytest.raises(ValueError, match=name):
            setattr(kv, name, bad)
    assert kv.k is k and kv.table is table and kv.len is length
    good = _rows(cfg, 5)
    kv.v, kv.table, kv.len = good, ints(2, 4), ints(4)[:2]
    assert kv.v is good
    with pytest.raises(ValueError, match="CUDA"):  # the books are kept by kernels
        sb.Pages(kv, mapped=ints(2), ref=ints(5), n_free=ints(1))


def test_books_put_in_place_later_are_looked_at():
    p = object.__new__(sb.Pages)
    p.__dict__.update(kv=types.SimpleNamespace(batch=2, n_pages=5, len=torch.zeros(2, dtype=torch.int32)))
    ints = lambda n: torch.zeros(n, dtype=torch.int32)
    for name, n in (("mapped", 2), ("ref", 5), ("n_free", 1)):
        for bad in (ints(n + 1), ints(n).long(), ints(2 * n)[::2] if n > 1 else ints(0), ints(n).to("meta")):
            with pytest.raises(ValueError, match=name):
                setattr(p, name, bad)
        setattr(p, name, ints(n))
