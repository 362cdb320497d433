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
