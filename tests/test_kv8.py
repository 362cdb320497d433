"""The 8-bit cache on the CPU: the oracle's rounding and scales, sizes, refusals of the entry points."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv8 as O8


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decoding_verification_pass_gb300 import binding
    return binding


def test_oracle_rounding_is_the_formats():
    every = O8.e4m3_of_byte(np.arange(256))
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(every, t)
    x = np.concatenate([every[~np.isnan(every)], np.random.default_rng(1).standard_normal(20000) * 60,
                        np.random.default_rng(2).standard_normal(20000) * 0.01])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O8.round_e4m3(x), want)
    v = np.sort(every[~np.isnan(every)])
    mid = (np.unique(v)[1:] + np.unique(v)[:-1]) / 2  # ties go to the even fraction
    want = torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O8.round_e4m3(mid), want)


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.5, 1), (1.75, -8), (1.7500001, -7), (0.0, -40), (1e-30, -40),
                                   (1e30, 40), (3.5, -7)])
def test_oracle_scale(top, e):
    assert O8.scale_of([0.0, -top, np.inf, np.nan]) == 2.0 ** e


def test_oracle_growth_and_commit_keep_values():
    """Re-rounding at a larger power of two keeps a row but for subnormals; a commit moves values."""
    g = np.random.default_rng(3)
    r = O8.Rows(2, 64, 64)
    a, b = g.standard_normal((5, 2, 64)), 40 * g.standard_normal((9, 2, 64))
    r.append(3, a)
    one = r.value(8)
    r.append(8, b)
    s = r.scale[:, 0].max()
    assert np.abs(r.value(8)[:, 3:] - one[:, 3:]).max() <= s * 2.0 ** -10
    before = r.value(17)
    r.commit(8, [2, 5, 8])
    after = r.value(12)
    assert np.abs(after[:, 9:12] - before[:, [10, 13, 16]]).max() <= r.scale.max() * 2.0 ** -10
    np.testing.assert_array_equal(after[:, :9], before[:, :9])


def test_sizes(lib):
    c = lib.LLAMA_8B
    L = lib.lib()
    assert L.spec_kv8_bytes(ctypes.byref(c.c()), 10) == 32 * 10 * 8 * 64 * 128
    assert L.spec_kv8_scale_bytes(ctypes.byref(c.c()), 10) == 32 * 10 * 8 * 4 * 4
    assert lib.spec_kv8_workspace_bytes(c, 2, 5) > lib.spec_kv8_workspace_bytes(c, 1, 5) > 0
    assert lib.spec_kv8_workspace_bytes(c, 1, 0) == 0
    assert lib.spec_kv8_workspace_bytes(lib.ModelConfig(0, 256, 0, 0, 0, 10), 1, 1) == 0


def _cache(lib, **kw):
    f = dict(k=4096, v=4096, k_scale=4096, v_scale=4096, len=4096, table=4096, batch=0, n_pages=4, max_pages=4)
    f.update(kw)
    return ctypes.byref(lib.spec_kv8_cache(*f.values()))


def test_refusals(lib):
    """Every bad argument is refused before any CUDA call; an empty batch is a no-op (no GPU here)."""
    L = lib.lib()
    P = ctypes.c_void_p
    ok = P(4096)
    c = ctypes.byref(lib.ModelConfig(2, 256, 4, 2, 256, 1000).c())
    E, S = lib.SPEC_EINVAL, lib.SPEC_ESIZE
    rope = lib.spec_rope_config(64, 0, 0, 1e4, 1.0, 1.0, 4.0)

    def append(cfg=c, kv=None, layer=0, n=5, q=ok, q_ld=256, k=ok, k_ld=128, v=ok, v_ld=128, f32=0, rc=rope, tab=ok,
               out=ok, ws=ok):
        return L.spec_kv8_append(cfg, kv or _cache(lib), layer, n, q, q_ld, k, k_ld, v, v_ld, f32, None,
                                 ctypes.byref(rc) if rc else None, tab, out, ws, None)

    def attend(cfg=c, kv=None, layer=0, n=5, q=ok, q_ld=256, anc=None, scale=0.0, o=ok, o_ld=256, ws=ok):
        return L.spec_kv8_attention(cfg, kv or _cache(lib), layer, n, q, q_ld, anc, scale, o, o_ld, ws, None)

    def commit(cfg=c, kv=None, path=ok, m=ok, n=5, ws=ok):
        return L.spec_kv8_tree_commit(cfg, kv or _cache(lib), path, m, n, ws, None)

    assert append() == attend() == commit() == lib.SPEC_OK
    assert L.spec_kv8_advance(_cache(lib), 5, ok, None) == lib.SPEC_OK
    bad_caches = [(_cache(lib, len=0), E), (_cache(lib, table=0), E), (_cache(lib, batch=-1), E),
                  (_cache(lib, n_pages=0), E), (_cache(lib, max_pages=0), E), (_cache(lib, batch=65536), S),
                  (_cache(lib, max_pages=16385), S), (_cache(lib, len=4098), E), (_cache(lib, table=4097), E)]
    for kv, want in bad_caches:
        assert append(kv=kv) == attend(kv=kv) == commit(kv=kv) == want
        assert L.spec_kv8_advance(kv, 5, ok, None) == want
        assert L.spec_kv8_truncate(kv, ok, 4, ok, None) == want
    for kv, want in [(_cache(lib, k=0), E), (_cache(lib, v=0), E), (_cache(lib, k_scale=0), E),
                     (_cache(lib, v_scale=0), E), (_cache(lib, k=4104), E), (_cache(lib, v_scale=4100), E),
                     (_cache(lib, n_pages=1 << 24), S)]:
        assert append(kv=kv) == attend(kv=kv) == commit(kv=kv) == want
    for kw in (dict(cfg=None), dict(q=None), dict(k=None), dict(v=None), dict(rc=None), dict(tab=None), dict(out=None),
               dict(ws=None), dict(layer=-1), dict(layer=2), dict(n=0), dict(q_ld=248), dict(q_ld=260), dict(k_ld=120),
               dict(v=P(4104)), dict(out=P(4098)), dict(k_ld=130, f32=1), dict(tab=P(4100)),
               dict(rc=lib.spec_rope_config(128, 0, 0, 1e4, 1.0, 1.0, 4.0)),
               dict(rc=lib.spec_rope_config(62, 0, 0, 1e4, 1.0, 1.0, 4.0)),
               dict(rc=lib.spec_rope_config(0, 0, 0, 1e4, 1.0, 1.0, 4.0)),
               dict(rc=lib.spec_rope_config(64, 0, 0, 1.0, 1.0, 1.0, 4.0)),
               dict(rc=lib.spec_rope_config(64, 0, 0, 1e4, 0.5, 1.0, 4.0)),
               dict(rc=lib.spec_rope_config(64, 0, 8192, 1e4, 2.0, 4.0, 4.0)),
               dict(rc=lib.spec_rope_config(64, 0, -1, 1e4, 2.0, 1.0, 4.0))):
        assert append(**kw) == E, kw
    assert append(n=129) == S
    assert append(k_ld=132, f32=1) == lib.SPEC_OK
    for kw in (dict(cfg=None), dict(q=None), dict(o=None), dict(ws=None), dict(layer=2), dict(n=0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q_ld=255), dict(o_ld=260), dict(o=P(4098))):
        assert attend(**kw) == E, kw
    assert attend(n=129) == S and attend(n=65, anc=ok) == S and attend(n=65) == lib.SPEC_OK
    for kw in (dict(cfg=None), dict(path=None), dict(m=None), dict(ws=None), dict(n=0)):
        assert commit(**kw) == E, kw
    assert commit(n=65) == S
    assert commit(path=P(4098)) == commit(m=P(4097)) == commit(ws=P(4099)) == E
    assert attend(anc=P(4100)) == attend(ws=P(4097)) == append(ws=P(4098)) == E
    big = ctypes.byref(lib.ModelConfig(70000, 256, 4, 2, 256, 1000).c())  # layers past a launch's grid
    assert append(cfg=big) == attend(cfg=big) == commit(cfg=big) == S
    assert L.spec_kv8_advance(_cache(lib), 0, ok, None) == E
    assert L.spec_kv8_advance(_cache(lib), 129, ok, None) == S
    assert L.spec_rope_table(ctypes.byref(rope), None, None) == E
    assert L.spec_rope_table(ctypes.byref(rope), P(4100), None) == E
    assert L.spec_rope_table(None, ok, None) == E
    assert L.spec_verify_forward_kv8(None, ok, None, None, 1, 5, _cache(lib), ok, ok, 1 << 30, None) == E


def test_a_changed_struct_is_its_callers_own(lib):
    """ModelConfig.c() may be edited: neither the config nor a later call sees it."""
    cfg = lib.ModelConfig(32, 4096, 32, 8, 14336, 128256)
    want = lib.spec_kv_bytes(cfg, 1, 64), lib.spec_kv8_workspace_bytes(cfg, 1, 5)
    cfg._kept()
    mine = cfg.c()
    mine.n_layers = 2
    assert cfg.c().n_layers == cfg._kept().n_layers == 32
    assert (lib.spec_kv_bytes(cfg, 1, 64), lib.spec_kv8_workspace_bytes(cfg, 1, 5)) == want
    assert lib.lib().spec_kv_bytes(ctypes.byref(mine), 1, 64) == want[0] // 16


def test_pass_refuses_another_models_cache(lib, monkeypatch):
    """spec_verify_forward_kv8 compares the cache, the logits and the device with the handle's model before any
    call of the library (which sees neither buffer's size)."""
    shape = dict(n_layers=2, d_model=256, n_heads=4, n_kv_heads=2, d_ffn=256, vocab=1000)

    def call(handle=77, model_dev=-1, vocab=1000, **cache):  # tensors of the CPU: device -1
        kv = object.__new__(lib.KV8Cache)
        object.__setattr__(kv, "cfg", lib.ModelConfig(**{**shape, **cache}))
        object.__setattr__(kv, "len", torch.zeros(1, dtype=torch.int32))
        object.__setattr__(kv, "pool", None)
        monkeypatch.setitem(lib._MODELS, 77, (lib.ModelConfig(**shape), model_dev))
        lib.spec_verify_forward_kv8(handle, torch.zeros(1, 3, dtype=torch.int32), 1, 3, kv,
                                    torch.zeros(1, 3, vocab), torch.zeros(4096, dtype=torch.uint8))

    def never():
        raise AssertionError("a call of the library")

    monkeypatch.setattr(lib, "lib", never)
    for kw, match in ((dict(n_layers=1), "cache"), (dict(n_kv_heads=1), "cache"), (dict(n_kv_heads=4), "cache"),
                      (dict(d_model=512), "cache"), (dict(n_layers=3), "cache"), (dict(vocab=999), "logits"),
                      (dict(handle=78), "live model"), (dict(handle=None), "live model"),
                      (dict(model_dev=1), "device")):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    with pytest.raises((AssertionError, RuntimeError)):  # nothing to refuse: on to the library
        call()


def test_pass_refuses_a_model_without_layers(lib, monkeypatch):
    """The handle of an LM head alone has no heads to compare."""
    kv = object.__new__(lib.KV8Cache)
    object.__setattr__(kv, "cfg", lib.ModelConfig(2, 256, 4, 2, 256, 1000))
    object.__setattr__(kv, "pool", None)
    monkeypatch.setitem(lib._MODELS, 77, (lib.ModelConfig(0, 256, 0, 0, 0, 1000), -1))
    with pytest.raises(ValueError, match="cache"):
        lib.spec_verify_forward_kv8(77, None, 1, 3, kv, None, None)
