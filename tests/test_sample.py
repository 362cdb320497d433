"""Truncated sampling without a GPU: the oracle pinned by enumeration and by the
acceptance oracle's own nucleus, and the refusals of the entry points."""
import ctypes
import itertools

import numpy as np
import pytest

from oracle import accept as OA
from oracle import sample as OS


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decoding_verification_pass_gb300 import binding
    return binding


def test_oracle_against_enumeration():
    """Every value pattern of four logits (ties included) against the rules written as sets."""
    for z in itertools.product([0.0, 0.7, 1.9], repeat=4):
        z = np.array(z)
        p = np.exp(z - z.max())
        p /= p.sum()
        for k, top_p, min_p in itertools.product([0, 1, 2, 3], [0.3, 0.62, 1.0], [0.0, 0.4, 1.0]):
            keep = {x for x in range(4) if p[x] >= min_p * p.max() * (1 - 1e-12)}
            if k:
                keep &= {x for x in range(4) if sum(z[y] > z[x] for y in range(4)) < k}
            if top_p < 1:
                tot = sum(p[x] for x in keep)
                keep = {x for x in keep if sum(p[y] for y in keep if z[y] > z[x]) < top_p * tot}
            got = OS.truncate(z, 1.0, k, top_p, min_p)
            assert set(np.flatnonzero(got.keep)) == keep, (z, k, top_p, min_p)
            np.testing.assert_allclose(got.p, [p[x] / sum(p[y] for y in keep) if x in keep else 0 for x in range(4)])


def test_oracle_top_p_is_the_acceptance_nucleus():
    rng = np.random.default_rng(3)
    for _ in range(20):
        z = rng.normal(size=200) * 2
        for top_p in (0.1, 0.5, 0.9):
            np.testing.assert_allclose(OS.truncate(z, 0.7, 0, top_p).p, OA.target_dist(z, 0.7, top_p)[0], atol=1e-15)


def test_oracle_draws_by_a_grid_of_uniforms():
    z = np.array([0.0, 1.0, -np.inf, 0.5, 2.0, np.nan])
    kept = OS.truncate(z, 0.8, 3)
    n = 4000
    got = np.bincount([OS.draw(kept, (i + 0.5) / n)[0] for i in range(n)], minlength=6)
    assert np.abs(got / n - kept.p).max() <= 1 / n
    assert OS.truncate([np.nan, -np.inf], 1.0) is None
    assert OS.truncate([1.0, 3.0, 3.0], 0.0).keep.tolist() == [False, True, False]


def test_refusals(lib):
    L = lib.lib()
    fake = ctypes.c_void_p(4096)

    def sampling(t=1.0, k=0, p=1.0, m=0.0, sets=1, dt=None):
        return ctypes.byref(lib.spec_sampling(t, k, p, m, dt, None, None, None, sets))

    def sample(z=fake, ld=10, rows=1, vocab=10, s=sampling(), u=fake, draws=1, tok=fake, probs=None, pld=10, ws=fake):
        return L.spec_sample(z, ld, 0, rows, vocab, s, u, draws, tok, probs, pld, ws, None)

    def filt(z=fake, ld=10, bf16=0, rows=1, vocab=10, s=sampling(), out=fake, old=10, ws=fake):
        return L.spec_filter_logits(z, ld, bf16, rows, vocab, s, out, old, ws, None)

    assert sample(rows=0) == lib.SPEC_OK and filt(rows=0) == lib.SPEC_OK
    for f in (sample, filt):
        for bad in (dict(z=None), dict(ws=None), dict(s=None), dict(ld=9), dict(rows=-1), dict(vocab=0),
                    dict(z=ctypes.c_void_p(4098)), dict(ws=ctypes.c_void_p(4098)), dict(s=sampling(t=-1.0)),
                    dict(s=sampling(t=float("nan"))), dict(s=sampling(t=float("inf"))), dict(s=sampling(k=-1)),
                    dict(s=sampling(p=0.0)), dict(s=sampling(p=1.5)), dict(s=sampling(p=float("nan"))),
                    dict(s=sampling(m=-0.1)), dict(s=sampling(m=1.1)), dict(s=sampling(sets=0)),
                    dict(s=sampling(dt=4098))):
            assert f(**bad) == lib.SPEC_EINVAL, bad
        assert f(rows=65536) == lib.SPEC_ESIZE
        assert f(vocab=(1 << 18) + 1, ld=1 << 19) == lib.SPEC_ESIZE
    for bad in (dict(u=None), dict(tok=None), dict(draws=0), dict(probs=fake, pld=9), dict(probs=ctypes.c_void_p(4098)),
                dict(tok=ctypes.c_void_p(4098)), dict(u=ctypes.c_void_p(4098))):
        assert sample(**bad) == lib.SPEC_EINVAL, bad
    assert sample(draws=65) == lib.SPEC_ESIZE
    for bad in (dict(out=None), dict(old=9), dict(old=11), dict(out=ctypes.c_void_p(4098), old=11)):
        assert filt(**bad) == lib.SPEC_EINVAL, bad  # (old = 11: in place with another row distance)
    assert filt(bf16=1, out=ctypes.c_void_p(4097)) == lib.SPEC_EINVAL
    # a scalar out of range does not matter where the array goes before it
    assert filt(rows=0, s=sampling(t=-1.0, dt=4096)) == lib.SPEC_OK


def test_python_refusals(lib):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        lib.Sampling(rows_per_set=0)
    with pytest.raises(ValueError):
        lib.Sampling(temperature=torch.ones(3))  # not on the GPU
    with pytest.raises(ValueError):
        lib.spec_sample(torch.zeros(2, 8), lib.Sampling(), torch.zeros(2, 1), torch.zeros(2, 1, dtype=torch.int32),
                        torch.zeros(256, dtype=torch.uint8))


def test_probs_over_the_logits_are_refused(lib):
    fake = ctypes.c_void_p(4096)
    s = ctypes.byref(lib.spec_sampling(1.0, 0, 1.0, 0.0, None, None, None, None, 1))
    other = ctypes.c_void_p(8192)
    assert lib.lib().spec_sample(fake, 10, 0, 0, 10, s, other, 1, other, fake, 10, other, None) == lib.SPEC_EINVAL
    assert lib.lib().spec_sample(fake, 10, 0, 0, 10, s, other, 1, other, other, 10, other, None) == lib.SPEC_OK
