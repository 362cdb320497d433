"""Truncated sampling at the ends of fp32: subnormal logits and temperatures,
against the fp64 oracle with the tolerances derived in test_gpu_sample.
"""
import numpy as np
import pytest
import torch

from oracle import sample as OS
from speculative_decoding_verification_pass_gb300 import binding as sb
from speculative_decoding_verification_pass_gb300 import workloads as wl
from test_gpu_sample import _cuda, _f32, _rows, check

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -149  # the smallest fp32 subnormal


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("V", [3, 900, 40000])
@pytest.mark.parametrize("bf16", [False, True])
def test_the_largest_of_subnormal_logits(V, bf16):
    """Greedy rows and rows of the k largest, all of whose logits are nearer to zero than the least normal number:
    they differ, though a product would flush them."""
    g = wl.rng(V, 60)
    step = TINY * (65536 if bf16 else 1)  # bf16's own least subnormal
    z = step * g.integers(-100, 101, size=(8, V))
    z[1] = -step * g.integers(1, 101, size=V)
    z[2] = step * g.integers(0, 2, size=V)
    z[3] = -0.0
    z[4] = 0.0
    z[4, V // 2] = step
    z[5] = -step
    z[5, V - 1] = 0.0
    z[6, 1] = 1.0
    z[7] = np.where(g.random(V) < 0.5, -np.inf, z[7])
    z[7, 0] = -step
    z = z.astype(np.float32)
    check(z, [(0.0, 0, 1.0, 0.0)] * 8, bf16=bf16, seed=1)
    for k in (1, 2, V // 3 + 1, max(V - 1, 1)):
        check(z, [(1.0, k, 1.0, 0.0)] * 8, bf16=bf16, seed=2)
    check(z, [(0.7, V // 3 + 1, 0.5, 0.0)] * 4 + [(1.0, 0, 0.6, 0.0)] * 2 + [(1.0, 0, 1.0, 1.0)] * 2, bf16=bf16, seed=3,
          least=0)


@pytest.mark.parametrize("V", [700, 40000])
@pytest.mark.parametrize("T", [2.0 ** -126, 3e-38, 1e-37, 1e-30, 2e-29, 1.7e-29, 1e-28])
def test_temperatures_that_part_subnormal_logits(V, T):
    """The least normal temperatures, where subnormal logits are as far apart as any, and the first at which they weigh
    the same."""
    g = wl.rng(V, 61)
    z = np.clip(T * 3 * g.standard_normal((6, V)), -T * 20, None)
    z[:, ::3] = TINY * g.integers(-2 ** 23, 2 ** 23, size=z[:, ::3].shape)
    z = z.astype(np.float32)
    check(z, [(T, 0, 1.0, 0.0), (T, 50, 0.9, 0.0), (T, 0, 0.8, 0.0), (T, 0, 1.0, 0.2), (T, V // 2, 0.95, 0.0),
              (T, 0, 0.3, 0.01)], seed=4)


def test_subnormal_temperatures_are_greedy():
    V = 5000
    z = _cuda(np.float32(3.0) * wl.rng(1, 62).standard_normal((4, V)).astype(np.float32))
    u, ws = _cuda(wl.uniforms(5, 4, 3)), sb.workspace(256)
    tok = torch.empty(4, 3, dtype=torch.int32, device="cuda")
    for s in (sb.Sampling(temperature=torch.full((4,), 1e-40, device="cuda")), sb.Sampling(1e-45), sb.Sampling(1.1e-38)):
        sb.spec_sample(z, s, u, tok, ws)
        assert torch.equal(tok.long(), z.argmax(1)[:, None].expand(4, 3))


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_pass_through_bit_for_bit(bf16):
    """Kept logits are the row's own, subnormal ones too; so is a row with a set out of range."""
    V = 3001
    z = (TINY * 65536 * wl.rng(2, 63).integers(-100, 101, size=(3, V))).astype(np.float32)
    z[2] = np.float32(_f32(1.0))
    z[2, ::2] = z[0, ::2]
    t, _, _ = _rows(z, bf16, 1)
    ws, out = sb.workspace(256), torch.empty(3, V, dtype=t.dtype, device="cuda")
    bits = torch.int16 if bf16 else torch.int32
    for s, status in ((sb.Sampling(), 0), (sb.Sampling(temperature=torch.full((3,), -1.0, device="cuda")), sb.DEV_BAD_PARAM)):
        sb.spec_filter_logits(t, s, out, ws)
        assert sb.spec_device_status(ws)[1] == status
        assert torch.equal(out.view(bits), t.contiguous().view(bits))


@pytest.mark.parametrize("far", [-29500.0, -22500.0, 21950.0, 25000.0, 29900.0])
def test_rows_whose_bins_are_by_difference(far):
    """|M| / T log2(e) between 21900 and 30000: weights by the 32-bit steps, bins by differences from M."""
    V = 30000
    g = wl.rng(3, 64)
    par = [(1.0, 0, 0.9, 0.0), (0.7, 2000, 0.95, 0.0), (0.5, 0, 1.0, 0.0), (2.0, 0, 0.4, 0.0), (1.0, 5000, 1.0, 0.0),
           (1.3, 0, 0.99, 1e-4)]
    T = np.array([_f32(p[0]) for p in par])
    z = 2.0 * T[:, None] * g.standard_normal((len(par), V))
    z += (far * T * np.log(2.0) - z.max(1))[:, None]
    check(z.astype(np.float32), par, seed=6, draws=4)


@pytest.mark.parametrize("V", [183325, 262144])
@pytest.mark.parametrize("gap", [20.0, 24.0, 25.0, 25.8, 27.0, 40.0])
def test_tails_below_the_units_of_the_sum(V, gap):
    """One id and a quarter of a million others, each about a unit of the sum or less: half a unit, 2^-35.5 of the
    largest, times V on the total, beside what a probability is off by itself."""
    z = (0.2 * wl.rng(7, 65).standard_normal((2, V))).astype(np.float32)
    z[:, 4] = gap
    probs = torch.empty(2, V, device="cuda")
    tok = torch.empty(2, 2, dtype=torch.int32, device="cuda")
    sb.spec_sample(_cuda(z), sb.Sampling(), _cuda(np.float32([[0.5, 0.9], [0.1, 0.99]])), tok, sb.workspace(256),
                   probs=probs)
    for got, x in zip(probs.double().cpu().numpy(), z):
        np.testing.assert_allclose(got, OS.truncate(x, 1.0).p, rtol=2.0 ** -21.4 + V * 2.0 ** -35.5)
    assert gap < 24 or (tok == 4).all()
