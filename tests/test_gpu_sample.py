"""GPU parity of truncated sampling and of the filter with the fp64 oracle.

Tokens and kept sets must be the oracle's.  A weight is (1 + t) 2^e with t off
by at most 2^-23.6 of 1 + t: g, at most 1/2, is rounded by 2^-26 twice and so 2^g by
2^-25 ln 2 sqrt 2, the polynomial's last step rounds t by 2^-26, and what goes
before it adds 2^-27; 1 + t >= 0.707.  In fixed point it is off by half a unit
more, 2^-36 of the row's largest.  A border between
two ids' cumulative masses is then off by at most 2 x 2^-23.6 + V 2^-35 of
the total: a decision that near to one is not compared (it is counted, and
rare by the sizes below).  Probabilities: 2^-23.6 of the weight and as much of
the total, and three fp32 roundings (the weight, 1 / total, the product) of
2^-24: 2^-21.4 in all; below 2^-120 of the largest they may be flushed.
"""
import numpy as np
import pytest
import torch

from oracle import accept as OA
from oracle import sample as OS
from speculative_decoding_verification_pass_gb300 import binding as sb
from speculative_decoding_verification_pass_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def margin(V):
    return 2 * 2.0 ** -23.6 + V * 2.0 ** -35


def _cuda(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).cuda()


def _rows(z, bf16, pad, fill=7.0):
    """The rows on the device, `pad` elements of something else between them; their values as the device sees them."""
    rows, V = z.shape
    t = torch.full((rows, V + pad), fill, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    t[:, :V] = _cuda(z)
    return t[:, :V], t[:, :V].double().cpu().numpy(), t


def _sampling(par, rows_per_set=1):
    T, k, p, m = zip(*par)
    return sb.Sampling(_cuda(T, torch.float32), _cuda(k, torch.int32), _cuda(p, torch.float32),
                       _cuda(m, torch.float32), rows_per_set=rows_per_set)


def _f32(x):
    return float(np.float32(x))


def check(z, par, bf16=False, pad=0, draws=3, seed=0, status=0, rows_per_set=1, least=1):
    """spec_sample and spec_filter_logits on rows z with the parameter sets par; how many decisions were compared."""
    rows, V = z.shape
    t, seen, whole = _rows(z, bf16, pad)
    u = wl.uniforms(seed, rows, draws)
    ws = sb.workspace(256)
    s = _sampling(par, rows_per_set)
    tok = torch.full((rows, draws), -9, dtype=torch.int32, device="cuda")
    probs = torch.full((rows, V + pad), 5.0, device="cuda")
    before = whole.clone()
    sb.spec_sample(t, s, _cuda(u), tok, ws, probs=probs[:, :V])
    assert sb.spec_device_status(ws)[1] == status
    bits = torch.int16 if bf16 else torch.int32
    assert torch.equal(whole.view(bits), before.view(bits))
    alone = torch.full_like(tok, -9)
    sb.spec_sample(t, s, _cuda(u), alone, ws)
    assert torch.equal(tok, alone)  # the same draws without the distribution
    out = torch.full_like(whole, 3.0)
    sb.spec_filter_logits(t, s, out[:, :V], ws)
    sb.spec_filter_logits(t, s, t, ws)  # in place
    sb.spec_device_status(ws)
    assert torch.equal(out[:, :V], t)
    if pad:
        assert (out[:, V:] == 3.0).all() and (whole[:, V:] == 7.0).all() and (probs[:, V:] == 5.0).all()
    tok, probs, out = tok.cpu().numpy(), probs[:, :V].double().cpu().numpy(), out[:, :V].double().cpu().numpy()
    compared = 0
    for r in range(rows):
        T, k, p, m = par[r // rows_per_set]
        ref = OS.truncate(seen[r], _f32(T), k, _f32(p), _f32(m))
        if ref is None:
            assert (tok[r] == -1).all() and (probs[r] == 0).all() and (out[r] == -np.inf).all()
            continue
        if ref.margin < margin(V):
            continue
        got = out[r] > -np.inf
        assert (got == ref.keep).all(), (r, par[r // rows_per_set], got.sum(), ref.keep.sum())
        assert (out[r][got] == seen[r][got]).all()
        near = ref.p < 2.0 ** -120
        np.testing.assert_allclose(probs[r][~near], ref.p[~near], rtol=2.0 ** -21.4)
        assert (probs[r][near] <= 2.0 ** -119).all() and (probs[r][~ref.keep] == 0).all()
        for d in range(draws):
            want, far = OS.draw(ref, float(u[r, d]))
            if far > margin(V):
                compared += 1
                assert tok[r, d] == want, (r, d, par[r // rows_per_set], far)
    assert compared >= least, compared
    return compared


ALL = [(1.0, 0, 1.0, 0.0), (0.7, 50, 0.95, 0.0), (0.8, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.08), (0.6, 40, 1.0, 0.0),
       (1.0, 1000, 0.9, 0.02), (0.0, 0, 1.0, 0.0), (1.0, 1, 1.0, 0.0), (0.9, 0, 0.4, 0.0), (1.0, 3000, 0.99, 0.0),
       (2.5, 5, 0.5, 0.3), (1.0, 0, 1.0, 1.0)]


def _peaked(seed, rows, V):
    """Rows from flat to one dominating id."""
    g = wl.rng(seed, 40)
    z = 2.0 * g.standard_normal((rows, V))
    for r in range(rows):
        ids = g.integers(0, V, size=min(48, V))
        z[r, ids] += (r % 4) * 1.5 * g.exponential(size=len(ids))
    return z.astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 3, 8, 31, 130, 1000, 1025, 2049, 4097, 16385, 32000, 50257, 128256, 131073,
                               151936, 262144])
@pytest.mark.parametrize("bf16", [False, True])
def test_rows_against_the_oracle(V, bf16):
    check(_peaked(V, len(ALL), V), ALL, bf16=bf16, seed=V, draws=4)


@pytest.mark.parametrize("pad", [1, 2, 3, 5])
@pytest.mark.parametrize("V", [7, 2050, 32001])
def test_rows_at_any_alignment(pad, V):
    """Row distances that are not multiples of 16 bytes, and a base that is not; what lies between the rows stays."""
    for bf16 in (False, True):
        check(_peaked(V + pad, len(ALL), V), ALL, bf16=bf16, pad=pad, seed=pad)


@pytest.mark.parametrize("rows", [1, 5, 33, 320, 700])
def test_batches(rows):
    """From one row over every SM to more rows than run at once; parameters per sequence of five rows."""
    V = 4099
    sets = [ALL[i % len(ALL)] for i in range(-(-rows // 5))]
    check(_peaked(rows, rows, V), sets, seed=rows, draws=2, rows_per_set=5)


@pytest.mark.parametrize("rows,V,bf16", [(60, 131077, False), (100, 40001, True), (170, 50257, False),
                                         (170, 32768, True), (90, 262144, False)])
def test_batches_of_long_rows(rows, V, bf16):
    """Rows that share the SMs by two, four and eight CTAs, kept on chip and read again."""
    sets = [ALL[(i * 5) % len(ALL)] for i in range(rows)]
    check(_peaked(rows, rows, V), sets, bf16=bf16, seed=rows, draws=2)


@pytest.mark.parametrize("draws", [1, 2, 17, 64])
def test_many_draws(draws):
    check(_peaked(draws, 6, 50257), ALL[:6], draws=draws, seed=draws)


@pytest.mark.parametrize("V", [20, 5000, 128256])
def test_ties(V):
    """Rows of few values: a threshold keeps all of its value or none; equal logits have equal chances."""
    g = wl.rng(V, 41)
    z = g.integers(-3, 4, size=(len(ALL), V)).astype(np.float32)
    z[0] = 1.5
    z[1] = -0.0
    z[2, ::2] = 0.0
    check(z, ALL, draws=5, seed=1)
    check(z, ALL, bf16=True, draws=5, seed=2)


def test_thresholds_inside_a_crowd():
    """Many logits within a bin of the first histogram (and within few steps of fp32), above the list's size: finer
    bins have to part them."""
    V = 128256
    g = wl.rng(5, 42)
    z = np.full((6, V), -1.0, np.float32)
    z[:, :100000] = 1.0 + g.integers(0, 4000, size=(6, 100000)) * np.float32(2.0 ** -23)
    z[3:, :100000] = 1.0 + g.integers(0, 30, size=(3, 100000)) * np.float32(2.0 ** -23)
    z[2, 0] = 40.0
    z[5, 1] = 9.0
    par = [(1.0, 5000, 1.0, 0.0), (1.0, 0, 0.31, 0.0), (1.0, 70000, 1.0, 0.0), (1.0, 0, 0.73, 0.0),
           (1.0, 50000, 0.5, 0.0), (0.5, 60001, 0.9, 0.0)]
    check(z, par, draws=2, seed=3)


def test_nucleus_deep_in_the_tail():
    """Rows where one id outweighs the rest by 2^28 and more, and top-p ends among the rest: beyond the bins that a
    first count has; heavy ids whose weights lie at a bin's edge."""
    V = 100000
    g = wl.rng(6, 43)
    z = (0.05 * g.standard_normal((8, V))).astype(np.float32)
    z[:, 777] = np.log(2.0) * np.array([30, 29, 27.9, 31, 20, 10, 33, 34])
    z[4:, 100:140] = z[4:, 777:778] - np.log(2.0) * (np.arange(40) * 0.25 + 0.0034)
    tail = np.exp(z.astype(np.float64) - z.max(1, keepdims=True)).sum(1) - 1
    par = [(1.0, 0, _f32(1 - 0.6 * t / (1 + t)), 0.0) for t in tail]
    check(z, par, draws=3, seed=8)
    check(z, [(1.0, 90000, p, 0.0) for _, _, p, _ in par], draws=3, seed=9)
    check(z, [(0.9, 0, p, 2.0 ** -60) for _, _, p, _ in par], draws=3, seed=10)


@pytest.mark.parametrize("top_p", [0.01, 0.05, 0.3, 0.999, 0.99999])
def test_nuclei_of_every_size(top_p):
    """From among the heaviest ids of flat rows to nearly all ids; temperatures that leave one id and nearly equal
    ones."""
    V = 128256
    z = _peaked(17, 8, V)
    check(z, [(T, 0, top_p, 0.0) for T in (0.05, 0.3, 0.7, 1.0, 1.5, 2.5, 8.0, 50.0)], draws=2, seed=11)


def test_zeros_of_both_signs_at_the_threshold():
    """0 and -0 are equal: neither is cut without the other, nor counted without it."""
    V = 30000
    g = wl.rng(7, 44)
    z = np.where(g.random((6, V)) < 0.5, np.float32(0.0), np.float32(-0.0)).astype(np.float32)
    z[:, ::3] = (-0.001 * g.random((6, len(z[0, ::3])))).astype(np.float32)
    z[:, 1::300] = 0.25
    par = [(1.0, 5000, 1.0, 0.0), (1.0, 0, 0.2, 0.0), (1.0, 5000, 0.6, 0.0), (1.0, 101, 0.9, 0.0), (1.0, 0, 0.5, 0.7),
           (1e-30, 0, 0.5, 0.0)]
    check(z, par, draws=2, seed=12)


def test_infinities_in_long_rows():
    """More infinite logits than a list holds."""
    V = 50000
    z = _peaked(18, 4, V)
    z[0, ::9] = np.inf
    z[1, ::2] = np.inf
    z[2, 5] = np.inf
    z[3, ::2] = np.nan
    check(z, [(1.0, 0, 0.9, 0.0), (0.7, 3000, 0.5, 0.1), (1.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0)], draws=4, seed=13)


def test_masked_rows():
    """-inf, the type's lowest value and NaN in masked places, rows with one id, with none, and with infinities."""
    V = 3000
    z = _peaked(9, 12, V)
    z[0, 5:] = -np.inf
    z[1] = -np.inf
    z[2] = np.nan
    z[3, ::2] = np.nan
    z[4, 1:] = np.finfo(np.float32).min
    z[5] = np.finfo(np.float32).min
    z[6, 17] = np.inf
    z[7, [3, 900, 2999]] = np.inf
    z[8] = -np.inf
    z[8, 2999] = -1e30
    z[9, :2000] = -np.inf
    par = [(0.7, 50, 0.95, 0.0), (1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 0.9, 0.0),
           (1.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.1), (1.0, 2, 1.0, 0.0), (1.0, 0, 0.5, 0.5), (1.0, 1500, 0.9, 0.0),
           (0.0, 0, 1.0, 0.0), (1.0, 0, 0.95, 0.0)]
    for first in (par, par[::-1]):
        check(z, first, status=sb.DEV_EMPTY_MASK, seed=4)
    z = np.where(np.isnan(z), -np.inf, z)
    z[~np.isfinite(z) & (z < 0)] = -np.inf
    check(z, par, bf16=True, status=sb.DEV_EMPTY_MASK, seed=5)


def test_masked_places_of_rows_far_from_zero():
    """Logits so large that their powers are taken in 64 bits: NaN and -inf there have no weight either."""
    g = np.random.default_rng(44)
    V = 5003
    z = (2.0 * g.standard_normal((8, V)) + np.array([4e4, -4e4, 3e5, 0.0])[np.arange(8) % 4, None])
    z[:, ::7] = np.nan
    z[:, 3::11] = -np.inf
    par = [(1.0, 0, 0.9, 0.0)] * 4 + [(0.7, 0, 1.0, 0.0), (0.7, 1000, 0.8, 0.0), (1.0, 0, 0.95, 1e-4), (0.9, 900, 1.0, 0.0)]
    check(z, par, seed=45)
    check(z[:1].repeat(2, 0), [(1.0, 0, 0.9, 0.0), (1.0, 0, 0.5, 0.0)], pad=1, seed=46)


def test_scales_of_temperature_and_logits():
    """Temperatures and offsets past where whole powers leave in 32 bits, far apart logits, tiny differences."""
    V = 2500
    z = _peaked(11, 9, V)
    z[1] += 1000.0
    z[2] -= 30000.0
    z[3] *= 1e20
    z[4] *= 1e-20
    z[5] = np.where(np.arange(V) % 3 == 0, np.float32(1e9), np.nextafter(np.float32(1e9), np.float32(0)))
    z[6] *= 40.0
    par = [(1e-3, 0, 0.9, 0.0), (0.7, 0, 0.9, 0.0), (0.5, 0, 1.0, 0.0), (1e20, 0, 0.9, 0.0), (1e-20, 0, 0.95, 0.05),
           (100.0, 0, 0.5, 0.0), (1.0, 0, 0.999, 0.0), (1e-30, 0, 1.0, 0.0), (3e38, 0, 0.5, 0.0)]
    check(z, par, seed=6, draws=5)


def test_uniforms_at_the_ends():
    V = 40000
    z = _peaked(12, 4, V)
    u = np.tile(np.array([0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0, 7.0, np.nan, -3.0, np.inf, 1e-45],
                         np.float32), (4, 1))
    for s, k in ((sb.Sampling(), 0), (sb.Sampling(top_k=30), 30)):
        tok = torch.empty(4, 8, dtype=torch.int32, device="cuda")
        sb.spec_sample(_cuda(z), s, _cuda(u), tok, sb.workspace(256))
        t = tok.cpu().numpy()
        for r in range(4):
            # a weight of half a unit, 2^-36 of 2^m with m the largest's own power rounded to the nearest, is the least
            # that is drawn: ids below 2^-37 of the largest never, above 2^-35 always
            p = OS.truncate(z[r], 1.0, k).p / OS.truncate(z[r], 1.0, k).p.max()
            sure, some = np.flatnonzero(p > 2.0 ** -35), np.flatnonzero(p > 2.0 ** -37)
            assert t[r, 0] == t[r, 4] == t[r, 5] == t[r, 7] and t[r, 0] in some and t[r, 0] <= sure[0]
            # the largest u below 1 leaves 2^-24 of the mass above it
            c = np.cumsum(p) / p.sum()
            assert t[r, 1] in some and c[t[r, 1]] > 1 - 2.0 ** -24 - margin(V)
            assert t[r, 2] == t[r, 3] == t[r, 6] and t[r, 2] in some and t[r, 2] >= sure[-1]


def test_draws_follow_the_distribution():
    """A grid of uniforms counts out the distribution to within one each."""
    V, n = 700, 64 * 40
    z = _peaked(13, 1, V)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32).reshape(40, 64)
    tok = torch.empty(40, 64, dtype=torch.int32, device="cuda")
    sb.spec_sample(_cuda(np.repeat(z, 40, 0)), sb.Sampling(0.9, 0, 0.97), _cuda(u), tok, sb.workspace(256))
    got = np.bincount(tok.cpu().numpy().ravel(), minlength=V)
    ref = OS.truncate(z[0], _f32(0.9), 0, _f32(0.97))
    assert np.abs(got - n * ref.p).max() <= 1.01


def test_parameters_out_of_range_on_the_device():
    V = 200
    z = _peaked(14, 9, V)
    bad = [(-1.0, 0, 1.0, 0.0), (float("nan"), 0, 1.0, 0.0), (float("inf"), 0, 1.0, 0.0), (1.0, -1, 1.0, 0.0),
           (1.0, 0, 0.0, 0.0), (1.0, 0, 1.1, 0.0), (1.0, 0, 1.0, -0.5), (1.0, 0, 1.0, 2.0), (1.0, 0, 1.0, 0.0)]
    ws, s = sb.workspace(256), _sampling(bad)
    tok = torch.full((9, 2), 5, dtype=torch.int32, device="cuda")
    probs = torch.full((9, V), 5.0, device="cuda")
    sb.spec_sample(_cuda(z), s, _cuda(wl.uniforms(1, 9, 2)), tok, ws, probs=probs)
    assert sb.spec_device_status(ws) == (sb.SPEC_EDEVICE, sb.DEV_BAD_PARAM)
    assert (tok[:8] == -1).all() and (tok[8] >= 0).all() and (probs[:8] == 0).all()
    out = torch.empty(9, V, device="cuda")
    sb.spec_filter_logits(_cuda(z), s, out, ws)
    assert sb.spec_device_status(ws)[1] == sb.DEV_BAD_PARAM
    assert torch.equal(out, _cuda(z))


def test_python_checks():
    z = torch.zeros(4, 10, device="cuda")
    ws, u, tok = sb.workspace(256), torch.zeros(4, 1, device="cuda"), torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    for f in (lambda: sb.spec_sample(z.t(), sb.Sampling(), u, tok, ws),
              lambda: sb.spec_sample(z.half(), sb.Sampling(), u, tok, ws),
              lambda: sb.spec_sample(z, sb.Sampling(), u[:3], tok, ws),
              lambda: sb.spec_sample(z, sb.Sampling(), u, tok.long(), ws),
              lambda: sb.spec_sample(z[:1].expand(4, 10), sb.Sampling(), u, tok, ws),
              lambda: sb.spec_sample(z, sb.Sampling(temperature=torch.ones(3, device="cuda")), u, tok, ws),
              lambda: sb.spec_sample(z, sb.Sampling(), u, tok, ws, probs=z[:, :9]),
              lambda: sb.spec_filter_logits(z, sb.Sampling(), z.bfloat16(), ws),
              lambda: sb.spec_filter_logits(z, sb.Sampling(), z[:, :9], ws),
              lambda: sb.Sampling(top_k=torch.ones(4, device="cuda"))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(sb.SpecError):
        sb.spec_sample(z, sb.Sampling(temperature=-1.0), u, tok, ws)
    # no rows, and a set more than needed
    sb.spec_sample(z[:0], sb.Sampling(), u[:0], tok[:0], ws)
    sb.spec_sample(z, sb.Sampling(temperature=torch.ones(9, device="cuda")), u, tok, ws)


def test_streams_captures_and_repeats():
    """On a side stream, captured and replayed with other contents, and again: the same bits."""
    V, rows = 32000, 20
    z1, z2 = _cuda(_peaked(15, rows, V)), _cuda(_peaked(16, rows, V))
    s = _sampling([ALL[i % len(ALL)] for i in range(rows)])
    u = _cuda(wl.uniforms(3, rows, 4))

    def run(z, out=None):
        o = out or (torch.empty(rows, 4, dtype=torch.int32, device="cuda"), torch.empty(rows, V, device="cuda"),
                    torch.empty(rows, V, device="cuda"))
        sb.spec_sample(z, s, u, o[0], ws, probs=o[1])
        sb.spec_filter_logits(z, s, o[2], ws)
        return o

    ws = sb.workspace(256)
    a, b = run(z1), run(z2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = run(z1)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, c))
    z = z1.clone()
    out = run(z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(z, out)
    for src, want in ((z2, b), (z1, a)):
        z.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_second_device():
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU in this process")
    z, u = _cuda(_peaked(17, 3, 5000)), _cuda(wl.uniforms(4, 3, 2))
    got = []
    for d in ("cuda:0", "cuda:1"):  # the current device stays 0
        tok = torch.empty(3, 2, dtype=torch.int32, device=d)
        sb.spec_sample(z.to(d), sb.Sampling(top_p=0.9), u.to(d), tok, sb.workspace(256, d))
        got.append(tok.cpu())
    assert torch.equal(*got)


@pytest.mark.parametrize("par", [(0.8, 40, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.7, 100, 0.95, 0.02), (0.0, 0, 1.0, 0.0)])
def test_round_of_drafts_with_one_truncation_on_both_sides(par):
    """Drafts drawn with spec_sample, the target's rows filtered with the same parameters, then spec_accept: what the
    acceptance oracle does with both truncated distributions."""
    B, gamma, V = 6, 4, 2003
    T, k, p, m = par
    zq, zp = wl.accept_logits(21, B, gamma, V)
    s = sb.Sampling(T, k, p, m)
    q = torch.empty(B * gamma, V, device="cuda")
    x = torch.empty(B * gamma, 1, dtype=torch.int32, device="cuda")
    ws = sb.workspace(sb.spec_accept_workspace_bytes(B, gamma, V))
    zq = np.ascontiguousarray(zq[:, :gamma].reshape(B * gamma, V))
    sb.spec_sample(_cuda(zq), s, _cuda(wl.uniforms(5, B * gamma, 1)), x, ws, probs=q)
    target = _cuda(zp).view(B * (gamma + 1), V)
    sb.spec_filter_logits(target, s, target, ws)
    u = wl.uniforms(6, B, gamma + 1)
    out = torch.empty(B, gamma + 1, dtype=torch.int32, device="cuda")
    n_acc = torch.empty(B, dtype=torch.int32, device="cuda")
    sb.spec_accept(target, q, x, _cuda(u), B, gamma, V, T, 1.0, out, n_acc, ws)
    assert sb.spec_device_status(ws) == (sb.SPEC_OK, 0)
    accepted = 0
    for b in range(B):
        z = []
        for i in range(gamma + 1):
            ref = OS.truncate(zp[b, i], _f32(T), k, _f32(p), _f32(m))
            z.append(np.where(ref.keep, zp[b, i].astype(np.float64), -np.inf))
        qs = q.view(B, gamma, V)[b].double().cpu().numpy()
        r = OA.accept(np.stack(z), None if T == 0 else qs, x.view(B, gamma)[b].cpu().numpy(), u[b], T)
        assert r.n_accepted == int(n_acc[b]) and r.tokens == out[b].tolist()
        accepted += r.n_accepted
    assert accepted > 0
