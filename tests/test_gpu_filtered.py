"""GPU: sampling and verification under top-k, top-p and min-p against the fp64
oracle.

Kept sets (the filter rows' integers and logits) and tokens must be equal to
the oracle's: both sides evaluate every cut and draw in fp64, so only a
decision within NEAR of its threshold may differ, and none of the seeded
decisions lies that close unless a check says so.  NEAR: the weights of the long
sums are exact to 5e-12 (2^-37), all others to 1e-14, and so are a sum and a
share of it; the units of integer masses are 2^-50 of the largest, for 2^12 of
them 2^-38 at most.
Probabilities are fp64 rounded once to fp32: half a step, 2^-24 relative, plus
fp64 noise far below it.
"""
import numpy as np
import pytest
import torch

from oracle import filtered as F
from synth.workloads import bf16_bits_to_f32, f32_to_bf16_bits
from tests.gpu_util import DEV, dev

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -35
EPS32 = 2.0 ** -24 * 1.001

SETTINGS = [  # T, top_k, top_p, min_p
    (1.0, 0, 1.0, 0.0), (0.7, 0, 0.9, 0.0), (1.0, 50, 1.0, 0.0), (0.6, 20, 0.95, 0.0),
    (1.0, 0, 1.0, 0.05), (0.8, 40, 0.95, 0.05), (1.3, 200, 0.98, 0.02), (0.0, 0, 1.0, 0.0),
    (1.0, 1, 1.0, 0.0), (2.0, 3, 0.5, 0.9), (0.7, 0, 1e-6, 0.0), (1.0, 0, 0.999, 0.0),
    (1.0, 0, 1.0, 1.0), (1.0, 0, 1.0, 1e-7), (1.5, 1000, 0.9, 0.0), (100.0, 5000, 0.7, 0.0),
]


def make_rows(rng, n, V, bf16, kinds=("normal",)):
    """[n, V] logits (bf16 bits or fp32), row i of kind kinds[i % len]."""
    lowest = float(bf16_bits_to_f32(np.uint16(0xFF7F))) if bf16 else float(np.finfo(np.float32).min)
    z = (3 * rng.standard_normal((n, V)) + 6.0 / (1 + rng.permutation(V))).astype(np.float32)
    for i in range(n):
        kind = kinds[i % len(kinds)]
        if kind == "ties":
            z[i] = np.round(z[i])
        elif kind == "equal":
            z[i] = 1.25
        elif kind == "masked":
            z[i, rng.random(V) < 0.9] = -np.inf
        elif kind == "lowest":
            z[i, rng.random(V) < 0.7] = lowest
        elif kind == "one":
            z[i] = -np.inf
            z[i, rng.integers(V)] = -3.0
        elif kind == "none":
            z[i] = -np.inf
            z[i, rng.random(V) < 0.5] = np.nan
        elif kind == "nan":
            z[i, rng.random(V) < 0.3] = np.nan
            z[i, 0] = 0.5
        elif kind == "inf":
            z[i, rng.integers(V, size=2)] = np.inf
        elif kind == "zeros":
            z[i] = np.where(rng.random(V) < 0.5, -0.0, 0.0)
        elif kind == "flat":
            z[i] *= 0.01
        elif kind == "peaked":
            z[i] *= 10
        elif kind == "sorted":
            z[i] = np.sort(z[i])
    return f32_to_bf16_bits(z) if bf16 else z


KINDS = ("normal", "ties", "equal", "masked", "lowest", "one", "none", "nan", "inf", "zeros",
         "flat", "peaked", "sorted")


def wide(z, bf16):
    return (bf16_bits_to_f32(z) if bf16 else z).astype(np.float64)


def settings_of(idx):
    s = [SETTINGS[i % len(SETTINGS)] for i in idx]
    col = lambda j, t: dev(np.array([x[j] for x in s], t))  # noqa: E731
    return s, dict(temperatures=col(0, np.float32), top_ks=col(1, np.int32),
                   top_ps=col(2, np.float32), min_ps=col(3, np.float32))


def unpack(rows):
    r = np.ascontiguousarray(rows.cpu().numpy())
    f8, f4 = r.view(np.float64), r.view(np.float32)
    return dict(scale=f8[..., 0], inv_sum=f8[..., 1], max=f4[..., 4], min_kept=f4[..., 5],
                last=r[..., 6], n_kept=r[..., 7])


def same_value(a, b):
    return a == b or (np.isnan(a) and np.isnan(b))


def check_row(got, i, want):
    assert int(got["n_kept"][i]) == want.n_kept, (int(got["n_kept"][i]), want[1:])
    assert int(got["last"][i]) == want.last
    assert same_value(float(got["min_kept"][i]), np.float32(want.min_kept))
    assert same_value(float(got["max"][i]), np.float32(want.max))
    assert got["scale"][i] == pytest.approx(want.scale, rel=1e-15)
    assert got["inv_sum"][i] == pytest.approx(want.inv_sum, rel=1e-11)


def check_sample(sv, z, bf16, idx, u, K=1, stride=None, row_index=None, probs=True):
    """One sampler call on rows z under settings idx (per sequence) against the oracle."""
    s, kw = settings_of(idx)
    V = z.shape[1]
    zt = dev(z)
    if stride:
        buf = torch.full((z.shape[0], stride), 77.0, dtype=zt.dtype, device=DEV)
        buf[:, :V] = zt
        zt = buf[:, :V]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tok, q, rows = sv.spec_draft_sample_filtered(
        zt, K, uniforms=dev(u), want_draft_probs=probs, want_filter_rows=True, device_error=err,
        row_index=None if row_index is None else dev(row_index), **kw)
    torch.cuda.synchronize()
    got = {n: v.reshape(-1) for n, v in unpack(rows).items()}
    tok = tok.cpu().numpy().reshape(-1)
    q = q.cpu().numpy().reshape(-1, V) if probs else None
    empty = False
    for i in range(tok.shape[0]):
        r = i if row_index is None else int(row_index.reshape(-1)[i])
        want = F.filter_row(wide(z[r], bf16), *s[i // K])
        empty |= want.n_kept == 0
        check_row(got, i, want)
        t, near = F.draw(want.probs, 0.0 if s[i // K][0] == 0 else float(u.reshape(-1)[i]))
        assert int(tok[i]) == t or near < NEAR, (i, s[i // K], int(tok[i]), t, near)
        if probs:
            assert np.all(np.abs(q[i] - want.probs) <= EPS32 * want.probs + 1e-45)
    assert int(err.item()) == (sv.DEVERR_EMPTY_ROW if empty else 0)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 17, 63, 64, 65, 511, 1000, 2048, 2049, 5003])
def test_sampler_small(gpu, V, bf16):
    rng = np.random.default_rng(1000 + V)
    n = len(KINDS) * len(SETTINGS)
    z = make_rows(rng, n, V, bf16, KINDS)
    check_sample(gpu, z, bf16, [i // len(KINDS) for i in range(n)],
                 rng.random((n, 1), dtype=np.float32))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("V", [30011, 32000, 151936])
def test_sampler_large(gpu, V, bf16):
    rng = np.random.default_rng(V)
    n = len(SETTINGS) * (2 if V > 100000 else 4)
    z = make_rows(rng, n, V, bf16, ("normal", "flat") if V > 100000 else ("normal", "masked",
                                                                          "sorted", "ties"))
    check_sample(gpu, z, bf16, [i // (n // len(SETTINGS)) for i in range(n)],
                 rng.random((n, 1), dtype=np.float32), probs=V < 100000)


def test_sampler_largest_vocabulary(gpu):
    rng = np.random.default_rng(9)
    V = 1 << 19
    z = make_rows(rng, 6, V, True, ("normal", "ties", "equal"))
    check_sample(gpu, z, True, [1, 2, 5, 11, 4, 14], rng.random((6, 1), dtype=np.float32),
                 probs=False)


@pytest.mark.parametrize("bf16", [True, False])
def test_sampler_rows_strides_and_drafts(gpu, bf16):
    """K drafts per sequence, rows by index, rows spaced wider than V at an odd distance."""
    rng = np.random.default_rng(31)
    B, K, V, per = 16, 3, 1237, 5
    z = make_rows(rng, B * per, V, bf16, KINDS[:4])
    ri = np.stack([b * per + rng.permutation(per)[:K] for b in range(B)]).astype(np.int32)
    u = rng.random((B, K), dtype=np.float32)
    check_sample(gpu, z, bf16, range(B), u, K, stride=V + 13, row_index=ri)
    check_sample(gpu, z[:B * K], bf16, range(B), u, K, stride=V + 3)


def test_uniform_ends_and_scalar_settings(gpu):
    """u = 0 and the largest u below 1 draw the first and last kept token; a
    scalar temperature, and no settings at all, equal the plain sampler's law."""
    rng = np.random.default_rng(3)
    V = 1000
    z = make_rows(rng, 4, V, False)
    for u in (0.0, np.float32(1 - 2.0 ** -24)):
        uu = np.full((4, 1), u, np.float32)
        tok, q, _ = gpu.spec_draft_sample_filtered(
            dev(z), 1, 0.9, uniforms=dev(uu), top_ks=dev(np.full(4, 30, np.int32)),
            want_draft_probs=True)
        for i in range(4):
            kept = np.nonzero(F.filter_row(z[i], 0.9, 30).probs)[0]
            assert int(tok[i]) == (kept[0] if u == 0 else kept[-1])
            assert np.array_equal(np.nonzero(q[i, 0].cpu().numpy())[0], kept)
    tok, _, rows = gpu.spec_draft_sample_filtered(dev(z), 1, 0.0, want_filter_rows=True)
    assert tok.view(-1).tolist() == z.argmax(1).tolist()
    assert unpack(rows)["n_kept"].reshape(-1).tolist() == [1] * 4


def test_bad_settings_are_flagged_and_off(gpu):
    rng = np.random.default_rng(4)
    V = 300
    z = make_rows(rng, 8, V, False)
    T = np.array([1, 1, 1, 1, 1, 1, -1, np.nan], np.float32)
    k = np.array([-1, 5, 5, 5, 5, 5, 0, 0], np.int32)
    p = np.array([1, 0, -0.5, 1.5, np.nan, 1, 1, 1], np.float32)
    mp = np.array([0, 0, 0, 0, 0, 1.5, 0, 0], np.float32)
    want = [F.filter_row(z[0], 1.0)] + [F.filter_row(z[i], 1.0, 5) for i in range(1, 6)] + \
        [F.filter_row(z[i], 0.0) for i in (6, 7)]
    bits = [gpu.DEVERR_FILTER] * 6 + [gpu.DEVERR_TEMPERATURE] * 2
    for i in range(8):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        s = slice(i, i + 1)
        _, q, rows = gpu.spec_draft_sample_filtered(
            dev(z[s]), 1, temperatures=dev(T[s]), top_ks=dev(k[s]), top_ps=dev(p[s]),
            min_ps=dev(mp[s]), uniforms=dev(np.array([[0.3]], np.float32)), want_filter_rows=True,
            want_draft_probs=True, device_error=err)
        assert int(err.item()) == bits[i], i
        check_row({n: v.reshape(-1) for n, v in unpack(rows).items()}, 0, want[i])
        assert np.allclose(q[0, 0].cpu().numpy(), want[i].probs, rtol=1e-6, atol=1e-30)


def test_bad_row_index(gpu):
    z = dev(np.zeros((2, 40), np.float32))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tok, q, rows = gpu.spec_draft_sample_filtered(
        z, 3, 1.0, uniforms=dev(np.full((1, 3), 0.5, np.float32)),
        row_index=dev(np.array([[-1, 1, 2]], np.int32)), want_draft_probs=True,
        want_filter_rows=True, device_error=err)
    assert tok.view(-1).tolist() == [-1, 20, -1]
    assert int(err.item()) == gpu.DEVERR_ROW_INDEX
    assert not q[0, 0].any() and not q[0, 2].any()
    assert unpack(rows)["n_kept"].reshape(-1).tolist() == [0, 40, 0]


# ---------------------------------------------------------------- verify
def verify_case(rng, B, K, V, bf16, noise=0.5, kinds=("normal",)):
    zt = make_rows(rng, B * (K + 1), V, bf16, kinds)
    base = wide(zt, bf16).reshape(B, K + 1, V)[:, :K].reshape(B * K, V)
    zd = (base + noise * rng.standard_normal((B * K, V))).astype(np.float32)
    return zt, f32_to_bf16_bits(zd) if bf16 else zd


def check_verify(sv, zt, zd, B, K, V, bf16, idx, rng, dense, bad_draft=False, stride=None):
    s, kw = settings_of(idx)
    rows = [[F.filter_row(wide(zt[b * (K + 1) + k], bf16), *s[b]) for k in range(K + 1)]
            for b in range(B)]
    q = np.zeros((B, K, V))
    tgt, dzd = dev(zt), dev(zd)
    if stride:
        buf = torch.zeros((B * (K + 1), stride), dtype=tgt.dtype, device=DEV)
        buf[:, :V] = tgt
        tgt = buf[:, :V]
    tgt = tgt.as_strided((B, K + 1, V), ((K + 1) * (stride or V), stride or V, 1))
    u = rng.random((B, K + 1), dtype=np.float32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if K:
        tok, probs, frows = sv.spec_draft_sample_filtered(
            dzd, K, uniforms=dev(rng.random((B, K), dtype=np.float32)), want_draft_probs=True,
            want_filter_rows=True, **kw)
        for b in range(B):
            for k in range(K):
                q[b, k] = F.filter_row(wide(zd[b * K + k], bf16), *s[b]).probs
    else:
        tok = torch.empty((B, 0), dtype=torch.int32, device=DEV)
        probs = torch.empty((B, 0, V), device=DEV)
        frows = torch.empty((B, 0, 8), dtype=torch.int32, device=DEV)
    if bad_draft and K:
        tok[::3, K // 2] = -1
        tok[1::3, 0] = V
    if dense:
        q = probs.cpu().numpy().astype(np.float64)
        out, acc, p = sv.spec_verify_filtered(tgt, probs, tok, dev(u), want_draft_target_prob=True,
                                              device_error=err, **kw)
    else:
        out, acc, p = sv.spec_verify_filtered_lq(tgt, dzd, frows, tok, dev(u),
                                                 want_draft_target_prob=True, device_error=err,
                                                 **kw)
    torch.cuda.synchronize()
    d, out, acc, p = tok.cpu().numpy(), out.cpu().numpy(), acc.cpu().numpy(), p.cpu().numpy()
    for b in range(B):
        a, c, want_p, near = F.verify_seq(rows[b], q[b], d[b], u[b], s[b][0])
        if near >= NEAR:
            assert int(acc[b]) == a, (b, s[b])
            assert out[b].tolist() == d[b, :a].tolist() + [c] + [-1] * (K - a), (b, s[b])
        assert np.all(np.abs(p[b] - want_p) <= EPS32 * want_p + 1e-45)
    flags = int(err.item())
    assert bool(flags & sv.DEVERR_DRAFT_TOKEN) == bool(((d < 0) | (d >= V)).any())
    assert bool(flags & sv.DEVERR_EMPTY_ROW) == any(r.n_kept == 0 for x in rows for r in x)
    return acc


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,K,V", [(1, 3, 32), (16, 1, 1), (32, 2, 7), (33, 5, 257), (16, 7, 5003),
                                   (3, 63, 100), (8, 0, 700), (8, 5, 32000)])
def test_verify(gpu, B, K, V, bf16, dense):
    rng = np.random.default_rng(B * 1000 + K * 10 + V)
    zt, zd = verify_case(rng, B, K, V, bf16)
    check_verify(gpu, zt, zd, B, K, V, bf16, range(B), rng, dense)


@pytest.mark.parametrize("dense", [True, False])
def test_verify_odd_rows_and_drafts(gpu, dense):
    rng = np.random.default_rng(17)
    B, K, V = 48, 4, 333
    zt, zd = verify_case(rng, B, K, V, False, kinds=KINDS)
    check_verify(gpu, zt, zd, B, K, V, False, range(B), rng, dense, bad_draft=True, stride=V + 5)


def test_verify_large_vocabulary(gpu):
    rng = np.random.default_rng(18)
    B, K, V = 8, 2, 151936
    zt, zd = verify_case(rng, B, K, V, True)
    check_verify(gpu, zt, zd, B, K, V, True, [0, 1, 2, 5, 6, 11, 13, 7], rng, False)


def test_verify_equal_distributions_accepts_everything(gpu):
    """Target rows equal to the drafter's under one setting: p = q, every draft
    is accepted (u < 1) and only the bonus row is drawn from."""
    rng = np.random.default_rng(19)
    B, K, V = 16, 3, 4000
    zt = make_rows(rng, B * (K + 1), V, True)
    zd = zt.reshape(B, K + 1, V)[:, :K].reshape(B * K, V).copy()
    acc = check_verify(gpu, zt, zd, B, K, V, True, range(B), rng, False)
    assert acc.tolist() == [K] * B


def test_greedy_sequences_need_no_q(gpu):
    """T = 0: neither q nor the uniforms are read (NaN in both changes nothing)."""
    rng = np.random.default_rng(20)
    B, K, V = 4, 3, 500
    zt = dev(make_rows(rng, B * (K + 1), V, False).reshape(B, K + 1, V))
    d = zt[:, :K].argmax(2).to(torch.int32)
    d[1, 2] = (d[1, 2] + 1) % V
    T = torch.zeros(B, device=DEV)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
    out, acc, _ = gpu.spec_verify_filtered(zt, nan(B, K, V), d, nan(B, K + 1), T)
    want, wacc = gpu.spec_verify_greedy(zt, d)
    assert torch.equal(out, want) and torch.equal(acc, wacc)


# ---------------------------------------------------------------- use
def test_streams_graphs_and_workspaces(gpu):
    """Captured calls replayed on new inputs, two graphs of one memory pool, and
    calls on two streams at once equal the eager ones."""
    rng = np.random.default_rng(21)
    B, K, V = 8, 3, 32000
    _, kw = settings_of(range(1, B + 1))
    sets = [(dev(make_rows(rng, B * K, V, True)), dev(rng.random((B, K), dtype=np.float32)))
            for _ in range(3)]
    eager = [gpu.spec_draft_sample_filtered(z, K, uniforms=u, want_filter_rows=True, **kw)
             for z, u in sets]
    z, u = sets[0][0].clone(), sets[0][1].clone()
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gpu.spec_draft_sample_filtered(z, K, uniforms=u, want_filter_rows=True, **kw)
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0][0].pool() if graphs else None):
            r = gpu.spec_draft_sample_filtered(z, K, uniforms=u, want_filter_rows=True, **kw)
        graphs.append((g, r))
    for i in (0, 1, 2, 1):
        z.copy_(sets[i][0])
        u.copy_(sets[i][1])
        for g, r in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(r[0], eager[i][0]) and torch.equal(r[2], eager[i][2])
        gpu.spec_draft_sample_filtered(*[sets[0][0], K], uniforms=sets[0][1], **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    res = []
    for rep in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                res.append((i, gpu.spec_draft_sample_filtered(
                    sets[i][0], K, uniforms=sets[i][1], want_filter_rows=True, **kw)))
    torch.cuda.synchronize()
    for i, r in res:
        assert torch.equal(r[0], eager[i][0]) and torch.equal(r[2], eager[i][2])


def test_repeated_calls_agree_bit_for_bit(gpu):
    rng = np.random.default_rng(22)
    B, K, V = 16, 2, 30011
    zt, zd = verify_case(rng, B, K, V, True)
    _, kw = settings_of(range(B))
    u, ud = dev(rng.random((B, K + 1), dtype=np.float32)), dev(rng.random((B, K), dtype=np.float32))
    tgt, dz = dev(zt).view(B, K + 1, V), dev(zd)
    first = None
    for _ in range(4):
        tok, q, rows = gpu.spec_draft_sample_filtered(dz, K, uniforms=ud, want_draft_probs=True,
                                                      want_filter_rows=True, **kw)
        r = gpu.spec_verify_filtered_lq(tgt, dz, rows, tok, u, want_draft_target_prob=True, **kw)
        now = [tok, q, rows, *r]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_rows_are_left_as_they_were(gpu):
    """A workspace and outputs inside larger buffers: nothing beyond them is written."""
    rng = np.random.default_rng(23)
    B, K, V = 5, 2, 999
    zt, zd = verify_case(rng, B, K, V, False)
    _, kw = settings_of(range(B))
    n = gpu.spec_filter_workspace_bytes(B * (K + 1), V)
    buf = torch.full((n + 512,), 171, dtype=torch.uint8, device=DEV)
    out = torch.full((B + 2, K + 1), -7, dtype=torch.int32, device=DEV)
    acc = torch.full((B + 2,), -7, dtype=torch.int32, device=DEV)
    q = torch.full((B, K, V), 1.0 / V, device=DEV)
    d = torch.zeros((B, K), dtype=torch.int32, device=DEV)
    gpu.spec_verify_filtered(dev(zt).view(B, K + 1, V), q, d,
                             dev(rng.random((B, K + 1), dtype=np.float32)), out_tokens=out[1:-1],
                             out_num_accepted=acc[1:-1], workspace=buf[256:256 + n], **kw)
    torch.cuda.synchronize()
    assert bool((buf[:256] == 171).all()) and bool((buf[256 + n:] == 171).all())
    assert out[0].tolist() == out[-1].tolist() == [-7] * (K + 1)
    assert acc[0] == acc[-1] == -7 and bool((out[1:-1] != -7).all())


def test_refusals(gpu):
    z = torch.zeros((4, 64), device=DEV)
    u = torch.zeros((4, 1), device=DEV)
    call = gpu.spec_draft_sample_filtered
    with pytest.raises(TypeError):
        call(z.half(), 1, uniforms=u)
    with pytest.raises(TypeError):
        call(z, 1, uniforms=u, top_ks=torch.zeros(4, device=DEV))
    with pytest.raises(ValueError):
        call(z, 1, uniforms=u, top_ps=torch.ones(3, device=DEV))
    with pytest.raises(ValueError):
        call(z.t(), 1, uniforms=u)
    with pytest.raises(ValueError):
        call(z[:, :1].expand(4, 64), 1, uniforms=u)
    with pytest.raises(ValueError):
        call(z, 3, uniforms=u)
    with pytest.raises(gpu.SpecVerifyError):
        call(z, 1)                                            # no uniforms
    with pytest.raises(gpu.SpecVerifyError):
        call(z, 1, -1.0, uniforms=u)
    with pytest.raises(gpu.SpecVerifyError):
        call(z, 1, uniforms=u, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        gpu.spec_verify_filtered(z, z, z, u, u)
    T = torch.ones(2, device=DEV)
    t3 = torch.zeros((2, 2, 64), device=DEV)
    with pytest.raises(ValueError):
        gpu.spec_verify_filtered(t3, t3, torch.zeros((2, 1), dtype=torch.int32, device=DEV),
                                 torch.zeros((2, 2), device=DEV), T)
    with pytest.raises(TypeError):
        gpu.spec_verify_filtered_lq(t3, torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV),
                                    torch.zeros((2, 1, 8), dtype=torch.int32, device=DEV),
                                    torch.zeros((2, 1), dtype=torch.int32, device=DEV),
                                    torch.zeros((2, 2), device=DEV), T)


# ---------------------------------------------------------------- many rows
# More rows than compute units: one kernel streams and cuts each row, rows
# without a candidate list follow in a second.
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("V", [777, 5003, 20011])
def test_sampler_many_rows(gpu, V, bf16):
    rng = np.random.default_rng(V + 1)
    n = 3 * len(KINDS) * len(SETTINGS)
    z = make_rows(rng, n, V, bf16, KINDS)
    check_sample(gpu, z, bf16, [i // len(KINDS) for i in range(n)],
                 rng.random((n, 1), dtype=np.float32))


@pytest.mark.parametrize("bf16", [True, False])
def test_sampler_many_large_rows(gpu, bf16):
    rng = np.random.default_rng(77)
    n, V = 528, 70001
    z = make_rows(rng, n, V, bf16, ("normal", "flat", "ties", "masked", "none", "inf", "lowest"))
    check_sample(gpu, z, bf16, [i // 7 for i in range(n)], rng.random((n, 1), dtype=np.float32),
                 probs=False)


@pytest.mark.parametrize("kind", ["none", "inf", "lowest", "equal", "one", "nan", "zeros"])
def test_sampler_few_large_rows_of_extremes(gpu, kind):
    """Rows that a kernel of their own streams (few, longer than 65536)."""
    rng = np.random.default_rng(78)
    n, V = len(SETTINGS), 66001
    for bf16 in (True, False):
        z = make_rows(rng, n, V, bf16, (kind,))
        check_sample(gpu, z, bf16, range(n), rng.random((n, 1), dtype=np.float32), probs=False)


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_verify_many_rows(gpu, bf16, dense):
    rng = np.random.default_rng(79)
    B, K, V = 130, 4, 4099
    zt, zd = verify_case(rng, B, K, V, bf16, kinds=("normal", "flat", "ties", "masked", "lowest"))
    check_verify(gpu, zt, zd, B, K, V, bf16, range(B), rng, dense, stride=V + 1)


def test_verify_many_large_rows(gpu):
    rng = np.random.default_rng(80)
    B, K, V = 176, 2, 33333
    zt, zd = verify_case(rng, B, K, V, True, noise=0.1, kinds=("normal", "flat"))
    check_verify(gpu, zt, zd, B, K, V, True, range(B), rng, False)


def test_verify_graph_and_streams(gpu):
    """A captured draft and verify replayed on new inputs, and on two streams at once."""
    rng = np.random.default_rng(81)
    B, K, V = 24, 3, 20000
    _, kw = settings_of(range(B))

    def step(i):
        tok, q, rows = gpu.spec_draft_sample_filtered(i[1], K, uniforms=i[3], want_filter_rows=True,
                                                      **kw)
        out, acc, _ = gpu.spec_verify_filtered_lq(i[0].view(B, K + 1, V), i[1], rows, tok, i[2],
                                                  **kw)
        return tok, rows, out, acc

    sets = []
    for _ in range(3):
        zt, zd = verify_case(rng, B, K, V, True)
        sets.append([dev(zt), dev(zd), dev(rng.random((B, K + 1), dtype=np.float32)),
                     dev(rng.random((B, K), dtype=np.float32))])
    eager = [step(i) for i in sets]
    static = [t.clone() for t in sets[0]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(static)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step(static)
    for i in (1, 2, 0, 2):
        for a, b in zip(static, sets[i]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, eager[i]))
        step(sets[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for rep in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((i, step(sets[i])))
    torch.cuda.synchronize()
    for i, r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, eager[i]))


@pytest.mark.parametrize("n,V", [(16, 5003), (16, 66001), (528, 5003)])
@pytest.mark.parametrize("kind", ["far", "steep", "gentle"])
def test_sampler_far_and_steep_logits(gpu, n, V, kind):
    """Logits far from 0 and temperatures at which an exponent's parts leave the
    range of the fast sums; each weight is then computed by itself."""
    rng = np.random.default_rng(90)
    z = (3 * rng.standard_normal((n, V))).astype(np.float32)
    z += {"far": np.float32(9000.0), "steep": np.float32(-2.0), "gentle": np.float32(1e-3)}[kind]
    T = {"far": 1.0, "steep": 1e-4, "gentle": 1e6}[kind]
    u = rng.random((n, 1), dtype=np.float32)
    p = rng.choice(np.array([1.0, 0.9, 0.5], np.float32), n)
    for bf16 in (False, True):
        zz = f32_to_bf16_bits(z) if bf16 else z
        tok, _, rows = gpu.spec_draft_sample_filtered(
            dev(zz), 1, uniforms=dev(u), temperatures=dev(np.full(n, T, np.float32)),
            top_ps=dev(p), want_filter_rows=True)
        got = {k: v.reshape(-1) for k, v in unpack(rows).items()}
        tok = tok.cpu().numpy().reshape(-1)
        for i in range(0, n, max(1, n // 64)):
            want = F.filter_row(wide(zz[i:i + 1], bf16)[0], float(np.float32(T)), 0, float(p[i]))
            check_row(got, i, want)
            t, near = F.draw(want.probs, float(u[i, 0]))
            assert int(tok[i]) == t or near < NEAR, (i, int(tok[i]), t, near)
