"""GPU: appending rotated keys, values and queries to a paged cache, against
the fp64 oracle.

Tolerances.  A rotated element is x0 c - x1 s in fp32: c and s are off by at
most 3 * 2^-24 (the reduced angle rounded to fp32, below pi/2 * 2^-24 twice, and
the function's own error), each product and the sum by 2^-24 of themselves, so
the value by less than 8 * 2^-24 (|x0| + |x1|); then half a step of the type it
is stored in.  e4m3: half a step is 2^-4 of the value, or 2^-10 below the
smallest normal value, both in units of the scale.  Copied elements are equal.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import filtered as F
from tests.gpu_util import DEV, dev

pytestmark = pytest.mark.gpu

STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
FP8 = torch.float8_e4m3fn


def f64(t):
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def rot_error(x, half, inter):
    """8 * 2^-24 (|x0| + |x1|) for rotated elements, 0 for copied ones."""
    e = np.zeros_like(x)
    i0 = 2 * np.arange(half) if inter else np.arange(half)
    i1 = i0 + 1 if inter else i0 + half
    s = (np.abs(x[..., i0]) + np.abs(x[..., i1])) * 8 * 2.0 ** -24
    e[..., i0] = e[..., i1] = s
    return e


def check_append(sv, rng, R, Hq, Hkv, D, rot, inter, dtype, fp8=False, packed=False, bs=16,
                 layout="nhd", slots=None, positions=None, scale=1.0, in_place=False,
                 scales=True, spare_blocks=2):
    nb = (R + bs - 1) // bs + spare_blocks
    if packed:
        x = torch.randn((R, (Hq + 2 * Hkv) * D), device=DEV).to(dtype)
        q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        q, k, v = (torch.randn((R, h, D), device=DEV).to(dtype) for h in (Hq, Hkv, Hkv))
    if slots is None:
        slots = rng.permutation(nb * bs)[:R].astype(np.int64)
        slots[rng.random(R) < 0.2] = -1
    if positions is None:
        positions = rng.integers(0, 200_000, R).astype(np.int64)
    cdt = FP8 if fp8 else dtype
    if layout == "nhd":
        kc, vc = (torch.zeros((nb, bs, Hkv, D), dtype=cdt, device=DEV) for _ in range(2))
    elif layout == "hnd":
        kc, vc = (torch.zeros((nb, Hkv, bs, D), dtype=cdt, device=DEV).transpose(1, 2)
                  for _ in range(2))
    else:                                              # halves of one buffer
        both = torch.zeros((nb, 2, bs, Hkv, D), dtype=cdt, device=DEV)
        kc, vc = both[:, 0], both[:, 1]
    fill = torch.randn((nb, bs, Hkv, D), device=DEV).clamp(-3, 3)
    kc.copy_(fill.to(cdt))
    vc.copy_((-fill).to(cdt))
    k0, v0 = f64(kc), f64(vc)
    inv = (1.0 / 10000.0 ** (np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    ks, vs = (dev((0.02 + 0.02 * rng.random(Hkv)).astype(np.float32)) if fp8 and scales else None
              for _ in range(2))
    q0 = f64(q)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sv.peagle_append_kv(
        k, v, dev(positions), dev(slots), kc, vc, inv_freq=dev(inv) if rot else None,
        interleaved=inter, rotary_scale=scale, query=q if Hq else None,
        out_query=q if in_place and Hq else None, k_scales=ks, v_scales=vs, device_error=err)
    torch.cuda.synchronize()
    nslots = nb * bs
    bad = (slots < -1) | (slots >= nslots)
    assert int(err.item()) == (sv.DEVERR_SLOT if bad.any() else 0)
    ok = (slots >= 0) & (slots < nslots)
    if Hq:
        want = F.rotate(q0, positions, inv, inter, scale)
        tol = STEP[dtype] * 1.001 * np.abs(want) + rot_error(q0, rot // 2, inter) * scale + TINY[dtype]
        tol[..., rot:] = 0
        assert np.all(np.abs(f64(out) - want) <= tol)
        if in_place:
            assert out.data_ptr() == q.data_ptr()
    for cache, before, x, sc, turned in ((kc, k0, k, ks, True), (vc, v0, v, vs, False)):
        xs = f64(x)
        want = F.rotate(xs, positions, inv, inter, scale) if turned else xs
        e = rot_error(xs, rot // 2, inter) * scale if turned else np.zeros_like(xs)
        if fp8:
            s = f64(sc)[:, None] if sc is not None else 1.0
            want, e = np.clip(want / s, -448, 448), e / s + np.abs(want / s) * 2.0 ** -23
            tol = 2.0 ** -4 * 1.001 * np.abs(want) + 2.0 ** -10 + 1.1 * e
        else:
            tol = STEP[dtype] * 1.001 * np.abs(want) + e + TINY[dtype]
            if not turned or rot < D:
                tol[..., 0 if not turned else rot:] = 0
        full = before.reshape(nslots, Hkv, D).copy()
        lim = np.zeros_like(full)
        full[slots[ok]], lim[slots[ok]] = want[ok], tol[ok]
        got = f64(cache).reshape(nslots, Hkv, D)
        assert np.all(np.abs(got - full) <= lim), np.abs(got - full).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("R,Hq,Hkv,D,rot,inter,packed", [
    (1, 64, 8, 64, 64, False, True), (1, 1, 1, 1, 0, False, False), (3, 2, 1, 2, 2, True, False),
    (17, 5, 5, 80, 40, True, True), (33, 8, 2, 96, 96, False, False), (64, 4, 1, 128, 64, False, True),
    (7, 3, 1, 7, 6, True, True), (7, 3, 1, 7, 6, False, True), (300, 16, 2, 256, 256, True, False),
    (5, 0, 3, 40, 20, False, False), (1200, 4, 4, 64, 34, False, False), (9, 2, 2, 100, 12, True, True),
    (2, 6, 2, 1000, 998, False, False), (4, 128, 16, 130, 2, False, True)])
def test_append(gpu, R, Hq, Hkv, D, rot, inter, packed, dtype):
    rng = np.random.default_rng(R * 7 + D)
    torch.manual_seed(R + D)
    check_append(gpu, rng, R, Hq, Hkv, D, rot, inter, dtype, packed=packed)
    check_append(gpu, rng, R, Hq, Hkv, D, rot, inter, dtype, fp8=True, packed=packed)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "halves"])
@pytest.mark.parametrize("bs", [1, 5, 16])
def test_layouts_and_blocks(gpu, layout, bs):
    rng = np.random.default_rng(bs)
    torch.manual_seed(bs)
    for fp8 in (False, True):
        check_append(gpu, rng, 100, 4, 2, 64, 64, False, torch.bfloat16, fp8=fp8, bs=bs,
                     layout=layout, in_place=True, scale=1.375)


def test_bad_and_padding_slots(gpu):
    rng = np.random.default_rng(2)
    torch.manual_seed(2)
    n = 3 * 16                     # R = 10 rows: one block and two spare ones
    slots = np.array([0, -1, n - 1, n, -2, 7, n + 12345, 1 << 40, -(1 << 62), 9], np.int64)
    check_append(gpu, rng, 10, 2, 2, 64, 32, False, torch.bfloat16, slots=slots)
    check_append(gpu, rng, 10, 2, 2, 64, 32, False, torch.bfloat16, slots=np.full(10, -1, np.int64))


def test_far_and_negative_positions(gpu):
    """Angles of positions up to 2^31 and below 0 stay exact."""
    rng = np.random.default_rng(3)
    torch.manual_seed(3)
    pos = np.array([0, 1, 2 ** 20 + 1, 2 ** 29 - 1, 2 ** 31 + 5, -1, -12345, 99_999], np.int64)
    check_append(gpu, rng, 8, 4, 2, 64, 64, False, torch.float32, positions=pos)


def test_values_beyond_e4m3(gpu):
    """Large values are limited to 448 scales, NaN stays NaN, infinities limit."""
    k = torch.tensor([1e4, -1e4, float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 464.0],
                     device=DEV).view(1, 1, 8)
    kc, vc = (torch.zeros((1, 1, 1, 8), dtype=FP8, device=DEV) for _ in range(2))
    one = torch.zeros(1, dtype=torch.int64, device=DEV)
    gpu.peagle_append_kv(k, k, one, one, kc, vc)
    got = kc.float().view(-1)
    assert got[:4].tolist() == [448.0, -448.0, 448.0, -448.0] and bool(got[4].isnan())
    assert got[5:].tolist() == [0.0, 0.0, 448.0]
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8))


def test_offsets_past_32_bits(gpu):
    """A cache of more than 2^32 elements, written at its far end."""
    nb, bs, H, D = 70_000, 128, 4, 128
    both = torch.empty((nb, 2, bs, H, D), dtype=FP8, device=DEV)
    kc, vc = both[:, 0], both[:, 1]
    slots = torch.tensor([0, nb * bs - 1], device=DEV)
    kc[-1, -1].view(torch.uint8).zero_()
    k = torch.randn((2, H, D), device=DEV).bfloat16()
    gpu.peagle_append_kv(k, k, torch.zeros(2, dtype=torch.int64, device=DEV), slots, kc, vc)
    assert torch.equal(kc[-1, -1].float(), k[1].float().to(FP8).float())
    assert torch.equal(vc[-1, -1].float(), k[1].float().to(FP8).float())
    assert torch.equal(kc[0, 0].float(), k[0].float().to(FP8).float())


def test_capture_and_streams(gpu):
    """A captured append replayed on new inputs, and appends on two streams."""
    R, H, D = 40, 4, 64
    mk = lambda: torch.randn((R, H, D), device=DEV).bfloat16()  # noqa: E731
    inv = torch.rand(D // 2, device=DEV)
    pos, slots = torch.arange(R, device=DEV), torch.randperm(64, device=DEV)[:R]
    sets = [(mk(), mk(), mk()) for _ in range(3)]

    def call(s, c):
        return gpu.peagle_append_kv(s[1], s[2], pos, slots, c[0], c[1], inv_freq=inv, query=s[0])

    cache = lambda: [torch.zeros((4, 16, H, D), dtype=torch.bfloat16, device=DEV)  # noqa: E731
                     for _ in range(2)]
    want = []
    for s in sets:
        c = cache()
        want.append((call(s, c), *c))
    buf, c = [t.clone() for t in sets[0]], cache()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        call(buf, c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(buf, c)
    for i in (0, 2, 1, 2):
        for a, b in zip(buf, sets[i]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((out, *c), want[i]))
        call(sets[0], cache())
    streams, cs, outs = [torch.cuda.Stream() for _ in range(2)], [cache(), cache()], []
    torch.cuda.synchronize()
    for rep in range(3):
        outs = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs.append(call(sets[i], cs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip((outs[i], *cs[i]), want[i]))


def test_refusals(gpu):
    k = torch.zeros((4, 2, 64), device=DEV).bfloat16()
    pos = torch.arange(4, device=DEV)
    kc, vc = (torch.zeros((2, 16, 2, 64), device=DEV).bfloat16() for _ in range(2))
    inv = torch.rand(32, device=DEV)
    call = gpu.peagle_append_kv
    call(k, k, pos, pos, kc, vc, inv_freq=inv)
    for bad, kind in (((k, k[:, :1], pos, pos, kc, vc), ValueError),
                      ((k, k.float(), pos, pos, kc, vc), TypeError),
                      ((k, k, pos.int(), pos, kc, vc), TypeError),
                      ((k, k, pos, pos[:3], kc, vc), ValueError),
                      ((k, k, pos, pos, kc, vc[:1]), ValueError),
                      ((k, k, pos, pos, kc.float(), vc.float()), TypeError),
                      ((k, k, pos, pos, kc, vc.transpose(1, 2).contiguous().transpose(1, 2)),
                       ValueError),
                      ((k, k, pos, pos, kc[..., :32], vc[..., :32]), ValueError),
                      ((k.transpose(1, 2).contiguous().transpose(1, 2), k, pos, pos, kc, vc),
                       ValueError),
                      ((k.double(), k.double(), pos, pos, kc, vc), TypeError)):
        with pytest.raises(kind):
            call(*bad)
    with pytest.raises(gpu.SpecVerifyError):
        call(k, k, pos, pos, kc, vc, inv_freq=torch.rand(33, device=DEV))
    with pytest.raises(gpu.SpecVerifyError):
        call(k, k, pos, pos, kc, vc, inv_freq=inv, rotary_scale=float("nan"))
    with pytest.raises(ValueError):
        call(k, k, pos, pos, kc, vc, k_scales=torch.ones(2, device=DEV))
    with pytest.raises(ValueError):
        call(k, k, pos, pos, kc, vc, out_query=k)


def test_decode_round(gpu):
    """One round of a server: filtered drafts, the filtered verify, the rebuilt
    drafter batch, and its keys and values into the paged cache."""
    rng = np.random.default_rng(40)
    torch.manual_seed(40)
    B, K, V, H, bs, Hkv, D = 6, 4, 2000, 64, 16, 2, 64
    T = dev(np.array([0.7, 1.0, 0.0, 0.9, 1.2, 0.6], np.float32))
    kw = dict(temperatures=T, top_ks=dev(np.array([50, 0, 0, 20, 0, 5], np.int32)),
              top_ps=dev(np.array([1, 0.9, 1, 0.95, 1, 0.8], np.float32)),
              min_ps=dev(np.array([0, 0, 0, 0, 0.1, 0.02], np.float32)))
    s = list(zip(*(t.cpu().tolist() for t in kw.values())))
    per = 2 * K
    zd = (3 * rng.standard_normal((B * per, V))).astype(np.float32)
    ri = np.stack([b * per + 1 + np.arange(K) for b in range(B)]).astype(np.int32)
    zt = np.stack([np.concatenate([zd[ri[b]] + 0.4 * rng.standard_normal((K, V)),
                                   3 * rng.standard_normal((1, V))]) for b in range(B)])
    zt = zt.astype(np.float32)
    ud, u = rng.random((B, K), dtype=np.float32), rng.random((B, K + 1), dtype=np.float32)
    tok, _, rows = gpu.spec_draft_sample_filtered(dev(zd), K, uniforms=dev(ud),
                                                  row_index=dev(ri), want_filter_rows=True, **kw)
    out, acc, _ = gpu.spec_verify_filtered_lq(dev(zt), dev(zd), rows, tok, dev(u),
                                              drafter_rows=dev(ri), **kw)
    L = np.array([3, 15, 16, 100, 0, 47], np.int64)
    table = np.arange(B * 9, dtype=np.int32).reshape(B, 9)[:, ::-1].copy()
    hid = torch.randn((B * (K + 1), H), device=DEV).bfloat16()
    batch = gpu.peagle_build_draft_batch(out, acc, tok, dev(L), dev(table), bs, hid,
                                         torch.randn(H, device=DEV).bfloat16(), V + 3)
    R = B * 2 * K
    kv = torch.randn((R, 2 * Hkv, D), device=DEV).bfloat16()
    kc, vc = (torch.zeros((B * 9, bs, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    inv = (1.0 / 10000.0 ** (np.arange(0, D, 2) / D)).astype(np.float32)
    gpu.peagle_append_kv(kv[:, :Hkv], kv[:, Hkv:], batch["positions"], batch["slot_mapping"], kc,
                         vc, inv_freq=dev(inv))
    torch.cuda.synchronize()
    d, o, a = tok.cpu().numpy(), out.cpu().numpy(), acc.cpu().numpy()
    for b in range(B):
        q = np.stack([F.filter_row(zd[ri[b, k]], *s[b]).probs for k in range(K)])
        for k in range(K):
            assert int(d[b, k]) == F.draw(q[k], 0.0 if s[b][0] == 0 else float(ud[b, k]))[0]
        wa, wc, _, _ = F.verify_seq([F.filter_row(zt[b, k], *s[b]) for k in range(K + 1)], q, d[b],
                                    u[b], s[b][0])
        assert int(a[b]) == wa and o[b].tolist() == d[b, :wa].tolist() + [wc] + [-1] * (K - wa)
    want = oracle.build_draft_batch(o, a, d, L, table, bs, hid.view(torch.int16).cpu().numpy(),
                                    np.zeros(H, np.int16), V + 3)
    slots = want["slot_mapping"]
    assert np.array_equal(batch["slot_mapping"].cpu().numpy(), slots)
    full_k, full_v = np.zeros((B * 9 * bs, Hkv, D)), np.zeros((B * 9 * bs, Hkv, D))
    x = f64(kv)
    ok = slots >= 0
    assert (~ok).sum() == sum(K - int(i) for i in a)
    full_k[slots[ok]] = F.rotate(x[:, :Hkv], want["positions"], inv, False)[ok]
    full_v[slots[ok]] = x[:, Hkv:][ok]
    assert np.array_equal(f64(vc).reshape(full_v.shape), full_v)
    assert np.allclose(f64(kc).reshape(full_k.shape), full_k, rtol=2.0 ** -8 * 1.001, atol=1e-5)


def test_refuses_an_expanded_cache(gpu):
    k = torch.zeros((4, 2, 64), device=DEV).bfloat16()
    pos = torch.arange(4, device=DEV)
    one = torch.zeros((1, 16, 2, 64), device=DEV).bfloat16()
    with pytest.raises(gpu.SpecVerifyError):
        gpu.peagle_append_kv(k, k, pos, pos, one.expand(3, 16, 2, 64), one.expand(3, 16, 2, 64))
    assert not one.any()
