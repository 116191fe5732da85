"""Host-side argument checks of the filtered calls and the paged append, without a GPU.

Every call below fails validation (or is empty), so nothing reaches the HIP
runtime; the pointers are never dereferenced."""
import pytest

from tests.test_abi_cpu import (EALIGN, EDTYPE, ENULL, ESHAPE, EVALUE, EWS, FAKE, OK,  # noqa: F401
                                declared_functions, lib)


def test_declared():
    names = declared_functions()
    for n in ("spec_filter_workspace_bytes", "spec_draft_sample_filtered", "spec_verify_filtered",
              "spec_verify_filtered_lq", "peagle_append_kv"):
        assert n in names


def test_kernel_names(lib):
    import draft_verification_vocab_amd as sv
    for name, i in sv.KERNEL_IDS.items():
        assert lib.sv_kernel_name(i) == name.encode()


def test_workspace_bytes(lib):
    f = lib.spec_filter_workspace_bytes
    assert f(0, 100) == f(-1, 100) == f(4, 0) == f(4, (1 << 19) + 1) == 0
    assert 0 < f(1, 1) <= f(7, 1000) < f(8192, 151936)


def sample(lib, z=FAKE, dtype=0, n=8, stride=64, ri=None, u=FAKE, T=1.0, Ts=None, k=None, p=None,
           mp=None, B=2, K=4, V=64, tok=FAKE, q=None, rows=None, ws=FAKE, wsb=1 << 30, err=None):
    return lib.spec_draft_sample_filtered(z, dtype, n, stride, ri, u, T, Ts, k, p, mp, B, K, V, tok,
                                          q, rows, ws, wsb, err, None)


def test_sampler_checks(lib):
    assert sample(lib, B=0, z=None, tok=None, u=None, ws=None, wsb=0) == OK
    for bad in (dict(B=-1), dict(K=0), dict(K=64), dict(V=0), dict(V=(1 << 19) + 1), dict(n=-1),
                dict(n=7), dict(stride=63), dict(stride=1 << 40), dict(B=(1 << 20) + 1, n=1 << 23)):
        assert sample(lib, **bad) == ESHAPE, bad
    assert sample(lib, dtype=2) == EDTYPE
    for T in (-1.0, float("nan"), float("inf"), 1e-40):
        assert sample(lib, T=T) == EVALUE
    for bad in (dict(z=None), dict(tok=None), dict(u=None), dict(u=None, T=0.0, Ts=FAKE)):
        assert sample(lib, **bad) == ENULL, bad
    assert sample(lib, ws=None) == EWS and sample(lib, wsb=8) == EWS
    for bad in (dict(z=FAKE + 2), dict(dtype=1, z=FAKE + 1), dict(tok=FAKE + 1), dict(ri=FAKE + 2),
                dict(u=FAKE + 1), dict(Ts=FAKE + 1), dict(k=FAKE + 1), dict(p=FAKE + 1),
                dict(mp=FAKE + 1), dict(q=FAKE + 2), dict(rows=FAKE + 8), dict(ws=FAKE + 8),
                dict(err=FAKE + 1)):
        assert sample(lib, **bad) == EALIGN, bad


def verify(lib, lq, z=FAKE, dtype=0, stride=64, q=FAKE, nd=6, ds=64, dr=None, rows=FAKE, d=FAKE,
           u=FAKE, T=FAKE, k=None, B=2, K=3, V=64, out=FAKE, acc=FAKE, p=None, ws=FAKE, wsb=1 << 30,
           err=None):
    if lq:
        return lib.spec_verify_filtered_lq(z, dtype, stride, q, nd, ds, dr, rows, d, u, T, k, None,
                                           None, B, K, V, out, acc, p, ws, wsb, err, None)
    return lib.spec_verify_filtered(z, dtype, stride, q, d, u, T, k, None, None, B, K, V, out, acc,
                                    p, ws, wsb, err, None)


@pytest.mark.parametrize("lq", [False, True])
def test_verify_checks(lib, lq):
    none = dict.fromkeys(("z", "q", "d", "u", "T", "out", "acc", "ws"))
    assert verify(lib, lq, B=0, wsb=0, **none) == OK
    for bad in (dict(B=-1), dict(K=-1), dict(K=64), dict(V=0), dict(V=(1 << 19) + 1),
                dict(stride=63), dict(B=(1 << 20) + 1)):
        assert verify(lib, lq, **bad) == ESHAPE, bad
    assert verify(lib, lq, dtype=2) == EDTYPE
    for n in ("z", "q", "d", "u", "T", "out", "acc"):
        assert verify(lib, lq, **{n: None}) == ENULL, n
    assert verify(lib, lq, ws=None) == EWS and verify(lib, lq, wsb=64) == EWS
    for bad in (dict(z=FAKE + 2), dict(q=FAKE + 1), dict(d=FAKE + 1), dict(u=FAKE + 2),
                dict(T=FAKE + 1), dict(k=FAKE + 2), dict(out=FAKE + 1), dict(acc=FAKE + 1),
                dict(p=FAKE + 2), dict(ws=FAKE + 4), dict(err=FAKE + 1)):
        assert verify(lib, lq, **bad) == EALIGN, bad
    if lq:
        for bad in (dict(nd=5), dict(nd=-1, dr=FAKE), dict(ds=63)):
            assert verify(lib, True, **bad) == ESHAPE, bad
        assert verify(lib, True, rows=None) == ENULL
        assert verify(lib, True, rows=FAKE + 8) == EALIGN
        assert verify(lib, True, dr=FAKE + 1) == EALIGN


def append(lib, q=FAKE, k=FAKE, v=FAKE, dtype=1, qs=256, ks=128, vs=128, pos=FAKE, slot=FAKE,
           inv=FAKE, rot=64, inter=0, scale=1.0, R=3, Hq=4, Hkv=2, D=64, kc=FAKE, vc=FAKE, cd=1,
           nb=4, bs=16, st=(2048, 128, 64), ksc=None, vsc=None, oq=FAKE, oqs=256, err=None):
    return lib.peagle_append_kv(q, k, v, dtype, qs, ks, vs, pos, slot, inv, rot, inter, scale, R, Hq,
                                Hkv, D, kc, vc, cd, nb, bs, *st, ksc, vsc, oq, oqs, err, None)


def test_append_checks(lib):
    none = dict.fromkeys(("q", "k", "v", "pos", "slot", "inv", "kc", "vc", "oq"))
    assert append(lib, R=0, **none) == OK
    for bad in (dict(R=-1), dict(R=1 << 31), dict(Hq=-1), dict(Hq=1025), dict(Hkv=0),
                dict(Hkv=1025), dict(D=0), dict(D=1025), dict(rot=-2), dict(rot=63), dict(rot=66),
                dict(nb=0), dict(bs=0), dict(qs=255), dict(ks=127), dict(vs=127), dict(oqs=255),
                dict(st=(-1, 128, 64)), dict(st=(2048, -1, 64)), dict(st=(2048, 128, -1))):
        assert append(lib, **bad) == ESHAPE, bad
    assert append(lib, dtype=3, cd=3) == EDTYPE and append(lib, dtype=1, cd=2) == EDTYPE
    assert append(lib, scale=float("inf")) == EVALUE
    assert append(lib, ksc=FAKE) == EVALUE                    # scales without e4m3
    for n in none:
        assert append(lib, **{n: None}) == ENULL, n
    for bad in (dict(q=FAKE + 1), dict(k=FAKE + 1), dict(v=FAKE + 1), dict(pos=FAKE + 4),
                dict(slot=FAKE + 4), dict(inv=FAKE + 2), dict(kc=FAKE + 1), dict(vc=FAKE + 1),
                dict(oq=FAKE + 1), dict(cd=3, ksc=FAKE + 1), dict(cd=3, vsc=FAKE + 2),
                dict(err=FAKE + 2)):
        assert append(lib, **bad) == EALIGN, bad


def test_append_refuses_caches_that_overlap_themselves(lib):
    """Strides below head_dim where the dimension is longer than 1; any stride where it is not."""
    base = dict(R=0)
    assert append(lib, **base) == OK
    for st in ((2048, 128, 63), (2048, 63, 64), (63, 128, 64), (0, 128, 64), (2048, 0, 64)):
        assert append(lib, st=st, **base) == ESHAPE, st
    assert append(lib, Hkv=1, st=(2048, 128, 0), **base) == OK
    assert append(lib, nb=1, st=(0, 128, 64), **base) == OK
    assert append(lib, bs=1, st=(2048, 0, 64), **base) == OK
