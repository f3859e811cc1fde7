"""Host-side checks of the row operators (no GPU): refusals before anything
reaches the device, and pins of the numpy oracle the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from oracle import rows as orow


@pytest.fixture(scope="module")
def ia():
    from integer_only_quantized_b200 import build
    build.build()
    import integer_only_quantized_b200 as mod
    mod.lib()
    return mod


P = 4096  # an aligned address that is never dereferenced


def _r(ia, ptr=P, sb=512, sh=64, sl=128):
    return ia._Rows(ptr, sb, sh, sl)


def _norm(ia, q=True, k=True, q_out=True, k_out=True, dtype=1, B=1, H=2, Hkv=1, L=3, d=64, **kw):
    f = dict(w_q=P, w_k=P, eps=1e-6, table=P, n_positions=10, rot=64, interleaved=0, positions=P)
    f.update(kw)
    mk = lambda x: _r(ia) if x is True else (x or None)
    return ia.lib().intattn_qk_norm_rope(mk(q), mk(k), ia._RopeNorm(**f), dtype, B, H, Hkv, L, d, mk(q_out), mk(k_out),
                                         None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=False), "INVALID_ARG"), (dict(q_out=False), "INVALID_ARG"), (dict(k_out=False), "INVALID_ARG"),
    (dict(k=False), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"), (dict(B=-1), "INVALID_ARG"),
    (dict(H=0), "INVALID_ARG"), (dict(L=-2), "INVALID_ARG"), (dict(d=32), "UNSUPPORTED"), (dict(d=96), "UNSUPPORTED"),
    (dict(dtype=2), "UNSUPPORTED"), (dict(rot=8), "UNSUPPORTED"), (dict(rot=80), "INVALID_ARG"),
    (dict(rot=-16), "INVALID_ARG"), (dict(n_positions=0), "INVALID_ARG"), (dict(positions=None), "INVALID_ARG"),
    (dict(positions=P + 2), "UNSUPPORTED"), (dict(table=P + 8), "UNSUPPORTED"), (dict(w_q=P + 4), "UNSUPPORTED"),
    (dict(eps=0.0), "PARAM_RANGE"), (dict(eps=float("nan")), "PARAM_RANGE"), (dict(eps=float("inf")), "PARAM_RANGE"),
    (dict(B=0), "OK"), (dict(L=0), "OK"), (dict(B=0, eps=-1.0), "PARAM_RANGE"),
])
def test_norm_rope_refusals(ia, kw, want):
    code = ia.OK if want == "OK" else getattr(ia, "ERR_" + want)
    assert _norm(ia, **kw) == code


@pytest.mark.parametrize("row,want", [(dict(ptr=P + 8), "UNSUPPORTED"), (dict(sl=12), "UNSUPPORTED"),
                                      (dict(sh=4), "UNSUPPORTED"), (dict(sb=1), "UNSUPPORTED"),
                                      (dict(ptr=None), "INVALID_ARG")])
@pytest.mark.parametrize("which", ["q", "k", "q_out", "k_out"])
def test_norm_rope_row_refusals(ia, row, want, which):
    assert _norm(ia, **{which: _r(ia, **row)}) == getattr(ia, "ERR_" + want)


def test_norm_rope_refuses_repeated_output_rows(ia):
    for kw in (dict(sl=0), dict(sh=0)):
        assert _norm(ia, q_out=_r(ia, **kw)) == ia.ERR_INVALID_ARG
    assert _norm(ia, q_out=_r(ia, sb=0), B=2) == ia.ERR_INVALID_ARG


def _scales(ia, **kw):
    f = dict(s_q=0.1, s_k=0.1, s_v=0.1, s_o=0.1)
    f.update(kw)
    return ia.Scales(**f)


def _write(ia, sc=None, k=True, v=True, q=False, bits=8, rn=None, B=1, H=2, Hkv=1, L=3, Lmax=9, d=64, start=P,
           lengths=None, kc=P, vc=P, q_out=None, dtype=1):
    s, keep = (sc or _scales(ia))._c()
    mk = lambda x: _r(ia) if x is True else (x or None)
    return ia.lib().intattn_cache_write(mk(k), mk(v), mk(q), dtype, s, bits, rn, B, H, Hkv, L, Lmax, d, start, lengths,
                                        kc, vc, q_out, None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=False), "INVALID_ARG"), (dict(v=False), "INVALID_ARG"), (dict(q=True), "INVALID_ARG"),
    (dict(q_out=P), "INVALID_ARG"), (dict(bits=5), "UNSUPPORTED"), (dict(d=72), "UNSUPPORTED"),
    (dict(dtype=-1), "UNSUPPORTED"), (dict(Hkv=0), "INVALID_ARG"), (dict(L=-1), "INVALID_ARG"),
    (dict(Lmax=-1), "INVALID_ARG"), (dict(start=None), "INVALID_ARG"), (dict(start=P + 1), "UNSUPPORTED"),
    (dict(lengths=P + 2), "UNSUPPORTED"), (dict(kc=None), "INVALID_ARG"), (dict(vc=P + 8), "UNSUPPORTED"),
    (dict(q=True, q_out=P + 4), "UNSUPPORTED"), (dict(q=True, q_out=P, H=0), "INVALID_ARG"),
    (dict(B=0, start=None), "OK"),
])
def test_cache_write_refusals(ia, kw, want):
    code = ia.OK if want == "OK" else getattr(ia, "ERR_" + want)
    assert _write(ia, **kw) == code


@pytest.mark.parametrize("sc,bits,want", [
    (dict(s_k=0.0), 8, "PARAM_RANGE"), (dict(s_v=-1.0), 8, "PARAM_RANGE"), (dict(s_k=float("inf")), 8, "PARAM_RANGE"),
    (dict(s_v=float("nan")), 4, "PARAM_RANGE"), (dict(z_k=256), 8, "INVALID_ARG"), (dict(z_k=-1), 8, "INVALID_ARG"),
    (dict(z_v=16), 4, "INVALID_ARG"), (dict(z_v=16), 8, "OK"), (dict(s_q=0.0), 8, "OK"), (dict(s_o=0.0), 8, "OK"),
])
def test_cache_scale_refusals(ia, sc, bits, want):
    """Checked before the launch: with no rows at all the call ends after the checks."""
    code = ia.OK if want == "OK" else getattr(ia, "ERR_" + want)
    assert _write(ia, sc=_scales(ia, **sc), bits=bits, B=0) == code
    s, keep = _scales(ia, **sc)._c()
    assert ia.lib().intattn_cache_read(P, P, s, bits, 0, 1, 3, 9, 64, P, None, 1, P, P, None) == code


def test_cache_heads_limit(ia):
    many = np.full(200, 0.1, np.float32)
    assert _write(ia, sc=_scales(ia, s_k=many, s_v=many, per_head=True), Hkv=129) == ia.ERR_UNSUPPORTED
    assert _write(ia, sc=_scales(ia, s_q=many, s_k=many, s_v=many, per_head=True), q=True, q_out=P,
                  H=129) == ia.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), "INVALID_ARG"), (dict(k_out=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"),
    (dict(v_out=None), "INVALID_ARG"), (dict(k=P + 8), "UNSUPPORTED"), (dict(v_out=P + 2), "UNSUPPORTED"),
    (dict(start=None), "INVALID_ARG"), (dict(bits=16), "UNSUPPORTED"), (dict(d=256), "UNSUPPORTED"),
    (dict(dtype=3), "UNSUPPORTED"), (dict(Hkv=0), "INVALID_ARG"), (dict(L=-1), "INVALID_ARG"), (dict(L=0, k=None), "OK"),
])
def test_cache_read_refusals(ia, kw, want):
    f = dict(k=P, v=P, bits=8, B=1, Hkv=1, L=3, Lmax=9, d=64, start=P, lengths=None, dtype=1, k_out=P, v_out=P)
    f.update(kw)
    s, keep = _scales(ia)._c()
    rc = ia.lib().intattn_cache_read(f["k"], f["v"], s, f["bits"], f["B"], f["Hkv"], f["L"], f["Lmax"], f["d"],
                                     f["start"], f["lengths"], f["dtype"], f["k_out"], f["v_out"], None)
    assert rc == (ia.OK if want == "OK" else getattr(ia, "ERR_" + want))


# ------------------------------------------------------------- oracle pins

def test_oracle_rotation_keeps_lengths_and_composes():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 5, 64))
    for il in (False, True):
        ang = np.arange(40)[:, None] * (10000.0 ** (-np.arange(16) / 16.0))
        table = np.stack([np.cos(ang), np.sin(ang)], -1)
        pos = rng.integers(0, 20, (2, 5))
        y, _ = orow.norm_rope(x, table=table, positions=pos, interleaved=il)
        assert np.allclose((y[..., :32] ** 2).sum(-1), (x[..., :32] ** 2).sum(-1))
        assert np.array_equal(y[..., 32:], x[..., 32:])  # past rot
        # turning by p and then by r is turning by p + r
        z, _ = orow.norm_rope(y, table=table, positions=pos * 0 + 13, interleaved=il)
        both, _ = orow.norm_rope(x, table=table, positions=pos + 13, interleaved=il)
        assert np.allclose(z, both)


def test_oracle_norm_has_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((1, 2, 4, 128)) * 7
    y, _ = orow.norm_rope(x, w=np.ones(128), eps=1e-12)
    assert np.allclose((y * y).mean(-1), 1.0)


def test_oracle_codes_by_hand():
    # s = 0.5: inv = 2; ties go to even, values past the range saturate, NaN is the code of 0
    x = np.array([0.25, 0.75, -0.25, -0.75, 63.5, 64.0, -1e30, np.inf, -np.inf, np.nan, 0.3, -0.0], np.float32)
    x = x.reshape(1, 1, 1, -1)
    assert orow.codes(x, [0.5]).ravel().tolist() == [0, 2, 0, -2, 127, 127, -127, 127, -127, 0, 1, 0]
    assert orow.codes(x, [0.5], [7], 4).ravel().tolist() == [7, 9, 7, 5, 15, 15, 0, 15, 0, 7, 8, 7]
    c = np.arange(-7, 8).repeat(2)[:16]
    assert np.array_equal(orow.unpack(orow.pack(c, 4, False), 4, False), c)


def test_positions_without_a_table_are_refused(ia):
    assert _norm(ia, table=None) == ia.ERR_INVALID_ARG
    assert _norm(ia, table=None, positions=None, B=0) == ia.OK
