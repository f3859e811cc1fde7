"""Outputs of the row operators that overlap are refused on the host (no GPU:
every call here ends at the refusal)."""
import pytest


@pytest.fixture(scope="module")
def ia():
    from integer_only_quantized_b200 import build
    build.build()
    import integer_only_quantized_b200 as mod
    mod.lib()
    return mod


A = 1 << 20  # aligned addresses that are never dereferenced
B, H, HKV, L, LMAX, D = 2, 4, 2, 3, 16, 64


def _write(ia, kc, vc, q_out=None, bits=8):
    s, keep = ia.Scales(0.1, 0.1, 0.1, 0.1)._c()
    r = ia._Rows(A, 4096, 64, 1024)
    return ia.lib().intattn_cache_write(r, r, r if q_out else None, 1, s, bits, None, B, H, HKV, L, LMAX, D, A, None, kc,
                                        vc, q_out, None)


@pytest.mark.parametrize("bits", [8, 4])
def test_caches(ia, bits):
    size = B * HKV * LMAX * D * bits // 8
    far = A + (1 << 22)
    for kc, vc in ((A, A), (A, A + size - 16), (A + size - 16, A), (A, A + 16)):
        assert _write(ia, kc, vc, bits=bits) == ia.ERR_INVALID_ARG
    q_size = B * H * L * D
    for q_out in (A, A + size - 16, A - q_size + 16, far, far + size - 16, far - q_size + 16):
        assert _write(ia, A, far, q_out, bits) == ia.ERR_INVALID_ARG


def test_values(ia):
    s, keep = ia.Scales(0.1, 0.1, 0.1, 0.1)._c()
    size = 2 * B * HKV * L * D
    for k_out, v_out in ((A, A), (A, A + size - 16), (A + size - 16, A)):
        assert ia.lib().intattn_cache_read(A, A, s, 8, B, HKV, L, LMAX, D, A, None, 1, k_out, v_out,
                                           None) == ia.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(q_out="k"), dict(k_out="q"), dict(q_out="x", k_out="x"), dict(q_out="q2"),
                                dict(k_out="k2")])
def test_norm_rope(ia, kw):
    rows = dict(q=ia._Rows(A, 4096, 64, 1024), k=ia._Rows(A + 512, 4096, 64, 1024), x=ia._Rows(A + 65536, 4096, 64, 1024),
                q2=ia._Rows(A, 4096, 192, 64), k2=ia._Rows(A + 512, 8192, 64, 1024))
    f = dict(q_out="q", k_out="k")
    f.update(kw)
    rn = ia._RopeNorm(A, A, 1e-6, None, 0, 0, 0, None)
    assert ia.lib().intattn_qk_norm_rope(rows["q"], rows["k"], rn, 1, B, H, HKV, L, D, rows[f["q_out"]], rows[f["k_out"]],
                                         None) == ia.ERR_INVALID_ARG
