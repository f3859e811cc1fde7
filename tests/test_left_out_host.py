"""The dtype flag for rows that a call leaves out, as the C ABI checks it (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def ia():
    from integer_only_quantized_b200 import build
    build.build()
    import integer_only_quantized_b200 as mod
    mod.lib()
    return mod


P = 4096  # an aligned address that is never dereferenced


def _calls(ia, dtype):
    """Return codes of the four calls without any row (they end after their checks)."""
    s, keep = ia.Scales(0.1, 0.1, 0.1, 0.1)._c()
    r = ia._Rows(P, 512, 64, 128)
    rn = ia._RopeNorm(P, P, 1e-6, P, 10, 64, 0, P)
    L = ia.lib()
    return {"norm": L.intattn_qk_norm_rope(r, r, rn, dtype, 0, 2, 1, 3, 64, r, r, None),
            "write": L.intattn_cache_write(r, r, r, dtype, s, 8, rn, 0, 2, 1, 3, 9, 64, P, None, P, P, P, None),
            "read": L.intattn_cache_read(P, P, s, 8, 0, 1, 3, 9, 64, P, None, dtype, P, P, None),
            "shared": L.intattn_decode_shared(P, P, P, 5, 5, P, P, P, s, 0, 4, 2, 7, 64, 8.0, dtype, P, P, 1 << 20, None)}


def test_accepted(ia):
    for dtype in (ia.DTYPE_FP16, ia.DTYPE_BF16):
        for flag in (0, ia.ZERO_LEFT_OUT):
            assert set(_calls(ia, dtype | flag).values()) == {ia.OK}


def test_refused(ia):
    for dtype in (3, -1, 3 | ia.ZERO_LEFT_OUT, 0x200, 0x300, -1 ^ ia.ZERO_LEFT_OUT, -256, -2 ** 31):
        assert set(_calls(ia, dtype).values()) == {ia.ERR_UNSUPPORTED}, dtype
    # the codes are an output type of the shared decode alone
    got = _calls(ia, ia.DTYPE_INT8 | ia.ZERO_LEFT_OUT)
    assert got.pop("shared") == ia.OK and set(got.values()) == {ia.ERR_UNSUPPORTED}
