"""Host-side refusals of the shared-prefix decode (no GPU)."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def ia():
    from integer_only_quantized_b200 import build
    build.build()
    import integer_only_quantized_b200 as mod
    mod.lib()
    return mod


P = 4096  # an aligned address that is never dereferenced


def _call(ia, q=P, kp=P, vp=P, Lp=5, Lp_max=5, kc=P, vc=P, lengths=P, sc=None, B=1, H=4, Hkv=2, Lmax=7, d=64,
          clip_c=8.0, dt=2, out=P, ws=P, ws_bytes=1 << 30, **scales):
    f = dict(s_q=0.1, s_k=0.1, s_v=0.1, s_o=0.1)
    f.update(scales)
    s, keep = ia.Scales(**f)._c()
    return ia.lib().intattn_decode_shared(q, kp, vp, Lp, Lp_max, kc, vc, lengths, s, B, H, Hkv, Lmax, d, clip_c, dt,
                                          out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), "INVALID_ARG"), (dict(kp=None), "INVALID_ARG"), (dict(vp=None), "INVALID_ARG"),
    (dict(kc=None), "INVALID_ARG"), (dict(vc=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(H=5), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"), (dict(B=-1), "INVALID_ARG"), (dict(Lp=-1), "INVALID_ARG"),
    (dict(Lp=6), "INVALID_ARG"), (dict(Lmax=-1), "INVALID_ARG"), (dict(Lp=0, Lp_max=0, Lmax=0), "INVALID_ARG"),
    (dict(Lp=60000, Lp_max=60000, Lmax=6000), "INVALID_ARG"), (dict(Lp=65536, Lp_max=65536), "INVALID_ARG"),
    (dict(d=80), "UNSUPPORTED"), (dict(dt=3), "UNSUPPORTED"), (dict(q=P + 8), "UNSUPPORTED"),
    (dict(kp=P + 1), "UNSUPPORTED"), (dict(vc=P + 4), "UNSUPPORTED"), (dict(lengths=P + 2), "UNSUPPORTED"),
    (dict(out=P + 8), "UNSUPPORTED"), (dict(ws=None), "WORKSPACE"), (dict(ws=P + 64), "WORKSPACE"),
    (dict(ws_bytes=8), "WORKSPACE"), (dict(clip_c=0.0), "PARAM_RANGE"), (dict(s_k=-1.0), "PARAM_RANGE"),
    (dict(s_o=float("nan")), "PARAM_RANGE"), (dict(z_k=256), "INVALID_ARG"), (dict(z_v=-3), "INVALID_ARG"),
    (dict(B=70000, H=1, Hkv=1), "UNSUPPORTED"), (dict(B=0), "OK"),
])
def test_refusals(ia, kw, want):
    assert _call(ia, **kw) == (ia.OK if want == "OK" else getattr(ia, "ERR_" + want))


def test_heads_limit_and_grouped_entries(ia):
    many = np.full(130, 0.1, np.float32)
    kw = dict(s_q=many, s_k=many, s_v=many, s_o=many, per_head=True, B=0)
    assert _call(ia, H=130, Hkv=130, **kw) == ia.ERR_UNSUPPORTED
    assert _call(ia, H=128, Hkv=2, **kw) == ia.OK
    # one bad K scale belongs to the whole group of its K / V head
    bad = many.copy()
    bad[1] = 0
    assert _call(ia, H=128, Hkv=2, **{**kw, "s_k": bad}) == ia.ERR_PARAM_RANGE
    assert _call(ia, H=128, Hkv=1, **{**kw, "s_k": bad}) == ia.OK


def test_workspace_size(ia):
    assert ia.decode_shared_workspace_size(2, 8, 3, 100, 64) == 0
    assert ia.decode_shared_workspace_size(2, 8, 4, -1, 64) == 0
    assert ia.decode_shared_workspace_size(2, 8, 4, 100, 96) == 0
    assert ia.decode_shared_workspace_size(2, 8, 4, 0, 64) > 0
