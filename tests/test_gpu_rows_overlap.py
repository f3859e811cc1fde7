"""Outputs of the row operators beside each other in one allocation are taken,
overlapping ones are refused before anything is written."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ia():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from integer_only_quantized_b200 import build
    build.build()
    import integer_only_quantized_b200 as mod
    mod.lib()
    return mod


def test_neighbours_and_overlaps(ia):
    import torch
    B, H, L, Lmax, d = 2, 2, 3, 5, 64
    x = torch.randn((B, L, 3 * H, d), device="cuda").to(torch.bfloat16)
    q, k, v = (t.transpose(1, 2) for t in x.split(H, dim=2))
    sc = ia.Scales(0.03, 0.03, 0.03, 1)
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    n, m = B * H * Lmax * d, B * H * L * d
    buf = torch.full((2 * n + m,), 77, dtype=torch.int8, device="cuda")
    kc, vc = buf[:n].view(B, H, Lmax, d), buf[n:2 * n].view(B, H, Lmax, d)
    qo = buf[2 * n:].view(B, H, L, d)
    for bad in (dict(v_cache=kc), dict(v_cache=buf[16:n + 16].view(B, H, Lmax, d)),
                dict(q_out=buf[n - 16:n - 16 + m].view(B, H, L, d))):
        with pytest.raises(ia.IntAttnError):
            ia.cache_write(**{**dict(k=k, v=v, scales=sc, k_cache=kc, v_cache=vc, start=st, q=q, q_out=qo), **bad})
    assert bool((buf == 77).all())
    ia.cache_write(k, v, sc, kc, vc, st, q=q, q_out=qo)
    own = [torch.full((B, H, Lmax, d), 77, dtype=torch.int8, device="cuda") for _ in range(2)]
    want = ia.cache_write(k, v, sc, *own, st, q=q)
    assert torch.equal(kc, own[0]) and torch.equal(vc, own[1]) and torch.equal(qo, want)
    out = torch.zeros(2 * m, dtype=torch.bfloat16, device="cuda")
    ko, vo = out[:m].view(B, H, L, d), out[m:].view(B, H, L, d)
    with pytest.raises(ia.IntAttnError):
        ia.cache_read(kc, vc, sc, st, L, k_out=ko, v_out=ko)
    ia.cache_read(kc, vc, sc, st, L, k_out=ko, v_out=vo)
    assert all(torch.equal(a, b) for a, b in zip((ko, vo), ia.cache_read(kc, vc, sc, st, L)))
    rn = ia.RopeNorm(w_q=torch.ones(d, device="cuda"), w_k=torch.ones(d, device="cuda"))
    want = [t.clone() for t in ia.qk_norm_rope(q, k, rn)]
    keep = x.clone()
    for bad in (dict(q_out=k), dict(k_out=q), dict(q_out=ko, k_out=ko)):
        with pytest.raises(ia.IntAttnError):
            ia.qk_norm_rope(q, k, rn, **{**dict(q_out=q, k_out=k), **bad})
    assert torch.equal(x, keep)
    ia.qk_norm_rope(q, k, rn, q_out=q, k_out=k)  # in place, in one packed buffer
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep[:, :, 2 * H:].transpose(1, 2))
    assert ia.device_error() == ia.OK
