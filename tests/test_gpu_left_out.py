"""Rows that a call leaves out (padding, lengths, positions and cache rows out of
range): 0 in an output that the call makes itself, whatever its memory held
before, and as they were in an output that the caller passes."""
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


@pytest.fixture(autouse=True)
def dirty():
    """Freed memory full of NaN patterns (0xFF bytes), in blocks of the sizes used here."""
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in [2048, 8192, 65536, 1 << 19] * 8 + [1 << 23] * 4]
    del old


def _packed(B, L, heads, d, dtype):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(B + L + d)
    x = torch.randn((B, L, sum(heads), d), device="cuda", generator=g).to(dtype)
    return [t.transpose(1, 2) for t in x.split(list(heads), dim=2)]


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48)])
@pytest.mark.parametrize("name", ["float16", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_padded_positions(ia, d, rot, name, interleaved):
    import torch
    B, L = 3, 70
    q, k, _ = _packed(B, L, (9, 2, 1), d, getattr(torch, name))
    pos = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
    for b, n in enumerate((70, 1, 33)):
        pos[b, n:] = -1
    w = torch.rand(d, device="cuda") + 0.5
    rn = ia.RopeNorm(ia.rope_table(L, rot), pos, w, w, interleaved=interleaved)
    live = (pos >= 0)[:, None, :, None]
    passed = [torch.full(t.shape, 3.0, dtype=t.dtype, device="cuda") for t in (q, k)]
    ia.qk_norm_rope(q, k, rn, q_out=passed[0], k_out=passed[1])
    fresh = ia.qk_norm_rope(q, k, rn)
    assert ia.device_error() == ia.OK
    for f, p in zip(fresh, passed):
        assert torch.equal(f, torch.where(live, p, 0)) and bool((p.masked_select(~live) == 3).all())
    # the next step over the whole tensor: a scale per tensor from the live rows alone
    codes = [ia.quantize(t, False) for t in (fresh[0], torch.where(live, passed[0], 0))]
    assert torch.equal(codes[0][0], codes[1][0]) and torch.equal(codes[0][1], codes[1][1])
    # one output passed, the other not; queries only
    mine = torch.full(k.shape, 3.0, dtype=k.dtype, device="cuda")
    fq, _ = ia.qk_norm_rope(q, k, rn, k_out=mine)
    assert torch.equal(fq, fresh[0]) and torch.equal(mine, passed[1])
    mine = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    _, fk = ia.qk_norm_rope(q, k, rn, q_out=mine)
    assert torch.equal(fk, fresh[1]) and torch.equal(mine, passed[0])
    assert torch.equal(ia.qk_norm_rope(q, None, rn)[0], fresh[0])


def test_positions_past_the_table(ia):
    import torch
    q, k, _ = _packed(1, 4, (3, 1, 1), 64, torch.bfloat16)
    rn = ia.RopeNorm(ia.rope_table(8, 64), _i32([[7, 8, -1, 2 ** 31 - 1]]))
    fq, fk = ia.qk_norm_rope(q, k, rn)
    assert ia.device_error() == ia.ERR_PARAM_RANGE
    assert not fq[:, :, 1:].any() and not fk[:, :, 1:].any() and bool(fq[:, :, 0].any())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rotated", [False, True])
def test_queries_of_cache_write(ia, d, rotated):
    import torch
    B, H, Hkv, L = 3, 6, 2, 9
    q, k, v = _packed(B, L, (H, Hkv, Hkv), d, torch.float16)
    ln = _i32([9, 0, 4])
    live = torch.arange(L, device="cuda") < ln[:, None]
    rn = None
    if rotated:
        pos = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
        pos[0, 5] = -1
        live[0, 5] = False
        rn = ia.RopeNorm(ia.rope_table(L, 16), pos, torch.ones(d, device="cuda"), torch.ones(d, device="cuda"))
    sc = ia.Scales(0.03, 0.03, 0.03, 1)
    mk = lambda: [torch.full((B, Hkv, 16, d), 5, dtype=torch.int8, device="cuda") for _ in range(2)]
    passed = torch.full((B, H, L, d), 99, dtype=torch.int8, device="cuda")
    c1, c2 = mk(), mk()
    ia.cache_write(k, v, sc, *c1, _i32([0, 3, 7]), lengths=ln, q=q, q_out=passed, norm=rn)
    fresh = ia.cache_write(k, v, sc, *c2, _i32([0, 3, 7]), lengths=ln, q=q, norm=rn)
    assert ia.device_error() == ia.OK
    live = live[:, None, :, None]
    assert torch.equal(fresh, torch.where(live, passed, 0)) and bool((passed.masked_select(~live) == 99).all())
    assert all(torch.equal(a, b) for a, b in zip(c1, c2)) and bool((c2[0][1] == 5).all())
    # cache rows that do not exist
    fresh = ia.cache_write(k, v, sc, *c2, _i32([-2, 100, 14]), q=q)
    assert ia.device_error() == ia.ERR_PARAM_RANGE
    assert not fresh[0, :, :2].any() and bool(fresh[0, :, 2].any())
    assert not fresh[1].any() and not fresh[2, :, 2:].any() and bool(fresh[2, :, :2].any())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits,zp", [(8, None), (8, 130), (4, None), (4, 9)])
@pytest.mark.parametrize("L", [1, 37, 300])
def test_values_read_back(ia, d, bits, zp, L):
    import torch
    B, H, Lmax = 4, 3, 320
    u8 = bits == 4 or zp is not None
    caches = [torch.randint(0, 256, (B, H, Lmax, d * bits // 8), device="cuda").to(torch.uint8) for _ in range(2)]
    caches = caches if u8 else [c.view(torch.int8) for c in caches]
    sc = ia.Scales(1, 0.02, 0.03, 1, z_k=zp, z_v=zp)
    st, ln = _i32([0, 5, 20, 19]), _i32([L, 0, max(L - 3, 0), L + 7])
    live = (torch.arange(L, device="cuda") < ln[:, None])[:, None, :, None]
    mk = lambda: torch.full((B, H, L, d), 7.0, dtype=torch.float16, device="cuda")
    passed = [mk(), mk()]
    kw = dict(lengths=ln, bits=bits, dtype=torch.float16)
    ia.cache_read(*caches, sc, st, L, k_out=passed[0], v_out=passed[1], **kw)
    fresh = ia.cache_read(*caches, sc, st, L, **kw)
    assert ia.device_error() == ia.OK
    for f, p in zip(fresh, passed):
        assert torch.equal(f, torch.where(live, p, 0)) and bool((p.masked_select(~live) == 7).all())
    assert torch.equal(ia.cache_read(caches[0], None, sc, st, L, **kw)[0], fresh[0])
    mine = mk()
    _, fv = ia.cache_read(*caches, sc, st, L, k_out=mine, **kw)
    assert torch.equal(fv, fresh[1]) and torch.equal(mine, passed[0])
    # cache rows that do not exist
    fk, fv = ia.cache_read(*caches, sc, _i32([-1, Lmax, -L, Lmax - 1]), L, bits=bits)
    assert ia.device_error() == ia.ERR_PARAM_RANGE
    for f in (fk, fv):
        assert not f[0, :, 0].any() and not f[1].any() and not f[2].any() and not f[3, :, 1:].any()
        assert bool(f[3, :, 0].any())


@pytest.mark.parametrize("name", ["int8", "float16", "bfloat16"])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_of_the_shared_decode(ia, d, name):
    import torch
    dt = getattr(torch, name)
    B, H, Hkv, Lp, Lmax = 5, 4, 2, 140, 30
    mk = lambda *s: torch.randint(-100, 101, s, device="cuda").to(torch.int8)
    q, kp, vp, kc, vc = mk(B, H, 1, d), mk(Hkv, Lp, d), mk(Hkv, Lp, d), mk(B, Hkv, Lmax, d), mk(B, Hkv, Lmax, d)
    sc = ia.Scales(0.02, 0.02, 0.03, 0.03)
    passed = torch.full((B, H, 1, d), 55, dtype=dt, device="cuda")
    ln = _i32([30, -1, 0, 31, 9])
    ia.decode_shared(q, kp, vp, kc, vc, ln, sc, 10.0, out=passed)
    assert ia.device_error() == ia.ERR_PARAM_RANGE
    fresh = ia.decode_shared(q, kp, vp, kc, vc, ln, sc, 10.0, dtype=dt)
    assert ia.device_error() == ia.ERR_PARAM_RANGE
    bad = _i32([1, 3]).long()
    assert bool((passed[bad] == 55).all()) and not fresh[bad].any()
    good = _i32([0, 2, 4]).long()
    assert torch.equal(fresh[good], passed[good]) and bool(fresh[good].any())
