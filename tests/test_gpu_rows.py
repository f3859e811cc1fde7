"""GPU tests of the row operators against the float64 oracle: norm and
rotation, cache_write (with and without them), cache_read, and their rows
left alone."""
import numpy as np
import pytest

from oracle import rows as orow

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


def _packed(rng, B, L, heads, d, dtype, scale=1.0):
    """Views [B, h, L, d] of one packed projection, and their float32 values."""
    import torch
    x = rng.standard_normal((B, L, sum(heads), d)).astype(np.float32)
    x *= np.exp(rng.standard_normal((sum(heads), d))).astype(np.float32) * np.float32(scale)
    t = torch.from_numpy(x).to(dtype).cuda()
    views = [v.transpose(1, 2) for v in t.split(list(heads), dim=2)]
    return views, [v.float().cpu().numpy() for v in views]


def _close(got, want, mag, dtype):
    """One rounding to dtype (half a step relative, half the smallest
    subnormal) of an fp32 value.  fp32 part, in units of 2^-24 of the magnitudes
    added: the sum of up to 128 squares (8 fused steps, 4 shuffled adds: 12,
    halved by the root: 6), mean and eps 2 (halved: 1), reciprocal root 4 (two units
    in the last place), two products 2, rotation 3: 16."""
    import torch
    eps = torch.finfo(dtype).eps
    tiny = torch.finfo(dtype).smallest_normal * eps
    bound = eps / 2 * np.abs(want) * (1 + 1e-3) + tiny / 2 + 16 * 2.0 ** -24 * mag
    bad = np.abs(got - want) > bound
    assert not bad.any(), f"{bad.sum()} of {bad.size}; first {np.argwhere(bad)[:3].tolist()}"


NORM = [  # B, H, Hkv, L, d, rot, interleaved, norm q, norm k
    (1, 1, 1, 1, 64, 64, False, True, True),
    (2, 12, 12, 1, 64, 64, True, True, True),
    (3, 5, 1, 7, 128, 128, False, True, False),
    (2, 6, 3, 33, 128, 64, False, False, True),
    (1, 3, 1, 19, 64, 16, True, True, True),
    (2, 4, 2, 5, 128, 112, True, True, True),
    (1, 7, 7, 3, 64, 48, False, True, True),
    (1, 32, 8, 700, 128, 128, False, True, True),
    (4, 12, 4, 301, 64, 0, False, True, True),
]


@pytest.mark.parametrize("dtype_name", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", NORM, ids=lambda c: "B{}H{}k{}L{}d{}r{}{}".format(*c[:6], "i" if c[6] else ""))
def test_norm_rope(ia, case, dtype_name):
    import torch
    B, H, Hkv, L, d, rot, il, nq, nk = case
    dtype = getattr(torch, dtype_name)
    rng = np.random.default_rng(sum(case))
    (q, k, _), (q32, k32, _) = _packed(rng, B, L, (H, Hkv, 2), d, dtype)
    w = [rng.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2)]
    table = ia.rope_table(50000, rot, 10000.0) if rot else None
    pos = rng.integers(0, 50000, (B, L)).astype(np.int32)
    dev = [torch.from_numpy(x).cuda() for x in w]
    rn = ia.RopeNorm(table, torch.from_numpy(pos).cuda() if rot else None, dev[0] if nq else None,
                     dev[1] if nk else None, 1e-6, il)
    got = ia.qk_norm_rope(q, k, rn)
    assert ia.device_error() == ia.OK
    tn = None if table is None else table.cpu().numpy()
    for g, x, wx in ((got[0], q32, w[0] if nq else None), (got[1], k32, w[1] if nk else None)):
        assert g.is_contiguous() and g.dtype == dtype
        want, mag = orow.norm_rope(x, wx, 1e-6, tn, pos, il)
        _close(g.float().cpu().numpy().astype(np.float64), want, mag, dtype)


def test_rope_table_far_positions(ia):
    t = ia.rope_table(60001, 64, 1e6).cpu().numpy().astype(np.float64)
    f = 1e6 ** (-np.arange(0, 64, 2) / 64.0)
    ang = 60000 * f
    assert np.abs(t[60000] - np.stack([np.cos(ang), np.sin(ang)], -1)).max() < 2.0 ** -24 + 1e-10
    assert t[0, :, 0].tolist() == [1.0] * 32 and t[0, :, 1].tolist() == [0.0] * 32


def test_norm_rope_in_place_and_strided_outputs(ia):
    import torch
    rng = np.random.default_rng(5)
    (q, k, v), (q32, k32, v32) = _packed(rng, 2, 9, (4, 2, 2), 64, torch.bfloat16)
    rn = ia.RopeNorm(ia.rope_table(100, 64), torch.arange(18, dtype=torch.int32, device="cuda").view(2, 9),
                     torch.ones(64, device="cuda"), torch.ones(64, device="cuda"))
    want = [t.clone() for t in ia.qk_norm_rope(q, k, rn)]
    outs = torch.zeros((2, 9, 6, 64), dtype=torch.bfloat16, device="cuda")
    qo, ko = (t.transpose(1, 2) for t in outs.split([4, 2], dim=2))
    ia.qk_norm_rope(q, k, rn, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    only, none = ia.qk_norm_rope(q, None, rn)
    assert none is None and torch.equal(only, want[0])
    ia.qk_norm_rope(q, k, rn, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert np.array_equal(v.float().cpu().numpy(), v32)  # the packed neighbour


def test_norm_rope_padding_and_positions_out_of_range(ia):
    import torch
    q = torch.randn((1, 2, 4, 64), device="cuda").to(torch.float16)
    out = torch.full_like(q, 3.0)
    rn = ia.RopeNorm(ia.rope_table(8, 32), torch.tensor([[0, -1, 8, 7]], dtype=torch.int32, device="cuda"))
    ia.qk_norm_rope(q, None, rn, q_out=out)
    assert ia.device_error() == ia.ERR_PARAM_RANGE and ia.device_error() == ia.OK
    assert torch.equal(out[:, :, 0], q[:, :, 0]) and (out[:, :, 1:3] == 3.0).all() and not (out[:, :, 3] == 3.0).any()


def test_norm_rope_special_values(ia):
    """A row of zeros stays zero; an infinity or NaN touches its own row only."""
    import torch
    x = torch.randn((1, 1, 4, 128), device="cuda").to(torch.bfloat16)
    x[0, 0, 0] = 0
    x[0, 0, 1, 5] = float("inf")
    x[0, 0, 2, 7] = float("nan")
    rn = ia.RopeNorm(w_q=torch.ones(128, device="cuda"))
    y, _ = ia.qk_norm_rope(x, None, rn)
    assert (y[0, 0, 0] == 0).all() and torch.isnan(y[0, 0, 1, 5]) and (y[0, 0, 1, 6:] == 0).all()
    assert torch.isnan(y[0, 0, 2]).all() and torch.isfinite(y[0, 0, 3]).all()


# ------------------------------------------------------------------- caches

CACHE = [  # B, Hkv, L, Lmax, d, bits, zp, per_head
    (1, 1, 1, 1, 64, 8, False, False),
    (2, 3, 1, 40, 128, 8, True, True),
    (3, 2, 17, 50, 64, 4, False, True),
    (2, 5, 33, 64, 128, 4, True, True),
    (64, 8, 1, 70, 128, 8, False, True),
    (2, 4, 700, 1024, 128, 8, True, False),
    (1, 12, 333, 400, 64, 8, False, True),
]


def _cache_inputs(rng, case, dtype):
    import torch
    B, H, L, Lmax, d, bits, zp, per_head = case
    views, vals = _packed(rng, B, L, (H, H, 2 * H), d, dtype)
    n = H if per_head else 1
    s = rng.uniform(0.02, 0.08, (2, n)).astype(np.float32) * (16 if bits == 4 else 1)
    z = rng.integers(0, 2 ** bits, (2, n)).astype(np.int32) if zp else (None, None)
    u8 = zp or bits == 4
    cache = [rng.integers(0, 200, (B, H, Lmax, d * bits // 8)).astype(np.uint8) for _ in range(2)]
    cache = [c if u8 else c.view(np.int8) for c in cache]
    start = rng.integers(0, Lmax - L + 1, B).astype(np.int32)
    lengths = rng.integers(0, L + 1, B).astype(np.int32)
    lengths[-1] = L
    return views, vals, s, z, cache, start, lengths


@pytest.mark.parametrize("dtype_name", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", CACHE, ids=lambda c: "B{}H{}L{}m{}d{}b{}{}{}".format(*c[:6], "z" if c[6] else "", "h" if c[7] else ""))
def test_cache_write_and_read(ia, case, dtype_name):
    import torch
    B, H, L, Lmax, d, bits, zp, per_head = case
    dtype = getattr(torch, dtype_name)
    rng = np.random.default_rng(sum(case) + 77)
    views, vals, s, z, cache, start, lengths = _cache_inputs(rng, case, dtype)
    sc = ia.Scales(0.05, s[0], s[1], 1.0, per_head=per_head, z_k=z[0], z_v=z[1])
    if per_head:
        sc.s_q = np.full(2 * H, 0.05, np.float32)
    dev = [torch.from_numpy(c.copy()).cuda() for c in cache]
    st, ln = torch.from_numpy(start).cuda(), torch.from_numpy(lengths).cuda()
    q_out = torch.full((B, 2 * H, L, d), 99, dtype=torch.int8, device="cuda")
    ia.cache_write(views[0], views[1], sc, dev[0], dev[1], st, lengths=ln, bits=bits, q=views[2], q_out=q_out)
    assert ia.device_error() == ia.OK
    for i in range(2):
        want = orow.write(cache[i], vals[i], s[i], z[i], bits, start, lengths)
        assert np.array_equal(dev[i].cpu().numpy(), want)
    want_q = np.where((np.arange(L) < lengths[:, None])[:, None, :, None], orow.codes(vals[2], [0.05]), 99)
    assert np.array_equal(q_out.cpu().numpy(), want_q)
    # reading back, rows past lengths left as they were
    outs = [torch.full((B, H, L, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    ia.cache_read(dev[0], dev[1], sc, st, L, lengths=ln, bits=bits, dtype=dtype, k_out=outs[0], v_out=outs[1])
    assert ia.device_error() == ia.OK
    for i in range(2):
        v = torch.from_numpy(orow.values(dev[i].cpu().numpy(), s[i], z[i], bits, start, L)).to(dtype)
        live = (torch.arange(L) < torch.from_numpy(lengths)[:, None])[:, None, :, None]
        assert torch.equal(outs[i].cpu(), torch.where(live, v, torch.tensor(7.0, dtype=dtype)))
    k_only, none = ia.cache_read(dev[0], None, sc, st, L, bits=bits, dtype=dtype)
    assert none is None
    v = torch.from_numpy(orow.values(dev[0].cpu().numpy(), s[0], z[0], bits, start, L)).to(dtype)
    assert torch.equal(k_only.cpu(), v)


@pytest.mark.parametrize("bits,zp", [(8, False), (4, True)])
def test_cache_write_with_norm_and_rotation(ia, bits, zp):
    """Codes of the normed and turned rows: each within half a step (and the
    fp32 error of 16 units, see _close, plus 2 for the reciprocal and product) of the
    float64 value; V untouched by the norm."""
    import torch
    B, H, Hkv, L, Lmax, d = 3, 8, 2, 29, 64, 128
    rng = np.random.default_rng(bits)
    (q, k, v), (q32, k32, v32) = _packed(rng, B, L, (H, Hkv, Hkv), d, torch.bfloat16)
    w = [rng.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2)]
    table = ia.rope_table(500, d)
    pos = rng.integers(0, 500, (B, L)).astype(np.int32)
    top = 2.0 ** (bits - 1) - 1
    s_q, s_k, s_v = (np.full(n, 3.0 / t, np.float32) for n, t in ((H, 127), (Hkv, top), (Hkv, top)))
    z = np.array([2 ** (bits - 1) + 1, 2 ** (bits - 1) - 2], np.int32) if zp else None
    sc = ia.Scales(s_q, s_k, s_v, 1.0, per_head=True, z_k=z, z_v=z)
    cache = [torch.zeros((B, Hkv, Lmax, d * bits // 8), dtype=torch.uint8 if zp or bits == 4 else torch.int8,
                         device="cuda") for _ in range(2)]
    start = np.array([0, 20, 35], np.int32)
    rn = ia.RopeNorm(table, torch.from_numpy(pos).cuda(), *(torch.from_numpy(x).cuda() for x in w))
    q_out = ia.cache_write(k, v, sc, *cache, torch.from_numpy(start).cuda(), bits=bits, q=q, norm=rn)
    assert ia.device_error() == ia.OK
    got = [orow.unpack(c.cpu().numpy(), bits, zp) for c in cache]
    rows = lambda c: np.stack([c[b, :, start[b]:start[b] + L] for b in range(B)])
    assert np.array_equal(rows(got[1]), orow.codes(v32, s_v, z, bits))
    tn = table.cpu().numpy()
    for codes, x, wx, s, zz, bb in ((q_out.cpu().numpy(), q32, w[0], s_q, None, 8), (rows(got[0]), k32, w[1], s_k, z, bits)):
        y, mag = orow.norm_rope(x, wx, 1e-6, tn, pos)
        sv = s.astype(np.float64)[None, :, None, None]
        zv = 0 if zz is None else zz[None, :, None, None]
        lo, hi = (-(2 ** (bb - 1) - 1), 2 ** (bb - 1) - 1) if zz is None else (0, 2 ** bb - 1)
        u = np.clip(y / sv + zv, lo, hi)
        slack = 0.5 + 18 * 2.0 ** -24 * mag / sv
        assert (np.abs(codes - u) <= slack).all()
        assert (np.abs(codes - zv) > 1).any()


def test_cache_write_special_values(ia):
    import torch
    x = torch.zeros((1, 1, 1, 64), dtype=torch.float16)
    x[0, 0, 0, :8] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.25, 0.75, -0.25, 6e4, -6e4])
    x = x.cuda()
    for bits, z, want in ((8, None, [0, 127, -127, 0, 2, 0, 127, -127]), (8, 9, [9, 255, 0, 9, 11, 9, 255, 0]),
                          (4, None, [0, 7, -7, 0, 2, 0, 7, -7]), (4, 3, [3, 15, 0, 3, 5, 3, 15, 0])):
        c = [torch.zeros((1, 1, 2, 64 * bits // 8), device="cuda",
                         dtype=torch.int8 if bits == 8 and z is None else torch.uint8) for _ in range(2)]
        ia.cache_write(x, x, ia.Scales(1, 0.5, 0.5, 1, z_k=z, z_v=z), *c, torch.tensor([1], dtype=torch.int32, device="cuda"),
                       bits=bits)
        for t in c:
            assert orow.unpack(t.cpu().numpy(), bits, z is not None)[0, 0, 1, :8].tolist() == want
            assert not t[0, 0, 0].any()


def test_cache_rows_out_of_range(ia):
    """Rows that would land outside the cache are left out, the others are
    written, and the error word says so."""
    import torch
    sc = ia.Scales(1, 0.5, 0.5, 1)
    x = torch.ones((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    c = [torch.zeros((2, 1, 6, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
    for start in ([4, -2], [2 ** 31 - 1, -2 ** 31]):
        st = torch.tensor(start, dtype=torch.int32, device="cuda")
        for t in c:
            t.zero_()
        ia.cache_write(x, x, sc, *c, st)
        assert ia.device_error() == ia.ERR_PARAM_RANGE
        for t in c:
            rows = t[:, 0, :, 0].cpu().tolist()
            assert rows == ([[0, 0, 0, 0, 2, 2], [2, 2, 0, 0, 0, 0]] if start[0] == 4 else [[0] * 6] * 2)
        out = torch.full((2, 1, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        ia.cache_read(c[0], None, sc, st, 4, k_out=out)
        assert ia.device_error() == ia.ERR_PARAM_RANGE
        got = out[:, 0, :, 0].cpu().tolist()
        assert got == ([[1, 1, 5, 5], [5, 5, 1, 1]] if start[0] == 4 else [[5] * 4] * 2)
    assert ia.device_error() == ia.OK


def test_cache_offsets_past_32_bits(ia):
    """Rows near the end of a cache of more than 2^31 elements."""
    import torch
    B, H, Lmax, d = 2, 128, 70000, 128
    sc = ia.Scales(1, 0.5, 0.5, 1)
    caches = [torch.zeros((B, H, Lmax, d), dtype=torch.int8, device="cuda") for _ in range(2)]
    assert caches[0].numel() > 2 ** 31
    x = torch.randn((B, H, 2, d), device="cuda").to(torch.bfloat16)
    st = torch.tensor([Lmax - 2, Lmax - 3], dtype=torch.int32, device="cuda")
    ia.cache_write(x, -x, sc, *caches, st)
    k, v = ia.cache_read(*caches, sc, st, 2)
    assert ia.device_error() == ia.OK
    want = torch.from_numpy(orow.codes(x.float().cpu().numpy(), [0.5]) * 0.5).to(torch.bfloat16)
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), -want)
    assert int((caches[0][1, H - 1, :Lmax - 3] != 0).sum()) == 0


def test_rows_on_another_stream_and_in_a_graph(ia):
    """A side stream, and a captured step replayed on new inputs."""
    import torch
    rng = np.random.default_rng(9)
    (q, k, v), _ = _packed(rng, 2, 3, (4, 2, 2), 64, torch.bfloat16)
    sc = ia.Scales(0.05, 0.05, 0.05, 1)
    rn = ia.RopeNorm(ia.rope_table(64, 64), torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3),
                     torch.ones(64, device="cuda"), torch.ones(64, device="cuda"))
    st = torch.tensor([1, 4], dtype=torch.int32, device="cuda")
    mk = lambda: [torch.zeros((2, 2, 9, 64), dtype=torch.int8, device="cuda") for _ in range(2)]

    def step(caches, stream=None):
        qo = ia.cache_write(k, v, sc, *caches, st, q=q, norm=rn, stream=stream)
        return [qo, *ia.cache_read(*caches, sc, st, 3, stream=stream), *ia.qk_norm_rope(q, k, rn, stream=stream)]

    want = step(mk())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        caches = mk()
        torch.cuda.synchronize()
        got = step(caches, stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    caches = mk()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(caches)
    k.copy_(k * 2)
    st.copy_(torch.tensor([0, 6], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    want = step(mk())
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and ia.device_error() == ia.OK


def test_python_refusals(ia):
    import torch
    sc = ia.Scales(1, 0.5, 0.5, 1)
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    c = torch.zeros((1, 2, 8, 64), dtype=torch.int8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ok = lambda **kw: ia.cache_write(**{**dict(k=x, v=x, scales=sc, k_cache=c, v_cache=c.clone(), start=st), **kw})
    ok()
    for err, kw in [(TypeError, dict(k=x.float())), (TypeError, dict(v=x.cpu())), (ValueError, dict(v=x[:, :1])),
                    (ValueError, dict(v=x.half())), (TypeError, dict(k_cache=c.to(torch.uint8))),
                    (ValueError, dict(v_cache=c[:, :, :7])), (TypeError, dict(start=st.long())),
                    (ValueError, dict(start=st.repeat(2))), (TypeError, dict(start=st.cpu())), (ValueError, dict(bits=3)),
                    (TypeError, dict(bits=4)), (ValueError, dict(q_out=c)), (ValueError, dict(k=x.transpose(2, 3))),
                    (ValueError, dict(scales=ia.Scales(1, [0.5], [0.5], 1, per_head=True))),
                    (ValueError, dict(norm=ia.RopeNorm(ia.rope_table(4, 64), st.view(1, 1)))),
                    (ValueError, dict(norm=ia.RopeNorm(w_k=torch.ones(128, device="cuda")))),
                    (TypeError, dict(norm=ia.RopeNorm(w_k=torch.ones(64))))]:
        with pytest.raises(err):
            ok(**kw)
    odd = torch.zeros((1, 2, 3, 65), dtype=torch.bfloat16, device="cuda")[..., :64]
    with pytest.raises(ia.IntAttnError):
        ok(v=odd)
    with pytest.raises(ia.IntAttnError):
        ia.qk_norm_rope(x, None, ia.RopeNorm(), q_out=torch.zeros(64, dtype=torch.bfloat16, device="cuda").expand(1, 2, 3, 64))
    with pytest.raises(TypeError):
        ia.cache_read(c, None, sc, st, 3, dtype=torch.float32)
    with pytest.raises(ValueError):
        ia.cache_read(c, None, sc, st, 3, v_out=x)
    assert ia.device_error() == ia.OK


def test_more_python_refusals(ia):
    """Tables and positions that would rotate nothing, and a stream of another device."""
    import torch
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((1, 3), dtype=torch.int32, device="cuda")

    class Elsewhere:
        cuda_stream, device = 0, torch.device("cuda", torch.cuda.current_device() + 1)

    table = ia.rope_table(4, 64)
    for rn in (ia.RopeNorm(None, pos), ia.RopeNorm(table[:0], pos), ia.RopeNorm(table[:, :0].contiguous(), pos)):
        with pytest.raises(ValueError):
            ia.qk_norm_rope(x, None, rn)
    with pytest.raises(ValueError):
        ia.qk_norm_rope(x, x, ia.RopeNorm(table, pos), k_out=x[:, :1])
    with pytest.raises(ValueError):
        ia.qk_norm_rope(x, None, ia.RopeNorm(table, pos), stream=Elsewhere())
    assert ia.device_error() == ia.OK


def test_scales_from_read_only_arrays(ia):
    """Scale arrays that cannot be written give the codes of those that can."""
    import torch
    rng = np.random.default_rng(31)
    k = torch.from_numpy(rng.standard_normal((1, 4, 5, 64)).astype(np.float32)).cuda().bfloat16()
    s = np.array([0.02, 0.03, 0.01, 0.05], np.float32)
    frozen = s.copy()
    frozen.flags.writeable = False
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = []
    for x in (s, frozen, s.tolist()):
        kc, vc = (torch.zeros((1, 4, 8, 64), dtype=torch.int8, device="cuda") for _ in range(2))
        ia.cache_write(k, k, ia.Scales(1, x, x, 1, per_head=True), kc, vc, st)
        out.append(torch.cat([kc, vc]))
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2]) and bool(out[0].any())
