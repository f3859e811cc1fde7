"""Norm and rotation on the way into the caches, at every geometry: both head
sizes, partial rotation, both pairings, every kind of code, ragged lengths,
padded positions and positions out of range."""
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


def _check(codes, y, mag, scale, zero, bits, live):
    """Codes of live rows within half a step of the float64 value y / s + z, and
    the fp32 part: 16 units of 2^-24 of the magnitudes added for norm and
    rotation (the sum of up to 128 squares 12, halved by the root: 6; mean and eps 2,
    halved: 1; reciprocal root 4; two products 2; rotation 3), 2 for the
    reciprocal of the scale and its product."""
    s = scale.astype(np.float64)[None, :, None, None]
    z = 0 if zero is None else zero[None, :, None, None]
    lo, hi = (-(2 ** (bits - 1) - 1), 2 ** (bits - 1) - 1) if zero is None else (0, 2 ** bits - 1)
    off = np.abs(codes - np.clip(y / s + z, lo, hi)) - (0.5 + 18 * 2.0 ** -24 * mag / s)
    assert (np.where(live, off, 0) <= 0).all()
    assert not live.any() or (np.abs(codes - z) * live > 1).any()


@pytest.mark.parametrize("bits,zp", [(8, False), (8, True), (4, False), (4, True)], ids=["i8", "u8", "i4", "u4"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["split", "pairs"])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 32), (64, 64), (128, 16), (128, 64), (128, 112), (128, 128), (64, 0)])
@pytest.mark.parametrize("name", ["float16", "bfloat16"])
def test_codes(ia, name, d, rot, interleaved, bits, zp):
    import torch
    B, H, Hkv, L, Lmax = 4, 9, 3, 13, 40
    rng = np.random.default_rng(d + rot + bits + 2 * zp + interleaved)
    norm_q, norm_k = bool(rng.integers(2)), bool(rng.integers(2))
    x = rng.standard_normal((B, L, H + 2 * Hkv, d)).astype(np.float32)
    x = torch.from_numpy(x).to(getattr(torch, name)).cuda()
    q, k, v = (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))
    q32, k32, v32 = (t.float().cpu().numpy() for t in (q, k, v))
    w = [rng.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2)]
    n_pos = 300
    pos = rng.integers(0, n_pos, (B, L)).astype(np.int32)
    lengths = np.array([13, 7, 0, 12], np.int32)
    if rot:
        pos[0, 3], pos[0, 12], pos[3, :5] = -1, -2 ** 31, -7  # padding
        pos[1, 2], pos[3, 6] = n_pos, 2 ** 31 - 1              # out of range: reported
        pos[1, 9] = n_pos + 5                                  # and not where the length ends before it
    live = (np.arange(L) < lengths[:, None]) & ((pos >= 0) & (pos < n_pos) if rot else True)
    top = 2.0 ** (bits - 1) - 1
    s_q = rng.uniform(0.9, 1.1, H).astype(np.float32) * np.float32(3 / 127)
    s_k, s_v = (rng.uniform(0.9, 1.1, Hkv).astype(np.float32) * np.float32(3 / top) for _ in range(2))
    z = rng.integers(2 ** (bits - 1) - 3, 2 ** (bits - 1) + 3, (2, Hkv)).astype(np.int32) if zp else (None, None)
    sc = ia.Scales(s_q, s_k, s_v, 1.0, per_head=True, z_k=z[0], z_v=z[1])
    u8 = zp or bits == 4
    before = [rng.integers(0, 250, (B, Hkv, Lmax, d * bits // 8)).astype(np.uint8) for _ in range(2)]
    before = before if u8 else [c.view(np.int8) for c in before]
    cache = [torch.from_numpy(c.copy()).cuda() for c in before]
    start = np.array([0, 27, 5, 20], np.int32)
    dev = lambda a: torch.from_numpy(a).cuda()
    table = ia.rope_table(n_pos, rot) if rot else None
    rn = ia.RopeNorm(table, dev(pos) if rot else None, dev(w[0]) if norm_q else None, dev(w[1]) if norm_k else None, 1e-6,
                     interleaved)
    q_out = torch.full((B, H, L, d), 99, dtype=torch.int8, device="cuda")
    ia.cache_write(k, v, sc, *cache, dev(start), lengths=dev(lengths), bits=bits, q=q, q_out=q_out, norm=rn)
    assert ia.device_error() == (ia.ERR_PARAM_RANGE if rot else ia.OK)

    # every byte that belongs to no live row is as it was: K, V and q_out alike
    written = np.zeros((B, Lmax), bool)
    for b in range(B):
        written[b, start[b]:start[b] + L] = live[b]
    for c, old in zip(cache, before):
        assert np.array_equal(np.where(written[:, None, :, None], 0, c.cpu().numpy()),
                              np.where(written[:, None, :, None], 0, old))
    rows_live = live[:, None, :, None]
    got_q = q_out.cpu().numpy().astype(np.int64)
    assert (np.where(rows_live, 99, got_q) == 99).all()

    got = [orow.unpack(c.cpu().numpy(), bits, zp) for c in cache]
    got = [np.stack([c[b, :, start[b]:start[b] + L] for b in range(B)]) for c in got]
    assert (np.where(rows_live, got[1] - orow.codes(v32, s_v, z[1], bits), 0) == 0).all()  # V: neither normed nor turned
    tn = None if table is None else table.cpu().numpy()
    inside = np.where((pos >= 0) & (pos < n_pos), pos, 0)
    for codes, x32, wx, s, zz, bb in ((got_q, q32, w[0] if norm_q else None, s_q, None, 8),
                                      (got[0], k32, w[1] if norm_k else None, s_k, z[0], bits)):
        y, mag = orow.norm_rope(x32, wx, 1e-6, tn, inside, interleaved)
        _check(codes, y, mag, s, zz, bb, rows_live)
