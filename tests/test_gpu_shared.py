"""GPU parity of the shared-prefix decode: byte-equal to the CPU oracle's
decode of each sequence over its joined keys."""
import numpy as np
import pytest

from integer_only_quantized_b200 import workloads as wl
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


class Case:
    """Inputs of one call, on the host.  spread: the logits' standard
    deviation (peaked rows keep weight on few keys)."""

    def __init__(self, B, H, Hkv, Lp, Lmax, d, seed, zk=False, zv=False, per_head=True, spread=3.0, lengths=None, clip=10.0,
                 Lp_max=None):
        rng = np.random.default_rng(seed)
        self.B, self.H, self.Hkv, self.Lp, self.Lmax, self.d, self.clip = B, H, Hkv, Lp, Lmax, d, clip
        n, nk = (H, Hkv) if per_head else (1, 1)
        self.per_head = per_head
        wob = lambda m: rng.uniform(0.9, 1.1, m).astype(np.float32)
        self.s_q, self.s_k = wob(n) * np.float32(spread ** 0.5 / 28), wob(nk) * np.float32(spread ** 0.5 / 28)
        self.s_v, self.s_o = wob(nk) / np.float32(28), wob(n) * np.float32(3 / 127)
        self.z_k = rng.integers(100, 156, nk).astype(np.int32) if zk else None
        self.z_v = rng.integers(0, 256, nk).astype(np.int32) if zv else None

        def codes(shape, z):
            x = np.rint(28 * rng.standard_normal(shape))
            if z is None:
                return np.clip(x, -127, 127).astype(np.int8)
            return np.clip(x + np.broadcast_to(z, (Hkv,))[:, None, None], 0, 255).astype(np.uint8)

        self.Lp_max = Lp if Lp_max is None else Lp_max
        self.q = codes((B, H, 1, d), None)
        self.kp, self.vp = codes((Hkv, self.Lp_max, d), self.z_k), codes((Hkv, self.Lp_max, d), self.z_v)
        self.kc, self.vc = codes((B, Hkv, Lmax, d), self.z_k), codes((B, Hkv, Lmax, d), self.z_v)
        if lengths is None:
            lengths = rng.integers(0, Lmax + 1, B)
            lengths[-1] = Lmax
        self.lengths = np.asarray(lengths, np.int32)

    def scales(self, ia):
        return ia.Scales(self.s_q, self.s_k, self.s_v, self.s_o, per_head=self.per_head, z_k=self.z_k, z_v=self.z_v)

    def dev(self):
        import torch
        return [torch.from_numpy(x).cuda() for x in (self.q, self.kp, self.vp, self.kc, self.vc, self.lengths)]

    def want(self, oracle_mod, rows=None):
        """int8 codes [B, H, 1, d] by the oracle (rows: only these sequences)."""
        G = self.H // self.Hkv
        rep = lambda x: x if x is None or not self.per_head else np.repeat(x, G)
        out = np.zeros(self.q.shape, np.int8)
        for b in range(self.B) if rows is None else rows:
            n = self.Lp + int(self.lengths[b])
            if n == 0:
                continue
            join = lambda p, c: np.repeat(np.concatenate([p[:, :self.Lp], c[b, :, :self.lengths[b]]], 1), G, 0)[None]
            out[b] = oracle_mod.decode(self.q[b:b + 1], join(self.kp, self.kc), join(self.vp, self.vc), self.per_head,
                                       self.s_q, rep(self.s_k), rep(self.s_v), self.s_o, n, self.clip,
                                       z_k=rep(self.z_k), z_v=rep(self.z_v))[0]
        return out


def _run(ia, c, **kw):
    q, kp, vp, kc, vc, ln = c.dev()
    out = ia.decode_shared(q, kp, vp, kc, vc, ln, c.scales(ia), c.clip, prefix_len=c.Lp, **kw)
    assert ia.device_error() == ia.OK
    return out


def _equal(got, want):
    got = got.cpu().numpy()
    if not np.array_equal(got, want):
        bad = np.argwhere(got != want)
        raise AssertionError(f"{len(bad)} of {want.size} codes differ; first {bad[:4].tolist()} got "
                             f"{got[tuple(bad[0])]} want {want[tuple(bad[0])]}")


SWEEP = [  # B, H, Hkv, Lp, Lmax, d
    (1, 1, 1, 1, 0, 64), (1, 1, 1, 0, 1, 64), (1, 2, 1, 1, 1, 128), (2, 2, 2, 127, 3, 64), (3, 4, 2, 128, 17, 128),
    (2, 8, 1, 129, 31, 64), (5, 3, 3, 300, 64, 128), (4, 12, 4, 1000, 33, 64), (33, 4, 4, 257, 100, 64),
    (40, 8, 2, 640, 130, 128), (64, 2, 2, 511, 5, 128), (65, 2, 1, 200, 9, 64), (70, 6, 2, 385, 40, 128),
    (1, 40, 1, 1500, 700, 128), (2, 9, 3, 0, 1030, 64), (130, 3, 3, 0, 65, 128), (3, 5, 5, 4100, 0, 64),
    (2, 4, 4, 5000, 1100, 128), (9, 32, 2, 130, 20, 64),
    # few queries over many tiles: four, then two key tiles side by side, the last group partly empty
    (2, 16, 16, 4900, 30, 64), (3, 32, 32, 2450, 20, 128), (1, 40, 10, 8200, 100, 128),
    (40, 20, 20, 2100, 17, 64), (7, 64, 8, 5050, 9, 128),
    # many short tiles: more than two (head, row tile) pairs per CTA
    (400, 100, 100, 100, 3, 64), (129, 32, 8, 250, 5, 128), (3, 128, 128, 600, 40, 64),
]


@pytest.mark.parametrize("zp", [(False, False), (True, True), (True, False), (False, True)],
                         ids=["i8", "zkzv", "zk", "zv"])
@pytest.mark.parametrize("shape", SWEEP, ids=lambda s: "B{}H{}k{}p{}m{}d{}".format(*s))
def test_parity(ia, oracle_mod, shape, zp):
    c = Case(*shape, seed=sum(shape) + 2 * zp[0] + zp[1], zk=zp[0], zv=zp[1], per_head=shape[0] % 2 == 1)
    _equal(_run(ia, c), c.want(oracle_mod))


@pytest.mark.parametrize("spread,clip", [(0.05, 8.0), (1.0, 2.0), (30.0, 14.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_flat_and_peaked_rows(ia, oracle_mod, d, spread, clip):
    c = Case(6, 8, 4, 700, 90, d, 3, spread=spread, clip=clip, zk=True, zv=True)
    _equal(_run(ia, c), c.want(oracle_mod))


def test_max_in_prefix_or_in_own_rows(ia, oracle_mod):
    """The row max (and all the weight) on one key, at every tile edge of the
    prefix and in the sequence's own rows."""
    c = Case(8, 2, 2, 400, 70, 128, 4, spread=0.01, lengths=[70] * 8)
    for b, j in enumerate([0, 127, 128, 255, 399, 400, 431, 469]):
        for h in range(2):
            k = np.sign(c.q[b, h, 0].astype(np.int32)) * 127
            if j < 400:
                c.kp[h, j] = k
            else:
                c.kc[b, h, j - 400] = k
    _equal(_run(ia, c), c.want(oracle_mod))


def test_extreme_codes(ia, oracle_mod):
    """The largest scores and sums the codes allow."""
    c = Case(3, 4, 2, 260, 40, 128, 6, zk=True, zv=True, lengths=[40, 0, 17])
    c.q[:] = np.where(c.q > 0, 127, -128)
    c.kp[:, ::2], c.kc[:, :, ::2] = 255, 0
    c.vp[:], c.vc[:] = 255, 255
    c.z_v[:] = 0
    _equal(_run(ia, c), c.want(oracle_mod))


def test_rows_without_keys(ia, oracle_mod):
    c = Case(4, 2, 1, 0, 50, 64, 7, zv=True, lengths=[0, 50, 0, 1])
    got = _run(ia, c)
    _equal(got, c.want(oracle_mod))
    assert not got[0].any() and not got[2].any()
    c = Case(2, 2, 2, 0, 33, 128, 8, lengths=[0, 0])
    assert not _run(ia, c).any()


def test_prefix_capacity_and_null_lengths(ia, oracle_mod):
    """Rows of the prefix past prefix_len are not read; lengths None: all rows."""
    import torch
    c = Case(3, 4, 2, 150, 20, 64, 9, Lp_max=310, lengths=[20] * 3)
    _equal(_run(ia, c), c.want(oracle_mod))
    q, kp, vp, kc, vc, _ = c.dev()
    got = ia.decode_shared(q, kp, vp, kc, vc, None, c.scales(ia), c.clip, prefix_len=150)
    _equal(got, c.want(oracle_mod))
    kp[:, 150:], vp[:, 150:] = 127, 127
    _equal(ia.decode_shared(q, kp, vp, kc, vc, None, c.scales(ia), c.clip, prefix_len=150), c.want(oracle_mod))


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
def test_value_outputs(ia, oracle_mod, name):
    import torch
    dt = getattr(torch, name)
    c = Case(5, 6, 3, 333, 50, 128, 10)
    got = _run(ia, c, dtype=dt)
    want = torch.from_numpy(c.want(oracle_mod).astype(np.float32) * c.s_o[None, :, None, None]).to(dt)
    assert torch.equal(got.cpu(), want)


def test_clip_per_head(ia, oracle_mod):
    import torch
    c = Case(3, 4, 2, 300, 40, 64, 11)
    clips = np.array([4.0, 8.0, 10.0, 6.5], np.float32)
    sc = c.scales(ia)
    sc.clip = clips
    q, kp, vp, kc, vc, ln = c.dev()
    got = ia.decode_shared(q, kp, vp, kc, vc, ln, sc, 1.0).cpu().numpy()
    for h in range(4):
        c.clip = float(clips[h])
        assert np.array_equal(got[:, h], c.want(oracle_mod)[:, h])


def test_lengths_out_of_range(ia, oracle_mod):
    """A bad length leaves that sequence's output alone; the others are right."""
    import torch
    c = Case(5, 2, 2, 140, 30, 64, 12, lengths=[30, 4, 0, 9, 30])
    want = c.want(oracle_mod)
    q, kp, vp, kc, vc, ln = c.dev()
    ln[1], ln[3] = -1, 31
    out = torch.full(c.q.shape, 55, dtype=torch.int8, device="cuda")
    ia.decode_shared(q, kp, vp, kc, vc, ln, c.scales(ia), c.clip, out=out)
    assert ia.device_error() == ia.ERR_PARAM_RANGE and ia.device_error() == ia.OK
    want[[1, 3]] = 55
    _equal(out, want)


def test_nothing_written_around(ia, oracle_mod):
    """Guard bands around out and the workspace, and a workspace full of
    another call's leftovers."""
    import torch
    c = Case(7, 6, 2, 517, 61, 64, 13)
    n = ia.decode_shared_workspace_size(7, 6, 2, 61, 64)
    ws = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    buf = torch.full((c.q.size + 8192,), 0x5A, dtype=torch.int8, device="cuda")
    out = buf[4096:4096 + c.q.size].view(c.q.shape)
    for _ in range(2):
        _run(ia, c, out=out, workspace=ws[4096:4096 + n])
        _equal(out, c.want(oracle_mod))
    assert (buf[:4096] == 0x5A).all() and (buf[4096 + c.q.size:] == 0x5A).all()
    assert (ws[:4096] == 0xA5).all() and (ws[4096 + n:] == 0xA5).all()


def test_equals_decode_on_the_joined_cache(ia):
    """Larger than the oracle does quickly: against intattn_decode, which the
    oracle checks, on the joined cache."""
    import torch
    for d, H, B, Lp, Lmax in ((128, 32, 64, 4001, 777), (64, 12, 70, 9000, 300)):
        g = torch.Generator(device="cuda")
        g.manual_seed(d)
        mk = lambda *s: torch.randn(s, generator=g, device="cuda").mul_(28).round_().clamp_(-127, 127).to(torch.int8)
        q, kp, vp, kc, vc = mk(B, H, 1, d), mk(H, Lp, d), mk(H, Lp, d), mk(B, H, Lmax, d), mk(B, H, Lmax, d)
        s = 3 ** 0.5 / 28
        sc = ia.Scales(s, s, 1 / 28, 3 / 127)
        ln = torch.randint(0, Lmax + 1, (B,), device="cuda", dtype=torch.int32, generator=g)
        got = ia.decode_shared(q, kp, vp, kc, vc, ln, sc, 10.0)
        assert ia.device_error() == ia.OK
        for b in range(0, B, 9):
            n = int(ln[b])
            join = lambda p, c: torch.cat([p, c[b, :, :n]], 1)[None].contiguous()
            want = ia.decode(q[b:b + 1], join(kp, kc), join(vp, vc), sc, Lp + n, 10.0)
            assert torch.equal(got[b:b + 1], want)


def test_longest_rows(ia, oracle_mod):
    """65535 keys in all: every sum stays in 32 bits when all keys are equal."""
    c = Case(2, 2, 1, 65000, 535, 64, 14, lengths=[535, 100])
    c.kp[:], c.kc[:] = 3, 3
    _equal(_run(ia, c), c.want(oracle_mod))
    c = Case(2, 3, 1, 65000, 535, 128, 15, zv=True, spread=6.0)
    _equal(_run(ia, c), c.want(oracle_mod))


def test_streams_and_graph(ia):
    """A side stream, and a captured decode loop replayed with growing
    lengths: cache_write of a token's rows, then the decode over them."""
    import torch
    c = Case(6, 8, 2, 700, 40, 64, 16, lengths=[3, 0, 7, 11, 20, 5])
    q, kp, vp, kc, vc, ln = c.dev()
    sc = c.scales(ia)
    want = ia.decode_shared(q, kp, vp, kc, vc, ln, sc, c.clip)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):
        got = ia.decode_shared(q, kp, vp, kc, vc, ln, sc, c.clip, stream=st)
        side.synchronize()
        assert torch.equal(got, want)
    # two calls at once on two streams, each with its own workspace
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ra = [ia.decode_shared(q, kp, vp, kc, vc, ln, sc, c.clip, stream=s) for _ in range(5) for s in (a, b)]
    torch.cuda.synchronize()
    assert all(torch.equal(r, want) for r in ra)

    new = torch.randn((6, 1, 12, 64), device="cuda").to(torch.bfloat16)
    qn, kn, vn = (t.transpose(1, 2) for t in new.split([8, 2, 2], dim=2))
    rn = ia.RopeNorm(ia.rope_table(1000, 64), torch.zeros((6, 1), dtype=torch.int32, device="cuda"),
                     torch.ones(64, device="cuda"), torch.ones(64, device="cuda"))
    start = ln.clone()
    ws = torch.empty(ia.decode_shared_workspace_size(6, 8, 2, 40, 64), dtype=torch.uint8, device="cuda")

    def step(kc, vc, start):
        rn.positions.copy_((start + 700).view(6, 1))
        q8 = ia.cache_write(kn, vn, sc, kc, vc, start, q=qn, norm=rn)
        start += 1
        return ia.decode_shared(q8, kp, vp, kc, vc, start, sc, c.clip, dtype=torch.bfloat16, workspace=ws)

    k1, v1, k2, v2 = kc.clone(), vc.clone(), kc.clone(), vc.clone()
    s1, s2 = start.clone(), start.clone()
    inputs = [torch.randn_like(new) for _ in range(4)]
    want = []
    for x in inputs:
        new.copy_(x)
        want.append(step(k1, v1, s1).clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(k2, v2, s2)
    for x, w in zip(inputs, want):
        new.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert torch.equal(k1, k2) and torch.equal(v1, v2) and torch.equal(s1, s2)
    assert ia.device_error() == ia.OK


def test_serving_run_against_the_oracle(ia, oracle_mod):
    """A prefix and prompts written by cache_write, one step of norm, rotation
    and quantising, and the decode: the oracle's decode over the codes in the
    caches, whose values are near the normed and turned rows."""
    import torch
    rng = np.random.default_rng(17)
    B, H, Hkv, d, Lp, L, Lmax = 3, 4, 2, 128, 210, 37, 64
    table = ia.rope_table(400, d)
    w = torch.ones(d, device="cuda")
    s = np.full(H, 4 / 127, np.float32)
    sc = ia.Scales(s * 3, s[:Hkv], s[:Hkv], s, per_head=True)

    def project(b, n):
        x = torch.from_numpy(rng.standard_normal((b, n, H + 2 * Hkv, d)).astype(np.float32)).to(torch.bfloat16).cuda()
        return [t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2)]

    zero = lambda *sh: torch.zeros(sh, dtype=torch.int8, device="cuda")
    idx = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kp, vp, kc, vc = zero(1, Hkv, Lp, d), zero(1, Hkv, Lp, d), zero(B, Hkv, Lmax, d), zero(B, Hkv, Lmax, d)
    _, k0, v0 = project(1, Lp)
    ia.cache_write(k0, v0, sc, kp, vp, idx([0]), norm=ia.RopeNorm(table, torch.arange(Lp, dtype=torch.int32, device="cuda")[None], w_k=w))
    own = idx([0, 20, 36])  # prompt rows of each sequence, right-padded to L
    _, k1, v1 = project(B, L)
    pos = (Lp + torch.arange(L, device="cuda").expand(B, L)).to(torch.int32).contiguous()
    ia.cache_write(k1, v1, sc, kc, vc, idx([0] * B), lengths=own, norm=ia.RopeNorm(table, pos, w_k=w))
    q2, k2, v2 = project(B, 1)
    rn = ia.RopeNorm(table, (Lp + own).view(B, 1).contiguous(), w, w)
    q8 = ia.cache_write(k2, v2, sc, kc, vc, own, q=q2, norm=rn)
    out = ia.decode_shared(q8, kp[0], vp[0], kc, vc, own + 1, sc, 10.0)
    assert ia.device_error() == ia.OK
    assert not kc[0, :, 1:].any() and not kc[1, :, 21:].any()
    G = H // Hkv
    for b, n in enumerate((own + 1).tolist()):
        join = lambda p, c: np.repeat(np.concatenate([p[0].cpu().numpy(), c[b, :, :n].cpu().numpy()], 1), G, 0)[None]
        want = oracle_mod.decode(q8[b:b + 1].cpu().numpy(), join(kp, kc), join(vp, vc), True, s * 3, s, s, s, Lp + n, 10.0)
        assert np.array_equal(out[b:b + 1].cpu().numpy(), want)
    values, _ = ia.cache_read(kc, None, sc, own, 1, dtype=torch.float16)
    y, mag = orow.norm_rope(k2.float().cpu().numpy(), w.cpu().numpy(), 1e-6, table.cpu().numpy(),
                            (Lp + own).view(B, 1).cpu().numpy())
    y = np.clip(y, -4, 4)
    # half a code, and half a step of the fp16 that holds the value
    assert (np.abs(values.float().cpu().numpy() - y) <= 0.501 * 4 / 127 + 2.0 ** -11 * np.abs(y) + 18 * 2.0 ** -24 * mag).all()
    # the same keys and queries through the floating rows and the int8 step of the library
    qf, kf = ia.qk_norm_rope(q2, k2, rn)
    assert np.abs(qf.float().cpu().numpy() - orow.norm_rope(q2.float().cpu().numpy(), w.cpu().numpy(), 1e-6, table.cpu().numpy(),
                                                            (Lp + own).view(B, 1).cpu().numpy())[0]).max() < 8 * 2.0 ** -8


def test_python_refusals(ia):
    c = Case(2, 4, 2, 20, 9, 64, 18)
    q, kp, vp, kc, vc, ln = c.dev()
    f = dict(q=q, k_prefix=kp, v_prefix=vp, k_cache=kc, v_cache=vc, lengths=ln, scales=c.scales(ia), clip_c=8.0)
    import torch
    ia.decode_shared(**f)
    for err, kw in [(TypeError, dict(q=q.float())), (ValueError, dict(q=q.expand(2, 4, 3, 64).contiguous())),
                    (TypeError, dict(k_prefix=kp.to(torch.uint8))), (ValueError, dict(v_prefix=vp[:, :5].contiguous())),
                    (ValueError, dict(k_cache=kc[:1])), (ValueError, dict(v_cache=vc[:, :, ::2].contiguous())),
                    (ValueError, dict(q=q[:, :3].contiguous())), (TypeError, dict(lengths=ln.long())),
                    (ValueError, dict(lengths=ln[:1])), (TypeError, dict(dtype=torch.float32)),
                    (ValueError, dict(out=q[:1])), (TypeError, dict(out=q, dtype=torch.float16)),
                    (ia.IntAttnError, dict(prefix_len=21)), (ia.IntAttnError, dict(clip_c=-1.0)),
                    (ia.IntAttnError, dict(workspace=torch.empty(4, dtype=torch.uint8, device="cuda")))]:
        with pytest.raises(err):
            ia.decode_shared(**{**f, **kw})


def test_workspace_of_another_place(ia):
    """A workspace that is not a contiguous tensor of the call's device."""
    import torch
    c = Case(2, 4, 2, 70, 20, 64, 77)
    q, kp, vp, kc, vc, ln = c.dev()
    n = ia.decode_shared_workspace_size(2, 4, 2, 20, 64)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty((n, 2), dtype=torch.uint8, device="cuda")[:, 0], n):
        with pytest.raises(ValueError):
            ia.decode_shared(q, kp, vp, kc, vc, ln, c.scales(ia), c.clip, workspace=ws)


def test_output_over_the_queries(ia, oracle_mod):
    """out = q: the queries are read before any output is written, with many
    row tiles and segments too."""
    for shape in ((2, 4, 2, 700, 40, 64), (40, 16, 2, 1500, 30, 128)):
        c = Case(*shape, 78)
        q, kp, vp, kc, vc, ln = c.dev()
        ia.decode_shared(q, kp, vp, kc, vc, ln, c.scales(ia), c.clip, out=q)
        _equal(q, c.want(oracle_mod))


@pytest.mark.parametrize("shape", [(4, 20, 37277, 229, 64), (7, 29, 15104, 60, 128), (5, 18, 12841, 300, 128),
                                   (1, 26, 37329, 20, 64), (32, 19, 4000, 21, 64)],
                         ids=lambda s: "B{}H{}p{}m{}d{}".format(*s))
def test_many_tiles_of_few_queries(ia, shape):
    """Four key tiles side by side and many tiles per CTA, over and over (the
    softmax teams run ahead of each other in any order): the bytes of decode
    on the joined cache."""
    import torch
    B, H, Lp, Lmax, d = shape
    g = torch.Generator(device="cuda")
    g.manual_seed(Lp)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").mul_(28).round_().clamp_(-127, 127).to(torch.int8)
    q, kp, vp, kc, vc = mk(B, H, 1, d), mk(H, Lp, d), mk(H, Lp, d), mk(B, H, Lmax, d), mk(B, H, Lmax, d)
    s = 3 ** 0.5 / 28
    sc = ia.Scales(s, s, 1 / 28, 3 / 127)
    ln = torch.randint(0, Lmax + 1, (B,), device="cuda", dtype=torch.int32, generator=g)
    got = [ia.decode_shared(q, kp, vp, kc, vc, ln, sc, 10.0) for _ in range(20)]
    assert ia.device_error() == ia.OK
    assert all(torch.equal(x, got[0]) for x in got)
    for b in {0, B - 1}:
        n = int(ln[b])
        join = lambda p, c: torch.cat([p, c[b, :, :n]], 1)[None].contiguous()
        want = ia.decode(q[b:b + 1], join(kp, kc), join(vp, vc), sc, Lp + n, 10.0)
        assert torch.equal(got[0][b:b + 1], want)


@pytest.mark.parametrize("shape", [(45, 18, 95, 555, 64), (64, 32, 200, 777, 128), (60, 8, 1500, 1000, 64)],
                         ids=lambda s: "B{}H{}p{}m{}d{}".format(*s))
def test_own_blocks_are_not_replaced_while_read(ia, shape):
    """Own rows streaming beside a busy prefix, over and over: always the
    bytes of the first call, and of decode on the joined cache."""
    import torch
    B, H, Lp, Lmax, d = shape
    g = torch.Generator(device="cuda")
    g.manual_seed(Lmax)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").mul_(28).round_().clamp_(-127, 127).to(torch.int8)
    q, kp, vp, kc, vc = mk(B, H, 1, d), mk(H, Lp, d), mk(H, Lp, d), mk(B, H, Lmax, d), mk(B, H, Lmax, d)
    s = 3 ** 0.5 / 28
    sc = ia.Scales(s, s, 1 / 28, 3 / 127)
    ln = torch.randint(0, Lmax + 1, (B,), device="cuda", dtype=torch.int32, generator=g)
    first = ia.decode_shared(q, kp, vp, kc, vc, ln, sc, 10.0)
    for _ in range(200):
        assert torch.equal(ia.decode_shared(q, kp, vp, kc, vc, ln, sc, 10.0), first)
    assert ia.device_error() == ia.OK
    for b in range(0, B, 13):
        n = int(ln[b])
        join = lambda p, c: torch.cat([p, c[b, :, :n]], 1)[None].contiguous()
        want = ia.decode(q[b:b + 1], join(kp, kc), join(vp, vc), sc, Lp + n, 10.0)
        assert torch.equal(first[b:b + 1], want)
