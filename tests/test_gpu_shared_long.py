"""GPU parity of the shared-prefix decode over long own caches: thousands of own
keys per sequence, up to the largest count, behind a short prefix or none."""
import numpy as np
import pytest

from test_gpu_shared import Case, _equal, _run

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


LONG = [  # B, H, Hkv, Lp, Lmax, d, lengths
    (1, 8, 1, 0, 10007, 128, [10007]), (3, 16, 2, 130, 12001, 64, [12001, 1, 7777]),
    (2, 40, 5, 500, 30011, 64, [29999, 30011]), (5, 6, 6, 1, 20000, 128, [0, 20000, 33, 19999, 16384]),
    (70, 4, 4, 300, 4099, 128, None), (1, 9, 1, 0, 65535, 128, [65535]), (2, 3, 3, 35, 65500, 64, [65500, 40001]),
    (2, 64, 4, 2000, 8200, 64, [8200, 5000]),
]


@pytest.mark.parametrize("zp", [(False, False), (True, True)], ids=["i8", "zkzv"])
@pytest.mark.parametrize("case", LONG, ids=lambda c: "B{}H{}k{}p{}m{}d{}".format(*c[:6]))
def test_parity(ia, oracle_mod, case, zp):
    import torch
    c = Case(*case[:6], seed=sum(case[:6]) + zp[0], zk=zp[0], zv=zp[1], per_head=case[0] % 2 == 1, lengths=case[6])
    got = _run(ia, c)
    rows = range(c.B) if c.B < 20 else range(0, c.B, 9)
    _equal(got[list(rows)], c.want(oracle_mod, rows)[list(rows)])
    assert torch.equal(_run(ia, c), got)


def test_equal_keys(ia, oracle_mod):
    """65535 own keys with one score: the largest row sum."""
    c = Case(2, 4, 2, 0, 65535, 64, 21, lengths=[65535, 65535])
    c.kc[:] = 3
    _equal(_run(ia, c), c.want(oracle_mod))


def test_equals_decode_over_long_caches(ia):
    """A batch of long caches, against intattn_decode on each sequence's rows."""
    import torch
    B, H, Lmax, d = 24, 16, 9000, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").mul_(28).round_().clamp_(-127, 127).to(torch.int8)
    q, kp, vp, kc, vc = mk(B, H, 1, d), mk(H, 200, d), mk(H, 200, d), mk(B, H, Lmax, d), mk(B, H, Lmax, d)
    s = 3 ** 0.5 / 28
    sc = ia.Scales(s, s, 1 / 28, 3 / 127)
    ln = torch.randint(0, Lmax + 1, (B,), device="cuda", dtype=torch.int32, generator=g)
    got = ia.decode_shared(q, kp, vp, kc, vc, ln, sc, 10.0)
    assert ia.device_error() == ia.OK
    for b in range(B):
        n = int(ln[b])
        join = lambda p, c: torch.cat([p, c[b, :, :n]], 1)[None].contiguous()
        assert torch.equal(got[b:b + 1], ia.decode(q[b:b + 1], join(kp, kc), join(vp, vc), sc, 200 + n, 10.0))
