"""The row operators and the shared-prefix decode at the ends of what they
take: the most sequences and heads, rows and values past 2^31 elements."""
import numpy as np
import pytest

from oracle import rows as orow
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


@pytest.mark.parametrize("shape", [(65535, 1, 1, 130, 3, 64), (255, 257, 257, 40, 2, 128), (1, 65535, 65535, 130, 3, 64),
                                   (1, 65408, 128, 300, 9, 64), (5, 13107, 13107, 1, 1, 128)],
                         ids=lambda s: "B{}H{}k{}p{}m{}d{}".format(*s))
def test_most_queries(ia, oracle_mod, shape):
    """65535 query rows or just below: all sequences, all heads, all of a group."""
    B, H = shape[:2]
    c = Case(*shape, seed=sum(shape), per_head=False, zv=True)
    got = _run(ia, c)
    rows = sorted({int(b) for b in np.linspace(0, B - 1, 300)})
    _equal(got[rows], c.want(oracle_mod, rows)[rows])


def test_more_queries_are_refused(ia):
    c = Case(2, 32768, 32768, 1, 1, 64, seed=1, per_head=False)
    with pytest.raises(ia.IntAttnError):
        _run(ia, c)


def test_many_heads_of_one_token(ia):
    import torch
    H = 65535
    x = torch.randn((1, H, 1, 64), device="cuda").to(torch.float16)
    rn = ia.RopeNorm(ia.rope_table(4, 64), torch.tensor([[3]], dtype=torch.int32, device="cuda"),
                     torch.ones(64, device="cuda"), torch.ones(64, device="cuda"))
    y, z = ia.qk_norm_rope(x, x[:, :H - 4], rn)
    part, _ = ia.qk_norm_rope(x[:, H - 5:], None, rn)
    assert torch.equal(y[:, H - 5:], part) and torch.equal(y[:, :H - 4], z)
    caches = [torch.zeros((1, H, 2, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
    ia.cache_write(x, -x, ia.Scales(1, 0.03, 0.03, 1), *caches, torch.tensor([1], dtype=torch.int32, device="cuda"))
    want = orow.codes(x.float().cpu().numpy(), [0.03])
    assert np.array_equal(caches[0][:, :, 1:].cpu().numpy(), want) and np.array_equal(caches[1][:, :, 1:].cpu().numpy(), -want)
    assert not caches[0][:, :, 0].any() and ia.device_error() == ia.OK


def test_rows_past_32_bits(ia):
    """Norm and rotation of more than 2^31 elements, in place: the last rows are
    those of a call of their own."""
    import torch
    H, L, d = 32, 530000, 128
    x = torch.zeros((1, L, H, d), dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    x[:, -3:].normal_()
    x[:, :2].normal_()
    q = x.transpose(1, 2)
    table = ia.rope_table(64, d)
    pos = (torch.arange(L, device="cuda") % 64).to(torch.int32).view(1, L)
    w = torch.rand(d, device="cuda") + 0.5
    ends = [q[:, :, s].clone() for s in (slice(0, 2), slice(L - 3, L))]
    want = [ia.qk_norm_rope(e, None, ia.RopeNorm(table, pos[:, s].contiguous(), w))[0]
            for e, s in zip(ends, (slice(0, 2), slice(L - 3, L)))]
    ia.qk_norm_rope(q, None, ia.RopeNorm(table, pos, w), q_out=q)
    assert torch.equal(q[:, :, :2], want[0]) and torch.equal(q[:, :, L - 3:], want[1])
    assert int(torch.count_nonzero(x[:, 2:-3])) == 0  # as values: 0 c - 0 s is -0 where the cosine is negative
    assert ia.device_error() == ia.OK


def test_values_past_32_bits(ia):
    """More than 2^31 values read back, rows past the lengths cleared."""
    import torch
    B, H, L, d = 2, 128, 70000, 128
    cache = torch.zeros((B, H, L, d), dtype=torch.int8, device="cuda")
    cache[:, :, -5:] = torch.randint(-127, 128, (B, H, 5, d), device="cuda").to(torch.int8)
    st, ln = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, 0], [L, L - 2]))
    k, _ = ia.cache_read(cache, None, ia.Scales(1, 0.5, 1, 1), st, L, lengths=ln)
    assert k.numel() > 2 ** 31 and ia.device_error() == ia.OK
    want = (cache[:, :, -5:].float() * 0.5).to(torch.bfloat16)
    want[1, :, -2:] = 0
    assert torch.equal(k[:, :, -5:], want) and int(torch.count_nonzero(k[:, :, :-5].view(torch.int16))) == 0
