"""GPU parity of the shared-prefix decode where a CTA has more than two
segments and loads its queries again in every phase, and where four key tiles fold
into the smallest ring.  The shapes, and what each is for, stand with the barrier
model, which runs them on the CPU."""
import numpy as np
import pytest

from test_gpu_shared import Case, _equal, _run
from test_shared_segments_protocol import SHAPES, name

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


@pytest.mark.parametrize("zp", [(False, False), (True, True)], ids=["i8", "zkzv"])
@pytest.mark.parametrize("shape", SHAPES, ids=name)
def test_parity(ia, oracle_mod, shape, zp):
    """Twelve sequences spread over the batch (every row tile among them), all
    heads of each; and the same bytes for the whole batch five times over."""
    import torch
    B, Hkv, G, Lp, Lmax, d = shape
    assert torch.cuda.get_device_properties(0).multi_processor_count == 148  # what the shapes are made for
    c = Case(B, Hkv * G, Hkv, Lp, Lmax, d, seed=sum(shape) + zp[0], zk=zp[0], zv=zp[1], per_head=False)
    got = _run(ia, c)
    rows = sorted({int(b) for b in np.linspace(0, B - 1, 12)})
    _equal(got[rows], c.want(oracle_mod, rows)[rows])
    for _ in range(4):
        assert torch.equal(_run(ia, c), got)
