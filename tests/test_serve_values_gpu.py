"""Decode over an E4M3 cache with block factors far apart and zero rows. Bounds: those of
test_serve_gpu.py, with no term for factors that a row gives no weight to."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_36_b200 import binding as fb
from tests import serve_ref as ref
from tests.gpu_util import f64
from tests.test_serve_gpu import DT, Cache, check_decode, decode, dev, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    fb.lib()
    yield
    assert fb.fa_get_last_device_error(None) == fb.FA_OK


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("Hq,Nq,d,dtype", [(8, 1, 128, "bf16"), (80, 1, 128, "bf16"), (40, 2, 64, "fp16"), (8, 2, 64, "bf16")])
def test_zero_queries_over_zero_keys(Hq, Nq, d, dtype, page, causal):
    """An all-zero step as a program's first one: zero queries, and keys whose append gave the blocks the
    smallest factor. Every key has the same weight."""
    Hkv, cap, lens = 2, 300, [100, 300, 1, 129]
    B = len(lens)
    cache = Cache(B, cap, Hkv, d, page, lens, seed=61)
    zero = ref.e4m3_encode(np.zeros(1))[0]
    for b, n in enumerate(lens):
        for pos in range(n):
            cache.k[(b, pos) if not page else (cache.table[b, pos // page], pos % page)] = zero
    cache.kf[:] = 2.0 ** -100
    q = torch.zeros(B, Nq, Hq, d, dtype=DT[dtype], device="cuda")
    q[1, :, 1] = 1.0  # one head of one sequence has queries
    o, lse = decode(cache, q, d ** -0.5, causal)
    check_decode(o, lse, cache.reference(q, d ** -0.5, causal), q.dtype)
