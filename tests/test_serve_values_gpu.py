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


def put_page(cache, b, tokens, k=None, v=None, vf=None):
    """Keys, values (before their factors) and the V factor of the blocks of sequence b that hold `tokens`."""
    for pos in tokens:
        i = pos // cache.unit
        at = (b, pos) if not cache.page else (cache.table[b, i], pos % cache.unit)
        if k is not None:
            cache.k[at] = ref.e4m3_encode(k)
        if v is not None:
            cache.v[at] = ref.e4m3_encode(v)
        if vf is not None:
            if cache.page:
                cache.vf[cache.table[b, i]] = vf
            else:
                cache.vf[b, :, i] = vf


FORMS = [(8, 1, 128, "bf16"), (80, 1, 128, "bf16"), (8, 1, 64, "bf16"), (80, 1, 64, "bf16"), (8, 1, 128, "fp16"),
         (80, 1, 128, "fp16"), (4, 4, 64, "fp16")]  # Hq (two KV heads), Nq, d, type


@pytest.mark.parametrize("log2", [24, 40, 60])
@pytest.mark.parametrize("where", [16, 32, 416], ids=["first", "early", "late"])
@pytest.mark.parametrize("Hq,Nq,d,dtype", FORMS, ids=str)
def test_large_factor_of_a_block_without_weight(Hq, Nq, d, dtype, where, log2):
    """A page whose V factor is far above the others', with scores so low that it adds nothing: the other pages'
    weights keep their bits."""
    B, Hkv, cap, page = 2, 2, 1000, 16
    cache = Cache(B, cap, Hkv, d, page, [1000, 700], seed=71)
    q = queries(B, Nq, Hq, d, dtype, 72).abs()  # its product with keys of -448 is far below the others'
    far = np.full((Hkv, d), -448.0)
    for b in range(B):
        cache.kf[cache.table[b, where // page]] = 0.5
        put_page(cache, b, range(where, where + page), k=far, vf=2.0 ** (log2 - 6))
    want = cache.reference(q, d ** -0.5, False)
    # what the page adds: exp of at least 448/2 sum|q| / sqrt(d) below, times its values
    assert float(q.float().sum(-1).min()) * 224 * d ** -0.5 > 2 * np.log(2.0) * (log2 + 40)
    o, lse = decode(cache, q, d ** -0.5, False)
    check_decode(o, lse, want, q.dtype)


@pytest.mark.parametrize("log2", [24, 40, 60])
@pytest.mark.parametrize("Hq,Nq,d,dtype", [(8, 3, 128, "bf16"), (40, 3, 128, "bf16"), (6, 3, 64, "fp16"), (40, 3, 64, "bf16")], ids=str)
def test_large_factor_of_a_block_that_is_masked(Hq, Nq, d, dtype, log2):
    """The newest draft's page has a V factor far above the others': the rows that do not see it, and their
    bits, are those of a cache without it."""
    B, Hkv, cap, page = 3, 2, 1000, 16
    lens = [992 + 1, 480 + 1, 128 + 1]  # the last token alone in its page; with the first page of a key tile too
    cache = Cache(B, cap, Hkv, d, page, lens, seed=73)
    q = queries(B, Nq, Hq, d, dtype, 74)
    ordinary = cache.reference(q, d ** -0.5, True)
    for b, n in enumerate(lens):
        put_page(cache, b, [n - 1], vf=2.0 ** (log2 - 6))
    o, lse = decode(cache, q, d ** -0.5, True)
    unseen = [x[:, :-1] if i != 1 else x[..., :-1] for i, x in enumerate(ordinary)]
    check_decode(o[:, :-1], lse[..., :-1], unseen, q.dtype)
    want = cache.reference(q, d ** -0.5, True)
    e, step = (2.0 ** -8 + 2.0 ** -11, 2.0 ** -8) if q.dtype == torch.bfloat16 else (2.0 ** -11, 2.0 ** -11)
    if dtype == "bf16":  # (beyond fp16's range)
        # the last row: the page is in its tile's products, the arithmetic's 1e-3 in its units
        assert (np.abs(f64(o) - want[0]) <= e * want[2] + step * np.abs(want[0]) + 1e-3 * max(1.0, 2.0 ** (log2 - 6)))[:, -1].all()


@pytest.mark.parametrize("Hq,Nq,d,dtype", FORMS[:4] + [(4, 4, 64, "bf16")], ids=str)  # (beyond fp16's range)
@pytest.mark.parametrize("page", [0, 16, 64])
def test_factors_that_rise_and_fall(page, Hq, Nq, d, dtype):
    """V factors over 2^60 along a sequence with values that make up for them, so every block matters alike;
    zero blocks with the smallest factor among them."""
    B, Hkv, cap = 2, 2, 1500
    lens = [1500, 1200]
    cache = Cache(B, cap, Hkv, d, page, lens, seed=75)
    g = np.random.default_rng(76)
    q = queries(B, Nq, Hq, d, dtype, 77, 0.2)
    unit = cache.unit
    for b, n in enumerate(lens):
        shift = 0
        for i in range(-(-n // unit)):
            shift = int(np.clip(shift + g.integers(-14, 15), -30, 30))
            tokens = range(i * unit, min((i + 1) * unit, n))
            if g.integers(0, 5) == 0:
                put_page(cache, b, tokens, v=np.zeros((Hkv, d)), vf=2.0 ** -100)
                continue
            put_page(cache, b, tokens, vf=2.0 ** (shift - 6))
            # keys along the queries' mean: a score of about -shift ln 2 evens the block's share out
            u = f64(q)[b].mean((0, 1))
            key = -shift * np.log(2.0) * d ** 0.5 * u / (u @ u)
            amp = max(np.abs(key).max() / 400, 1e-30)
            f = 2.0 ** np.ceil(np.log2(amp))
            put_page(cache, b, tokens, k=np.tile(key / f, (Hkv, 1)))
            if page:
                cache.kf[cache.table[b, i]] = f
            else:
                cache.kf[b, :, i] = f
    o_ref, l_ref, w = cache.reference(q, d ** -0.5, False)
    o, lse = decode(cache, q, d ** -0.5, False)
    e, step = (2.0 ** -8 + 2.0 ** -11, 2.0 ** -8) if q.dtype == torch.bfloat16 else (2.0 ** -11, 2.0 ** -11)
    # scores to 60: fp32 arithmetic moves each by 2^-23 of the sum of its d products' magnitudes at most, a
    # weight by as much, so L by their largest and O by that share of sum p |v|
    moved = np.abs(l_ref).max() + 64
    small = 2.0 ** -20 * moved
    assert np.abs(f64(lse) - l_ref).max() <= 1e-3 + small
    assert (np.abs(f64(o) - o_ref) <= (e + small + 2.0 ** -14) * w + step * np.abs(o_ref)).all()
