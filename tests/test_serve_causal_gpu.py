"""Decode over an E4M3 cache with several causal query tokens where every CTA takes many key tiles and
many segments, so that its warps run far ahead of one another: tiles that only some rows see one after
the other at a segment's end, and sequences of a single such tile, with NaN codes among the new tokens.
Bounds: those of test_serve_gpu.py."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_36_b200 import binding as fb
from tests import serve_ref as ref
from tests.gpu_util import f64
from tests.test_serve_gpu import Cache, check_decode, dev, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    fb.lib()
    yield
    assert fb.fa_get_last_device_error(None) == fb.FA_OK


class BigCache(Cache):
    """As Cache, with values drawn from a table (encoding millions one by one takes long)."""

    def __init__(self, B, cap, Hkv, d, page, lens, seed):
        super().__init__(B, 1, Hkv, d, page, [0] * B, seed)
        g = np.random.default_rng(seed)
        table = ref.e4m3_encode(np.clip(g.standard_normal(1 << 16) * 64, -448, 448))
        self.lens, per = lens, -(-cap // self.unit)
        shape = (B, cap, Hkv, d) if not page else (B * per + 2, page, Hkv, d)
        fshape = (B, Hkv, per) if not page else (B * per + 2, Hkv)
        self.k, self.v = (table[g.integers(0, 1 << 16, shape, dtype=np.uint16)] for _ in "kv")
        self.kf, self.vf = (np.exp2(g.integers(-8, -3, fshape)).astype(np.float32) for _ in "kv")
        if page:
            self.table = g.permutation(B * per + 2)[:B * per].reshape(B, per).astype(np.int32)

    def at(self, b, pos):
        return (b, pos) if not self.page else (self.table[b, pos // self.page], pos % self.page)


def several_tiles(g, Nq, B):
    """Lengths just past a tile's end: the last two tiles of a segment are both seen by some rows only."""
    return (128 * g.integers(4, 9, B) + g.integers(1, Nq - 1, B)).tolist()


def one_tile(g, Nq, B):
    return g.integers(2, 129, B).tolist()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Nq", [(8, 4), (4, 7), (20, 4), (32, 7), (2, 32), (2, 128)])  # 14 to 128 rows of a KV head
@pytest.mark.parametrize("lengths,page,B", [(several_tiles, 0, 110), (several_tiles, 64, 110), (one_tile, 16, 600)])
def test_causal_tiles_in_a_row(lengths, page, B, Hq, Nq, d, dtype):
    Hkv, g = 2, np.random.default_rng(Hq + Nq + d)
    lens = lengths(g, Nq, B)
    cache = BigCache(B, max(lens), Hkv, d, page, lens, seed=Hq + d)
    q = queries(B, Nq, Hq, d, dtype, 51)
    bad = np.zeros((B, Nq, Hq, d), dtype=bool)
    put = []
    for b in range(0, B, 3):
        pos, h, c = max(lens[b] - 1 - int(g.integers(0, Nq)), 0), int(g.integers(0, Hkv)), int(g.integers(0, d))
        put.append((*cache.at(b, pos), h, c))
        for t in range(Nq):
            bad[b, t, h * Hq // Hkv:(h + 1) * Hq // Hkv, c] |= pos <= t + lens[b] - Nq
    for x in put:
        cache.v[x] = 0
    want = cache.reference(q, d ** -0.5, True)
    for x in put:
        cache.v[x] = 0xFF
    args, bt = cache.cuda(), None if not page else torch.from_numpy(cache.table).cuda()
    runs = [fb.attention_decode_fp8(q, *args, dev(lens), causal=True, block_table=bt) for _ in range(20)]
    torch.cuda.synchronize()
    assert fb.fa_get_last_device_error(None) == fb.FA_OK
    o, lse = runs[0]
    for o2, l2 in runs[1:]:
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)
    assert np.array_equal(np.isnan(f64(o)), bad)
    check_decode(torch.where(torch.from_numpy(bad).cuda(), torch.from_numpy(want[0]).cuda().to(o.dtype), o), lse, want, q.dtype)
