"""Appends to an E4M3 cache where many blocks have no page: their rows are on their way to shared memory
when that is found out, and the neighbours' results must not show it."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_36_b200 import binding as fb
from tests import serve_ref as ref
from tests.gpu_util import f64
from tests.test_serve_gpu import DT, dev, run_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("page", [16, 64, 128, 256])  # one warp to 256 threads a block
def test_append_among_blocks_without_a_page(page, d, dtype):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B, Hkv, per = 24, 4, 5
    g = np.random.default_rng(page + d)
    olds = g.integers(0, page, B).tolist()
    counts = [per * page - o for o in olds]
    cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
    lens = [o + c for o, c in zip(olds, counts)]
    n = B * per + 1
    place = g.permutation(B * per).reshape(B, per).astype(np.int32)
    codes = [ref.e4m3_encode(np.clip(g.standard_normal((n, page, Hkv, d)) * 64, -448, 448)) for _ in "kv"]
    fac = [np.exp2(g.integers(-8, -4, (n, Hkv))) for _ in "kv"]
    x = torch.from_numpy(g.standard_normal((cu[-1], 2, Hkv, d))).to(DT[dtype])
    table = place.copy()
    lost = g.random((B, per)) < 0.5
    table[lost] = g.choice([-1, n, n + 77, -2 ** 31, 2 ** 31 - 1], int(lost.sum()))
    pools = [torch.from_numpy(c.copy()).cuda() for c in codes]
    facs = [torch.from_numpy(f.astype(np.float32)).cuda() for f in fac]
    xd = x.cuda()
    fb.cache_append_fp8(xd[:, 0], xd[:, 1], *pools, *facs, dev(cu), dev(olds), dev(lens), max(counts),
                        block_table=torch.from_numpy(table).cuda())
    assert fb.fa_get_last_device_error(None) == fb.FA_ERR_INVALID_ARG
    kept = place[lost]
    for i in range(2):
        want, wf = codes[i].copy(), fac[i].copy()
        ref.append_fp8(f64(x[:, i]), want, wf, place, cu, olds, lens, page)
        want[kept], wf[kept] = codes[i][kept], fac[i][kept]
        assert np.array_equal(facs[i].cpu().numpy(), wf.astype(np.float32))
        assert np.array_equal(pools[i].cpu().numpy(), want)


@pytest.mark.parametrize("page", [16, 64])
def test_append_of_a_prompt_beside_single_tokens(page):
    """One long prompt, single tokens and idle sequences in one call."""
    g = np.random.default_rng(page)
    B = 40
    counts = g.integers(0, 2, B).tolist()
    counts[17] = 1900
    olds = [int(g.integers(0, 140)) for _ in range(B)]
    got_c, got_f, codes, fac = run_append((page, 2048, 2, 64, "bf16", olds, counts))
    for i in range(2):
        assert np.array_equal(got_f[i], fac[i])
        assert np.array_equal(got_c[i], codes[i])
