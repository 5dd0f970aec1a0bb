"""The serving entry points without a GPU: invalid arguments are refused before anything touches the
device, and the torch helpers refuse tensors they would have to copy or convert."""
import numpy as np
import pytest
import torch

import oracle
from exact_tiled_attention_36_b200 import binding as fb
from exact_tiled_attention_36_b200 import build as fbuild
from tests import serve_ref as ref

FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
INV, UNS, MIS, OK = fb.FA_ERR_INVALID_ARG, fb.FA_ERR_UNSUPPORTED, fb.FA_ERR_MISALIGNED, fb.FA_OK


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbuild.build()
    fb.lib()


def contiguous(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, o=FAKE, lse=FAKE, sl=FAKE, ws=FAKE, B=2, Hq=8, Hkv=2, Nq=1,
             Nk=64, d=128, scale=0.1, causal=0, dtype=fb.FA_BF16, stream=None)
    a.update(kw)
    return fb.fa_decode_fp8(*a.values())


def paged(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, o=FAKE, lse=FAKE, sl=FAKE, bt=FAKE, ws=FAKE, B=2, Hq=8, Hkv=2,
             Nq=1, num_pages=9, page=64, max_pages=4, d=64, scale=0.1, causal=0, dtype=fb.FA_FP16, stream=None)
    a.update(kw)
    return fb.fa_decode_paged_fp8(*a.values())


@pytest.mark.parametrize("call,kw,code", [
    (contiguous, dict(q=None), INV), (contiguous, dict(ks=None), INV), (contiguous, dict(v=None), INV),
    (contiguous, dict(ws=None), INV), (contiguous, dict(lse=None), INV), (contiguous, dict(B=0), INV),
    (contiguous, dict(Nq=-1), INV), (contiguous, dict(Nk=-1), INV), (contiguous, dict(Hq=9), INV),
    (contiguous, dict(Hkv=0), INV), (contiguous, dict(scale=0.0), INV), (contiguous, dict(scale=float("nan")), INV),
    (contiguous, dict(causal=2), INV), (contiguous, dict(d=96), UNS), (contiguous, dict(d=256), UNS),
    (contiguous, dict(dtype=5), UNS), (contiguous, dict(Hq=64, Nq=5), UNS), (contiguous, dict(B=65536), UNS),
    (contiguous, dict(q=FAKE + 8), MIS), (contiguous, dict(k=FAKE + 4), MIS), (contiguous, dict(ks=FAKE + 2), MIS),
    (contiguous, dict(Nk=2 ** 31 - 1), UNS), (paged, dict(page=64, max_pages=2 ** 25 - 1), UNS),
    (contiguous, dict(sl=FAKE + 1), MIS), (contiguous, dict(ws=FAKE + 8), MIS), (contiguous, dict(Nq=0), OK),
    (paged, dict(sl=None), INV), (paged, dict(bt=None), INV), (paged, dict(num_pages=0), INV),
    (paged, dict(max_pages=0), INV), (paged, dict(page=8), INV), (paged, dict(page=48), UNS),
    (paged, dict(page=96), UNS), (paged, dict(page=1 << 20, max_pages=1 << 12), UNS), (paged, dict(bt=FAKE + 2), MIS),
    (paged, dict(vs=None), INV), (paged, dict(Nq=0), OK),
])
def test_decode_refuses_before_launch(call, kw, code):
    assert call(**kw) == code


def test_decode_workspace_size_of_invalid_sizes():
    for a in ((0, 8, 2, 1, 128), (1, 9, 2, 1, 128), (1, 8, 2, 1, 96), (1, 64, 2, 5, 128), (1, 8, 2, -1, 64)):
        assert fb.fa_decode_fp8_workspace_size(*a) == 0


def tables(**kw):
    a = dict(sl=FAKE, new=FAKE + 4, free=FAKE, bt=FAKE, slots=FAKE, cu=FAKE, lens=FAKE + 8, used=FAKE, B=2,
             num_free=4, num_pages=9, page=64, max_pages=4, total=5, stream=None)
    a.update(kw)
    return fb.fa_build_block_tables(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INV), (dict(num_free=-1), INV), (dict(num_pages=-1), INV), (dict(page=0), INV),
    (dict(max_pages=0), INV), (dict(total=-1), INV), (dict(new=None), INV), (dict(free=None), INV),
    (dict(bt=None), INV), (dict(slots=None), INV), (dict(cu=None), INV), (dict(lens=None), INV),
    (dict(used=None), INV), (dict(lens=FAKE), INV), (dict(lens=FAKE + 4), INV),
    (dict(cu=FAKE + 2), MIS), (dict(sl=FAKE + 1), MIS),
    (dict(page=1 << 16, num_pages=1 << 15), UNS), (dict(page=1 << 16, max_pages=1 << 15), UNS),
])
def test_tables_refuse_before_launch(kw, code):
    assert tables(**kw) == code


def append16(**kw):
    a = dict(k=FAKE, v=FAKE, ks=None, vs=None, kp=FAKE, vp=FAKE, slots=FAKE, total=5, Hkv=2, num_pages=9, page=16,
             d=64, dtype=fb.FA_BF16, stream=None)
    a.update(kw)
    return fb.fa_cache_append_paged(*a.values())


def append8(**kw):
    a = dict(k=FAKE, v=FAKE, ks=None, vs=None, kc=FAKE, vc=FAKE, kf=FAKE, vf=FAKE, cu=FAKE, sl=FAKE, lens=FAKE, B=2,
             total=5, most=5, Hkv=2, Nk=100, d=64, dtype=fb.FA_BF16, stream=None)
    a.update(kw)
    return fb.fa_cache_append_fp8(*a.values())


def append8p(**kw):
    a = dict(k=FAKE, v=FAKE, ks=None, vs=None, kc=FAKE, vc=FAKE, kf=FAKE, vf=FAKE, cu=FAKE, sl=FAKE, lens=FAKE,
             bt=FAKE, B=2, total=5, most=5, Hkv=2, num_pages=9, page=64, max_pages=4, d=64, dtype=fb.FA_BF16,
             stream=None)
    a.update(kw)
    return fb.fa_cache_append_paged_fp8(*a.values())


@pytest.mark.parametrize("call", [append16, append8, append8p])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(total=-1), INV), (dict(Hkv=0), INV), (dict(d=32), UNS),
    (dict(dtype=3), UNS), (dict(k=FAKE + 8), MIS), (dict(ks=(128, 0)), INV), (dict(ks=(128, 60)), MIS),
    (dict(vs=(-8, 64)), INV), (dict(vs=(130, 64)), MIS), (dict(total=0), OK),
])
def test_appends_refuse_before_launch(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("call,kw,code", [
    (append16, dict(kp=None), INV), (append16, dict(vp=FAKE + 8), MIS), (append16, dict(slots=None), INV),
    (append16, dict(num_pages=0), INV), (append16, dict(page=0), INV), (append16, dict(slots=FAKE + 2), MIS),
    (append16, dict(num_pages=1 << 20, page=1 << 11), UNS),
    (append8, dict(kc=None), INV), (append8, dict(kf=None), INV), (append8, dict(cu=None), INV),
    (append8, dict(lens=None), INV), (append8, dict(B=0), INV), (append8, dict(most=-1), INV),
    (append8, dict(Nk=-1), INV), (append8, dict(vf=FAKE + 2), MIS), (append8, dict(most=0), OK),
    (append8, dict(Nk=0), OK),
    (append8p, dict(bt=None), INV), (append8p, dict(page=8), INV), (append8p, dict(page=80), UNS),
    (append8p, dict(num_pages=0), INV), (append8p, dict(max_pages=0), INV), (append8p, dict(bt=FAKE + 2), MIS),
    (append8p, dict(page=1 << 20, max_pages=1 << 12), UNS),
])
def test_append_own_refusals(call, kw, code):
    assert call(**kw) == code


def test_helpers_refuse_cpu_tensors_and_wrong_types():
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 128, 2, 64, dtype=torch.uint8)
    f = torch.ones(1, 2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        fb.attention_decode_fp8(q, k, k, f, f)
    with pytest.raises(TypeError, match="q must be"):
        fb.attention_decode_fp8(q.float(), k, k, f, f)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fb.build_block_tables(i, i, i, i.view(2, 1), 16, 2, 0)
    with pytest.raises(TypeError, match="new_lens"):
        fb.build_block_tables(i, i.long(), i, i.view(2, 1), 16, 2, 0)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fb.cache_append_paged(x, x, x, x, i)
    with pytest.raises(ValueError, match="CUDA"):
        fb.cache_append_fp8(x, x, k, k, f, f, i, i, i, 3)


def test_row_strides_of_views():
    """Views of a packed projection keep their strides; a transposed head is refused."""
    meta = torch.zeros(5, 3, 2, 64, dtype=torch.bfloat16)

    class Fake:  # a CUDA tensor's shape and strides on a machine without one
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def get_device(self):
            return 0

        def __getattr__(self, name):
            return getattr(self.t, name)

    assert fb._rows(Fake(meta[:, 0]), "k", 0) == (384, 64)
    assert fb._rows(Fake(meta[:, 0].contiguous()), "k", 0) == (128, 64)
    assert fb._rows(Fake(meta[:1, 0, :1]), "k", 0) == (64, 64)
    assert fb._rows(Fake(meta[:, 0, :1]), "k", 0) == (384, 64)
    with pytest.raises(ValueError, match="contiguous"):
        fb._rows(Fake(meta[:, 0].transpose(1, 2)), "k", 0)
    with pytest.raises(ValueError, match="tokens"):
        fb._rows(Fake(meta), "k", 0)


# The references themselves, against torch and by hand.
def test_reference_encoder_is_the_format_s_rounding():
    x = torch.cat([torch.randn(20000) * 2.0 ** torch.randint(-12, 8, (20000,)), torch.linspace(-448, 448, 7169),
                   torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 447.9, 17.0, 19.0])])
    x = x.clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn)
    got = ref.e4m3_encode(x.numpy())
    assert np.array_equal(got, want.view(torch.uint8).numpy())
    assert ref.e4m3_encode([np.inf, np.nan]).tolist() == [0x7F, 0x7F]


def test_reference_factor():
    for a, f in ((448.0, 1.0), (448.1, 2.0), (0.0, 2.0 ** -100), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7),
                 (3.38e38, 2.0 ** 120)):
        assert ref.factor_of(a) == f


def test_reference_append_rescales_a_growing_block():
    codes = np.zeros((1, 16, 1, 2), np.uint8)
    fac = np.array([[1.0]])
    codes[0, :2, 0] = ref.e4m3_encode([[1.0, -448.0], [2.0 ** -9, 3 * 2.0 ** -9]])
    ref.append_fp8(np.array([[[1000.0, 1.0]]]), codes, fac, [[0]], [0, 1], [2], [3], 16)
    assert fac[0, 0] == 4.0
    # 2^-9 / 4 rounds to 0; 3 2^-9 / 4 = 0.75 steps rounds to one step
    assert oracle.e4m3_decode(codes[0, :3, 0]).tolist() == [[0.25, -112.0], [0.0, 2.0 ** -9], [256.0, 0.25]]


def test_reference_tables_by_hand():
    table, slots, cu, lens, used = ref.tables([3, 0], [2, 5], [8, 9, 7], [[4, -1], [-1, -1]], 4, 10, 8)
    assert table == [[4, 8], [9, 7]] and lens == [5, 5] and cu == [0, 2, 7] and used == 3
    assert slots == [19, 32, 36, 37, 38, 39, 28, -1]
