"""The serving operators on the GPU against plain 64-bit references: decode over an E4M3 cache
(fa_decode_fp8, fa_decode_paged_fp8), the appends that write the caches, block tables with slot
maps, and a run of them together.

Bounds of the decode. P is rounded to fp16 (half a step of 10 mantissa bits: 2^-11 of a weight); for
bf16 up to 32 rows of a KV head (d = 64: 24) it is then split into two E4M3 terms, which leave at most 2^-8 of it
(half a step of a 3-bit mantissa is 2^-4 of the value, and so of the remainder; the three terms of fp16
hold all 11 bits), or 2^-22 of the key tile's largest weight below E4M3's normal range (2^-25 of the
running reference in the form for more rows, fp16 throughout), so
    |O - O_ref| <= e sum_j p_j |v_j| + half a step of the output type at O_ref + 1e-3,
e = 2^-8 + 2^-11 for bf16 and 2^-11 for fp16, the last for the fp32 arithmetic (as for the FP8 forward)
and the smallest weights. L comes from the exact scores and keeps max|L - L_ref| <= 1e-3.
Integers, codes and factors are exact."""
import numpy as np
import pytest
import torch

import oracle
from exact_tiled_attention_36_b200 import binding as fb
from tests import serve_ref as ref
from tests.gpu_util import _record as record, check_l, f64, guarded

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    fb.lib()
    yield
    assert fb.fa_get_last_device_error(None) == fb.FA_OK


def guarded_bytes(shape, guard=4096):
    """A byte tensor inside a filled buffer, and a checker of the guards (gpu_util.guarded for bytes)."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf[guard:guard + n].view(*shape), lambda: bool((buf[:guard] == 0xA5).all() and (buf[guard + n:] == 0xA5).all())


def dev(x, dtype=I32):
    return torch.tensor(x, dtype=dtype, device="cuda")


# ------------------------------------------------------------------------------- decode
class Cache:
    """Random E4M3 caches: page 0 contiguous [B, cap, Hkv, d], else a shuffled page pool. Rows past
    a sequence's length hold NaN codes."""

    def __init__(self, B, cap, Hkv, d, page, lens, seed, spread=2, factors=None):
        g = np.random.default_rng(seed)
        self.unit, self.page, self.lens = page or 128, page, lens
        per = -(-cap // self.unit)
        shape = (B, cap, Hkv, d) if not page else (B * per + 2, page, Hkv, d)
        fshape = (B, Hkv, per) if not page else (B * per + 2, Hkv)
        self.k, self.v = (ref.e4m3_encode(np.clip(g.standard_normal(shape) * 64, -448, 448)) for _ in "kv")
        self.kf, self.vf = (np.exp2(g.integers(-6 - spread, -5 + spread, fshape)).astype(np.float32) for _ in "kv")
        if factors is not None:  # not powers of two: a caller's own
            self.kf, self.vf = (f * g.uniform(1, 1.99, fshape).astype(np.float32) for f in (self.kf, self.vf))
        self.table = None
        if page:
            self.table = g.permutation(B * per + 2)[:B * per].reshape(B, per).astype(np.int32)
            for b, n in enumerate(lens):
                for i in range(per):
                    first = max(0, min(page, n - i * page))
                    self.k[self.table[b, i], first:] = self.v[self.table[b, i], first:] = 0x7F
        else:
            for b, n in enumerate(lens):
                self.k[b, n:] = self.v[b, n:] = 0xFF

    def cuda(self):
        return [torch.from_numpy(x).cuda() for x in (self.k, self.v, self.kf, self.vf)]

    def reference(self, q, scale, causal):
        return ref.decode_fp8(f64(q), self.k, self.v, self.kf.astype(np.float64), self.vf.astype(np.float64),
                              self.lens, scale, causal, self.unit, self.table)


def check_decode(o, lse, want, dtype):
    o_ref, l_ref, w = want
    o, lse = f64(o), f64(lse)
    empty = np.isneginf(l_ref)
    assert np.isneginf(lse[empty]).all() and (o[np.moveaxis(empty, 1, 2)] == 0).all(), "rows without keys"
    assert np.isfinite(lse[~empty]).all() and np.isfinite(o).all()
    check_l(lse[~empty], l_ref[~empty])
    e, step = (2.0 ** -8 + 2.0 ** -11, 2.0 ** -8) if dtype == torch.bfloat16 else (2.0 ** -11, 2.0 ** -11)
    bound = e * w + step * np.abs(o_ref) + 1e-3
    err = np.abs(o - o_ref)
    record("O", err.max(), (err - bound).max())
    assert (err <= bound).all(), (err.max(), (err - bound).max())


def decode(cache, q, scale, causal, ws=None, stream=0):
    B, Nq, Hq, d = q.shape
    Hkv = cache.k.shape[2]
    k, v, kf, vf = cache.cuda()
    o, o_ok = guarded((B, Nq, Hq, d), q.dtype)
    lse, l_ok = guarded((B, Hq, Nq), torch.float32)
    if ws is None:
        ws = torch.full((fb.fa_decode_fp8_workspace_size(B, Hq, Hkv, Nq, d),), 255, dtype=torch.uint8, device="cuda")
    dt = fb.FA_BF16 if q.dtype == torch.bfloat16 else fb.FA_FP16
    sl = dev(cache.lens)
    if cache.page:
        bt = torch.from_numpy(cache.table).cuda()
        st = fb.fa_decode_paged_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), kf.data_ptr(), vf.data_ptr(),
                                    o.data_ptr(), lse.data_ptr(), sl.data_ptr(), bt.data_ptr(), ws.data_ptr(), B, Hq,
                                    Hkv, Nq, k.shape[0], cache.page, bt.shape[1], d, scale, int(causal), dt, stream)
    else:
        full = all(n == k.shape[1] for n in cache.lens)  # a full batch gives no lengths
        st = fb.fa_decode_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), kf.data_ptr(), vf.data_ptr(), o.data_ptr(),
                              lse.data_ptr(), 0 if full else sl.data_ptr(), ws.data_ptr(), B, Hq, Hkv, Nq, k.shape[1],
                              d, scale, int(causal), dt, stream)
    assert st == fb.FA_OK, fb.fa_status_string(st)
    torch.cuda.synchronize()
    assert fb.fa_get_last_device_error(None) == fb.FA_OK
    assert o_ok() and l_ok(), "write outside O / L"
    return o, lse


def queries(B, Nq, Hq, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, Nq, Hq, d, generator=g) * scale).to(DT[dtype]).cuda()


DECODES = [
    # B, Hq, Hkv, Nq, cap, d, type, page, causal, lengths
    (1, 1, 1, 1, 1, 128, "bf16", 0, False, [1]),                       # one key, one row
    (3, 8, 2, 1, 1000, 128, "bf16", 0, False, [1000, 1000, 1000]),     # full caches, a ragged last tile
    (5, 8, 2, 2, 2048, 128, "bf16", 0, True, [0, 1, 129, 1000, 2047]),  # an empty sequence, rows without keys
    (3, 4, 4, 1, 777, 64, "fp16", 0, False, [777, 5, 640]),            # one row an item, d = 64
    (3, 6, 3, 1, 900, 64, "bf16", 0, False, [900, 1, 128]),            # d = 64, odd Hkv
    (3, 32, 4, 4, 1500, 128, "bf16", 0, True, [1500, 3, 1024]),        # 32 rows
    (3, 6, 2, 20, 300, 128, "fp16", 0, True, [300, 260, 17]),          # 60 rows
    (2, 16, 1, 8, 900, 64, "bf16", 0, True, [900, 411]),               # 128 rows
    (2, 5, 1, 5, 600, 64, "fp16", 32, True, [600, 2]),                 # 25 rows of one small head
    (40, 32, 8, 1, 700, 128, "bf16", 0, False, list(range(0, 680, 17))),  # many short items
    (4, 8, 2, 2, 1100, 128, "bf16", 16, True, [1100, 0, 33, 640]),
    (4, 8, 2, 2, 1100, 128, "fp16", 32, False, [1, 31, 1099, 512]),
    (4, 8, 2, 1, 1100, 128, "bf16", 64, True, [1100, 65, 64, 63]),
    (3, 10, 2, 3, 1200, 128, "fp16", 192, True, [1200, 193, 5]),       # pages that end inside a key tile
    (4, 8, 4, 2, 1300, 64, "bf16", 16, True, [1300, 17, 0, 1000]),
    (3, 7, 7, 1, 1280, 64, "bf16", 256, False, [1280, 257, 100]),
    (2, 24, 1, 1, 500, 64, "bf16", 32, True, [500, 77]),               # three chunks of rows
    (2, 32, 1, 1, 500, 128, "bf16", 0, False, [500, 77]),              # two, in step
    (2, 33, 1, 1, 1000, 128, "bf16", 0, False, [1000, 1]),             # just past the transposed form
    (3, 64, 1, 2, 700, 128, "fp16", 64, True, [700, 1, 130]),          # 128 rows
    (3, 80, 2, 1, 1500, 128, "bf16", 16, False, [1500, 0, 129]),       # 40 rows, small pages, an empty sequence
    (2, 144, 3, 2, 640, 64, "bf16", 32, True, [640, 333]),             # 96 rows of one of two loaded heads, odd Hkv
    (5, 32, 1, 3, 2000, 64, "fp16", 0, True, [2000, 2, 128, 1025, 0]),
    (30, 96, 2, 1, 600, 128, "bf16", 0, False, list(range(0, 600, 20))),  # many short items
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: "-".join(map(str, c[:9])))
def test_decode(case):
    B, Hq, Hkv, Nq, cap, d, dtype, page, causal, lens = case
    cache = Cache(B, cap, Hkv, d, page, lens, seed=sum(lens) + d)
    q = queries(B, Nq, Hq, d, dtype, 3)
    o, lse = decode(cache, q, d ** -0.5, causal)
    check_decode(o, lse, cache.reference(q, d ** -0.5, causal), q.dtype)


@pytest.mark.parametrize("Hq", [8, 80])
@pytest.mark.parametrize("page", [0, 16, 64])
def test_decode_factors_of_any_value(page, Hq):
    """Factors that are no powers of two and differ by 2^12 between a sequence's blocks."""
    cache = Cache(2, 1000, 2, 128, page, [1000, 413], seed=5, spread=6, factors="own")
    q = queries(2, 1, Hq, 128, "bf16", 6, 0.1)
    o, lse = decode(cache, q, 128 ** -0.5, False)
    o_ref, l_ref, w = cache.reference(q, 128 ** -0.5, False)
    # 2^-22 of the tile's largest weight times the largest value of the tile, 128 times (in the form for
    # many rows 2^-25 of the reference, which is at most 2^8 times the tile's: less)
    floor = 2.0 ** -22 * 128 * 448 * float(cache.vf.max())
    assert np.abs(f64(lse) - l_ref).max() <= 1e-3
    assert (np.abs(f64(o) - o_ref) <= (2.0 ** -8 + 2.0 ** -11) * w + 2.0 ** -8 * np.abs(o_ref) + 1e-3 + floor).all()


@pytest.mark.parametrize("Hq", [4, 36])
def test_decode_one_key_above_a_long_tail(Hq):
    """One key well above 20000 others, whose small weights together still matter."""
    B, Hkv, cap, d = 1, 1, 20000, 128
    cache = Cache(B, cap, Hkv, d, 0, [cap], seed=8)
    q = queries(B, 1, Hq, d, "bf16", 9)
    cache.k[0, :, 0] = ref.e4m3_encode(np.zeros((cap, d)))
    cache.v[0, :, 0] = ref.e4m3_encode(np.full((cap, d), 64.0))
    cache.kf[:], cache.vf[:] = 2.0 ** -6, 2.0 ** -6
    u = f64(q)[0, 0]
    key = u.sum(0) / max(1, Hq / 12)  # q . key about 12 after scaling (between 2 and 6 of many heads)
    cache.k[0, 777, 0] = ref.e4m3_encode(np.clip(key * 64, -448, 448))
    cache.v[0, 777, 0] = ref.e4m3_encode(np.full(d, -64.0))
    o, lse = decode(cache, q, d ** -0.5, False)
    check_decode(o, lse, cache.reference(q, d ** -0.5, False), q.dtype)


@pytest.mark.parametrize("Hq", [8, 72])
def test_decode_large_and_small_queries(Hq):
    """Query rows of very different sizes side by side, zeros among them."""
    cache = Cache(2, 500, 2, 128, 0, [500, 300], seed=10)
    q = queries(2, 1, Hq, 128, "bf16", 11)
    sizes = torch.tensor([1e-20, 1.0, 0.0, 3.0, 1e-3, 0.1, 1.0, 2.0] * (Hq // 8), device="cuda")
    q *= sizes.to(q.dtype)[None, None, :, None]
    o, lse = decode(cache, q, 128 ** -0.5, False)
    check_decode(o, lse, cache.reference(q, 128 ** -0.5, False), q.dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [4, 8, 80])
def test_decode_nan_stays_in_its_rows(Hq, d):
    """A NaN in one query row, or in one KV head's keys, reaches that row or head alone."""
    cache = Cache(2, 400, 2, d, 64, [400, 222], seed=12)
    q = queries(2, 1, Hq, d, "bf16", 13)
    q[0, 0, 0, 5] = float("nan")
    q[0, 0, 1, 5] = float("inf")
    cache.k[cache.table[1, 1], 3, 1, 7] = 0x7F
    o, lse = decode(cache, q, d ** -0.5, False)
    bad = torch.zeros(2, Hq, dtype=torch.bool)
    bad[0, :2] = True
    bad[1, Hq // 2:] = True
    assert torch.equal(torch.isnan(o[:, 0]).all(-1).cpu(), bad) and torch.equal(torch.isnan(o[:, 0]).any(-1).cpu(), bad)
    assert torch.equal(torch.isnan(lse[:, :, 0]).cpu(), bad)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [2, 4, 8, 16, 36])
@pytest.mark.parametrize("page", [0, 16])
def test_decode_nan_values_of_new_tokens(page, Hq, d):
    """A NaN among a new token's values (an infinity that was appended) reaches the rows that see the
    token, at its own index, and no row before it; its key's NaN reaches their whole outputs."""
    Hkv, Nq, cap = 2, 3, 600
    lens = [600, 129, 257, 2, 600]
    cache = Cache(5, cap, Hkv, d, page, lens, seed=41)
    q = queries(5, Nq, Hq, d, "bf16", 42)

    def put(x, b, pos, h, c):
        x[(b, pos, h, c) if not page else (cache.table[b, pos // page], pos % page, h, c)] = 0xFF

    place = [(0, 598, 0, 3), (0, 599, 0, 3), (0, 599, 1, d - 1), (1, 128, 1, 17), (1, 127, 0, 40), (2, 256, 0, 0),
             (3, 1, 1, 5)]  # values: sequence, position, head, index
    g = Hq // Hkv
    bad = np.zeros((5, Nq, Hq, d), dtype=bool)
    for b, pos, h, c in place:
        for t in range(Nq):
            bad[b, t, h * g:h * g + g, c] |= pos <= t + lens[b] - Nq
    zero = Cache(5, cap, Hkv, d, page, lens, seed=41)  # the same with zeros there
    for b, pos, h, c in place:
        put(cache.v, b, pos, h, c)
        zero.v[(b, pos, h, c) if not page else (cache.table[b, pos // page], pos % page, h, c)] = 0
    want = zero.reference(q, d ** -0.5, True)
    o, lse = decode(cache, q, d ** -0.5, True)
    assert np.array_equal(np.isnan(f64(o)), bad)
    check_decode(torch.where(torch.from_numpy(bad).cuda(), torch.from_numpy(want[0]).cuda().to(o.dtype), o), lse, want, q.dtype)
    put(cache.k, 4, 599, 1, 9)  # a key of the last token
    o, lse = decode(cache, q, d ** -0.5, True)
    bad[4, 2, g:] = True
    assert np.array_equal(np.isnan(f64(o)), bad)
    assert np.array_equal(np.isnan(f64(lse)), np.moveaxis(bad.all(-1), 1, 2))


@pytest.mark.parametrize("B,Hq,page", [(700, 1, 0), (700, 4, 16), (1300, 40, 16)])
def test_decode_many_sequences(B, Hq, page):
    """More sequences than a block has threads, most of them short or empty, long ones at the end."""
    lens = [(7 * b) % 5 * (b % 3) for b in range(B)]
    lens[B - 2], lens[520], lens[3] = 300, 290, 131
    cache = Cache(B, 304, 1, 128, page, lens, seed=43)
    q = queries(B, 1, Hq, 128, "bf16", 44)
    o, lse = decode(cache, q, 128 ** -0.5, False)
    check_decode(o, lse, cache.reference(q, 128 ** -0.5, False), q.dtype)


@pytest.mark.parametrize("Hq", [8, 72])
def test_decode_captured_behind_other_work(Hq):
    """A captured call behind a memset, a copy and another stream's work, replayed over new contents; two
    calls at once on two streams, each with its workspace."""
    caches = [Cache(3, 900, 2, 128, 0, [900, 33, 512], seed=s) for s in (45, 46)]
    q = queries(3, 1, Hq, 128, "bf16", 47)
    data = [c.cuda() for c in caches]
    want = [c.reference(q, 128 ** -0.5, False) for c in caches]
    sl = dev([900, 33, 512])
    k, v, kf, vf = (torch.empty_like(x) for x in data[0])
    src = [x.clone() for x in data[0]]
    side, here = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=here):
        for x in (k, v):
            x.zero_()  # a memset
        side.wait_stream(here)
        with torch.cuda.stream(side):
            for x, y in zip((v, vf), (src[1], src[3])):
                x.copy_(y)
        for x, y in zip((k, kf), (src[0], src[2])):
            x.copy_(y)
        first = fb.attention_decode_fp8(q, k, k, kf, kf, sl)
        here.wait_stream(side)
        out = fb.attention_decode_fp8(q, k, v, kf, vf, sl)
        again = fb.attention_decode_fp8(q, k, v, kf, vf, sl)
        k.zero_()  # (only after both have read it)
    for i in (0, 1, 0):
        for x, y in zip(src, data[i]):
            x.copy_(y)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_decode(*out, want[i], q.dtype)
        assert all(torch.equal(a, b) for a, b in zip(out, again)) and torch.isfinite(first[0]).all()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(10):
        outs.append((0, fb.attention_decode_fp8(q, *data[0], sl)))
        outs.append((1, fb.attention_decode_fp8(q, *data[1], sl, stream=side)))
    torch.cuda.synchronize()
    for i, (a, b) in outs:
        check_decode(a, b, want[i], q.dtype)
    assert fb.fa_get_last_device_error(None) == fb.FA_OK


@pytest.mark.parametrize("Hq", [8, 70])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_pages_outside_the_pool_read_zeros(page, Hq):
    cache = Cache(3, 700, 2, 128, page, [700, 300, 650], seed=14)
    n = cache.k.shape[0]
    for b, i, pg in ((0, 1, -1), (0, 5, n), (1, 0, n + 1000), (2, 650 // page, -7)):
        cache.table[b, i] = pg
    q = queries(3, 2, Hq, 128, "bf16", 15)
    o, lse = decode(cache, q, 128 ** -0.5, True)
    check_decode(o, lse, cache.reference(q, 128 ** -0.5, True), q.dtype)


def test_decode_no_keys():
    q = queries(2, 3, 8, 64, "bf16", 16)
    cache = Cache(2, 64, 2, 64, 64, [0, 0], seed=17)
    o, lse = decode(cache, q, 0.1, True)
    assert (o == 0).all() and torch.isneginf(lse).all()
    z = torch.zeros(0, dtype=torch.uint8, device="cuda")
    o, lse = fb.attention_decode_fp8(q, z.view(2, 0, 2, 64), z.view(2, 0, 2, 64), z.float().view(2, 2, 0),
                                     z.float().view(2, 2, 0))
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = fb.attention_decode_fp8(q[:, :0], *[x for x in cache.cuda()], dev([0, 0]),
                                     block_table=torch.from_numpy(cache.table).cuda())
    assert o.shape == (2, 0, 8, 64) and lse.shape == (2, 8, 0)


def test_decode_workspace_kept_between_layouts():
    """A workspace that holds another call's partial results gives the right answer."""
    B, Hq, Hkv, d = 16, 8, 2, 128
    ws = torch.empty(fb.fa_decode_fp8_workspace_size(B, Hq, Hkv, 1, d), dtype=torch.uint8, device="cuda")
    q = queries(B, 1, Hq, d, "bf16", 18)
    for lens in (list(range(0, 1600, 100)), [0] * 8 + [1600] * 8, list(range(0, 1600, 100))):
        cache = Cache(B, 1600, Hkv, d, 0, lens, seed=19)
        o, lse = decode(cache, q, d ** -0.5, False, ws=ws)
        check_decode(o, lse, cache.reference(q, d ** -0.5, False), q.dtype)


@pytest.mark.parametrize("Hq", [8, 68])
@pytest.mark.parametrize("word", [-2 ** 31, 2 ** 31 - 1, 0, -1])
def test_decode_workspace_contents_do_not_matter(word, Hq):
    """Empty sequences among others, one of them alone, whatever the workspace holds on entry."""
    for lens, cap in (([0, 700, 0, 1, 0], 700), ([0], 128)):
        B = len(lens)
        ws = torch.empty(fb.fa_decode_fp8_workspace_size(B, Hq, 2, 1, 128) // 4, dtype=I32, device="cuda").fill_(word)
        cache = Cache(B, cap, 2, 128, 0, lens, seed=23)
        q = queries(B, 1, Hq, 128, "bf16", 24)
        k, v, kf, vf = cache.cuda()
        o, lse = fb.attention_decode_fp8(q, k, v, kf, vf, dev(lens), workspace=ws.view(torch.uint8))
        check_decode(o, lse, cache.reference(q, 128 ** -0.5, False), q.dtype)


@pytest.mark.parametrize("Hq", [16, 100])
def test_decode_is_deterministic_and_takes_any_stream(Hq):
    cache = Cache(6, 3000, 2, 128, 64, [3000, 1, 2999, 128, 1500, 777], seed=20)
    q = queries(6, 1, Hq, 128, "bf16", 21)
    k, v, kf, vf = cache.cuda()
    sl, bt = dev(cache.lens), torch.from_numpy(cache.table).cuda()
    o, lse = fb.attention_decode_fp8(q, k, v, kf, vf, sl, block_table=bt)
    check_decode(o, lse, cache.reference(q, 128 ** -0.5, False), q.dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [fb.attention_decode_fp8(q, k, v, kf, vf, sl, block_table=bt, stream=side) for _ in range(4)]
    f8 = torch.float8_e4m3fn  # the codes under their own type
    outs += [fb.attention_decode_fp8(q, k.view(f8), v.view(f8), kf, vf, sl, block_table=bt) for _ in range(2)]
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)


# ------------------------------------------------------------------------------- block tables
TABLES = [
    # page, table width, lengths before, new lengths, free pages beyond the need (negative: too few)
    (16, 8, [0], [1], 0),
    (64, 4, [0, 64, 65, 100], [1, 1, 63, 0], 3),
    (16, 40, [5, 0, 16, 600, 31, 7], [0, 0, 0, 40, 1, 300], 0),
    (1, 9, [3, 0, 8], [2, 9, 1], 1),
    (192, 6, [191, 192, 1000], [1, 1, 152], 5),
    (16, 8, [0, 10, 20], [100, 6, 30], -2),           # the free list ends: the last request gets nothing
    (16, 8, [0, 10, 20], [100, 6, 12], -7),           # the first one too; the others need no page
    (16, 4, [60, 10, -3, 5], [5, 4, 3, -1], 2),       # past the table, and negative lengths
    (32, 3, [0] * 700, [i % 50 for i in range(700)], 11),  # more requests than one scan step takes
]


@pytest.mark.parametrize("case", TABLES, ids=lambda c: f"p{c[0]}-b{len(c[2])}-{c[4]}")
@pytest.mark.parametrize("pad", [0, 37])
def test_block_tables(case, pad):
    page, width, olds, news, spare = case
    B = len(olds)
    g = np.random.default_rng(B + page)
    need = sum(max(0, -(-(n + c) // page) - -(-n // page)) for n, c in zip(olds, news)
               if n >= 0 and c >= 0 and n + c <= width * page)
    num_pages = B * width + max(spare, 0) + need
    order = g.permutation(num_pages).astype(np.int32)
    table = np.full((B, width), -9, np.int32)
    for b, n in enumerate(olds):
        have = max(0, -(-n // page))
        table[b, :have] = order[b * width:b * width + have]
    free = order[B * width:][:need + spare]
    total = sum(max(c, 0) for c in news) + pad
    want = ref.tables(olds, news, free, table, page, num_pages, total)
    bt = torch.from_numpy(table).cuda()
    got = fb.build_block_tables(dev(olds), dev(news), torch.from_numpy(free.copy()).cuda(), bt, page, num_pages, total)
    short = want[3] != [n + max(c, 0) for n, c in zip(olds, news)] or min(news) < 0
    assert fb.fa_get_last_device_error(None) == (fb.FA_ERR_INVALID_ARG if short else fb.FA_OK)
    for name, a, b in zip(("slots", "cu", "lens"), got, want[1:4]):
        assert a.tolist() == b, name
    assert int(got[3]) == want[4] and bt.tolist() == want[0]


def test_block_tables_many_tokens_and_no_room():
    """Slots over many CTAs; a packed buffer that ends inside a request; a page outside the pool."""
    g = np.random.default_rng(3)
    page, B, width = 16, 300, 64
    olds, news = g.integers(0, 500, B).tolist(), g.integers(0, 500, B).tolist()
    order = g.permutation(B * width * 2).astype(np.int32)
    table = order[:B * width].reshape(B, width).copy()
    free = order[B * width:].copy()
    num = 2 * B * width
    for total, pages in ((sum(news), num), (sum(news) - 700, num), (0, num), (sum(news), num - 3)):
        want = ref.tables(olds, news, free, table, page, pages, total)
        bt = torch.from_numpy(table).cuda()
        got = fb.build_block_tables(dev(olds), dev(news), torch.from_numpy(free).cuda(), bt, page, pages, total)
        cut = total < sum(news) or -1 in want[1]
        assert fb.fa_get_last_device_error(None) == (fb.FA_ERR_INVALID_ARG if cut else fb.FA_OK)
        for name, a, b in zip(("slots", "cu", "lens"), got, want[1:4]):
            assert a.tolist() == b, name
        assert int(got[3]) == want[4] and bt.tolist() == want[0]


def test_block_tables_of_new_requests_need_no_lengths():
    bt = torch.full((2, 3), -1, dtype=I32, device="cuda")
    slots, cu, lens, used = fb.build_block_tables(None, dev([40, 3]), dev([7, 5, 2, 9]), bt, 16, 10, 43)
    assert bt.tolist() == [[7, 5, 2], [9, -1, -1]] and cu.tolist() == [0, 40, 43] and lens.tolist() == [40, 3]
    assert slots.tolist() == [7 * 16 + i for i in range(16)] + [5 * 16 + i for i in range(16)] + \
        [2 * 16 + i for i in range(8)] + [9 * 16 + i for i in range(3)]
    assert int(used) == 4


# ------------------------------------------------------------------------------- appends
@pytest.mark.parametrize("d,Hkv,dtype,strided", [(128, 8, "bf16", True), (64, 3, "fp16", False), (64, 1, "bf16", True)])
def test_append_16bit(d, Hkv, dtype, strided):
    T, n, page = 301, 40, 16
    g = torch.Generator().manual_seed(1)
    if strided:
        kv = torch.randn(T, 2, Hkv, d, generator=g).to(DT[dtype]).cuda()
        k, v = kv[:, 0], kv[:, 1]
    else:
        k, v = (torch.randn(T, Hkv, d, generator=g).to(DT[dtype]).cuda() for _ in "kv")
    slots = torch.randperm(n * page, generator=g)[:T].to(I32)
    slots[[3, 100]] = -1
    slots[7] = n * page
    kp, k_ok = guarded((n, page, Hkv, d), DT[dtype])
    vp, v_ok = guarded((n, page, Hkv, d), DT[dtype])
    want_k, want_v = kp.clone(), vp.clone()
    live = (slots >= 0) & (slots < n * page)
    want_k.view(-1, Hkv, d)[slots[live].cuda().long()] = k[live.cuda()]
    want_v.view(-1, Hkv, d)[slots[live].cuda().long()] = v[live.cuda()]
    fb.cache_append_paged(k, v, kp, vp, slots.cuda())
    torch.cuda.synchronize()
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v) and k_ok() and v_ok()
    fb.cache_append_paged(k[:0], v[:0], kp, vp, slots[:0].cuda())


APPENDS = [
    # page (0: contiguous), capacity, Hkv, d, type, lengths before, new tokens
    (64, 640, 8, 128, "bf16", [0, 63, 64, 65, 500], [1, 1, 1, 1, 1]),       # one decode step
    (16, 320, 3, 64, "fp16", [0, 5, 16, 30], [300, 0, 17, 2]),
    (0, 384, 2, 128, "bf16", [0, 100, 128, 383], [384, 200, 129, 1]),
    (0, 300, 1, 64, "bf16", [299, 0, 127], [1, 300, 2]),                    # a last block of 44 tokens
    (256, 1024, 2, 128, "fp16", [0, 255, 200], [1000, 300, 600]),           # more rows than registers hold
    (192, 576, 1, 128, "bf16", [10, 0], [500, 192]),
    (128, 256, 4, 64, "bf16", [100, 1], [28, 30]),
]


def append_case(case, seed=0, bump=None):
    page, cap, Hkv, d, dtype, olds, counts = case
    B, unit = len(olds), page or 128
    g = np.random.default_rng(seed + cap + d)
    per = -(-cap // unit)
    n = B * per + (3 if page else 0)
    place = g.permutation(n)[:B * per].reshape(B, per) if page else np.arange(B * per).reshape(B, per)
    codes = [ref.e4m3_encode(np.clip(g.standard_normal((n, unit, Hkv, d)) * 64, -448, 448)) for _ in "kv"]
    fac = [np.exp2(g.integers(-8, -4, (n, Hkv))) for _ in "kv"]
    T = sum(counts)
    x = torch.from_numpy(g.standard_normal((T, 2, Hkv, d)) * np.exp2(g.integers(-3, 4, (T, 2, Hkv, 1)))).to(DT[dtype])
    if bump:
        bump(x)
    x = x.cuda()
    cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
    lens = [o + c for o, c in zip(olds, counts)]
    return page, cap, unit, per, place, codes, fac, x, cu, lens


def run_append(case, seed=0, bump=None):
    """The caches after the append: ([k codes, v codes], [k factors, v factors]) by block, and the
    reference's."""
    olds = case[5]
    page, cap, unit, per, place, codes, fac, x, cu, lens = append_case(case, seed, bump)
    B, (n, _, Hkv, d) = len(olds), codes[0].shape
    pools, intact = [], []
    for c in codes:
        p, ok = guarded_bytes((n, unit, Hkv, d) if page else (B, cap, Hkv, d))
        if page:
            p.copy_(torch.from_numpy(c))
        else:  # the capacity may end inside the last block
            p.copy_(torch.from_numpy(c.reshape(B, per * 128, Hkv, d)[:, :cap].copy()))
        pools.append(p)
        intact.append(ok)
    dev_fac = []
    for f in fac:
        f = f if page else f.reshape(B, per, Hkv).transpose(0, 2, 1)
        dev_fac.append(torch.from_numpy(f.astype(np.float32).copy()).cuda())
    bt = torch.from_numpy(place.astype(np.int32)).cuda() if page else None
    fb.cache_append_fp8(x[:, 0], x[:, 1], *pools, *dev_fac, dev(cu), dev(olds), dev(lens),
                        max(l - o for l, o in zip(lens, olds)), block_table=bt)
    assert fb.fa_get_last_device_error(None) == fb.FA_OK
    assert intact[0]() and intact[1](), "write outside the caches"
    for i in range(2):
        ref.append_fp8(f64(x[:, i]), codes[i], fac[i], place, cu, olds, lens, unit)
    got_c, got_f = [], []
    for p, f in zip(pools, dev_fac):
        f = f.cpu().numpy().astype(np.float64)
        got_c.append(p.cpu().numpy())
        got_f.append(f if page else f.transpose(0, 2, 1).reshape(B * per, Hkv))
    if not page:
        codes = [c.reshape(B, per * 128, Hkv, d)[:, :cap] for c in codes]
    return got_c, got_f, codes, fac


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:5])))
def test_append_fp8(case):
    got_c, got_f, codes, fac = run_append(case)
    for i in range(2):
        assert np.array_equal(got_f[i], fac[i])
        assert np.array_equal(got_c[i], codes[i])


def test_append_fp8_extreme_values():
    """Zeros, the types' largest and smallest values, infinities and NaN; a block that grows by much."""
    def bump(x):
        x[0] = 0
        x[1] = torch.finfo(x.dtype).max
        x[2] = torch.finfo(x.dtype).smallest_normal
        x[3, :, :, ::2] = float("inf")
        x[4, :, :, 1::3] = float("nan")
        x[5] = -float("inf")
    for page in (0, 16, 64):
        for dtype in ("bf16", "fp16"):
            case = (page, 256, 2, 128, dtype, [0, 10, 20, 30, 40, 50], [1, 1, 1, 1, 1, 1])
            got_c, got_f, codes, fac = run_append(case, bump=bump)
            for i in range(2):
                assert np.array_equal(got_f[i], fac[i]) and np.array_equal(got_c[i], codes[i])
            case = (page, 256, 2, 64, dtype, [3], [40])
            got_c, got_f, codes, fac = run_append(case, bump=bump)
            for i in range(2):
                assert np.array_equal(got_f[i], fac[i]) and np.array_equal(got_c[i], codes[i])


def test_append_fp8_leaves_out_what_does_not_fit():
    """Bad lengths and pages write nothing and are reported; the other sequences are served."""
    Hkv, d, page, per = 2, 64, 16, 4
    x = torch.randn(40, 2, Hkv, d).to(torch.bfloat16).cuda()
    k = torch.zeros(20, page, Hkv, d, dtype=torch.uint8, device="cuda")
    v, kf, vf = k.clone(), torch.ones(20, Hkv, device="cuda"), torch.ones(20, Hkv, device="cuda")
    bt = torch.arange(20, dtype=I32, device="cuda").view(5, per)
    bt[3, 0] = 20  # outside the pool
    olds, lens = dev([0, 60, -1, 0, 4]), dev([8, 68, 7, 8, 12])  # fine, past the table, negative, bad page, fine
    fb.cache_append_fp8(x[:, 0], x[:, 1], k, v, kf, vf, dev([0, 8, 16, 24, 32, 40]), olds, lens, 8, block_table=bt)
    assert fb.fa_get_last_device_error(None) == fb.FA_ERR_INVALID_ARG
    touched = k.view(20, -1).ne(0).any(1).cpu()
    assert touched.nonzero().flatten().tolist() == [0, 16]
    # more new tokens than the bound, and tokens past the packed rows
    for olds, lens, cu, most in (([0], [9], [0, 40], 8), ([0], [9], [35, 44], 9), ([0], [9], [0, 8], 9),
                                 ([5], [4], [0, 8], 9)):
        before = k.clone()
        fb.cache_append_fp8(x[:, 0], x[:, 1], k, v, kf, vf, dev(cu), dev(olds), dev(lens), most, block_table=bt[1:2])
        assert fb.fa_get_last_device_error(None) == fb.FA_ERR_INVALID_ARG
        assert torch.equal(k, before)


# ------------------------------------------------------------------------------- together
@pytest.mark.parametrize("d,Hkv,Hq,dtype", [(128, 2, 8, "bf16"), (64, 4, 4, "fp16")])
def test_serving_loop(d, Hkv, Hq, dtype):
    """Prompts, then decode steps, over an 8-bit and a 16-bit paged cache side by side: tables, appends and
    attention on one stream, the last steps replayed from a captured graph."""
    B, page, width, pages = 4, 16, 12, 60
    g = torch.Generator().manual_seed(5)
    bt = torch.full((B, width), -1, dtype=I32, device="cuda")
    free = torch.randperm(pages, generator=g).to(I32).cuda()
    dt = DT[dtype]
    k8, v8 = (torch.full((pages, page, Hkv, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv")
    kf, vf = (torch.full((pages, Hkv), float("nan"), device="cuda") for _ in "kv")
    k16, v16 = (torch.full((pages, page, Hkv, d), float("nan"), dtype=dt, device="cuda") for _ in "kv")
    lens = torch.zeros(B, dtype=I32, device="cuda")
    hist = [torch.zeros(0, 2, Hkv, d) for _ in range(B)]
    taken = 0

    def step(x, news, total, q):
        nonlocal lens, taken
        slots, cu, after, used = fb.build_block_tables(lens, news, free[taken:].contiguous(), bt, page, pages, total)
        fb.cache_append_fp8(x[:, 0], x[:, 1], k8, v8, kf, vf, cu, lens, after, total, block_table=bt)
        fb.cache_append_paged(x[:, 0], x[:, 1], k16, v16, slots)
        o8, l8 = fb.attention_decode_fp8(q, k8, v8, kf, vf, after, causal=True, block_table=bt)
        o16, l16 = fb.attention_decode(q, k16, v16, after, causal=True, block_table=bt)
        return after, used, o8, l8, o16, l16

    for counts in ([37, 0, 5, 64], [1, 20, 1, 1], [1, 1, 1, 1], [2, 2, 2, 2], [1, 1, 1, 1]):
        total = sum(counts)
        x = torch.randn(total, 2, Hkv, d, generator=g).to(dt)
        q = torch.randn(B, 2, Hq, d, generator=g).to(dt).cuda()
        xd, news = x.cuda(), dev(counts)
        after, used, o8, l8, o16, l16 = step(xd, news, total, q)
        graph = torch.cuda.CUDAGraph()  # the same step again, captured and replayed: it writes the same rows
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            again = step(xd, news, total, q)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(again, (after, used, o8, l8, o16, l16)):
            assert torch.equal(a, b)
        at = 0
        for b, c in enumerate(counts):
            hist[b] = torch.cat([hist[b], x[at:at + c].float()])
            at += c
        lens, taken = after, taken + int(used)
        assert lens.tolist() == [len(h) for h in hist]
        n = max(len(h) for h in hist)
        k, v = (torch.stack([torch.cat([h[:, i], torch.zeros(n - len(h), Hkv, d)]) for h in hist]) for i in (0, 1))
        o_ref, l_ref = oracle.attn_decode(q, k, v, d ** -0.5, lens.tolist(), True)
        live = np.isfinite(l_ref)
        assert np.array_equal(live, np.isfinite(f64(l16))) and np.array_equal(live, np.isfinite(f64(l8)))
        # the 8-bit cache holds exactly what its codes say
        table = bt.cpu().numpy()
        want = ref.decode_fp8(f64(q), k8.cpu().numpy(), v8.cpu().numpy(), f64(kf), f64(vf), lens.tolist(), d ** -0.5,
                              True, page, table)
        check_decode(o8, l8, want, dt)
        # and its codes are the tokens to half a step of 3 mantissa bits (once more where a block grew)
        for b in range(B):
            for i in range(len(hist[b])):
                pg, r = table[b, i // page], i % page
                val = oracle.e4m3_decode(k8[pg, r].cpu().numpy()) * f64(kf[pg])[:, None]
                x0 = hist[b][i, 0].double().numpy()
                assert (np.abs(val - x0) <= 2.0 ** -4 * np.abs(x0) + 2.0 ** -8 * f64(kf[pg])[:, None]).all()
                if i > 40:
                    break
        assert np.abs(f64(o16) - o_ref)[np.moveaxis(live, 1, 2)].max() <= 1e-2 + 2.0 ** -7 * np.abs(o_ref).max()
    assert taken <= pages and fb.fa_get_last_device_error(None) == fb.FA_OK


@pytest.mark.parametrize("page", [0, 64])
def test_offsets_past_32_bits(page):
    """Appends to, and attention over, the end of a cache of more than 2^32 bytes of codes, against the
    same tokens in a small cache."""
    Hkv, d, new = 8, 128, 300
    N = (1 << 22) + 512  # 2^32 + 2^19 bytes of keys, and of values
    g = torch.Generator().manual_seed(48)
    x = torch.randn(new, 2, Hkv, d, generator=g).to(torch.bfloat16).cuda()

    def run(N, first):
        """Tokens first .. first + 299 of N, the earlier ones zeros."""
        shape = (1, N, Hkv, d) if not page else (N // page, page, Hkv, d)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in "kv")
        fshape = (1, Hkv, -(-N // 128)) if not page else (N // page, Hkv)
        kf, vf = (torch.ones(fshape, device="cuda") for _ in "kv")
        bt = None
        if page:  # a short sequence in the last pages
            bt = torch.arange(first // page, N // page, dtype=I32, device="cuda")[None]
            at = first % page
        else:
            at = first
        fb.cache_append_fp8(x[:, 0], x[:, 1], k, v, kf, vf, dev([0, new]), dev([at]), dev([at + new]), new, block_table=bt)
        outs = []
        for Hq in (8, 320):
            q = queries(1, 1, Hq, d, "bf16", 49, 20.0)  # scores far above the zeros' before
            outs.append(fb.attention_decode_fp8(q, k, v, kf, vf, dev([at + new]), block_table=bt))
        if page:
            k16 = torch.zeros((max(N // 2, 512) // page, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
            n = k16.shape[0] * page
            fb.cache_append_paged(x[:, 0], x[:, 1], k16, k16.clone(), torch.arange(n - new, n, dtype=I32, device="cuda"))
            assert torch.equal(k16.view(-1, Hkv, d)[-new:], x[:, 0])
        assert fb.fa_get_last_device_error(None) == fb.FA_OK
        return k.view(-1, Hkv, d)[first:first + new].clone(), v.view(-1, Hkv, d)[first:first + new].clone(), outs

    k0, v0, small = run(512, 192)
    k1, v1, large = run(N, N - 320)
    assert torch.equal(k0, k1) and torch.equal(v0, v1)
    for (o0, l0), (o1, l1) in zip(small, large):
        # the split differs, and its rounding: P to 2^-9 of itself, O to bf16
        assert (f64(l0) > 20).all() and np.abs(f64(l0) - f64(l1)).max() <= 2e-3
        assert np.abs(f64(o0) - f64(o1)).max() <= 2.0 ** -6 * np.abs(f64(o0)).max()
