"""The torch helpers on a stream that is not the current one: what they allocate is that stream's own
memory, so neither stream's pending work can touch the other's."""
import contextlib

import numpy as np
import pytest
import torch

from exact_tiled_attention_36_b200 import binding as fb

I32 = torch.int32


def test_cpu_tensors_are_refused_with_a_stream_too():
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    k, f = torch.zeros(1, 128, 2, 64, dtype=torch.uint8), torch.ones(1, 2, 1)
    i = torch.zeros(2, dtype=I32)
    for call in (lambda: fb.attention_decode_fp8(q, k, k, f, f, stream=0), lambda: fb.attention_fwd(q, q, q, stream=7),
                 lambda: fb.build_block_tables(i, i, i, i.view(2, 1), 16, 2, 0, stream=0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


class FakeDevice:
    """What _on_stream asks of torch.cuda, on the CPU: it keeps the order of events."""

    class Stream:
        def __init__(self, handle, device):
            self.cuda_stream, self.device = handle, device

    def __init__(self, device):
        self.log, self.device, self.current = [], device, self.Stream(1, device)

    def ExternalStream(self, handle, device):
        return self.Stream(handle, device)

    def default_stream(self, device):
        return self.Stream(0, device)

    def current_stream(self, device):
        return self.current

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before


@pytest.mark.parametrize("handle", [0, 1, 9])
@pytest.mark.parametrize("as_stream", [False, True])
def test_calls_allocate_on_their_stream(handle, as_stream, monkeypatch):
    device = torch.device("cuda", 0)
    fake = FakeDevice(device)
    monkeypatch.setattr(torch, "cuda", fake)

    class Result:
        def record_stream(self, s):
            fake.log.append((self, s.cuda_stream))

    mine, new = Result(), Result()

    def fn(x, out=None, lse=None):
        assert fake.current.cuda_stream == handle and x == 5
        return out, new

    res = fb._on_stream(fake.Stream(handle, device) if as_stream else handle, device, fn, 5, out=mine, lse=None)
    assert res == (mine, new) and fake.current.cuda_stream == 1
    assert fake.log == ([] if handle == 1 else [(new, 1)])  # on the current stream itself there is nothing to order
    with pytest.raises(ValueError, match="cuda:1"):
        fb._on_stream(fake.Stream(3, torch.device("cuda", 1)), device, fn, 5)


@pytest.fixture
def side():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    fb.lib()
    yield torch.cuda.Stream()
    torch.cuda.synchronize()
    assert fb.fa_get_last_device_error(None) == fb.FA_OK


def caches(B, N, Hkv, d, seed):
    g = np.random.default_rng(seed)
    k, v = (torch.from_numpy((g.integers(0x18, 0x58, (B, N, Hkv, d)) | g.integers(0, 2, (B, N, Hkv, d)) << 7)
                             .astype(np.uint8)).cuda() for _ in "kv")
    kf, vf = (torch.from_numpy(np.exp2(g.integers(-4, 0, (B, Hkv, -(-N // 128)))).astype(np.float32)).cuda() for _ in "kv")
    return k, v, kf, vf


def pending(n):
    """Some milliseconds of work on the current stream."""
    x = torch.ones(4096, 4096, device="cuda")
    for _ in range(n):
        x = x @ x * 0
    return x


@pytest.mark.gpu
def test_workspaces_of_two_streams_are_apart(side, monkeypatch):
    """A call on the current stream drops its workspace while it still runs; one on another stream right after
    it must not get the same memory, nor its outputs any that the first stream still reads."""
    B, N, Hkv, Hq, d = 4, 1024, 2, 8, 128
    k, v, kf, vf = caches(B, N, Hkv, d, 1)
    q = torch.randn(B, 1, Hq, d, device="cuda").to(torch.bfloat16)
    k16 = torch.randn(B, N, Hkv, d, device="cuda").to(torch.bfloat16)
    ws = {}
    at = {"fa_decode_fp8": 8, "fa_decode": 6}
    real = {n: getattr(fb.lib(), n) for n in at}

    class Spy:
        def __getattr__(self, name):
            if name not in at:
                return getattr(fb_lib, name)
            return lambda *a: (ws.setdefault(name, []).append(a[at[name]]), real[name](*a))[1]

    fb_lib = fb.lib()
    monkeypatch.setattr(fb, "lib", lambda: Spy())
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    busy = pending(20)
    outs = []
    for call in (lambda **s: fb.attention_decode_fp8(q, k, v, kf, vf, **s), lambda **s: fb.attention_decode(q, k16, k16, **s)):
        scrap = torch.zeros_like(q), torch.zeros(B, Hq, 1, device="cuda")
        taken = [x.data_ptr() for x in scrap]
        del scrap  # free for the current stream, whose zeros are not written yet
        outs += [call(), call(stream=side), call(stream=side.cuda_stream), call()]
        for o, lse in outs[-3:-1]:
            assert o.data_ptr() not in taken and lse.data_ptr() not in taken
    for name, p in ws.items():
        assert len(p) == 4 and not {p[0], p[3]} & {p[1], p[2]}, name
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, outs[i // 4 * 4][0]) and torch.equal(lse, outs[i // 4 * 4][1])
    del busy


@pytest.mark.gpu
def test_dropped_results_wait_for_the_stream_that_read_them(side):
    k, v, kf, vf = caches(2, 256, 2, 128, 2)
    q = torch.randn(2, 1, 8, 128, device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    o, lse = fb.attention_decode_fp8(q, k, v, kf, vf, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    busy = pending(20)
    seen = o.clone()  # behind the pending work
    at = o.data_ptr()
    want = None
    del o, lse
    o2, _ = fb.attention_decode_fp8(q * 2, k, v, kf, vf, stream=side)
    assert o2.data_ptr() != at
    torch.cuda.synchronize()
    want, _ = fb.attention_decode_fp8(q, k, v, kf, vf)
    assert torch.equal(seen, want)
    del busy


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [8, 80])
def test_two_streams_at_once(side, Hq):
    """Calls that outlast the host's part of them, on both streams in turn."""
    B, N, Hkv, d = 16, 8192, 2, 128
    data = [caches(B, N, Hkv, d, s) for s in (3, 4)]
    q = torch.randn(B, 1, Hq, d, device="cuda").to(torch.bfloat16)
    want = []
    for x in data:
        want.append(fb.attention_decode_fp8(q, *x))
        torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    busy = pending(5)
    outs = []
    for _ in range(12):
        outs.append((0, fb.attention_decode_fp8(q, *data[0])))
        outs.append((1, fb.attention_decode_fp8(q, *data[1], stream=side)))
    torch.cuda.synchronize()
    for i, (o, lse) in outs:
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    del busy


@pytest.mark.gpu
def test_other_helpers_on_another_stream(side):
    """Forward, backward, packed forward and backward, FP8 and block tables: a call with `stream` gives what one
    on the current stream gives, with the current stream kept busy."""
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(1, 320, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2, 4))
    cu = torch.tensor([0, 100, 320], device="cuda")  # int64: converted within the call
    codes = [torch.randint(0, 100, (1, 320, h, 128), generator=g).to(torch.uint8).cuda() for h in (4, 2, 2)]
    fac = [torch.ones(1, h, 3, device="cuda") for h in (4, 2, 2)]
    free, table = torch.arange(40, dtype=I32, device="cuda"), torch.zeros(3, 8, dtype=I32, device="cuda")
    old, new = (torch.tensor(x, dtype=I32, device="cuda") for x in ([0, 3, 20], [30, 1, 0]))

    def calls(**s):
        o, lse = fb.attention_fwd(q, k, v, causal=True, **s)
        o2, l2 = fb.attention_varlen_fwd(q[0], k[0], v[0], cu, cu, 220, 220, causal=True, **s)
        return [o, lse, *fb.attention_bwd(q, k, v, o, lse, do, causal=True, **s), o2, l2,
                *fb.attention_varlen_bwd(q[0], k[0], v[0], o2, l2, do[0], cu, cu, 220, 220, causal=True, **s),
                *fb.attention_fwd_fp8(*codes, *fac, **s), *fb.build_block_tables(old, new, free, table, 16, 40, 31, **s)]

    want = calls()
    torch.cuda.synchronize()
    busy = pending(20)
    got = calls(stream=side)
    side.synchronize()
    names = "o lse dq dk dv o2 l2 dq2 dk2 dv2 o8 l8 slots cu lens used".split()
    for name, a, b in zip(names, want, got, strict=True):
        if name.startswith("dq"):  # its sums are taken in any order
            assert (a.float() - b.float()).norm() <= 2.0 ** -7 * a.float().norm(), name
        else:
            assert torch.equal(a, b), name
    del busy


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [8, 80])
def test_captured_on_a_forked_stream(side, Hq):
    """A call with `stream` inside a capture, on a stream that joined it: replayed over new contents, twice,
    with eager calls on both streams between the replays."""
    B, N, Hkv, d = 3, 700, 2, 128
    data = [caches(B, N, Hkv, d, s) for s in (6, 7)]
    q = torch.randn(B, 1, Hq, d, device="cuda").to(torch.bfloat16)
    want = [fb.attention_decode_fp8(q, *x) for x in data]
    lens, news = torch.tensor([5, 0], dtype=I32, device="cuda"), torch.tensor([20, 9], dtype=I32, device="cuda")
    free, table = torch.arange(9, dtype=I32, device="cuda"), torch.zeros(2, 4, dtype=I32, device="cuda")
    tables = [x.clone() for x in fb.build_block_tables(lens, news, free, table, 16, 9, 29)]
    now = [x.clone() for x in data[0]]
    here, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=here):
        first = fb.attention_decode_fp8(q, *now)
        side.wait_stream(here)
        forked = fb.attention_decode_fp8(q, *now, stream=side)
        built = fb.build_block_tables(lens, news, free, table, 16, 9, 29, stream=side)
        beside = fb.attention_decode_fp8(q, *now)
        here.wait_stream(side)
        fb.attention_decode_fp8(q, *now, stream=side)  # its results dropped within the capture
        here.wait_stream(side)
        last = fb.attention_decode_fp8(q, *now)
    for i in (1, 0, 1):
        for x, y in zip(now, data[i]):
            x.copy_(y)
        side.wait_stream(torch.cuda.current_stream())
        eager = fb.attention_decode_fp8(q, *data[1 - i]), fb.attention_decode_fp8(q, *data[1 - i], stream=side)
        torch.cuda.synchronize()
        for x in (first, forked, beside, last):
            for t in x:
                t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for x in (first, forked, beside, last):
            assert torch.equal(x[0], want[i][0]) and torch.equal(x[1], want[i][1])
        for x in eager:
            assert torch.equal(x[0], want[1 - i][0]) and torch.equal(x[1], want[1 - i][1])
        assert all(torch.equal(a, b) for a, b in zip(built, tables))
