"""Prompt operators on a given stream: whose memory has to outlive the call.

On the CPU with stand-ins for tensors and streams (nothing is launched); on a
GPU with inputs that are freed, and their memory written, while the stream is
still busy with other work."""
import threading

import pytest
import torch

import confidence_gated_kv_gb300 as ck
from confidence_gated_kv_gb300 import binding, prompt


class Stream:
    cuda_stream = 1 << 20


class External(Stream):
    pass


class Tensor:
    """What the bindings ask of a contiguous CUDA tensor."""
    is_cuda, requires_grad, device = True, False, torch.device("cuda", 0)

    def __init__(self, *shape, dtype=torch.float16):
        self.shape, self.dtype, self.used_on = torch.Size(shape), dtype, []

    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def __len__(self):
        return self.shape[0]

    def record_stream(self, s):
        self.used_on.append(s)


@pytest.fixture
def calls(monkeypatch):
    """Names of the library calls, none of which is made."""
    names = []
    for module in (binding, prompt):
        monkeypatch.setattr(module, "call_on", lambda index, fn, name, args, stream: names.append(name))
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    prompt._bind()
    return names


def every_call(stream):
    """Each call with a stream, and the tensors that the work reads or writes."""
    i32 = lambda *s: Tensor(*s, dtype=torch.int32)  # noqa: E731
    q, k, v, out, cu, cuk = Tensor(9, 4, 64), Tensor(9, 2, 64), Tensor(9, 2, 64), Tensor(9, 4, 64), i32(2), i32(2)
    lse = Tensor(9, 4, dtype=torch.float32)
    ck.prompt_attention(q, k, v, cu, cuk, out=out, lse=lse, stream=stream)
    yield "attention", [q, k, v, out, cu, cuk, lse]
    rotary = ck.Rotary(64, device="cpu")
    rotary.turns, rotary.device_index = Tensor(32, dtype=torch.int64), 0
    q, k, qo, ko, pos = Tensor(9, 4, 64), Tensor(9, 2, 64), Tensor(9, 4, 64), Tensor(9, 2, 64), i32(9)
    qw, kw = Tensor(64), Tensor(64)
    ck.qk_rotary(q, k, pos, rotary, qw, kw, q_out=qo, k_out=ko, stream=stream)
    yield "rotary", [q, k, qo, ko, pos, qw, kw, rotary.turns]
    c = ck.Cache.__new__(ck.Cache)
    c._h, c._dev_index, c.B, c.Hkv, c.d, c.workspace = None, 0, 1, 2, 64, Tensor(1)
    k, v = Tensor(9, 2, 64), Tensor(9, 2, 64)
    c.prefill_begin([9], stream=stream)
    yield "begin", [c.workspace]
    c.workspace = Tensor(1)
    c.prefill_layer(0, k, v, stream=stream)
    yield "layer", [k, v, c.workspace]
    c.workspace = Tensor(1)
    o = dict(k=Tensor(9, 2, 64), v=Tensor(9, 2, 64), positions=i32(9), cu_seqlens=i32(2))
    c.read_layer(0, out=o, stream=stream)
    yield "read", [*o.values(), c.workspace]


def test_tensors_are_held_for_a_given_stream(calls):
    s = Stream()
    for name, tensors in every_call(s):
        for i, t in enumerate(tensors):
            assert t.used_on == [s], (name, i)
    assert len(calls) == 5


@pytest.mark.parametrize("stream", [None, External(), 1 << 20])
def test_nothing_is_told_of_other_streams(calls, stream):
    # the current stream needs nothing; one that torch does not own may be gone when the tensors are freed
    for name, tensors in every_call(stream):
        assert all(t.used_on == [] for t in tensors), name


def test_a_raw_handle_is_a_stream_of_the_tensors_device(monkeypatch):
    # new outputs on another device than the current one belong to a stream of theirs
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: made.append((handle, device)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: binding._same)
    with binding.allocating_on(1 << 20, 3):
        pass
    assert made == [(1 << 20, 3)]
    monkeypatch.setattr(prompt, "allocating_on", lambda stream, index: made.append((stream, index)) or binding._same)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: None)
    t = Tensor(4, 2, 64)
    t.get_device = lambda: 5
    prompt._bind()
    prompt._like(t, 1 << 20)
    assert made[1] == (1 << 20, 5)


@pytest.mark.gpu
def test_inputs_freed_behind_the_call():
    n, Hq, Hkv, d = 700, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    make = lambda h: torch.randn((n, h, d), generator=g, device="cuda").half()  # noqa: E731
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    keep = make(Hq), make(Hkv), make(Hkv)
    rotary = ck.Rotary(d)
    cfg = ck.make_config(L=1, Hq=Hq, Hkv=Hkv, d=d, V=1000, B=1, cap=1024, W=64, P=1, n_high=[1024], n_low=[1024])
    cache = ck.Cache(cfg)

    def run(q, k, v, stream):
        """out of every operator, all on `stream`"""
        a = ck.prompt_attention(q, k, v, cu, stream=stream)
        b = ck.qk_rotary(q, k, pos, rotary, stream=stream)
        cache.prefill_begin([n], stream=stream)
        cache.prefill_layer(0, k, v, stream=stream)
        r = cache.read_layer(0, stream=stream)
        return a, *b, r["k"], r["v"]

    want = run(*keep, None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        q, k, v = (x.clone() for x in keep)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)                     # about 10 ms before the operators start
        got = run(q, k, v, s)
        del q, k, v
        new = [torch.full_like(x, 100.0) for x in keep]       # the freed memory, were it handed out
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        del new


@pytest.mark.gpu
def test_raw_handles():
    q, k, v = (torch.randn(50, h, 64, device="cuda").half() for h in (4, 2, 2))
    cu = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = ck.prompt_attention(q, k, v, cu, return_lse=True)
    for handle in (s.cuda_stream, 0):
        got = ck.prompt_attention(q, k, v, cu, return_lse=True, stream=handle)
        a = ck.qk_rotary(q, k, None, None, torch.ones(64, device="cuda").half(), stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(a[1], k)


@pytest.mark.gpu
def test_two_caches_in_two_threads():
    # the library's per-device records are shared by all threads
    lens = [300, 70, 1500]
    g = torch.Generator(device="cuda").manual_seed(3)
    data, caches, want = [], [], []
    for d, H in ((64, 3), (128, 2)):
        cfg = ck.make_config(L=2, Hq=H, Hkv=H, d=d, V=1000, B=3, cap=1500, W=32, P=1, n_high=[1500] * 2, n_low=[1500] * 2)
        data.append([torch.randn((sum(lens), H, d), generator=g, device="cuda").half() for _ in range(4)])
        caches.append(ck.Cache(cfg))

    def work(i, stream, rounds):
        c, x = caches[i], data[i]
        for _ in range(rounds):
            c.prefill_begin(lens, stream=stream)
            for l in range(2):
                c.prefill_layer(l, x[2 * l], x[2 * l + 1], stream=stream)
            got[i] = [c.read_layer(l, stream=stream) for l in range(2)]
        stream.synchronize()

    got = [None, None]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i, streams[i], 30)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    want, got = got, [None, None]
    for i in range(2):                                  # the same, one after the other
        work(i, streams[i], 1)
        for a, b in zip(want[i], got[i]):
            assert all(torch.equal(a[key], b[key]) for key in a)
        assert caches[i].stats()["device_status"] == 0
