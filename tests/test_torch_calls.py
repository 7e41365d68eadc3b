"""The extension that makes the paged cache's and the adapters' calls from torch
tensors: it takes what the kernels take, leaves everything else to the Python
functions, and both ways give the same bits."""
import types

import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_02_b200 as qoq  # noqa: E402

DEV = "cuda"
D = 128
Hq, Hkv, PAGE, PAGES, B, T = 4, 2, 32, 9, 2, 7


def _batch(dev):
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).half().to(dev)  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    n = PAGES * Hkv * (PAGE // 16) * 1024
    codes = [torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8).to(dev)
             .view(PAGES, Hkv, PAGE // 16, 1024) for _ in range(2)]
    scales = torch.rand(PAGES, Hkv, PAGE, 4, generator=g).half().to(dev)
    return dict(qkv=rnd(T, (Hq + 2 * Hkv) * D), Q=rnd(T, Hq, D), cache=(*codes, scales),
                q_start=i32([0, 5, 7]), seqlen=i32([70, 33]),
                table=i32([[0, 3, 5, 1], [7, 8, 2, 4]]),
                freq=torch.logspace(0, -4, 64, dtype=torch.float64).to(dev))


def _adapters(dev):
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g).half().to(dev)  # noqa: E731
    return dict(Y=rnd(T, 256), X=rnd(T, 384), A=rnd(3, 8, 384), Bm=rnd(3, 256, 8),
                ids=torch.tensor([0, 2, 2, -1, 1, 0, 3], dtype=torch.int32, device=dev),
                scaling=torch.tensor([0.5, 1.0, 2.0], device=dev))


def _append_args(s, **o):
    a = dict(qkv=s["qkv"], cache=s["cache"], q_start=s["q_start"], seqlen=s["seqlen"],
             table=s["table"], Hq=Hq, freq=s["freq"], inter=0, factor=1.0, q_out=None, values=None)
    a.update(o)
    return tuple(a.values())


def _attend_args(s, **o):
    a = dict(Q=s["Q"], cache=s["cache"], q_start=s["q_start"], seqlen=s["seqlen"],
             table=s["table"], max_q=5, scale=0.1, out=None, ws=None)
    a.update(o)
    return tuple(a.values())


def _lora_args(s, **o):
    a = dict(Y=s["Y"], X=s["X"], A=s["A"], Bm=s["Bm"], ids=s["ids"], scaling=s["scaling"], out=None,
             ws=None)
    a.update(o)
    return tuple(a.values())


def test_host_tensors_and_wrong_counts():
    c = qoq._load_calls()
    s, a = _batch("cpu"), _adapters("cpu")
    assert c.paged_append(*_append_args(s)) is None
    assert c.paged_attention(*_attend_args(s)) is None
    assert c.lora_add(*_lora_args(a)) is None
    assert c.paged_append(*[None] * 11) is None
    assert c.paged_attention(*[3] * 9) is None
    assert c.lora_add(*["x"] * 8) is None
    for f in (c.paged_append, c.paged_attention, c.lora_add):
        with pytest.raises(TypeError):
            f(1, 2)


def _wrong(t):
    """Forms of a tensor that a kernel does not take."""
    yield None
    yield t.cpu()
    yield t.double() if t.dtype != torch.float64 else t.float()
    yield t[:-1]
    if t.dim() > 1:
        yield torch.empty(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=DEV)[..., ::2]
        yield t.flatten()


@pytest.mark.gpu
def test_wrong_tensors_are_left_to_python():
    c = qoq._load_calls()
    s, a = _batch(DEV), _adapters(DEV)
    before = [t.clone() for t in s["cache"]]
    for name in ("q_start", "seqlen", "table", "freq"):
        for bad in _wrong(s[name]):
            if name == "freq" and (bad is None or (bad.is_cuda and bad.dtype == torch.float64)):
                continue                          # (no rotation; 63 frequencies: refused below)
            assert c.paged_append(*_append_args(s, **{name: bad})) is None, name
            if name != "freq":
                assert c.paged_attention(*_attend_args(s, **{name: bad})) is None, name
    for i in range(3):
        for bad in _wrong(s["cache"][i]):
            if bad is None or i < 2 or bad.shape[1:] != s["cache"][2].shape[1:] or not bad.is_cuda:
                cache = tuple(bad if j == i else t for j, t in enumerate(s["cache"]))
                assert c.paged_append(*_append_args(s, cache=cache)) is None, i
                assert c.paged_attention(*_attend_args(s, cache=cache)) is None, i
    for bad in (dict(Hq=3), dict(Hq=1 << 40), dict(Hq=-1), dict(Hq=4.0), dict(factor=1),
                dict(freq=s["freq"][:60]), dict(cache=s["cache"][:2]), dict(inter=2),
                dict(qkv=s["qkv"][:, 4:]), dict(qkv=s["qkv"].float()), dict(qkv=s["qkv"][0]),
                dict(values=(s["Q"],)), dict(values=(s["Q"], s["Q"])),
                dict(q_out=torch.empty(T, Hq + 1, D, dtype=torch.float16, device=DEV))):
        assert c.paged_append(*_append_args(s, **bad)) is None, bad
    for bad in (dict(max_q=0), dict(max_q=-2), dict(max_q=1.0), dict(scale=float("inf")), dict(scale=1),
                dict(Q=s["Q"][..., :64]), dict(Q=s["Q"].float()), dict(Q=s["Q"][:, :3]),
                dict(out=s["Q"][1:]), dict(ws=torch.empty(16, dtype=torch.uint8, device=DEV)),
                dict(ws=torch.empty(1 << 24, dtype=torch.uint8))):
        assert c.paged_attention(*_attend_args(s, **bad)) is None, bad
    for name in a:
        for bad in _wrong(a[name]):
            assert c.lora_add(*_lora_args(a, **{name: bad})) is None, name
    assert all(torch.equal(t, u) for t, u in zip(s["cache"], before))


@pytest.mark.gpu
def test_both_ways_give_the_same_bits(monkeypatch):
    c = qoq._load_calls()
    quick = []

    def watch(name):
        def call(*args):
            out = getattr(c, name)(*args)
            quick.append(out is not None)
            return out
        return call
    names = ("paged_append", "paged_attention", "lora_add")
    watched = types.SimpleNamespace(**{n: watch(n) for n in names})
    never = types.SimpleNamespace(**{n: lambda *args: None for n in names})
    results = []
    for way in (watched, never):
        monkeypatch.setattr(qoq, "_calls", way)
        s, a = _batch(DEV), _adapters(DEV)
        wide = torch.zeros(T, Hq + 1, D, dtype=torch.float16, device=DEV)
        wide[:, :Hq] = s["Q"]
        values = tuple(torch.zeros(T, Hkv, D, dtype=torch.float16, device=DEV) for _ in range(2))
        mine = torch.zeros(T, Hq, D, dtype=torch.float16, device=DEV)
        q = qoq.kv4_paged_append(s["qkv"], s["cache"], s["q_start"], s["seqlen"], s["table"], Hq,
                                 inv_freq=s["freq"], values=values)
        qoq.kv4_paged_append(s["qkv"], s["cache"], s["q_start"], s["seqlen"], s["table"], Hq,
                             inv_freq=s["freq"], rope_layout="interleaved", rope_factor=1.25,
                             q_out=mine)
        o = [qoq.kv4_paged_attention(s["Q"], s["cache"], s["q_start"], s["seqlen"], s["table"]),
             qoq.kv4_paged_attention(wide[:, :Hq], s["cache"], s["q_start"], s["seqlen"], s["table"],
                                     max_q=5, out=torch.empty_like(s["Q"]))]
        same = qoq.lora_add(a["Y"], a["X"], a["A"], a["Bm"], a["ids"], a["scaling"])
        into = a["Y"].clone()
        assert qoq.lora_add(into, a["X"], a["A"], a["Bm"], a["ids"], a["scaling"], out=into) is into
        results.append([q, mine, *values, *s["cache"], *o, same, into])
    assert quick == [True] * 6
    for x, y in zip(*results):
        assert x.dtype == y.dtype and torch.equal(x, y)
    assert torch.equal(results[0][-1], results[0][-2])


@pytest.mark.gpu
def test_quick_calls_follow_the_current_stream():
    s = _batch(DEV)
    side = torch.cuda.Stream()
    want = qoq.kv4_paged_attention(s["Q"], s["cache"], s["q_start"], s["seqlen"], s["table"])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        Q = torch.zeros_like(s["Q"])
        torch.cuda._sleep(2000000)       # (the queries come late: a call on another stream misses them)
        Q.copy_(s["Q"])
        got = qoq.kv4_paged_attention(Q, s["cache"], s["q_start"], s["seqlen"], s["table"])
    side.synchronize()
    assert torch.equal(got, want)
