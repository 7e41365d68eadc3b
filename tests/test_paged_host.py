"""Host side of the paged 4-bit KV cache: the index arithmetic that the kernels
share (compiled here as plain C++), refusals of the entry points, and the
frequency helper."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import w4a8_quantized_gemm_02_b200 as qoq
import paged_reference as ref

CSRC = os.path.join(os.path.dirname(qoq.__file__), "csrc")
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    return qoq.lib()


@pytest.fixture(scope="module")
def idx(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged")
    src = d / "idx.cpp"
    src.write_text("""
#include "qoq_paged.h"
using namespace qoq;
extern "C" {
void c_rows(const int* q, int b, int T, int* first, int* n) {
  const RowRange r = rows_of(q, b, T);
  *first = r.first;
  *n = r.n;
}
int c_len(int s, int c) { return clamp_len(s, c); }
long long c_pos(int s, int n, int i) { return position_of(s, n, i); }
int c_vis(long long p, int len) { return visible(p, len); }
int c_blk(const int* t, int blk, int ppb, int pages, int Hkv, int hk) {
  return pool_block(t, blk, ppb, pages, Hkv, hk);
}
int c_slot(int f, int b, int g, int tile) { return slot_base(f, b, g, tile); }
}
""")
    so = d / "idx.so"
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(src)])
    lib = ctypes.CDLL(str(so))
    lib.c_pos.restype = ctypes.c_longlong
    lib.c_vis.argtypes = [ctypes.c_longlong, ctypes.c_int]
    return lib


def _ints(a):
    return (ctypes.c_int * len(a))(*a)


def test_row_ranges_stay_inside(idx):
    T = 10
    rng = np.random.default_rng(0)
    wild = [-2 ** 31, -1, 0, 3, 10, 11, 2 ** 31 - 1]
    for a in wild:
        for e in wild:
            f, n = ctypes.c_int(), ctypes.c_int()
            idx.c_rows(_ints([a, e]), 0, T, ctypes.byref(f), ctypes.byref(n))
            if 0 <= a <= e <= T:
                assert (f.value, n.value) == (a, e - a)
            else:
                assert n.value == 0
    assert [idx.c_len(s, 7) for s in (-5, 0, 6, 7, 8, 2 ** 31 - 1)] == [0, 0, 6, 7, 7, 7]
    assert idx.c_pos(-2 ** 31, 2 ** 31 - 1, 0) == -2 ** 31 - (2 ** 31 - 1)
    for _ in range(200):
        p, n = int(rng.integers(-5, 30)), int(rng.integers(0, 20))
        assert idx.c_vis(p, n) == sum(1 for t in range(n) if t <= p)


def test_page_numbers_outside_the_pool_give_no_block(idx):
    table = [3, -1, 4, 0, 2 ** 31 - 1, -2 ** 31]
    pages, Hkv, ppb = 4, 3, 2
    for blk in range(2 * len(table)):
        pid = table[blk // ppb]
        for hk in range(Hkv):
            got = idx.c_blk(_ints(table), blk, ppb, pages, Hkv, hk)
            if 0 <= pid < pages:
                assert got == (pid * Hkv + hk) * ppb + blk % ppb < pages * Hkv * ppb
            else:
                assert got == -1


def test_tile_slots_hold_every_sequence(idx):
    rng = np.random.default_rng(1)
    for _ in range(300):
        g, tile = int(rng.integers(1, 70)), int(rng.choice([64, 128, 256]))
        q = rng.integers(0, 3 * tile, int(rng.integers(1, 9)))
        start = np.concatenate([[0], np.cumsum(q)])
        base = [idx.c_slot(int(s), b, g, tile) for b, s in enumerate(start)]
        for b, n in enumerate(q):
            assert base[b + 1] - base[b] >= -(-int(n) * g // tile)
        assert base[-1] <= int(start[-1]) * g // tile + len(q)


def test_prompt_splits_fit_the_grid_and_the_workspace():
    """The rule by which the prompt kernel splits slots, over random batches: units
    of equal length `chunk`, at least the batch's work over `target`.  No batch has
    more units than target + pairs, nor more units of split slots (the ones that
    leave partial results) than 2 target; every unit has work."""
    rng = np.random.default_rng(2)
    target, least = 148, 8
    for _ in range(400):
        B, Hkv = int(rng.integers(1, 200)), int(rng.integers(1, 65))
        n = rng.integers(0, int(10 ** rng.uniform(0, 4.2)) + 1, B)
        if rng.random() < 0.3:
            n[rng.integers(0, B)] = 100000
        chunk = max(least, -(-int(n.sum()) * Hkv // target))
        splits = np.where(n <= chunk, 1, -(-n // chunk))
        assert splits.sum() * Hkv <= target + B * Hkv
        assert (splits[splits > 1].sum() * Hkv) <= 2 * target
        for m, k in zip(n[splits > 1], splits[splits > 1]):
            per = -(-int(m) // int(k))
            assert per <= chunk and (k - 1) * per < m and (k - 1) * chunk < m


def test_decode_runs_cover_every_pair_once():
    """The decode kernel's runs, over random batches: with every pair's length in
    blocks and a constant in front of it, a CTA's run is cut at the pairs' ends;
    every block is in one piece, and a pair's unfinished pieces are the last of its
    first CTA and the first of the next ones, where the merge looks for them."""
    rng = np.random.default_rng(3)
    cost = 12
    for grid in (1, 7, 592):
        for _ in range(60):
            B, Hkv = int(rng.integers(1, 40)), int(rng.integers(1, 9))
            n = rng.integers(0, int(10 ** rng.uniform(0, 3)) + 1, B)
            w = np.maximum(n, 1) + cost
            total, mean = int(w.sum()) * Hkv, -(-int(w.sum()) // len(w))
            run = max(-(-total // grid), min(cost + 16, mean))
            assert run * grid >= total
            places, at = set(), 0
            for b, m in enumerate(w):
                for h in range(Hkv):
                    lo, hi = at, at + int(m)
                    at = hi
                    pieces = []
                    for k in range(lo // run, (hi - 1) // run + 1):
                        assert k < grid
                        f, t = max(lo, k * run) - lo, min(hi, (k + 1) * run) - lo
                        c0, c1 = max(0, f - cost), t - cost
                        if c1 > 0:
                            pieces.append((k, c0, c1, c0 == 0 and t == hi - lo))
                    first, last = pieces[0][0], (hi - 1) // run
                    assert [p[0] for p in pieces] == list(range(first, last + 1))
                    assert pieces[0][1] == 0 and pieces[-1][2] == m - cost
                    assert all(p[2] == q[1] for p, q in zip(pieces, pieces[1:]))
                    assert pieces[0][3] == (first == last)
                    for k, c0, _, whole in pieces:
                        if not whole:
                            place = 2 * k + (c0 == 0)
                            assert place not in places and place < 2 * grid
                            assert place == (2 * first + 1 if k == first else 2 * k)
                            places.add(place)


def test_nibble_tables_are_permutations():
    for at in (ref.K_AT, ref.V_AT):
        assert sorted(at.tolist()) == list(range(2048))
    codes = np.random.default_rng(0).integers(0, 16, (3, 16, 128)).astype(np.uint8)
    for at in (ref.K_AT, ref.V_AT):
        assert np.array_equal(ref.unpack(ref.pack(codes, at), at), codes)


def _append(L, qkv=FAKE, ld=6 * 128, T=4, Hq=4, Hkv=1, d=128, start=FAKE, lens=FAKE, B=2,
            table=FAKE, width=4, pages=8, page=16, freq=FAKE, rot=128, inter=0, q=FAKE, kc=FAKE,
            vc=FAKE, sc=FAKE, kh=None, vh=None):
    return L.qoq_kv4_paged_append(qkv, ld, T, Hq, Hkv, d, start, lens, B, table, width, pages,
                                  page, freq, rot, inter, 1.0, q, kc, vc, sc, kh, vh, None)


def test_append_refusals(L):
    INV, UNS = qoq.QOQ_ERR_INVALID_ARG, qoq.QOQ_ERR_UNSUPPORTED
    for name in ("qkv", "start", "lens", "table", "q", "kc", "vc", "sc"):
        assert _append(L, **{name: None}) == INV, name
    for name in ("qkv", "q", "kc", "vc", "sc"):
        assert _append(L, **{name: ODD}) == INV, name
    for name in ("start", "lens", "table"):
        assert _append(L, **{name: ctypes.c_void_p(0x10002)}) == INV, name
    assert _append(L, freq=None) == INV
    assert _append(L, freq=ctypes.c_void_p(0x10004)) == INV
    assert _append(L, kh=FAKE) == INV and _append(L, vh=FAKE) == INV
    assert _append(L, kh=ODD, vh=FAKE) == INV
    for bad in (dict(T=-1), dict(B=-1), dict(width=0), dict(pages=0), dict(page=0), dict(Hq=0),
                dict(Hkv=0), dict(rot=-16), dict(rot=144), dict(inter=2), dict(ld=6 * 128 - 8),
                dict(ld=6 * 128 + 4)):
        assert _append(L, **bad) == INV, bad
    for bad in (dict(d=64), dict(page=24), dict(rot=20), dict(width=1 << 28),
                dict(pages=1 << 30, page=64), dict(Hq=65536, ld=1 << 24)):
        assert _append(L, **bad) == UNS, bad
    # nothing to do: fine without a device
    assert _append(L, T=0) == qoq.QOQ_OK
    assert _append(L, B=0) == qoq.QOQ_OK


def _attend(L, Q=FAKE, ldq=4 * 128, T=4, Hq=4, Hkv=1, d=128, kc=FAKE, vc=FAKE, sc=FAKE, start=FAKE,
            lens=FAKE, B=2, table=FAKE, width=64, pages=8, page=16, max_q=1, scale=0.1, out=FAKE,
            ws=FAKE, ws_bytes=1 << 40):
    return L.qoq_kv4_paged_attention(Q, ldq, T, Hq, Hkv, d, kc, vc, sc, start, lens, B, table,
                                     width, pages, page, max_q, scale, out, ws, ws_bytes, None)


def test_attention_refusals(L):
    INV, UNS = qoq.QOQ_ERR_INVALID_ARG, qoq.QOQ_ERR_UNSUPPORTED
    for name in ("Q", "start", "lens", "table", "out", "kc", "vc", "sc"):
        assert _attend(L, **{name: None}) == INV, name
    for name in ("Q", "out", "kc", "vc", "sc"):
        assert _attend(L, **{name: ODD}) == INV, name
    for name in ("start", "lens", "table"):
        assert _attend(L, **{name: ctypes.c_void_p(0x10001)}) == INV, name
    for bad in (dict(T=-1), dict(B=-2), dict(width=0), dict(pages=-1), dict(page=0), dict(Hq=0),
                dict(Hkv=3), dict(max_q=0), dict(ldq=4 * 128 - 8), dict(ldq=4 * 128 + 4),
                dict(scale=math.inf), dict(scale=math.nan)):
        assert _attend(L, **bad) == INV, bad
    for bad in (dict(d=256), dict(page=40), dict(width=1 << 27, page=64), dict(B=1 << 23)):
        assert _attend(L, **bad) == UNS, bad
    # a workspace that is missing, misaligned or one byte short
    need = L.qoq_kv4_paged_attention_workspace_bytes(4, 4, 1, 128, 2, 64, 16, 1)
    assert need > 0
    for bad in (dict(ws=None), dict(ws=ODD), dict(ws_bytes=need - 1)):
        assert _attend(L, **bad) == qoq.QOQ_ERR_WORKSPACE, bad
    assert _attend(L, T=0) == qoq.QOQ_OK
    assert _attend(L, B=0, ws=None, ws_bytes=0) == qoq.QOQ_OK


def test_attention_refuses_what_its_block_counts_cannot_hold(L):
    """A table may name a page many times: more blocks than the pool has."""
    UNS = qoq.QOQ_ERR_UNSUPPORTED
    for bad in (dict(width=1 << 22, page=256, Hq=32, Hkv=32, ldq=32 * 128),   # 2^31 blocks and more
                dict(width=1 << 22, page=256, B=1 << 14),                     # 2^40 in the batch
                dict(width=(1 << 27) - 1)):                                   # tokens up to 2^31 - 16
        assert _attend(L, **bad) == UNS, bad
    assert _append(L, width=(1 << 27) - 1) == UNS
    f = L.qoq_kv4_paged_attention_workspace_bytes
    assert f(4, 32, 32, 128, 2, 1 << 22, 256, 1) == 0
    assert f(4, 4, 1, 128, 2, 1 << 22, 256, 1) > 0


def test_workspace_is_bounded_and_zero_for_nothing(L):
    f = L.qoq_kv4_paged_attention_workspace_bytes
    assert f(0, 4, 1, 128, 2, 64, 16, 1) == 0
    assert f(4, 4, 1, 128, 0, 64, 16, 1) == 0
    assert f(4, 4, 3, 128, 2, 64, 16, 1) == 0       # an invalid shape
    for B in (1, 64, 4096):
        # partial results of the splits: some thousand units of at most 16 rows
        assert f(B, 32, 8, 128, B, 8192, 16, 1) <= (16 * 148 + 8 * B) * 8 * 528 + (8 * B + 64) * 8
    assert f(4, 4, 1, 128, 2, 64, 16, 1) == f(4, 4, 1, 128, 2, 64, 16, 1)


def test_paged_bytes():
    assert qoq.kv4_paged_bytes(3, 2, 48) == (3 * 2 * 3 * 1024, 3 * 2 * 3 * 1024, 3 * 2 * 48 * 8)
    for bad in ((0, 1, 16), (1, 0, 16), (1, 1, 0)):
        with pytest.raises(qoq.QoQError) as e:
            qoq.kv4_paged_bytes(*bad)
        assert e.value.status == qoq.QOQ_ERR_INVALID_ARG
    with pytest.raises(qoq.QoQError):
        qoq.kv4_paged_bytes(1, 1, 20)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    cache = tuple(torch.zeros(s, dtype=t) for s, t in
                  (((2, 1, 1, 1024), torch.uint8), ((2, 1, 1, 1024), torch.uint8),
                   ((2, 1, 16, 4), torch.float16)))
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        qoq.kv4_paged_append(torch.zeros(1, 512).half(), cache, i, i[:1], t, 2)
    with pytest.raises(ValueError):
        qoq.kv4_paged_attention(torch.zeros(1, 2, 128).half(), cache, i, i[:1], t)
    with pytest.raises(ValueError):
        qoq.kv4_paged_append(torch.zeros(1, 512).half(), cache, i, i[:1], t, 2,
                             rope_layout="neox")


def test_rope_frequencies():
    torch = pytest.importorskip("torch")
    f, a = qoq.rope_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and a == 1.0
    assert np.allclose(f.numpy(), 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-15)
    g, _ = qoq.rope_frequencies(64, 10000.0, {"type": "linear", "factor": 4}, device="cpu")
    assert torch.equal(g, f / 4)
    g, _ = qoq.rope_frequencies(64, 10000.0, {"type": "ntk", "factor": 4}, device="cpu")
    assert g[0] == 1.0 and math.isclose(float(g[-1]), float(f[-1]) / 4, rel_tol=1e-12)
    # llama3: fast pairs kept, slow ones divided, in between monotone
    g, a = qoq.rope_frequencies(128, 500000.0, {
        "type": "llama3", "factor": 8, "low_freq_factor": 1, "high_freq_factor": 4,
        "original_length": 8192}, device="cpu")
    f, _ = qoq.rope_frequencies(128, 500000.0, device="cpu")
    ratio = (f / g).numpy()
    assert a == 1.0 and (np.diff(ratio) >= -1e-12).all()
    turns = 8192 * f.numpy() / (2 * np.pi)
    assert np.allclose(ratio[turns >= 4], 1.0) and np.allclose(ratio[turns <= 1], 8.0)
    # yarn: the same ends, and the factor on the values
    g, a = qoq.rope_frequencies(128, 500000.0, {"type": "yarn", "factor": 16,
                                                "original_length": 8192}, device="cpu")
    ratio = (f / g).numpy()
    assert math.isclose(a, 0.1 * math.log(16) + 1) and ratio[0] == 1.0
    assert math.isclose(ratio[-1], 16.0) and (np.diff(ratio) >= -1e-9).all()
    for bad in (dict(rot=20), dict(rot=0), dict(rot=144), dict(base=1.0),
                dict(scaling={"type": "other"}), dict(scaling={"type": "linear"}),
                dict(scaling={"type": "linear", "factor": 0}),
                dict(scaling={"type": "linear", "factor": 2, "low_freq_factor": 1}),
                dict(scaling={"type": "llama3", "factor": 2, "low_freq_factor": 4,
                              "high_freq_factor": 4, "original_length": 8})):
        with pytest.raises(ValueError):
            qoq.rope_frequencies(**{"device": "cpu", **bad})
