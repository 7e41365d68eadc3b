"""Attention over the paged 4-bit KV cache in binary64 on the GPU, for long sequences and
values of any size, with an allowance that follows the values.

Allowance of an output o = sum p v / sum p, with v = s (c - 8) + (m + 8 s) and the averages
A = sum p |s (c - 8)| / sum p, F = sum p |m + 8 s| / sum p and V = sum p |v| / sum p over the n
tokens that the row sees:

* its own rounding to FP16: 2^-11 |o|, at least 2^-25;
* the weights p s as FP16 numbers: 2^-11 A;
* sums in FP32, n / 16 additions in a row at the most (16 tokens an MMA, and no thread adds
  more than one token in 8 to its sums), each rounded or cut to 2^-23 of the sum so far:
  n / 16 2^-23 (A + F + |o|), the last for the denominator;
* scores in FP32: eight roundings (of the scale, its products, the two terms, the reference)
  of terms of at most G = scale log2(e) max (15 s_K + |m_K|) sum |q| together, 2^-24 each,
  and 2^-22 for the exponential: d = 8 2^-24 (G + 1), of every weight, in numerator and
  denominator: 2 d V.

Queries are counted as exact: a caller takes such as the kernels' formats hold (0 and +-a).
"""
import math

import numpy as np
import torch

import paged_reference as ref

D = 128


def pool_of(rng, total, page, Hkv, k_scale, k_offset, v_scale, v_offset, codes=(0, 16)):
    """A pool of random codes (in V those of even dimensions in the upper half of the range
    given, of odd ones in the lower half, so that errors of the weights do not average out)
    with the scales given per token: functions of (sequence, tokens) -> array.  Returns
    (k_codes, v_codes, scales, table)."""
    need = [-(-t // page) for t in total]
    pages = sum(need) + 1
    order = rng.permutation(pages)
    table = np.full((len(total), max(need)), -1, np.int32)
    shape = (pages, Hkv, page // 16, 16, D)
    kc = ref.pack(rng.integers(0, 16, shape).astype(np.uint8), ref.K_AT)
    mid = (codes[0] + codes[1]) // 2
    low = rng.integers(codes[0], mid, shape)
    v = np.where(np.arange(D) % 2 == 0, low + (codes[1] - mid), low).astype(np.uint8)
    vc = ref.pack(v, ref.V_AT)
    sc = np.zeros((pages, Hkv, page, 4), np.float16)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        t = n * page
        for i, f in enumerate((k_scale, k_offset, v_scale, v_offset)):
            sc[table[b, :n], :, :, i] = np.broadcast_to(
                np.asarray(f(b, t), np.float64), (t,)).reshape(n, 1, page)
    return kc, vc, sc, table


def attention(Q, kc, vc, sc, q_start, seqlen, table, scale):
    """(out, allowance), (T, Hq, 128) binary64 on the GPU; rows of no sequence NaN."""
    dev = "cuda"
    T, Hq, _ = Q.shape
    pages, Hkv, page = sc.shape[:3]
    g = Hq // Hkv
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=dev)
    tol = torch.zeros(T, Hq, D, dtype=torch.float64, device=dev)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    for b in range(len(seqlen)):
        lo, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        L = min(int(seqlen[b]), table.shape[1] * page)
        if n <= 0:
            continue
        if L <= 0:
            out[lo:lo + n] = 0.0
            continue
        mine = table[b, :-(-L // page)]
        for h in range(Hkv):
            s = to(sc[mine, h].reshape(-1, 4)[:L].astype(np.float64))
            ck = to(ref.unpack(kc[mine, h], ref.K_AT).reshape(-1, D)[:L]).double()
            cv = to(ref.unpack(vc[mine, h], ref.V_AT).reshape(-1, D)[:L]).double()
            k = ck * s[:, 0:1] + s[:, 1:2]
            v = cv * s[:, 2:3] + s[:, 3:4]
            q = to(Q[lo:lo + n, h * g:(h + 1) * g].astype(np.float64)).reshape(n * g, D)
            pos = int(seqlen[b]) - n + torch.arange(n, device=dev).repeat_interleave(g)
            sees = torch.arange(L, device=dev) <= pos.view(-1, 1)
            z = (q @ k.T * scale).masked_fill(~sees, -math.inf)
            top = z.amax(-1, keepdim=True)
            p = torch.where(sees, (z - torch.where(top.isinf(), 0.0, top)).exp(), 0.0)
            den = p.sum(-1, keepdim=True)
            p = p / torch.where(den == 0, 1.0, den)
            o = p @ v
            A = p @ ((cv - 8) * s[:, 2:3]).abs()
            F = p @ (s[:, 3:4] + 8 * s[:, 2:3]).abs()
            V = p @ v.abs()
            count = sees.sum(-1, keepdim=True).double()
            G = scale * math.log2(math.e) * (15 * s[:, 0] + s[:, 1].abs()).max() * \
                q.abs().sum(-1, keepdim=True)
            e = (2.0 ** -11 * o.abs() + 2.0 ** -25 + 2.0 ** -11 * A +
                 count / 16 * 2.0 ** -23 * (A + F + o.abs()) + 2 * 8 * 2.0 ** -24 * (G + 1) * V)
            sl = (slice(lo, lo + n), slice(h * g, (h + 1) * g))
            out[sl], tol[sl] = o.view(n, g, D), e.view(n, g, D)
    return out, tol
