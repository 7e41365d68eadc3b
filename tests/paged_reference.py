"""Plain references for the paged 4-bit KV cache, in binary64, and its nibble
layout read from the public header's description."""
import numpy as np

D = 128


def tables():
    """(flat token * 128 + dimension) of every (run, word, nibble) of a block's
    1024 bytes, for K and for V."""
    r, w, p = (a.ravel() for a in np.meshgrid(np.arange(32), np.arange(8), np.arange(8),
                                              indexing="ij"))
    gid, tig, j, e = r >> 2, r & 3, p & 3, p >> 2
    k = (gid + 8 * (j & 1)) * D + 16 * w + 2 * tig + e + 8 * (j >> 1)
    v = (2 * tig + e + 8 * (j >> 1)) * D + 16 * w + gid + 8 * (j & 1)
    return k, v


K_AT, V_AT = tables()


def unpack(codes, at):
    """(..., 1024) bytes of blocks -> (..., 16, 128) codes."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2048)
    out = np.empty_like(nib)
    out[..., at] = nib
    return out.reshape(*codes.shape[:-1], 16, D)


def pack(codes, at):
    nib = codes.reshape(*codes.shape[:-2], 2048)[..., at]
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).astype(np.uint8)


def rotate(x, pos, freq, layout, factor):
    """x (T, heads, 128) float16 -> binary64, its first 2 * len(freq) dimensions
    turned."""
    y = x.astype(np.float64)
    if freq is None:
        return y
    rot = 2 * len(freq)
    angle = np.asarray(pos, np.float64)[:, None] * freq[None, :]
    c, s = (np.cos(angle) * factor)[:, None, :], (np.sin(angle) * factor)[:, None, :]
    if layout == "half":
        a, b = y[..., :rot // 2].copy(), y[..., rot // 2:rot].copy()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., 0:rot:2].copy(), y[..., 1:rot:2].copy()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def rows(q_start, seqlen):
    """[(sequence, row, position)] of a well-formed batch."""
    out = []
    for b in range(len(seqlen)):
        n = q_start[b + 1] - q_start[b]
        out += [(b, q_start[b] + i, int(seqlen[b]) - int(n) + i) for i in range(n)]
    return out


def attention(Q, kc, vc, sc, q_start, seqlen, table, scale):
    """(out (T, Hq, 128) binary64 with NaN in rows of no sequence, the FP32 and
    FP16 error allowance of every output).

    Allowance, per row and KV head: half an FP16 step of the output (2^-11
    relative, 2^-25 absolute below the normal range); the weights p s enter the
    products as FP16 (2^-11 relative, 2^-25 absolute), times codes centred on 8:
    2^-11 * 8 max s + n 2^-22 for n tokens and a largest weight of at least 1; FP32
    scores and sums, the allowance of the unpaged attention: 5e-5 max |v^|."""
    T, Hq, _ = Q.shape
    pages, Hkv, page = sc.shape[:3]
    g, cap = Hq // Hkv, table.shape[1] * page
    out = np.full((T, Hq, D), np.nan)
    tol = np.zeros((T, Hq, 1))
    for b in range(len(seqlen)):
        n = int(q_start[b + 1] - q_start[b])
        if n <= 0:
            continue
        L = max(0, min(int(seqlen[b]), cap))
        held = [(t, int(table[b, t // page])) for t in range(L)]
        held = [(t, p) for t, p in held if 0 <= p < pages]
        t_at = np.array([t for t, _ in held], np.int64)
        p_at = np.array([p for _, p in held], np.int64)
        for h in range(Hkv):
            mine = sorted(set(p_at.tolist()))
            s = np.zeros((len(held), 4))
            qk = np.zeros((len(held), D))
            qv = np.zeros((len(held), D))
            for p in mine:
                at = p_at == p
                slot = t_at[at] % page
                qk[at] = unpack(kc[p, h], K_AT).reshape(page, D)[slot]
                qv[at] = unpack(vc[p, h], V_AT).reshape(page, D)[slot]
                s[at] = sc[p, h].astype(np.float64)[slot]
            k = qk * s[:, 0:1] + s[:, 1:2]
            v = qv * s[:, 2:3] + s[:, 3:4]
            for i in range(n):
                row = q_start[b] + i
                see = t_at <= int(seqlen[b]) - n + i
                m = int(see.sum())
                hs = slice(h * g, (h + 1) * g)
                if m == 0:
                    out[row, hs] = 0.0
                    continue
                z = Q[row, hs].astype(np.float64) @ k[see].T * scale
                z = np.exp(z - z.max(-1, keepdims=True))
                out[row, hs] = (z @ v[see]) / z.sum(-1, keepdims=True)
                tol[row, hs] = (2.0 ** -8 * s[see, 2].max() + m * 2.0 ** -22 + 2.0 ** -25
                                + 5e-5 * np.abs(v[see]).max())
    return out, tol + 2.0 ** -11 * np.abs(out)
