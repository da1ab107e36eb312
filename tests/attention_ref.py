"""Plain 64-bit forms of the attention operators, for their tests: numpy, on the host, written
from the definitions in include/w4a8_attn.h."""
import numpy as np


def rope(x, positions, inv_freq, weight, eps, offset, interleaved, attn_factor):
    """Head norm and rotation of x [M, H, D] in 64 bits, and the magnitude its error scales with."""
    x = x.astype(np.float64)
    d, r = x.shape[-1], 2 * len(inv_freq)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (weight.astype(np.float64) + offset)
    i = np.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    t = positions.astype(np.float64)[:, None, None] * inv_freq
    c, s = np.cos(t) * attn_factor, np.sin(t) * attn_factor
    y, size = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(attn_factor)
    return y, size


def append(x, codes, scales, page_table, cu, lens, num_pages):
    """In-place append of x [M, Hkv, D] fp32 to codes and scales, bit for bit as defined."""
    P = codes.shape[2]
    f127 = np.float32(127)
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        length = max(0, min(int(lens[b]), page_table.shape[1] * P))
        pos = max(0, length - n)
        while n > 0 and pos < length:
            slot, page = pos % P, int(page_table[b, pos // P])
            take = min(P - slot, length - pos)
            if 0 <= page < num_pages:
                for h in range(codes.shape[1]):
                    row = cu[b] + pos - (length - n)
                    v = x[row:row + take, h].astype(np.float32)
                    top = np.abs(v).max()
                    old = scales[page, h]
                    s = top / f127
                    if slot and old > 0:
                        s, room = old, f127 * old
                        with np.errstate(over="ignore"):
                            while top > room:
                                room, s = room * np.float32(2), s * np.float32(2)
                        codes[page, h, :slot] = np.rint(codes[page, h, :slot].astype(np.float64) * (np.float64(old) / s)).astype(np.int8)
                    with np.errstate(divide="ignore", invalid="ignore"):
                        q = np.clip(np.rint(v / s), -127, 127) if s > 0 else np.zeros_like(v)
                    codes[page, h, slot:slot + take] = q.astype(np.int8)
                    scales[page, h] = s
            pos += take


def attention(q, kc, ks, vc, vs, page_table, cu, lens, scale, causal, window):
    """o [M, Hq, D] in 64 bits, NaN in rows of no sequence, and per row and column
    (A = sum p |v|, T = the largest p * scale times sum |codes|, delta = the largest |scale| sum |q k|)."""
    M, hq, d = q.shape
    P, hkv = kc.shape[2], kc.shape[1]
    g = hq // hkv
    q = q.astype(np.float64)
    o = np.full((M, hq, d), np.nan)
    A, T, delta = np.zeros((M, hq, d)), np.zeros((M, hq, d)), np.zeros((M, hq, 1))
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        length = max(0, min(int(lens[b]), page_table.shape[1] * P))
        if n == 0:
            continue
        t = np.arange(length)
        page = page_table[b, t // P].astype(np.int64)
        ok = (page >= 0) & (page < kc.shape[0])
        at = np.where(ok, page, 0)
        for h in range(hkv):
            k = kc[at, h, t % P].astype(np.float64) * ks[at, h].astype(np.float64)[:, None]
            vcode = vc[at, h, t % P].astype(np.float64)
            sv = vs[at, h].astype(np.float64)
            for i in range(n):
                pos = length - n + i
                see = ok.copy()
                if causal:
                    see &= t <= pos
                    if window:
                        see &= t > pos - window
                m = int(cu[b]) + i
                heads = slice(h * g, (h + 1) * g)
                if not see.any():
                    o[m, heads] = 0
                    continue
                z = q[m, heads] @ k[see].T * scale
                delta[m, heads, 0] = (np.abs(q[m, heads]) @ np.abs(k[see]).T).max(-1) * abs(scale)
                p = np.exp(z - z.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                w = p * sv[see]
                o[m, heads] = w @ vcode[see]
                A[m, heads] = w @ np.abs(vcode[see])
                T[m, heads] = w.max(-1, keepdims=True) * np.abs(vcode[see]).sum(0)
    return o, A, T, delta
