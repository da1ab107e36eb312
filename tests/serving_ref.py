"""Plain forms of the serving operators, for their tests: numpy, on the host, written from the
definitions in include/w4a8_serve.h.  What is defined to the bit is computed to the bit."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
STEPS = np.array([b if b < 16 else (16 + b % 16) * 2 ** (b // 16 - 1) for b in range(256)], np.float64)


def norm(h, w, eps, offset):
    """y of the rounded h (fp32 [M, K]), to the bit: the mean and the root in 64 bits."""
    f = (1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(-1, keepdims=True) + np.float64(np.float32(eps)))).astype(np.float32)
    return (h * f) * (w + np.float32(offset))


def assign(table, lens, free, count, new, page, M):
    """pages_assign on copies: table, cu, lens, positions, slots, count, missing."""
    table, pages, most = table.copy(), len(free), table.shape[1] * page
    count, cu, missing, out_lens = min(max(int(count), 0), pages), [0], 0, []
    positions, slots = np.zeros(M, np.int32), np.full(M, -1, np.int64)
    for b in range(len(lens)):
        old = min(max(int(lens[b]), 0), most)
        n = min(max(int(new[b]), 0), M - cu[-1])
        have, want = -(-old // page), -(-(old + n) // page)
        for e in range(have, want):
            if e >= table.shape[1]:
                missing += 1
            elif count > 0:
                count -= 1
                table[b, e] = free[count]
            else:
                table[b, e] = -1
                missing += 1
        for i in range(n):
            pos = old + i
            positions[cu[-1] + i] = pos
            p = int(table[b, pos // page]) if pos < most else -1
            slots[cu[-1] + i] = p * page + pos % page if 0 <= p < pages else -1
        cu.append(cu[-1] + n)
        out_lens.append(min(old + n, most))
    return table, np.array(cu), np.array(out_lens), positions, slots, count, missing


def release(table, lens, free, count, keep, page):
    """pages_release on copies: free, lens, count."""
    free, pages, most = free.copy(), len(free), table.shape[1] * page
    count, out = min(max(int(count), 0), pages), [0] * len(lens)
    for b in reversed(range(len(lens))):
        old = min(max(int(lens[b]), 0), most)
        out[b] = min(max(int(keep[b]), 0), old)
        for e in reversed(range(-(-out[b] // page), -(-old // page))):
            if 0 <= table[b, e] < pages and count < pages:
                free[count] = table[b, e]
                count += 1
    return free, np.array(out), count


def _nearest(x, points):
    """Index of the nearest of ascending points, ties to the even index, the last one beyond; x fp32 or fp64."""
    x = x.astype(np.float64)
    hi = np.clip(np.searchsorted(points, x), 1, len(points) - 1)
    up, down = points[hi] - x, x - points[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise4(x, unit):
    """Codes [..., D / 2] and scale bytes [..., D / 16] of fp32 x [..., H, D], unit [H], to the bit."""
    u = unit.astype(np.float32)[:, None]
    g = x.astype(np.float32).reshape(*x.shape[:-1], -1, 16)
    with np.errstate(over="ignore", invalid="ignore"):
        t = np.abs(g).max(-1) / (np.float32(6) * u)
        byte = np.maximum(_nearest(np.minimum(t, np.float32(1e9)), STEPS), 1)
        s = STEPS[byte].astype(np.float32) * u
        y = g / s[..., None]
    code = _nearest(np.minimum(np.abs(y), np.float32(100)), GRID) + 8 * np.signbit(y)
    code = code.reshape(*x.shape[:-1], -1, 2)
    return (code[..., 0] + 16 * code[..., 1]).astype(np.uint8), byte.astype(np.uint8)


def values4(codes, scales, unit):
    """The values that codes [..., H, P, D / 2] and scales [..., H, P, D / 16] stand for, in 64 bits."""
    grid = np.concatenate([GRID, -GRID])
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    s = STEPS[scales] * unit.astype(np.float64)[:, None, None]
    return (grid[c].reshape(*scales.shape, 16) * s[..., None]).reshape(c.shape)
