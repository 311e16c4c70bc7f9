"""Plain references of the 4-bit operands and the expert plan, written from the definitions in include/pnq.h, in 64 bits,
element by element of the layouts (numpy; shares nothing with the package)."""
import numpy as np

NVFP4, MXFP4 = 1004, 1006
GROUP = {NVFP4: 16, MXFP4: 32}
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m * 2.0 ** -9) if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])[:127]


def nearest_even_place(v, table):
    """Place in the rising table of the value nearest to each v >= 0, ties to the even place, past the end the last."""
    v = np.minimum(v, table[-1])
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    down, up = v - table[lo], table[hi] - v
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def scale_values(words, kind):
    words = np.asarray(words).astype(np.int64)
    if kind == NVFP4:
        return np.where(words == 127, np.nan, E4M3[np.minimum(words, 126)])
    return np.where(words == 255, np.nan, np.ldexp(1.0, words - 127))


def quantize(x, kind, g):
    """(codes [rows][K], scale words [rows][K / group]) of float32 x."""
    rows, K = x.shape
    with np.errstate(all="ignore"):
        r = np.float32(1.0) / np.float32(g)
        y = (x.astype(np.float32) * r).astype(np.float32).reshape(rows, -1, GROUP[kind])
        top = np.abs(y).max(-1)
        finite = np.isfinite(y).all(-1)
        amax = np.where(finite, top, 0.0).astype(np.float32)
        if kind == NVFP4:
            raw = (amax / np.float32(6.0)).astype(np.float32).astype(np.float64)
            words = nearest_even_place(raw, E4M3)
            words = np.where(finite, words, 127)
        else:
            e = np.where(amax > 0, np.frexp(amax.astype(np.float64))[1] - 1 - 2, -127)
            words = np.where(finite, np.maximum(e, -127) + 127, 255)
        s = scale_values(words, kind)[..., None]
        empty = ~finite[..., None] | (s == 0)
        t = np.where(empty, 0.0, np.abs(y.astype(np.float64)) / np.where(empty, 1.0, s))
        codes = nearest_even_place(t, GRID) + 8 * np.signbit(y)
        codes = np.where(empty, 0, codes)
    return codes.reshape(rows, K).astype(np.uint8), words.astype(np.uint8)


def values(codes, words, kind):
    """e2m1 * scale in 64 bits (no global multiplier)."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(scale_values(words, kind), GROUP[kind], axis=1)


def tiled_place(r, group, groups):
    """Byte of the word of tiled row r, group `group` of `groups`."""
    chunks = -(-groups // 4)
    return ((r // 128) * chunks + group // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + group % 4


def scales_of(tiled, rows, groups):
    """Scale words [len(rows)][groups] of tiled rows `rows`."""
    rows = np.asarray(rows)
    return tiled[tiled_place(rows[:, None], np.arange(groups)[None, :], groups)]


def matrix_rows(rows, matrices):
    """Tiled rows of the rows of every matrix."""
    pad = -(-rows // 128) * 128
    return np.concatenate([m * pad + np.arange(rows) for m in range(matrices)]) if rows else np.zeros(0, np.int64)


def codes_of(packed, K):
    """Codes [rows][K] of packed rows [rows][pitch]."""
    return np.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1)[:, :K]


def plan(ids, experts):
    """offsets, block_start, order, position, scale_row of ids [tokens][slots]."""
    flat = np.asarray(ids).reshape(-1)
    n = flat.size
    order, position, scale_row = [np.full(n, -1, np.int64) for _ in range(3)]
    offsets, blocks = [0], [0]
    for e in range(experts):
        mine = np.nonzero(flat == e)[0]
        at = offsets[-1] + np.arange(mine.size)
        order[at] = mine
        position[mine] = at
        scale_row[at] = 128 * blocks[-1] + np.arange(mine.size)
        offsets.append(offsets[-1] + mine.size)
        blocks.append(blocks[-1] + -(-mine.size // 128))
    return np.array(offsets), np.array(blocks), order, position, scale_row
