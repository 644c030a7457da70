"""Position rotation and the 4-bit cache (oracle; test infrastructure).

``rotate`` follows the formula in fp32, one rounding per product and sum; ``encode`` and ``decode``
are the 4-bit format's definition: the nearest scale to max |y| / 6, the nearest code to y / s,
quotients in fp32, ties to the even code, by searching the values that can be held."""
import numpy as np

PAGE, BLOCK = 16, 16
CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                   for e in range(16) for m in range(8)])


def rotary_table(max_position, dim, base=10000.0):
    angle = np.arange(max_position)[:, None] * base ** (-2.0 * np.arange(dim // 2) / dim)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def rotate(x, table_rows, interleaved=False, exact=False):
    """``x`` [tokens, heads, hd] (bf16 values) turned by ``table_rows`` [tokens, rotary]; fp32, or
    float64 if ``exact``; not yet rounded to bf16."""
    t = np.float64 if exact else np.float32
    x = np.array(x, t)
    half = table_rows.shape[1] // 2
    cos, sin = (table_rows[:, None, a:a + half].astype(t) for a in (0, half))
    one = np.arange(half)
    i, j = (2 * one, 2 * one + 1) if interleaved else (one, one + half)
    a, b = x[..., i].copy(), x[..., j].copy()
    x[..., i] = (a * cos).astype(t) - (b * sin).astype(t)
    x[..., j] = (b * cos).astype(t) + (a * sin).astype(t)
    return x


def nearest(x, grid):
    """Index of the nearest of ascending ``grid`` values, the even one of two as near."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


def encode(x, layer_scale=1.0):
    """Codes [..., hd] and scale bytes [..., hd / 16] of values [..., hd]."""
    f32 = np.float32
    with np.errstate(all="ignore"):
        x = np.asarray(x, f32)
        y = (np.where(np.isnan(x), f32(0), x) / f32(layer_scale)).astype(f32)
        y = y.reshape(*y.shape[:-1], -1, BLOCK)
        top = np.minimum(np.abs(y).max(-1) / f32(6.0), f32(448.0))
        sb = nearest(top.astype(np.float64), SCALES[:127])
        s = SCALES[sb][..., None].astype(f32)
        t = np.where(s > 0, np.abs(y) / np.where(s > 0, s, f32(1)), f32(0))
        code = nearest(np.minimum(t, f32(6.0)).astype(np.float64), CODES)
    code = code + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def decode(code, sb, layer_scale=1.0):
    """float64 values of codes [..., hd] and scale bytes [..., hd / 16]."""
    c = np.asarray(code).reshape(*code.shape[:-1], -1, BLOCK)
    v = np.where(c >= 8, -1.0, 1.0) * CODES[c & 7] * SCALES[np.asarray(sb) & 127][..., None]
    return v.reshape(code.shape) * layer_scale


def pack(code, sb, values):
    """Bytes [pages, nkv, 9 hd] of codes [pages, 16, nkv, hd] and scales [pages, 16, nkv, hd / 16]."""
    b = (code[..., ::2] | code[..., 1::2] << 4).transpose(0, 2, 1, 3)
    s = sb.transpose(0, 2, 3, 1) if values else sb.transpose(0, 2, 1, 3)
    flat = lambda a: a.reshape(a.shape[0], a.shape[1], -1)
    return np.concatenate([flat(b), flat(s)], 2)


def unpack(cache, hd, values):
    """Codes [pages, 16, nkv, hd] and scale bytes [pages, 16, nkv, hd / 16] of a cache's bytes."""
    pages, nkv, _ = cache.shape
    b = cache[..., :8 * hd].reshape(pages, nkv, PAGE, hd // 2).transpose(0, 2, 1, 3)
    s = cache[..., 8 * hd:]
    s = s.reshape(pages, nkv, hd // BLOCK, PAGE).transpose(0, 3, 1, 2) if values else \
        s.reshape(pages, nkv, PAGE, hd // BLOCK).transpose(0, 2, 1, 3)
    return np.stack([b & 15, b >> 4], -1).reshape(pages, PAGE, nkv, hd), s
