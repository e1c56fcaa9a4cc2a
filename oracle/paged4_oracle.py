"""Plain CPU implementation of the 4-bit paged cache's format (include/paged4.h):
the quantizer of 32 channels of a token, and where a block of 16 tokens has its
codes, scales and zeros.

Test infrastructure: numpy, place by place from the format's description,
nothing shared with the library's kernels.
"""
import numpy as np

D, G, BLOCK = 128, 32, 2560


def quantise(x):
    """Rows x [..., 128] (fp32 values of the cache's type): codes uint8 [..., 128], scales and zeros fp16 [..., 4]."""
    x = np.asarray(x, np.float32)
    y = x.reshape(*x.shape[:-1], 4, G)
    with np.errstate(all="ignore"):
        fine = np.isfinite(y).all(-1)
        lo, hi = (np.clip(np.where(fine, f(-1), 0), -65504, 65504).astype(np.float32) for f in (y.min, y.max))
        s = ((hi - lo) / np.float32(15)).astype(np.float16)
        z = lo.astype(np.float16)
        s = np.where(z.astype(np.float64) + 15 * s.astype(np.float64) > 65504, np.nextafter(s, np.float16(0)), s)
        sf, zf = s.astype(np.float32)[..., None], z.astype(np.float32)[..., None]
        c = np.rint((y - zf) / np.where(sf > 0, sf, np.float32(1)))
        c = np.where((sf > 0) & fine[..., None], np.clip(np.nan_to_num(c), 0, 15), 0)
    z = np.where(fine, z, np.float16("nan")).astype(np.float16)
    return c.astype(np.uint8).reshape(x.shape), s, z


def held(x):
    """What rows read back as, in 64 bits (NaN where a group is not finite)."""
    c, s, z = quantise(x)
    return (c.reshape(*c.shape[:-1], 4, G) * s.astype(np.float64)[..., None] + z.astype(np.float64)[..., None]).reshape(c.shape)


def key_place(token, channel):
    """Byte and shift of a key code in its block."""
    group, c, i = channel // G, channel % G // 8, channel % 8
    nibble = i // 2 + 4 * (i % 2)
    return 64 * token + 16 * c + 4 * group + nibble // 2, 4 * (nibble % 2)


def value_place(token, channel):
    half, m, high, g = channel // 64, channel // 16 % 4, channel // 8 % 2, channel % 8
    c, e, odd = token % 8 // 2, token // 8, token % 2
    return 1280 + 512 * half + 64 * g + 16 * c + 4 * m + 2 * odd + e, 4 * high


def key_scale_place(token, group):
    """Bytes of a scale and its zero."""
    return 1024 + 16 * token + 2 * group, 1024 + 16 * token + 8 + 2 * group


def value_scale_place(token, group):
    c, e, odd = token % 8 // 2, token // 8, token % 2
    at = 2304 + 32 * c + 16 * e + 4 * group + 2 * odd
    return at, at + 128


def _places():
    kc = np.array([[key_place(t, d) for d in range(D)] for t in range(16)])
    vc = np.array([[value_place(t, d) for d in range(D)] for t in range(16)])
    ks = np.array([[key_scale_place(t, j) for j in range(4)] for t in range(16)])
    vs = np.array([[value_scale_place(t, j) for j in range(4)] for t in range(16)])
    return kc, ks, vc, vs


PLACES = _places()


def write(block, token, k=None, v=None):
    """Put a token's key and value rows [128] into a block [2560] uint8, nothing else of it touched."""
    for row, codes, scales in ((k, PLACES[0], PLACES[1]), (v, PLACES[2], PLACES[3])):
        if row is None:
            continue
        c, s, z = quantise(row)
        for d in range(D):
            at, shift = codes[token, d]
            block[at] = (block[at] & (0xF0 if shift == 0 else 0x0F)) | int(c[d]) << shift
        for j in range(4):
            for x, at in zip((s[j], z[j]), scales[token, j]):
                block[at:at + 2] = np.frombuffer(np.float16(x).tobytes(), np.uint8)


def parts(blocks, values):
    """Blocks [..., 2560] -> codes [..., 16, 128], scales and zeros [..., 16, 4] (float64)."""
    blocks = np.asarray(blocks)
    place, scale = (PLACES[2], PLACES[3]) if values else (PLACES[0], PLACES[1])
    codes = blocks[..., place[..., 0]] >> place[..., 1].astype(np.uint8) & 15

    def half(at):
        lo, hi = blocks[..., at], blocks[..., at + 1]
        return (lo.astype(np.uint16) | hi.astype(np.uint16) << 8).view(np.float16).astype(np.float64)
    return codes, half(scale[..., 0]), half(scale[..., 1])


def rows(blocks, values):
    """What blocks [..., 2560] stand for: [..., 16, 128] in 64 bits."""
    c, s, z = parts(blocks, values)
    c = c.reshape(*c.shape[:-1], 4, G)
    return (c * s[..., None] + z[..., None]).reshape(*c.shape[:-2], D)
