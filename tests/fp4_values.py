"""The 4-bit KV row format (CSA_MIXED_MXFP4_BF16) in numpy, from its definition."""
import numpy as np

from long_context_sparse_08_b200 import workloads as W

C, R, NOPE, WIN = 512, 64, 448, 128
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)


def row_bytes(c, r):
    return (c - r) // 2 + -(-((c - r) // 32) // 16) * 16 + 2 * r


def encode_rows(x, r=R):
    """float32 rows [n, c] -> uint8 [n, row_bytes(c, r)], by the format's definition."""
    x = np.asarray(x, np.float32)
    n, c = x.shape
    nb = (c - r) // 32
    blk = x[:, :c - r].reshape(n, nb, 32)
    amax = np.abs(blk).max(-1)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(amax.astype(np.float64))) - 2
    e = np.clip(np.where(amax > 0, e, -14), -14, 13)
    v = (blk / np.exp2(e)[..., None]).reshape(n, c - r).astype(np.float64)
    a = np.minimum(np.abs(v), 6.0)
    # nearest grid value, the even code at a midpoint
    d = np.abs(a[..., None] - E2M1)
    lo = d.argmin(-1)
    tie = np.isclose(d[np.arange(n)[:, None], np.arange(c - r), np.minimum(lo + 1, 7)], d.min(-1),
                     rtol=0, atol=0) & (lo < 7)
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    code = np.where((v < 0) & (code > 0), code + 8, code).astype(np.uint8)
    out = np.zeros((n, row_bytes(c, r)), np.uint8)
    out[:, :(c - r) // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    out[:, (c - r) // 2:(c - r) // 2 + nb] = (e + 127).astype(np.uint8)
    out[:, out.shape[1] - 2 * r:] = W.f32_to_bf16_bits(np.ascontiguousarray(x[:, c - r:])).view(np.uint8)
    return out


def decode_rows(b, c=C, r=R):
    """uint8 rows [..., bytes] -> float64 [..., c]."""
    b = np.asarray(b)
    nb = (c - r) // 32
    cod = b[..., :(c - r) // 2]
    code = np.stack((cod & 15, cod >> 4), -1).reshape(b.shape[:-1] + (c - r,))
    v = np.where(code >= 8, -E2M1[code & 7], E2M1[code & 7])
    ex = b[..., (c - r) // 2:(c - r) // 2 + nb].astype(np.float64) - 127
    v = v * np.repeat(np.exp2(ex), 32, -1)
    rope = np.ascontiguousarray(b[..., b.shape[-1] - 2 * r:]).view(np.uint16)
    return np.concatenate((v, W.bf16_bits_to_f32(rope).astype(np.float64)), -1)


def exponent_and_code(v):
    """Exponent and e2m1 code of a value that is its block's largest."""
    a = abs(float(v))
    e = 13 if a >= 2.0 ** 16 else (-14 if a == 0 else int(np.clip(np.floor(np.log2(a)) - 2, -14, 13)))
    x = min(a / 2.0 ** e, 6.0)
    d = np.abs(E2M1 - x)
    best = [i for i in range(8) if d[i] == d.min()]
    code = best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)
    return e, code + 8 if v < 0 and code else code
