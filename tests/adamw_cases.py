"""AdamW's definition on the CPU, for the tests: the moments in fp32 operations whose roundings the interface states (so to
the last bit, codes among it), the parameters in 64 bits."""
import numpy as np
import torch

BLOCK = 256


def mix(x):
    x = np.asarray(x, np.uint64) & 0xFFFFFFFF
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def random_bits(seed, t, place, first, n):
    """The 32 bits of elements [first, first + n) of the tensor at `place`."""
    key = mix(mix(mix(t) ^ np.uint64(seed & 0xFFFFFFFF)) + np.uint64(place))
    i = np.arange(first, first + n, dtype=np.uint64)
    return mix(key + (i & np.uint64(0xFFFFFFFF)) + np.uint64(0x9E3779B9) * (i >> np.uint64(32)))


def decode_codes(code, e, top):
    """code: (blocks, 256) without a sign; e: (blocks,) bytes; in 64 bits.  top: the highest exponent's field."""
    f, k = code.astype(np.int64) >> 3, code.astype(np.int64) & 7
    x = np.ldexp(np.where(f > 0, 8 + k, k).astype(np.float64), np.maximum(f, 1) - top - 3 + e[:, None].astype(np.int64) - 100)
    return np.where(e[:, None] == 255, np.nan, x)


def decode(state, bits):
    """(m, v) of a state buffer as (blocks, 256), in 64 bits."""
    if bits == 32:
        s = state.reshape(-1, 2, BLOCK).astype(np.float64)
        return s[:, 0], s[:, 1]
    s = state.reshape(-1, 2 * BLOCK + 16)
    cm, cv, em, ev = s[:, :BLOCK], s[:, BLOCK:2 * BLOCK], s[:, 2 * BLOCK], s[:, 2 * BLOCK + 1]
    m = decode_codes(cm & 127, em, 15)
    return np.where(cm & 128, -m, m), decode_codes(cv, ev, 31)


def encode(x, top, u, exact=None):
    """Codes and exponent bytes of |x| (blocks, 256) in 64 bits; u: 16 random bits over 2^16.  A number is taken down to a
    multiple of its step after adding u steps; one that lies on it then, but above `exact`, to the multiple below."""
    most = np.max(np.where(np.isnan(x), np.inf, np.abs(x)), axis=1)
    bad = ~np.isfinite(most)
    most = np.where(bad, 1.0, most)
    m, e = np.frexp(np.where(most > 0, most, 1.0))            # most = m 2^e, m in [1/2, 1)
    e = np.where(most > 0, e - 1 + (m >= 15 / 16), -127)       # the next exponent where 1.875 2^e could round up
    e = np.clip(e, -100, 127)
    y = np.where(bad[:, None], 0.0, np.ldexp(np.abs(x), -e[:, None]))
    _, ey = np.frexp(np.where(y > 0, y, 2.0 ** -1000))
    f = np.clip(ey - 1 + top, 0, top)                          # field of y's binade, 0 below the least
    step = np.ldexp(1.0, np.maximum(f, 1) - top - 3)
    q = np.floor(y / step + u)                                 # 8 + k, or k for f = 0; 16 is the next binade's first
    code = np.where(f > 0, f * 8 + q - 8, q)
    if exact is not None:
        code = code - ((y / step + u == q) & (np.abs(exact) < np.abs(x)))
    return np.minimum(code, top * 8 + 7).astype(np.uint8), np.where(bad, 255, e + 100).astype(np.uint8)


def step_moments(g, state, bits, betas, seed, t, place, first=0):
    """(m, v) in fp32 before they are rounded to codes, and the new state buffer.  g: n numbers in fp32."""
    n = len(g)
    m, v = (a.astype(np.float32) for a in decode(state, bits))
    G = np.zeros(m.size, np.float32)
    G[:n] = g
    G = G.reshape(m.shape)
    b1, b2 = (np.float32(b) for b in betas)
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        v64 = v.astype(np.float64) * betas[1] + (1.0 - betas[1]) * G.astype(np.float64) ** 2
        m = m * b1 + G * np.float32(1.0 - betas[0])
        v = v * b2 + (G * G) * np.float32(1.0 - betas[1])
    if bits == 32:
        return m, v, np.stack((m, v), 1).reshape(-1)
    new = np.zeros((len(m), 2 * BLOCK + 16), np.uint8)
    r = random_bits(seed, t, place, first, m.size).reshape(m.shape)
    cm, em = encode(m.astype(np.float64), 15, (r & np.uint64(0xFFFF)).astype(np.float64) / 65536)
    cv, ev = encode(v.astype(np.float64), 31, (r >> np.uint64(16)).astype(np.float64) / 65536, v64)
    gone = em == 255
    cm = np.where(gone[:, None], 0, cm + 128 * ((m < 0) & (cm > 0)))
    cv = np.where((ev == 255)[:, None], 0, np.where((v > 0) & (cv == 0), 1, cv))
    new[:, :BLOCK], new[:, BLOCK:2 * BLOCK], new[:, 2 * BLOCK], new[:, 2 * BLOCK + 1] = cm, cv, em, ev
    return m, v, new.reshape(-1)


def step_param(p, m, v, betas, eps, lr, wd, t):
    """The new parameters in 64 bits, and the size of what was taken off."""
    p, m, v = (np.asarray(a, np.float64) for a in (p, m, v))
    with np.errstate(invalid="ignore", over="ignore"):
        u = lr * m / (1 - betas[0] ** t) / (np.sqrt(v / (1 - betas[1] ** t)) + eps)
    return p - lr * wd * p - u, np.abs(u)


def as_numpy(x):
    return x.detach().float().cpu().numpy() if x.dtype in (torch.bfloat16, torch.float16) else x.detach().cpu().numpy()
