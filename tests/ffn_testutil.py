"""Plain 64-bit forms of the expert feed-forward operators, with the error that
the kernels' arithmetic allows, for the tests."""
import numpy as np

SWIGLU = dict(alpha=1.0, limit=float("inf"), beta=0.0)
CLAMPED = dict(alpha=1.702, limit=7.0, beta=1.0)
DROPOUT_TAG = 0x44524F50
BF16_HALF = 2.0 ** -8      # half a bf16 step, relative
FLOOR = 2.0 ** -125        # below the normal range relative bounds end


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def gated(z, alpha, limit, beta):
    """h of interleaved pre-activations z [M, 2I], 64 bits."""
    g = np.minimum(z[:, 0::2], limit)
    u = np.clip(z[:, 1::2], -limit, limit)
    return g * sigmoid(alpha * g) * (u + beta)


def gated_bound(z, ez, alpha, limit, beta):
    """Error of a bf16 h whose pre-activations are off by at most ez.

    d(g s)/dg = s + x s (1 - s), x = alpha g, is within 1.1 in magnitude and
    d h/du = g s, so |dh| <= 1.1 |u + beta| eg + |g s| eu + 1.1 eg eu; the
    sigmoid's exponent is off by |x| 2^-23 and its exponential and reciprocal by
    2^-21: 1e-5 relative for |x| < 60 (beyond, s is 1 or h is below 1e-20); one
    bf16 rounding."""
    g = np.minimum(z[:, 0::2], limit)
    u = np.clip(z[:, 1::2], -limit, limit)
    eg, eu = ez[:, 0::2], ez[:, 1::2]
    gs = g * sigmoid(alpha * g)
    h = gs * (u + beta)
    inner = 1.1 * np.abs(u + beta) * eg + np.abs(gs) * eu + 1.1 * eg * eu + 1e-5 * np.abs(h)
    return BF16_HALF * (np.abs(h) + inner) + inner + FLOOR


def gated_backward(dh, z, alpha, limit, beta):
    """dz [M, 2I] of dh [M, I] at z, 64 bits."""
    zg, zu = z[:, 0::2], z[:, 1::2]
    g, u = np.minimum(zg, limit), np.clip(zu, -limit, limit)
    s = sigmoid(alpha * g)
    dz = np.empty_like(z)
    dz[:, 0::2] = np.where(zg > limit, 0.0, dh * (u + beta) * s * (1 + alpha * g * (1 - s)))
    dz[:, 1::2] = np.where(np.abs(zu) > limit, 0.0, dh * g * s)
    return dz


def gated_backward_bound(dh, eh, z, alpha, limit, beta):
    """Error of a bf16 dz whose dh is off by at most eh.  s is 1e-5 off as above;
    in t = 1 + x (1 - s) that and the roundings are 1e-5 (1 + |x|) absolute."""
    zg, zu = z[:, 0::2], z[:, 1::2]
    g, u = np.minimum(zg, limit), np.clip(zu, -limit, limit)
    x = alpha * g
    s = sigmoid(x)
    fg, fu = (u + beta) * s * (1 + x * (1 - s)), g * s
    efg = 1e-5 * np.abs(u + beta) * s * (1 + np.abs(x)) + 1e-5 * np.abs(fg)
    efu = 1e-5 * np.abs(fu)
    out = np.empty_like(z)
    for k, (f, ef) in enumerate(((fg, efg), (fu, efu))):
        inner = np.abs(f) * eh + (np.abs(dh) + eh) * ef
        out[:, k::2] = BF16_HALF * (np.abs(dh * f) + inner) + inner + FLOOR
    return out


def int8_quantize(x32):
    """Codes and scales of fp32 rows (bf16 values), each operation rounded as defined."""
    x32 = x32.astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(x32).max(axis=1)
        ok = np.isfinite(amax)
        a = np.maximum(np.where(ok, amax, 1), np.float32(2.0 ** -100)).astype(np.float32)
        inv = ((np.float32(1.0) / a).astype(np.float32) * np.float32(127.0)).astype(np.float32)
        q = np.rint(np.where(ok[:, None], x32, 0) * inv[:, None]).astype(np.int8)
        scale = np.where(ok, (a / np.float32(127.0)).astype(np.float32), np.float32(np.nan))
    return q, scale.astype(np.float32)


def philox(counter, key):
    """Philox4x32-10 (Salmon et al., SC'11) of counter words [n, 4] under key (lo, hi)."""
    c = [np.asarray(counter[:, i], np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             p0 & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=1)


def dropout_words(n, seed, elem_offset=0):
    g = np.arange(elem_offset // 4, (elem_offset + n + 3) // 4, dtype=np.uint64)
    z = np.zeros_like(g)
    ctr = np.stack([g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), z, z + np.uint64(DROPOUT_TAG)], axis=1)
    return philox(ctr, (seed & 0xFFFFFFFF, seed >> 32)).reshape(-1)[:n]


def dropout_f32(x32, p, seed, elem_offset=0, residual32=None):
    """The FP32 value before the output's rounding, each operation rounded as defined."""
    keep = (dropout_words(x32.size, seed, elem_offset) >= np.uint64(round(p * 2.0 ** 32))).reshape(x32.shape)
    scale = np.float32(1.0 / (1.0 - p)) if p < 1 else np.float32(0)
    y = np.where(keep, x32.astype(np.float32) * scale, np.float32(0))
    return y if residual32 is None else (y + residual32.astype(np.float32)).astype(np.float32)
