"""Plain 64-bit reference of the 4-bit formats, the scale atoms and the root-mean-square norm (numpy only).

Values are encoded by nearest-value search over the format's exact values (ties to the even code), so
nothing here shares a method with the kernels."""
import numpy as np

MXFP8, MXFP4, NVFP4 = 2, 3, 4
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])
E5M2 = np.array([m / 4 * 2.0 ** -14 for m in range(4)] +
                [(1 + m / 4) * 2.0 ** (e - 15) for e in range(1, 31) for m in range(4)])


def encode(v, values, sign_bit):
    """Codes of v (float64): nearest of the sorted non-negative values, ties to the even code, saturating;
    the sign of v (-0 included) in sign_bit. NaN is the caller's."""
    a = np.minimum(np.abs(v), values[-1])
    half = (values[1:] + values[:-1]) / 2
    lo, hi = np.searchsorted(half, a, side="left"), np.searchsorted(half, a, side="right")
    at = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))          # lo != hi only at a tie
    return (at | np.where(np.signbit(v), sign_bit, 0)).astype(np.uint8)


def decode(code, values, sign_bit):
    v = values[code & (sign_bit - 1)]
    return np.where(code & sign_bit, -v, v)


def bf16_f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e8m0_exponent(amax, emax):
    """floor(log2(amax)) - emax in [-127, 127] (amax finite or infinite, >= 0)."""
    m, e = np.frexp(amax)
    e = np.where(amax == 0, -127, np.where(np.isinf(amax), 127, e - 1 - emax))
    return np.clip(e, -127, 127).astype(np.int64)


def quantise(x_bits, kind, g=1.0):
    """Blocks along the rows of BF16 patterns [rows, K]: (codes [rows, K], scale bytes [rows, K / block])."""
    rows, K = x_bits.shape
    B = 32 if kind == MXFP4 else 16
    x32 = (x_bits.astype(np.uint32) << 16).view(np.float32).reshape(rows, K // B, B)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore", under="ignore"):
        amax = np.abs(x32).max(-1)                                       # NaN if any is
        nan = np.isnan(amax)
        if kind == MXFP4:
            X = np.where(nan, 0, e8m0_exponent(np.where(nan, 1, amax).astype(np.float64), 2))
            sf = np.where(nan, 255, X + 127).astype(np.uint8)
            v = x32.astype(np.float64) * np.exp2(-X.astype(np.float64))[..., None]
        else:
            t = (amax * np.float32(g)) / np.float32(6)
            nan = np.isnan(t)
            sf = np.where(nan, 0x7F, encode(np.where(nan, 0, t).astype(np.float64), E4M3, 128))
            s = E4M3[np.where(nan, 0x38, sf)].astype(np.float32)         # 0x38 stands for 1
            f = np.where(nan, np.float32(1), np.where(s > 0, np.float32(g) / np.where(s > 0, s, 1), np.float32(0)))
            v = (x32 * f.astype(np.float32)[..., None]).astype(np.float64)
    codes = encode(np.where(np.isnan(v), 6.0, v), E2M1, 8)               # E2M1 has no NaN: +6
    return codes.reshape(rows, K), sf.astype(np.uint8)


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(q):
    return np.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)


def atoms(sf, kind):
    """Scale bytes [MN, n] -> atoms (zero where padded)."""
    MN, n = sf.shape
    per = {MXFP8: 4, MXFP4: 8, NVFP4: 16}[kind]
    R, N = -(-MN // 128) * 128, -(-n // per) * per
    full = np.zeros((R, N), np.uint8)
    full[:MN, :n] = sf
    return np.ascontiguousarray(full.reshape(R // 128, 4, 32, N // 4, 4).transpose(0, 3, 2, 1, 4)).reshape(-1)


def from_atoms(a, MN, n, kind):
    """Atoms -> (scale bytes [MN, n], bytes that pad K for those rows)."""
    per = {MXFP8: 4, MXFP4: 8, NVFP4: 16}[kind]
    R, N = -(-MN // 128) * 128, -(-n // per) * per
    full = a.reshape(R // 128, N // 4, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(R, N)
    return np.ascontiguousarray(full[:MN, :n]), full[:MN, n:]


def scale_values(sf, kind):
    """Scale bytes as numbers (NaN for the NaN byte)."""
    if kind == NVFP4:
        return np.where(sf & 0x7F == 0x7F, np.nan, E4M3[np.minimum(sf, 0x7E)])
    return np.where(sf == 255, np.nan, np.exp2(sf.astype(np.float64) - 127))


def values(codes, sf, kind):
    """The numbers 4-bit codes [rows, K] with scale bytes [rows, K / block] stand for (without 1 / g)."""
    s = scale_values(sf, kind)
    return (decode(codes, E2M1, 8).reshape(*sf.shape, -1) * s[..., None]).reshape(codes.shape)


def rmsnorm(x, res, gamma, eps):
    """float64 (h, rstd, y) of BF16-valued float64 inputs; h = bf16(f32(x + res)) as float64."""
    h = x
    if res is not None:
        f = (x.astype(np.float32) + res.astype(np.float32)).view(np.uint32)
        h = bf16_f64(((f + 0x7FFF + ((f >> 16) & 1)) >> 16).astype(np.uint16))
    rstd = 1 / np.sqrt((h * h).sum(1) / h.shape[1] + eps)
    return h, rstd, h * rstd[:, None] * gamma


def rmsnorm_grad(dy, h, gamma, rstd, dres=None):
    """float64 (dh, dgamma)."""
    xh = h * rstd[:, None]
    g = dy * gamma
    dh = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    return dh if dres is None else dh + dres, (dy * xh).sum(0)
