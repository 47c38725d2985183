"""The 8-bit operators from their definitions, in 64 bits (numpy, on the CPU),
and the error bounds the tests hold the kernels to.

Bounds.  A rounding to nearest is off by at most half a step, eps / 2 of the
value: with p significant bits the steps in [1, 2) are 2^(1-p), so 2^-8 for
bf16 (p = 8), 2^-11 for fp16 (11), 2^-24 for fp32 (24); below the normal range
half a step of the smallest normal's.  fp32 arithmetic: u = 2^-24
bounds one operation, n u a chain of n (n u < 2^-10 throughout, so second-order
terms are covered by the factor 1.01).

The 8-bit matrix instructions.  Measured on gfx950 with single products: the
128 products of a block are added in groups of 8 neighbours, aligned to the
group's largest; of 2^16 beside it, 2^3 is kept and 2^2 is lost.  A product p
in a group whose largest is P is therefore off by less than 2^-13 of the power
of two under P (of the operands' exponents' sum, which is at most |P|), and the sum of 8
by less than 8 * 2^-13 * max |p| of the group; the groups' sums are added in fp32.
"""
import numpy as np

BLOCK = 128
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
SMALLEST = {"bf16": 2.0 ** -126, "f16": 2.0 ** -14, "f32": 2.0 ** -126}   # smallest normal
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
U = 2.0 ** -24


def blocks(n):
    return -(-n // BLOCK)


def decode(raw, fp8):
    """The values of uint8 bit patterns, from the formats' definitions."""
    raw = np.asarray(raw, dtype=np.uint8).astype(np.int64)
    m_bits, bias = (3, 7) if fp8 == "e4m3" else (2, 15)
    sign = np.where(raw & 0x80, -1.0, 1.0)
    e, m = (raw & 0x7F) >> m_bits, raw & ((1 << m_bits) - 1)
    frac = m / float(1 << m_bits)
    v = np.where(e == 0, frac * 2.0 ** (1 - bias), (1.0 + frac) * np.exp2((e - bias).astype(np.float64)))
    if fp8 == "e4m3":
        v = np.where((raw & 0x7F) == 0x7F, np.nan, v)
    else:
        v = np.where(e == 31, np.where(m == 0, np.inf, np.nan), v)
    return sign * v


def _table(fp8):
    """Non-negative finite values in order, and their bit patterns."""
    raw = np.arange(128, dtype=np.uint8)
    v = decode(raw, fp8)
    keep = np.isfinite(v)
    return v[keep], raw[keep]


def encode(x, fp8):
    """Bit patterns nearest to x (float64, |x| within the type's range), ties to even."""
    v, raw = _table(fp8)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(v, a), 1, len(v) - 1)
    lo = hi - 1
    d_lo, d_hi = a - v[lo], v[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (raw[hi] % 2 == 0))
    r = np.where(up, raw[hi], raw[lo])
    r = np.where(np.isnan(x), 0x7F, r)
    return (r | np.where(np.signbit(x) & ~np.isnan(x), 0x80, 0)).astype(np.uint8)


def block_amax(x, rows):
    """Largest |x| of each block (NaN does not enter)."""
    m, k = x.shape
    p = np.zeros((-(-m // rows) * rows, blocks(k) * BLOCK))
    p[:m, :k] = np.where(np.isnan(x), 0.0, np.abs(x))
    return p.reshape(p.shape[0] // rows, rows, blocks(k), BLOCK).max(axis=(1, 3)) if p.size else \
        np.zeros((p.shape[0] // rows, blocks(k)))


def spread(s, rows, m, k):
    return np.repeat(np.repeat(s, rows, 0)[:m], BLOCK, 1)[:, :k]


def quantize_fp32(x, fp8, rows, pow2=False):
    """The quantisation exactly as it is defined, operation by operation in
    fp32: (bit patterns, scales).  x: float32 values."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        amax = block_amax(x, rows).astype(np.float32)
        s = np.maximum(amax / np.float32(TOP[fp8]), np.float32(2.0 ** -126))
        if pow2:
            m, e = np.frexp(s)
            s = np.where(np.isinf(s), s, np.ldexp(np.float32(1), np.where(m == 0.5, e - 1, e))).astype(np.float32)
        r = (np.float32(1) / s).astype(np.float32)
        y = (x * spread(r, rows, *x.shape)).astype(np.float32)
    return encode(y.astype(np.float64), fp8), s


def product(a, sa, b, sb, sb_rows):
    """C in float64, and the bound on what fp32 sums over blocks and (16-bit
    outputs) the 8-bit instructions leave: (C, exact_path, instruction_path).
    a, b: decoded values; sa, sb: float64 scales."""
    M, K = a.shape
    N = b.shape[0]
    C, path, instr = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    nb = blocks(K)
    with np.errstate(all="ignore"):
        for kb in range(nb):
            ab, bb = a[:, kb * BLOCK:(kb + 1) * BLOCK], b[:, kb * BLOCK:(kb + 1) * BLOCK]
            s = sa[:, kb][:, None] * np.repeat(sb[:, kb], sb_rows)[:N][None, :]
            C += s * (ab @ bb.T)
            # per block: 128 products' sums, two scales' product, the product with it, nb sums
            path += s * (np.abs(ab) @ np.abs(bb).T) * (128 + 3 + nb) * U
            for g in range(0, ab.shape[1], 8):
                pmax = (np.abs(ab[:, None, g:g + 8]) * np.abs(bb[None, :, g:g + 8])).max(axis=2)
                instr += s * pmax * 8 * 2.0 ** -13
    return C, 1.01 * path, 1.01 * instr


def rms(x, residual, w, eps):
    """(h as float64 before its rounding is the caller's; here h is given rounded): y, rstd."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h ** 2).mean(axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def rms_backward(dy, h, w, rstd, dh):
    g = dy * w
    dx = rstd[:, None] * (g - h * (rstd ** 2 * (g * h).mean(axis=1))[:, None])
    if dh is not None:
        dx = dx + dh
    return dx, (dy * h * rstd[:, None]).sum(axis=0)


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound everywhere; NaN exactly where ref has NaN."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), "%s: NaN in other places" % what
    with np.errstate(invalid="ignore"):
        bad = np.argwhere(~((np.abs(got - ref) <= bound) | (got == ref) | np.isnan(ref)))
    assert bad.size == 0, "%s: %d of %d off, first at %s: %r, not %r (bound %r)" % (
        what, len(bad), got.size, bad[0], got[tuple(bad[0])], ref[tuple(bad[0])],
        np.broadcast_to(bound, ref.shape)[tuple(bad[0])])


def half_step(ref, t):
    """Half a step of type t at ref (and what fp32 arithmetic of a few operations adds is the caller's)."""
    return np.maximum(np.abs(ref), SMALLEST[t]) * HALF_STEP[t]
