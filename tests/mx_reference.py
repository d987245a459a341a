"""The router and the MXFP4 operators in 64 bits, plainly, for the tests: numpy only, no
code of the library.  Error bounds beside the values are derived where they are made."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E2M1 = np.concatenate([E2M1, -E2M1])


def to_f64(x, kind):
    """Values of a float32 / float16 array, or of bfloat16 bit patterns (uint16)."""
    if kind == "bf16":
        return (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return x.astype(np.float64)


def scale_byte(amax):
    """max(floor(log2 a) - 2, -127) + 127; 0 for 0."""
    e = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1
    return np.where(amax > 0, np.maximum(e - 2, -127) + 127, 0).astype(np.int64)


def round_e2m1(y):
    """Magnitudes y to the nearest of 0 .. 6, ties to the even code; the code 0..7."""
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    up_at_tie = np.array([False, True, False, True, False, True, False])
    y = y[..., None]
    return np.where(up_at_tie, y >= mid, y > mid).sum(-1)


def quantise(x):
    """Codes 0..15 [..., D] and scale bytes [..., D / 32] of x (64 bits)."""
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    s = scale_byte(np.abs(b).max(-1))
    code = round_e2m1(np.abs(b) * 2.0 ** (127 - s[..., None])) + 8 * np.signbit(b)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def values(codes, scales):
    v = E2M1[codes].reshape(scales.shape + (32,))
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(codes.shape)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def scale_planes(scales):
    """[rows][D / 32] bytes -> [ceil(D / 128)][pitch] words, as the library holds them."""
    rows, n = scales.shape
    q, pitch = (n + 3) // 4, (rows + 3) // 4 * 4
    out = np.zeros((q, pitch, 4), np.uint8)
    padded = np.zeros((rows, q * 4), np.uint8)
    padded[:, :n] = scales
    out[:, :rows] = padded.reshape(rows, q, 4).transpose(1, 0, 2)
    return out.view(np.uint32)[..., 0]


def blocks(codes, scales, gate_up):
    """The documented weight blocks of codes [E][N][D] and scales [E][N][D / 32], element by element."""
    E, N, D = codes.shape
    KB, packed = (D + 255) // 256, pack(codes)
    out = np.zeros((E, N // 128, KB, 17408), np.uint8)
    for nb in range(N // 128):
        for r in range(128):
            ch = ((r // 32) % 2) * (N // 2) + nb * 64 + (r // 64) * 32 + r % 32 if gate_up else nb * 128 + r
            for k in range(D // 32):
                kb, c = k // 8, k % 8
                at = r * 128 + (c ^ (r % 8)) * 16
                out[:, nb, kb, at:at + 16] = packed[:, ch, k * 16:k * 16 + 16]
                out[:, nb, kb, 16384 + 512 * (c // 4) + 4 * r + c % 4] = scales[:, ch, k]
    return out


def sum_error(a, w):
    """How far an fp32 sum over k of a[.., k] w[n, k] may be off, each [.., n]: the products of one
    scaled block pair are exact and so is their sum (multiples of a quarter below 2^11, scaled), so
    at most D / 32 block sums are added; every addition may drop 2^-22 of the magnitude summed so
    far (truncation instead of rounding, and once more where operands are aligned)."""
    n = a.shape[-1] // 32 + 8
    return n * 2.0 ** -22 * (np.abs(a) @ np.abs(w).T)


def f16_error(v):
    """Rounding to binary16: half a unit in the last place, or in the smallest subnormal's."""
    return np.abs(v) * 2.0 ** -11 + 2.0 ** -25


def silu_mul(g, u, eg, eu):
    """h = silu(g) u and its error: silu' is within 1.1 of 0, exp and the division are good to a few
    units of 2^-23 (2^-19 allowed, and what exp's argument loses: 2^-22 of |g|)."""
    s = g / (1.0 + np.exp(-g))
    h = s * u
    return h, 1.1 * np.abs(u) * eg + (np.abs(s) + 1.1 * eg) * eu + np.abs(h) * (2.0 ** -19 + 2.0 ** -22 * np.abs(g))


def quantise_interval(h, err):
    """Smallest and largest magnitude that an element of h, off by up to err, may have as MXFP4,
    and the smallest and largest scale byte of its block."""
    b, d = np.abs(h).reshape(h.shape[:-1] + (h.shape[-1] // 32, 32)), err.reshape(h.shape[:-1] + (h.shape[-1] // 32, 32))
    lo, hi = np.maximum(b - d, 0.0), b + d
    s0, s1 = scale_byte(lo.max(-1)), scale_byte(hi.max(-1))
    both = []
    for v in (lo, hi):
        for s in (s0, s1):
            both.append(E2M1[round_e2m1(v * 2.0 ** (127 - s[..., None]))] * 2.0 ** (s[..., None] - 127.0))
    return np.min(both, 0).reshape(h.shape), np.max(both, 0).reshape(h.shape), s0, s1


def route(logits, topK, sigmoid, renormalise, scale, bias=None):
    """expert_idx, probs, keys [M][E] (-inf where masked) in 64 bits."""
    l = np.where(np.isnan(logits), -np.inf, np.minimum(logits, np.finfo(np.float32).max))
    masked = l == -np.inf
    if sigmoid:
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-l))
    else:
        top = np.where(masked.all(1), 0.0, l.max(1))[:, None]
        ex = np.where(masked, 0.0, np.exp(np.where(masked, top, l) - top))
        p = ex / np.maximum(ex.sum(1, keepdims=True), 1e-300)
    p = np.where(masked, 0.0, p)
    key = np.where(masked, -np.inf, l if bias is None else p + bias)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :topK]
    w = np.take_along_axis(p, idx, 1)
    none = np.take_along_axis(masked, idx, 1)
    if renormalise:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return np.where(none, -1, idx).astype(np.int32), np.where(none, 0.0, w * scale), key, p


def layer(x, expert_idx, probs, w1, w2):
    """Output and error bound of the MXFP4 layer: x [M][K] quantised values, w1 [E][2I][K], w2 [E][K][I]."""
    M, K = x.shape
    I = w2.shape[2]
    out, err = np.zeros((M, K)), np.zeros((M, K))
    for t in range(M):
        for j, e in enumerate(expert_idx[t]):
            if not 0 <= e < w1.shape[0]:
                continue
            gu, eg = x[t:t + 1] @ w1[e].T, sum_error(x[t:t + 1], w1[e])
            h, eh = silu_mul(gu[:, :I], gu[:, I:], eg[:, :I], eg[:, I:])
            q = values(*quantise(h))
            lo, hi, _, _ = quantise_interval(h, eh)
            y = q @ w2[e].T
            ey = sum_error(np.maximum(np.abs(q), hi), w2[e]) + (hi - lo) @ np.abs(w2[e]).T
            p = float(probs[t, j])
            out[t] += p * y[0]
            # a product's own result may be held in binary16 before it is weighted, and the
            # weighted sum of topK terms rounds that often in fp32
            err[t] += abs(p) * (ey[0] + f16_error(np.abs(y[0]) + ey[0]) + np.abs(y[0]) * 2.0 ** -20)
    return out, err + f16_error(np.abs(out) + err)
