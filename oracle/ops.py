"""fp64 definitions of the layer's operators around the bottleneck block: rotary
positions, the counter-based dropout mask, 8-bit floating point with a power-of-two scale
for each block of 128, and the product of such operands; attention over packed sequences
and its gradients, the norm behind a residual, and gradient clipping. NumPy on the CPU,
written from the formulas; nothing here is shared with the CUDA path.
"""

from __future__ import annotations

import decimal

import numpy as np

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA_BITS = {"e4m3": 3, "e5m2": 2}
BIAS = {"e4m3": 7, "e5m2": 15}


# ------------------------------------------------------------------ rotary positions
_TWO_PI = decimal.Decimal("6.28318530717958647692528676655900576839433879875021")


def rope_angles(positions, inv_freq, pair_axis):
    """[T, pairs] angles in radians within a turn: positions [axes, T] integers, inv_freq
    [pairs] fp64. Python integers hold each frequency as a 128-bit fraction of a turn."""
    pos = [[int(p) for p in row] for row in np.asarray(positions)]
    out = np.empty((len(pos[0]), len(inv_freq)))
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        for i, w in enumerate(np.asarray(inv_freq, dtype=np.float64)):
            turn = int(decimal.Decimal(float(w)) / _TWO_PI * (1 << 128))
            out[:, i] = [(p * turn % (1 << 128)) / (1 << 128) for p in pos[pair_axis[i]]]
    return 2 * np.pi * out


def rope(x, positions, inv_freq, pair_axis, interleaved=False, inverse=False):
    """x [T, heads, dim] fp64."""
    x = np.asarray(x, dtype=np.float64)
    pairs = len(inv_freq)
    phi = rope_angles(positions, inv_freq, pair_axis)[:, None, :]
    c, s = np.cos(phi), np.sin(phi) * (-1.0 if inverse else 1.0)
    out = x.copy()
    if interleaved:
        u, v = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
        out[..., 0:2 * pairs:2], out[..., 1:2 * pairs:2] = u * c - v * s, v * c + u * s
    else:
        u, v = x[..., :pairs], x[..., pairs:2 * pairs]
        out[..., :pairs], out[..., pairs:2 * pairs] = u * c - v * s, v * c + u * s
    return out


# ------------------------------------------------------------------------- dropout
def philox4x32_10(counter, key):
    """The Philox4x32-10 block (Salmon, Moraes, Dror and Shaw, SC 2011) of one counter
    (four 32-bit words) and key (two), with Python integers."""
    mask = 0xFFFFFFFF
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & mask, (a >> 32) ^ c[3] ^ k[1], a & mask]
        k = [(k[0] + 0x9E3779B9) & mask, (k[1] + 0xBB67AE85) & mask]
    return c


def dropout_drop(p):
    """Of the 65536 draws, how many drop an element."""
    return int(np.floor(p * 65536.0 + 0.5))


def dropout_keep(elements, p, seed, offset):
    """keep of the given flat element indices."""
    mask = 0xFFFFFFFF
    drop, blocks, out = dropout_drop(p), {}, []
    for e in elements:
        g, j = divmod(int(e), 8)
        if g not in blocks:
            blocks[g] = philox4x32_10((g & mask, g >> 32, offset & mask, offset >> 32 & mask),
                                      (seed & mask, seed >> 32))
        word = blocks[g][j // 2]
        out.append((word >> 16 if j & 1 else word & 0xFFFF) >= drop)
    return np.array(out, dtype=bool)


# --------------------------------------------------------------------- 8-bit values
def fp8_values(fmt):
    """The values of the 256 codes of a format."""
    m, bias = MANTISSA_BITS[fmt], BIAS[fmt]
    out = np.empty(256)
    for code in range(256):
        e, f = (code & 127) >> m, code & ((1 << m) - 1)
        v = f * 2.0 ** (1 - bias - m) if e == 0 else (1 + f / (1 << m)) * 2.0 ** (e - bias)
        if fmt == "e4m3" and code & 127 == 127:
            v = np.nan
        if fmt == "e5m2" and e == 31:
            v = np.inf if f == 0 else np.nan
        out[code] = -v if code & 128 else v
    return out


def fp8_round(v, fmt):
    """To the nearest value of the format, ties to the even code; finite |v| <= FMAX."""
    table = fp8_values(fmt)[:128]
    table = table[np.isfinite(table)]
    a = np.abs(v)
    hi = np.searchsorted(table, a).clip(0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - a, a - table[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.copysign(np.where(take_hi, table[hi], table[lo]), v)


def fp8_quantize(x, fmt, block_rows=1):
    """(values [rows, cols] after the scale, exponents [rows, blocks]) of x [rows, cols] fp64,
    blocks of block_rows x 128."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    blocks = -(-cols // 128)
    q, e = np.empty_like(x), np.zeros((rows, blocks), dtype=np.int64)
    for r0 in range(0, rows, block_rows):
        for b in range(blocks):
            part = x[r0:r0 + block_rows, b * 128:(b + 1) * 128]
            fine = np.abs(part[np.isfinite(part)])
            top = fine.max() if fine.size else 0.0
            ex = 0
            if top > 0:
                ex = max(-127, int(np.floor(np.log2(top / FMAX[fmt]))) - 1)
                while top > FMAX[fmt] * 2.0 ** ex:
                    ex += 1
            e[r0:r0 + block_rows, b] = ex
            done = fp8_round(np.where(np.isfinite(part), part, 0.0) * 2.0 ** -ex, fmt)
            done = np.where(np.isnan(part), np.nan, done)
            inf = np.nan if fmt == "e4m3" else np.inf
            done = np.where(np.isinf(part), np.copysign(inf, part), done)
            q[r0:r0 + block_rows, b * 128:(b + 1) * 128] = done
    return q, e


def fp8_scales(exponents):
    """Scale bytes of exponents [rows, blocks] in tiles of 128 rows x 4 blocks."""
    rows, blocks = exponents.shape
    kt = -(-blocks // 4)
    out = np.full(-(-rows // 128) * kt * 512, 127, dtype=np.uint8)
    for r in range(rows):
        for b in range(blocks):
            at = (r // 128 * kt + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
            out[at] = exponents[r, b] + 127
    return out


def fp8_dequantize(values, exponents):
    """values [rows, K] times their blocks' scales."""
    scale = np.repeat(2.0 ** exponents, 128, axis=1)
    return values * scale[:, :values.shape[1]]


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def fp8_matmul(a, b, row_scale=None, act="identity"):
    """(act(row_scale * a b^T), the sum of the magnitudes that each value adds up) of
    dequantised operands."""
    with np.errstate(invalid="ignore"):
        z, size = a @ b.T, np.abs(a) @ np.abs(b).T
    if row_scale is not None:
        z, size = z * row_scale[:, None], size * np.abs(row_scale)[:, None]
    return (silu(z) if act == "silu" else z), size


# ----------------------------------------------------------------------- attention
def attention(q, k, v, lengths, causal=True, scale=None, dout=None):
    """q [Tq, hq, dim], k and v [Tk, hk, dim]; lengths: (queries, keys) of each sequence. A dict
    of out, lse [hq, Tq] and, with dout, dq, dk, dv; rows of no sequence are NaN. Also the sums of
    magnitudes that a relative rounding of the probabilities P, of their gradients dS and of out
    scales with: out_size = sum P |v|, dv_size = sum P |dout|, dq_size and dk_size = sum E |k|,
    sum E |q| with E = |dS| + scale P sum |dout| (|out| + out_size), the last for what a rounded
    out makes of dS = scale P (dP - sum dout out)."""
    group = q.shape[1] // k.shape[1]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    like = {"out": q, "out_size": q}
    if dout is not None:
        like |= {"dq": q, "dq_size": q, "dk": k, "dk_size": k, "dv": k, "dv_size": k}
    r = {name: np.full(x.shape, np.nan) for name, x in like.items()}
    r["lse"] = np.full((q.shape[1], q.shape[0]), np.nan)
    q0 = k0 = 0
    for nq, nk in lengths:
        i, j = slice(q0, q0 + nq), slice(k0, k0 + nk)
        seen = np.ones((nq, nk), dtype=bool)
        if causal:
            seen = np.arange(nk)[None] <= np.arange(nq)[:, None] + nk - nq
        for name in like:
            if name[:2] in ("dk", "dv"):
                r[name][j] = 0.0
        for h in range(q.shape[1]):
            g = h // group
            s = np.where(seen, scale * q[i, h] @ k[j, g].T, -np.inf)
            top = s.max(1, initial=-np.inf)
            e = np.exp(s - np.where(np.isinf(top), 0.0, top)[:, None])
            total = e.sum(1)
            with np.errstate(divide="ignore"):
                r["lse"][h, i] = top + np.log(total)
            p = e / np.where(total == 0, 1.0, total)[:, None]
            r["out"][i, h] = p @ v[j, g]
            r["out_size"][i, h] = p @ np.abs(v[j, g])
            if dout is None:
                continue
            do = dout[i, h]
            dp = do @ v[j, g].T
            ds = scale * p * (dp - (p * dp).sum(1)[:, None])
            size = (np.abs(do) * (np.abs(r["out"][i, h]) + r["out_size"][i, h])).sum(1)
            size = np.abs(ds) + scale * p * size[:, None]
            r["dq"][i, h], r["dq_size"][i, h] = ds @ k[j, g], size @ np.abs(k[j, g])
            r["dk"][j, g] += ds.T @ q[i, h]
            r["dk_size"][j, g] += size.T @ np.abs(q[i, h])
            r["dv"][j, g] += p.T @ do
            r["dv_size"][j, g] += p.T @ np.abs(do)
        q0, k0 = q0 + nq, k0 + nk
    return r


# ------------------------------------------------------- norm behind a residual
def row_scale(h, eps):
    """1 / rms of the rows of h."""
    return 1.0 / np.sqrt(np.mean(np.square(h), axis=1) + eps)


# --------------------------------------------------------------- gradient clipping
def grad_clip(grads, max_norm):
    """(norm over all, gradients scaled to it)."""
    norm = np.sqrt(sum(float(np.sum(np.square(g))) for g in grads))
    by = max_norm / (norm + 1e-6)
    return norm, [g if by >= 1 else g * by for g in grads]
