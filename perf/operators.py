"""Cases of the layer's operators beyond the bottleneck block: what to run, at which
sizes, and what each operator computes, written out.

Four operators, each with a plain form of elementary torch operations (``own`` false) and
the library's own call (``own`` true):

* ``rope``      rotary positions with one or more position axes on the q and k planes of a
                QKV block, and the inverse rotation of their gradients;
* ``dropout``   dropout of a branch output added to the residual, the mask regenerated
                from a counter (Philox4x32-10) and never stored, and its gradient;
* ``quantise``  bf16 to 8-bit floating point with one power-of-two scale for each block
                of 128 along the contracted dimension, as stored and transposed;
* ``product``   the matrix product of two such operands, with the deferred row scale and
                the activation of the bottleneck block.

Scale bytes hold the exponent plus 127 and lie in tiles of 128 rows x 4 blocks: the byte
of row r, block b is at ((r // 128) * ceil(blocks / 4) + b // 4) * 512 + (r % 32) * 16 +
(r // 32 % 4) * 4 + b % 4; bytes of rows and blocks outside the operand are 127.
"""

import functools
import math

import numpy as np
import torch

own = False

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA = {"e4m3": 3, "e5m2": 2}
LOWEST = {"e4m3": -6, "e5m2": -14}      # exponent of the smallest normal value
DTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of a 2048-wide layer: pure latency
        dict(name="rope_token", op="rope", T=1, hq=16, hk=16, D=128, R=128, axes=1, far=8192,
             interleaved=False, inverse=False, packed=True),
        # q and k of the 4096-wide layer at the benchmark's token count
        dict(name="rope_text", op="rope", T=16384, hq=32, hk=32, D=128, R=128, axes=1,
             far=16384, interleaved=False, inverse=False, packed=False),
        # gradients of a video batch: time, height and width, shared key heads, an odd token
        # count, adjacent pairs, and times far from zero
        dict(name="rope_video_grad", op="rope", T=12007, hq=40, hk=8, D=128, R=128, axes=3,
             far=4000000, interleaved=True, inverse=True, packed=True),
        # a short fine-tuning batch of a 2048-wide layer, forward and backward
        dict(name="dropout_short", op="dropout", T=77, n=2048, p=0.05, way="step"),
        # the residual branch of the 4096-wide layer at the benchmark's token count
        dict(name="dropout_residual", op="dropout", T=16384, n=4096, p=0.1, way="forward"),
        # the branch's gradient in the 5120-wide layer, an odd token count
        dict(name="dropout_grad", op="dropout", T=8191, n=5120, p=0.1, way="backward"),
        # the 4096-wide activations of a training step: rows for the forward product,
        # columns for the weight gradient, read once
        dict(name="quantise_training", op="quantise", rows=16384, cols=4096, fmt="e4m3",
             block_rows=1, way="both"),
        # a 2048-wide QKV block's down-projection weight, square blocks, both products' layouts
        dict(name="quantise_weight", op="quantise", rows=2048, cols=1536, fmt="e4m3",
             block_rows=128, way="both"),
        # one token through the two up-projections of the 4096-wide MLP
        dict(name="product_token", op="product", G=2, M=1, N=11008, K=1024, fa="e4m3", fb="e4m3",
             scaled=False, act="identity"),
        # the gate/up down-projection of the 4096-wide MLP with its row scale and activation
        dict(name="product_down", op="product", G=1, M=16384, N=2048, K=4096, fa="e4m3",
             fb="e4m3", scaled=True, act="silu"),
        # the two up-projections of the 4096-wide MLP
        dict(name="product_up", op="product", G=2, M=16384, N=11008, K=1024, fa="e4m3", fb="e4m3",
             scaled=False, act="identity"),
        # a weight gradient: tokens contracted, an odd number of them, 5-bit-exponent gradients
        dict(name="product_weight_grad", op="product", G=1, M=2048, N=4096, K=16383, fa="e5m2",
             fb="e4m3", scaled=False, act="identity"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "dropout", "quantise", "product", "product"])
    if op == "rope":
        D = rng.choice([64, 72, 80, 96, 128, 256])
        hk = rng.choice([1, 2, 4, 8, 16])
        hq = hk * rng.choice([1, 2, 4])
        T = min(_log(rng, 1, 16384), (1 << 27) // ((hq + hk) * D))
        return dict(op=op, T=T, hq=hq, hk=hk, D=D, R=D if rng.random() < 0.7 else D // 16 * 8,
                    axes=rng.choice([1, 2, 3]), far=_log(rng, 64, 16000000),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    packed=rng.random() < 0.5)
    if op == "dropout":
        n = 8 * _log(rng, 8, 1024)
        return dict(op=op, T=min(_log(rng, 1, 20000), (1 << 26) // n), n=n,
                    p=rng.choice([0.0, 0.01, 0.1, 0.25, 0.5]),
                    way=rng.choice(["forward", "backward", "step"]))
    if op == "quantise":
        cols = 8 * _log(rng, 8, 1376)
        return dict(op=op, rows=min(_log(rng, 1, 16384), (1 << 26) // cols), cols=cols,
                    fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), block_rows=rng.choice([1, 1, 128]),
                    way=rng.choice(["rows", "columns", "both"]))
    G = rng.choice([1, 1, 2, 3])
    N, K = 8 * _log(rng, 8, 1376), 8 * _log(rng, 8, 1024)
    M = min(_log(rng, 1, 16384), max(1, int(3.5e11 / (G * N * K))))
    return dict(op=op, G=G, M=M, N=N, K=K, fa=rng.choice(["e4m3", "e4m3", "e5m2"]), fb="e4m3",
                scaled=rng.random() < 0.5, act=rng.choice(["identity", "silu"]))


# ------------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _sections(pairs, axes):
    """How many of the pairs turn with each axis: a quarter with time, the rest shared."""
    if axes == 1:
        return [pairs]
    rest = pairs - pairs // 4
    return [pairs // 4] + [rest // (axes - 1)] * (axes - 2) + [rest - rest // (axes - 1) * (axes - 2)]


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    if c["op"] == "rope":
        T, hq, hk, D = c["T"], c["hq"], c["hk"], c["D"]
        if c["packed"]:     # slices of one [T, (hq + 2 hk) D] projection
            whole = _normal(g, (T, hq + 2 * hk, D))
            q, k = whole[:, :hq], whole[:, hq:hq + hk]
        else:               # planes of their own
            q, k = _normal(g, (T, hq, D)), _normal(g, (T, hk, D))
        span = [c["far"]] + [max(2, min(c["far"], 128))] * (c["axes"] - 1)
        pos = torch.stack([torch.randint(0, s, (T,), generator=g, device="cuda") for s in span])
        pairs = c["R"] // 2
        inv_freq = 10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
        sections = _sections(pairs, c["axes"])
        axis = np.repeat(np.arange(c["axes"]), sections)     # the axis that each pair turns with
        return dict(case=c, q=q, k=k, positions=pos.to(torch.int32), inv_freq=inv_freq,
                    sections=sections, axis=torch.from_numpy(axis).cuda(),
                    q_out=torch.empty_like(q).contiguous(), k_out=torch.empty_like(k).contiguous())
    if c["op"] == "dropout":
        shape = (c["T"], c["n"])
        return dict(case=c, x=_normal(g, shape), res=_normal(g, shape), dout=_normal(g, shape),
                    seed=0x5DEECE66D1234567 ^ (int(seed) * 0x9E3779B97F4A7C15 & (1 << 63) - 1),
                    offset=int(seed) % 1000 + (1 << 33), out=torch.empty(shape, device="cuda", dtype=torch.bfloat16),
                    dx=torch.empty(shape, device="cuda", dtype=torch.bfloat16))
    if c["op"] == "quantise":
        # rows of different magnitude, as activations and gradients have them
        x = torch.randn((c["rows"], c["cols"]), generator=g, device="cuda")
        x = x * torch.exp2(torch.randint(-6, 7, (c["rows"], 1), generator=g, device="cuda").float())
        return dict(case=c, x=x.to(torch.bfloat16))
    G, M, N, K = c["G"], c["M"], c["N"], c["K"]
    a, a_sf = quantise_plain(_normal(g, (G * M, K)), c["fa"], 1)
    b, b_sf = zip(*(quantise_plain(_normal(g, (N, K), K ** -0.5), c["fb"], 128) for _ in range(G)))
    # (the blocks of one operand's scale tiles start anew with every matrix of the batch)
    a_sf = torch.stack([pack_scales(s) for s in unpack_scales(a_sf, G * M, K).view(G, M, -1)])
    scale = torch.rand(M, generator=g, device="cuda") + 0.5 if c["scaled"] else None
    return dict(case=c, a=a.view(G, M, -1), a_sf=a_sf, b=torch.stack(b), b_sf=torch.stack(b_sf),
                row_scale=scale, out=torch.empty(G, M, N, device="cuda", dtype=torch.bfloat16))


def work(case):
    c = case
    if c["op"] == "rope":
        values = c["T"] * (c["hq"] + c["hk"]) * c["D"]
        return {"bytes": 4 * values + 4 * c["axes"] * c["T"] + 4 * c["R"],
                "flops": 3 * c["T"] * (c["hq"] + c["hk"]) * c["R"]}
    if c["op"] == "dropout":
        n = c["T"] * c["n"]
        return {"bytes": {"forward": 6, "backward": 4, "step": 10}[c["way"]] * n, "flops": 2 * n}
    if c["op"] == "quantise":
        n, ways = c["rows"] * c["cols"], 2 if c["way"] == "both" else 1
        return {"bytes": 2 * n + ways * n * 129 / 128, "flops": 3 * n * ways}
    G, M, N, K = c["G"], c["M"], c["N"], c["K"]
    return {"bytes": G * ((M + N) * K * 129 / 128 + 2 * M * N) + (4 * M if c["scaled"] else 0),
            "flops": 2 * G * M * N * K}


# ----------------------------------------------------------------------- scale layout
def pack_scales(e):
    """Scale bytes [rows, blocks] in tiles of 128 rows x 4 blocks."""
    rows, blocks = e.shape
    rt, bt = -(-rows // 128), -(-blocks // 4)
    full = torch.nn.functional.pad(e, (0, bt * 4 - blocks, 0, rt * 128 - rows), value=127)
    return full.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def unpack_scales(sf, rows, K):
    blocks = -(-K // 128)
    rt, bt = -(-rows // 128), -(-blocks // 4)
    return sf.view(rt, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)[:rows, :blocks]


# ------------------------------------------------------------------------- plain forms
def rope_plain(x, positions, inv_freq, axis, interleaved, inverse):
    """Pair i of the first 2 * len(inv_freq) values of each head turns by the angle
    positions[axis[i], t] * inv_freq[i] (its negative for the inverse)."""
    pairs = inv_freq.numel()
    # angles of far positions: 32 bits lose them
    angle = positions.double()[axis].T * inv_freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    sin = -sin if inverse else sin
    r = x[..., :2 * pairs].float()
    u, v = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :pairs], r[..., pairs:])
    u, v = u * cos - v * sin, v * cos + u * sin
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned.to(x.dtype), x[..., 2 * pairs:]], -1)


def _philox_round(state, _):
    # a product of two 32-bit words wraps in the signed 64-bit type to the same 64 bits
    c0, c1, c2, c3, k0, k1 = state
    p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    low = 0xFFFFFFFF
    return ((p1 >> 32 & low) ^ c1 ^ k0, p1 & low, (p0 >> 32 & low) ^ c3 ^ k1, p0 & low,
            (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low)


def keep_plain(count, p, seed, offset, device):
    """Element 8 g + j is kept when 16-bit half j of the Philox4x32-10 block with counter
    (g, offset) and key `seed` is at least round(65536 p)."""
    g = torch.arange(-(-count // 8), device=device, dtype=torch.int64)
    o = torch.full_like(g, offset & 0xFFFFFFFF), torch.full_like(g, offset >> 32)
    start = (g & 0xFFFFFFFF, g >> 32, *o, seed & 0xFFFFFFFF, seed >> 32)
    words = torch.stack(functools.reduce(_philox_round, range(10), start)[:4], -1)
    halves = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(-1)[:count]
    return halves >= dropped(p)


def dropped(p):
    """Of 65536 values of a 16-bit half, how many drop the element."""
    return int(math.floor(p * 65536.0 + 0.5))


def dropout_plain(x, res, p, seed, offset):
    keep = keep_plain(x.numel(), p, seed, offset, x.device).view(x.shape)
    y = torch.where(keep, x.float() * (65536.0 / (65536 - dropped(p))), 0.0)
    return (y if res is None else res.float() + y).to(x.dtype)


def quantise_plain(x, fmt, block_rows):
    """8-bit values [rows, pitch] (pitch: columns rounded up to 16, zeros behind them) and
    scale bytes: the smallest power of two s, at least 2^-127, with max|block| <= s * FMAX."""
    rows, cols = x.shape
    blocks, pitch = -(-cols // 128), -(-cols // 16) * 16
    rt = -(-rows // block_rows)
    full = torch.nn.functional.pad(x.float(), (0, blocks * 128 - cols, 0, rt * block_rows - rows))
    full = full.view(rt, block_rows, blocks, 128)
    largest = full.abs().amax((1, 3))
    bits = largest.view(torch.int32)
    byte = (bits >> 23) - (8 if fmt == "e4m3" else 15) + ((bits & 0x7FFFFF) > 0x600000).int()
    byte = torch.where(largest == 0, 127, byte.clamp(min=0)).to(torch.uint8)
    scale = ((254 - byte.int()) << 23).view(torch.float32)[:, None, :, None]
    q = (full * scale).view(rt * block_rows, blocks * 128)[:rows, :pitch].to(DTYPE[fmt])
    return q.contiguous(), pack_scales(byte.repeat_interleave(block_rows, 0)[:rows])


def dequantise_plain(q, sf, K):
    rows = q.shape[0]
    scale = (unpack_scales(sf, rows, K).int() << 23).view(torch.float32)   # 2^(byte - 127)
    return q[:, :K].float() * scale.repeat_interleave(128, 1)[:, :K]


def product_plain(a, a_sf, b, b_sf, K, row_scale, act):
    z = dequantise_plain(a, a_sf, K) @ dequantise_plain(b, b_sf, K).T
    z = z if row_scale is None else z * row_scale[:, None]
    z = z / (1 + torch.exp(-z)) if act == "silu" else z
    return z.to(torch.bfloat16)


def run(state):
    c = state["case"]
    return (run_own if own else run_plain)(state, c)


def run_plain(s, c):
    if c["op"] == "rope":
        args = (s["positions"], s["inv_freq"], s["axis"], c["interleaved"], c["inverse"])
        return rope_plain(s["q"], *args), rope_plain(s["k"], *args)
    if c["op"] == "dropout":
        rng = (c["p"], s["seed"], s["offset"])
        out = dropout_plain(s["x"], s["res"], *rng) if c["way"] != "backward" else None
        dx = dropout_plain(s["dout"], None, *rng) if c["way"] != "forward" else None
        return out, dx
    if c["op"] == "quantise":
        x, rows, cols = s["x"], None, None
        if c["way"] != "columns":
            rows = quantise_plain(x, c["fmt"], c["block_rows"])
        if c["way"] != "rows":
            cols = quantise_plain(x.T, c["fmt"], c["block_rows"])
        return rows, cols
    one = functools.partial(product_plain, K=c["K"], row_scale=s["row_scale"], act=c["act"])
    return torch.stack(list(map(one, s["a"], s["a_sf"], s["b"], s["b_sf"])))


def run_own(s, c):
    from rank_bottleneck_online_gb300 import binding as B
    if c["op"] == "rope":
        return B.rope(s["q"], s["k"], s["positions"], s["inv_freq"], sections=s["sections"],
                      interleaved=c["interleaved"], inverse=c["inverse"], q_out=s["q_out"],
                      k_out=s["k_out"])
    if c["op"] == "dropout":
        rng = (c["p"], s["seed"], s["offset"])
        out = dx = None
        if c["way"] != "backward":
            out = B.dropout_add(s["x"], *rng, residual=s["res"], out=s["out"])
        if c["way"] != "forward":
            dx = B.dropout_bwd(s["dout"], *rng, dx=s["dx"])
        return out, dx
    if c["op"] == "quantise":
        return B.fp8_quantize(s["x"], fmt=c["fmt"], block_rows=c["block_rows"], way=c["way"])
    if "ws" not in s:       # the workspace that a program keeps beside its weights
        s["ws"] = B.Workspace(B.fp8_matmul_workspace_bytes(c["M"], c["N"], c["K"], c["G"]))
    return B.fp8_matmul(s["a"], s["a_sf"], s["b"], s["b_sf"], c["K"], s["ws"],
                        row_scale=s["row_scale"], act=c["act"], out=s["out"])


# ------------------------------------------------------------------- definitions, 64 bits
def _rope_exact(x, s, c):
    x = x.double()
    out, first = x.clone(), 0
    for a, n in enumerate(s["sections"]):
        for i in range(first, first + n):
            turn = s["positions"][a].double() * s["inv_freq"][i] * (-1 if c["inverse"] else 1)
            at = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["R"] // 2)
            z = torch.complex(x[..., at[0]], x[..., at[1]]) * torch.polar(torch.ones_like(turn), turn)[:, None]
            out[..., at[0]], out[..., at[1]] = z.real, z.imag
        first += n
    return out


def _keep_exact(count, p, seed, offset):
    g = np.arange(-(-count // 8), dtype=np.uint64)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [g & low, g >> half, np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> half) ^ x[1] ^ np.uint64(key[0]), b & low, (a >> half) ^ x[3] ^ np.uint64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    drawn = np.stack(x, 1).astype("<u4").view("<u2").reshape(-1)[:count]
    return torch.from_numpy(drawn >= dropped(p)).cuda()


def _two_to(e):
    """2^e in 64 bits, from the bits of the format (pow and exp2 need not be exact)."""
    return (e.to(torch.int64) + 1023 << 52).view(torch.float64)


def _round8(v, fmt):
    """To the nearest 8-bit value, ties to even."""
    e = torch.frexp(v)[1] - 1
    step = _two_to(e.clamp(min=LOWEST[fmt]) - MANTISSA[fmt])
    return torch.round(v / step) * step


def _quantise_exact(x, fmt, block_rows):
    rows, cols = x.shape
    rt, blocks, pitch = -(-rows // block_rows), -(-cols // 128), -(-cols // 16) * 16
    full = torch.zeros(rt * block_rows, blocks * 128, dtype=torch.float64, device=x.device)
    full[:rows, :cols] = x
    tiles = full.unflatten(0, (rt, block_rows)).unflatten(2, (blocks, 128))
    m, e = torch.frexp(tiles.abs().amax((1, 3), keepdim=True) / FMAX[fmt])
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-127)
    e = torch.where(m == 0, 0, e)
    values = _round8(tiles * _two_to(-e), fmt).reshape(rt * block_rows, blocks * 128)
    return values[:rows, :pitch].contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _rope_exact(s["q"], s, c), _rope_exact(s["k"], s, c)
    if c["op"] == "dropout":
        keep = _keep_exact(s["x"].numel(), c["p"], s["seed"], s["offset"]).view(s["x"].shape)
        weight = keep.double() / (1.0 - dropped(c["p"]) / 65536.0)
        return (s["res"].double() + s["x"].double() * weight if c["way"] != "backward" else None,
                s["dout"].double() * weight if c["way"] != "forward" else None)
    if c["op"] == "quantise":
        x, rows, cols = s["x"].double(), None, None
        if c["way"] != "columns":
            rows = (_quantise_exact(x, c["fmt"], c["block_rows"]), None)
        if c["way"] != "rows":
            cols = (_quantise_exact(x.T, c["fmt"], c["block_rows"]), None)
        return rows, cols
    K, blocks = c["K"], -(-c["K"] // 128)
    out = []
    for g in range(c["G"]):
        operands = []
        for v, sf, rows in ((s["a"][g], s["a_sf"][g], c["M"]), (s["b"][g], s["b_sf"][g], c["N"])):
            r = torch.arange(rows, device="cuda")[:, None]
            b = torch.arange(K, device="cuda")[None] // 128
            at = ((r // 128) * -(-blocks // 4) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
            operands.append(v[:, :K].double() * _two_to(sf[at].int() - 127))
        z = operands[0] @ operands[1].mT
        if s["row_scale"] is not None:
            z *= s["row_scale"].double()[:, None]
        out.append(z * torch.sigmoid(z) if c["act"] == "silu" else z)
    return torch.stack(out)
