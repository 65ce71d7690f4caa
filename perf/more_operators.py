"""Cases of the layer's attention core, of the norm in front of an 8-bit block and of its
gradients' clipping: what to run, at which sizes, and what each operator computes, written out.

Four operators, each with a plain form of elementary torch operations (``own`` false) and
the library's own call (``own`` true):

* ``forward``   softmax attention over packed sequences, with the logarithms of the rows' sums;
* ``backward``  its gradients from the forward's outputs, probabilities regenerated (``step``
                is both, as a short training step runs them);
* ``norm``      the residual added, the sum's root-mean-square scale, and its values in 8-bit
                floating point with a power-of-two scale for each block of 128;
* ``clip``      the norm over all gradients of a model, and the gradients scaled down to it.

Sequence s has the queries [q_starts[s], q_starts[s + 1]) and the keys [k_starts[s],
k_starts[s + 1]). With ``causal`` its last query sees all its keys, the one before all but the
last, and so on, so that more queries than keys leave the first ones without any: their output
and their gradients are 0, their logarithm -inf. Rows behind the last sequence stay as they were.

Scale bytes hold the exponent plus 127 and lie in tiles of 128 rows x 4 blocks: the byte
of row r, block b is at ((r // 128) * ceil(blocks / 4) + b // 4) * 512 + (r % 32) * 16 +
(r // 32 % 4) * 4 + b % 4; bytes of rows and blocks outside the operand are 127.
"""

import math

import torch

own = False

EPS = 1e-5
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA = {"e4m3": 3, "e5m2": 2}
LOWEST = {"e4m3": -6, "e5m2": -14}      # exponent of the smallest normal value
DTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------------------- cases
def _attention(name, op, lengths, hq, hk, D, causal, packed, tail=0):
    return dict(name=name, op=op, lengths=lengths, hq=hq, hk=hk, D=D, causal=causal,
                packed=packed, tail=tail)


def listed():
    return [
        # a decoding step: one new token each of eight sequences over their long contexts, key
        # heads shared by five query heads
        _attention("attention_token", "forward", ",".join(
            f"1:{n}" for n in (8192, 4097, 16384, 63, 12007, 1, 9999, 8191)), 40, 8, 128, True, False),
        # the attention core of the 4096-wide layer at the benchmark's token count
        _attention("attention_layer", "forward", ",".join(["4096:4096"] * 4), 32, 32, 128, True,
                   False),
        # a chunk of new tokens behind contexts of any length, odd sizes, a packed projection
        _attention("attention_chunk", "forward", "1000:3001,77:77,1:2500,515:4111,200:129,3:0", 40,
                   8, 128, True, True, 5),
        # a short fine-tuning batch of the 2048-wide layer, forward and backward
        _attention("attention_short", "step", "77:77", 16, 16, 128, True, True),
        # the gradients of the 2048-wide layer's attention core at the benchmark's token count
        _attention("attention_grad", "backward", ",".join(["4096:4096"] * 4), 16, 16, 128, True,
                   False),
        # gradients of shared key heads, ragged sequences, no causal mask, narrower heads
        _attention("attention_grad_shared", "backward", "2047:2047,513:1030,1:77,1291:1291", 24, 8,
                   96, False, True, 3),
        # one token of the 2048-wide layer
        dict(name="norm_token", op="norm", T=1, d=2048, fmt="e4m3", residual=True, gamma=False),
        # the second norm of the 4096-wide layer at the benchmark's token count
        dict(name="norm_layer", op="norm", T=16384, d=4096, fmt="e4m3", residual=True, gamma=False),
        # the 5120-wide layer's first norm with its weight applied here, an odd token count
        dict(name="norm_weighted", op="norm", T=8191, d=5120, fmt="e5m2", residual=False, gamma=True),
        # the gradients of the 2048-wide attention block
        dict(name="clip_block", op="clip", d=2048, r=512, ffn=0, layers=1, odd=0, wide=False,
             most=1.0),
        # those of one 5120-wide layer
        dict(name="clip_layer", op="clip", d=5120, r=1280, ffn=13824, layers=1, odd=0, wide=False,
             most=1.0),
        # many tensors, in 32 bits as they are accumulated over steps, odd ones among them
        dict(name="clip_model", op="clip", d=1024, r=256, ffn=2752, layers=24, odd=50257, wide=True,
             most=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "step", "norm", "clip"])
    if op == "norm":
        d = 8 * _log(rng, 8, 1376)
        return dict(op=op, T=min(_log(rng, 1, 16384), (1 << 26) // d), d=d,
                    fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), residual=rng.random() < 0.7,
                    gamma=rng.random() < 0.3)
    if op == "clip":
        return dict(op=op, d=8 * _log(rng, 8, 256), r=8 * _log(rng, 4, 64), ffn=8 * _log(rng, 8, 512),
                    layers=_log(rng, 1, 24), odd=_log(rng, 1, 100000), wide=rng.random() < 0.5,
                    most=rng.choice([0.1, 1.0, 1.0, 1e6]))
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 1, 2, 3, 4])
    one = op == "forward" and rng.random() < 0.3      # a decoding step
    lengths, left = [], 8e8 / hq                      # scores of one head, all sequences
    longest_q = longest_k = 1
    for _ in range(rng.choice([1, 1, 2, 3, 4, 7])):
        nk = _log(rng, 1, 8192)
        nq = 1 if one else nk if rng.random() < 0.6 else _log(rng, 1, 4096)
        nk = rng.choice([nk] * 9 + [0])
        longest = max(longest_q, nq) * max(longest_k, nk)
        if longest * (len(lengths) + 1) > left and lengths:
            break
        while nq * nk > left:
            nq, nk = max(1, nq // 2), max(1, nk // 2)
        longest_q, longest_k = max(longest_q, nq), max(longest_k, nk)
        lengths.append(f"{nq}:{nk}")
    return dict(op=op, lengths=",".join(lengths), hq=hq, hk=hk,
                D=rng.choice([40, 64, 64, 72, 80, 96, 128, 128, 128]), causal=rng.random() < 0.7,
                packed=rng.random() < 0.5, tail=rng.choice([0, 0, 1, 130]))


def _lengths(c):
    return [tuple(map(int, p.split(":"))) for p in c["lengths"].split(",")]


def _shapes(c):
    """The gradients of ``layers`` layers of bottleneck blocks (``ffn`` 0: the QKV block alone)
    and one tensor of ``odd`` values."""
    d, r, n = c["d"], c["r"], c["ffn"]
    layer = [(d,), (d, 3 * r), (3, r, d)]
    if n:
        layer += [(d, r), (r, d), (d,), (d, 2 * r), (2, r, n), (n, r), (r, d)]
    return layer * c["layers"] + ([(c["odd"],)] if c["odd"] else [])


# ------------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    if c["op"] == "norm":
        shape = (c["T"], c["d"])
        # rows of different magnitude, as a residual stream has them
        x = torch.randn(shape, generator=g, device="cuda")
        x = x * torch.exp2(torch.randint(-3, 4, (c["T"], 1), generator=g, device="cuda").float())
        gamma = _normal(g, (c["d"],), 0.1) + 1 if c["gamma"] else None
        return dict(case=c, x=x.to(torch.bfloat16), gamma=gamma,
                    residual=_normal(g, shape) if c["residual"] else None)
    if c["op"] == "clip":
        dtype = torch.float32 if c["wide"] else torch.bfloat16
        grads = [_normal(g, s, 0.01, dtype) for s in _shapes(c)]
        # (scaled into a buffer of their own, so that a pass finds the gradients as they were)
        flat = torch.empty(sum(t.numel() for t in grads), dtype=dtype, device="cuda")
        outs = [o.view(t.shape) for o, t in zip(flat.split([t.numel() for t in grads]), grads)]
        return dict(case=c, grads=grads, flat=flat, outs=outs)
    lengths = _lengths(c)
    hq, hk, D = c["hq"], c["hk"], c["D"]
    starts = torch.tensor([(0, 0)] + lengths).cumsum(0).to(torch.int32).cuda()
    Tq, Tk = sum(n for n, _ in lengths) + c["tail"], sum(n for _, n in lengths) + c["tail"]
    # heads of different sharpness: the spread of a row's scores is 0.5 to 4
    sharp = torch.exp2(torch.rand((hq, 1), generator=g, device="cuda") * 3 - 1).to(torch.bfloat16)
    if c["packed"]:     # heads side by side in a token's row
        q = torch.cat([_normal(g, (Tq, hq, D)) * sharp, _normal(g, (Tq, 2, D))], 1)[:, :hq]
        k, v = _normal(g, (Tk, 2, hk, D)).unbind(1)
    else:               # planes of their own
        q, k, v = _normal(g, (Tq, hq, D)) * sharp, _normal(g, (Tk, hk, D)), _normal(g, (Tk, hk, D))
    zeros = torch.zeros_like
    s = dict(case=c, q=q, k=k, v=v, q_starts=starts[:, 0].contiguous(),
             k_starts=starts[:, 1].contiguous(), longest=tuple(max(n) for n in zip(*lengths)),
             out=zeros(q).contiguous(), lse=torch.zeros(hq, Tq, device="cuda"))
    if c["op"] != "forward":
        s.update(dout=_normal(g, (Tq, hq, D)), dq=zeros(s["out"]), dk=zeros(k).contiguous(),
                 dv=zeros(v).contiguous())
    if c["op"] == "backward":       # what the forward has left
        s["saved"] = forward_plain(s)
    return s


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["d"]
        return {"bytes": n * (2 + 129 / 128 + (4 if c["residual"] else 0)) + 4 * c["T"], "flops": 6 * n}
    if c["op"] == "clip":
        n = sum(math.prod(s) for s in _shapes(c))
        return {"bytes": (8 if c["wide"] else 4) * n, "flops": 3 * n}
    lengths = _lengths(c)
    hq, hk, D = c["hq"], c["hk"], c["D"]
    rows, keys = sum(n for n, _ in lengths), sum(n for _, n in lengths)
    pairs = sum(sum(max(0, k - n + 1 + i) for i in range(n)) if c["causal"] else n * k
                for n, k in lengths)
    products = {"forward": 2, "backward": 5, "step": 7}[c["op"]]
    ins, outs = 2 * rows * hq * D, 4 * keys * hk * D          # q; k and v
    moved = {"forward": 2 * ins + outs, "backward": 4 * ins + 2 * outs, "step": 5 * ins + 2 * outs}
    return {"bytes": moved[c["op"]] + 4 * rows * hq, "flops": 2 * products * pairs * hq * D}


# ----------------------------------------------------------------------- plain forms
def _padded(t, starts, longest):
    """[sequences, heads, longest, D] in 32 bits of packed [T, heads, D], with where each row
    comes from and whether it is one."""
    t = t if t.shape[0] else t.new_zeros((1,) + t.shape[1:])      # (no rows at all)
    at = starts[:-1, None] + torch.arange(longest, device=t.device)
    inside = at < starts[1:, None]
    at = torch.where(inside, at, 0)
    rows = torch.where(inside[..., None, None], t[at].float(), 0.0)
    return rows.transpose(1, 2), at, inside


def _packed(rows, at, inside, like):
    """Back to [T, heads, D] as `like`; rows of no sequence 0."""
    out = torch.zeros(like.shape, dtype=like.dtype, device=like.device)
    out[at[inside]] = rows.transpose(1, 2)[inside].to(like.dtype)
    return out


def _scores(s):
    """Scaled scores [sequences, hk, hq / hk, queries, keys], -inf where a query does not see a
    key, and the padded operands."""
    c = s["case"]
    longest_q, longest_k = s["longest"]
    q, at_q, in_q = _padded(s["q"], s["q_starts"], longest_q)
    k, at_k, in_k = _padded(s["k"], s["k_starts"], max(longest_k, 1))
    v = _padded(s["v"], s["k_starts"], max(longest_k, 1))[0]
    q = q.unflatten(1, (c["hk"], c["hq"] // c["hk"]))
    x = q @ k[:, :, None].mT * c["D"] ** -0.5
    seen = in_q[:, :, None] & in_k[:, None]
    if c["causal"]:
        behind = (s["k_starts"] - s["q_starts"]).diff()[:, None, None]
        i = torch.arange(x.shape[-2], device=x.device)[:, None]
        seen = seen & (torch.arange(x.shape[-1], device=x.device) <= i + behind)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    return x, q, k[:, :, None], v[:, :, None], (at_q, in_q), (at_k, in_k)


def forward_plain(s):
    x, _, _, v, rows, _ = _scores(s)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v / torch.where(total == 0, 1.0, total)).flatten(1, 2)
    lse = (top + torch.log(total)).flatten(1, 2)
    lse_out = torch.zeros(s["lse"].shape, device=o.device)
    lse_out[:, rows[0][rows[1]]] = lse[..., 0].transpose(1, 2)[rows[1]].T
    return _packed(o, *rows, s["out"]), lse_out


def backward_plain(s, out, lse):
    c = s["case"]
    x, q, k, v, rows, keys = _scores(s)
    lse = _padded(lse.T[..., None], s["q_starts"], x.shape[-2])[0].unflatten(1, q.shape[1:3])
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse))
    dout = _padded(s["dout"], s["q_starts"], x.shape[-2])[0].unflatten(1, q.shape[1:3])
    dv = (p.mT @ dout).sum(2)
    dp = dout @ v.mT
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * c["D"] ** -0.5
    dq, dk = (ds @ k).flatten(1, 2), (ds.mT @ q).sum(2)
    return (_packed(dq, *rows, s["dq"]), _packed(dk, *keys, s["dk"]), _packed(dv, *keys, s["dv"]))


def pack_scales(e):
    """Scale bytes [rows, blocks] in tiles of 128 rows x 4 blocks."""
    rows, blocks = e.shape
    rt, bt = -(-rows // 128), -(-blocks // 4)
    full = torch.nn.functional.pad(e, (0, bt * 4 - blocks, 0, rt * 128 - rows), value=127)
    return full.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def norm_plain(x, residual, gamma, fmt):
    """(sum, 1 / rms of its rows, 8-bit values [T, pitch], scale bytes): the smallest power of
    two s, at least 2^-127, with max|block| <= s * FMAX; 1 for a block of zeros."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    y = h.float() if gamma is None else (h.float() * gamma.float()).to(x.dtype).float()
    T, d = y.shape
    blocks, pitch = -(-d // 128), -(-d // 16) * 16
    full = torch.nn.functional.pad(y, (0, blocks * 128 - d)).view(T, blocks, 128)
    largest = full.abs().amax(2)
    bits = largest.view(torch.int32)
    byte = (bits >> 23) - (8 if fmt == "e4m3" else 15) + ((bits & 0x7FFFFF) > 0x600000).int()
    byte = torch.where(largest == 0, 127, byte.clamp(min=0)).to(torch.uint8)
    scale = ((254 - byte.int()) << 23).view(torch.float32)[:, :, None]
    q = (full * scale).view(T, blocks * 128)[:, :pitch].to(DTYPE[fmt])
    return h, rstd, q.contiguous(), pack_scales(byte)


def clip_plain(grads, most, outs):
    """Norm over all; gradients times min(1, most / (norm + 1e-6)) into outs."""
    # (a sum of many squares: 64 bits)
    norm = torch.stack([t.double().square().sum() for t in grads]).sum().sqrt()
    by = torch.clamp(most / (norm + 1e-6), max=1.0).float()
    _ = [torch.mul(t.float(), by, out=o) for t, o in zip(grads, outs)]
    return norm.float().view(1)


def run(state):
    return (run_own if own else run_plain)(state, state["case"])


def run_plain(s, c):
    if c["op"] == "norm":
        return norm_plain(s["x"], s["residual"], s["gamma"], c["fmt"])
    if c["op"] == "clip":
        return clip_plain(s["grads"], c["most"], s["outs"]), s["flat"]
    if c["op"] == "backward":
        return backward_plain(s, *s["saved"])
    out, lse = forward_plain(s)
    return (out, lse) if c["op"] == "forward" else (out, lse, *backward_plain(s, out, lse))


def run_own(s, c):
    from rank_bottleneck_online_gb300 import binding as B
    if c["op"] == "norm":
        h, rstd, (q, scales) = B.norm_quantize(s["x"], residual=s["residual"], gamma=s["gamma"],
                                               eps=EPS, fmt=c["fmt"])
        return h, rstd, q, scales
    if "ws" not in s:       # the workspace that a program keeps beside its weights
        s["ws"] = B.Workspace(B.grad_clip_workspace_bytes() if c["op"] == "clip" else
                              B.attention_workspace_bytes(s["q"].shape[0], s["k"].shape[0], c["hq"],
                                                          c["hk"], c["D"], len(s["q_starts"]) - 1))
    if c["op"] == "clip":
        return B.grad_clip(s["grads"], c["most"], s["ws"], outs=s["outs"]), s["flat"]
    args = dict(causal=c["causal"], q_starts=s["q_starts"], k_starts=s["k_starts"])
    qkv = s["q"], s["k"], s["v"]
    if c["op"] == "backward":
        out, lse = s["saved"]
    else:
        out, lse = B.attention(*qkv, s["ws"], out=s["out"], lse=s["lse"], **args)
        if c["op"] == "forward":
            return out, lse
    grads = B.attention_bwd(*qkv, out, lse, s["dout"], s["ws"], dq=s["dq"], dk=s["dk"], dv=s["dv"],
                            **args)
    return grads if c["op"] == "backward" else (out, lse, *grads)


# ------------------------------------------------------------------- definitions, 64 bits
def _attention_exact(s, c):
    """Head by head of each sequence, over the keys of each query alone."""
    group, scale = c["hq"] // c["hk"], 1.0 / math.sqrt(c["D"])
    found = {name: torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
             for name in ("out", "lse", "dq", "dk", "dv") if name in s}
    q0 = k0 = 0
    for n, m in _lengths(c):
        rows, keys = slice(q0, q0 + n), slice(k0, k0 + m)
        q0, k0 = q0 + n, k0 + m
        hidden = torch.zeros(n, m, dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        none = hidden.all(1)
        for h in range(c["hq"]):
            q, k, v = (t.double() for t in (s["q"][rows, h], s["k"][keys, h // group],
                                            s["v"][keys, h // group]))
            x = (q @ k.T * scale).masked_fill(hidden, -math.inf)
            found["lse"][h, rows] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1).masked_fill(none[:, None], 0.0)
            o = p @ v
            found["out"][rows, h] = o
            if c["op"] == "forward":
                continue
            do = s["dout"][rows, h].double()
            ds = p * (do @ v.T - (do * o).sum(1, keepdim=True)) * scale
            found["dq"][rows, h] = ds @ k
            found["dk"][keys, h // group] += ds.T @ q
            found["dv"][keys, h // group] += p.T @ do
    return tuple(found[name] for name in ("out", "lse", "dq", "dk", "dv")
                 if name in found and (c["op"] != "backward" or name[0] == "d"))


def _two_to(e):
    """2^e in 64 bits, from the bits of the format (pow and exp2 need not be exact)."""
    return (e.to(torch.int64) + 1023 << 52).view(torch.float64)


def _norm_exact(s, c):
    h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    r = h.to(torch.bfloat16).double()         # the sum is stored: its scale and values are its
    rstd = 1.0 / torch.sqrt((r * r).sum(1) / c["d"] + EPS)
    y = r if s["gamma"] is None else (r * s["gamma"].double()).to(torch.bfloat16).double()
    T, d = y.shape
    blocks, pitch = -(-d // 128), -(-d // 16) * 16
    full = torch.zeros(T, blocks * 128, dtype=torch.float64, device="cuda")
    full[:, :d] = y
    tiles = full.view(T, blocks, 128)
    m, e = torch.frexp(tiles.abs().amax(2, keepdim=True) / FMAX[c["fmt"]])
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-127)
    v = tiles * _two_to(torch.where(m == 0, 0, -e))
    step = _two_to((torch.frexp(v)[1] - 1).clamp(min=LOWEST[c["fmt"]]) - MANTISSA[c["fmt"]])
    return h, rstd, (torch.round(v / step) * step).view(T, -1)[:, :pitch].contiguous(), None


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        return _norm_exact(s, c)
    if c["op"] == "clip":
        norm = math.sqrt(sum(float((t.double() ** 2).sum()) for t in s["grads"]))
        by = min(1.0, c["most"] / (norm + 1e-6))
        return (torch.tensor([norm], dtype=torch.float64),
                torch.cat([t.double().view(-1) * by for t in s["grads"]]))
    return _attention_exact(s, c)
