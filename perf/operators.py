"""The expert feed-forward operators, as they are measured.

Five operators of the MXFP4 expert layer: the gated gate_up product (dense and
grouped by expert), its backward pass (the down projection's data gradient with
the activation's derivative), the int8 token quantizer, the int8 product with
token and channel scales, and dropout from the counter-based generator.  `run`
computes each in elementary torch operations, or, where `own` is true, by the
framework's entry points.  Sizes follow the expert layer this framework is
built around (hidden 2880, gate_up 5760, 32 experts, top-4) or are generic.
"""
import math
import random

import torch

own = False

HIDDEN, INTER, EXPERTS, TOPK = 2880, 2880, 32, 4
# activation: h = g s(alpha g) (u + beta) with g = min(gate, limit), u = up clamped to +-limit
CLAMPED = {"alpha": 1.702, "limit": 7.0, "beta": 1.0}   # the clamped form of the repository's expert layer
SWIGLU = {"alpha": 1.0, "limit": math.inf, "beta": 0.0}
DROPOUT_TAG = 0x44524F50
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the gate_up projection: decoding, where latency counts
        {"name": "gated_1_token", "op": "gated", "m": 1, "k": HIDDEN, "i": INTER, "groups": 0, "clamped": True, "z": False},
        # a ragged batch of prompts at sizes that fill no tile
        {"name": "gated_333_odd", "op": "gated", "m": 333, "k": 1472, "i": 1112, "groups": 0, "clamped": False, "z": False},
        # a training batch: h for the down projection, z kept for the backward pass
        {"name": "gated_4096_train", "op": "gated", "m": 4096, "k": HIDDEN, "i": INTER, "groups": 0, "clamped": True, "z": True},
        # 16384 tokens routed to 4 of 32 experts, skewed as routers are: the largest call
        {"name": "gated_moe_65536", "op": "gated", "m": 65536, "k": HIDDEN, "i": INTER, "groups": EXPERTS, "clamped": True, "z": True},
        # the backward pass of the training batch
        {"name": "gated_bwd_4096", "op": "gated_bwd", "m": 4096, "k": HIDDEN, "i": INTER, "groups": 0, "clamped": True},
        # the backward pass of a ragged batch over a few experts, one of them empty
        {"name": "gated_bwd_moe_2999", "op": "gated_bwd", "m": 2999, "k": 1472, "i": 1112, "groups": 7, "clamped": False},
        # the activations of a training batch into 8-bit tokens
        {"name": "int8_tokens_4096", "op": "int8_quantize", "m": 4096, "k": INTER},
        # a prefill's worth of wide rows
        {"name": "int8_tokens_16384_wide", "op": "int8_quantize", "m": 16384, "k": 11520},
        # one token through the 8-bit down projection
        {"name": "int8_gemm_1_token", "op": "int8_gemm", "m": 1, "n": HIDDEN, "k": INTER, "groups": 0, "f32": False},
        # the down projection of a training batch or long prompt
        {"name": "int8_gemm_4096", "op": "int8_gemm", "m": 4096, "n": HIDDEN, "k": INTER, "groups": 0, "f32": False},
        # the block's output onto the residual stream
        {"name": "dropout_residual_4096", "op": "dropout", "m": 4096, "n": HIDDEN, "p": 0.1, "residual": True, "f32": False},
        # the gradient of a large batch through the same mask
        {"name": "dropout_grad_65536", "op": "dropout", "m": 65536, "n": HIDDEN, "p": 0.1, "residual": False, "f32": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "int8_quantize", "int8_gemm", "dropout"])
    if op == "int8_quantize":
        k = 16 * _log(rng, 1, 720)
        return {"op": op, "m": _log(rng, 1, min(65536, 180_000_000 // k)), "k": k}
    if op == "dropout":
        n = _log(rng, 1, 11520)
        return {"op": op, "m": _log(rng, 1, min(65536, 180_000_000 // n)), "n": n, "p": rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]),
                "residual": rng.random() < 0.5, "f32": rng.random() < 0.25}
    groups = rng.choice([0, 0, rng.randint(1, EXPERTS)])
    m = _log(rng, 1, 16384)
    if op == "int8_gemm":
        return {"op": op, "m": m, "n": 8 * _log(rng, 4, 720), "k": 16 * _log(rng, 4, 360), "groups": groups, "f32": rng.random() < 0.3}
    case = {"op": op, "m": m, "k": 64 * _log(rng, 1, 90), "i": 8 * _log(rng, 4, 360), "groups": groups, "clamped": rng.random() < 0.5}
    if op == "gated":
        case["z"] = rng.random() < 0.5
    return case


# -------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + salt)
    return g


def _activations(rows, cols, seed, salt, std=1.0):
    """N(0, std^2) with 1% of the columns 20 times larger, as activations have them."""
    g = _gen(seed, salt)
    x = torch.randn((rows, cols), generator=g, device="cuda") * std
    loud = torch.rand((cols,), generator=g, device="cuda") < 0.01
    x[:, loud] *= 20.0
    return x


def _to_mxfp4(x):
    """Codes (two per byte, low nibble first) and scale codes of blocks of 32 along
    the rows: the scale is the power of two below the largest magnitude, over 4."""
    rows, k = x.shape
    b = x.view(rows, k // 32, 32)
    e = (b.abs().amax(-1).view(torch.int32) >> 23) - 2
    e = e.clamp(1, 252)
    v = b * ((254 - e) << 23).view(torch.float32).unsqueeze(-1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(v.abs().contiguous(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(rows, k)
    return code[:, 0::2] | (code[:, 1::2] << 4), e.to(torch.uint8)


def _gemm_ready(scales, k):
    """Row-major scale codes [rows, k/32] in the order the GEMMs read them: 512-byte
    atoms of 128 rows x 4 blocks."""
    rows, nb = scales.shape
    atoms = (nb + 3) // 4
    tiles = (rows + 127) // 128
    full = torch.zeros((tiles * 128, atoms * 4), dtype=torch.uint8, device=scales.device)
    full[:rows, :nb] = scales
    return full.view(tiles, 4, 32, atoms, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _weights(n, k, groups, seed):
    """Weights N(0, 0.02^2) in MXFP4: codes [G, n, k/2], row-major scales [G, n, k/32], GEMM-ready scales."""
    codes, scales, ready = [], [], []
    for e in range(max(groups, 1)):
        w = torch.randn((n, k), generator=_gen(seed, 100 + e), device="cuda") * 0.02
        c, s = _to_mxfp4(w)
        codes.append(c)
        scales.append(s)
        ready.append(_gemm_ready(s, k))
    return torch.stack(codes), torch.stack(scales), torch.cat(ready)


def _groups(m, groups, seed):
    """(sizes, offsets) of m routed rows over the experts, skewed as a router's are:
    each expert starts on a multiple of 128 rows; the last of several is empty."""
    r = random.Random(seed)
    share = [(e + 1) ** -1.2 for e in range(groups)]
    if groups > 1:
        share[-1] = 0.0
    r.shuffle(share)
    total = sum(share)
    sizes = [int(m * s / total) for s in share]
    sizes[share.index(max(share))] += m - sum(sizes)
    offsets = [0]
    for s in sizes:
        offsets.append(offsets[-1] + (s + 127) // 128 * 128)
    return sizes, offsets


def prepare(case, seed):
    c = dict(case)
    op, m = c["op"], c["m"]
    st = {"case": c}
    if op == "int8_quantize":
        st["x"] = _activations(m, c["k"], seed, 1).to(torch.bfloat16)
        return st
    if op == "dropout":
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        st["x"] = _activations(m, c["n"], seed, 1).to(dtype)
        st["residual"] = _activations(m, c["n"], seed, 2, 3.0).to(dtype) if c["residual"] else None
        st["seed"] = (seed * 0x9E3779B97F4A7C15 + 1) & 0xFFFFFFFFFFFFFFFF
        return st
    rows = m
    if c["groups"]:
        st["sizes"], st["offsets"] = _groups(m, c["groups"], seed)
        rows = max(st["offsets"][-1], 128)
        st["d_sizes"] = torch.tensor(st["sizes"], dtype=torch.int32, device="cuda")
        st["d_offsets"] = torch.tensor(st["offsets"], dtype=torch.int32, device="cuda")
    k = c["k"]
    if op == "int8_gemm":
        # codes as a token and channel quantizer leaves them: bell-shaped, the largest of a row at 127
        st["a"] = (torch.randn((rows, k), generator=_gen(seed, 1), device="cuda") * 32).round().clamp(-127, 127).to(torch.int8)
        st["a_scales"] = torch.rand((rows,), generator=_gen(seed, 2), device="cuda") * 0.05 + 0.005
        g = max(c["groups"], 1)
        st["b"] = (torch.randn((g, c["n"], k), generator=_gen(seed, 3), device="cuda") * 32).round().clamp(-127, 127).to(torch.int8)
        st["b_scales"] = torch.rand((g, c["n"]), generator=_gen(seed, 4), device="cuda") * 5e-4 + 1e-4
        if c["groups"]:
            st["out"] = torch.zeros((rows, c["n"]), dtype=torch.float32 if c["f32"] else torch.bfloat16, device="cuda")
        else:
            st["b"], st["b_scales"] = st["b"][0], st["b_scales"][0]
        return st
    std = 1.0 if op == "gated" else 1e-2
    st["a"], st["a_rows"] = _to_mxfp4(_activations(rows, k, seed, 1, std))
    st["a_scales"] = _gemm_ready(st["a_rows"], k)
    n = 2 * c["i"] if op == "gated" else c["i"]
    st["b"], st["b_rows"], st["b_scales"] = _weights(n, k, c["groups"], seed)
    if not c["groups"]:
        st["b"], st["b_rows"] = st["b"][0], st["b_rows"][0]
    if op == "gated_bwd":
        # pre-activations of both signs, some past the clamp
        st["z"] = (torch.randn((rows, 2 * c["i"]), generator=_gen(seed, 9), device="cuda") * 3.0).to(torch.bfloat16)
    if c["groups"]:  # rows between the experts stay as they are
        if op == "gated":
            st["h"] = torch.zeros((rows, c["i"]), dtype=torch.bfloat16, device="cuda")
            st["z"] = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda") if c["z"] else None
        else:
            st["dz"] = torch.zeros((rows, 2 * c["i"]), dtype=torch.bfloat16, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms
def _decode(codes, scales):
    grid = torch.tensor(GRID + [-v for v in GRID], device=codes.device)
    v = grid[torch.stack((codes & 15, codes >> 4), -1).int()]
    v = v.view(codes.shape[0], scales.shape[1], 32) * (scales.int() << 23).view(torch.float32).unsqueeze(-1)
    return v.view(codes.shape[0], 2 * codes.shape[1])


def _per_group(st, a_of, b_of, rows):
    """The product of each expert's rows with its weights; zero rows between them."""
    if not st["case"]["groups"]:
        return a_of(slice(None)) @ b_of(None).t()
    spans = list(zip(range(len(st["sizes"])), st["offsets"], st["sizes"], st["offsets"][1:]))
    parts = [torch.nn.functional.pad(a_of(slice(o, o + s)) @ b_of(g).t(), (0, 0, 0, nxt - o - s)) for g, o, s, nxt in spans]
    full = torch.cat(parts)
    return torch.nn.functional.pad(full, (0, 0, 0, rows - full.shape[0]))


def _mx_product(st):
    pick = lambda t, g: t if g is None else t[g]  # noqa: E731
    return _per_group(st, lambda r: _decode(st["a"][r], st["a_rows"][r]),
                      lambda g: _decode(pick(st["b"], g), pick(st["b_rows"], g)), st["a"].shape[0])


def _valid_rows(st, rows):
    at = torch.arange(rows, device="cuda")
    seg = torch.bucketize(at, st["d_offsets"][1:].long(), right=True).clamp(max=len(st["sizes"]) - 1)
    return at < st["d_offsets"].long()[seg] + st["d_sizes"].long()[seg]


def _gated_plain(st):
    c, act = st["case"], CLAMPED if st["case"]["clamped"] else SWIGLU
    z = _mx_product(st)
    g = z[:, 0::2].clamp(max=act["limit"])
    u = z[:, 1::2].clamp(-act["limit"], act["limit"])
    h = g / (1 + torch.exp(-act["alpha"] * g)) * (u + act["beta"])
    return [h.to(torch.bfloat16)] + ([z.to(torch.bfloat16)] if c["z"] else [])


def _gated_bwd_plain(st):
    act = CLAMPED if st["case"]["clamped"] else SWIGLU
    dh = _mx_product(st)
    zg, zu = st["z"][:, 0::2].float(), st["z"][:, 1::2].float()
    g, u = zg.clamp(max=act["limit"]), zu.clamp(-act["limit"], act["limit"])
    s = 1 / (1 + torch.exp(-act["alpha"] * g))
    dg = dh * (u + act["beta"]) * s * (1 + act["alpha"] * g * (1 - s)) * (zg <= act["limit"])
    du = dh * g * s * (zu.abs() <= act["limit"])
    dz = torch.stack((dg, du), -1).view(dh.shape[0], -1)
    if st["case"]["groups"]:
        dz = dz * _valid_rows(st, dz.shape[0]).unsqueeze(-1)
    return [dz.to(torch.bfloat16)]


def _int8_quantize_plain(st):
    x = st["x"].float()
    a = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    return [(x * (127.0 / a)).round().to(torch.int8), (a / 127.0).squeeze(-1)]


def _int8_gemm_plain(st):
    pick = lambda t, g: t if g is None else t[g]  # noqa: E731
    c = _per_group(st, lambda r: st["a"][r].float(), lambda g: pick(st["b"], g).float(), st["a"].shape[0])
    c = c * st["a_scales"].unsqueeze(-1)
    if st["case"]["groups"]:
        at = torch.bucketize(torch.arange(c.shape[0], device="cuda"), st["d_offsets"][1:].long(), right=True)
        c = c * st["b_scales"][at.clamp(max=len(st["sizes"]) - 1)]
    else:
        c = c * st["b_scales"]
    return [c if st["case"]["f32"] else c.to(torch.bfloat16)]


def _round(c, keys):
    p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
    low = 0xFFFFFFFF
    return ((p1 >> 32) & low) ^ c[1] ^ keys[0], p1 & low, ((p0 >> 32) & low) ^ c[3] ^ keys[1], p0 & low


def _philox_words(n, seed):
    """Philox4x32-10 words of elements 0 .. n-1: word g mod 4 of the counter (g / 4, 0, tag)."""
    at = torch.arange((n + 3) // 4, device="cuda", dtype=torch.int64)
    c = (at, torch.zeros_like(at), torch.zeros_like(at), torch.full_like(at, DROPOUT_TAG))
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    keys = [((k0 + r * 0x9E3779B9) & 0xFFFFFFFF, (k1 + r * 0xBB67AE85) & 0xFFFFFFFF) for r in range(10)]
    c = _round(_round(_round(_round(_round(c, keys[0]), keys[1]), keys[2]), keys[3]), keys[4])
    c = _round(_round(_round(_round(_round(c, keys[5]), keys[6]), keys[7]), keys[8]), keys[9])
    return torch.stack(c, -1).view(-1)[:n]


def _dropout_plain(st):
    x, p = st["x"], st["case"]["p"]
    keep = (_philox_words(x.numel(), st["seed"]) >= round(p * 2 ** 32)).view(x.shape)
    y = torch.where(keep, x.float() * (1.0 / (1.0 - p)), 0.0)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return [y.to(x.dtype)]


PLAIN = {"gated": _gated_plain, "gated_bwd": _gated_bwd_plain, "int8_quantize": _int8_quantize_plain,
         "int8_gemm": _int8_gemm_plain, "dropout": _dropout_plain}


# ------------------------------------------------------- the framework's calls
def _own(st):
    import quantize_block_scaled_rht_b200 as mx
    c = st["case"]
    op, k = c["op"], c.get("k")
    if op == "int8_quantize":
        q = mx.mxfp4_int8_quantize(st["x"])
        return [q.codes, q.scales]
    if op == "dropout":
        return [mx.mxfp4_dropout(st["x"], c["p"], st["seed"], residual=st["residual"])]
    if op == "int8_gemm":
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        if c["groups"]:
            return [mx.mxfp4_int8_grouped_gemm(st["a"], st["a_scales"], st["d_offsets"], st["d_sizes"], st["b"], st["b_scales"],
                                               out=st["out"])]
        return [mx.mxfp4_int8_gemm(st["a"], st["a_scales"], st["b"], st["b_scales"], out_dtype=dtype)]
    act = CLAMPED if c["clamped"] else SWIGLU
    if op == "gated":
        if c["groups"]:
            h, z = mx.mxfp4_grouped_gated_gemm(st["a"], st["a_scales"], st["d_offsets"], st["d_sizes"], st["b"], st["b_scales"], k,
                                               **act, save_z=c["z"], out=st["h"], z_out=st["z"])
        else:
            h, z = mx.mxfp4_gated_gemm(st["a"], st["a_scales"], st["b"], st["b_scales"], k, **act, save_z=c["z"])
        return [h, z] if c["z"] else [h]
    if c["groups"]:
        return [mx.mxfp4_grouped_gated_gemm_backward(st["a"], st["a_scales"], st["d_offsets"], st["d_sizes"], st["b"], st["b_scales"],
                                                     st["z"], k, **act, out=st["dz"])]
    return [mx.mxfp4_gated_gemm_backward(st["a"], st["a_scales"], st["b"], st["b_scales"], st["z"], k, **act)]


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- the work
def work(case):
    c = case
    op, m, k = c["op"], c["m"], c.get("k", 0)
    if op == "int8_quantize":
        return {"bytes": m * k * 3 + 4 * m, "flops": 2 * m * k}
    if op == "dropout":
        return {"bytes": m * c["n"] * (4 if c["f32"] else 2) * (3 if c["residual"] else 2), "flops": 2 * m * c["n"]}
    # an empty expert's weights are not read
    g = max(c["groups"] - 1, 1)
    if op == "int8_gemm":
        n = c["n"]
        return {"bytes": m * k + g * n * k + 4 * (m + g * n) + m * n * (4 if c["f32"] else 2), "flops": 2 * m * n * k}
    n = 2 * c["i"] if op == "gated" else c["i"]
    operands = (m + g * n) * k * 17 / 32
    if op == "gated":
        return {"bytes": operands + 2 * m * c["i"] + (2 * m * n if c["z"] else 0), "flops": 2 * m * n * k}
    return {"bytes": operands + 2 * 2 * m * 2 * c["i"], "flops": 2 * m * n * k}


# ------------------------------------------------- from the definition, 64 bits
def _value64(codes, scales):
    """E2M1 by its fields: exponent 0 gives mantissa / 2, exponent e gives 2^(e-1) (1 + mantissa / 2)."""
    nib = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int32, device=codes.device)
    nib[:, 0::2] = codes.int() % 16
    nib[:, 1::2] = codes.int() // 16
    e, mant, sign = (nib // 2) % 4, (nib % 2).double(), 1.0 - 2.0 * (nib // 8).double()
    mag = torch.where(e == 0, mant / 2, torch.pow(2.0, (e - 1).double()) * (1 + mant / 2))
    x = torch.pow(2.0, scales.double() - 127.0)
    return sign * mag * x.repeat_interleave(32, dim=1)


def _spans(st):
    if not st["case"]["groups"]:
        return [(None, 0, st["a"].shape[0])]
    return [(g, o, s) for g, (o, s) in enumerate(zip(st["offsets"], st["sizes"])) if s]


def _act64(case):
    return (1.702, 7.0, 1.0) if case["clamped"] else (1.0, float("inf"), 0.0)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "int8_quantize":
        a = st["x"].double().abs().max(dim=1).values
        return [None, torch.clamp(a, min=2.0 ** -100) / 127]
    if op == "dropout":
        return [_dropout64(st)]
    rows = st["a"].shape[0]
    if op == "int8_gemm":
        out = torch.zeros((rows, case["n"]), dtype=torch.float64, device="cuda")
        for g, o, s in _spans(st):
            b, sb = (st["b"], st["b_scales"]) if g is None else (st["b"][g], st["b_scales"][g])
            out[o:o + s] = torch.matmul(st["a"][o:o + s].double(), b.double().transpose(0, 1))
            out[o:o + s] *= torch.outer(st["a_scales"][o:o + s].double(), sb.double())
        return [out]
    alpha, limit, beta = _act64(case)
    i = case["i"]
    if op == "gated":
        h = torch.zeros((rows, i), dtype=torch.float64, device="cuda")
        zs = torch.zeros((rows, 2 * i), dtype=torch.float64, device="cuda") if case["z"] else None
    else:
        dz = torch.zeros((rows, 2 * i), dtype=torch.float64, device="cuda")
    for g, o, s in _spans(st):
        b, bs = (st["b"], st["b_rows"]) if g is None else (st["b"][g], st["b_rows"][g])
        y = torch.matmul(_value64(st["a"][o:o + s], st["a_rows"][o:o + s]), _value64(b, bs).transpose(0, 1))
        if op == "gated":
            gate, up = torch.clamp(y[:, 0::2], max=limit), torch.clamp(y[:, 1::2], min=-limit, max=limit)
            h[o:o + s] = gate * torch.sigmoid(alpha * gate) * (up + beta)
            if zs is not None:
                zs[o:o + s] = y
        else:
            z = st["z"][o:o + s].double()
            gate, up = torch.clamp(z[:, 0::2], max=limit), torch.clamp(z[:, 1::2], min=-limit, max=limit)
            sg = torch.sigmoid(alpha * gate)
            dz[o:o + s, 0::2] = torch.where(z[:, 0::2] > limit, 0.0, y * (up + beta) * (sg + alpha * gate * sg * torch.sigmoid(-alpha * gate)))
            dz[o:o + s, 1::2] = torch.where(z[:, 1::2].abs() > limit, 0.0, y * gate * sg)
    if op == "gated":
        return [h] + ([zs] if zs is not None else [])
    return [dz]


def _mul_hi_lo(x, m):
    """High and low 32 bits of x * m from 16-bit pieces."""
    xl, xh, ml, mh = x % 65536, x // 65536, m % 65536, m // 65536
    mid = xh * ml + (xl * ml) // 65536
    mid2 = xl * mh + mid % 65536
    return xh * mh + mid // 65536 + mid2 // 65536, (mid2 % 65536) * 65536 + (xl * ml) % 65536


def _dropout64(st):
    x, p, seed = st["x"].double(), st["case"]["p"], st["seed"]
    n = x.numel()
    q = torch.arange((n + 3) // 4, device="cuda", dtype=torch.int64)
    w = [q % 2 ** 32, q // 2 ** 32, torch.zeros_like(q), torch.zeros_like(q) + DROPOUT_TAG]
    k = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        h0, l0 = _mul_hi_lo(w[0], 0xD2511F53)
        h1, l1 = _mul_hi_lo(w[2], 0xCD9E8D57)
        w = [h1 ^ w[1] ^ k[0], l1, h0 ^ w[3] ^ k[1], l0]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    drawn = torch.stack(w, 1).flatten()[:n].view(x.shape)
    y = torch.where(drawn < round(p * 2 ** 32), torch.zeros_like(x), x / (1.0 - p))
    return y if st["residual"] is None else y + st["residual"].double()
