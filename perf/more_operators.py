"""Cases and plain forms of the operators around the wrapped projections of an
attention layer: a frozen base in 4 bits (rows and weights stored and restored,
the projection's product on 4-bit weights with 8-bit or 4-bit rows), and the
norm of every query and key head with the position rotation, forward and back.

A run with own = False is elementary torch; with own = True it makes the
library's calls. Widths are those of the package's own workloads (2560,
19456 = 2 x 9728, 4096, 14336), heads of 64 and 128.
"""
import math

import torch

own = False

PANEL = 128  # columns of one panel of a 4-bit store
GROUP = 32   # columns that share a 4-bit scale
EPS = 1e-6


def listed():
    return [
        # a decode batch's activations stored in 4 bits and read back: launch latency
        {"name": "rows4_decode", "op": "rows4", "tokens": 256, "width": 2560},
        # the checkpoint of a wrapped projection in packed training
        {"name": "rows4_train", "op": "rows4", "tokens": 32768, "width": 4096},
        # a frozen weight stored once for the forward and for dX, both read back
        {"name": "weights4_gate_up", "op": "weights4", "rows": 19456, "width": 2560},
        # a single request's token through an attention projection
        {"name": "matmul4_one_token", "op": "matmul4", "x": "q8", "tokens": 1, "k": 2560, "n": 2560, "add": False},
        # a decode batch through the widest projection: the weights' bytes
        {"name": "matmul4_decode_gate_up", "op": "matmul4", "x": "q8", "tokens": 256, "k": 2560, "n": 19456, "add": False},
        # a few requests through the down projection, all operands in 4 bits: long sums, few rows
        {"name": "matmul4_down_ragged", "op": "matmul4", "x": "q4", "tokens": 37, "k": 9728, "n": 2560, "add": False},
        # a prefill chunk whose last tile is ragged, added to the residual rows
        {"name": "matmul4_prefill_add", "op": "matmul4", "x": "q8", "tokens": 8191, "k": 4096, "n": 4096, "add": True},
        # the MLP-up projection of a long mixed batch, all operands in 4 bits
        {"name": "matmul4_mlp_up", "op": "matmul4", "x": "q4", "tokens": 8192, "k": 4096, "n": 14336, "add": False},
        # a decode step's queries and keys: launch latency
        {"name": "qk_decode", "op": "qk", "tokens": 64, "heads_q": 32, "heads_k": 8, "dim": 128, "rot": 128, "pairs": "halves"},
        # those of a training batch
        {"name": "qk_train", "op": "qk", "tokens": 16384, "heads_q": 32, "heads_k": 8, "dim": 128, "rot": 128, "pairs": "halves"},
        # the gradient in a short ragged batch, half of each small head turned, neighbours paired
        {"name": "qk_backward_short", "op": "qk_backward", "tokens": 333, "heads_q": 12, "heads_k": 3, "dim": 64, "rot": 32, "pairs": "neighbours"},
        # that of a training batch
        {"name": "qk_backward_train", "op": "qk_backward", "tokens": 16384, "heads_q": 32, "heads_k": 8, "dim": 128, "rot": 128, "pairs": "halves"},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["rows4", "weights4", "matmul4", "matmul4", "qk", "qk_backward"])
    if op == "rows4":
        return {"op": op, "tokens": _log(rng, 1, 32768), "width": _log(rng, 8, 4096, 8)}
    if op == "weights4":
        return {"op": op, "rows": _log(rng, 8, 19456, 8), "width": _log(rng, 8, 4096, 8)}
    if op == "matmul4":
        case = {"op": op, "x": rng.choice(["q8", "q4"]), "tokens": _log(rng, 1, 8192), "k": _log(rng, 64, 14336, 8),
                "n": _log(rng, 64, 14336, 8), "add": rng.random() < 0.3}
        while case["tokens"] * case["k"] * case["n"] > 8192 * 4096 * 14336:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    rot = dim if rng.random() < 0.6 else 16 * rng.randint(1, dim // 16)
    heads_k = rng.randint(1, 8)
    case = {"op": op, "tokens": _log(rng, 1, 16384), "heads_q": heads_k * rng.randint(1, 8), "heads_k": heads_k, "dim": dim,
            "rot": rot, "pairs": rng.choice(["halves", "halves", "neighbours"])}
    while case["tokens"] * (case["heads_q"] + heads_k) * dim > 16384 * 40 * 128:
        case["tokens"] //= 2
    return case


# ---------------------------------------------------------------------------
# The stored forms
# ---------------------------------------------------------------------------
def _count(width, n):
    return -(-width // n)


def _power(s):
    """2**s in float32 for whole s in [-126, 127], from the number's own bits
    (the device's pow is an ulp off for some whole exponents)."""
    return ((s.int() + 127) << 23).view(torch.float32)


def _nibbles(v):
    """The e2m1 codes of float32 values of magnitude up to 6, ties to even."""
    a = v.abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
    code += (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte()
    return code + 8 * (v < 0).byte()


def _store4(x, group_rows=1):
    """(values, exponents) of a float32 matrix in 4 bits: panels of 128 columns,
    [panels, rows, 64] bytes of two codes each (the even column in the low half)
    and [panels, rows, 4] biased power-of-two exponents, one per 32 columns
    (shared by group_rows rows)."""
    rows, width = x.shape
    np_, nr = _count(width, PANEL), _count(rows, group_rows)
    p = torch.zeros((nr * group_rows, np_ * PANEL), dtype=torch.float32, device=x.device)
    p[:rows, :width] = x
    b = p.view(nr, group_rows, np_ * 4, GROUP)
    m, ex = torch.frexp(b.abs().amax(dim=(1, 3)))
    s = torch.where(m > 0, (ex - 3 + (m > 0.75).int()).clamp(-126, 126), torch.full_like(ex, -126))
    code = _nibbles(b * _power(-s)[:, None, :, None]).view(nr * group_rows, np_, 64, 2)[:rows]
    e = (s + 127).byte().repeat_interleave(group_rows, 0)[:rows].view(rows, np_, 4)
    return (code[..., 0] + 16 * code[..., 1]).transpose(0, 1).contiguous(), e.transpose(0, 1).contiguous()


def _restored4(values, exps, width):
    """float32 values of a 4-bit store."""
    np_, rows, _ = values.shape
    code = torch.stack([values & 15, values >> 4], dim=3).view(np_, rows, 4, GROUP)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=values.device)
    table = torch.cat([table, -table])
    v = table[code.int()] * _power(exps.int() - 127)[..., None]
    return v.view(np_, rows, PANEL).transpose(0, 1).reshape(rows, np_ * PANEL)[:, :width]


def _store8(x):
    """(values, exponents) of a float32 matrix in 8 bits: e4m3 bytes padded to
    whole blocks of 128 columns, one biased power-of-two exponent per block."""
    rows, width = x.shape
    nb = _count(width, PANEL)
    p = torch.zeros((rows, nb * PANEL), dtype=torch.float32, device=x.device)
    p[:, :width] = x
    b = p.view(rows, nb, PANEL)
    m, ex = torch.frexp(b.abs().amax(dim=2))
    s = torch.where(m > 0, (ex - 9 + (m > 0.875).int()).clamp(-126, 126), torch.full_like(ex, -126))
    e = torch.zeros((rows, _count(nb, 4) * 4), dtype=torch.uint8, device=x.device)
    e[:, :nb] = (s + 127).to(torch.uint8)
    return (b * _power(-s)[:, :, None]).to(torch.float8_e4m3fn).view(rows, nb * PANEL).view(torch.uint8), e


def _restored8(values, exps, width):
    nb = _count(width, PANEL)
    v = values.view(torch.float8_e4m3fn).float().view(values.shape[0], nb, PANEL)
    return (v * _power(exps[:, :nb].int() - 127)[:, :, None]).view(values.shape[0], nb * PANEL)[:, :width]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _activations(g, tokens, width):
    """Normal rows with a few channels far above the rest and rows of
    different size, as the activations between two projections have them."""
    x = torch.randn((tokens, width), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((tokens, 1), generator=g, device="cuda"))
    x[:, torch.rand((width,), generator=g, device="cuda") < 0.005] *= 20.0
    return x.to(torch.bfloat16)


def _positions(g, tokens, decode):
    """Decode: a token of each of many requests, far into them. Otherwise
    sequences of about 2000 tokens behind each other."""
    if decode:
        return torch.randint(0, 131072, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    first = torch.rand((tokens,), generator=g, device="cuda") < 1 / 2000
    at = torch.arange(tokens, device="cuda")
    start = torch.where(first, at, torch.zeros_like(at)).cummax(0).values
    return (at - start).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    empty = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "rows4":
        T, W = case["tokens"], case["width"]
        return {"op": op, "x": _activations(g, T, W), "out": empty(T, W)}
    if op == "weights4":
        R, W = case["rows"], case["width"]
        w = (torch.randn((R, W), generator=g, device="cuda") / math.sqrt(W)).to(torch.bfloat16)
        return {"op": op, "w": w, "out": empty(R, W), "out_t": empty(W, R)}
    if op == "matmul4":
        T, K, N = case["tokens"], case["k"], case["n"]
        x = _activations(g, T, K).float()
        w = torch.randn((N, K), generator=g, device="cuda") / math.sqrt(K)
        st = {"op": op, "x": case["x"], "k": K, "add": case["add"], "y": empty(T, N)}
        st["xq"], st["xe"] = _store8(x) if case["x"] == "q8" else _store4(x)
        st["wq"], st["we"] = _store4(w.to(torch.bfloat16).float())
        if case["add"]:
            st["y0"] = torch.randn((T, N), generator=g, device="cuda").to(torch.bfloat16)
        return st
    T, D, rot = case["tokens"], case["dim"], case["rot"]
    hq, hk = case["heads_q"], case["heads_k"]
    # queries, keys and values of a token side by side, as a joint projection leaves them
    qkv = _activations(g, T, (hq + 2 * hk) * D)
    weight = lambda: (1.0 + 0.2 * torch.randn((D,), generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    st = {"op": op, "D": D, "hq": hq, "hk": hk, "pairs": case["pairs"],
          "q": qkv[:, :hq * D], "k": qkv[:, hq * D:(hq + hk) * D], "wq": weight(), "wk": weight(),
          "freqs": 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / (rot // 2)),
          "positions": _positions(g, T, op == "qk" and T <= 1024)}
    if op == "qk":
        st["q_out"], st["k_out"] = empty(T, hq * D), empty(T, hk * D)
    else:
        st["gq"] = torch.randn((T, hq * D), generator=g, device="cuda").to(torch.bfloat16)
        st["gk"] = torch.randn((T, hk * D), generator=g, device="cuda").to(torch.bfloat16)
        dqkv = empty(T, (hq + 2 * hk) * D)
        st["dq"], st["dk"] = dqkv[:, :hq * D], dqkv[:, hq * D:(hq + hk) * D]
        st["dweight"] = empty(2, D, dtype=torch.float32)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _objects(st):
    """The library's handles on a state's buffers, made once and kept."""
    if "kept" in st:
        return st["kept"]
    import lora_adapter_batching_amd as L
    op, kept = st["op"], {}
    if op == "rows4":
        kept["q"] = L.new_q4(*st["x"].shape)
    elif op == "weights4":
        kept["q"], kept["qt"] = L.new_q4(*st["w"].shape), L.new_q4(*reversed(st["w"].shape))
    elif op == "matmul4":
        kept["x"] = L.Q8Rows(st["xq"], st["xe"], st["k"]) if st["x"] == "q8" else L.Q4(st["xq"], st["xe"], st["k"])
        kept["w"] = L.Q4(st["wq"], st["we"], st["k"])
    else:
        kept["heads"] = L.QKHeads(st["hq"], st["hk"], st["D"], st["wq"], st["wk"], st["freqs"], eps=EPS,
                                  neighbours=st["pairs"] == "neighbours")
        if op == "qk_backward":
            kept["ws"] = L.new_workspace_qk(kept["heads"], st["q"].shape[0])
    st["kept"] = kept
    return kept


def _rotation(st):
    """cos and sin [T, 1, rot / 2] of every position's angles, taken in 64 bits."""
    angle = st["positions"].double()[:, None, None] * st["freqs"]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _split(st, n):
    """The two members of each turned pair and the columns that stay."""
    half = st["freqs"].numel()
    if st["pairs"] == "halves":
        return n[..., :half], n[..., half:2 * half], n[..., 2 * half:]
    return n[..., 0:2 * half:2], n[..., 1:2 * half:2], n[..., 2 * half:]


def _join(st, a, b, rest):
    if st["pairs"] == "halves":
        return torch.cat([a, b, rest], dim=-1)
    return torch.cat([torch.stack([a, b], dim=-1).flatten(-2), rest], dim=-1)


def _turned(st, n, cos, sin):
    a, b, rest = _split(st, n)
    return _join(st, a * cos - b * sin, b * cos + a * sin, rest)


def run(st):
    op = st["op"]
    if own:
        import lora_adapter_batching_amd as L
        k = _objects(st)
        if op == "rows4":
            L.q4_quantize(st["x"], k["q"])
            L.q4_dequantize(k["q"], st["out"])
            return st["out"]
        if op == "weights4":
            L.q4_quantize(st["w"], k["q"], k["qt"])
            L.q4_dequantize(k["q"], st["out"])
            L.q4_dequantize(k["qt"], st["out_t"])
            return {"w": st["out"], "wt": st["out_t"]}
        if op == "matmul4":
            if st["add"]:
                st["y"].copy_(st["y0"])
            L.q4_matmul(k["x"], k["w"], st["y"], accumulate=st["add"])
            return st["y"]
        if op == "qk":
            L.qk_norm_rope(st["q"], st["k"], k["heads"], st["positions"], st["q_out"], st["k_out"])
            return {"q": st["q_out"], "k": st["k_out"]}
        L.qk_norm_rope_backward(st["q"], st["k"], k["heads"], st["positions"], st["gq"], st["gk"], st["dq"], st["dk"],
                                dweight=st["dweight"], ws=k["ws"])
        return {"dq": st["dq"], "dk": st["dk"], "dweight": st["dweight"]}
    if op == "rows4":
        return _restored4(*_store4(st["x"].float()), st["x"].shape[1]).to(torch.bfloat16)
    if op == "weights4":
        w = st["w"].float()
        return {"w": _restored4(*_store4(w, GROUP), w.shape[1]).to(torch.bfloat16),
                "wt": _restored4(*_store4(w.t(), GROUP), w.shape[0]).to(torch.bfloat16)}
    if op == "matmul4":
        x = (_restored8 if st["x"] == "q8" else _restored4)(st["xq"], st["xe"], st["k"])
        y = x @ _restored4(st["wq"], st["we"], st["k"]).t()
        return (st["y0"].float() + y if st["add"] else y).to(torch.bfloat16)
    cos, sin = _rotation(st)
    T, D = st["q"].shape[0], st["D"]
    out = {}
    for name, heads in (("q", st["hq"]), ("k", st["hk"])):
        x, w = st[name].float().view(T, heads, D), st["w" + name].float()
        n = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
        if op == "qk":
            out[name] = _turned(st, n * w, cos, sin).to(torch.bfloat16).view(T, heads * D)
            continue
        m = _turned(st, st["g" + name].float().view(T, heads, D), cos, -sin)
        g = m * w
        r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
        out["d" + name] = (r * (g - n * (g * n).mean(dim=-1, keepdim=True))).to(torch.bfloat16).view(T, heads * D)
        # per token first: a sum over all tokens in one go would lose bits
        out["dw" + name] = (m * n).sum(dim=1).sum(dim=0)
    if op == "qk":
        return out
    return {"dq": out["dq"], "dk": out["dk"], "dweight": torch.stack([out["dwq"], out["dwk"]])}


# ---------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "rows4":  # x read; the store written and read; the restored rows written
        T, W = case["tokens"], case["width"]
        return {"bytes": T * (5 * W + 2 * _count(W, GROUP)), "flops": 4 * T * W}
    if op == "weights4":  # w read; both stores written and read; both restored
        R, W = case["rows"], case["width"]
        return {"bytes": R * W * 8 + 2 * (R * _count(W, GROUP) + W * _count(R, GROUP)), "flops": 8 * R * W}
    if op == "matmul4":
        T, K, N = case["tokens"], case["k"], case["n"]
        x = K + _count(K, PANEL) if case["x"] == "q8" else K // 2 + _count(K, GROUP)
        return {"bytes": T * x + N * (K // 2 + _count(K, GROUP)) + T * N * (4 if case["add"] else 2), "flops": 2 * T * K * N}
    n = case["tokens"] * (case["heads_q"] + case["heads_k"]) * case["dim"]
    small = 4 * case["tokens"] + 4 * case["dim"] + 4 * case["rot"]
    if op == "qk":
        return {"bytes": 4 * n + small, "flops": 8 * n}
    return {"bytes": 6 * n + small + 8 * case["dim"], "flops": 16 * n}


def _power64(s):
    """2**s in float64 for whole s, from the number's own bits."""
    return ((s.long() + 1023) << 52).view(torch.float64)


def _e2m1_64(code):
    """The values of 4-bit codes (sign, two exponent bits, one mantissa bit), from the definition."""
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * _power64(e.long() - 1))
    return torch.where(code >= 8, -mag, mag)


def _read4_64(values, exps, width):
    col = torch.arange(width, device="cuda")
    panel, at = col // PANEL, col % PANEL
    v = values.permute(1, 0, 2)[:, panel, at // 2]
    code = torch.where(at % 2 == 1, v >> 4, v & 15)
    return _e2m1_64(code) * _power64(exps.permute(1, 0, 2)[:, panel, at // GROUP].long() - 127)


def _read8_64(values, exps, width):
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        mag = math.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-mag if b & 128 else mag)
    table = torch.tensor(v, dtype=torch.float64, device="cuda")
    at = torch.arange(width, device="cuda") // PANEL
    return table[values[:, :width].int()] * _power64(exps.long() - 127)[:, at]


def _through_4_bits64(x, group_rows):
    """x rounded to its block's grid: multiples of the e2m1 step at each
    value's size, ties to even."""
    rows, width = x.shape
    p = torch.nn.functional.pad(x, (0, -width % GROUP, 0, -rows % group_rows))
    b = p.view(p.shape[0] // group_rows, group_rows, p.shape[1] // GROUP, GROUP)
    top = b.abs().amax(dim=(1, 3), keepdim=True)
    k = torch.floor(torch.log2(top / 6.0)).clamp(-126, 126)
    unit = _power64(torch.where(6.0 * _power64(k) >= top, k, k + 1))
    step = _power64(torch.floor(torch.log2((b / unit).abs().clamp(min=1.0))) - 1.0) * unit
    return (torch.round(b / step) * step).view(p.shape)[:rows, :width]


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "rows4":
        return _through_4_bits64(st["x"].double(), 1)
    if op == "weights4":
        w = _through_4_bits64(st["w"].double(), GROUP)
        return {"w": w, "wt": w.t()}
    if op == "matmul4":
        x = (_read8_64 if st["x"] == "q8" else _read4_64)(st["xq"], st["xe"], st["k"])
        y = torch.matmul(x, _read4_64(st["wq"], st["we"], st["k"]).t())
        return y + st["y0"].double() if st["add"] else y
    T, D, half = st["q"].shape[0], st["D"], st["freqs"].numel()
    # each pair is a complex number that the position turns
    angle = st["positions"].double()[:, None] * st["freqs"][None, :]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    col = torch.arange(2 * half, device="cuda")
    re, im = (col[:half], col[half:]) if st["pairs"] == "halves" else (col[0::2], col[1::2])

    def rotate(v, t):
        z = torch.complex(v[..., re], v[..., im]) * t
        v = v.clone()
        v[..., re], v[..., im] = z.real, z.imag
        return v

    out, dweight = {}, []
    for name, heads in (("q", st["hq"]), ("k", st["hk"])):
        x, w = st[name].double().view(T, heads, D), st["w" + name].double()
        rms = torch.sqrt((x ** 2).sum(dim=-1, keepdim=True) / D + EPS)
        if op == "qk":
            out[name] = rotate(x / rms * w, turn).view(T, heads * D)
            continue
        m = rotate(st["g" + name].double().view(T, heads, D), turn.conj())
        dweight.append((m * x / rms).sum(dim=(0, 1)))
        along = (m * w * x).sum(dim=-1, keepdim=True) / (D * rms ** 3)
        out["d" + name] = (m * w / rms - x * along).view(T, heads * D)
    if op == "qk":
        return out
    return {"dq": out["dq"], "dk": out["dk"], "dweight": torch.stack(dweight)}
