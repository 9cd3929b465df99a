"""Cases and plain forms of the 8-bit operators that stand beside the LoRA
projections: rows stored in 8 bits and restored, the frozen projection's
block-scaled product, the packed backward that reads an 8-bit checkpoint, and
the gated activation between two projections.

A run with own = False is elementary torch; with own = True it makes the
library's calls. Widths are those of the package's own workloads (2560,
19456 = 2 x 9728, 4096, 14336, 3584).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128


def listed():
    return [
        # a decode batch's activations stored and read back: launch latency
        {"name": "rows_decode", "op": "rows", "tokens": 256, "width": 2560},
        # the checkpoint of one wrapped projection in packed training
        {"name": "rows_train", "op": "rows", "tokens": 65536, "width": 3584},
        # a single request's token through an attention projection
        {"name": "matmul_one_token", "op": "matmul", "tokens": 1, "k": 2560, "n": 2560, "add": False},
        # a decode batch through the widest projection (reads 50 MB of weights)
        {"name": "matmul_decode_gate_up", "op": "matmul", "tokens": 256, "k": 2560, "n": 19456, "add": False},
        # a few requests through the down projection: long sums, few rows
        {"name": "matmul_down_ragged", "op": "matmul", "tokens": 37, "k": 9728, "n": 2560, "add": False},
        # a prefill chunk whose last tile is ragged, added to the residual rows
        {"name": "matmul_prefill_add", "op": "matmul", "tokens": 8191, "k": 4096, "n": 4096, "add": True},
        # the MLP-up projection of a long mixed batch: the largest product
        {"name": "matmul_mlp_up", "op": "matmul", "tokens": 8192, "k": 4096, "n": 14336, "add": False},
        # the smallest packed step: four adapters over sixteen tokens
        {"name": "backward_tiny", "op": "backward", "tokens": 16, "h_in": 256, "h_out": 256, "adapters": 4, "max_rank": 8},
        # packed training: 32 adapters of mixed ranks, one of them without tokens
        {"name": "backward_train", "op": "backward", "tokens": 65536, "h_in": 3584, "h_out": 3584, "adapters": 32, "max_rank": 64},
        # the activation of a decode batch, straight into the down projection's 8 bits
        {"name": "swiglu_decode", "op": "swiglu", "tokens": 256, "width": 9728},
        # the same for a training batch, which keeps the bf16 rows too
        {"name": "swiglu_train", "op": "swiglu", "tokens": 16384, "width": 9728},
        # its gradient
        {"name": "swiglu_backward_train", "op": "swiglu_backward", "tokens": 16384, "width": 9728},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["rows", "matmul", "matmul", "backward", "swiglu", "swiglu_backward"])
    if op == "rows":
        return {"op": op, "tokens": _log(rng, 1, 65536), "width": _log(rng, 8, 3584, 8)}
    if op == "matmul":
        case = {"op": op, "tokens": _log(rng, 1, 8192), "k": _log(rng, 64, 14336, 8), "n": _log(rng, 64, 14336, 8),
                "add": rng.random() < 0.3}
        while case["tokens"] * case["k"] * case["n"] > 8192 * 4096 * 14336:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    if op == "backward":
        return {"op": op, "tokens": _log(rng, 1, 32768), "h_in": _log(rng, 64, 3584, 8), "h_out": _log(rng, 64, 3584, 8),
                "adapters": rng.randint(1, 32), "max_rank": rng.choice([4, 8, 13, 16, 32, 64])}
    return {"op": op, "tokens": _log(rng, 1, 16384), "width": _log(rng, 8, 9728, 8)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _blocks(width):
    return -(-width // BLOCK)


def _power(s):
    """2**s in float32 for whole s in [-126, 127], from the number's own bits
    (the device's pow is an ulp off for some whole exponents)."""
    return ((s.int() + 127) << 23).view(torch.float32)


def _store(x, block_rows):
    """(values, exponents) of a float32 matrix in 8 bits: e4m3 bytes padded to
    whole blocks, and one biased power-of-two exponent per block."""
    rows, width = x.shape
    nb, nr = _blocks(width), -(-rows // block_rows)
    p = torch.zeros((nr * block_rows, nb * BLOCK), dtype=torch.float32, device=x.device)
    p[:rows, :width] = x
    b = p.view(nr, block_rows, nb, BLOCK)
    m, ex = torch.frexp(b.abs().amax(dim=(1, 3)))
    s = torch.where(m > 0, (ex - 9 + (m > 0.875).int()).clamp(-126, 126), torch.full_like(ex, -126))
    q = (b * _power(-s)[:, None, :, None]).to(torch.float8_e4m3fn)
    lde = -(-nb // 4) * 4
    e = torch.zeros((nr, lde), dtype=torch.uint8, device=x.device)
    e[:, :nb] = (s + 127).to(torch.uint8)
    return q.view(nr * block_rows, nb * BLOCK)[:rows].contiguous().view(torch.uint8), e


def _restored(values, exps, width, block_rows):
    """float32 values of an 8-bit store."""
    nb = _blocks(width)
    scale = _power(exps[:, :nb].int() - 127)
    scale = scale.repeat_interleave(block_rows, 0)[:values.shape[0]]
    v = values.view(torch.float8_e4m3fn)[:, :nb * BLOCK].float().view(values.shape[0], nb, BLOCK)
    return (v * scale[:, :, None]).view(values.shape[0], nb * BLOCK)[:, :width]


def _activations(g, tokens, width):
    """Normal rows with a few channels far above the rest and rows of
    different size, as the activations between two projections have them."""
    x = torch.randn((tokens, width), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((tokens, 1), generator=g, device="cuda"))
    x[:, torch.rand((width,), generator=g, device="cuda") < 0.005] *= 20.0
    return x.to(torch.bfloat16)


def _ranks(case):
    """The adapters' ranks: the largest first, then 8, 16, 32, 64 in turn."""
    some = [r for r in (8, 16, 32, 64) if r <= case["max_rank"]] or [case["max_rank"]]
    return np.array([case["max_rank"]] + [some[i % len(some)] for i in range(case["adapters"] - 1)], dtype=np.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, T = case["op"], case["tokens"]
    if op == "rows":
        return {"op": op, "x": _activations(g, T, case["width"]), "out": torch.empty((T, case["width"]), dtype=torch.bfloat16, device="cuda")}
    if op == "matmul":
        K, N = case["k"], case["n"]
        xq, xe = _store(_activations(g, T, K).float(), 1)
        w = (torch.randn((N, K), generator=g, device="cuda") / math.sqrt(K)).to(torch.bfloat16)
        wq, we = _store(w.float(), BLOCK)
        st = {"op": op, "k": K, "n": N, "add": case["add"], "xq": xq, "xe": xe, "wq": wq, "we": we,
              "y": torch.empty((T, N), dtype=torch.bfloat16, device="cuda")}
        if case["add"]:
            st["y0"] = torch.randn((T, N), generator=g, device="cuda").to(torch.bfloat16)
        return st
    if op == "backward":
        hi, ho, n = case["h_in"], case["h_out"], case["adapters"]
        ranks = _ranks(case)
        scales = rng.uniform(0.5, 2.0, size=n).astype(np.float32)
        # tokens grouped by adapter; the last of several adapters has none, and
        # one token in fifty belongs to no adapter (its rows come last)
        ids = rng.integers(0, n - 1 if n > 2 else n, size=T)
        ids[rng.random(T) < 0.02] = n
        ids = np.sort(ids).astype(np.int32)
        starts = np.searchsorted(ids, np.arange(n + 2)).astype(np.int32)
        seg_adapter = np.append(np.arange(n), -1).astype(np.int32)
        rmax, R = int(ranks.max()), int(ranks.sum())
        A = [(torch.randn((int(r), hi), generator=g, device="cuda") / math.sqrt(hi)).to(torch.bfloat16) for r in ranks]
        B = [(torch.randn((ho, int(r)), generator=g, device="cuda") / math.sqrt(int(r))).to(torch.bfloat16) for r in ranks]
        xq, xe = _store(_activations(g, T, hi).float(), 1)
        first = np.concatenate([[0], np.cumsum(ranks)])
        # place of dB_i[j][k] in the flat list of all dB_i, as a place in [h_out, R]
        flat = np.concatenate([(np.arange(ho)[:, None] * R + first[i] + np.arange(ranks[i])[None, :]).reshape(-1) for i in range(n)])
        dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=t)  # noqa: E731
        return {"op": op, "h_in": hi, "h_out": ho, "ranks": ranks, "scales": scales, "starts": starts, "seg_adapter": seg_adapter,
                "A": A, "B": B, "xq": xq, "xe": xe,
                "dy": torch.randn((T, ho), generator=g, device="cuda").to(torch.bfloat16),
                "u": torch.randn((T, rmax), generator=g, device="cuda"),
                "dx0": torch.randn((T, hi), generator=g, device="cuda").to(torch.bfloat16),
                "dx": torch.empty((T, hi), dtype=torch.bfloat16, device="cuda"),
                "dA": torch.empty((R, hi), dtype=torch.float32, device="cuda"),
                "dB": torch.empty((R * ho,), dtype=torch.float32, device="cuda"),
                "ids": dev(ids, torch.int32),
                "col_adapter": dev(np.repeat(np.arange(n), ranks), torch.int32),
                "col_rank": dev(np.concatenate([np.arange(r) for r in ranks]), torch.int64),
                "col_scale": dev(np.repeat(scales, ranks), torch.float32),
                "flat": dev(flat, torch.int64)}
    F = case["width"]
    gate_up = (1.5 * torch.randn((T, 2 * F), generator=g, device="cuda")).to(torch.bfloat16)
    st = {"op": op, "width": F, "gate_up": gate_up}
    if op == "swiglu":
        st["h"] = torch.empty((T, F), dtype=torch.bfloat16, device="cuda")
        st["restored"] = torch.empty((T, F), dtype=torch.bfloat16, device="cuda")
    else:
        st["dh"] = torch.randn((T, F), generator=g, device="cuda").to(torch.bfloat16)
        st["dgate_up"] = torch.empty((T, 2 * F), dtype=torch.bfloat16, device="cuda")
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
    if op == "rows":
        kept["q"] = L.new_q8_rows(*st["x"].shape)
    elif op == "matmul":
        kept["x"] = L.Q8Rows(st["xq"], st["xe"], st["k"])
        kept["w"] = L.Q8Weights(st["wq"], st["we"], st["k"])
    elif op == "backward":
        first = np.concatenate([[0], np.cumsum(st["ranks"])])
        table = lambda t, row: torch.tensor([t.data_ptr() + 4 * int(row) * int(f) for f in first[:-1]], dtype=torch.int64, device="cuda")  # noqa: E731
        kept["x"] = L.Q8Rows(st["xq"], st["xe"], st["h_in"])
        kept["adapters"] = L.Adapters(st["A"], st["B"], st["ranks"], st["scales"], st["h_in"], st["h_out"])
        kept["segments"] = L.Segments(st["starts"], st["seg_adapter"])
        kept["dA"], kept["dB"] = table(st["dA"], st["h_in"]), table(st["dB"], st["h_out"])
        kept["ws"] = L.new_workspace(L.OP_BACKWARD, kept["adapters"], kept["segments"])
    elif op == "swiglu":
        kept["hq"] = L.new_q8_rows(*st["h"].shape)
    st["kept"] = kept
    return kept


def run(st):
    op = st["op"]
    if own:
        import lora_adapter_batching_amd as L
        k = _objects(st)
        if op == "rows":
            L.q8_quantize(st["x"], k["q"])
            L.q8_dequantize(k["q"], st["out"])
            return st["out"]
        if op == "matmul":
            if st["add"]:
                st["y"].copy_(st["y0"])
            L.q8_matmul(k["x"], k["w"], st["y"], accumulate=st["add"])
            return st["y"]
        if op == "backward":
            st["dx"].copy_(st["dx0"])
            L.packed_backward_q8(k["x"], st["dy"], st["u"], k["adapters"], k["segments"], st["dx"], k["dA"], k["dB"], ws=k["ws"])
            return {"dx": st["dx"], "dA": st["dA"], "dB": st["dB"]}
        if op == "swiglu":
            L.swiglu(st["gate_up"], st["h"], k["hq"])
            L.q8_dequantize(k["hq"], st["restored"])
            return {"h": st["h"], "restored": st["restored"]}
        L.swiglu_backward(st["gate_up"], st["dh"], st["dgate_up"])
        return st["dgate_up"]
    if op == "rows":
        return _round_trip(st["x"].float())
    if op == "matmul":
        y = _restored(st["xq"], st["xe"], st["k"], 1) @ _restored(st["wq"], st["we"], st["k"], BLOCK).t()
        return (st["y0"].float() + y if st["add"] else y).to(torch.bfloat16)
    if op == "backward":
        mine = (st["ids"][:, None] == st["col_adapter"][None, :]).float() * st["col_scale"]
        x, dy = _restored(st["xq"], st["xe"], st["h_in"], 1), st["dy"].float()
        du = (dy @ torch.cat(st["B"], 1).float()) * mine
        dx = st["dx0"].float() + du @ torch.cat(st["A"]).float()
        dB = dy.t() @ (st["u"][:, st["col_rank"]] * mine)
        return {"dx": dx.to(torch.bfloat16), "dA": du.t() @ x, "dB": dB.reshape(-1)[st["flat"]]}
    gate, up = st["gate_up"].float().split(st["width"], dim=1)
    s = 1.0 / (1.0 + torch.exp(-gate))
    if op == "swiglu":
        h = gate * s * up
        return {"h": h.to(torch.bfloat16), "restored": _round_trip(h)}
    dh = st["dh"].float()
    return torch.cat([dh * up * s * (1.0 + gate * (1.0 - s)), dh * gate * s], dim=1).to(torch.bfloat16)


def _round_trip(x):
    return _restored(*_store(x, 1), x.shape[1], 1).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------
def work(case):
    op, T = case["op"], case["tokens"]
    if op == "rows":  # x read; the store written and read; the restored rows written
        return {"bytes": T * case["width"] * 6 + 2 * T * _blocks(case["width"]), "flops": 4 * T * case["width"]}
    if op == "matmul":
        K, N = case["k"], case["n"]
        return {"bytes": T * (K + _blocks(K)) + N * K + _blocks(N) * _blocks(K) + T * N * (4 if case["add"] else 2), "flops": 2 * T * K * N}
    if op == "backward":
        hi, ho, ranks = case["h_in"], case["h_out"], _ranks(case)
        R, mean = int(ranks.sum()), float(ranks.mean())
        return {"bytes": T * (ho * 2 + hi + _blocks(hi) + hi * 4 + mean * 4) + R * (hi + ho) * (2 + 4),
                "flops": T * mean * 4 * (hi + ho)}
    F = case["width"]
    if op == "swiglu":  # gate and up read; bf16 rows and the store written; the store read and restored
        return {"bytes": T * F * (4 + 2 + 1 + 1 + 2) + 2 * T * _blocks(F), "flops": 8 * T * F}
    return {"bytes": T * F * (4 + 2 + 4), "flops": 12 * T * F}


def _table64():
    """The 256 values of e4m3, from its definition."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        mag = math.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-mag if b & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _power64(s):
    """2**s in float64 for whole s, from the number's own bits."""
    return ((s.long() + 1023) << 52).view(torch.float64)


def _read64(values, exps, width, block_rows):
    row = torch.arange(values.shape[0], device="cuda") // block_rows
    out = _table64()[values[:, :width].int()]
    at = torch.arange(width, device="cuda") // BLOCK
    return out.mul_(_power64(exps.long() - 127)[row[:, None], at[None, :]])


def _through_8_bits64(x):
    """x rounded to its 1 x 128 block's grid: multiples of the e4m3 step at
    each value's size, ties to even."""
    rows, width = x.shape
    p = torch.nn.functional.pad(x, (0, _blocks(width) * BLOCK - width)).view(rows, -1, BLOCK)
    top = p.abs().amax(dim=2, keepdim=True)
    k = torch.floor(torch.log2(top / 448.0)).clamp(-126, 126)
    unit = _power64(torch.where(448.0 * _power64(k) >= top, k, k + 1))
    step = _power64(torch.floor(torch.log2((p / unit).abs().clamp(min=2.0 ** -6))) - 3.0) * unit
    return (torch.round(p / step) * step).view(rows, -1)[:, :width]


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "rows":
        return _through_8_bits64(st["x"].double())
    if op == "matmul":
        y = torch.matmul(_read64(st["xq"], st["xe"], st["k"], 1), _read64(st["wq"], st["we"], st["k"], BLOCK).t())
        return y + st["y0"].double() if st["add"] else y
    if op == "backward":
        dx, dA, dB = st["dx0"].double(), [], []
        x, dy, u = _read64(st["xq"], st["xe"], st["h_in"], 1), st["dy"], st["u"]
        for i, (a, b) in enumerate(zip(st["A"], st["B"])):
            lo, hi, r = int(st["starts"][i]), int(st["starts"][i + 1]), int(st["ranks"][i])
            d = dy[lo:hi].double() * float(st["scales"][i])
            du = d @ b.double()
            dx[lo:hi] += du @ a.double()
            dA.append(du.t() @ x[lo:hi])
            dB.append((d.t() @ u[lo:hi, :r].double()).reshape(-1))
        return {"dx": dx, "dA": torch.cat(dA), "dB": torch.cat(dB)}
    F = st["width"]
    g, u = st["gate_up"][:, :F].double(), st["gate_up"][:, F:].double()
    if op == "swiglu":
        h = g * torch.sigmoid(g) * u
        return {"h": h, "restored": _through_8_bits64(h)}
    dh, s = st["dh"].double(), torch.sigmoid(g)
    return torch.cat([dh * u * (s + g * s * (1 - s)), dh * g * s], dim=1)
