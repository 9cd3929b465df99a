"""The operators around an attention layer's wrapped q/k/v projection as they
are used together: a frozen base in 4 bits, adapters on top, the norm and
rotation of queries and keys, forward, backward and as a captured decode step.
Each stage is checked on the stage before's own output, with the tolerances of
the stages' own tests (the adapters': a low-rank vector enters as two bf16
parts, 2^-15 of it left out)."""
import numpy as np
import pytest
import torch

import lora_adapter_batching_amd as L
from tests import q8_ref as R8
from tests.helpers import to_f64
from tests.test_gpu_q4 import check_matmul
from tests.test_gpu_q8 import bf16, rows
from tests.test_gpu_q8 import held as held_np
from tests.test_gpu_qk import Case

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -23


class Layer:
    """One q/k/v projection of `width` columns and its case of heads, whose rows are the projection's y."""

    def __init__(self, T, width, hq, hk, D, ranks, seed):
        rng = np.random.default_rng(seed)
        self.T, self.width, self.ranks, self.scales = T, width, ranks, [1.0, 0.5, 2.0][:len(ranks)]
        self.case = Case(T, hq, hk, D, D, seed=seed)
        self.out = (hq + 2 * hk) * D
        self.A = [bf16(rng.standard_normal((r, width)) / np.sqrt(width)) for r in ranks]
        self.B = [bf16(rng.standard_normal((self.out, r)) / np.sqrt(r)) for r in ranks]
        self.w, self.wt = L.new_q4(self.out, width), L.new_q4(width, self.out)
        L.q4_quantize(rows(rng, self.out, width, 0.1) / np.sqrt(width), self.w, self.wt)
        self.x = rows(rng, T, width)
        self.ids = rng.integers(-1, len(ranks), T).astype(np.int32)
        self.y = self.case.x[:T, 8:]                                   # [T, out], strided

    def adapted(self, base, x, ids):
        """(y, sum of magnitudes) of the adapters on top of base."""
        want, mag, x = base.copy(), np.abs(base), to_f64(x)
        for a in range(len(self.ranks)):
            t = ids == a
            low, A, Bm = x[t], to_f64(self.A[a]), to_f64(self.B[a])
            want[t] += self.scales[a] * (low @ A.T) @ Bm.T
            mag[t] += self.scales[a] * (np.abs(low) @ np.abs(A).T) @ np.abs(Bm).T
        return want, mag


@pytest.mark.parametrize("T", [150, 2100])
def test_forward_and_backward(T):
    y = Layer(T, 256, 3, 1, 64, [8, 16, 4], 3)
    c, hq, hk, D = y.case, 3, 1, 64
    # tokens grouped by adapter, those without one last
    perm, starts, adap = L.segments_from_ids(y.ids, 3)
    ids = y.ids[perm]
    seg, ad = L.Segments(starts, adap), L.Adapters(y.A, y.B, y.ranks, y.scales, y.width, y.out)
    xq, u = L.new_q8_rows(T, y.width), torch.zeros((T, 16), device="cuda")
    L.q8_quantize(y.x, xq)
    L.q4_matmul(xq, y.w, y.y)
    check_matmul(xq, y.w, y.y)
    base = to_f64(y.y)
    L.sgmv_fused(y.x, ad, seg, y.y, u, L.new_workspace(L.OP_FUSED, ad, seg))
    want, mag = y.adapted(base, y.x, ids)
    held_np(to_f64(y.y), want, BF * np.abs(want) + (2.0 ** -15 + 400 * F32) * mag)
    c.check_forward(c.forward())
    # back: the attention's dq, dk and dv, the projection's dy in place of the first two
    dw = torch.empty((2, D), device="cuda")
    dy = c.backward(dw, ws=L.new_workspace_qk(c.heads, T))
    c.check_backward(dy, dw)
    dy = dy[:T, 8:]
    dy[:, (hq + hk) * D:] = c.gr[:T, 8 + (hq + hk) * D:]
    dyq, dx = L.new_q8_rows(T, y.out), torch.zeros((T, y.width), dtype=torch.bfloat16, device="cuda")
    L.q8_quantize(dy, dyq)
    L.q4_matmul(dyq, y.wt, dx)
    check_matmul(dyq, y.wt, dx)
    base_dx = to_f64(dx)
    gA, gB = [torch.zeros((r, y.width), device="cuda") for r in y.ranks], [torch.zeros((y.out, r), device="cuda") for r in y.ranks]
    tab = lambda ts: torch.tensor([t.data_ptr() for t in ts], dtype=torch.int64, device="cuda")  # noqa: E731
    L.packed_backward_q8(xq, dy, u, ad, seg, dx, tab(gA), tab(gB), ws=L.new_workspace(L.OP_BACKWARD, ad, seg))
    torch.cuda.synchronize()
    xv, d64, uu = R8.read_store(xq), to_f64(dy), u.cpu().numpy().astype(np.float64)
    want, tol = base_dx.copy(), np.zeros_like(base_dx)
    for a, r in enumerate(y.ranks):
        t = ids == a
        n, A, Bm, s = int(t.sum()), to_f64(y.A[a]), to_f64(y.B[a]), y.scales[a]
        du, dm = s * d64[t] @ Bm, s * np.abs(d64[t]) @ np.abs(Bm)
        held_np(gA[a].cpu().numpy(), du.T @ xv[t], (n + y.out + 16) * F32 * (dm.T @ np.abs(xv[t])), "dA")
        held_np(gB[a].cpu().numpy(), s * d64[t].T @ uu[t, :r], (n + 8) * F32 * (s * np.abs(d64[t]).T @ np.abs(uu[t, :r])), "dB")
        want[t] += du @ A
        tol[t] += (2.0 ** -16 + (y.out + r + 16) * F32) * (dm @ np.abs(A))
    held_np(to_f64(dx), want, BF * (np.abs(want) + tol) + tol, "dx")


@pytest.mark.parametrize("x4", [False, True])
def test_a_captured_decode_step_is_replayed(x4):
    """Rows stored, the 4-bit product, device-planned adapters and the rotation
    in place, in one graph: replays with new tokens, ids and positions, the
    program's eager work between them."""
    y = Layer(24, 512, 4, 2, 128, [8, 16], 4)
    c = y.case
    dev = lambda v, t: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    ga = L.GraphAdapters(dev([t.data_ptr() for t in y.A], torch.int64), dev([t.data_ptr() for t in y.B], torch.int64),
                         dev(y.ranks, torch.int32), dev(y.scales, torch.float32), y.width, y.out, 16)
    ids = dev(y.ids, torch.int32)
    ws = L.new_workspace_graph(ga, 24)
    q = L.new_q4(24, 512) if x4 else L.new_q8_rows(24, 512)
    plain = c.wide()                                                   # the projection's rows before the rotation

    def step():
        (L.q4_quantize if x4 else L.q8_quantize)(y.x, q)
        L.q4_matmul(q, y.w, y.y)
        L.sgmv_fused_graph(y.x, ga, ids, y.y, ws)
        plain.copy_(c.x)
        L.qk_norm_rope(c.cols(c.x, 0), c.cols(c.x, 1), c.heads, c.pos, c.cols(c.x, 0), c.cols(c.x, 1))

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(9)
    for k in range(4):
        y.x.copy_(rows(rng, 24, 512))
        y.ids = rng.integers(-1, 2, 24).astype(np.int32)
        ids.copy_(torch.from_numpy(y.ids))
        c.pos.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = c.x.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, c.x)
        base = torch.empty((24, y.out), dtype=torch.bfloat16, device="cuda")
        L.q4_matmul(q, y.w, base)
        check_matmul(q, y.w, base)
        want, mag = y.adapted(to_f64(base), y.x, y.ids)
        held_np(to_f64(plain[:24, 8:]), want, BF * np.abs(want) + (2.0 ** -15 + 600 * F32) * mag)
        big = c.wide()
        for kind in (0, 1):
            c.cols(big, kind)[:] = c.cols(c.x, kind)
        c.check_forward(big, plain)
