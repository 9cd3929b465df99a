"""The query/key norm without a GPU: the struct's layout, every refusal (all
before any HIP call), calls without tokens, the binding's checks, and the
64-bit form that the GPU tests compare with."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import lora_adapter_batching_amd as L
from lora_adapter_batching_amd import binding as B
from tests import qk_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [(1 << 40) + (i << 36) for i in range(12)]  # aligned stand-in addresses, never read
by = ctypes.byref


def heads(hq=4, hk=2, dim=64, rot=64, nb=0, eps=1e-6, wq=A[8], wk=A[9], f=A[10]):
    return B.CQKHeads(hq, hk, dim, rot, nb, eps, wq, wk, f)


def forward(h=None, q=(A[0], 256), k=(A[1], 128), pos=A[11], T=4, qo=(A[2], 256), ko=(A[3], 128)):
    st = L.load().lora_qk_norm_rope(*q, *k, by(h or heads()), pos, T, *qo, *ko, None)
    return st, L.load().lora_last_error().decode()


def backward(h=None, q=(A[0], 256), k=(A[1], 128), pos=A[11], T=4, gq=(A[2], 256), gk=(A[3], 128), dq=(A[4], 256), dk=(A[5], 128),
             dw=A[6], flags=0, ws=A[7], wb=1 << 30):
    st = L.load().lora_qk_norm_rope_backward(*q, *k, by(h or heads()), pos, T, *gq, *gk, *dq, *dk, dw, flags, ws, wb, None)
    return st, L.load().lora_last_error().decode()


def test_struct_matches_the_c_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in B.CQKHeads._fields_]
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "lora_sgmv.h"\nint main(void) {\n'
    src += '  printf("%zu\\n", sizeof(lora_qk_heads_t));\n'
    src += "".join(f'  printf("%zu\\n", offsetof(lora_qk_heads_t, {n}));\n' for n in names) + "  return 0;\n}\n"
    (tmp_path / "q.c").write_text(src)
    exe = tmp_path / "q"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "q.c"), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(B.CQKHeads)] + [getattr(B.CQKHeads, n).offset for n in names]


@pytest.mark.parametrize("bad,word,want", [
    (dict(hq=-1), "heads_q", 1), (dict(hk=-1), "heads_k", 1), (dict(hq=0, hk=0), "both 0", 1), (dict(hq=65537), "65536", 2),
    (dict(dim=0), "head_dim", 1), (dict(dim=60), "head_dim", 1), (dict(dim=264, rot=64), "256", 2), (dict(rot=-16), "rot_dim", 1),
    (dict(rot=80), "rot_dim", 1), (dict(rot=24), "rot_dim", 1), (dict(eps=0.0), "eps", 1), (dict(eps=-1.0), "eps", 1),
    (dict(eps=float("nan")), "eps", 1), (dict(eps=float("inf")), "eps", 1), (dict(eps=1e-39), "eps", 1), (dict(eps=2e30), "eps", 1),
    (dict(wq=0), "weight", 1), (dict(wk=0), "weight", 1), (dict(wq=A[8] + 8), "aligned", 1), (dict(f=0), "freqs", 1),
    (dict(f=A[10] + 4), "freqs", 1)])
def test_every_entry_refuses_bad_heads(bad, word, want):
    n = ctypes.c_size_t(0)
    lib = L.load()
    for st, msg in (forward(heads(**bad)), backward(heads(**bad)),
                    (lib.lora_workspace_size_qk(by(heads(**bad)), 4, by(n)), lib.lora_last_error().decode())):
        assert st == want and word in msg, (st, msg)
    assert lib.lora_workspace_size_qk(None, 4, by(n)) == 1
    assert lib.lora_workspace_size_qk(by(heads()), -1, by(n)) == 1 and lib.lora_workspace_size_qk(by(heads()), 4, None) == 1


@pytest.mark.parametrize("bad,word,want", [
    (dict(T=-1), "num_tokens", 1), (dict(T=0x7fffffff), "num_tokens", 2), (dict(pos=0), "positions", 1), (dict(pos=A[11] + 2), "positions", 1),
    (dict(q=(0, 256)), "q is NULL", 1), (dict(k=(0, 128)), "k is NULL", 1), (dict(q=(A[0] + 8, 256)), "aligned", 1),
    (dict(q=(A[0], 248)), "below its width", 1), (dict(k=(A[1], 132)), "multiple of 8", 1)])
def test_both_directions_refuse(bad, word, want):
    for st, msg in (forward(**bad), backward(**bad)):
        assert st == want and word in msg, (st, msg)


def test_forward_refusals():
    for bad, word in [(dict(qo=(0, 256)), "q_out is NULL"), (dict(ko=(A[3], 120)), "below its width"), (dict(qo=(A[2] + 2, 256)), "aligned"),
                      (dict(qo=(A[3], 256)), "starts at"), (dict(qo=(A[1], 256)), "starts at"), (dict(ko=(A[0], 128)), "starts at"),
                      (dict(qo=(A[0], 264)), "row stride"), (dict(ko=(A[1], 136)), "row stride")]:
        st, msg = forward(**bad)
        assert st == 1 and word in msg, (bad, msg)


def test_backward_refusals():
    for bad, word, want in [(dict(gq=(0, 256)), "dq_out is NULL", 1), (dict(gk=(A[3], 120)), "below its width", 1), (dict(dq=(0, 256)), "dq is NULL", 1),
                            (dict(dk=(A[5] + 4, 128)), "aligned", 1), (dict(dq=(A[0], 256)), "starts at", 1), (dict(dq=(A[2], 256)), "starts at", 1),
                            (dict(dk=(A[1], 128)), "starts at", 1), (dict(dk=(A[3], 128)), "starts at", 1), (dict(dk=(A[4], 128)), "starts at", 1),
                            (dict(dq=(A[1], 256)), "starts at", 1), (dict(dk=(A[2], 128)), "starts at", 1), (dict(flags=2), "flags", 1),
                            (dict(dw=A[6] + 2), "dweight", 1), (dict(ws=0), "workspace", 1), (dict(ws=A[7] + 8), "workspace", 1),
                            (dict(wb=2047), "workspace", 3)]:
        st, msg = backward(**bad)
        assert st == want and word in msg, (bad, st, msg)


def test_workspace_holds_every_workgroups_share():
    lib, n, last = L.load(), ctypes.c_size_t(0), 0
    for T in (0, 1, 4, 300, 512, 513, 2047, 2048, 3071, 4096, 1 << 20, 0x7fff0000):
        assert lib.lora_workspace_size_qk(by(heads(dim=128, rot=0)), T, by(n)) == 0
        assert n.value % 1024 == 0 and n.value <= 768 * 1024 and (T == 0 or n.value > 0)
        last = max(last, n.value)
    assert last == 768 * 1024


def test_no_tokens_is_no_work():
    assert forward(T=0, pos=0, q=(0, 0), k=(0, 0), qo=(0, 0), ko=(0, 0))[0] == 0
    none = dict(T=0, pos=0, q=(0, 0), k=(0, 0), gq=(0, 0), gk=(0, 0), dq=(0, 0), dk=(0, 0))
    assert backward(dw=0, ws=0, wb=0, **none)[0] == 0


def test_a_kind_without_heads_has_its_pointers_ignored():
    """(what is refused is something else, behind those checks)"""
    st, msg = forward(heads(hk=0, wk=0), k=(0, 0), ko=(0, 0), qo=(A[2], 248))
    assert st == 1 and "q_out" in msg
    st, msg = backward(heads(hq=0, wq=0), q=(0, 0), gq=(0, 0), dq=(0, 0), flags=4)
    assert st == 1 and "flags" in msg
    st, msg = backward(heads(hq=0, wq=0), q=(0, 0), gq=(0, 0), dq=(0, 0), wb=0)
    assert st == 3, msg


def test_binding_refuses_wrong_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    f = torch.zeros(32, dtype=torch.float64)
    h = L.QKHeads(4, 2, 64, bf(64), bf(64), f)
    assert h.rot_dim == 64
    L.QKHeads(4, 0, 64, bf(64), None, f), L.QKHeads(0, 2, 64, None, bf(64), None)
    for args in [(4, 2, 64, bf(32), bf(64), f), (4, 2, 64, bf(64), None, f), (4, 2, 64, bf(64).float(), bf(64), f),
                 (4, 2, 64, bf(64), bf(64), f.float()), (4, 2, 64, bf(128)[::2], bf(64), f), (4, 2, 64, bf(64), bf(64), f[None])]:
        with pytest.raises(ValueError):
            L.QKHeads(*args)
    pos = torch.zeros(3, dtype=torch.int32)
    ok = dict(q=bf(3, 256), k=bf(3, 128), p=pos, qo=bf(3, 256), ko=bf(3, 128))
    call = lambda **a: L.qk_norm_rope(*[{**ok, **a}[n] for n in ("q", "k")], h, *[{**ok, **a}[n] for n in ("p", "qo", "ko")])  # noqa: E731
    for bad in [dict(q=bf(2, 256)), dict(q=bf(3, 255)), dict(k=bf(3, 128).float()), dict(k=None), dict(p=pos.long()), dict(p=pos[None]),
                dict(p=torch.zeros(6, dtype=torch.int32)[::2]), dict(qo=bf(3, 128)), dict(ko=bf(128, 3).t()), dict(qo=None)]:
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError, match="device tensors"):
        call()
    back = lambda **a: L.qk_norm_rope_backward(ok["q"], ok["k"], h, pos, bf(3, 256), bf(3, 128), bf(3, 256), bf(3, 128), **a)  # noqa: E731
    for dw in (torch.zeros(2, 32), torch.zeros(2, 64).double(), torch.zeros(64, 2).t(), torch.zeros(128)):
        with pytest.raises(ValueError, match="dweight"):
            back(dweight=dw)
    with pytest.raises(ValueError, match="device tensors"):
        back(dweight=torch.zeros(2, 64))


@pytest.mark.parametrize("neighbours", [False, True])
def test_reference_gradient_against_autograd_and_differences(neighbours):
    torch.manual_seed(0)
    T, H, D, rot = 3, 2, 48, 32
    x, w, g = torch.randn(T, H, D).double(), torch.randn(D).double(), torch.randn(T, H, D).double()
    pos, f = torch.tensor([0, 5, -70000]), torch.rand(rot // 2).double()
    x.requires_grad_(), w.requires_grad_()
    out = R.forward(x, w, pos, f, 1e-3, neighbours)
    (out * g).sum().backward()
    dx, dw = R.backward(x.detach(), w.detach(), pos, f, 1e-3, neighbours, g)
    assert torch.allclose(dx, x.grad, rtol=1e-12, atol=1e-13) and torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-13)
    loss = lambda a, b: float((R.forward(a, b, pos, f, 1e-3, neighbours) * g).sum())  # noqa: E731
    step = 1e-6
    for t, h, d in [(0, 0, 0), (1, 1, 31), (2, 0, 47), (2, 1, 17)]:
        e = torch.zeros_like(dx)
        e[t, h, d] = step
        num = (loss(x.detach() + e, w.detach()) - loss(x.detach() - e, w.detach())) / (2 * step)
        assert abs(num - float(dx[t, h, d])) < 1e-6 * (1 + abs(num))  # step^2 and 1e-16 / step of sums of some tens
    # a rotation keeps lengths, and position 0 turns nothing
    n = x.detach() / torch.sqrt((x.detach() ** 2).mean(-1, keepdim=True) + 1e-3) * w.detach()
    assert torch.allclose(out.detach().norm(dim=-1), n.norm(dim=-1)) and torch.allclose(out.detach()[0], n[0])


def test_the_weight_of_no_heads_is_ignored():
    """At any address (what is refused is something else, behind that check)."""
    st, msg = forward(heads(hk=0, wk=A[9] + 2), k=(0, 0), ko=(0, 0), qo=(A[2], 248))
    assert st == 1 and "q_out" in msg
    st, msg = backward(heads(hq=0, wq=A[8] + 2), q=(0, 0), gq=(0, 0), dq=(0, 0), flags=4)
    assert st == 1 and "flags" in msg
    st, msg = forward(heads(hk=0, wq=A[8] + 2, wk=0), k=(0, 0), ko=(0, 0))
    assert st == 1 and "aligned" in msg
