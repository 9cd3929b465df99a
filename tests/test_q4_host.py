"""4-bit operators without a GPU: the struct's layout, every refusal (all of
them before any HIP call), calls without rows, the binding's checks, the
choice of the product's kernel, and the 64-bit forms that the GPU tests
compare with."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import lora_adapter_batching_amd as L
from lora_adapter_batching_amd import binding as B
from tests import q4_ref as R
from tests.q4_products import LONG_SUMS, PRODUCTS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, D = 1 << 40, 1 << 41  # aligned stand-in addresses, never read
by = ctypes.byref


def q4(rows=4, width=256, ld=256, lde=16, values=P, exps=P):
    return B.CQ4(values, ld, exps, lde, rows, width)


def q8(rows=4, width=256, ld=256, lde=4, block_rows=1, values=P, exps=P):
    return B.CQ8(values, ld, exps, lde, rows, width, block_rows)


def status(fn, *args):
    st = fn(*args)
    return st, L.load().lora_last_error().decode()


def test_struct_matches_the_c_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in B.CQ4._fields_]
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "lora_sgmv.h"\nint main(void) {\n'
    src += '  printf("%zu\\n", sizeof(lora_q4_t));\n'
    src += "".join(f'  printf("%zu\\n", offsetof(lora_q4_t, {n}));\n' for n in names) + "  return 0;\n}\n"
    (tmp_path / "q.c").write_text(src)
    exe = tmp_path / "q"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "q.c"), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(B.CQ4)] + [getattr(B.CQ4, n).offset for n in names]


@pytest.mark.parametrize("bad,word,want", [
    (dict(rows=-1), "rows", 1), (dict(width=0), "width", 1), (dict(width=12), "width", 1), (dict(width=-8), "width", 1),
    (dict(ld=248), "panel stride", 1), (dict(ld=264), "panel stride", 1), (dict(ld=192), "panel stride", 1),
    (dict(lde=12), "exponent panel stride", 1), (dict(lde=18), "exponent panel stride", 1),
    (dict(values=0), "NULL", 1), (dict(exps=0), "NULL", 1), (dict(values=P + 8), "aligned", 1), (dict(exps=P + 2), "aligned", 1),
    (dict(rows=0x7ffffff8, ld=1 << 40, lde=1 << 40), "larger than", 2), (dict(width=0x7ffffff8), "larger than", 2)])
def test_every_entry_refuses_a_bad_store(bad, word, want):
    lib = L.load()
    r = by(q4(**bad))
    calls = [(lib.lora_q4_quantize, D, 1 << 33, r, None), (lib.lora_q4_quantize, D, 1024, by(q4()), r),
             (lib.lora_q4_dequantize, r, D, 1 << 33), (lib.lora_q4_matmul, r, by(q4(rows=8, ld=512, lde=32)), D, 1024, 0),
             (lib.lora_q4_matmul, by(q4()), r, D, 1024, 0), (lib.lora_q4_matmul_q8, by(q8()), r, D, 1024, 0)]
    for fn, *args in calls:
        st, msg = status(fn, *args, None)
        assert st == want and word in msg, (fn, st, msg)


def test_quantize_refusals():
    lib = L.load()
    o, t = q4(rows=8, ld=512, lde=32), q4(rows=256, width=8, ld=1 << 14, lde=1 << 10, values=D)
    for x, ld, a, b, word in [(0, 256, o, None, "NULL"), (P + 4, 256, o, None, "aligned"), (D * 2, 248, o, None, "below its width"),
                              (D * 2, 260, o, None, "multiple of 8"), (P, 256, None, None, "NULL"),
                              (D * 2, 256, o, q4(rows=248, width=8, ld=1 << 14, lde=1 << 10), "transpose"),
                              (D * 2, 256, o, q4(rows=256, width=16, ld=1 << 14, lde=1 << 10), "transpose"),
                              (D * 2, 256, q4(rows=4), q4(rows=256, width=4, ld=1 << 14, lde=1 << 10), "multiple of 8"),
                              (P, 256, o, None, "starts at"), (D, 256, o, t, "starts at"),
                              (D * 2, 256, o, q4(rows=256, width=8, ld=1 << 14, lde=1 << 10), "starts at")]:
        st, msg = status(lib.lora_q4_quantize, x, ld, by(a) if a else None, by(b) if b else None, None)
        assert st == B.LORA_INVALID_ARGUMENT and word in msg, (word, msg)
    for x, ld, word in [(P, 256, "starts at"), (0, 256, "NULL"), (P + 2, 256, "aligned"), (D, 128, "below its width"), (D, 260, "multiple of 8")]:
        st, msg = status(lib.lora_q4_dequantize, by(o), x, ld, None)
        assert st == B.LORA_INVALID_ARGUMENT and word in msg, msg


@pytest.mark.parametrize("bits", [4, 8])
def test_matmul_refusals(bits):
    lib = L.load()
    fn, mk = (lib.lora_q4_matmul, q4) if bits == 4 else (lib.lora_q4_matmul_q8, q8)
    x, w = mk(), q4(rows=16, ld=1024, lde=64)
    cases = [((None, by(w), D, 16, 0), "NULL", 1), ((by(x), None, D, 16, 0), "NULL", 1),
             ((by(x), by(q4(rows=16, width=128, ld=1024, lde=64)), D, 16, 0), "wide", 1),
             ((by(x), by(q4(rows=12, ld=1024, lde=64)), D, 16, 0), "multiple of 8", 1),
             ((by(x), by(w), 0, 16, 0), "NULL", 1), ((by(x), by(w), D + 2, 16, 0), "aligned", 1),
             ((by(x), by(w), D, 8, 0), "below its width", 1), ((by(x), by(w), D, 20, 0), "multiple of 8", 1),
             ((by(x), by(w), D, 16, 2), "flags", 1), ((by(x), by(w), P, 16, 0), "starts at an operand", 1),
             ((by(mk(values=2 * D)), by(w), 2 * D, 16, 0), "starts at an operand", 1)]
    if bits == 8:
        cases += [((by(q8(ld=1 << 24)), by(w), D, 16, 0), "strides", 2), ((by(q8(lde=1 << 24)), by(w), D, 16, 0), "strides", 2),
                  ((by(q8(block_rows=128)), by(w), D, 16, 0), "block_rows", 1)]
    for args, word, want in cases:
        st, msg = status(fn, *args, None)
        assert st == want and word in msg, (msg, word)


def test_more_than_one_launch_holds_is_refused():
    """Grids of 2^32 threads and more (stand-in addresses: nothing is launched)."""
    lib = L.load()
    big = 0x7ffff000
    store = q4(rows=big, width=1 << 16, ld=1 << 40, lde=1 << 40)
    for fn, *args in [(lib.lora_q4_quantize, D, 1 << 16, by(store), None),
                      (lib.lora_q4_quantize, D, 1 << 16, by(store), by(q4(rows=1 << 16, width=big, ld=1 << 40, lde=1 << 40, values=4 * D))),
                      (lib.lora_q4_dequantize, by(store), D, 1 << 16),
                      (lib.lora_q4_matmul, by(q4(rows=big, ld=1 << 40, lde=1 << 40)), by(q4(rows=big, ld=1 << 40, lde=1 << 40)), D, 1 << 32, 0),
                      (lib.lora_q4_matmul_q8, by(q8(rows=big)), by(q4(rows=big, ld=1 << 40, lde=1 << 40)), D, 1 << 32, 0)]:
        st, msg = status(fn, *args, None)
        assert st == B.LORA_UNSUPPORTED and "too large" in msg, (fn, st, msg)


def test_no_rows_is_no_work():
    """No HIP call is made without rows: these succeed without a GPU."""
    lib = L.load()
    e, w = q4(rows=0, values=0, exps=0, ld=0, lde=0), q4(rows=8, ld=512, lde=32)
    assert lib.lora_q4_quantize(None, 0, by(e), None, None) == 0
    assert lib.lora_q4_dequantize(by(e), None, 0, None) == 0
    assert lib.lora_q4_matmul(by(e), by(w), None, 0, 0, None) == 0
    assert lib.lora_q4_matmul(by(q4()), by(e), None, 0, 0, None) == 0
    assert lib.lora_q4_matmul_q8(by(q8(rows=0, values=0, exps=0)), by(w), None, 0, 0, None) == 0
    assert lib.lora_q4_matmul_q8(by(q8()), by(e), None, 0, 0, None) == 0


def test_binding_refuses_wrong_tensors():
    v, e = torch.zeros((2, 8, 64), dtype=torch.uint8), torch.zeros((2, 8, 4), dtype=torch.uint8)
    L.Q4(v, e, 256), L.Q4(v, e, 136), L.Q4(v, e, 256, rows=3), L.Q4(v, e, 8), L.Q4(v[:, 4:], e[:, 4:], 256)
    for args in [(v.float(), e, 256), (v, e.int(), 256), (v, e, 264), (v[0], e, 256), (v, e[:, :7], 256), (v, e[:1], 256),
                 (v[:, :, :32], e, 256), (v, e.expand(2, 8, 4)[:, :, :2], 256), (v[:, ::2], e[:, ::2], 256),
                 (v.transpose(0, 1).contiguous().transpose(0, 1), e, 256), (v, torch.zeros((2, 4, 8), dtype=torch.uint8).transpose(1, 2), 256)]:
        with pytest.raises(ValueError):
            L.Q4(*args)
    for rows in (9, -1):
        with pytest.raises(ValueError):
            L.Q4(v, e, 256, rows=rows)
    x, x8, w = L.new_q4(4, 256, "cpu"), L.new_q8_rows(4, 256, "cpu"), L.new_q4(16, 256, "cpu")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    for fn, args in [(L.q4_quantize, (bf(3, 256), x)), (L.q4_quantize, (bf(4, 128), x)), (L.q4_quantize, (torch.zeros(4, 256), x)),
                     (L.q4_dequantize, (x, bf(4, 255))), (L.q4_matmul, (x, w, bf(4, 8))), (L.q4_matmul, (x8, w, bf(3, 16))),
                     (L.q4_matmul, (x, L.new_q8_weights(16, 256, "cpu"), bf(4, 16))), (L.q4_matmul, (L.new_q8_weights(4, 256, "cpu"), w, bf(4, 16)))]:
        with pytest.raises(ValueError):
            fn(*args)
    # a store of the other form is no store of this one
    for fn, args in [(L.q4_quantize, (bf(4, 256), x8)), (L.q4_quantize, (bf(4, 256), x, L.new_q8_weights(256, 4, "cpu"))),
                     (L.q4_dequantize, (x8, bf(4, 256)))]:
        with pytest.raises(ValueError, match="must be a Q4"):
            fn(*args)
    for fn, args in [(L.q8_quantize, (bf(4, 256), x)), (L.q8_dequantize, (x, bf(4, 256))), (L.q8_matmul, (x8, w, bf(4, 16))),
                     (L.swiglu, (bf(4, 512), None, x))]:
        with pytest.raises(AttributeError):
            fn(*args)
    for fn, args in [(L.q4_quantize, (bf(4, 256), x)), (L.q4_matmul, (x, w, bf(4, 16))), (L.q4_matmul, (x8, w, bf(4, 16)))]:
        with pytest.raises(ValueError, match="device tensors"):
            fn(*args)


def test_binding_hands_over_the_strides_of_views():
    """Rows of a larger store, a single panel or row of any stride."""
    v, e = torch.zeros((3, 20, 64), dtype=torch.uint8), torch.zeros((3, 20, 4), dtype=torch.uint8)
    q = L.Q4(v[:, 4:9], e[:, 4:9], 384)
    assert (q._c.values, q._c.ld, q._c.ld_exps, q.rows) == (v.data_ptr() + 256, 1280, 80, 5)
    assert q._c.exps == e.data_ptr() + 16
    one = L.Q4(v[1:2, :5], e[1:2, :5], 128)
    assert (one._c.ld, one._c.ld_exps) == (320, 20)
    odd = torch.zeros((1, 128), dtype=torch.uint8)[:, None, ::2]            # [1, 1, 64], unit stride missing
    with pytest.raises(ValueError):
        L.Q4(odd, torch.zeros((1, 1, 4), dtype=torch.uint8), 128)
    row = torch.zeros((3, 5, 64), dtype=torch.uint8)[:, 2:3]                 # one row of three panels
    q = L.Q4(row, torch.zeros((3, 1, 4), dtype=torch.uint8), 384)
    assert (q._c.ld, q._c.ld_exps) == (320, 4)


def test_reference_rounding_is_nearest_even_on_every_code():
    """The 64-bit rounding against a search over the whole e2m1 table."""
    g = R.GRID
    mids = (g[1:] + g[:-1]) / 2
    for v in np.concatenate([g, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9)]):
        d = np.abs(g - v)
        near = np.flatnonzero(d == d.min())
        want = g[near[0]] if len(near) == 1 else g[[n for n in near if n % 2 == 0][0]]
        assert R.round_e2m1(np.array([v]))[0] == want, v


def test_reference_exponent_is_the_smallest_that_fits():
    rng = np.random.default_rng(0)
    x = np.ldexp(rng.uniform(0.5, 1, 500), rng.integers(-130, 128, 500))[:, None]
    e = R.block_exponents(x)[:, 0]
    assert np.all(x[:, 0] <= np.ldexp(6.0, e - 127))
    assert np.all((x[:, 0] > np.ldexp(6.0, e - 128)) | (e == 1))
    top = np.array([[float(torch.finfo(torch.bfloat16).max)], [2.0 ** -133], [0.0], [np.inf], [np.nan]])
    assert R.block_exponents(top)[:, 0].tolist() == [253, 1, 1, 255, 255]


def test_every_kernel_of_the_product_is_reached_by_a_tested_size():
    """The sizes that the GPU tests multiply take every kernel, ragged in each
    direction, with short sums and (8-bit rows) with sums behind its staged
    exponents. The choice is made from measured times, so another fit of them
    moves sizes from one kernel to another: this says when the list has to follow."""
    for bits in (4, 8):
        chosen = {}
        for b, T, K, N in PRODUCTS:
            if b != bits:
                continue
            k = B.inspect_matmul4(bits, T, K, N)
            if k.stages:
                assert T > k.tokens and N > k.columns, (T, K, N)     # more than one tile each way
                assert T % k.tokens
            assert N % k.columns and K % 128, (T, K, N)
            chosen.setdefault(k.kernel, []).append(k)
        assert sorted(chosen) == list(range(k.kernels))
        for ks in chosen.values():
            if ks[0].stages == 0:
                assert any(q.blocks > 1 for q in ks)
                continue
            assert any(q.blocks > q.stages for q in ks)
            if bits == 8:
                assert any(q.blocks > q.exps for q in ks) and any(q.stages < q.blocks <= q.exps for q in ks)


def test_matmul_inspection_refusals():
    lib, out = L.load(), B.CMatmulKernel()
    B.inspect_matmul4(4, 1, 8, 8), B.inspect_matmul4(8, 1, 8, 8)
    for args in [(4, 0, 8, 8, by(out)), (4, 1, 0, 8, by(out)), (8, 1, 8, 0, by(out)), (4, 1, 12, 8, by(out)), (4, 1, 8, 12, by(out)),
                 (4, 1, 8, 8, None), (16, 1, 8, 8, by(out))]:
        assert lib.lora_inspect_matmul4(*args) == B.LORA_INVALID_ARGUMENT


def test_long_sums_fetch_their_exponents_three_times():
    """The long sums that the GPU tests multiply take every tile, each past two refills of its staged exponents."""
    chosen = {}
    for bits, T, K, N in LONG_SUMS:
        k = B.inspect_matmul4(bits, T, K, N)
        assert bits == 8 and (k.blocks - 1) // k.exps >= 2, (T, K, N)
        chosen[k.kernel] = k
    assert sorted(chosen) == list(range(1, k.kernels))


def test_binding_names_what_is_no_store():
    q, x = L.new_q4(4, 128, device="cpu"), torch.zeros((4, 128), dtype=torch.bfloat16)
    for call in (lambda: L.q4_quantize(x, x), lambda: L.q4_quantize(x, None), lambda: L.q4_quantize(x, q, x), lambda: L.q4_dequantize(x, x),
                 lambda: L.q4_matmul(x, q, x), lambda: L.q4_matmul(q, x, x), lambda: L.q4_matmul(None, q, x)):
        with pytest.raises(ValueError, match="must be a Q4"):
            call()
