"""8-bit operators without a GPU: the struct's layout, every refusal (all of
them before any HIP call), calls without rows, and the 64-bit forms that the
GPU tests compare with."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import lora_adapter_batching_amd as L
from lora_adapter_batching_amd import binding as B
from tests import q8_ref as R
from tests.q8_products import PRODUCTS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 40  # an aligned stand-in address, never read


def q8(rows=4, width=256, ld=256, lde=4, block_rows=1, values=P, exps=P):
    return B.CQ8(values, ld, exps, lde, rows, width, block_rows)


def status(fn, *args):
    st = fn(*args)
    return st, L.load().lora_last_error().decode()


def test_struct_matches_the_c_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in B.CQ8._fields_]
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "lora_sgmv.h"\nint main(void) {\n'
    src += '  printf("%zu\\n", sizeof(lora_q8_t));\n'
    src += "".join(f'  printf("%zu\\n", offsetof(lora_q8_t, {n}));\n' for n in names) + "  return 0;\n}\n"
    (tmp_path / "q.c").write_text(src)
    exe = tmp_path / "q"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "q.c"), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(B.CQ8)] + [getattr(B.CQ8, n).offset for n in names]


BAD_Q8 = [
    (dict(rows=-1), "rows"), (dict(width=0), "width"), (dict(width=12), "width"), (dict(ld=255), "row stride"),
    (dict(ld=264), "row stride"), (dict(width=264, ld=272), "row stride"), (dict(lde=3), "exponent stride"),
    (dict(width=1024, ld=1024, lde=4), "exponent stride"), (dict(block_rows=2), "block_rows"),
    (dict(values=0), "NULL"), (dict(exps=0), "NULL"), (dict(values=P + 8), "aligned"), (dict(exps=P + 2), "aligned"),
]


@pytest.mark.parametrize("bad,word", BAD_Q8)
def test_every_entry_refuses_a_bad_store(bad, word):
    lib = L.load()
    b = q8(**bad)
    r = ctypes.byref(b)
    w = ctypes.byref(q8(rows=8, block_rows=128))
    wbad = ctypes.byref(q8(**{"rows": 8, "block_rows": 128, **bad}))
    calls = [(lib.lora_q8_quantize, P, 1024, r, None, None), (lib.lora_q8_dequantize, r, P, 1024, None),
             (lib.lora_q8_matmul, r, w, P, 1024, 0, None), (lib.lora_q8_matmul, ctypes.byref(q8()), wbad, P, 1024, 0, None),
             (lib.lora_swiglu, P, 2048, max(b.rows, 0), 256, None, 0, r, None),
             (lib.lora_swiglu_backward, P, 2048, P, 1024, max(b.rows, 0), 128, None, 0, r, None)]
    for fn, *args in calls:
        st, msg = status(fn, *args)
        assert st == B.LORA_INVALID_ARGUMENT, (fn, msg)
        assert word in msg, msg


def test_quantize_refusals():
    lib = L.load()
    o = q8()
    for args, word in [((0, 256, o, None), "NULL"), ((P + 4, 256, o, None), "aligned"), ((P, 248, o, None), "below its width"),
                       ((P, 260, o, None), "multiple of 8"), ((P, 256, None, None), "NULL"),
                       ((P, 256, o, q8(rows=256, width=8, ld=128, block_rows=128)), "128 x 128"),
                       ((P, 256, q8(rows=8, block_rows=128), q8(rows=248, width=8, ld=128, block_rows=128)), "transpose"),
                       ((P, 256, q8(rows=8, block_rows=128), q8(rows=256, width=8, ld=128)), "block_rows")]:
        st, msg = status(lib.lora_q8_quantize, args[0], args[1], ctypes.byref(args[2]) if args[2] else None,
                         ctypes.byref(args[3]) if args[3] else None, None)
        assert st == B.LORA_INVALID_ARGUMENT and word in msg, (args, msg)
    D = 1 << 41
    wq, wt = q8(rows=8, block_rows=128), q8(rows=256, width=8, ld=128, block_rows=128)
    for x, a, b in [(P, o, None), (P, wq, q8(rows=256, width=8, ld=128, block_rows=128, values=D)), (D, wq, wt)]:
        st, msg = status(lib.lora_q8_quantize, x, 256, ctypes.byref(a), ctypes.byref(b) if b else None, None)
        assert st == B.LORA_INVALID_ARGUMENT and "starts at" in msg, msg
    for x, ld, word in [(P, 256, "starts at"), (0, 256, "NULL"), (P + 2, 256, "aligned"), (P, 128, "below its width")]:
        st, msg = status(lib.lora_q8_dequantize, ctypes.byref(o), x, ld, None)
        assert st == B.LORA_INVALID_ARGUMENT and word in msg, msg


def test_matmul_refusals():
    lib = L.load()
    x, w = q8(), q8(rows=16, block_rows=128)
    by, D = ctypes.byref, 1 << 41
    for args, word, want in [
            ((None, by(w), P, 16, 0), "NULL", 1), ((by(x), None, P, 16, 0), "NULL", 1),
            ((by(x), by(q8(rows=16)), P, 16, 0), "block_rows", 1), ((by(w), by(w), P, 16, 0), "block_rows", 1),
            ((by(x), by(q8(rows=16, width=128, block_rows=128)), P, 16, 0), "wide", 1),
            ((by(x), by(q8(rows=12, block_rows=128)), P, 16, 0), "multiple of 8", 1),
            ((by(x), by(w), 0, 16, 0), "NULL", 1), ((by(x), by(w), P + 2, 16, 0), "aligned", 1),
            ((by(x), by(w), P, 8, 0), "below its width", 1), ((by(x), by(w), P, 20, 0), "multiple of 8", 1),
            ((by(x), by(w), P, 16, 2), "flags", 1),
            ((by(q8(ld=1 << 24)), by(w), D, 16, 0), "strides", 2), ((by(x), by(q8(rows=16, ld=1 << 24, block_rows=128)), D, 16, 0), "strides", 2),
            ((by(q8(lde=1 << 24)), by(w), D, 16, 0), "strides", 2),
            ((by(x), by(w), P, 16, 0), "starts at an operand", 1)]:
        st, msg = status(lib.lora_q8_matmul, *args, None)
        assert st == want and word in msg, (msg, word)


def test_swiglu_refusals():
    lib = L.load()
    hq, gq = q8(rows=4, width=128, ld=128), q8(rows=4, width=256)
    by = ctypes.byref
    D = 1 << 41
    for args, word in [((P, 256, -1, 128, D, 128, None), "num_tokens"), ((P, 256, 4, 12, D, 128, None), "width"),
                       ((P, 256, 4, 0, D, 128, None), "width"), ((P, 256, 4, 128, None, 0, None), "both NULL"),
                       ((0, 256, 4, 128, D, 128, None), "NULL"), ((P + 2, 256, 4, 128, D, 128, None), "aligned"),
                       ((P, 248, 4, 128, D, 128, None), "below its width"), ((P, 256, 4, 128, D, 120, None), "below its width"),
                       ((P, 256, 5, 128, None, 0, by(hq)), "expected 5"), ((P, 256, 4, 136, None, 0, by(hq)), "expected 4"),
                       ((P, 256, 4, 128, P, 256, None), "starts at"), ((P, 256, 4, 128, None, 0, by(hq)), "starts at"),
                       ((D, 256, 4, 128, P, 128, by(hq)), "starts at")]:
        st, msg = status(lib.lora_swiglu, *args, None)
        assert st == B.LORA_INVALID_ARGUMENT and word in msg, (args, msg)
    for args, word in [((P, 256, D, 128, -1, 128, D * 2, 256, None), "num_tokens"), ((P, 256, 0, 128, 4, 128, D * 2, 256, None), "NULL"),
                       ((P, 256, D, 120, 4, 128, D * 2, 256, None), "below its width"), ((P, 256, D, 128, 4, 128, None, 0, None), "both NULL"),
                       ((P, 256, D, 128, 4, 128, D * 2, 128, None), "below its width"),
                       ((P, 256, D, 128, 4, 128, None, 0, by(hq)), "expected 4 x 256"), ((P, 256, D, 128, 5, 128, None, 0, by(gq)), "expected 5"),
                       ((P, 256, D, 128, 4, 128, P, 256, None), "starts at"), ((P, 256, D, 128, 4, 128, D, 256, None), "starts at"),
                       ((D, 256, P, 128, 4, 128, None, 0, by(gq)), "starts at"), ((P, 256, D, 128, 4, 128, None, 0, by(gq)), "starts at")]:
        st, msg = status(lib.lora_swiglu_backward, *args, None)
        assert st == B.LORA_INVALID_ARGUMENT and word in msg, (args, msg)


def _backward_args(x=None, T=4, rows=None, u=P, **seg):
    ranks, scales = np.array([4, 8], np.int32), np.ones(2, np.float32)
    ad = B.CAdapters(2, 256, 128, P, P, ranks.ctypes.data, scales.ctypes.data, 0, 0)
    starts, adap = np.array([0, T], np.int32), np.array([0], np.int32)
    sg = B.CSegments(T, 1, starts.ctypes.data, adap.ctypes.data, seg.get("rows_dev", 0), 0)
    xs = x if x is not None else q8(rows=T if rows is None else rows)
    keep = (ranks, scales, starts, adap, ad, sg, xs)
    return keep, (ctypes.byref(xs), P, 128, u, 8, ctypes.byref(ad), ctypes.byref(sg), P, 256, P, P)


def test_backward_refusals():
    lib = L.load()

    def call(want, word, args, flags=0, ws=P, wb=1 << 40):
        keep, a = args
        st, msg = status(lib.lora_packed_backward_q8, *a, flags, ws, wb, None)
        assert st == want and word in msg, msg

    call(1, "u is NULL", _backward_args(u=0))
    call(1, "x has 3 rows", _backward_args(rows=3))
    call(1, "wide", _backward_args(x=q8(width=128)))
    call(1, "block_rows", _backward_args(x=q8(block_rows=128)))
    call(1, "values/exps", _backward_args(x=q8(values=0)))
    call(2, "strides", _backward_args(x=q8(ld=1 << 26)))
    call(1, "gather limit", _backward_args(x=q8(rows=200, ld=1 << 24), T=200, rows_dev=P))
    call(1, "exponent stride", _backward_args(x=q8(lde=512), rows_dev=P))
    call(1, "flags", _backward_args(), flags=2)
    call(3, "workspace", _backward_args(), wb=16)
    keep, a = _backward_args()
    st, msg = status(lib.lora_packed_backward_q8, None, *a[1:], 0, P, 1 << 40, None)
    assert st == 1 and "x is NULL" in msg


def test_more_than_one_launch_holds_is_refused():
    """Grids of 2^32 threads and more (stand-in addresses: nothing is launched)."""
    lib = L.load()
    by, big, D = ctypes.byref, 0x7fffff00, 1 << 41
    for fn, *args in [(lib.lora_q8_quantize, D, 4096, by(q8(rows=big, width=4096, ld=4096, lde=32)), None),
                      (lib.lora_q8_quantize, D, 1 << 20, by(q8(rows=big, width=1 << 20, ld=1 << 20, lde=1 << 13, block_rows=128)), None),
                      (lib.lora_q8_dequantize, by(q8(rows=big, width=4096, ld=4096, lde=32)), D, 4096),
                      (lib.lora_q8_matmul, by(q8(rows=big)), by(q8(rows=big, block_rows=128)), D, big, 0),
                      (lib.lora_swiglu, D, 8192, big, 4096, 2 * D, 4096, None),
                      (lib.lora_swiglu_backward, D, 8192, 4 * D, 4096, big, 4096, 2 * D, 8192, None)]:
        st, msg = status(fn, *args, None)
        assert st == B.LORA_UNSUPPORTED, (fn, st, msg)


def test_no_rows_is_no_work():
    """No HIP call is made without rows: these succeed without a GPU."""
    lib = L.load()
    by = ctypes.byref
    e = q8(rows=0, values=0, exps=0)
    assert lib.lora_q8_quantize(None, 0, by(e), None, None) == 0
    assert lib.lora_q8_dequantize(by(e), None, 0, None) == 0
    assert lib.lora_q8_matmul(by(e), by(q8(rows=8, block_rows=128)), None, 0, 0, None) == 0
    assert lib.lora_q8_matmul(by(q8()), by(q8(rows=0, block_rows=128)), None, 0, 0, None) == 0
    assert lib.lora_swiglu(None, 0, 0, 256, P, 256, by(e), None) == 0
    assert lib.lora_swiglu_backward(None, 0, None, 0, 0, 128, None, 0, by(e), None) == 0


def test_binding_refuses_wrong_tensors():
    v, e = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8)
    L.Q8Rows(v, e, 256), L.Q8Rows(v.view(torch.float8_e4m3fn), e, 136), L.Q8Rows(v, e, 256, rows=2)
    for args in [(v.float(), e, 256), (v, e.int(), 256), (v, e, 264), (v.t(), e, 4), (v, e[:3], 256), (v, e[:, :1], 256),
                 (v[0], e, 256)]:
        with pytest.raises(ValueError):
            L.Q8Rows(*args)
    with pytest.raises(ValueError):
        L.Q8Rows(v, e, 256, rows=5)
    with pytest.raises(ValueError):  # a stride of two bytes holds two blocks, but not in whole dwords
        L.Q8Rows(v, torch.zeros((4, 2), dtype=torch.uint8), 256)
    q, w = L.new_q8_rows(4, 256, "cpu"), L.new_q8_weights(16, 256, "cpu")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    for fn, args in [(L.q8_quantize, (bf(3, 256), q)), (L.q8_quantize, (bf(4, 128), q)), (L.q8_quantize, (torch.zeros(4, 256), q)),
                     (L.q8_dequantize, (q, bf(4, 255))), (L.q8_matmul, (q, w, bf(4, 8))), (L.q8_matmul, (q, w, bf(3, 16))),
                     (L.swiglu, (bf(4, 256), bf(4, 256))), (L.swiglu, (torch.zeros(4, 256), bf(4, 128))),
                     (L.swiglu_backward, (bf(4, 256), bf(4, 120), bf(4, 256))), (L.swiglu_backward, (bf(4, 256), bf(4, 128), bf(4, 128)))]:
        with pytest.raises(ValueError):
            fn(*args)
    with pytest.raises(ValueError, match="device tensors"):
        L.q8_quantize(bf(4, 256), q)


def test_reference_rounding_is_nearest_even_on_every_code():
    """The 64-bit rounding against a search over the whole e4m3 table."""
    grid = np.unique(R.TABLE[np.isfinite(R.TABLE) & (R.TABLE >= 0)])
    assert grid[-1] == 448 and len(grid) == 127
    mids = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9), [0.0]])
    got = R.round_e4m3(v)
    for x, q in zip(v, got):
        d = np.abs(grid - x)
        near = np.flatnonzero(d == d.min())
        want = grid[near[0]] if len(near) == 1 else grid[[n for n in near if n % 2 == 0][0]]
        assert q == want, x


def test_reference_exponent_is_the_smallest_that_fits():
    rng = np.random.default_rng(0)
    x = np.ldexp(rng.uniform(0.5, 1, 500), rng.integers(-130, 128, 500))[:, None]
    e = R.block_exponents(x, 1)[:, 0]
    assert np.all(x[:, 0] <= np.ldexp(448.0, e - 127))
    assert np.all((x[:, 0] > np.ldexp(448.0, e - 128)) | (e == 1))


def test_reference_swiglu_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, dh = rng.standard_normal((3, 32)) * 2, rng.standard_normal((3, 16))
    g = R.swiglu_grad(x, dh)
    step = 1e-6
    for i in range(3):
        for j in range(32):
            d = np.zeros_like(x)
            d[i, j] = step
            num = (np.sum(dh * R.swiglu(x + d)[3]) - np.sum(dh * R.swiglu(x - d)[3])) / (2 * step)
            assert abs(num - g[i, j]) < 1e-7 * (1 + abs(num)), (i, j)  # step^2 and 1e-16 / step


def test_binding_refuses_a_u_that_is_narrower_than_its_ranks():
    """A column slice has the stride of the matrix it is cut from, so only its
    width says that it does not hold the ranks."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    ad = L.Adapters([bf(16, 256), bf(8, 256)], [bf(64, 16), bf(64, 8)], [16, 8], [1.0, 1.0], 256, 64, device="cpu")
    q, dy, tab = L.new_q8_rows(4, 256, "cpu"), bf(4, 64), torch.zeros(2, dtype=torch.int64)
    full = torch.zeros((4, 64))
    wide, narrow = L.Segments([0, 2, 4], [0, -1]), L.Segments([0, 4], [1])
    call = lambda u, seg: L.packed_backward_q8(q, dy, u, ad, seg, None, tab, tab)  # noqa: E731
    for u, seg in [(full[:, :8], wide), (full[:, 56:], wide), (full[:, :4], narrow), (full[:3], narrow), (full.double(), narrow),
                   (torch.zeros((4, 64), dtype=torch.int32), narrow), (full.t(), narrow), (None, narrow)]:
        with pytest.raises(ValueError, match="u must be"):
            call(u, seg)
    for u, seg in [(full, wide), (full[:, :16], wide), (full[:, :8], narrow)]:
        with pytest.raises(ValueError, match="device tensors"):
            call(u, seg)


def test_binding_refuses_another_devices_stream():
    class Stream:
        device_index, cuda_stream = 1, 0

    def launch(*_):
        raise AssertionError("launched")

    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        L.binding._call_on(0, Stream(), launch)


def test_binding_takes_rows_that_no_other_follows_with_any_stride():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    one = bf(256, 1).t()                                         # [1, 256] with strides (1, 1)
    none = bf(256, 4).t()[:0]                                    # [0, 256] with strides (1, 4)
    assert L.binding._rows_arg("x", one, 1, 256, -1) == 256 and L.binding._rows_arg("x", none, 0, 256, -1) == 256
    for rows in (0, 1, 4):                                       # (a call of one token may name any of the rows)
        assert L.binding._rows_arg("x", bf(4, 264)[:, :256], rows, 256, -1) == 264
    with pytest.raises(ValueError):
        L.binding._rows_arg("x", bf(256, 2).t(), 1, 256, -1)     # a row that is itself strided


def test_binding_takes_a_single_stored_row_of_any_stride():
    """A store whose row no other follows, as a slice of a tensor of another
    layout: the strides it hands over are those of a store of its own."""
    wide = lambda n: torch.zeros((n, 1), dtype=torch.uint8).t()                   # noqa: E731  [1, n] with strides (1, 1)
    exps = torch.zeros((3, 6), dtype=torch.uint8)[1:2, :4]                        # a stride of 6
    for q, want in [(L.Q8Rows(wide(256), wide(4), 256), (256, 4)), (L.Q8Rows(wide(640), wide(8), 600), (640, 8)),
                    (L.Q8Rows(torch.zeros((1, 256), dtype=torch.uint8), exps, 256), (256, 4)),
                    (L.Q8Rows(torch.zeros((4, 264), dtype=torch.uint8)[:, :256], exps, 256, rows=1), (256, 4)),
                    (L.Q8Weights(torch.zeros((128, 256), dtype=torch.uint8), exps, 256), (256, 4)),
                    (L.Q8Rows(torch.zeros((256, 4), dtype=torch.uint8).t()[:0], torch.zeros((4, 2), dtype=torch.uint8).t()[:0], 256), (256, 4))]:
        assert (q._c.ld, q._c.ld_exps) == want
        # (the store's own checks pass: what is refused is the matrix beside it)
        st, msg = status(L.load().lora_q8_dequantize, ctypes.byref(B.CQ8(P, q._c.ld, P, q._c.ld_exps, 1, q.width, q.block_rows)), 0, 0, None)
        assert st == B.LORA_INVALID_ARGUMENT and "x is NULL" in msg, msg
    for v, e in [(wide(256), wide(2)),                                           # two bytes of exponents: not a whole dword
                 (torch.zeros((2, 256), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8).t()),  # two rows, strides (1, 2)
                 (torch.zeros((256, 2), dtype=torch.uint8).t(), torch.zeros((2, 4), dtype=torch.uint8))]:
        with pytest.raises(ValueError):
            L.Q8Rows(v, e, 256)


# Kernels of the product that no size takes with a sum behind the exponents it
# holds: two-stage 128 x 128 tiles cost more than three-stage ones from 31 blocks.
SHORT_SUMS_ONLY = {(128, 128, 2)}


def test_every_kernel_of_the_product_is_reached_by_a_tested_size():
    """The sizes that the GPU tests multiply take every kernel, ragged in each
    direction, with short sums and with sums behind its staged exponents. The
    choice is made from measured times, so another fit of them moves sizes from
    one kernel to another: this says when the list has to follow."""
    chosen = {}
    for T, K, N in PRODUCTS:
        k = B.inspect_matmul(T, K, N)
        if k.stages:
            assert T > k.tokens and N > k.columns, (T, K, N)     # more than one tile each way
        assert T % k.tokens or not k.stages, (T, K, N)
        assert N % k.columns and K % 128, (T, K, N)
        chosen.setdefault(k.kernel, []).append(k)
    assert sorted(chosen) == list(range(k.kernels))
    for kernel, ks in chosen.items():
        k = ks[0]
        long = [q for q in ks if q.blocks > q.exps]
        short = [q for q in ks if k.stages < q.blocks <= q.exps]
        if k.stages == 0:
            assert any(q.blocks > 1 for q in ks)
        else:
            assert short, (kernel, k.tokens, k.columns)
            assert long or (k.tokens, k.columns, k.stages) in SHORT_SUMS_ONLY, (kernel, k.tokens, k.columns)


def test_kernels_left_out_of_long_sums_never_take_one():
    rng = np.random.default_rng(7)
    for _ in range(20000):
        T, N = int(2 ** rng.uniform(0, 20)), 8 * int(2 ** rng.uniform(0, 14))
        k = B.inspect_matmul(T, 128 * int(rng.integers(61, 600)), N)
        assert not (k.blocks > k.exps > 0 and (k.tokens, k.columns, k.stages) in SHORT_SUMS_ONLY)


def test_matmul_inspection_refusals():
    lib, out = L.load(), B.CMatmulKernel()
    B.inspect_matmul(1, 8, 8)
    for args in [(0, 8, 8, ctypes.byref(out)), (1, 0, 8, ctypes.byref(out)), (1, 8, 0, ctypes.byref(out)), (1, 12, 8, ctypes.byref(out)),
                 (1, 8, 12, ctypes.byref(out)), (1, 8, 8, None)]:
        assert lib.lora_inspect_matmul(*args) == B.LORA_INVALID_ARGUMENT


def test_whole_number_products_show_any_misplaced_part():
    """What the GPU test of every kernel compares: with a mistake planted in
    the 64-bit form, y differs in every 32 x 32 fragment that it touches."""
    from tests.test_gpu_q8_products import exact_case
    T, K, N = 96, 1352, 264
    x, w, y0, ref, y064 = exact_case(T, K, N, 1, "cpu")
    xq, xe = R.quantize(x.double().numpy())
    wq, we = R.quantize(w.double().numpy(), 128)
    want = ref.float().to(torch.bfloat16)
    product = lambda a, b: torch.from_numpy(a @ b.T).float().to(torch.bfloat16)  # noqa: E731
    xs, ws = R.restore(xq, xe), R.restore(wq, we, 128)
    assert torch.equal(product(xs, ws), want)                    # the operands are exact, and so is the product
    same = lambda got: (got == want)[:96, :256].reshape(3, 32, 8, 32).all(3).all(1)  # noqa: E731
    for b in range(11):
        gone = ws.copy()
        gone[:, 128 * b:128 * b + 128] = 0                       # block b left out
        assert not same(product(xs, gone)).any(), b
    for b in range(10):
        turned = xe.copy()
        turned[:, [b, b + 1]] = turned[:, [b + 1, b]]            # two blocks' exponents exchanged
        if (xe[:, b] != xe[:, b + 1]).all():
            assert not same(product(R.restore(xq, turned), ws)).any(), b
    assert not same(torch.roll(want, 1, 1)).any() and not same(torch.roll(want, 1, 0)).any()
    assert not same((ref + y064).float().to(torch.bfloat16)).any()


def test_written_exponents_end_at_the_largest_finite_values():
    """The header's range of stored exponents: 1 for zeros and subnormals, 247 for the largest fp32 and bf16 values."""
    top = np.array([[np.finfo(np.float32).max], [float(torch.finfo(torch.bfloat16).max)], [2.0 ** -149], [0.0]])
    assert R.block_exponents(top, 1)[:, 0].tolist() == [247, 247, 1, 1]


def test_binding_refuses_tables_that_the_kernels_would_overrun():
    """Row and address tables of another type, shorter than the batch or the adapters, or with gaps."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    ad = L.Adapters([bf(8, 256), bf(8, 256)], [bf(64, 8), bf(64, 8)], [8, 8], [1.0, 1.0], 256, 64, device="cpu")
    q, dy, u = L.new_q8_rows(4, 256, "cpu"), bf(4, 64), torch.zeros((4, 8))
    tab, rows_ = torch.zeros(2, dtype=torch.int64), torch.arange(4, dtype=torch.int32)

    def call(rows=None, a=tab, b=tab):
        L.packed_backward_q8(q, dy, u, ad, L.Segments([0, 2, 4], [0, 1], rows), None, a, b)

    for rows in (rows_.long(), rows_[:3], torch.arange(8, dtype=torch.int32)[::2], rows_.short()):
        with pytest.raises(ValueError, match="token_rows must be"):
            call(rows)
    for bad in (tab.int(), tab[:1], torch.zeros(4, dtype=torch.int64)[::2], tab.double()):
        with pytest.raises(ValueError, match="dA_ptrs must be"):
            call(a=bad)
        with pytest.raises(ValueError, match="dB_ptrs must be"):
            call(b=bad)
    for ok in (dict(), dict(rows=rows_), dict(a=torch.zeros(3, dtype=torch.int64), b=tab.view(torch.uint64))):
        with pytest.raises(ValueError, match="device tensors"):
            call(**ok)
