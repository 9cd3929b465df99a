"""Invariants of the compiled gfx950 code of the 4-bit product and of the
query/key norm (CPU only: hipcc cross-compiles the device code to assembly)."""
import os
import re

import pytest

from tests.test_isa_invariants import CSRC, _device_asm, _early_lds_loads


@pytest.fixture(scope="module")
def product_asm(tmp_path_factory):
    return _device_asm(os.path.join(CSRC, "lora_q4_matmul.hip"), tmp_path_factory.mktemp("asm"))


def test_lds_loads_scalar_operands(product_asm):
    """M0, the descriptor and the offset of every LDS-destination load are
    scalar registers, and M0 has no other use."""
    in_asm, loads = False, 0
    for l in product_asm.splitlines():
        if "ASMSTART" in l or "ASMEND" in l:
            in_asm = "ASMSTART" in l
            continue
        s = l.split(";")[0].strip()
        if in_asm:
            m = re.match(r"s_mov_b32 m0, (\S+)", s)
            if m:
                assert re.fullmatch(r"s\d+|vcc_(lo|hi)", m.group(1)), s
            if s.startswith("buffer_load"):
                loads += 1
                assert re.fullmatch(r"buffer_load_dword(x4)? v\d+, s\[\d+:\d+\], (s\d+|vcc_(lo|hi)) offen lds", s), s
        else:
            assert not re.search(r"\bm0\b", s), s
    assert loads > 0


def test_lds_loads_wait_for_their_scalar_registers(product_asm):
    """M0 is one wait state old and every scalar register that a vector
    instruction wrote five when an LDS-destination load reads it."""
    loads, early = _early_lds_loads(product_asm)
    assert loads > 0
    assert not early, (len(early), early[:3])


def test_main_loops_hold_the_rings_loads_alone(product_asm):
    """Between two barriers of the main loops there is no other vector memory
    access: their explicit waits count the ring's loads."""
    n = 0
    for k in re.split(r"\n(?=_ZN4lora\S*q4_tile_kernel\S*:)", product_asm)[1:]:
        body = k.split(".Lfunc_end")[0]
        loops = [b for b in body.split("s_barrier") if b.count("v_mfma") and "buffer_load_dwordx4" in b]
        assert loops
        n += 1
        for b in loops:
            inner = re.split(r"v_mfma", b)[1:-1]
            assert not any(re.search(r"global_(load|store)|buffer_store|flat_", p) for p in inner), k.split(":")[0]
    assert n > 0


def test_no_scratch(product_asm, tmp_path):
    for text in (product_asm, _device_asm(os.path.join(CSRC, "lora_qk.hip"), tmp_path), _device_asm(os.path.join(CSRC, "lora_q4.hip"), tmp_path)):
        sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)
        assert sizes and all(int(v) == 0 for v in sizes), sizes
