"""The empty loads of the products' rings, in the compiled gfx950 code (CPU
only). Behind a group's last block the ring's loads have empty descriptors.
The range of a buffer load ends at its descriptor's bytes less the scalar
offset, so an empty one with an offset above 0 would have a range below 0 and
depend on how that is compared: the scalar offset of every such load has to be
0 wherever its descriptor can be empty."""
import os
import re

import pytest

from tests.test_isa_invariants import CSRC, _device_asm


def scalar_offsets(text):
    """The instructions that last wrote the scalar offset of every 16-byte
    LDS-destination load, in program order, with register numbers left out."""
    ins = [s for s in (re.split(r";|//", l)[0].strip() for l in text.splitlines()) if s and not s.startswith(".") and not s.endswith(":")]
    found = []
    for i, s in enumerate(ins):
        m = re.match(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], (\S+) offen lds", s)
        if not m:
            continue
        if not re.fullmatch(r"s\d+|vcc_(lo|hi)", m.group(1)):
            found.append(m.group(1))
            continue
        for o, _, rest in (ins[j].partition(" ") for j in range(i - 1, -1, -1)):
            dst = rest.split(",")[0].strip()
            pair = re.fullmatch(r"s\[(\d+):(\d+)\]", dst)
            hit = dst == m.group(1) or pair and m.group(1)[0] == "s" and int(pair[1]) <= int(m.group(1)[1:]) <= int(pair[2])
            if hit and o.startswith(("s_", "v_")) and not o.startswith(("s_cmp", "s_bitcmp", "s_wait")):
                found.append(f"{o} " + ", ".join(re.sub(r"\d+", "N", a) if re.fullmatch(r"s\d+", a) else a
                                                 for a in (p.strip() for p in rest.split(",")[1:])))
                break
        else:
            found.append("nothing")
    return found


@pytest.mark.parametrize("source", ["lora_q4_matmul.hip", "lora_q8_matmul.hip"])
def test_scalar_offsets_can_be_zero(source, tmp_path):
    found = scalar_offsets(_device_asm(os.path.join(CSRC, source), tmp_path))
    assert found
    bad = [f for f in found if not re.fullmatch(r"s_mov_b32 0|s_cselect_b32 (0, \S+|\S+, 0)", f)]
    assert not bad, (len(bad), len(found), sorted(set(bad)))


def test_scalar_offsets_are_found():
    """The look-up itself, on a short listing."""
    load = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"
    for line, want in [("s_cselect_b32 s9, s2, 0", "s_cselect_b32 sN, 0"), ("s_mov_b32 s9, 0", "s_mov_b32 0"),
                       ("s_movk_i32 s9, 0x80", "s_movk_i32 0x80"), ("s_mov_b64 s[8:9], 0", "s_mov_b64 0")]:
        assert scalar_offsets("\n".join([line, "s_cmp_lt_i32 s9, s2", "s_mov_b32 m0, s3", "s_nop 0", load])) == [want]
