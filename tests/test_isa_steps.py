"""The steps of the products' main loops in the compiled gfx950 code (CPU only):
their explicit waits count the ring's loads, so a step holds exactly those and
no other access that the same counter would count."""
import os
import re

import pytest

from tests.test_isa_invariants import CSRC, _device_asm

VECTOR_MEMORY = re.compile(r"(buffer|global|flat|scratch|tbuffer|image)_")


def listing(body):
    """(instructions, label -> place) of one kernel."""
    ins, labels = [], {}
    for line in body.splitlines():
        s = re.split(r";|//", line)[0].strip()
        if re.fullmatch(r"[.\w$]+:", s):
            labels[s[:-1]] = len(ins)
        elif s and not s.startswith("."):
            ins.append(s)
    return ins, labels


def innermost_loops(body):
    """The instructions from the target of each backward branch to the branch, without those that hold another."""
    ins, labels = listing(body)
    spans = []
    for i, s in enumerate(ins):
        op, _, target = s.partition(" ")
        if op.startswith(("s_cbranch", "s_branch")) and labels.get(target.strip(), i + 1) <= i:
            spans.append((labels[target.strip()], i))
    inner = [a for a in spans if not any(b != a and a[0] <= b[0] and b[1] <= a[1] for b in spans)]
    return [ins[a:b + 1] for a, b in inner]


def steps(text, kernel):
    """(template arguments, the loops that multiply) of every instance of a kernel."""
    for k in re.split(rf"\n(?=_ZN4lora\S*{kernel}\S*:)", text)[1:]:
        name, body = k.split(":", 1)
        args = [int(v) for v in re.findall(r"L[ib](\d+)E", name)]
        loops = [l for l in innermost_loops(body.split(".Lfunc_end")[0]) if any(i.startswith("v_mfma") for i in l)]
        yield name, args, loops


def check_step(name, loop, loads, stages, multiplications):
    memory = [i for i in loop if VECTOR_MEMORY.match(i)]
    ring = [i for i in memory if re.match(r"buffer_load_dword(x4)? .* lds$", i)]
    assert len(ring) == loads and len(memory) == loads, (name, len(ring), loads, [i for i in memory if i not in ring][:3])
    assert sum(i.startswith("v_mfma") for i in loop) == multiplications, name
    waits = [i for i in loop if i.startswith("s_waitcnt") and "vmcnt" in i]
    assert [re.search(r"vmcnt\((\d+)\)", i).group(1) for i in waits] == [str((stages - 2) * loads)], (name, waits)


def up(a, b):
    return -(-a // b)


def test_steps_on_four_bit_weights(tmp_path):
    n = 0
    for name, args, loops in steps(_device_asm(os.path.join(CSRC, "lora_q4_matmul.hip"), tmp_path), "q4_tile_kernel"):
        bt, bn, wt, wn, s, x8, ks, _, _ = args
        waves = wt * wn
        pieces = bn // 16 + bt * (128 if x8 else 64) // 1024
        loads = up(pieces, waves) + up(up(bn, 64) + (0 if x8 else up(bt, 64)), waves)
        assert len(loops) == 1, (name, len(loops))
        check_step(name, loops[0], loads, s, 2 * (bt // wt // 32) * (bn // wn // 32))
        n += 1
    assert n == 2 * 20  # ten tiles for either form of x, stored and added to


def test_steps_on_eight_bit_weights(tmp_path):
    n = 0
    for name, args, loops in steps(_device_asm(os.path.join(CSRC, "lora_q8_matmul.hip"), tmp_path), "q8_tile_kernel"):
        bt, bn, wt, wn, s, ks, _, _ = args
        assert len(loops) == 1, (name, len(loops))
        check_step(name, loops[0], (bn + bt) // 8 // (wt * wn), s, 2 * (bt // wt // 32) * (bn // wn // 32))
        n += 1
    assert n == 2 * 8


def test_the_check_itself():
    step = "\n".join([".L1:", "buffer_load_dwordx4 v1, s[4:7], s9 offen lds", "v_mfma_f32_x v[0:3], v1, v2", "s_waitcnt vmcnt(2)",
                      "buffer_load_dword v1, s[4:7], s9 offen lds", "s_cbranch_scc1 .L1"])
    outer = "\n".join([".L0:", step, "s_branch .L0"])
    loop, = innermost_loops(outer)
    check_step("k", loop, 2, 3, 1)
    for other in ("buffer_load_dword v1, v0, s[4:7], 0 offen", "scratch_load_dword v1, off, s0", "global_store_dword v0, v1, off",
                  "s_waitcnt vmcnt(0)", "buffer_load_dword v1, s[4:7], s9 offen lds", "v_mfma_f32_x v[0:3], v1, v2"):
        with pytest.raises(AssertionError):
            check_step("k", loop[:2] + [other] + loop[2:], 2, 3, 1)
