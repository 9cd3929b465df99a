"""Invariants of the compiled gfx950 code that the kernels rely on (CPU only:
hipcc cross-compiles the device code to assembly; no GPU needed).

- The shrink's LDS-destination loads are inline assembly that sets M0 to the
  LDS address: every such M0 source and buffer descriptor must be a scalar
  register, and the compiler must not use M0 anywhere else.
- No kernel spills to scratch memory (a spill would also add vector memory
  operations that the explicit load counts of the shrink do not expect).
- The output rows y are streamed: every 16-byte buffer store of the forward
  kernels (the y stores) carries the non-temporal bit, and so do the x loads
  of one-item-per-tile launches (a second form of the LDS-destination load).
- M0 and scalar registers that vector instructions wrote have aged the wait
  states that an LDS-destination load needs (one and five): the compiler does
  not insert them inside inline assembly.
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lora_adapter_batching_amd", "csrc")
HIPCC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")


def _device_asm(src, tmp_path):
    if not os.path.exists(HIPCC) and not shutil.which("hipcc"):
        pytest.skip("hipcc not available")
    out = tmp_path / (os.path.basename(src) + ".s")
    from lora_adapter_batching_amd.build import CODEGEN_FLAGS
    cmd = [HIPCC if os.path.exists(HIPCC) else "hipcc"] + CODEGEN_FLAGS + [
        "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S", "-o", str(out), src]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text()


@pytest.fixture(scope="module")
def fwd_asm(tmp_path_factory):
    return _device_asm(os.path.join(CSRC, "lora_fwd.hip"), tmp_path_factory.mktemp("asm"))


@pytest.fixture(scope="module")
def bwd_asm(tmp_path_factory):
    return _device_asm(os.path.join(CSRC, "lora_bwd.hip"), tmp_path_factory.mktemp("asm"))


def test_lds_loads_use_scalar_m0_and_descriptor(fwd_asm):
    lines = fwd_asm.splitlines()
    n_loads = n_stream = 0
    in_asm = False
    for i, l in enumerate(lines):
        s = l.split(";")[0].strip()
        if "ASMSTART" in l:
            in_asm = True
            continue
        if "ASMEND" in l:
            in_asm = False
            continue
        if not s:
            continue
        if in_asm:
            m = re.match(r"s_mov_b32 m0, (\S+)", s)
            if m:
                assert re.fullmatch(r"s\d+", m.group(1)), f"line {i}: M0 from {m.group(1)}"
            m = re.match(r"buffer_load_dwordx4 v\d+, (\S+), 0 offen( nt)? lds", s)
            if m:
                n_loads += 1
                n_stream += m.group(2) is not None
                assert re.fullmatch(r"s\[\d+:\d+\]", m.group(1)), f"line {i}: descriptor {m.group(1)}"
        else:
            assert not re.search(r"\bm0\b", s), f"line {i}: compiler use of M0: {s}"
    assert n_loads > 0
    assert 0 < n_stream < n_loads, (n_stream, n_loads)


def test_output_row_stores_are_streamed(fwd_asm):
    stores = [l.split(";")[0].strip() for l in fwd_asm.splitlines() if "buffer_store_dwordx4" in l]
    assert stores
    plain = [s for s in stores if not re.search(r"\bnt\b", s)]
    assert not plain, plain[:3]


def test_no_scratch(fwd_asm, bwd_asm):
    for text in (fwd_asm, bwd_asm):
        sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)
        assert sizes and all(int(v) == 0 for v in sizes), sizes


def test_part_loads_are_whole_device_scope_vectors(fwd_asm):
    """The split hand-off sums its parts from 16-byte device-scope loads:
    every forward kernel instance has some, and no part is read with
    narrower device-scope loads (a bit cast of a vector element once turned
    the vector loads into single-word reads of element 0)."""
    kernels = re.split(r"\n(?=_ZN4lora15sgmv_fwd_kernel\S*:)", fwd_asm)
    n = 0
    for k in kernels:
        if not k.startswith("_ZN4lora15sgmv_fwd_kernel"):
            continue
        body = k.split(".Lfunc_end")[0]
        n += 1
        assert re.search(r"buffer_load_dwordx4 .*\bsc1\b", body), k.split(":")[0]
        assert not re.search(r"buffer_load_dword v\d+, .*\bsc1\b", body), k.split(":")[0]
    assert n > 0


@pytest.fixture(scope="module")
def q8_matmul_asm(tmp_path_factory):
    return _device_asm(os.path.join(CSRC, "lora_q8_matmul.hip"), tmp_path_factory.mktemp("asm"))


def test_q8_matmul_lds_loads_scalar_operands_and_no_scratch(q8_matmul_asm):
    """The 8-bit product's LDS-destination loads: M0, the descriptor and the k
    offset are scalar registers, M0 has no other use, no kernel spills vectors
    to memory, and the steps of the main loops hold no other vector memory
    access (their explicit waits count the ring's loads)."""
    in_asm, loads = False, 0
    for l in q8_matmul_asm.splitlines():
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
    sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", q8_matmul_asm)
    assert sizes and all(int(v) == 0 for v in sizes), sizes
    # between two barriers of the main loops nothing but the ring's loads
    for k in re.split(r"\n(?=_ZN4lora\S*q8_tile_kernel\S*:)", q8_matmul_asm)[1:]:
        body = k.split(".Lfunc_end")[0]
        loops = [b for b in body.split("s_barrier") if b.count("v_mfma") and "buffer_load_dwordx4" in b]
        assert loops
        for b in loops:
            inner = re.split(r"v_mfma", b)[1:-1]
            assert not any(re.search(r"global_(load|store)|buffer_store|flat_", p) for p in inner), k.split(":")[0]


# ---------------------------------------------------------------------------
# Wait states in front of the LDS-destination loads
# ---------------------------------------------------------------------------
_SGPR = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(vcc|m0)(?:_lo|_hi)?\b")


def _scalar_registers(text):
    regs = set()
    for lo, hi, one, name in _SGPR.findall(text):
        regs |= {name} if name else {f"s{i}" for i in (range(int(lo), int(hi) + 1) if lo else [int(one)])}
    return regs


def _early_lds_loads(text):
    """(loads, those that read M0 less than one wait state after its write or a
    scalar register less than five after a vector instruction's write of it).
    Every instruction is one wait state, s_nop n is n + 1; all paths into a
    load are followed, through branches too."""
    ins, labels = [], {}                       # (opcode, operands) in order; label -> place
    for line in text.splitlines():
        s = re.split(r";|//", line)[0].strip()
        if re.fullmatch(r"[.\w$]+:", s):
            labels[s[:-1]] = len(ins)
        elif s and not s.startswith("."):
            op, _, rest = s.partition(" ")
            ins.append((op, rest))
    from_branch = {}
    for i, (op, rest) in enumerate(ins):
        if op.startswith(("s_cbranch", "s_branch")):
            from_branch.setdefault(labels[rest.strip()], []).append(i)

    def before(i):
        prev = from_branch.get(i, [])
        return prev + ([i - 1] if i and ins[i - 1][0] not in ("s_branch", "s_endpgm", "s_setpc_b64") else [])

    loads, early = 0, []
    for i, (op, rest) in enumerate(ins):
        if not op.startswith("buffer_load") or not re.search(r"\blds\b", rest):
            continue
        loads += 1
        reads, todo = _scalar_registers(rest), [(j, 0) for j in before(i)]
        while todo:
            j, waited = todo.pop()
            o, r = ins[j]
            dst = r.split(",")[0]
            if o.startswith("v_"):             # carries are the second destination
                dst += "," + r.split(",")[1] if re.search(r"_co_|div_scale", o) and "," in r else ""
                if _scalar_registers(dst) & reads:
                    early.append((i, o, r, rest, waited))
            elif waited < 1 and "m0" in _scalar_registers(dst) and not o.startswith(("s_cmp", "buffer_")):
                early.append((i, o, r, rest, waited))
            waited += int(r, 0) + 1 if o == "s_nop" else 1
            if waited < 5:
                todo += [(k, waited) for k in before(j)]
    return loads, early


def test_lds_loads_wait_for_their_scalar_registers(fwd_asm, q8_matmul_asm):
    """M0 is one wait state old and every scalar register that a vector
    instruction wrote five when an LDS-destination load reads it."""
    for text in (fwd_asm, q8_matmul_asm):
        loads, early = _early_lds_loads(text)
        assert loads > 0
        assert not early, (len(early), early[:3])


def test_wait_state_count_follows_branches_and_nops():
    """The counting itself, on short listings of each kind."""
    load = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"
    first = "v_readfirstlane_b32 s6, v0"
    for lines, n in [(["s_mov_b32 m0, s2", load], 1), (["s_mov_b32 m0, s2", "s_nop 0", load], 0),
                     ([first, "s_mov_b32 m0, s2", "s_nop 3", load], 0), ([first, "s_mov_b32 m0, s2", "s_nop 2", load], 1),
                     (["v_readfirstlane_b32 s9, v0", "s_mov_b32 m0, s2", "s_nop 0", load], 1),
                     (["v_readfirstlane_b32 s8, v0", "s_mov_b32 m0, s2", "s_nop 0", load], 0),
                     ([first, "s_cbranch_scc1 .L1", "s_nop 7", ".L1:", "s_mov_b32 m0, s2", "s_nop 1", load], 1),
                     ([first, "s_branch .L1", ".L2:", "s_endpgm", ".L1:", "s_mov_b32 m0, s2", "s_nop 3", load], 0),
                     ([".L1:", "s_mov_b32 m0, s2", "s_nop 0", load, first, "s_cbranch_scc1 .L1"], 1),
                     (["v_cmp_eq_u32_e64 s[6:7], v0, v1", "s_mov_b32 m0, s2", "s_nop 0", load], 1),
                     (["v_add_co_u32_e64 v0, s[6:7], v0, v1", "s_mov_b32 m0, s2", "s_nop 0", load], 1)]:
        loads, early = _early_lds_loads("\n".join(lines))
        assert loads == 1 and len(early) == n, lines
