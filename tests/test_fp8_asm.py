"""Static checks of the gfx950 assembly of the 8-bit expert kernels (CPU only).

1. No instruction touches the destination of an LDS read before a wait has
   retired it, by the analysis of tests/asm_check.py with one refinement: where
   two paths meet with the same newest reads in flight (the MFMA-tile kernel
   carries reads over its loop's back edge), their order is kept, so that a
   wait for all but the N newest of them counts.
2. No scalar load inside the MFMA-tile kernel's item loop: scalar loads return
   out of order and would spoil those counts.
3. The stage loops keep everything in registers, and the streaming kernel's
   loop never waits for all of its loads.
4. No packed fp32 arithmetic anywhere in the new units.
"""
import re
import subprocess

import pytest

import tests.asm_check as A
from routed_expert_ffn_03_amd.build import CSRC, HIPCC_FLAGS
from tests.test_kernel_asm import _hipcc

UNITS = ["fp8_fat.hip", "fp8_ffn.hip", "fp8_quant.hip", "balance.hip", "combine_bwd.hip"]


def merge_keeping_order(a, b):
    """Join of two in-flight states: the newest reads that both have, in order; the rest in any order."""
    if a == b:
        return a
    ra, rb = list(a[1]), list(b[1])
    n = 0
    while n < min(len(ra), len(rb)) and (ra[-1 - n][0], ra[-1 - n][2]) == (rb[-1 - n][0], rb[-1 - n][2]):
        n += 1
    rest = {(x[0], x[2]): x for x in [*a[0], *b[0], *ra[:len(ra) - n], *rb[:len(rb) - n]]}
    return (frozenset(rest.values()), tuple(ra[len(ra) - n:]))


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    out = {}
    for u in UNITS:
        s = tmp_path_factory.mktemp("asm") / (u + ".s")
        res = subprocess.run([hipcc, *HIPCC_FLAGS, "--cuda-device-only", "-S", f"{CSRC}/{u}", "-o", str(s)],
                             capture_output=True, text=True, timeout=900)
        assert res.returncode == 0, res.stderr[-2000:]
        out[u] = s.read_text()
    return out


def test_join_keeps_the_common_newest_reads():
    r = lambda *regs: (frozenset(regs), 1, False)
    a = (frozenset(), (r("v0"), r("v4"), r("v8")))
    b = (frozenset(), (r("v9"), r("v4"), r("v8")))
    old, new = merge_keeping_order(a, b)
    assert [x[0] for x in new] == [frozenset({"v4"}), frozenset({"v8"})]
    assert {x[0] for x in old} == {frozenset({"v0"}), frozenset({"v9"})}


def test_no_lds_result_used_before_its_wait(asm, monkeypatch):
    monkeypatch.setattr(A, "_merge", merge_keeping_order)
    seen = 0
    for u in ("fp8_fat.hip", "fp8_ffn.hip"):
        for name, lines in A.kernel_bodies(asm[u]).items():
            bad = A.stale_lds_uses(lines)
            assert not bad, (name, bad[:3])
            seen += "ffn_fp8" in name
    assert seen == 4


def _loops(lines):
    """The lines of every innermost loop: its header block and every block tagged as inside it."""
    starts = [i for i, x in enumerate(lines) if re.match(r"^(\.LBB\w+:|; %bb\.\d+:)", x.strip())]
    blocks = [lines[i:j] for i, j in zip(starts, starts[1:] + [len(lines)])]
    out = []
    for blk in blocks:
        if not any("Inner Loop Header" in x for x in blk[:3]):
            continue
        tag = "Header=" + blk[0].strip().split(":")[0][2:] + " "
        out.append([x for b in blocks if b is blk or any(tag in y for y in b[:3]) for x in b])
    return out


def test_stage_loops_stay_in_registers(asm):
    for u in ("fp8_fat.hip", "fp8_ffn.hip"):
        for name, lines in A.kernel_bodies(asm[u]).items():
            if "ffn_fp8" not in name:
                continue
            loops = [b for b in _loops(lines) if any("v_mfma" in x for x in b)]
            assert len(loops) >= (7 if "fat" in name else 1), name
            for body in loops:
                assert not [x for x in body if "scratch_" in x], name
                if "stream" in name:
                    assert not [x for x in body if re.search(r"vmcnt\(0\)", x)], name
                    assert sum(" lds" in x and "buffer_load_dwordx4" in x for x in body) >= 8
                else:
                    assert not [x for x in body if re.match(r"\s*s_(buffer_)?load", x)], name


def test_no_scalar_load_in_the_item_loop(asm):
    for name, lines in A.kernel_bodies(asm["fp8_fat.hip"]).items():
        if "ffn_fp8_fat" not in name:
            continue
        first = next(i for i, x in enumerate(lines) if "This Loop Header: Depth=1" in x)
        assert not [x for x in lines[first:] if re.match(r"\s*s_(buffer_)?load", x)], name


def test_no_packed_fp32_arithmetic(asm):
    for u, text in asm.items():
        assert not re.search(r"v_pk_(add|mul|fma)_f32", text), u
