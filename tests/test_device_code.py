"""A defect of hipcc 7.2 looked for in the device code that was built here: the select
of a uniform 64-bit minimum, such as `lo + step < R ? lo + step : R`, is made to take
the carry of the addition before it (scalar condition code) instead of the
comparison, which is done by a vector instruction."""
import os
import re
import shutil
import subprocess

import pytest

from byte_level_bpe_pretokenize_amd.build import LIB

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
# scalar instructions that leave the condition code as it is
KEEPS = re.compile(r"s_(mov|cmov|cselect|load|buffer_load|mul_|waitcnt|nop|branch|cbranch|barrier|ff[01]|flbit|brev|sext|"
                   r"pack|getpc|setpc|swappc|endpgm|bfm|bitset|getreg|setreg|setprio|sleep|code_end|bitreplicate)")


def selects_by_a_carry(text: str):
    """(function, instruction) of each scalar select of two values, or branch, whose condition
    is a scalar addition's or subtraction's carry.  The carry as a truth value
    (-1 or 0) is how 64-bit arithmetic goes on and is no such select."""
    found, fn, last = [], "", ""
    for line in text.splitlines():
        if (m := re.match(r"^(?:[0-9a-f]+ )?<?([\w.$]+)>?:", line)):
            # (a place that is branched to: what came before need not be what ran before)
            fn, last = (m.group(1) if m.group(1).startswith("_Z") else fn), ""
        elif (m := re.match(r"^\s+(s_\w+)\s*([^/;]*)", line)):
            op, args = m.groups()
            if op.startswith(("s_cselect", "s_cbranch_scc")):
                if last.startswith(("s_add", "s_sub")) and not args.rstrip().endswith("-1, 0"):
                    found.append((fn, f"{op} {args.strip()} after {last}"))
            elif not KEEPS.match(op):
                last = op
    return found


def test_the_search_finds_the_defect():
    """Made by hipcc 7.2 of a search in growing steps, and the same as it should be."""
    head = "_Z4findPKlllPl:\n.LBB0_6:\n"
    bad = ("\ts_add_u32 s16, s12, s2\n\ts_addc_u32 s17, s13, s3\n\tv_cmp_lt_i64_e32 vcc, s[16:17], v[6:7]\n"
           "\ts_cselect_b32 s17, s17, s7\n\ts_cselect_b32 s16, s16, s6\n")
    good = bad.replace("\ts_cselect_b32 s17", "\ts_and_b64 s[20:21], vcc, exec\n\ts_cselect_b32 s17")
    assert [x[0] for x in selects_by_a_carry(head + bad)] == ["_Z4findPKlllPl"] * 2
    assert selects_by_a_carry(head + good) == []
    truth = "\ts_add_u32 s2, s4, s6\n\ts_cselect_b64 s[12:13], -1, 0      // 000000014580: 859080C1\n"
    assert selects_by_a_carry(head + truth) == []


def test_the_library_is_free_of_it(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(LIB):
        pytest.skip("libbpe.so is not built")
    # (the objects are written beside the library that they come from)
    lib = shutil.copy(LIB, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True)
    objects = sorted(f for f in os.listdir(tmp_path) if "amdgcn" in f)
    assert objects
    kernels = 0
    for f in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", str(tmp_path / f)],
                              check=True, capture_output=True, text=True).stdout
        kernels += text.count("s_endpgm")
        assert selects_by_a_carry(text) == [], f
    assert kernels > 20
