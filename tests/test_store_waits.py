"""The kernels that let a tile's stores run on under the next tile's steps: in their
compiled form no store may follow a load into LDS without a wait for every load in
between. What is left to be waited for afterwards is then never counted against a
number of stores, which is the compiler's choice (it joins equal neighbours, such as
the stores of rows that are not there).

Read from the listing of the library's own gfx950 code, on the CPU."""
import os
import re
import shutil
import subprocess

import pytest

from mixture_experts_expert_amd import build

OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.HIPCC))), "llvm", "bin", "llvm-objdump")
OBJDUMP = OBJDUMP if os.path.exists(OBJDUMP) else "/opt/rocm/llvm/bin/llvm-objdump"
LOAD = re.compile(r"\bbuffer_load_\w+ .*\blds\b")
STORE = re.compile(r"\bbuffer_store_")
ALL = re.compile(r"\bs_waitcnt\b.*\bvmcnt\(0\)")


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler for gfx950")
    d = tmp_path_factory.mktemp("code")
    lib = shutil.copy(build.LIB, d)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=d, check=True, capture_output=True)
    return sorted(str(p) for p in d.iterdir() if "gfx950" in p.name)


def kernels(code, name):
    """Listings of the kernels whose mangled name holds `name`."""
    found = {}
    for obj in code:
        table = subprocess.run([OBJDUMP, "-t", obj], capture_output=True, text=True, check=True).stdout
        names = [l.split()[-1] for l in table.splitlines() if " F .text" in l and name in l]
        for n in names:
            out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f"--disassemble-symbols={n}", obj],
                                 capture_output=True, text=True, check=True).stdout
            found[n] = out.splitlines()
    return found


def unwaited(lines):
    """Stores before which a load into LDS may still be on its way, in order of the listing."""
    bad, loads = [], False
    for l in lines:
        if LOAD.search(l):
            loads = True
        elif ALL.search(l):
            loads = False
        elif STORE.search(l) and loads:
            bad.append(l.strip())
    return bad


@pytest.mark.parametrize("name, n", [("i8_duo_kernel", 3), ("i8_tile_kernel", 1), ("gate_up_ckpt8_kernel", 2),
                                     ("down_dgrad_ckpt8_kernel", 1), ("block_tile_kernel", 4)])
def test_no_store_behind_loads_into_lds(code, name, n):
    found = kernels(code, name)
    assert len(found) == n, list(found)
    for k, lines in found.items():
        assert any(LOAD.search(l) for l in lines) and any(STORE.search(l) for l in lines)
        assert unwaited(lines) == [], k


def test_the_reading_itself():
    load, store = "  buffer_load_dwordx4 v1, s[0:3], 0 offen lds", "  buffer_store_dwordx4 v[0:3], v1, s[0:3], 0 offen"
    assert unwaited([load, "  s_waitcnt vmcnt(6) lgkmcnt(0)", store]) == [store.strip()]
    assert unwaited([load, "  s_waitcnt vmcnt(0)", store, store]) == []
    assert unwaited([load, "  s_waitcnt vmcnt(0)", store, load, store]) == [store.strip()]
    assert unwaited(["  buffer_load_dwordx4 v[0:3], v1, s[0:3], 0 offen", store]) == []


def test_sum_over_split_columns_loads_each_chunk_once(code):
    """Its instance for few tokens has one band of chunks a workgroup: eight loads where the slots fit one batch, eight
    in the loop over batches. (Not about waits; it is read from the same listing.)"""
    (name, lines), = [(k, v) for k, v in kernels(code, "gather_sum_kernel").items() if "shared8" in k and "Lb1E" in k]
    assert sum("global_load_dwordx4" in l for l in lines) == 16, name
    assert sum("global_store_dwordx4" in l for l in lines) == 2, name
