"""The library's device code, as built: where branches that lanes took apart join again, the execution mask is restored
before anything is computed, spilled or reloaded for all of them.

The compiler places spills (and constants that it makes anew) at the head of a join at times, ahead of that restore: lanes
that were not in the branch then lose what the others keep.  Where registers are scarce such a kernel is wrong only for the
lengths that leave lanes out, so its instructions are looked at, not its results alone.

CPU only; the disassembler is the one of the toolchain that builds the library."""
import os
import re
import subprocess

import pytest

import draft_selection_amd as ds

TOOLS = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
VECTOR = re.compile(r"(v_(?!readlane|writelane|readfirst|nop)|scratch_|global_|ds_|flat_|buffer_)")


def disassembly(lib, where):
    fat, dev, copy = (os.path.join(where, n) for n in ("fat", "dev.o", "copy.so"))
    run = lambda tool, *a: subprocess.run([os.path.join(TOOLS, tool), *a], check=True, capture_output=True, text=True).stdout
    run("llvm-objcopy", "--dump-section", f".hip_fatbin={fat}", lib, copy)
    run("clang-offload-bundler", "--type=o", "--unbundle", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--input={fat}",
        f"--output={dev}")
    return run("llvm-objdump", "-d", dev)


def late_restores(text):
    """(kernel, address, instructions ahead of the restore) of every join that has any."""
    found, functions = [], 0
    for part in re.split(r"\n(?=[0-9a-f]{16} <)", text):
        head = re.match(r"[0-9a-f]{16} <(\S+)>:", part)
        if not head:
            continue
        functions += 1
        ins, at, saved, joins, targets = [], {}, None, {}, set()
        for line in part.split("\n")[1:]:
            m = re.match(r"\t(\S.*?)\s*// ([0-9A-F]+): \S+.*?(?:<\S+\+0x([0-9a-f]+)>)?$", line)
            if not m:
                continue
            op, addr = m.group(1), int(m.group(2), 16)
            at[addr] = len(ins)
            ins.append((op, addr))
            s = re.match(r"s_\w+_saveexec_b64 (s\[\d+:\d+\]|vcc)", op)
            if s:
                saved = s.group(1)
            s = re.match(r"s_xor_b64 (s\[\d+:\d+\]), exec, (s\[\d+:\d+\])", op)
            if s and s.group(2) == saved:
                saved = s.group(1)
            if re.match(r"s_c?branch", op) and m.group(3):
                to = ins[0][1] + int(m.group(3), 16)
                targets.add(to)
                if op.startswith("s_cbranch_execz"):
                    joins.setdefault(to, set()).add(saved)
        for addr, masks in joins.items():
            ahead = []
            for op, here in ins[at.get(addr, len(ins)):]:
                if here != addr and here in targets:  # a block of its own
                    break
                r = re.match(r"s_or_b64 exec, exec, (s\[\d+:\d+\]|vcc)", op)
                if r:
                    if ahead and r.group(1) in masks:
                        found.append((head.group(1), hex(addr), ahead))
                    break
                if re.match(r"s_(c?branch|endpgm|\w+_saveexec)", op):
                    break
                if VECTOR.match(op):
                    ahead.append(op)
    return found, functions


def test_masks_are_restored_first(tmp_path):
    if not all(os.path.exists(os.path.join(TOOLS, t)) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-objdump")):
        pytest.skip("no disassembler")
    found, functions = late_restores(disassembly(ds.LIB_PATH, str(tmp_path)))
    assert functions > 100
    assert not found, [(k, a, len(x), x[:3]) for k, a, x in found]


def test_the_search_finds_one():
    """A join whose mask comes late, and the same one in order."""
    def text(*tail):
        ops = ["s_and_saveexec_b64 s[0:1], vcc", "s_cbranch_execz 1", "v_mov_b32_e32 v1, v2", *tail, "s_endpgm"]
        return "\n" + "0" * 16 + " <k>:\n" + "\n".join(
            f"\t{op:<60} // {0x100 + 4 * i:012X}: BF880000" + (" <k+0xc>" if "execz" in op else "") for i, op in enumerate(ops))
    late = text("scratch_store_dword off, v3, off", "s_or_b64 exec, exec, s[0:1]")
    assert [(k, x) for k, _, x in late_restores(late)[0]] == [("k", ["scratch_store_dword off, v3, off"])]
    assert late_restores(text("s_or_b64 exec, exec, s[0:1]", "scratch_store_dword off, v3, off"))[0] == []
