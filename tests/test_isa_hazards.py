"""Wait states of the built library's code that the compiler does not keep inside
inline assembly: the code objects are disassembled and every load to shared memory is
looked at.  On gfx950 such a load takes its base from m0, one wait state after a
scalar write of it at the earliest, and a memory instruction reads a scalar register
five wait states after a vector instruction wrote it.  m0 cannot be listed as
overwritten by an asm block, so in a kernel with such loads nothing else may use it."""
import os
import re
import shutil
import subprocess

import pytest

import draft_token_verification_vocab_amd as sv

LLVM = "/opt/rocm/llvm/bin/llvm-objdump"
OBJDUMP = LLVM if os.path.exists(LLVM) else shutil.which("llvm-objdump")

SCALAR = re.compile(r"\bs(\d+)\b|\bs\[(\d+):(\d+)\]|\b(vcc)\b")


def scalars(text):
    """The scalar registers that text names."""
    found = set()
    for one, low, high, vcc in SCALAR.findall(text):
        if vcc:
            found.add("vcc")
        elif one:
            found.add(int(one))
        else:
            found.update(range(int(low), int(high) + 1))
    return found


def waits(instruction):
    """Wait states that an instruction makes up."""
    op, _, rest = instruction.partition(" ")
    return int(rest, 0) + 1 if op == "s_nop" else 1


def to_shared(instruction):
    op = instruction.split()[0]
    return op.startswith(("global_load_lds", "buffer_load")) and (
        "_lds" in op or re.search(r"\blds\b", instruction) is not None)


def hazards(lines):
    """(loads to shared memory, those too close behind what they read, functions with
    such loads that name m0 beside their writes for each)."""
    loads, bad, before, name = 0, [], [], None
    names, per = {}, {}
    for line in lines:
        label = re.match(r"[0-9a-f]* ?<(.*)>:", line)
        if label:
            name, before = label.group(1), []
            continue
        text = " ".join(line.split("//")[0].split())
        if not re.match(r"[a-z]", text):
            continue
        if re.search(r"\bm0\b", text):
            names[name] = names.get(name, 0) + 1
        if to_shared(text):
            loads += 1
            per[name] = per.get(name, 0) + 1
            reads, since = scalars(text), 0
            for old in reversed(before):
                op, _, args = old.partition(" ")
                written = args.split(",")[0]
                if since < 1 and op.startswith("s_") and written == "m0":
                    bad.append((name, old, text))
                if op.startswith("v_") and scalars(written) & reads:
                    bad.append((name, old, text))
                since += waits(old)
                if since >= 5:
                    break
        before = before[-5:] + [text]
    return loads, bad, [f for f in per if names.get(f, 0) != per[f]]


def test_the_scan_finds_what_it_looks_for():
    near = ["0 <f>:", " s_mov_b32 m0, s3  // 00: 00", " global_load_lds_dwordx4 v1, s[4:5]"]
    assert hazards(near) == (
        1, [("f", "s_mov_b32 m0, s3", "global_load_lds_dwordx4 v1, s[4:5]")], [])
    assert hazards(near[:2] + [" s_nop 0"] + near[2:]) == (1, [], [])
    assert hazards(near[:2] + [" v_add_u32_e32 v2, v3, v4"] + near[2:]) == (1, [], [])
    lane = ["0 <f>:", " v_readlane_b32 s5, v7, 3", " s_mov_b32 m0, s3", " s_nop 2"] + near[2:]
    assert len(hazards(lane)[1]) == 1
    lane[3] = " s_nop 3"
    assert hazards(lane) == (1, [], [])
    assert hazards(near + [" s_mov_b32 s9, m0"])[2] == ["f"]
    near[2] = " buffer_load_dwordx4 v1, s[0:3], 0 offen lds"
    assert len(hazards(near)[1]) == 1
    near[2] = " buffer_load_dwordx4 v[0:3], v5, s[0:3], 0"
    assert hazards(near) == (0, [], [])


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_loads_to_shared_memory_wait_for_what_they_read(tmp_path):
    if not os.path.exists(sv.lib_path()):
        from draft_token_verification_vocab_amd import build
        build.build()
    shutil.copy(sv.lib_path(), tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True,
                   capture_output=True)
    objects = [p for p in sorted(tmp_path.iterdir()) if "gfx950" in p.name and p.stat().st_size]
    assert objects
    loads = 0
    for path in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], check=True,
                              capture_output=True, text=True).stdout
        n, bad, others = hazards(text.splitlines())
        loads += n
        assert not bad, (len(bad), bad[:3])
        assert not others
    assert loads > 0
