"""The built attention kernels' code, read back (CPU only): where a lane
branch ends, no copy of a value that all lanes hold may stand before the
execution mask is restored, because it would move only the lanes that took the
branch.  The compiler was seen to put copies to accumulation registers there in
a kernel that fills the register file.  Two signs of it are looked for: such a
register (or a spill) touched under a mask at all, and any register copy
between the place where skipping lanes arrive and the restore."""
import os
import re
import shutil
import subprocess

import pytest

import implicit_gemm_nhwc_amd as igc

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
COPY = re.compile(r"v_accvgpr_|v_mov_b(32|64)\S* v\S+, v|scratch_")
HELD = re.compile(r"v_accvgpr_|scratch_")
RESTORE = re.compile(r"s_or_b64 exec, exec,")


def copies_before_a_restore(body):
    """[(restore, copies)] of a kernel's lines: copies in a block where lanes
    that skipped a branch arrive, before its restore of the mask."""
    joins = {x.split()[-1] for x in body if x.startswith("s_cbranch_execz")}
    found, block = [], None
    for line in body:
        if line.startswith("<"):
            block = [] if line[1:].split(">")[0] in joins else None
        elif line.startswith(("s_cbranch", "s_branch")) or "saveexec" in line:
            block = None
        elif block is not None:
            if RESTORE.match(line):
                copies = [x for x in block if COPY.match(x)]
                if copies:
                    found.append((line, copies))
                block = None
            else:
                block.append(line)
    return found


def under_a_lane_branch(body, what):
    """Lines that match `what` between a change of the mask and its restore."""
    depth, found = 0, []
    for line in body:
        if "saveexec" in line:
            depth += 1
        elif RESTORE.match(line):
            depth = max(0, depth - 1)
        elif depth and what.match(line):
            found.append(line)
    return found


def kernels(lib, folder):
    """{name: lines} of the attention and norm kernels in a built library."""
    copy = os.path.join(folder, "lib.so")
    shutil.copy(lib, copy)
    subprocess.run([OBJDUMP, "--offloading", copy], cwd=folder, check=True, timeout=120,
                   stdout=subprocess.DEVNULL)
    found = {}
    for name in sorted(os.listdir(folder)):
        path = os.path.join(folder, name)
        if "gfx950" not in name:
            continue
        with open(path, "rb") as f:
            if not re.search(rb"attn_|qk_norm_", f.read()):
                continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", path],
                              check=True, timeout=300, capture_output=True, text=True).stdout
        body = None
        for line in text.split("\n"):
            line = line.split("//")[0].strip()
            start = re.search(r"<(_Z\w+)>:$", line)
            if start:
                body = found.setdefault(start.group(1), [])
            elif line and body is not None:
                body.append(line)
    return found


@pytest.fixture(scope="module", params=["LIB_PATH", "POISON_LIB_PATH"])
def built(request, tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    lib = getattr(igc, request.param)
    if not os.path.exists(lib):
        import __graft_entry__
        __graft_entry__.build()
    return request.param, kernels(lib, str(tmp_path_factory.mktemp("code")))


def test_the_scan_finds_what_it_looks_for():
    lost = ["s_and_saveexec_b64 s[0:1], vcc", "s_cbranch_execz L1", "v_add_f32_e32 v1, v2, v3",
            "<L1>:", "v_accvgpr_write_b32 a3, v1", "s_or_b64 exec, exec, s[0:1]"]
    assert copies_before_a_restore(lost) == [(lost[5], [lost[4]])]
    kept = lost[:4] + [lost[5], lost[4]]
    assert copies_before_a_restore(kept) == []
    # copies that the branch itself makes for its lanes
    assert copies_before_a_restore(lost[:2] + ["v_mov_b32_e32 v1, v2"] + kept[3:]) == []
    assert copies_before_a_restore([lost[0], "v_mov_b32_e32 v1, v2", lost[5]]) == []
    # without a jump the join has no label (the form that was seen)
    seen = [lost[0], "v_add3_u32 v5, v5, v7, v6", "v_accvgpr_write_b32 a160, v18",
            "s_mov_b64 s[2:3], s[0:1]", lost[5]]
    assert under_a_lane_branch(seen, HELD) == [seen[2]]
    assert under_a_lane_branch([lost[0], lost[5], seen[2]], HELD) == []


def test_no_copy_before_a_mask_is_restored(built):
    _, code = built
    assert sum("attn_" in n for n in code) > 100 and sum("qk_norm_" in n for n in code) > 30
    assert all(any(x.startswith("s_endpgm") for x in body) for body in code.values())
    for name, body in code.items():
        assert copies_before_a_restore(body) == [], name
        assert under_a_lane_branch(body, HELD) == [], name
