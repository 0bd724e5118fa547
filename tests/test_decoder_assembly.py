"""The built code of the decoder operators' kernels, read back (CPU only) for
the same register copies as the attention kernels' (test_attn_assembly.py), and
for what the deep pipelines count on: no wait for all loads, and no spill,
inside the loops of the products."""
import os
import re
import shutil
import subprocess

import pytest

import implicit_gemm_nhwc_amd as igc
from test_attn_assembly import (HELD, OBJDUMP, copies_before_a_restore, kernels,
                                under_a_lane_branch)

NAMES = rb"layer_norm_|quantize_rows|kv_cache_|cache_attn_|linear_i8_"


def _kernels(lib, folder):
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
            if not re.search(NAMES, f.read()):
                continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", path],
                              check=True, timeout=300, capture_output=True, text=True).stdout
        body = None
        for line in text.split("\n"):
            line = re.sub(r"^[0-9a-f]+ (<L\d+>:)$", r"\1", line.split("//")[0].strip())
            start = re.search(r"<(_Z\w+)>:$", line)
            if start:
                body = found.setdefault(start.group(1), [])
            elif line and body is not None:
                body.append(line)
    return {n: b for n, b in found.items() if re.search(NAMES.decode(), n)}


@pytest.fixture(scope="module", params=["LIB_PATH", "POISON_LIB_PATH"])
def built(request, tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    lib = getattr(igc, request.param)
    if not os.path.exists(lib):
        import __graft_entry__
        __graft_entry__.build()
    return request.param, _kernels(lib, str(tmp_path_factory.mktemp("code")))


def test_no_copy_before_a_mask_is_restored(built):
    _, code = built
    for part, least in (("layer_norm_", 50), ("quantize_rows", 28), ("kv_cache_", 12),
                        ("cache_attn_", 18), ("linear_i8_", 10)):
        assert sum(part in n for n in code) >= least, part
    for name, body in code.items():
        assert copies_before_a_restore(body) == [], name
        assert under_a_lane_branch(body, HELD) == [], name


def _product_loops(body):
    """Blocks between a label and a backward jump to it that hold a product."""
    at = {}
    loops = []
    for i, line in enumerate(body):
        if line.startswith("<"):
            at[line[1:].split(">")[0]] = i
        m = re.match(r"s_c?branch\S* (\S+)$", line)
        if m and m.group(1) in at:
            inner = body[at[m.group(1)]:i]
            if any(x.startswith("v_mfma") for x in inner):
                loops.append(inner)
    return loops


def test_no_spills(built):
    """None but two registers that the product of 256 x 256 tiles, whose sums
    fill half of the file, puts aside between its loop and its results."""
    _, code = built
    for name, body in code.items():
        spills = [x for x in body if x.startswith("scratch_")]
        assert len(spills) <= (4 if "linear_i8_tile_kernelILi0ELi256" in name
                               or "linear_i8_tile_kernelILi1ELi256" in name else 0), name
        for inner in _product_loops(body):
            assert not any(x.startswith("scratch_") for x in inner), name


def test_product_loops_do_not_drain_their_loads(built):
    """A stage's wait leaves the later ones under way: a wait for everything
    would come from a barrier that is more than a barrier."""
    _, code = built
    seen = 0
    for name, body in code.items():
        if "linear_i8_tile" not in name:
            continue
        loops = _product_loops(body)
        assert loops, name
        for inner in loops:
            seen += 1
            waits = [x for x in inner if x.startswith("s_waitcnt") and "vmcnt(0)" in x]
            stages = int(re.search(r"kernelILi\dELi\d+ELi(\d+)E", name).group(1))
            assert len(waits) <= (1 if stages == 2 else 0), (name, waits)
    assert seen >= 4


LABEL = re.compile(r"^[0-9a-f]+ (<L\d+>:)$")


def _labels(body):
    """A listing's lines with labels bare: it prints their addresses before them,
    and a rule that looks for `<` at a line's start sees none of those."""
    return [LABEL.sub(r"\1", x) for x in body]


def test_labels_are_seen():
    lost = ["s_and_saveexec_b64 s[0:1], vcc", "s_cbranch_execz L1", "v_add_f32_e32 v1, v2, v3",
            "0000000000001a40 <L1>:", "v_accvgpr_write_b32 a3, v1", "s_or_b64 exec, exec, s[0:1]"]
    assert copies_before_a_restore(_labels(lost)) == [(lost[5], [lost[4]])]


@pytest.mark.parametrize("lib", ["LIB_PATH", "POISON_LIB_PATH"])
def test_no_copy_where_a_branch_of_an_attention_kernel_arrives(lib, tmp_path):
    """The rule on the places where skipping lanes arrive, over the attention and
    norm kernels with their labels bare."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(getattr(igc, lib)):
        import __graft_entry__
        __graft_entry__.build()
    code = {n: _labels(b) for n, b in kernels(getattr(igc, lib), str(tmp_path)).items()}
    jumps = {n: {x.split()[-1] for x in b if x.startswith("s_cbranch_execz")}
             for n, b in code.items()}
    assert sum(map(bool, jumps.values())) > 100   # kernels with such branches
    for name, body in code.items():
        places = {x[1:].split(">")[0] for x in body if x.startswith("<")}
        assert jumps[name] <= places, name
        assert copies_before_a_restore(body) == [], name
