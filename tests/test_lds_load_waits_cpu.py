"""Loads to LDS stand far enough behind the writes of the scalar registers that they read (the build's check of
its machine code, on listings and on the product's own, compiled here), and results exchanged over LDS are ordered."""
import os
import subprocess

import pytest

from gradient_sync_zr_amd import _build

LOAD = "global_load_lds_dwordx4 v2, s[4:5]"


def found(*lines):
    return _build.unwaited_lds_loads("kernel:\n" + "\n".join("\t" + x for x in lines))


def test_m0():
    write = "s_add_u32 m0, s33, 0x1000"
    assert [i for _, i in found(write, LOAD)] == [LOAD]
    assert found(write, ";;#ASMEND", "; %bb.1:", LOAD)               # nothing that runs in between
    assert not found(write, "s_nop 0", LOAD)
    assert not found(write, "v_add_u32_e32 v1, v2, v3", LOAD)
    assert found("s_mov_b32 m0, s2", "buffer_load_dword v1, s[8:11], 0 offen lds")
    assert found("s_nop 0", write, LOAD) and not found("s_add_u32 s6, s33, 0x1000", LOAD)
    assert not found(write, "global_load_dwordx4 v[0:3], v2, s[4:5]")   # not to LDS


def test_scalar_registers_written_by_vector_instructions():
    write = "v_readfirstlane_b32 s5, v7"
    assert found(write, LOAD) and found(write, "s_nop 3", LOAD) and not found(write, "s_nop 4", LOAD)
    assert found("v_cmp_lt_u32_e64 s[4:5], v0, v1", *["s_mov_b32 s9, 0"] * 4, LOAD)
    assert not found(write, *["s_mov_b32 s9, 0"] * 5, LOAD)
    assert not found("v_readfirstlane_b32 s6, v7", LOAD)


@pytest.fixture(scope="module")
def product(tmp_path_factory):
    """The product's machine code."""
    out = tmp_path_factory.mktemp("linear") / "zr_linear.s"
    cmd = [_build.HIPCC] + [f for f in _build.FLAGS if f != "-fPIC"] + \
          ["--offload-device-only", "-S", os.path.join(_build.CSRC, "zr_linear.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    return out.read_text()


def test_product(product):
    loads = [x for x in product.split("\n") if "global_load_lds_dwordx4" in x]
    writes = [x for x in product.split("\n") if "m0" in x.split(";")[0].replace(",", " ").split()]
    assert loads and len(writes) == len(loads)      # M0 is used for nothing else
    assert _build.unwaited_lds_loads(product) == []


def test_results_exchanged_over_lds_are_ordered(tmp_path):
    """The tiled product's results go through LDS within a wave: between one lane's writes and another's reads, and
    between those and the next writes, the compiler has a fence in every form."""
    out = tmp_path / "zr_linear.ll"
    cmd = [_build.HIPCC] + [f for f in _build.FLAGS if f != "-fPIC"] + \
          ["--offload-device-only", "-emit-llvm", "-S", os.path.join(_build.CSRC, "zr_linear.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    forms = [f for f in out.read_text().split("\ndefine ")[1:] if "13linear_kernel" in f.split("\n", 1)[0]]
    assert len(forms) == 14
    for form in forms:
        order = ""
        for line in form.split("\n}", 1)[0].split("\n"):
            if "store <4 x float>" in line and "ptr addrspace(3)" in line:
                order += "w"
            elif "load <4 x float>, ptr addrspace(3)" in line:
                order += "r"
            elif 'fence syncscope("wavefront")' in line:
                order += "|"
        groups = [{*g} for g in order.split("|") if g]
        assert len(groups) == 4 and all(len(g) == 1 for g in groups), order
