"""Waits of the windowed-attention kernels on the tensor cores are bounded, so that a step that never comes ends in a
status and not in a hang.  Read from the source: a kernel that waits for ever must not run."""

import os
import re
import shutil
import subprocess

import pytest

from delta_rule_recurrent_scan_b200 import build

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "delta_rule_recurrent_scan_b200", "csrc")
FILES = ["window_attn_tc.cu", "window_bwd_tc.cu", "window_tc.cuh"]


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def _kernels(text):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__[^;{]*?(\w+)\((?=const|WindowArgs)", text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield m.group(1), text[at:end]


@pytest.mark.parametrize("name", FILES)
def test_no_barrier_waits_for_warps_that_may_have_given_up(name):
    """A warp whose bounded wait gives up leaves its role at once.  Every barrier that counts threads (named ones and
    __syncthreads) would wait for it for ever, except before the roles begin and where all of them end."""
    text = _code(name)
    assert "named_sync" not in text and "bar.sync" not in text and "barrier.sync" not in text
    assert re.findall(r"mbarrier\.\w+", text) == [], "waits go through sm100::mbar_wait_bounded"
    assert "mbar_try_wait" not in text
    for kernel, body in _kernels(text):
        if "mbar_wait_bounded" not in body and "warp_wait" not in body:
            continue
        roles = body.index("bool fine = true;")
        assert body[:roles].count("__syncthreads()") == 1, kernel
        after = body[roles:]
        assert after.count("__syncthreads()") == 1, kernel
        assert not re.search(r"\bwarp_wait|mbar_wait_bounded|\bfor \(", after[after.index("__syncthreads()"):]), kernel


def test_the_scan_finds_the_kernels():
    names = [k for f in FILES for k, body in _kernels(_code(f)) if "warp_wait" in body]
    assert names == ["window_fwd_tc_kernel", "window_dkdv_tc_kernel", "window_dq_tc_kernel"]


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_the_last_word_of_a_bounded_wait_is_a_try(tmp_path):
    """The loop behind every bounded wait, compiled for the host against a fake clock."""
    exe = tmp_path / "bounded_wait_check"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "bounded_wait_check.cpp")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, src, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_mbarrier_waits_use_that_loop():
    text = _code("sm100.cuh")
    assert text.count("mbarrier.try_wait") == 1 and text.count("mbar_try_wait(") == 2
    body = text[text.index("bool mbar_wait_bounded"):]
    assert "return wait_bounded(" in body[:body.index("}\n\n")]


def _host_check(name, tmp_path):
    """Compiles a check that includes a kernel's source and runs its host part (no GPU call is made)."""
    exe = tmp_path / name
    native = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native")
    subprocess.run([build._nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2", "--expt-relaxed-constexpr",
                    "-I", CSRC, "-I", build.INCLUDE, os.path.join(native, name + ".cu"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


needs_nvcc = pytest.mark.skipif(shutil.which(build._nvcc()) is None, reason="nvcc not available")


def _role_ends(kernel, call):
    """In the kernel's source: after its work loop, a warp whose wait gave up makes this call."""
    for f in FILES:
        for k, body in _kernels(_code(f)):
            if k == kernel:
                return re.search(r"if \(!fine\)\s*\{?\s*" + call, body) is not None
    raise AssertionError(kernel)


@needs_nvcc
def test_forward_marks_every_row_it_could_not_make(tmp_path):
    """A CTA takes work after work; behind a wait that gave up, every row of the work at hand and of all later ones is
    NaN in o and lse (zero behind a sequence's end where the call asks for it), and nothing else is touched."""
    assert _role_ends("window_fwd_tc_kernel", r"mark_rest<D>\(")
    _host_check("window_fwd_marks_check", tmp_path)


@needs_nvcc
def test_backward_marks_every_row_it_could_not_make(tmp_path):
    """dq: as the forward.  dk and dv: a CTA's key tile, or the slot of its part of a cut one, which the join then adds
    up to NaN."""
    assert _role_ends("window_dq_tc_kernel", r"mark_queries<D>\(") and _role_ends("window_dkdv_tc_kernel", r"mark_key<D>\(")
    _host_check("window_bwd_marks_check", tmp_path)
