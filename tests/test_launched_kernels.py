"""Every kernel of the experts' products that the library holds is one that some call launches:
calls over the sizes that the tiles are chosen by, on the CPU, with
``tests/launched_kernels.c`` in place of the launch."""
import itertools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB_DIR = os.path.join(ROOT, "combine_ep_layout_08_amd")
LIB = os.path.join(LIB_DIR, "libep.so")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
FAMILIES = ("::expert_kernel<", "::grad_weight_kernel<", "::row_sums_kernel(")


def _held():
    """Kernels of the library: name by place.  (Their handles are data; the host functions that
    launch them are in the text.)"""
    nm = shutil.which("nm")
    if nm is None or not os.path.exists(LIB):
        pytest.skip("libep.so is not built, or there is no nm")
    out = subprocess.run([nm, "-C", LIB], capture_output=True, text=True, check=True).stdout
    held = {}
    for line in out.splitlines():
        place, kind, name = line.split(maxsplit=2) if line[:1] != " " else ("", "", "")
        if kind.lower() in "drb" and any(f in name for f in FAMILIES) and "stub" not in name:
            held[int(place, 16)] = name.split("::", 2)[2].rsplit("(", 1)[0]
    return held


def _calls():
    tokens = [1, 3, 12, 40, 47, 60, 100, 130, 400, 512, 1400, 4096]
    for t, topk, e, own in itertools.product(tokens, (1, 8), (1, 8, 64), (0, 1)):
        for k, n in ((128, 16), (1024, 1024), (7168, 4096), (4096, 6016), (2048, 7168)):
            for gated in (0, 1):
                yield 0, t, topk, e, own, k, n, gated, 0
        for k, n in ((128, 24), (1024, 504), (7168, 2048), (2048, 6016), (6016, 2048), (512, 16384)):
            yield 1, t, topk, e, own, k, n, 0, t % 2


def test_every_kernel_is_launched_by_some_call(tmp_path):
    held = _held()
    assert len(held) > 40
    exe = str(tmp_path / "launched_kernels")
    res = subprocess.run(
        ["gcc", "-O1", "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROCM, "include"),
         os.path.join(ROOT, "tests", "launched_kernels.c"), "-o", exe, "-rdynamic",
         "-L", LIB_DIR, "-l:libep.so", "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-ldl",
         "-Wl,-rpath," + LIB_DIR], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    calls = list(_calls())
    text = "\n".join(" ".join(map(str, c)) for c in calls) + "\n"
    res = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr
    lines = [line.split() for line in res.stdout.splitlines()]
    assert len(lines) == len(calls)
    seen = set()
    for call, line in zip(calls, lines):
        assert line[-1] == "0" and len(line) > 1, (call, line)
        seen |= {int(p, 16) for p in line[:-1]}
    assert seen <= set(held), "a kernel that the symbols do not name"
    left = sorted(held[p] for p in set(held) - seen)
    assert not left, "\n".join(["no call launches:"] + left)
