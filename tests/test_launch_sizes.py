"""The quantiser's launches on the CPU: however many rows a call has, every launch has fewer than
2^32 threads (HIP refuses the others) and together they take each row once.  A row of at most
4096 channels is one wave's, a longer one four waves', in blocks of four waves.
``tests/launch_sizes.c`` stands in for the launch and prints what it is asked for."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB_DIR = os.path.join(ROOT, "combine_ep_layout_08_amd")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not os.path.exists(os.path.join(LIB_DIR, "libep.so")):
        pytest.skip("libep.so is not built")
    out = str(tmp_path_factory.mktemp("launch") / "launch_sizes")
    cmd = ["gcc", "-O1", "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROCM, "include"),
           os.path.join(ROOT, "tests", "launch_sizes.c"), "-o", out, "-rdynamic",
           "-L", LIB_DIR, "-l:libep.so", "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
           "-Wl,-rpath," + LIB_DIR]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    return out


def _check(program, args, rows, channels):
    res = subprocess.run([program, *map(str, args)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stderr
    lines = [list(map(int, line.split())) for line in res.stdout.splitlines()]
    status, launches = [x for x in lines if len(x) == 1], [x for x in lines if len(x) == 3]
    assert status == [[0]] and launches
    a_block = 1 if channels > 4096 else 4
    reached = 0
    for blocks, threads, first in launches:
        assert threads == 256 and blocks * threads < 2 ** 32, (blocks, threads)
        assert first == reached, (first, reached)
        reached += blocks * a_block
    # the last block may have waves without a row; no launch is without one
    assert reached - a_block < rows <= reached and launches[-1][2] < rows


@pytest.mark.parametrize("channels", [16, 4096, 4112, 32768])
@pytest.mark.parametrize("rows", [2048, 2 ** 22 - 1, 2 ** 22, 2 ** 22 + 1, 2 ** 24 - 1, 2 ** 24,
                                  2 ** 24 + 1, 2 ** 26 + 3])
def test_rows(program, rows, channels):
    _check(program, ("rows", rows, channels), rows, channels)


@pytest.mark.parametrize("channels", [4096, 4112])
@pytest.mark.parametrize("tokens,topk", [(2 ** 21 - 1, 8), (2 ** 21, 8), (2 ** 21 + 1, 8),
                                         (2 ** 24 + 1, 1), (2 ** 22 + 3, 8)])
def test_slots_of_expert_rows(program, tokens, topk, channels):
    _check(program, ("slots", tokens, topk, channels), tokens * topk, channels)
