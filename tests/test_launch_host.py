"""The host side of the layer-norm and Muon calls over sizes that no test can
allocate: built with the undefined-behaviour sanitizer over a stand-in for the HIP
runtime that checks each launch against the card's limits and launches nothing.
CPU only."""

from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

import sharded_mixed_precision_zero_amd as Z

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sharded_mixed_precision_zero_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = shutil.which("hipcc") or os.path.join(ROCM, "bin", "hipcc")
CLANG = os.path.join(ROCM, "llvm", "bin", "clang++")

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                                reason="no hipcc")


@pytest.fixture(scope="module")
def call(tmp_path_factory):
    """call(line, ...) -> (workspace bytes, status, launches) of each line."""
    d = str(tmp_path_factory.mktemp("launch"))
    objs, symbols = [], []
    for name in ("zero_shard_muon", "zero_shard_norm"):
        objs.append(os.path.join(d, name + ".o"))
        subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g",
                        "-std=c++17", "-ffp-contract=off", "-Xarch_host", "-fsanitize=undefined",
                        "-I" + os.path.join(ROOT, "include"), "-c",
                        os.path.join(CSRC, name + ".hip"), "-o", objs[-1]],
                       check=True, capture_output=True, timeout=300)
        out = subprocess.run(["nm", "-u", objs[-1]], check=True, capture_output=True, text=True)
        symbols += re.findall(r"__hip_fatbin_\w+", out.stdout)  # the kernels, which are not built
    exe = os.path.join(d, "launch_host")
    subprocess.run([CLANG, "-std=c++17", "-O1", "-g", "-fsanitize=undefined",
                    "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROCM, "include"),
                    "-I" + os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "native", "launch_host.cpp"), *objs,
                    *[f"-Wl,--defsym={s}=0" for s in symbols], "-pthread", "-o", exe],
                   check=True, capture_output=True, timeout=300)

    def run(*lines):
        env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
        r = subprocess.run([exe], input="\n".join(lines) + "\n", env=env, capture_output=True,
                           text=True, timeout=60)
        assert r.returncode == 0, r.stderr[-2000:]
        assert "runtime error" not in r.stderr, r.stderr[:2000]
        out = [tuple(int(v) for v in line.rpartition(": ")[2].split())
               for line in r.stdout.splitlines()]
        assert len(out) == len(lines)
        return out

    return run


def test_ordinary_sizes(call):
    lines = [f"ortho {b} {r} {c} {t} 5" for b, r, c, t in (
        (1, 96, 128, 0), (4, 1024, 1024, 1), (1, 5120, 5120, 0), (1, 13824, 5120, 1),
        (3, 100, 3000, 2), (1, 1, 1, 0), (16, 300, 2000, 0))]
    lines += ["norm 1 5120 1", "norm 8192 5120 1", "norm 3 20480 2", "norm_grad 37 1601 0",
              "norm_grad 8192 5120 1", "norm_grad 1030 20480 0", "momentum 1000003 64 0",
              "momentum 26214400 16 1", "apply 1", "apply 70778880"]
    for line, (_, rc, launches) in zip(lines, call(*lines)):
        assert rc == Z.ZS_OK and launches >= 1, line


def test_ortho_sides_of_every_power_of_two(call):
    sides = [1 << k for k in range(21)]
    lines = [f"ortho 1 {r} {c} 0 5" for r in sides for c in sides if r * c <= 1 << 38]
    for line, (need, _, _) in zip(lines, call(*lines)):
        assert need > 0, line


def test_ortho_refuses_what_no_launch_takes(call):
    """Products of more tiles than a launch takes: no workspace and no launch; up
    to there every call is queued, whatever shape its tiles would take alone."""
    huge = ["ortho 65535 65536 65536 0 5", "ortho 65535 1048576 200 1 5", "ortho 1 1048576 1048576 0 1",
            "ortho 600 32768 32768 0 5"]
    for line, (need, rc, launches) in zip(huge, call(*huge)):
        assert (need, rc, launches) == (-1, Z.ZS_EINVAL, 0), line
    sides = [1 << k for k in range(5, 21)]
    lines = [f"ortho {b} {r} {c} 0 5" for b in (1, 1000, 65535) for r in sides for c in sides]
    for line, (need, rc, launches) in zip(lines, call(*lines)):
        assert (rc == Z.ZS_OK and need > 0 and launches > 0) or (
            rc == Z.ZS_EINVAL and need == -1 and launches == 0), line


def test_layernorm_of_any_number_of_rows_is_queued(call):
    lines = [f"{op} {rows} {cols} {t}" for op in ("norm", "norm_grad") for t in (0, 1)
             for rows in (1, 4194303, 4194304, 1 << 31, 1 << 40)
             for cols in (1, 512, 8192, 16384, 16385, 1 << 31)]
    for line, (need, rc, launches) in zip(lines, call(*lines)):
        assert need > 0 and rc == Z.ZS_OK and launches > 0, line


def test_muon_passes_of_any_length_are_queued(call):
    sizes = [1, (1 << 34) - 1, 1 << 34, (1 << 34) + 1, (1 << 35) - 1, 1 << 35, (1 << 35) + 5,
             1 << 38]
    lines = [f"momentum {n} {k} {t}" for n in sizes for k in (1, 64) for t in (0, 1)]
    lines += [f"apply {n}" for n in sizes]
    for line, (_, rc, launches) in zip(lines, call(*lines)):
        assert rc == Z.ZS_OK and launches >= 1, line
