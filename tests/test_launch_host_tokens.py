"""The host side of the seam, embedding and AdamW calls over sizes that no test can
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
    """call(line, ...) -> (bytes, status, launches) of each line."""
    d = str(tmp_path_factory.mktemp("launch"))
    names = ("zero_shard_seam", "zero_shard_embed", "zero_shard_adamw")
    objs = [os.path.join(d, name + ".o") for name in names]
    builds = [subprocess.Popen(
        [HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17",
         "-ffp-contract=off", "-Xarch_host", "-fsanitize=undefined",
         "-I" + os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, name + ".hip"), "-o", obj])
        for name, obj in zip(names, objs)]
    assert [b.wait(timeout=300) for b in builds] == [0] * len(names)
    symbols = []
    for obj in objs:
        out = subprocess.run(["nm", "-u", obj], check=True, capture_output=True, text=True)
        symbols += re.findall(r"__hip_fatbin_\w+", out.stdout)  # the kernels, which are not built
    exe = os.path.join(d, "launch_host_tokens")
    subprocess.run([CLANG, "-std=c++17", "-O1", "-g", "-fsanitize=undefined",
                    "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROCM, "include"),
                    "-I" + os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "native", "launch_host_tokens.cpp"), *objs,
                    *[f"-Wl,--defsym={s}=0" for s in symbols], "-pthread", "-o", exe],
                   check=True, capture_output=True, timeout=300)

    def run(*lines):
        env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
        r = subprocess.run([exe], input="\n".join(lines) + "\n", env=env, capture_output=True,
                           text=True, timeout=120)
        assert r.returncode == 0, r.stderr[-2000:]
        assert "runtime error" not in r.stderr, r.stderr[:2000]
        out = [tuple(int(v) for v in line.rpartition(": ")[2].split())
               for line in r.stdout.splitlines()]
        assert len(out) == len(lines)
        return out

    return run


def test_seams_of_every_size(call):
    rows = [1, 37, 255, 256, 1023, 1024, 8192, 1 << 20, (1 << 31) + 7, 1 << 40]
    cols = [1, 7, 512, 513, 2048, 4096, 6144, 6145, 8192, 8193, 12288, 12289, 16383, 16384]
    for dtype in (Z.ZS_F32, Z.ZS_BF16):
        for gate in (Z.ZS_GATE_NONE, Z.ZS_GATE_COLUMN, Z.ZS_GATE_SIGMOID):
            lines = [f"{{}} {r} {c} {dtype} {gate}" for r in rows for c in cols]
            for what, most in (("seam", 1), ("seam_grad", 2)):
                for bytes_, rc, launches in call(*[line.format(what) for line in lines]):
                    assert rc == Z.ZS_OK and launches == most
                    assert 0 <= bytes_ <= 4 * 256 * 16384 * 4


def test_embeddings_of_every_size(call):
    """All within the stated limits run, all beyond are refused without a launch."""
    tokens = [1, 8, 9, 2048, 2049, 8192, 8193, 1 << 20, 1 << 24, (1 << 27) - 1, 1 << 27]
    vocab = [1, 1009, 32000, 1 << 17, (1 << 37) // 5120, Z.ZS_EMBEDDING_MAX_VOCAB]
    cols = [1, 8, 9, 120, 121, 127, 128, 129, 384, 385, 5120, 16384, 1 << 20]
    for dtype in (Z.ZS_F32, Z.ZS_BF16):
        cases = [(t, v, c) for t in tokens for v in vocab for c in cols]
        for what in ("embed", "embed_grad"):
            got = call(*[f"{what} {t} {v} {c} {dtype} 0" for t, v, c in cases])
            for (t, v, c), (bytes_, rc, launches) in zip(cases, got):
                fits = t * ((c + 7) // 8 * 8) < 1 << 34 and v * c <= 1 << 37
                assert rc == (Z.ZS_OK if fits else Z.ZS_EINVAL), (what, t, v, c)
                # at most the sort, log8(2^27 / 2^11) = 6 merges, the sums, the join
                assert (1 <= launches <= 9) if fits else launches == 0
                assert bytes_ >= 0 if fits else bytes_ == -1


def test_adamw_of_every_size(call):
    """Within the limits of a tensor and of all together; launches a group of 440."""
    most = Z.ZS_ADAMW_MAX_ELEMENTS
    cases = {(1, 0, 8): 0, (1, 1, 8): 1, (1, most, 8): 1, (1, most, 32): 1, (2, most, 32): None,
             (3, most, 8): 1, (4, most, 8): None, (1, most + 1, 8): None, (440, 1000, 8): 1,
             (441, 1000, 32): 2, (1 << 20, 5, 32): 2384, (1 << 20, 5, 8): 2384,
             ((1 << 20) + 1, 5, 8): None, (0, 0, 32): 0}
    got = call(*[f"adamw {c} {n} {bits}" for c, n, bits in cases])
    for case, want, (bytes_, rc, launches) in zip(cases, cases.values(), got):
        if want is None:
            assert rc == Z.ZS_EINVAL and launches == 0, case
        else:  # the norm's and its total, and the step's
            assert rc == Z.ZS_OK and launches == 2 * want + 1 and bytes_ > 0, case
