"""The rule of mx_launch.h, compiled for the host: the cases of mx_shapes.py take
the shapes that they are listed for, all shapes are among them, dense and for
experts, and each runs its main loop and its last partial stage."""
from __future__ import annotations

import os
import subprocess

import pytest

from mx_shapes import CASES
from quantized_gemv_gguf_amd import build

TERMS = {"mxfp4": 0, "bf16": 1, "f16": 2, "f32": 3}


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    """(shape, shapes there are, blocks of a stage) of (x, pair, places, rows, blocks, experts)."""
    exe = str(tmp_path_factory.mktemp("rule") / "mx_rule")
    cmd = [build.hipcc(), f"--offload-arch={build.ARCH}", "--cuda-host-only", "-std=c++17", "-O1", f"-I{build.INC}",
           f"-I{build.CSRC}", os.path.join(build.ROOT, "tests", "mx_rule.hip"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]

    def ask(problems):
        text = "".join(f"{TERMS[x]} {int(pair)} {m} {n} {nb} {e}\n" for x, pair, m, n, nb, e in problems)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return ask


def test_cases_take_every_shape(chosen):
    answers = chosen([(x, pair, m, n, nb, e) for x, pair, _, m, n, nb, e in CASES])
    assert len(answers) == len(CASES)
    seen, wanted = set(), set()
    for (x, pair, shape, m, n, nb, e), (got, shapes, stage) in zip(CASES, answers):
        assert got == shape, f"{x} {'pair ' if pair else ''}{m} x {n}, {nb} blocks, {e} experts: shape {got}, not {shape}"
        assert nb // stage >= 4 and nb % stage != 0, (x, pair, shape, nb, stage)
        seen.add((x, pair, shape, e > 0))
        wanted |= {(x, pair, s, experts) for s in range(shapes) for experts in (False, True)}
    assert {(x, pair) for x, pair, _, _ in wanted} == {(x, pair) for x in TERMS for pair in (False, True)}
    assert seen == wanted, f"no case: {sorted(wanted - seen)}"


def test_no_shape_for_grids_past_32_bits(chosen):
    """2^32 threads in every shape: nothing is chosen; of fewer rows it is."""
    many = [(x, pair, 1 << 30, 1 << 30, 1, 0) for x in TERMS for pair in (False, True)]
    assert all(a[0] == -1 for a in chosen(many))
    assert all(a[0] >= 0 for a in chosen([(x, pair, 1 << 12, 1 << 20, 1, 0) for x, pair, *_ in many]))
