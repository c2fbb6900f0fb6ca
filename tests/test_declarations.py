"""The operators' files declare each other's functions in one place, and the
library links against nothing that it does not hold (CPU only)."""
import os
import re
import subprocess

import routing_grouped_expert_amd as moe
from routing_grouped_expert_amd import build

SRC = os.path.join(moe.PKG, "csrc")
PROTOTYPE = re.compile(r"^(?:hipError_t|size_t|int|bool|void) (\w+)\([^;{}]*\);", re.M)


def text(f):
    return open(os.path.join(SRC, f)).read()


def test_one_declaration():
    names = set(PROTOTYPE.findall(text("operators.h")))
    assert {"launch_grouped", "launch_skinny", "skinny_rows", "compute_units", "launch_mx_dense",
            "launch_grouped_dense", "launch_rms_norm", "launch_quantize_mx"} <= names
    for f in sorted(os.listdir(SRC)):
        if f != "operators.h":
            assert not names & set(PROTOTYPE.findall(text(f))), f
        for n in names:
            if re.search(rf"^\w+ {n}\([^;{{}}]*\) {{", text(f), re.M):
                assert '#include "operators.h"' in text(f), f
    assert sum("typedef uint32_t u32x4" in text(f) for f in os.listdir(SRC)) == 1


def test_nothing_undefined(monkeypatch, tmp_path):
    moe.lib()
    out = subprocess.run(["nm", "-D", "--undefined-only", "-C", moe.LIB_PATH], check=True,
                         capture_output=True, text=True).stdout
    assert "moe::" not in out
    ran = []
    monkeypatch.setattr(build.subprocess, "check_call", lambda cmd: ran.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    build._link(["a.o"], str(tmp_path / "x.so"))
    assert "-Wl,-z,defs" in ran[0]
