"""Host code of the entry points of include/gdn_linattn.h under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): the instrumented library objects of
test_host_sanitizers, driven by tests/csrc/linattn_sanitize_main.c."""
import os
import subprocess

from gated_delta_rule_64_b200 import build as gdn_build
from tests import test_host_sanitizers as base


def test_linattn_host_code_under_sanitizers():
    base.test_library_host_code_under_sanitizers()  # (builds the objects where they are stale)
    main = os.path.join(base.HERE, "csrc", "linattn_sanitize_main.c")
    exe, mobj = os.path.join(base.OUT, "linattn_san"), os.path.join(base.OUT, "linattn_sanitize_main.o")
    if base._stale(exe, gdn_build.deps() + [main]):
        objs = [os.path.join(base.OUT, os.path.basename(src) + ".o") for src in gdn_build.sources()]
        subprocess.run(["gcc", *base.SAN, "-g", "-I", gdn_build.INCLUDE, "-c", main, "-o", mobj], check=True)
        subprocess.run([gdn_build.nvcc(), *gdn_build.ARCH, *objs, mobj, "-o", exe,
                        *[a for f in base.SAN for a in ("-Xcompiler", f)]], check=True)
    assert "0 failures" in base._run(exe, ASAN_OPTIONS="detect_leaks=0:protect_shadow_gap=0")


def test_linattn_limits_under_sanitizers():
    base.test_library_host_code_under_sanitizers()
    main = os.path.join(base.HERE, "csrc", "linattn_limits_main.c")
    exe, mobj = os.path.join(base.OUT, "linattn_limits"), os.path.join(base.OUT, "linattn_limits_main.o")
    if base._stale(exe, gdn_build.deps() + [main]):
        objs = [os.path.join(base.OUT, os.path.basename(src) + ".o") for src in gdn_build.sources()]
        subprocess.run(["gcc", *base.SAN, "-g", "-I", gdn_build.INCLUDE, "-c", main, "-o", mobj], check=True)
        subprocess.run([gdn_build.nvcc(), *gdn_build.ARCH, *objs, mobj, "-o", exe,
                        *[a for f in base.SAN for a in ("-Xcompiler", f)]], check=True)
    assert "0 failures" in base._run(exe, ASAN_OPTIONS="detect_leaks=0:protect_shadow_gap=0")
