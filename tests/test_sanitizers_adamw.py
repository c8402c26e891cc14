"""The AdamW step's host side (table validation, work list, defaults) built with
the compiler's sanitizers and driven on the CPU over random tables:
AddressSanitizer + UndefinedBehaviorSanitizer, and ThreadSanitizer from eight
threads. No HIP code is built here."""
import os

import pytest

from test_sanitizers import ASAN, ASAN_ENV, CSRC, SAN, _build, _run

SOURCES = [os.path.join(SAN, "adamw_stress.cpp"), os.path.join(CSRC, "adamw.cpp")]


def test_adamw_tables_under_asan_ubsan(tmp_path):
    r = _run(_build(tmp_path, "adamw_asan", ASAN, extra_sources=SOURCES), ["300", "2"], ASAN_ENV)
    assert r.returncode == 0 and "adamw stress ok" in r.stdout, r.stdout + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-4000:]


def test_adamw_tables_under_tsan_from_eight_threads(tmp_path):
    exe = _build(tmp_path, "adamw_tsan", ["-fsanitize=thread"], extra_sources=SOURCES)
    r = _run(exe, ["30", "8"], {"TSAN_OPTIONS": "halt_on_error=1"})
    if r.returncode != 0 and "FATAL: ThreadSanitizer: unexpected memory mapping" in r.stderr:
        pytest.skip("ThreadSanitizer cannot run in this process environment (memory layout)")
    assert r.returncode == 0 and "adamw stress ok" in r.stdout, r.stdout + r.stderr[-4000:]
    assert "WARNING: ThreadSanitizer" not in r.stderr, r.stderr[-4000:]
