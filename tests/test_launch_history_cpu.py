"""Which decode kernels may start before the kernel in front of them: the
launch history's rules, compiled for the host."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_token_gb300", "csrc")

MAIN = r"""
#include <cstdio>
#include <cstdint>
#include <thread>
#include <vector>
#include "launch_history.h"
using kve::LaunchHistory;
static int bad = 0;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); ++bad; } } while (0)
static const void* S(std::uintptr_t i) { return reinterpret_cast<const void*>(i * 64); }

int main() {
  const void *a = S(1), *b = S(2), *c = S(3);
  {  // one stream: a step after a step, and after kernels that write what it reads
    LaunchHistory h;
    CHECK(h.attend_early(a));
    h.attend(0, a); CHECK(h.epilogue_early(0)); CHECK(!h.epilogue_early(1));
    h.epilogue(0, a); CHECK(h.attend_early(a)); CHECK(!h.epilogue_early(0));
    h.apply(a); CHECK(!h.attend_early(a));
    h.attend(1, a); CHECK(h.attend_early(a)); CHECK(h.epilogue_early(1));
    h.inputs(a); CHECK(!h.attend_early(a)); CHECK(!h.epilogue_early(1));
    h.other(a, true); CHECK(h.attend_early(a));       // behind an ordinary kernel, which waits
  }
  {  // a launch on another stream does not stand between the two
    LaunchHistory h;
    h.inputs(a); h.other(b, true); CHECK(!h.attend_early(a)); CHECK(h.attend_early(b));
    h.attend(0, a); CHECK(h.attend_early(a));
    h.apply(a); h.other(b, true); h.epilogue(3, b); CHECK(!h.attend_early(a));
    h.inputs(b); CHECK(!h.attend_early(a)); CHECK(!h.attend_early(b)); CHECK(h.attend_early(c));
    h.attend(2, b); CHECK(!h.attend_early(a)); CHECK(h.attend_early(b));
    h.attend(2, a); CHECK(h.attend_early(a));
  }
  {  // a launch that failed has put nothing there
    LaunchHistory h;
    h.inputs(a); h.other(a, false); CHECK(!h.attend_early(a));
    h.attend(0, a); h.other(a, false); CHECK(!h.epilogue_early(0));
  }
  {  // two handles of the legacy default stream
    LaunchHistory h;
    h.inputs(nullptr); CHECK(!h.attend_early(reinterpret_cast<const void*>(1)));
    h.attend(0, reinterpret_cast<const void*>(1)); CHECK(h.attend_early(nullptr));
  }
  {  // more held streams than it notes: never wrongly early
    LaunchHistory h;
    for (int i = 1; i <= 128; ++i) h.inputs(S(i));
    for (int i = 1; i <= 128; ++i) CHECK(!h.attend_early(S(i)));
    CHECK(h.attend_early(S(500)));
    h.inputs(S(129));
    for (int i = 1; i <= 129; ++i) { CHECK(!h.attend_early(S(i))); h.attend(0, S(i)); CHECK(!h.attend_early(S(i))); }
  }
  {  // several host threads, a stream each
    LaunchHistory h;
    std::vector<std::thread> t;
    std::vector<int> wrong(8, 0);
    for (int i = 0; i < 8; ++i)
      t.emplace_back([&, i] {
        for (int k = 0; k < 20000; ++k) {
          h.inputs(S(i + 1));
          if (h.attend_early(S(i + 1))) ++wrong[i];
          h.other(S(i + 1), true);
          if (!h.attend_early(S(i + 1))) ++wrong[i];
        }
      });
    for (auto& x : t) x.join();
    for (int w : wrong) CHECK(w == 0);
  }
  return bad != 0;
}
"""


def test_launch_history_rules(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "history.cpp", tmp_path / "history"
    src.write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_calls_that_write_a_steps_rows_hold_its_stream():
    """The calls whose outputs a decode step reads are noted as such, the
    others as ordinary: each entry point's own line."""
    src = open(os.path.join(CSRC, "abi.cu")).read()
    body = lambda f: re.search(r"kvevict_status %s\(.*?\n}" % f, src, re.S).group(0)
    for f in ("kvevict_norm_rope", "kvevict_kv4_read"):
        assert "history.inputs(stream)" in body(f) and "launched(" not in body(f)
    for f in ("kvevict_attend_prompt", "kvevict_kv4_write", "kvevict_kv4_pack", "kvevict_kv4_attend"):
        assert "launched(ctx, stream" in body(f)
