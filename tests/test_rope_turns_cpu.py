"""The rotation's frequency tables, compiled for the host."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_token_gb300", "csrc")


def run(tmp_path, main, *args):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "turns.cpp", tmp_path / "turns"
    src.write_text("#include <cstdio>\n#include <cstdlib>\n#include <cstring>\n#include <thread>\n#include <vector>\n"
                   "#include \"rope_turns.h\"\n" + main)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, timeout=120)


def test_threads_with_bases_of_their_own(tmp_path):
    r = run(tmp_path, r"""
int main() {
  std::vector<std::thread> t;
  std::vector<int> wrong(8, 0);
  for (int i = 0; i < 8; ++i)
    t.emplace_back([&, i] {
      for (int k = 0; k < 5000; ++k) {
        // one base more than a thread keeps, taken in turn, and one asked for again
        const double base = 10000.0 * (i + 1) + k % 5;
        const int r = 16 * (1 + (i + k % 5) % 8);
        uint64_t ref[kve::kRopePairs];
        kve::turn_fractions(base, r, ref);
        for (int again = 0; again < 2; ++again)
          if (std::memcmp(ref, kve::turn_table(base, r), r / 2 * sizeof(uint64_t)) != 0) ++wrong[i];
      }
    });
  for (auto& x : t) x.join();
  for (int w : wrong)
    if (w) return 1;
  return 0;
}
""")
    assert r.returncode == 0


@pytest.mark.parametrize("r", [16, 48, 96, 128])
@pytest.mark.parametrize("base", [1.0, 1.5, 1e4, 5e5, 1e6, 1e300, 0.5, 1e-3])
def test_tables_against_exact_arithmetic(tmp_path, base, r):
    """A frequency is off by at most 2^-61 turn a position for bases from 1, and
    1 / base times that below (the arithmetic is beside the function)."""
    mp = pytest.importorskip("mpmath")
    out = run(tmp_path, r"""
int main(int, char** v) {
  const int r = std::atoi(v[2]);
  const uint64_t* f = kve::turn_table(std::atof(v[1]), r);
  for (int i = 0; i < r / 2; ++i) std::printf("%llu\n", static_cast<unsigned long long>(f[i]));
}
""", repr(base), r)
    with mp.workdps(80):
        worst = mp.mpf(0)
        for i, line in enumerate(out.stdout.split()):
            t = mp.mpf(base) ** (mp.mpf(-2 * i) / r) / (2 * mp.pi)
            d = mp.mpf(int(line)) / mp.mpf(2) ** 64 - t
            worst = max(worst, abs(d - mp.nint(d)))
        assert worst <= mp.mpf(2) ** -61 * max(1, 1 / base)
