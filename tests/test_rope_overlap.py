"""A q_out that shares bytes with q, k or v: the host's test of two strided
sets of rows against brute force, and the entry points' refusals."""

import os
import shutil
import subprocess

import pytest

from tests.test_rope_refusals import PTR, _call

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_128_gb300", "csrc")

MODEL = r"""
#include <cstdio>
#include "token_rows.h"

static bool brute(const pagedkv::TokenRows& a, const pagedkv::TokenRows& b, int64_t n) {
  for (int64_t i = 0; i < n; ++i)
    for (int64_t j = 0; j < n; ++j) {
      const int64_t x = int64_t(a.at) + i * a.stride, y = int64_t(b.at) + j * b.stride;
      if (x < y + b.row && y < x + a.row) return true;
    }
  return false;
}

int main() {
  long cases = 0;
  for (int ra = 1; ra <= 4; ++ra)
    for (int rb = 1; rb <= 4; ++rb)
      for (int sa = ra; sa <= 9; ++sa)
        for (int sb = rb; sb <= 9; ++sb)
          for (int n = 1; n <= 5; ++n)
            for (int at = 0; at <= 120; ++at) {
              const pagedkv::TokenRows a{60, ra, sa}, b{uintptr_t(at), rb, sb};
              if (pagedkv::rows_overlap(a, b, n) != brute(a, b, n) || pagedkv::rows_overlap(b, a, n) != brute(a, b, n)) {
                std::printf("%d %d %d %d %d %d\n", ra, rb, sa, sb, n, at);
                return 1;
              }
              ++cases;
            }
  // extents past 64 bits
  const pagedkv::TokenRows big{1 << 20, 16, int64_t(1) << 60}, small{1 << 21, 16, 16};
  if (pagedkv::rows_overlap(big, small, int64_t(1) << 20) || pagedkv::rows_overlap(big, small, 0)) return 1;
  std::printf("%ld\n", cases);
  return 0;
}
"""


def test_rows_overlap(tmp_path):
    cxx = os.environ.get("CXX", "g++")
    if not shutil.which(cxx):
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "rows.cpp", tmp_path / "rows"
    src.write_text(MODEL)
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
    assert int(done.stdout) > 100000


# what is not refused would go on to a launch, on pointers that are the host's
@pytest.mark.skipif(os.path.exists("/dev/nvidiactl"), reason="host pointers")
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over", [
    dict(q=PTR + 64, q_out=PTR),                       # 4 heads of 64 bf16: rows of 512 bytes
    dict(q=PTR, q_out=PTR + 496),
    dict(q=PTR, q_out=PTR + 512, num_tokens=2),        # on the next token's row
    dict(q=PTR, q_out=PTR + 768, num_tokens=2, q_token_stride=512, q_out_token_stride=256, k=PTR + 8192, v=PTR + 8192),
    dict(q=PTR + 4096, q_out=PTR, k=PTR + 256, v=PTR + 8192),
    dict(q=PTR + 4096, q_out=PTR, k=PTR + 8192, v=PTR + 496),
    # q, k and v side by side (rows of 1024 bytes), q_out over the values
    dict(q=PTR, k=PTR + 512, v=PTR + 768, q_out=PTR + 640, q_token_stride=512, k_token_stride=512, v_token_stride=512,
         q_out_token_stride=512, num_tokens=3),
], ids=str)
def test_overlapping_outputs_are_refused(fp8, over):
    a = dict(num_tokens=1)
    a.update(over)
    assert _call(fp8, **a) == 1
