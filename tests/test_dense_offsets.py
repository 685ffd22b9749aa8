"""Offsets of the 16-bit products' buffer loads, without a GPU: a lane whose
row or channel does not exist reads past the buffer (zeros) at every step,
also where a step adds to its offset."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_moe_expert_top_amd", "csrc")

CHECKS = """
#include "offsets.h"
using moe::kOut;
using moe::offset_sum;
// a descriptor's bytes are below 2^32 - 15 (16-byte units), so kOut is past them all
static_assert(kOut >= 0xFFFFFFF0u, "");
constexpr bool stays_out() {
  for (uint32_t add = 0; add < 4096; ++add)
    if (offset_sum(kOut, add) != kOut) return false;
  return offset_sum(kOut, 0xFFC00000u) == kOut && offset_sum(kOut, ~0u) == kOut;
}
static_assert(stays_out(), "a lane that is out came back in");
static_assert(offset_sum(0, 64) == 64 && offset_sum(128, 0) == 128 && offset_sum(0xFFC00000u, 512) == 0xFFC00200u, "");
// the rows past 2040 of 2^20 inputs (just below 4 GiB): plain products wrap from row 2048 on
constexpr uint32_t N = 2040, K = 1u << 20;
constexpr bool rows_stay_out() {
  for (uint32_t row = N; row < N + 512; ++row)
    for (uint32_t col = 0; col < 64; col += 8)
      if (moe::row_offset(row, N, K, col) != kOut) return false;
  return true;
}
static_assert(rows_stay_out() && (N + 10) * K * 2 < N * K * 2, "");
static_assert(moe::row_offset(N - 1, N, K, K - 8) == N * K * 2 - 16 && moe::row_offset(0, N, K, 8) == 16, "");
int main() { return 0; }
"""


def test_a_lane_that_is_out_stays_out(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "checks.cpp"
    src.write_text(CHECKS)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o", str(tmp_path / "checks")],
                   check=True)


def bare_sums(text):
    """Lines that add to a lane's offset (po, qo) outside offset_sum."""
    out = []
    for line in re.sub(r"//.*", "", text).splitlines():
        line = re.sub(r"offset_sum\(.*", "", line)
        if re.search(r"\b[pq]o(\[(?:[^\[\]]|\[[^\]]*\])*\])+\s*[+-]\s*[\w(]|[\w)]\s*[+-]\s*[pq]o\[", line):
            out.append(line.strip())
    return out


def test_no_bare_sum_with_a_lanes_offset():
    assert bare_sums("x = a ? qo[x] + 64 * u : kOut;") and bare_sums("at + po[twin(i)]") and bare_sums("qo[x][u]+4")
    assert not bare_sums("qo[i] = (r + 8) * 2;  // qo[x] + 64\n offset_sum(po[twin(i)], at), 0);\n dma(qr, qo[twin(i)], 0)")
    with open(os.path.join(CSRC, "gemm16.hip")) as f:
        text = f.read()
    assert bare_sums(text) == []
    assert not re.search(r"\bpo\[.*=.*\bch \* \(uint32_t\)p\.K", text)  # a channel's row: row_offset
