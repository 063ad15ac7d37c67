"""Which copies of a warp's ring are under way when it gives up a wait (host code, compiled here), and what the
kernels' sources say about orders that a run need not show."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "nvfp4_block_scaled_gemv_gb300", "csrc_layer")

# A loader that is `stages` tiles ahead, as far as there are tiles, and a reader that gives up at each tile in turn:
# the fills that await_fills names must be the ones loaded and not read, with the parity of their round.
PROGRAM = r"""
#include "ring.h"
#include <cstdio>
#include <vector>
int main() {
  for (uint32_t stages = 2; stages <= 6; ++stages)
    for (uint32_t tiles = 1; tiles <= 40; ++tiles)
      for (uint32_t stop = 0; stop < tiles; ++stop) {
        uint32_t reads_left = tiles, loads_left = tiles, stage = 0, parity = 0;
        auto load = [&] { if (loads_left) --loads_left; };
        for (uint32_t i = 0; i < stages; ++i) load();
        for (uint32_t i = 0; i < stop; ++i) {
          --reads_left;
          load();
          if (++stage == stages) stage = 0, parity ^= 1u;
        }
        const uint32_t loaded = tiles < stop + stages ? tiles : stop + stages;
        std::vector<uint32_t> got;
        nvfp4::await_fills(reads_left, loads_left, stage, parity, stages, [&](uint32_t s, uint32_t p) {
          got.push_back(s * 2 + p);
          return true;
        });
        std::vector<uint32_t> want;
        for (uint32_t fill = stop; fill < loaded; ++fill) want.push_back(fill % stages * 2 + (fill / stages & 1u));
        uint32_t asked = 0;  // a wait that runs out is the last
        nvfp4::await_fills(reads_left, loads_left, stage, parity, stages, [&](uint32_t, uint32_t) { return ++asked < 2; });
        if (got != want || asked != (want.size() < 2 ? want.size() : 2)) {
          std::printf("stages %u tiles %u stop %u: %zu fills, expected %zu\n", stages, tiles, stop, got.size(), want.size());
          return 1;
        }
      }
  return 0;
}
"""


def test_fills_under_way(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    (tmp_path / "ring.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", SOURCE, "ring.cpp", "-o", "ring"], cwd=tmp_path, check=True)
    done = subprocess.run(["./ring"], cwd=tmp_path, capture_output=True, text=True)
    assert done.returncode == 0, done.stdout


def test_the_kernel_of_few_tokens_waits_for_them():
    """Where that kernel leaves a run early, it waits for its fills first and adds up no pieces of the CTA."""
    with open(os.path.join(SOURCE, "attention.cu")) as f:
        code = f.read()
    left = code[code.index("mbar_wait<false>(bar, parity, ok"):]
    left = left[left.index("if (!ok) {"):]
    assert "await_fills(" in left[: left.index("break;")]
    assert "__syncthreads_or(!ok)" in code


def kernel_sources():
    return {name: open(os.path.join(SOURCE, name)).read() for name in sorted(os.listdir(SOURCE))}


def test_arrivals_at_another_cta_name_the_cluster():
    """An arrive at a barrier of the cluster's shared memory is not at a CTA's scope, the default."""
    found = 0
    for name, code in kernel_sources().items():
        for line in re.findall(r"mbarrier\.arrive[^\"]*shared::cluster", code):
            found += 1
            assert ".cluster.shared::cluster" in line, (name, line)
    assert found >= 3


def test_the_pair_releases_what_it_wrote():
    """The warps that fill shared memory for the pair's MMAs release it to the cluster, those that have read marks too, and
    who issues the MMAs acquires it there."""
    code = kernel_sources()["attention_prompt.cu"]
    for what in ("slot_full(si)", "q_full", "p_ready(x & 1)"):
        assert f"arrive_issuer_filled<CTAS>({what}, lane == 0)" in code
    filled = code[code.index("void arrive_issuer_filled"):]
    assert "fence.release.sync_restrict::shared::cta.cluster" in filled[: filled.index("\n}\n")]
    for what in ("q_full, 0", "slot_full(i)", "s_free(x & 1)", "p_ready(x & 1)"):
        assert f"wait_phase<CTAS>({what}" in code and f"wait_phase({what}" not in code


def test_no_read_only_loads():
    """Kernels of the layer may be launched before those in front of them end; what they read may have been written by
    one of these, and does not go by the read-only path."""
    for name, code in kernel_sources().items():
        for word in ("__ldg(", "global.nc", "ld_stream_256(", "ld_shared_2x128(", "ld_scale_32("):
            assert word not in code, (name, word)
