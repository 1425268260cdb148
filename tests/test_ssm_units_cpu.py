"""Units of packed sequences on the host: the index arithmetic that the state-space kernels use on offsets, compiled
from their own header. A call has room for T / unit + B units; offsets are on the device, where nothing can refuse them, so
whatever they hold, the units that are written and read lie in that room, and with ascending offsets they are all there."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <algorithm>
#include <cstdio>
#include <vector>
#include "ssm_common.cuh"
// stdin: unit T B, then B + 1 offsets, until the end; per case one line: room, then base, count and held of every sequence
int main() {
    long long unit, T, B;
    while (std::scanf("%lld %lld %lld", &unit, &T, &B) == 3) {
        std::vector<int> off(B + 1);
        for (int& v : off) std::scanf("%d", &v);
        const gdn2::Seqs s{off.data(), (int)B, (int)T};
        std::printf("%lld", s.units((int)unit));
        long long base = 0;
        for (int b = 0; b < B; ++b) {
            const int lo = std::min(std::max(off[b], 0), (int)T), hi = std::min(std::max(off[b + 1], 0), (int)T);
            const int count = gdn2::Seqs::units_of(std::max(hi - lo, 0), (int)unit);
            std::printf(" %lld %d %d", base, count, gdn2::Seqs::held(base, count, (int)s.units((int)unit)));
            base += count;
        }
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    d = tmp_path_factory.mktemp("units")
    src, exe = str(d / "units.cu"), str(d / "units")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "gated_deltanet_mixer_gdn2_gb300", "csrc"), src, "-o", exe], check=True)

    def go(cases):
        text = "\n".join(" ".join(map(str, (u, T, len(off) - 1, *off))) for u, T, off in cases)
        lines = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(lines) == len(cases)
        return [[int(v) for v in line.split()] for line in lines]

    return go


def test_ascending_offsets_have_room_for_all(run):
    rng = np.random.default_rng(0)
    cases = []
    for _ in range(300):
        T, B = int(rng.integers(1, 5000)), int(rng.integers(1, 40))
        cases.append((int(rng.choice([16, 32, 128, 1024, 5000])), T, sorted(int(v) for v in rng.integers(-3, T + 4, B + 1))))
    for room, *rest in run(cases):
        at = 0
        for base, count, held in zip(*[iter(rest)] * 3):
            assert base == at and held == count and base + count <= room
            at += count


def test_other_offsets_stay_in_their_room(run):
    T = 4096
    cases = [(128, T, [0, T] * 3), (32, T, [0, T] * 40), (128, 1 << 29, [0, 1 << 29] * 400), (128, T, list(range(T, -1, -64))),
             (32, T, [100, 50, T, 0, 2 ** 31 - 1, -(2 ** 31), 77]), (T, T, [0, T, 0, T, T])]
    rng = np.random.default_rng(1)
    cases += [(int(rng.choice([32, 128, 1024])), T, [int(v) for v in rng.integers(-10, 2 * T, 12)]) for _ in range(200)]
    beyond = 0
    for room, *rest in run(cases):
        for base, count, held in zip(*[iter(rest)] * 3):
            assert 0 <= held <= count and (held == 0 or base + held <= room)
            assert held == count or base + held >= room  # nothing that there is room for is left out
            beyond += base + count > room
    assert beyond > 500  # units that an unbounded index would have put outside
