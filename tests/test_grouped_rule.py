"""Which kernel takes the products of rows grouped by expert, and in which clusters: the rule is host arithmetic, compiled
here by itself and held against values worked out by hand."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_gemv_dequant_gb300", "csrc")
MAIN = """
#include <cstdio>
#include <cstdlib>
#include "fp8_group_rule.cuh"
int main(int, char** v) {
    int room[9] = {0};
    for (int i = 1; i < 9; ++i) room[i] = atoi(v[i]);
    const int sms = atoi(v[9]);
    const long long M = atoll(v[10]), E = atoll(v[11]), N = atoll(v[12]), K = atoll(v[13]);
    const qg::fp8::FewPlan p = qg::fp8::few_plan(room, M, E, N, K);
    printf("%d %lld %d\\n", p.split, p.chain, (int)qg::fp8::takes_few(p, sms, M, E, N, K));
}
"""
SMS = 152
ROOM = [SMS // i for i in range(1, 9)]


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("rule")
    (d / "main.cpp").write_text(MAIN)
    # signed overflow ends the program
    r = subprocess.run(["g++", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", "-I" + CSRC,
                        "-o", str(d / "rule"), str(d / "main.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(M, E, N, K, room=ROOM):
        args = [str(n) for n in [*room, SMS, M, E, N, K]]
        r = subprocess.run([str(d / "rule"), *args], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        split, chain, few = r.stdout.split()
        return int(split), int(chain), few == "1"

    return ask


@pytest.mark.parametrize("M", [1, 8, 32 * 64, 32 * 64 + 1, 64 * 64, 64 * 64 + 1])
def test_without_room_for_any_cluster(rule, M):
    """Where the GPU holds no cluster of the kernel of few rows, the other kernel takes every call."""
    assert rule(M, 64, 4096, 4096, [0] * 8) == (0, 0, False)


def test_clusters(rule):
    # 256 tiles of 16 k blocks: one round of 152, one of 104; sharing the second costs 18 for each of two waves
    assert rule(8, 64, 4096, 2048) == (1, 32, True)
    # 162 tiles of 41: a round, then 12 tiles for 25 clusters of six, 7 blocks and the join
    assert rule(302, 9, 2200, 5200) == (6, 58, True)
    # the same where there is room for clusters of four and less
    assert rule(302, 9, 2200, 5200, ROOM[:4] + [0] * 4) == (4, 62, True)
    # one tile: the most CTAs that two blocks each allow
    assert rule(1, 1, 128, 2048) == (8, 12, True) and rule(1, 1, 128, 384) == (1, 3, True)
    # 1024 tiles of 32: six rounds and one of 112 tiles
    assert rule(48 * 32, 32, 4096, 4096)[:2] == (1, 224)


def test_kernels(rule):
    for E, N, K in ((1, 128, 128), (9, 2200, 5200), (64, 4096, 4096), (128, 1024, 4096)):
        assert rule(32 * E, E, N, K)[2] and not rule(64 * E + 1, E, N, K)[2]
    # between 32 and 64 rows per expert by the longer chain: 7 rounds of 32 for both, a fifth off is asked for
    assert not rule(48 * 32, 32, 4096, 4096)[2]
    # 81 tiles of 256 rows are two rounds of 76 pairs, 82 blocks; 58 as above
    assert rule(9 * 34, 9, 2200, 5200)[2]


def test_sizes_next_to_31_bits(rule):
    most = (1 << 31) - (1 << 14)
    for M, E, N, K in ((most, 1, 1, 1), (1, 1, most, 16), (1, 1, 1, most), (most, 1024, most // 1024, most),
                       (32 * 1024, 1024, most // 1024, most), (1, 1, most, most)):
        split, chain, _ = rule(M, E, N, K)
        assert split >= 1 and chain >= 1
