"""How the log probabilities' tiles are shared out and where their parts lie: the header's own code, walked through on the host
without a GPU; and the workspace that the parts take, against the documented bound."""
import os
import shutil
import subprocess

import pytest

import gated_delta_rule_12_gb300 as gdn
import torch
from gated_delta_rule_12_gb300 import build as gbuild

# Every tile has to be taken once, a run's tiles to follow one another with rising words and to be alone with their part, parts of
# a row to rise with the words, has() to say what at() has handed out, and parts to lie apart within total().
WALK = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "part_order.h"
using gdn::PartOrder;

static const char *walk(int N, int nt)
{
    const int mt = (N + 255) / 256, tiles = mt * nt, pairs = tiles < 76 ? tiles : 76;
    const PartOrder o = PartOrder::make(mt, nt, pairs);
    std::vector<int> owner((size_t)tiles, -1);                    // a tile's part
    std::vector<std::vector<int>> taken((size_t)mt);              // of each part of a row tile: its tiles
    for (int m = 0; m < mt; ++m) {
        if (o.of(m).parts > nt + 1) return "more parts than tiles and one";
        taken[m].resize(o.of(m).parts);
    }
    for (int pair = 0; pair < pairs; ++pair) {
        int was_m = -1, was_part = -1, was_n = -1;
        for (int round = 0; round < o.rounds(); ++round) {
            int m, n, part;
            if (!o.at(pair, round, m, n, part)) { was_m = -1; continue; }
            if (m < 0 || m >= mt || n < 0 || n >= nt) return "no such tile";
            if (part < 0 || part >= o.of(m).parts) return "no such part";
            int &own = owner[(size_t)m * nt + n];
            if (own >= 0) return "a tile twice";
            own = part;
            const bool follows = m == was_m && part == was_part;
            if (follows && n <= was_n) return "words do not rise in a run";
            if (!follows && taken[m][part]) return "two runs with one part";
            ++taken[m][part];
            was_m = m; was_part = part; was_n = n;
        }
    }
    for (int m = 0; m < mt; ++m) {
        for (int n = 0; n < nt; ++n) {
            if (owner[(size_t)m * nt + n] < 0) return "a tile that nobody takes";
            if (n && owner[(size_t)m * nt + n] < owner[(size_t)m * nt + n - 1]) return "parts do not rise with the words";
        }
        for (int part = 0; part < o.of(m).parts; ++part)
            if (o.has(m, part) != (taken[m][part] > 0)) return "has() and at() differ";
    }
    // the rows at the groups' ends and beside them
    std::vector<bool> used((size_t)o.total(N), false);
    for (int row = 0; row < N; ++row) {
        const int parts = o.of(row / 256).parts;
        for (int part = 0; part < parts; ++part) {
            const int64_t at = o.first(row) + part * o.step(row, N);
            if (at < 0 || at >= o.total(N)) return "a part outside";
            if (used[at]) return "two parts in one place";
            used[at] = true;
        }
    }
    for (bool u : used) if (!u) return "room that no part has";
    return nullptr;
}

int main()
{
    int count = 0;
    const int rows[] = {1, 255, 256, 257, 700, 2100, 8191, 8192, 8193, 8448, 8449, 9000, 15617, 16384, 16385, 20000, 24833, 33000};
    const int words[] = {1, 2, 3, 5, 9, 17, 18, 19, 20, 38, 57, 64, 76, 77, 100, 118, 128, 129, 152, 153, 256, 300};
    for (int N : rows)
        for (int nt : words) {
            if ((int64_t)N * nt > 4000000) continue;
            if (const char *e = walk(N, nt)) { std::printf("%d rows, %d tiles of words: %s\n", N, nt, e); return 1; }
            ++count;
        }
    // few words: groups of up to 608 row tiles
    const int more[][2] = {{155648, 1}, {155649, 1}, {156000, 1}, {77824, 2}, {77825, 2}, {80000, 2}, {51968, 3}, {52225, 3}, {257, 609}, {8193, 609}};
    for (auto &s : more) {
        if (const char *e = walk(s[0], s[1])) { std::printf("%d rows, %d tiles of words: %s\n", s[0], s[1], e); return 1; }
        ++count;
    }
    std::srand(1);
    for (int i = 0; i < 600; ++i) {
        const int nt = 1 + std::rand() % (1 << (1 + std::rand() % 9)), most = 3000000 / nt, N = 1 + std::rand() % (most < 60000 ? most : 60000);
        if (const char *e = walk(N, nt)) { std::printf("%d rows, %d tiles of words: %s\n", N, nt, e); return 1; }
        ++count;
    }
    // every number of row tiles that a group may have
    for (int nt = 1; nt <= 1500; ++nt) {
        const int size = PartOrder::make(1 << 20, nt, 76).size;
        for (int rows = 1; rows <= size; ++rows)
            if (PartOrder::group(rows, nt, 76).parts > nt + 1) { std::printf("%d row tiles, %d tiles of words: many parts\n", rows, nt); return 1; }
    }
    std::printf("%d shapes\n", count);
    return 0;
}
"""


def test_every_tile_and_every_part_once(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(WALK)
    subprocess.run([cc, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", os.path.join(gbuild.PKG, "csrc"), "-o", str(exe), str(src)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


def documented(N, V, k, tc):
    """The header's bound, and what 256-byte boundaries add."""
    words = 256 if tc else 128
    return N * (V / words + 2) * (16 + 8 * k) + 8 * N + 2048


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.bfloat16, 61), (torch.float32, 64)])
@pytest.mark.parametrize("k", [0, 1, 8, 20])
def test_workspace_within_the_documented_bound(k, dtype, D):
    gbuild.build()
    for N in (1, 255, 256, 8192, 8193, 8448, 8449, 16384, 16385, 65537, 1 << 20):
        for V in (20, 256, 257, 700, 4608, 4609, 32768, 50257, 65536, 151936, 155905, 262144):
            size = gdn.linear_log_probs_workspace_size(N, D, V, k, dtype)
            assert 0 < size <= documented(N, V, k, dtype is torch.bfloat16 and D % 8 == 0), (N, V)


@pytest.mark.parametrize("V", [6000, 32768, 65536, 151936, 262144])
@pytest.mark.parametrize("N", [8192, 16384, 65536])
def test_one_token_more_takes_one_token_more(N, V):
    """A last group of one row tile has its own parts and leaves those of the other rows as they are."""
    gbuild.build()
    for k in (0, 20):
        a, b = (gdn.linear_log_probs_workspace_size(n, 64, V, k) for n in (N, N + 1))
        assert a <= b <= a + documented(1, V, k, True)
