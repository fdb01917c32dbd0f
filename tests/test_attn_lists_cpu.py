"""The window attention's own work list, replayed on the host from the rules that
the kernel and its launch use (gdn_attn_impl.h, gdn_attn_launch.h): every
(sequence, head, row tile, key tile) is the work of exactly one workgroup, no two
pieces share a place in the workspace, and the join looks for each piece where it
was left.  Over both types, every head size, windows up to 64 tokens and up to
1024 query heads a key/value head."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

REPLAY = r"""
#include "gdn_attn_launch.h"
#include <cstdio>
#include <map>
#include <vector>
using namespace gdn;
using namespace gdn::attn;

// `before`: workgroups that the shared list takes first (0: none; many: it fills the grid)
static bool replay(bool bf16, int D, int B, int K, int Hq, int Hkv, int prefix, bool ragged, int len0, int before)
{
    AttnArgs a{};
    const int page = 16;
    a.B = B; a.K = K; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.page_log2 = 4; a.prefix = prefix;
    a.P = (prefix + len0 + 40 * B + K + page - 1) / page;
    a.count = ragged ? reinterpret_cast<const int32_t*>(16) : nullptr;
    const Pick p = pick(a, bf16);
    const int N = 8192 / D, M = p.MO, nb = p.blocks;
    if (!countable(a, p, N)) return true;
    a.G = Hq / Hkv;
    a.listed = row_tiles_listed(a, M, nb);
    a.at = layout(a, nb, p.MS, M);
    const size_t places = (a.at.bytes - a.at.o_o) / ((size_t)M * D * 4);
    std::vector<Seq> seq;
    std::vector<int> base;
    int tiles = 0, segs = 0;
    for (int b = 0; b < B; ++b) {
        const int len = b % 5 == 4 ? 0 : prefix + len0 + 37 * (b % 3), cnt = ragged ? (b % 4 == 1 ? 0 : 1 + (K - 1) * b / B) : K;
        seq.push_back(seq_from(a, len, cnt, N, M));
        tiles += seq[b].segs * seq[b].tiles;
        segs += seq[b].segs;
    }
    const RowTiles rts = row_tiles_of(a, M);
    const OwnList l = own_list_of(rts, tiles, segs, nb);
    for (int b = 0, u = 0; b < B; ++b) {
        base.push_back(u);
        u += seq[b].segs * (seq[b].tiles + l.extra);
    }
    const int blocks = before + l.blocks < nb ? before + l.blocks : nb;
    // [b][h][row tile] -> how often each key tile was taken; the places of its pieces, in order
    std::map<std::vector<int>, std::vector<int>> taken;
    std::map<std::vector<int>, std::vector<size_t>> left;
    std::map<size_t, int> used;
    for (int own_block = 0; own_block < blocks && own_block < l.blocks; ++own_block) {
        const int part = own_block / rts.grouped, rt_block = own_block - part * rts.grouped;
        const int u1 = first_unit(l.units, l.parts, part + 1);
        std::vector<int> last;
        for (int u = first_unit(l.units, l.parts, part); u < u1; ++u) {
            int b = 0;
            while (u >= base[b] + seq[b].segs * (seq[b].tiles + l.extra)) ++b;
            const Seq& q = seq[b];
            const int span = q.tiles + l.extra, seg = (u - base[b]) / span, k = (u - base[b]) % span - l.extra;
            if (k < 0) continue;
            const int h = a.listed ? seg / q.rts : seg, rt_list = a.listed ? seg - h * q.rts : 0;
            const std::vector<int> tile{b, h, rt_list + rt_block};
            taken[tile].resize(q.tiles);
            ++taken[tile][k];
            if (tile != last) {
                const size_t slot = ((size_t)part + ((size_t)b * Hkv + h) * rts.in_list + rt_list) * rts.grouped + rt_block;
                if (slot >= places || used[slot]++) return printf("place %zu of %zu\n", slot, places), false;
                left[tile].push_back(slot);
                last = tile;
            }
        }
    }
    for (int b = 0; b < B; ++b) {
        const Seq& q = seq[b];
        if (q.tiles == 0) continue;
        for (int h = 0; h < Hkv; ++h)
            for (int rt = 0; rt < q.rts; ++rt) {
                const std::vector<int> tile{b, h, rt};
                if (taken[tile] != std::vector<int>(q.tiles, 1)) return printf("b %d h %d row tile %d\n", b, h, rt), false;
                const int rt_list = a.listed ? rt : 0, rt_block = a.listed ? 0 : rt;
                const int u = base[b] + (h * (a.listed ? q.rts : 1) + rt_list) * (q.tiles + l.extra) + l.extra;
                const int p0 = part_of(l.units, l.parts, u), n = part_of(l.units, l.parts, u + q.tiles - 1) - p0 + 1;
                const size_t slot = ((size_t)p0 + ((size_t)b * Hkv + h) * rts.in_list + rt_list) * rts.grouped + rt_block;
                if ((size_t)n != left[tile].size()) return printf("%d pieces, not %zu\n", n, left[tile].size()), false;
                for (int i = 0; i < n; ++i)
                    if (left[tile][i] != slot + (size_t)i * rts.grouped) return printf("join\n"), false;
            }
    }
    return true;
}

int main()
{
    int n = 0, wrong = 0;
    for (int bf16 = 0; bf16 < 2; ++bf16)
        for (int D : {64, 128, 256})
            for (int K : {1, 2, 5, 16, 32, 33, 48, 63, 64})
                for (int G : {1, 3, 8, 24, 100, 512, 513, 700, 1023, 1024})
                    for (int Hkv : {1, 2, 5, 64})
                        for (int B : {1, 3, 40})
                            for (int prefix : {0, 32})
                                for (int ragged = 0; ragged < 2; ++ragged)
                                    for (int len0 : {0, 300}) {
                                        if (G * Hkv > 1024 || (long long)B * K * G * Hkv > 300000) continue;
                                        for (int before : {0, 1 << 20}) {
                                            ++n;
                                            if (replay(bf16, D, B, K, G * Hkv, Hkv, prefix, ragged, len0, before)) continue;
                                            printf("bf16 %d D %d B %d K %d Hq %d Hkv %d prefix %d ragged %d len %d\n", bf16, D, B,
                                                   K, G * Hkv, Hkv, prefix, ragged, len0);
                                            if (++wrong == 10) return 1;
                                        }
                                    }
    printf("%d lists\n", n);
    return wrong != 0;
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_every_tile_is_taken_once(tmp_path):
    src, exe = tmp_path / "replay.cpp", tmp_path / "replay"
    src.write_text(REPLAY)
    r = subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-w",
                        "-I" + os.path.join(ROOT, "include"),
                        "-I" + os.path.join(ROOT, "speculative_verify_gdn_amd", "csrc"), str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    assert int(r.stdout.split()[0]) > 2000
