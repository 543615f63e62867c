"""The packed attention's host arithmetic over all sizes that its checks let through: the grid and split rules,
taken from the sources as they are, run with traps on overflow, bad shifts and divisions by zero."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "layerwise_weight_offload_slot_gb300", "csrc")

PROGRAM = """
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "dlo.h"
#define __host__
#define __device__
#define __forceinline__ inline
constexpr int kGb300Sms = 152;
constexpr int TQ = 128, TK = 128, kTile = 128;
constexpr int kStatBytes = kTile * 32;
%s
int main() {
    const int rows[] = {1, 127, 128, 129, 5000, 65535, 622592, 7000000, 1 << 23, 100000000, 1 << 29, (1 << 30) - 1, 1 << 30};
    const int heads[][2] = {{1, 1}, {2, 1}, {8, 8}, {40, 8}, {24, 1}, {77, 1}, {127, 127}, {1024, 8}, {60000, 60000}, {65535, 1}, {65535, 65535}};
    long n = 0, split = 0;
    for (int batch : {1, 2, 33, 700, 65535})
        for (auto& h : heads)
            for (int hd : {8, 64, 72, 128})
                for (int rq : rows)
                    for (int rk : rows) {
                        dlo_attn_packed a = {};
                        a.batch = batch, a.heads = h[0], a.kv_heads = h[1], a.head_dim = hd, a.rows_q = rq, a.rows_k = rk;
                        const PackedGrid p = packed_grid(a);
                        const PackedBwdSplit b = packed_bwd_split(a);
                        const long long keys = (rk + 127LL) / 128;
                        // every key tile has a part, parts fit their bound, and the launch its limits
                        if (p.parts < 1 || p.parts > 64 || p.ctas < 1 || a.heads / a.kv_heads %% p.gh) return 1;
                        if (p.parts > 1 && (p.per < 1 || (long long)p.per * p.parts < keys || (long long)TK * p.per > 1LL << 30 || p.ctas > 0x7FFFFFFF ||
                                            (double)p.parts * a.heads * rq * (hd + 1) * 4 > 512.0 * (1 << 20)))
                            return 2;
                        if (b.q < 1 || b.k < 1 || b.q > 64 || b.k > 64 || b.total < b.part_v || b.part_v < b.part_k || b.part_k < b.part_q) return 3;
                        ++n, split += p.parts > 1;
                    }
    std::printf("%%ld %%ld\\n", n, split);
}
"""


def part(name, pattern):
    with open(os.path.join(CSRC, name)) as f:
        return re.search(pattern, f.read(), re.S | re.M).group()


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_grid_and_split_rules_hold_for_all_sizes(tmp_path):
    rules = "\n".join([part("attention.cuh", r"^__host__ __device__ __forceinline__ int packed_slots\(.*?\}$"),
                       part("attention_packed.cu", r"^constexpr int kParts = .*?^PackedGrid packed_grid\(.*?^\}$"),
                       part("attention_packed_bwd.cu", r"^struct PackedBwdSplit \{.*?^PackedBwdSplit packed_bwd_split\(.*?^\}$")])
    src, exe = tmp_path / "sizes.cpp", tmp_path / "sizes"
    src.write_text(PROGRAM % rules)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.returncode
    n, split = map(int, r.stdout.split())
    assert n == 5 * 11 * 4 * 13 * 13 and split > 500
