"""How a paged attention call is divided (csrc/attention_plan.h), compiled with the host's C++ compiler: no GPU."""
import os
import shutil
import subprocess

import pytest

import gemm_int8_act_amd as pq2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "attention_plan.h"
#include <cstdio>
int main() {
    long long s, n, h, kv, d, len;
    while (std::scanf("%lld %lld %lld %lld %lld %lld", &s, &n, &h, &kv, &d, &len) == 6) {
        const pq2::PagedPlan p = pq2::paged_plan(s, n, h, kv, d, len);
        std::printf("%lld %lld %lld %lld %lld %lld %d\n", (long long)p.splits, (long long)p.row_tiles, (long long)p.partial_floats,
                    (long long)p.counter_words, (long long)pq2::paged_places(p, s, kv), (long long)pq2::paged_workgroups(p, s, kv),
                    pq2::kPagedThreads);
    }
}
"""


def compiled(tmp_path, source):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(source)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "gemm_int8_act_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    return str(exe)


def sizes():
    """Sizes that the entry point accepts, up to its largest: 2^23 tiles of 16 query rows."""
    out = []
    for seqs in (1, 2, 3, 5, 9, 63, 64, 65, 1000, 65535):
        for kv in (1, 2, 3, 5, 7, 8, 9, 128, 1024):
            for group in (1, 5, 16, 64, 1024):
                if kv * group > 1024:
                    continue
                tiles = (1 << 23) // (seqs * kv)
                news = {1, 2, 17, 1 << 20, max(1, tiles * 16 // group), max(1, tiles // 2 * 16 // group), max(1, (tiles * 8 // 15) * 16 // group)}
                for new in news:
                    for d in (64, 256):
                        for length in (1, 256, 257, 2048, 100000, (1 << 31) - 1):
                            out.append((seqs, new, kv * group, kv, d, length))
    return out


def test_launches_fit(tmp_path):
    """Every accepted size divides into fewer than 2^32 threads, a workgroup for each tile of each part, and no padding
    where there are fewer places than XCDs; the library's workspace is the plan's."""
    exe = compiled(tmp_path, PROGRAM)
    cases, accepted = sizes(), []
    pq2.pq2_attention_paged_workspace.cache_clear()
    for c in cases:
        try:
            accepted.append((c, pq2.pq2_attention_paged_workspace(*c)))
        except ValueError:
            pass
    pq2.pq2_attention_paged_workspace.cache_clear()
    assert len(accepted) > 1000
    assert ((1, 1 << 20, 64, 1, 256, 2048), (0, 0)) in accepted
    out = subprocess.run([exe], input="".join(" ".join(map(str, c)) + "\n" for c, _ in accepted), capture_output=True, text=True, check=True).stdout
    largest = 0
    for (case, work), line in zip(accepted, out.splitlines()):
        splits, row_tiles, floats, words, places, workgroups, threads = map(int, line.split())
        seqs, _, _, kv, _, _ = case
        assert (floats, words) == work, case
        assert places == kv * splits * min(seqs, 64), case
        assert workgroups == places * row_tiles if places < 8 else places * row_tiles <= workgroups < (places + 8) * row_tiles, case
        assert workgroups * threads < 1 << 32, (case, workgroups)
        largest = max(largest, workgroups)
    assert largest > 1 << 23           # (the padding is among the cases)
    assert len(out.splitlines()) == len(accepted)


PARTS = r"""
#include "attention_plan.h"
#include <cstdio>
int main() {
    long long most, chunk, about;
    while (std::scanf("%lld %lld %lld", &most, &chunk, &about) == 3)
        std::printf("%d\n", pq2::parts_of((int)most, (int)chunk, (int)about));
}
"""


def test_parts_of_the_longest_tables(tmp_path):
    """Parts from a quotient that is off by one at most, up to the 2^30 keys that a table may hold in one part."""
    exe = compiled(tmp_path, PARTS)
    cases = []
    for splits in (1, 2, 8, 128):
        for most in (0, 1, 2, 127, 128, 129, 255, 256, 257, 5000, (1 << 23) + 1, (1 << 30) - 129, (1 << 30) - 1, 1 << 30):
            for least in (256, 2048):
                chunk = max(least, ((most + splits - 1) // splits + 127) & ~127)
                exact = max(most - 1, 0) // chunk
                cases += [(most, chunk, about, exact + 1) for about in (exact - 1, exact, exact + 1) if about >= 0]
    out = subprocess.run([exe], input="".join(f"{m} {c} {a}\n" for m, c, a, _ in cases), capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == [want for *_, want in cases]
