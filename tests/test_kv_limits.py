"""The paged cache at the limits of what its calls are told, on the host: the tokens that an append
stores, whatever the lengths say, and the first key that a row tile sees; and no loads by the
read-only path; and outputs in their inputs' memory."""
import os
import re
import shutil
import subprocess

import pytest

from test_kv_abi import CUDA, FAKE, INVALID, append, attend, lib  # noqa: F401 (lib: the fixture)
from w8a8_quantised_moe_gb300 import build

STORED = r"""
#include <climits>
#include <cstdio>
#include <set>
#include <utility>
#include <vector>
#include "kv_plan.h"
using namespace moe;
static unsigned long long state = 1234567890123ull;
static int rnd(int n) { state ^= state << 13; state ^= state >> 7; state ^= state << 17; return (int)(state % n); }
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s (case %d)\n", __LINE__, #x, kase); return 1; } } while (0)
int main() {
    for (int kase = 0; kase < 6000; ++kase) {
        const int pages[4] = {16, 32, 64, 128}, page = pages[rnd(4)];
        const int B = 1 + rnd(6), max_pages = rnd(5), cap = max_pages * page;
        std::vector<int> q_start(B + 1), lengths(B);
        int at = rnd(3);
        for (int b = 0; b <= B; ++b) {
            q_start[b] = at;
            at += rnd(3) ? rnd(5) : rnd(300);
        }
        const int T = q_start[B] + rnd(4);
        for (int b = 0; b < B; ++b) {
            const int n = q_start[b + 1] - q_start[b];
            const int choice[8] = {rnd(cap + 1), cap, cap + 1, cap + rnd(n + 2), cap + n, cap + n + 1 + rnd(200), INT_MAX, -rnd(50)};
            lengths[b] = choice[rnd(8)];
        }
        KvBatch bt{q_start.data(), lengths.data(), nullptr, max_pages, B, T, max_pages};
        const bool by_token = kv_slot_by_token(B, T, page);
        std::set<std::pair<int, int>> stored, want;
        int reported = 0, reports = 0;
        for (int slot = 0; slot < kv_slots(B, T, page); ++slot) {
            int b = 0;
            while (b + 1 < B && kv_first_slot(bt, b + 1, page, by_token) <= slot) ++b;
            int over;
            const KvSeq s = kv_seq_stored(bt, b, page, over);
            const int run = slot - kv_first_slot(bt, b, page, by_token);
            if (over > 0 && run == 0) ++reported;
            const int p = kv_slot_page(s, run, page, by_token);
            if (p < 0) continue;
            CHECK(p < max_pages);
            const int lo = kv_max(p * page, kv_max(s.len - s.n, 0)), hi = kv_min(p * page + page, s.len);
            CHECK(hi > lo);
            for (int pos = lo; pos < hi; ++pos) {
                const int row = s.q0 + pos - (s.len - s.n);
                CHECK(row >= q_start[b] && row < q_start[b + 1]);
                CHECK(stored.insert({row, pos}).second);
            }
        }
        for (int b = 0; b < B; ++b) {
            const long long n = q_start[b + 1] - q_start[b], L = lengths[b] < 0 ? 0 : lengths[b];
            for (int i = 0; i < n; ++i) {
                const long long pos = L - n + i;
                if (pos >= 0 && pos < cap) want.insert({q_start[b] + i, (int)pos});
            }
            reports += n > 0 && L > cap;
            int over;
            const KvSeq s = kv_seq_stored(bt, b, page, over);
            CHECK(s.q0 == q_start[b] && s.n >= 0 && over >= 0 && s.n + over == n && s.len <= cap);
            CHECK(s.n == 0 || (long long)s.len - s.n == L - n);
        }
        CHECK(stored == want);
        CHECK(reported == reports);
    }
    std::printf("ok\n");
    return 0;
}
"""

FIRST_KEY = r"""
#include <cstdio>
#include "kv_plan.h"
using namespace moe;
static unsigned long long state = 987654321987ull;
static int rnd(int n) { state ^= state << 13; state ^= state >> 7; state ^= state << 17; return (int)(state % n); }
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s (case %d)\n", __LINE__, #x, kase); return 1; } } while (0)
int main() {
    for (int kase = 0; kase < 20000; ++kase) {
        const int rows[3] = {8, 16, 256};
        const KvShape sh{1 + rnd(rnd(2) ? 40 : 3), rows[rnd(3)], 128, rnd(3) ? 1 + rnd(rnd(2) ? 20 : 400) : 0, 16, 0};
        const KvSeq s{0, 1 + rnd(rnd(2) ? 5 : 300), rnd(900)};
        for (int rt = 0; rt < kv_row_tiles(s, sh); ++rt) {
            int unit, count;
            kv_units(s, sh, rt, unit, count);
            const int got = kv_first_key(s, sh, rt);
            int first = 1 << 30;  // key that a row sees
            const int end = kv_min((rt + 1) * sh.rows, s.n * sh.group);
            for (int r = rt * sh.rows; r < end; ++r) {
                const int pos = s.len - s.n + r / sh.group;
                if (pos >= 0) first = kv_min(first, sh.window ? kv_max(pos - sh.window + 1, 0) : 0);
            }
            CHECK(first == 1 << 30 || got == first);
            CHECK(got >= 0 && (got == 0 || got / sh.tokens == unit));
        }
    }
    std::printf("ok\n");
    return 0;
}
"""


def compiled(tmp_path, text):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    (tmp_path / "program.cc").write_text(text)
    exe = str(tmp_path / "program")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", build.CSRC,
                    str(tmp_path / "program.cc"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_first_key_that_a_row_tile_sees(tmp_path):
    compiled(tmp_path, FIRST_KEY)


def test_an_append_stores_each_token_at_its_position_or_not_at_all(tmp_path):
    compiled(tmp_path, STORED)
    with open(os.path.join(build.CSRC, "kv_append.cu")) as f:
        text = f.read()
    assert "kv_seq_stored(" in text and "kv_seq(" not in text


def test_no_load_by_the_read_only_path():
    """Kernels that start before the one that writes their input has ended may not use it."""
    names = [n for n in os.listdir(build.CSRC) if re.match(r"(api_)?kv.*\.(cu|cuh|h)$", n)]
    assert {"kv_append.cu", "kv_attend.cu", "kv_attend_few.cu", "kv_dev.cuh"} <= set(names)
    for name in names:
        with open(os.path.join(build.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"__ldg\b|\.nc\b|__restrict__", text), name


def meets(out, width, rows, w, stride, T):
    """Whether bytes [out, out + 2 width T) are in one of the T rows of 2 w bytes, 2 stride apart."""
    return any(rows + 2 * i * stride < out + 2 * width * T and out < rows + 2 * (i * stride + w) for i in range(T))


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("stride", [512, 520, 4096])
def test_outputs_that_share_memory_with_their_inputs(lib, monkeypatch, T, stride):
    """4 heads of 128 channels: rows of 1024 bytes."""
    monkeypatch.setenv("MOE_INJECT", "launch_fail")  # what passes the checks ends there
    far, seen = 1 << 28, set()
    for off in [*range(-6 * 1024, 6 * 8192, 16 * 13), -1024 * T, -1024 * T - 16, -1024 * T + 16, 0, 16, -16, 1008, 1024, 1040]:
        hit = meets(FAKE + off, 512, FAKE, 512, stride, T)
        seen.add(hit)
        assert attend(lib, T=T, q=FAKE, q_stride=stride, out=FAKE + off) == (INVALID if hit else CUDA), off
        away = dict(T=T, key=far, value=far, q=2 * far, q_stride=stride, k_stride=stride, v_stride=stride)
        want = CUDA if not hit or (off == 0 and stride == 512) else INVALID
        assert append(lib, **{**away, "q": FAKE, "q_out": FAKE + off}) == want, off
        for name in ("key", "value"):  # 2 heads: rows of 512 bytes
            hit = meets(FAKE + off, 512, FAKE, 256, stride, T)
            assert append(lib, **{**away, name: FAKE, "q_out": FAKE + off}) == (INVALID if hit else CUDA), (name, off)
    assert seen == {False, True}
