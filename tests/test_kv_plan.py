"""The index arithmetic of the paged cache's kernels (csrc/kv_plan.h), compiled for the
host: every unit of work is done once, in the order that the parts are joined in, and no
number in the caller's arrays leads outside a buffer."""
import os
import shutil
import subprocess

import pytest

from w8a8_quantised_moe_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>
#include "kv_plan.h"
using namespace moe;
static unsigned long long state = 88172645463325252ull;
static int rnd(int n) { state ^= state << 13; state ^= state >> 7; state ^= state << 17; return (int)(state % n); }
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s (case %d)\n", __LINE__, #x, kase); return 1; } } while (0)
int main() {
    for (int kase = 0; kase < 4000; ++kase) {
        const int pages[4] = {16, 32, 64, 128}, page = pages[rnd(4)];
        const int B = 1 + rnd(9), heads = 1 + rnd(5), max_pages = 1 + rnd(40);
        const bool wild = rnd(3) == 0;  // arrays that say anything
        std::vector<int> q_start(B + 1), lengths(B), table(B * max_pages);
        int at = wild ? rnd(400) - 100 : rnd(3);
        for (int b = 0; b <= B; ++b) {
            q_start[b] = at;
            at += wild ? rnd(400) - 150 : rnd(4) ? rnd(6) : rnd(200);
        }
        const int T = wild ? rnd(300) : q_start[B] + rnd(4);
        for (int b = 0; b < B; ++b) lengths[b] = wild ? rnd(100000) - 50000 : rnd(max_pages * page + 1);
        KvBatch bt{q_start.data(), lengths.data(), table.data(), max_pages, B, T, max_pages};
        // pages of new tokens
        std::vector<std::pair<int, int>> by_sequence, by_slot;
        for (int b = 0; b < B; ++b) {
            const KvSeq s = kv_seq(bt, b, page);
            CHECK(s.q0 >= 0 && s.n >= 0 && s.q0 + s.n <= T && s.len >= 0 && s.len <= max_pages * page);
            const int n = kv_run_pages(s, page), first = kv_first_page(s, page);
            int tokens = 0;
            for (int i = 0; i < n; ++i) {
                CHECK(first + i < max_pages);
                int lo = kv_max((first + i) * page, kv_max(s.len - s.n, 0)), hi = kv_min((first + i + 1) * page, s.len);
                CHECK(hi > lo);
                CHECK(lo - (s.len - s.n) >= 0 && hi - (s.len - s.n) <= s.n);  // rows of the sequence
                tokens += hi - lo;
                by_sequence.push_back({b, first + i});
            }
            CHECK(tokens == kv_min(s.n, s.len));
        }
        const bool by_token = kv_slot_by_token(B, T, page);
        for (int slot = 0; slot < kv_slots(B, T, page); ++slot) {
            int b = 0;  // the last sequence that begins at the slot or before; any one where they are wild
            if (wild) b = rnd(B);
            else while (b + 1 < B && kv_first_slot(bt, b + 1, page, by_token) <= slot) ++b;
            const KvSeq s = kv_seq(bt, b, page);
            const int at = kv_slot_page(s, slot - kv_first_slot(bt, b, page, by_token), page, by_token);
            CHECK(at >= -1 && at < max_pages);
            if (at >= 0) by_slot.push_back({b, at});
            if (at >= 0) CHECK(at >= kv_first_page(s, page) && at < kv_first_page(s, page) + kv_run_pages(s, page));
        }
        if (!wild) CHECK(by_slot == by_sequence);
        // attention
        const int row_choice[2] = {16, 256}, tok_choice[2] = {64, 128};
        KvShape sh{1 + rnd(rnd(2) ? 20 : 3), row_choice[rnd(2)], tok_choice[rnd(2)], rnd(2) ? 0 : 1 + rnd(300), page, rnd(3) ? rnd(6) : 0};
        long long U = 0;
        std::vector<long long> before;
        for (int b = 0; b < B; ++b) {
            before.push_back(U);
            U += kv_seq_units(kv_seq(bt, b, page), sh) * heads;
        }
        if (U == 0) continue;
        for (int b = 0; b < B; ++b) {  // sums by formula and one by one
            const KvSeq s = kv_seq(bt, b, page);
            long long sum = 0;
            for (int rt = 0; rt < kv_row_tiles(s, sh); ++rt) {
                int first, count;
                kv_units(s, sh, rt, first, count);
                CHECK(first >= 0 && count >= 1);
                CHECK(kv_units_before(s, sh, rt) == sum);
                sum += count + sh.extra;
            }
            CHECK(kv_seq_units(s, sh) == sum);
        }
        const int most = 1 + rnd(400), ctas = kv_ctas(U, most, 1 + rnd(4));
        CHECK(ctas >= 1 && ctas <= most && ctas <= U);
        std::map<std::tuple<int, int, int, int>, int> done;
        std::map<std::tuple<int, int, int>, std::vector<int>> parts;
        long long last = 0, units = 0;
        for (int c = 0; c < ctas; ++c) {
            const long long u0 = kv_deal(U, ctas, c), u1 = kv_deal(U, ctas, c + 1);
            CHECK(u0 == last && u1 > u0);
            last = u1;
            int b = 0;
            while (b + 1 < B && before[b + 1] <= u0) ++b;
            while (kv_seq_units(kv_seq(bt, b, page), sh) == 0) --b;
            KvPlace p;
            p.b = b;
            p.s = kv_seq(bt, b, page);
            const long long per = kv_seq_units(p.s, sh);
            p.head = (int)((u0 - before[b]) / per);
            int found = 0;
            KvPlace q = p;
            for (int rt = 0; rt < kv_row_tiles(q.s, sh); ++rt)
                if (kv_enter_if(q, sh, rt, u0 - before[b] - p.head * per, before[b] + p.head * per)) {
                    p = q;
                    ++found;
                }
            CHECK(found == 1);
            for (;;) {
                const long long u = p.base + (p.unit - p.first);
                CHECK(u >= u0);
                if (u >= u1) break;
                CHECK(kv_owner(U, ctas, u) == c);
                CHECK(p.b < B && p.head < heads && p.rt < kv_row_tiles(p.s, sh));
                CHECK(p.unit >= 0 && (long long)p.unit * sh.tokens <= kv_max(p.s.len - 1, 0));
                ++units;
                ++done[std::make_tuple(p.b, p.head, p.rt, p.unit)];
                auto& list = parts[std::make_tuple(p.b, p.head, p.rt)];
                if (list.empty() || list.back() != c) list.push_back(c);
                CHECK(list.front() == kv_owner(U, ctas, p.base));
                if (p.unit + 1 == p.end) CHECK(c == kv_owner(U, ctas, p.base + (p.end - p.first) - 1));
                if (u1 <= p.base + (p.end - p.first) && p.unit + 1 == p.end) break;
                kv_next(p, bt, sh, heads);
            }
        }
        long long tiles = 0;
        for (int b = 0; b < B; ++b) tiles += (long long)kv_row_tiles(kv_seq(bt, b, page), sh) * heads;
        CHECK(last == U && (long long)done.size() == units && units == U - tiles * sh.extra);
        for (auto& d : done) CHECK(d.second == 1);
        for (auto& l : parts)
            for (size_t i = 0; i < l.second.size(); ++i) CHECK(l.second[i] == l.second[0] + (int)i);
        // every key that a row sees is in one of its units
        for (int b = 0; b < B; ++b) {
            const KvSeq s = kv_seq(bt, b, page);
            for (int i = 0; i < s.n; ++i)
                for (int g = 0; g < sh.group; g += kv_max(1, sh.group - 1)) {
                    const int rt = (int)(((long long)i * sh.group + g) / sh.rows), p = s.len - s.n + i;
                    if (p < 0) continue;
                    const int lo = sh.window && p >= sh.window ? p - sh.window + 1 : 0;
                    CHECK(done.count(std::make_tuple(b, 0, rt, lo / sh.tokens)));
                    CHECK(done.count(std::make_tuple(b, 0, rt, p / sh.tokens)));
                }
        }
    }
    std::printf("ok\n");
    return 0;
}
"""


def test_every_unit_is_done_once_and_no_index_leaves_its_buffer(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    (tmp_path / "plan.cc").write_text(PROGRAM)
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", build.CSRC,
                    str(tmp_path / "plan.cc"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_header_is_the_one_that_is_built():
    assert "kv_plan.h" in build.HEADERS and os.path.exists(os.path.join(build.CSRC, "kv_plan.h"))
