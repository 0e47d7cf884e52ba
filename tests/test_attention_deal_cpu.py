"""How paged attention deals its work out to warps (csrc/wsm_deal.cuh), compiled for the host: every group of tokens
belongs to one warp's range, and the join looks for an item's partials where the ranges leave them."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <vector>
#include "wsm_deal.cuh"
using namespace wsm;

#define CHECK(x) do { if (!(x)) { printf("%s: line %d, %s\n", what, __LINE__, #x); exit(1); } } while (0)

static unsigned long long seed = 1;
static int upto(int n) {   // 0 .. n - 1
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return (int)((seed >> 33) % (unsigned)n);
}

// Walk all ranges as the warps do, note who has which group and which partials are written; then join as the join does.
static void walk(const char *what, const std::vector<int> &lengths, int max_tokens, int window, int hq, int workers) {
    const int batch = (int)lengths.size();
    std::vector<int> prefix(batch + 1, 0);
    for (int b = 0; b < batch; ++b) prefix[b + 1] = prefix[b] + span_of(max_tokens, window, lengths[b]).groups;
    const int total = line_of(prefix.data(), hq, batch), per = share_of(total, workers);
    std::vector<std::vector<int>> seen((size_t)batch * hq);
    for (int i = 0; i < batch * hq; ++i) seen[i].assign(prefix[i / hq + 1] - prefix[i / hq], 0);
    std::map<int, int> wrote;                              // slot -> item
    long long all = 0;
    for (int w = 0; w < workers; ++w) {
        Place a = place_of(prefix.data(), batch, hq, total, per, w);
        const Place z = place_of(prefix.data(), batch, hq, total, per, w + 1);
        const int n = groups_before(prefix.data(), hq, z, batch) - groups_before(prefix.data(), hq, a, batch);
        CHECK(n >= 0);
        all += n;
        int left = n;
        while (left > 0) {
            while (prefix[a.b + 1] == prefix[a.b]) { ++a.b; a.item = a.g = 0; CHECK(a.b < batch); }
            const int groups = prefix[a.b + 1] - prefix[a.b], here = std::min(left, groups - a.g), i = a.b * hq + a.item;
            for (int g = a.g; g < a.g + here; ++g) ++seen[i][g];
            if (here < groups) {
                CHECK(groups > kSnapGroups);
                const int slot = slot_of(w, per, line_of(prefix.data(), hq, a.b) + a.item * (groups + kItemCost));
                CHECK(slot >= 0 && slot < 2 * workers && wrote.emplace(slot, i).second);
            }
            left -= here;
            a.g = 0;
            if (++a.item == hq) { a.item = 0; ++a.b; }
        }
    }
    CHECK(all == (long long)prefix[batch] * hq);
    for (auto &item : seen) for (int n : item) CHECK(n == 1);
    for (int i = 0; i < batch * hq; ++i) {
        const int b = i / hq, n = prefix[b + 1] - prefix[b];
        if (n <= kSnapGroups) continue;
        const int at = line_of(prefix.data(), hq, b) + (i - b * hq) * (n + kItemCost);
        const Ranges r = ranges_of(at, n, per);
        if (r.first == r.last) continue;
        for (int w = r.first; w <= r.last; ++w) {
            auto it = wrote.find(w == r.first ? slot_of(w, per, at) : 2 * w);
            CHECK(it != wrote.end() && it->second == i);
            wrote.erase(it);
        }
    }
    CHECK(wrote.empty());
}

// A line of `items` items of n groups: the ranges reach its end, and ascend.
static void reach(const char *what, int items, int n, int workers) {
    std::vector<int> prefix = {0, n};
    const long long line = (long long)items * (n + kItemCost);
    CHECK(line <= 0x7fffffffll);
    const int total = line_of(prefix.data(), items, 1), per = share_of(total, workers);
    CHECK((long long)total == line && per >= 1 && (long long)per * workers >= line);
    long long before = 0;
    for (int w = 0; w <= workers; ++w) {
        const int now = groups_before(prefix.data(), items, place_of(prefix.data(), 1, items, total, per, w), 1);
        CHECK(now >= before);
        before = now;
    }
    CHECK(before == (long long)items * n);
    const int at = total - n - kItemCost;                  // the last item
    const Ranges r = ranges_of(at, n, per);
    CHECK(r.first >= 0 && r.first <= r.last && r.last < workers);
}

int main() {
    const char *what = "random";
    for (int i = 0; i < 3000; ++i) {
        std::vector<int> lengths(1 + upto(i % 3 ? 6 : 90));
        const int most = 1 + upto(i % 2 ? 300 : 6000), max_tokens = most - upto(3);
        for (int &n : lengths) n = upto(5) ? upto(most + 2) - 1 : 0;
        if (i % 7 == 0) for (int &n : lengths) n = 0;
        walk(what, lengths, max_tokens, upto(3) ? 0 : 1 + upto(most), 1 + upto(i % 5 ? 4 : 70), 1 + upto(i % 4 ? 1800 : 9));
    }
    const int sizes[] = {148 * 4, 148 * 8, 148 * 12};
    for (int workers : sizes) {
        reach("short line", 1, 1, workers);
        // the longest lines that are accepted, and some just below
        for (int n : {1, 5, 8, 9, 125, 1021, 8189, 131068})
            for (int less = 0; less < 3; ++less) reach("long line", (int)(0x7fffffffll / (n + kItemCost)) - less, n, workers);
        reach("one item", 1, 0x7fffffff - kItemCost, workers);
    }
    puts("dealt");
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    folder = tmp_path_factory.mktemp("deal")
    src, exe = folder / "deal.cpp", folder / "deal"
    src.write_text("#include <algorithm>\n" + PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all", "-x", "c++",
                    "-I", os.path.join(ROOT, "weight_streaming_megakernel_b200", "csrc"), "-o", str(exe), str(src)], check=True)
    return str(exe)


def test_every_group_is_dealt_once_and_joined(program):
    run = subprocess.run([program], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "dealt", run.stdout + run.stderr
