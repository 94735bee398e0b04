"""The order of prompt attention's work items: every item once, by falling cost, whatever the order in which indexes are asked for.

The host program below runs the kernels' own arithmetic (csrc/prompt_order.h) with 32 lanes as a loop; the reference counts
the items of a problem one by one.
"""
import os
import random
import shutil
import subprocess

import pytest
import torch

from masked_attention_tri_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "prompt_order.h"
using namespace triattn::prompt;
struct HostSeqs {
    std::vector<Seq> v;
    mutable long long passes = 0;
    int n() const { return (int)v.size(); }
    Seq at(int s) const { return v[s]; }
    int end(int s0) const { return s0 + 32 < n() ? s0 + 32 : n(); }
    template <typename F> int sum(int s0, F f) const {
        ++passes;
        int x = 0;
        for (int s = s0; s < end(s0); ++s) x += f(v[s]);
        return x;
    }
    template <typename F> int most(int s0, F f) const {
        ++passes;
        int x = -1;
        for (int s = s0; s < end(s0); ++s) x = f(v[s]) > x ? f(v[s]) : x;
        return x;
    }
    template <typename F> bool find(int s0, F f, int& place, int& s) const {
        ++passes;
        for (s = s0; s < end(s0); ++s) {
            const int c = f(v[s]);
            if (place < c) return true;
            place -= c;
        }
        return false;
    }
};
template <int PER> void run(const HostSeqs& seqs, int tq, int ng, int heads, int asks) {
    Order<PER> o;
    int bits = 0;
    while (1 << bits < tq) ++bits;
    o.begin(seqs, bits, ng, heads);
    for (int i = 0; i < asks; ++i) {
        long long at;
        if (std::scanf("%lld", &at) != 1) return;
        int s = -1, item = -1, h = -1;
        if (!o.locate(seqs, at, s, item, h)) s = item = h = -1;
        std::printf("%d %d %d %lld\n", s, item, h, seqs.passes);
    }
}
int main() {
    int per, tq, ng, heads, n, asks;
    while (std::scanf("%d %d %d %d %d %d", &per, &tq, &ng, &heads, &n, &asks) == 6) {
        HostSeqs seqs;
        for (int i = 0; i < n; ++i) {
            Seq q{};
            if (std::scanf("%d %d", &q.lq, &q.lk) != 2) return 1;
            q.shift = q.lk - q.lq;
            seqs.v.push_back(q);
        }
        if (per == 1) run<1>(seqs, tq, ng, heads, asks);
        else run<2>(seqs, tq, ng, heads, asks);
    }
}
"""


@pytest.fixture(scope="module")
def locate(tmp_path_factory):
    d = tmp_path_factory.mktemp("order")
    src, exe = d / "order.cpp", d / "order"
    src.write_text(PROGRAM)
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", build.CSRC, str(src), "-o",
                    str(exe)], check=True)

    def run(per, tq, ng, heads, seqs, asks):
        text = " ".join(str(x) for x in [per, tq, ng, heads, len(seqs), len(asks)] + [y for s in seqs for y in s] + list(asks))
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [tuple(int(x) for x in line.split()) for line in out if line]
    return run


def _items(per, tq, ng, heads, seqs):
    """{(sequence, item, head): key tiles that the item's last tile sees}."""
    all_items = {}
    for s, (lq, lk) in enumerate(seqs):
        tiles = [(b, g) for b in range(-(-lq // tq)) for g in range(ng)]
        for i in range(-(-len(tiles) // per)):
            b = tiles[i * per:(i + 1) * per][-1][0]
            keys = max(0, min((b + 1) * tq, lq) + lk - lq)
            for h in range(heads):
                all_items[s, i, h] = -(-keys // 128)
    return all_items


def _problem(r):
    tq = r.choice([1, 2, 8, 32, 64, 128])
    n = r.choice([1, 2, 5, 31, 32, 33, 70])
    lens = [r.choice([0, 1, r.randint(0, 40), r.randint(0, 600)]) * (4 if tq >= 32 else 1) for _ in range(n)]
    seqs = [(lq, r.choice([lq, lq, 0, r.randint(0, 3000), lq + r.randint(0, 20000)])) for lq in lens]
    return r.choice([1, 2]), tq, r.choice([1, 1, 2, 3, 5]), r.choice([1, 2, 3, 8]), seqs


@pytest.mark.parametrize("seed", range(12))
def test_every_item_once_by_falling_cost(locate, seed):
    r = random.Random(seed)
    for _ in range(4):
        per, tq, ng, heads, seqs = _problem(r)
        want = _items(per, tq, ng, heads, seqs)
        got = [x[:3] for x in locate(per, tq, ng, heads, seqs, range(len(want) + 5))]
        assert got[len(want):] == [(-1, -1, -1)] * 5
        assert len(set(got[:len(want)])) == len(want) and set(got[:len(want)]) == set(want)
        cost = [want[x] for x in got[:len(want)]]
        assert cost == sorted(cost, reverse=True)


@pytest.mark.parametrize("seed", range(6))
def test_any_order_of_asking(locate, seed):
    r = random.Random(100 + seed)
    per, tq, ng, heads, seqs = _problem(r)
    n = len(_items(per, tq, ng, heads, seqs))
    got = [x[:3] for x in locate(per, tq, ng, heads, seqs, range(n + 3))]
    asks = [r.randrange(n + 3) for _ in range(200)] + [n + 2, 0, n, max(0, n - 1), 0]
    assert [x[:3] for x in locate(per, tq, ng, heads, seqs, asks)] == [got[a] for a in asks]


def _chunks(seqs):
    return -(-len(seqs) // 32)


def test_a_long_prefix_beside_many_short_prompts(locate):
    """Levels without items cost nothing, and the items of a level one pass: 128k keys and 2000 prompts."""
    r = random.Random(7)
    seqs = [(r.randint(1, 64), 0) for _ in range(2000)]
    seqs = [(a, a) for a, _ in seqs]
    seqs.insert(900, (64, 131072))
    per, tq, ng, heads = 2, 32, 1, 8
    want = _items(per, tq, ng, heads, seqs)
    got = locate(per, tq, ng, heads, seqs, range(len(want)))
    assert set(x[:3] for x in got) == set(want) and got[0][0] == 900
    # begin (two passes), two levels with items, one between them; then one look an item
    assert got[-1][3] <= 8 * _chunks(seqs) + len(want)
    # a block that takes a short one alone
    one = locate(per, tq, ng, heads, seqs, [len(want) - 1])
    assert one[0][:3] == got[-1][:3] and one[0][3] <= 8 * _chunks(seqs)


def test_past_the_last_item(locate):
    seqs = [(65 * i, 65 * i) for i in range(1, 129)] * 2
    n = len(_items(2, 32, 1, 8, seqs))
    for x in locate(2, 32, 1, 8, seqs, [n, n + 1, n + 1000]):
        assert x[:3] == (-1, -1, -1) and x[3] == 2 * _chunks(seqs)


def test_many_sequences_and_levels(locate):
    """The most sequences that a call may have, and keys up to 2^30: as many passes as 256 levels take."""
    r = random.Random(9)
    seqs = [(r.choice([0, 1, 1, 2]), r.choice([1, 5, r.randint(1, 1 << 20)])) for _ in range(65535)]
    seqs[30000] = (3, (1 << 30) - 1)
    items = sum(a > 0 for a, _ in seqs)
    asks = [0, 1, 2, items // 2, items - 1, items, 5]
    got = locate(2, 128, 1, 1, seqs, asks)
    assert got[0][:2] == (30000, 0) and got[5][0] == -1
    assert got[-1][3] <= 2 * (3 * 256 + 8) * _chunks(seqs)
    seqs = [(1 << 15, 1 << 15)] + [(1, r.randint(1, 1 << 15)) for _ in range(5000)]  # items at every level
    want = _items(1, 128, 1, 1, seqs)
    got = locate(1, 128, 1, 1, seqs, range(len(want)))
    assert set(x[:3] for x in got) == set(want)
    cost = [want[x[:3]] for x in got]
    assert cost == sorted(cost, reverse=True) and got[-1][3] <= (3 * 257 + 4) * _chunks(seqs) + len(want)


@pytest.mark.parametrize("per,tq,ng", [(2, 32, 1), (1, 128, 3), (2, 1, 2)])
def test_levels_of_several_key_tiles(locate, per, tq, ng):
    """Past 32768 keys a level is several key tiles: every item once, and no item more than a level's key tiles after a cheaper one."""
    seqs = [(300, 100000), (70, 70), (129, 33000), (5, 2), (64, 99000), (1, 0)]
    want = _items(per, tq, ng, 2, seqs)
    got = [x[:3] for x in locate(per, tq, ng, 2, seqs, range(len(want)))]
    assert len(set(got)) == len(want) and set(got) == set(want)
    least, step = None, -(-(-(-100000 // 128)) // 256)
    for x in got:
        least = want[x] if least is None else min(least, want[x])
        assert want[x] < least + step


@pytest.mark.gpu
def test_values_of_a_long_prefix_beside_many_short_prompts():
    from test_prompt_attention import BF, _run
    r = random.Random(11)
    lq = [r.randint(0, 40) for _ in range(200)]
    lk = [n + r.choice([0, 0, 0, r.randint(0, 200)]) for n in lq]
    lq[123], lk[123] = 64, 40000
    _run(lq, lk, 4, 2, 64, BF)


@pytest.mark.gpu
def test_values_of_prompts_of_many_lengths():
    from test_prompt_attention import F16, _run
    r = random.Random(12)
    lq = [r.randint(1, 700) for _ in range(100)]
    _run(lq, lq, 4, 2, 128, F16)


@pytest.mark.gpu
def test_values_where_most_sequences_are_empty():
    """The grid has a block for each item that there could be: most of them none."""
    from test_prompt_attention import BF, _run
    lq = [(5 + i % 60) if i % 150 == 7 else 0 for i in range(3000)]
    lk = [n + (100 if i % 300 == 7 else 0) for i, n in enumerate(lq)]
    _run(lq, lk, 16, 8, 64, BF)


@pytest.mark.gpu
def test_values_of_more_places_without_an_item_than_a_block_passes_over():
    from test_prompt_attention import BF, _inputs, _within, reference
    import masked_attention_tri_gb300 as ta
    n = [0] * 30000 + [3] + [0] * 30000 + [40]
    q, k, v, g = _inputs([43], [43], 32, 32, 64, BF)
    cu = torch.zeros(len(n) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(n).cumsum(0)
    a = q, k, v, cu.cuda(), cu.cuda(), 40, 40
    o, lse = ta.prompt_attention(*a, return_aux=True)
    s = float(torch.tensor(0.125, dtype=torch.float32))
    R, T = reference(q, k, v, [3, 40], [3, 40], s, g, out=o)
    _within(o, *reference(q, k, v, [3, 40], [3, 40], s), "o")
    for x, name in zip(ta.prompt_attention_backward(*a, o, lse, g), ("dq", "dk", "dv")):
        _within(x, R, T, name)
    assert ta.get_status() == 0
