"""The backward of the sink window takes every (q block, key block) that holds a kept pair exactly once.

The host program below runs the kernel's own arithmetic (csrc/sink_window.h) for all CTAs of one sequence: the one of
each key block and, where the first key blocks are shared, those of the far q blocks.  The mask itself, pair by pair, is
the reference.
"""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from masked_attention_tri_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "sink_window.h"
using namespace triattn;
int main() {
    int S, tq, H, mq, mk, window, batch_sinks, Lq, Lk, sinks;
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d", &S, &tq, &H, &mq, &mk, &window, &batch_sinks, &Lq, &Lk, &sinks) == 10) {
        const SinkSharing s = sink_sharing(S, tq, H, mq, mk, window, batch_sinks);
        std::printf("P %d\n", s.nb);
        const int nqb = (Lq + 127) / 128;
        for (int kb = 0; kb * 128 < Lk; ++kb) {
            const bool shared = kb < s.nb;
            for (int far = -1; far < (shared ? s.chunks : 0); ++far) {
                if (far >= 0 && sink_far_first(kb, window, s.chunk, far) >= nqb) continue;
                const QBlocks r = sink_q_blocks(kb, Lq, Lk, window, sinks, s.chunk, far);
                for (int qb = r.qb0; qb < r.qb1; ++qb) {
                    const int st = sink_q_state(qb, kb, Lq, Lk, window, sinks, r.all_valid, shared, far);
                    if (st >= 0) std::printf("%d %d %d %d\n", kb, qb, far, st);
                }
            }
        }
    }
}
"""


@pytest.fixture(scope="module")
def lists(tmp_path_factory):
    d = tmp_path_factory.mktemp("lists")
    src, exe = d / "lists.cpp", d / "lists"
    src.write_text(PROGRAM)
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)

    def run(problems):
        text = "\n".join(" ".join(str(x) for x in p) for p in problems) + "\n"
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        parts = [p.splitlines() for p in out.split("P ")[1:]]
        return [(int(p[0]), [tuple(int(x) for x in line.split()) for line in p[1:]]) for p in parts]
    return run


def _check(problem, nb, listed):
    *_, window, _, Lq, Lk, sinks = problem
    q, k = np.arange(Lq)[:, None], np.arange(Lk)
    keep = (k <= q) & ((k > q - window) | (k < sinks))
    at_q, at_k = np.arange(0, Lq, 128), np.arange(0, Lk, 128)
    blocks = lambda m: np.add.reduceat(np.add.reduceat(m.astype(np.int64), at_q, 0), at_k, 1) > 0  # noqa: E731
    kept, past_sinks = blocks(keep), blocks(keep & (k >= sinks))
    lost_rows = np.add.reduceat((~keep.any(1)).astype(np.int64), at_q) > 0
    seen = {}
    for kb, qb, far, st in listed:
        assert (kb, qb) not in seen, (problem, kb, qb)
        seen[kb, qb] = st
        assert (st == 1) == kept[qb, kb], (problem, kb, qb)
        if far >= 0:  # a far CTA adds to the keys below `sinks` alone
            assert st == 1 and kb < nb and not past_sinks[qb, kb], (problem, kb, qb)
    for qb, kb in zip(*np.nonzero(kept | lost_rows[:, None])):
        assert (kb, qb) in seen, (problem, kb, qb)


def _alone(Lq, Lk, window, sinks):
    return (1, Lq, 1, Lq, Lk, window, sinks, Lq, Lk, sinks)


def test_more_queries_than_keys(lists):
    """The window of a q block starts past the last key, but inside the last key block's 128 columns."""
    problems = [_alone(2048, 100, 16, 4), _alone(4096, 200, 40, 130), _alone(2100, 100, 20, 4), _alone(2100, 129, 100, 1),
                (2, 2348, 1, 2048, 300, 16, 4, 2048, 100, 4), (2, 3400, 1, 2100, 1900, 60, -1, 1300, 60, 30)]
    for p, (nb, listed) in zip(problems, lists(problems)):
        assert nb > 0
        _check(p, nb, listed)


def test_random_problems(lists):
    rng = np.random.default_rng(1)
    problems = []
    for i in range(400):
        Lq = int(rng.integers(1200, 3000))
        Lk = Lq if i % 4 == 0 else int(rng.integers(1, 700 if i % 2 else 3000))
        window = int(2 ** rng.uniform(0, 10))
        sinks = int(rng.integers(1, 520)) if i % 3 else int(rng.integers(1, 20))
        per_sequence = i % 5 == 0
        other = int(rng.integers(0, 2000))
        total = max(2 * 256 * -(-sinks // 128), Lq + other)
        own = int(rng.integers(-1, 300)) if per_sequence else sinks
        problems.append((2, total, 1, max(Lq, other), max(Lk, other), window, -1 if per_sequence else sinks, Lq, Lk, own))
    shared = 0
    for p, (nb, listed) in zip(problems, lists(problems)):
        _check(p, nb, listed)
        shared += nb > 0
    assert shared > 200


B16, F16 = torch.bfloat16, torch.float16


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [B16, F16])
@pytest.mark.parametrize("lens,lens_k,D,window,sinks", [
    ([2048], [100], 64, 16, 4), ([4096], [200], 64, 40, 130), ([2048, 300], [2048, 100], 64, 16, 4),
    ([2100], [100], 128, 20, 4), ([2100, 1300], [1900, 60], 96, 60, 30), ([4096], [200], 128, 40, [130]),
    ([2100, 1300], [1900, 60], 32, 60, [3, 30])])
def test_gradients_with_more_queries_than_keys(lens, lens_k, D, window, sinks, dtype):
    """Against fp64, tolerances as in test_sink_window.py."""
    import math

    from test_sink_window import _check as check
    from test_sink_window import _dense, _problem, _run
    q, k, v, g = _problem(lens, lens_k, 1, D, dtype, seed=sum(lens) + D)
    s = 1 / math.sqrt(D)
    check(_run(q, k, v, g, lens, lens_k, window, sinks, s), _dense(q, k, v, g, lens, lens_k, window, sinks, s, dtype))
