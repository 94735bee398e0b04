"""Prompt attention where many rows see no key: more queries than keys, so that whole tiles of rows have nothing to read.

Such tiles come after those with keys, and one that a CTA takes hands the tensor core nothing to do; the rows get O = 0,
lse = -inf and dQ = 0 all the same.  The sizes give each of 152 SMs several of them in a row after tiles with keys.
Tolerances: test_prompt_attention.py's.
"""
import pytest

from masked_attention_tri_gb300 import build
from test_prompt_attention import BF, F16, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("lq,lk,Hq,Hk,D,dtype", [
    ([4096], [1024], 32, 8, 128, BF),                       # 384 pairs of tiles without a key after 128 with some
    ([4096] * 4, [1024, 900, 129, 1], 16, 16, 64, F16),     # 768 and more, of several sequences
    ([2500, 2500, 300], [200, 0, 300], 24, 8, 96, BF),      # a sequence without keys beside one with fewer than queries
    ([1500] * 12, [1, 0, 17, 130, 300, 1, 1, 500, 0, 0, 64, 2000], 16, 4, 64, BF),
])
def test_many_tiles_without_a_key(lq, lk, Hq, Hk, D, dtype):
    _run(lq, lk, Hq, Hk, D, dtype)
