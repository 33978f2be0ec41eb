"""w4_attn_shared where its lists and its join take their other forms: batches of more sequences than a CTA has
threads, and more rows (sequences times heads) than 8 and 16 an SM."""
import pytest
import torch

from helpers import ensure_built
from test_gpu_attn_shared import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


@pytest.mark.parametrize("Hq,Hkv,D", [(28, 4, 128), (32, 8, 64), (20, 10, 128), (16, 1, 64), (40, 2, 128)])
@pytest.mark.parametrize("per", [1, 3, 9, 17, 33])
def test_rows_an_sm(w4, Hq, Hkv, D, per):
    """A little more than `per` rows an SM: each form of the join, rows of many parts and of one."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = per * sms // Hq + 2
    own = [1 + (37 * b) % 90 for b in range(B - 1)]
    Batch([(900, own), (130, [700])], Hq, Hkv, D, 64, seed=B).check(w4, rows=sorted({*range(0, B, max(1, B // 24)), B - 1}))


@pytest.mark.parametrize("Hq,Hkv,D,B", [(4, 2, 128, 257), (4, 2, 128, 700), (4, 4, 64, 513), (2, 1, 64, 1300), (16, 1, 64, 300),
                                        (16, 1, 128, 300)])
def test_more_sequences_than_threads(w4, Hq, Hkv, D, B):
    """Each thread of a CTA lists a run of sequences: groups, unused rows and sequences of no group in one run, and
    items that begin and end in any of them."""
    groups, left, i = [], B - 12, 0
    while left > 0:
        n = min(left, (1, 5, 0, 40, 2, 130)[i % 6])
        groups.append(((70, 16, 33, 200, 0, 129)[i % 6], [None if b % 7 == 3 else 1 + (b * b + i) % 61 for b in range(n)]))
        left, i = left - n, i + 1
    b = Batch(groups, Hq, Hkv, D, 16, before=5, after=7, seed=B)
    assert len(b.lens) == B
    b.check(w4, rows=sorted({*range(0, B, 5), *range(B - 8, B)}))


def test_one_prefix_before_many_sequences(w4):
    """600 sequences behind one prefix: 34 tiles of one key-value head."""
    Batch([(1500, [1 + b % 3 for b in range(600)])], 7, 1, 128, 64, seed=1).check(w4, rows=range(0, 600, 17))
