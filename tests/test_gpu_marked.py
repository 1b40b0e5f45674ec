"""Chunks and windowed decodes of contexts that are cut and joined, walked by one CTA or counted from several
planners, where every tile has left its mark (marked_cases.py): none may be lost, doubled or misplaced."""
import numpy as np
import pytest
import torch

from paged_kv_cache_87_gb300 import binding
from tests.marked_cases import Marked
from tests.test_gpu_chunk import TYPES, chunk
from tests.test_gpu_chunk_few import KINDS, many
from tests.test_gpu_window import TYPES as DECODE_TYPES, decode

pytestmark = pytest.mark.gpu


def run(call, *a, **kw):
    c = Marked(*a, **kw)
    out = call(c)
    assert binding.pkv_get_device_status() == 0
    c.check(out)


@pytest.mark.parametrize("q_type,kv_type", TYPES)
def test_items_cut_over_many_sms(q_type, kv_type):
    rng = np.random.default_rng(3)
    run(chunk, rng, [20011], [3], 4, 1, 128, 16, q_type, kv_type, None, 0)
    run(chunk, rng, [9000, 7000, 100], [70, 1, 100], 8, 2, 64, 32, q_type, kv_type, None, 0)
    run(chunk, rng, [9000, 7000], [70, 300], 4, 1, 128, 8, q_type, kv_type, 5000, 300)
    # two row tiles an item; more sequences than plan for themselves
    run(chunk, rng, [9000], [70], 16, 2, 128, 16, q_type, kv_type, None, 0)
    run(chunk, rng, [7000] + [60] * 39, [1] + [40] * 39, 4, 1, 64, 16, q_type, kv_type, None, 0)


@pytest.mark.parametrize("q_type,kv_type", DECODE_TYPES)
def test_windows_cut_into_pieces(q_type, kv_type):
    rng = np.random.default_rng(4)
    run(decode, rng, [9000, 4000], [1] * 2, 4, 1, 128, 16, q_type, kv_type, 8000, 20)
    run(decode, rng, [30011], [1], 8, 2, 64, 32, q_type, kv_type, 4097, 5)
    run(decode, rng, [30011, 12, 1000], [1] * 3, 4, 1, 128, 16, q_type, kv_type, 30011, 0)
    run(decode, rng, [1900] * 90, [1] * 90, 8, 2, 64, 16, q_type, kv_type, 1500, 3)


@pytest.mark.parametrize("q_type,kv_type,d", KINDS)
def test_few_rows_of_long_contexts(q_type, kv_type, d):
    rng = np.random.default_rng(5)
    lens, new = many(24, [20, 40, 33], [5, 1, 2])
    lens[7], new[7] = 5001, 6
    lens[9], new[9] = 2999, 3
    run(chunk, rng, lens, new, 96, 24, d, 16, q_type, kv_type, None, 0)
    run(chunk, rng, lens, new, 96, 24, d, 32, q_type, kv_type, 2000, 300)
