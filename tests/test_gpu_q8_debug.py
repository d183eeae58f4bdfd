"""The 8-bit paged cache in the debug build (GQA_DEBUG_BOUNDS), in which every global access whose
index comes from offsets, lengths or page tables is checked before it is made: odd shapes, splits,
blocks of rows and contradictory contents give the same results, and no check fires."""
import pytest

import test_gpu_q8 as t_q8
import test_gpu_q8_corners as t_co
import test_gpu_q8_planted as t_pl
import test_gpu_q8_short as t_sh
from test_gpu_debug_bounds import _clean, debug_lib

pytestmark = pytest.mark.gpu


def test_append_and_read(debug_lib):
    for d in (64, 128, 512):
        t_q8.test_append(d, 16, True, 5, 5, [3, 0, 40], [0, 7, 16])
        t_q8.test_append(d, 128, False, 4, 3, [609, 1, 700], [3, 0, 33])
        t_q8.test_read(d, 3, 32, [3, 0, 40, 200], [3, 5, 90, 333])
    for what, code in (("page", -1), ("table", -8), ("lens", -1), ("pages", -4)):
        t_q8.test_append_bad_device_contents(what, code, 650)
    for what, code in (("page", -1), ("lens", -1), ("pages", -4), ("cu", -1)):
        t_q8.test_read_bad_device_contents(what, code)
    t_co.test_append_in_place(40)
    _clean()


def test_attention(debug_lib):
    for page in (16, 128):
        t_q8.test_decode(6, 2, page, 70)
        t_q8.test_decode(64, 1, page, 0)
        t_q8.test_chunks(page, 7, 1, 128)
    t_q8.test_drafts([5, 17, 2, 12], 6, 2, 33)
    for t in (1, 2, 6, 40):
        t_q8.test_long(t, 2048, 16)
    t_q8.test_many_sequences()
    t_q8.test_many_ragged_drafts(8)
    for t in ([1, 1], [4, 2], [100, 1]):
        t_q8.test_bounds_exceeded(t)
        t_q8.test_more_keys_than_pages(t)
        t_q8.test_bad_page(t, 2 ** 31 - 1)
    _clean()


def test_short_and_blocks(debug_lib):
    t_sh.test_decode(3, 1, 16, 70)
    t_sh.test_drafts(2, 1, 4, 33)
    for what, code in (("page", -1), ("lens", -1), ("bound", -4)):
        t_sh.test_bad_device_contents(what, code)
    for Hq, Hkv, most in ((40, 1, 1), (24, 1, 2), (12, 1, 1), (7, 1, 13)):
        t_co.test_rows_in_blocks(Hq, Hkv, most, 900, 130)
    for cu in t_co.FEW:
        t_co.test_attention_with_contradictory_offsets(cu, 6, 64, 64, 64)
        t_co.test_attention_with_contradictory_offsets(cu, 6, 2, 2, 600)
    for cu in t_co.BAD:
        t_co.test_attention_with_contradictory_offsets(cu, 10, 4, 1, 600)
        t_co.test_attention_with_contradictory_offsets(cu, 10, 16, 1, 64)
        t_co.test_read_and_append_with_contradictory_offsets(cu)
    _clean()


def test_planted(debug_lib):
    t_pl.test_one_long_sequence_among_short_ones(8, 21)
    t_pl.test_a_chunk_per_sm(64, 8, [1] * 5, [513, 9000, 577, 4097, 100], 2048)
    t_pl.test_tiles_and_spans(64, 8, [4, 2, 3, 4, 0, 1, 4, 3], [2000 + 700 * i for i in range(8)], 0)
    _clean()
