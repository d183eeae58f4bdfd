"""The packed and paged operators in the debug build (GQA_DEBUG_BOUNDS), in which every global
access whose index comes from offsets, lengths or page tables is checked before it is made:
odd shapes, splits, long caches and contradictory contents give the same results, and no check
fires."""
import math

import pytest

import test_gpu_append_offsets as t_ao
import test_gpu_packed as t_pk
import test_gpu_packed_offsets as t_po
import test_gpu_packed_ragged as t_rg
import test_gpu_paged_batches as t_pb
import test_gpu_paged_planted as t_pl
import test_gpu_paged_rows as t_pr
from test_gpu_debug_bounds import _clean, debug_lib

pytestmark = pytest.mark.gpu


def test_packed_prompts(debug_lib):
    for Hq, Hkv in ((8, 2), (6, 2), (5, 1), (64, 1)):
        for window in (0, 100):
            t_pk.test_packed_shapes([129, 0, 1, 127, 300], Hq, Hkv, window)
    t_pk.test_packed_many_sequences()
    t_pk.test_packed_hidden_values_do_not_leak(math.nan, 50, 8, 1)
    t_rg.test_ragged_prompts()
    _clean()


def test_append(debug_lib):
    for d in (64, 128, 512):
        t_pk.test_append(d, 16, True, 5, 5, [3, 0, 40], [0, 7, 16])
        t_pk.test_append(d, 128, False, 3, 1, [70, 259], [1, 0])
    t_pk.test_append_without_a_cache_and_in_place()
    t_pk.test_append_k_only()
    for what, code in (("page", -1), ("table", -8), ("lens", -1), ("pages", -4)):
        t_pk.test_append_bad_device_contents(what, code)
    t_pb.test_append_many_sequences(1025)
    _clean()


def test_append_of_many_tokens(debug_lib):
    for total in (609, 2000):
        t_ao.test_append_behind_many_sound_ones(total, 40)
    t_pb.test_append_many_sequences(3000)
    t_ao.test_sound_offsets_leave_the_status_alone(700)
    _clean()


def test_contradictory_offsets(debug_lib):
    for cu in t_po.BAD:
        t_po.test_packed_attention(cu, 16, 1)
        t_ao.test_append(cu)
    _clean()


def test_paged(debug_lib):
    for page in (16, 128):
        t_pk.test_paged_decode(6, 2, page, 70)
        t_pk.test_paged_chunks(page, 7, 1, 300)
        t_pr.test_rows(64, 2, [1, 0, 1, 1, 1], page, 70)
    t_pk.test_paged_drafts([5, 17, 2, 12], 8, 1, 33)
    t_pk.test_paged_many_sequences()
    t_pk.test_paged_bad_page([90, 1], 2 ** 31 - 1)
    t_pk.test_paged_bad_page([1, 1], -1)
    t_pk.test_paged_bounds_exceeded([100, 1])
    t_pk.test_paged_more_queries_than_keys([4, 2])
    t_pk.test_paged_hidden_values_do_not_leak(70, 40, math.inf)
    t_rg.test_ragged_chunks(16)
    _clean()


def test_paged_split(debug_lib):
    for t in (1, 3, 40, 200):
        t_pk.test_paged_long(t, 0)
    t_pl.test_a_chunk_per_sm(64, 8, [1] * 5, [513, 9000, 577, 4097, 100], 0)
    t_pl.test_tiles_and_spans(64, 8, [150, 1, 20], [9000, 3000, 12000], 0)
    t_pl.test_levels(32, [4, 1, 3, 2, 0, 4, 4, 1], 64)
    _clean()
