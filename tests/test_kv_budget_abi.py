"""Refusals of the calls that keep a cache within a budget (no GPU needed)."""
import math

import pytest

tbw = pytest.importorskip("ternary_bit_weight_gb300")
from test_attention_abi import ALIGN, FAKE, NULL, OK, SHAPE, call  # noqa: E402

WEIGHTS = dict(x_type=0, kv_type=1, B=2, cu_q=FAKE, Tq=5, Hq=16, Hkv=8, D=128, scale=0.1, Q=FAKE, ldq=2048, lse=FAKE,
               num_pages=10, page_size=16, k=FAKE, ks=FAKE, table=FAKE, max_pages=7, lens=FAKE, known=FAKE, decay=1.0,
               weight=FAKE, err=FAKE, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x_type=2), SHAPE), (dict(kv_type=3), SHAPE), (dict(B=-1), SHAPE), (dict(B=1 << 31), SHAPE), (dict(Tq=-1), SHAPE),
    (dict(Tq=1 << 31), SHAPE), (dict(Hq=12), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=144), SHAPE), (dict(D=24), SHAPE),
    (dict(scale=-0.1), SHAPE), (dict(scale=math.nan), SHAPE), (dict(decay=-0.5), SHAPE), (dict(decay=math.inf), SHAPE),
    (dict(page_size=24), SHAPE), (dict(num_pages=-1), SHAPE), (dict(max_pages=-1), SHAPE), (dict(max_pages=1 << 28), SHAPE),
    (dict(cu_q=None), SHAPE), (dict(ldq=2040), SHAPE), (dict(Q=None), NULL), (dict(lse=None), NULL), (dict(k=None), NULL),
    (dict(ks=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(weight=None), NULL),
    (dict(Q=FAKE + 8), ALIGN), (dict(ldq=2052), ALIGN), (dict(lse=FAKE + 2), ALIGN), (dict(k=FAKE + 8), ALIGN),
    (dict(cu_q=FAKE + 2), ALIGN), (dict(known=FAKE + 1), ALIGN), (dict(weight=FAKE + 2), ALIGN), (dict(lens=FAKE + 2), ALIGN),
    (dict(table=FAKE + 2), ALIGN), (dict(ks=FAKE + 1), ALIGN), (dict(err=FAKE + 2), ALIGN),
    (dict(B=0), OK), (dict(Tq=0), OK),
    (dict(B=0, cu_q=None, Tq=0, Q=None, weight=None), OK)])
def test_weights_refusals(change, status):
    assert call("tern_attn_weights", WEIGHTS, **change) == status


KEEP = dict(B=2, Hkv=8, num_pages=10, page_size=16, weight=FAKE, table=FAKE, max_pages=7, lens=FAKE, budget=64, first=4,
            recent=16, keep=FAKE, new_lens=FAKE, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), SHAPE), (dict(B=1 << 28), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=5000), SHAPE), (dict(page_size=12), SHAPE),
    (dict(num_pages=-1), SHAPE), (dict(max_pages=-1), SHAPE), (dict(max_pages=1 << 28), SHAPE), (dict(budget=0), SHAPE),
    (dict(budget=1 << 31), SHAPE), (dict(first=-1), SHAPE), (dict(recent=-1), SHAPE), (dict(first=49), SHAPE),
    (dict(recent=61), SHAPE), (dict(first=1 << 62, recent=1 << 62), SHAPE), (dict(weight=None), NULL), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(keep=None), NULL), (dict(new_lens=None), NULL), (dict(weight=FAKE + 2), ALIGN),
    (dict(keep=FAKE + 2), ALIGN), (dict(new_lens=FAKE + 1), ALIGN), (dict(lens=FAKE + 2), ALIGN), (dict(table=FAKE + 2), ALIGN),
    (dict(B=0), OK)])
def test_keep_refusals(change, status):
    assert call("tern_kv_keep", KEEP, **change) == status


COMPACT = dict(kv_type=1, B=2, Hkv=8, D=128, num_pages=10, page_size=16, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, weight=FAKE,
               table=FAKE, max_pages=7, keep=FAKE, budget=64, to=FAKE + 64, to_pages=4, err=FAKE, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(kv_type=-1), SHAPE), (dict(B=-1), SHAPE), (dict(B=1 << 23), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=8), SHAPE),
    (dict(D=256), SHAPE), (dict(page_size=0), SHAPE), (dict(num_pages=1 << 31), SHAPE), (dict(max_pages=-1), SHAPE),
    (dict(max_pages=1 << 28), SHAPE), (dict(budget=0), SHAPE), (dict(budget=65), SHAPE), (dict(to_pages=3), SHAPE),
    (dict(to_pages=-1), SHAPE), (dict(to_pages=1 << 28), SHAPE), (dict(to=FAKE), SHAPE), (dict(k=None), NULL),
    (dict(v=None), NULL), (dict(ks=None), NULL), (dict(vs=None), NULL), (dict(table=None), NULL), (dict(keep=None), NULL),
    (dict(k=FAKE + 8), ALIGN), (dict(vs=FAKE + 2), ALIGN), (dict(weight=FAKE + 2), ALIGN), (dict(keep=FAKE + 2), ALIGN),
    (dict(to=FAKE + 2), ALIGN), (dict(err=FAKE + 2), ALIGN), (dict(B=0), OK)])
def test_compact_refusals(change, status):
    assert call("tern_kv_compact", COMPACT, **change) == status


@pytest.mark.parametrize("name,args", [("tern_attn_weights", WEIGHTS), ("tern_kv_keep", KEEP)])
@pytest.mark.parametrize("page_size", [1, 16, 1024])
def test_tables_of_more_tokens_than_a_tile_can_count(name, args, page_size):
    """A tile that begins below 2^31 tokens must not end past them: tables hold 2^30 at most."""
    limit = (1 << 30) // page_size
    assert call(name, args, page_size=page_size, max_pages=limit + 1) == SHAPE
    assert call(name, args, page_size=page_size, max_pages=(2 ** 31 - 1) // page_size) == SHAPE
    assert call(name, args, page_size=page_size, max_pages=limit, lens=None) == NULL   # (the shape itself passes)


def test_new_lengths_have_a_place_of_their_own():
    assert call("tern_kv_keep", KEEP, lens=FAKE, new_lens=FAKE) == SHAPE
