"""Paged-cache calls of the C ABI refuse bad arguments before they touch a
device: every case here is turned down on the host (no GPU needed)."""
import ctypes

import pytest

from lossless_bit_weight_encode_gb300 import build as libbuild
from lossless_bit_weight_encode_gb300 import w12

INVALID, SHAPE, ALIGN = 1, 2, 4
A = 1 << 20  # an aligned address that no call here gets to use


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def cache(**kw):
    f = dict(k_dev=A, v_dev=A, scales_dev=None, num_pages=4, page_stride=2 * 16 * 64, head_stride=16 * 64,
             row_stride=64, page_size=16, kv_heads=2, head_dim=64, dtype=w12.KV_BF16)
    f.update(kw)
    return w12.w12_kv_cache(**f)


def attend(**kw):
    f = dict(q=A, out=A, lse=None, q_stride=256, out_stride=256, tables=A, table_stride=8, lens=A, cu_new=A, tree=None,
             requests=2, max_blocks=8, tokens=3, heads=4, max_new=1, window=0, scale=0.1)
    f.update(kw)
    return w12.w12_kv_attend_args(**f)


def store(**kw):
    f = dict(q=A, k=A, v=A, q_out=A, q_stride=256, k_stride=128, v_stride=128, q_out_stride=256, q_norm=None,
             k_norm=None, rope=A, positions=A, slots=A, rope_rows=10, tokens=3, heads=4, rot=64, interleaved=0, eps=1e-6)
    f.update(kw)
    return w12.w12_kv_store_args(**f)


def plan(**kw):
    f = {n: A for n in ("lens", "new_lens", "owned_in", "owned_out", "tables", "ring", "ring_state_in",
                        "ring_state_out", "cu_new", "positions", "slots")}
    f.update(table_stride=8, requests=2, max_blocks=8, page_size=16, ring_size=10, tokens=3, trim=0)
    f.update(kw)
    return w12.w12_kv_plan_args(**f)


BAD_CACHES = [(dict(k_dev=None), INVALID), (dict(v_dev=None), INVALID), (dict(dtype=2), INVALID),
              (dict(scales_dev=A), INVALID), (dict(dtype=w12.KV_Q8), INVALID), (dict(head_dim=96), SHAPE),
              (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 31), SHAPE), (dict(kv_heads=0), SHAPE),
              (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(row_stride=32), SHAPE),
              (dict(head_stride=1 << 37), SHAPE), (dict(row_stride=68), ALIGN), (dict(page_stride=2052), ALIGN),
              (dict(k_dev=A + 8), ALIGN), (dict(dtype=w12.KV_Q8, scales_dev=A + 4), ALIGN),
              (dict(dtype=w12.KV_Q8, scales_dev=A, row_stride=72), ALIGN)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refused(kw, status):
    L, c, size = w12.lib(), cache(**kw), ctypes.c_size_t()
    assert L.w12_kv_store(c, store(), None) == status
    assert L.w12_kv_read(c, A, 1, A, A, None) == status
    assert L.w12_kv_attend(c, attend(), A, 1 << 30, None) == status
    assert L.w12_kv_attend_workspace_size(c, attend(), ctypes.byref(size)) == status
    assert w12.w12_last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(tables=None), INVALID), (dict(lens=None), INVALID),
    (dict(cu_new=None), INVALID), (dict(requests=0), INVALID), (dict(tokens=0), INVALID), (dict(max_blocks=0), INVALID),
    (dict(window=-1), INVALID), (dict(max_new=-1), INVALID), (dict(heads=3), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=1 << 16, tokens=1 << 15, q_stride=1 << 22, out_stride=1 << 22), SHAPE),
    (dict(max_blocks=1 << 27, table_stride=1 << 27), SHAPE), (dict(table_stride=7), SHAPE), (dict(q_stride=248), SHAPE),
    (dict(out_stride=128), SHAPE), (dict(q_stride=260), ALIGN), (dict(q=A + 8), ALIGN), (dict(out=A + 2), ALIGN),
    (dict(lse=A + 2), ALIGN), (dict(tree=A + 1), ALIGN), (dict(tables=A + 2), ALIGN)])
def test_attend_refused(kw, status):
    assert w12.lib().w12_kv_attend(cache(), attend(**kw), A, 1 << 30, None) == status


def test_attend_workspace_refused():
    L = w12.lib()
    assert L.w12_kv_attend(cache(), attend(), None, 1 << 30, None) == INVALID
    assert L.w12_kv_attend(cache(), attend(), A + 128, 1 << 30, None) == ALIGN
    assert L.w12_kv_attend(cache(), None, A, 1 << 30, None) == INVALID
    assert L.w12_kv_attend_workspace_size(cache(), attend(), None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(heads=-1), INVALID), (dict(tokens=-1), INVALID), (dict(rope=None), INVALID),
    (dict(positions=None), INVALID), (dict(rope_rows=0), INVALID), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE),
    (dict(rot=-16), SHAPE), (dict(rot=7, interleaved=1), SHAPE), (dict(k_stride=64), SHAPE), (dict(q_stride=128), SHAPE),
    (dict(k_stride=132), ALIGN), (dict(q_out_stride=257), ALIGN), (dict(q=A + 8), ALIGN), (dict(k_norm=A + 2), ALIGN),
    (dict(rope=A + 4), ALIGN), (dict(slots=A + 4), ALIGN), (dict(positions=A + 1), ALIGN)])
def test_store_refused(kw, status):
    assert w12.lib().w12_kv_store(cache(), store(**kw), None) == status


@pytest.mark.parametrize("kw,status", [(dict(requests=0), INVALID), (dict(max_blocks=0), INVALID),
                                       (dict(ring_size=0), INVALID), (dict(tokens=-1), INVALID),
                                       (dict(page_size=20), SHAPE), (dict(page_size=0), SHAPE),
                                       (dict(table_stride=7), SHAPE), (dict(requests=1 << 28), SHAPE),
                                       (dict(lens=A + 2), ALIGN),
                                       (dict(slots=A + 4), ALIGN), (dict(ring_state_in=A + 4), ALIGN)] +
                         [(dict([(n, None)]), INVALID) for n in ("lens", "new_lens", "owned_in", "owned_out", "tables",
                                                                 "ring", "ring_state_in", "ring_state_out", "cu_new",
                                                                 "positions", "slots")])
def test_plan_refused(kw, status):
    assert w12.lib().w12_kv_plan(plan(**kw), None) == status


def test_read_refused():
    L = w12.lib()
    assert L.w12_kv_read(cache(), None, 1, A, A, None) == INVALID
    assert L.w12_kv_read(cache(), A, -1, A, A, None) == INVALID
    assert L.w12_kv_read(cache(), A, 1, A, A + 8, None) == ALIGN
    assert L.w12_kv_read(cache(), A + 4, 1, A, A, None) == ALIGN


def test_attend_positions_refused():
    assert w12.lib().w12_kv_attend(cache(), attend(tree=A, window=4, positions=A + 2), A, 1 << 30, None) == ALIGN
