"""Refusals of the target's side of a step: host-side validation returns before anything is
launched, so these run without a GPU."""
import ctypes

import pytest

import speculative_decoding_03_gb300 as ds
from speculative_decoding_03_gb300.target import _CacheStruct

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000000          # an aligned address that is never dereferenced by these calls
F32, BF16, F16 = 0, 1, 2
NAN, INF = float("nan"), float("inf")


def cache(k=FAKE, v=FAKE, dtype=BF16, layers=2, pages=10, page=16, heads=4, D=128, layer_s=81920, page_s=8192,
          slot_s=512, head_s=128):
    return _CacheStruct(k, v, dtype, layers, pages, page, heads, D, layer_s, page_s, slot_s, head_s)


def append(c=None, layer=0, starts=None, counts=FAKE, parents=None, B=2, N=4, rows=8, pages=FAKE, most=5, lengths=FAKE,
           k=FAKE, k_row=512, k_head=128, v=FAKE, v_row=512, v_head=128, q=FAKE, q_row=1024, q_head=128, q_heads=8,
           out=FAKE + 4096, out_row=1024, out_head=128, inv=FAKE, rotated=128, inter=0, qw=FAKE, kw=FAKE, eps=1e-6,
           ws=FAKE, ws_bytes=256):
    c = cache() if c is None else c
    return ds.lib().dspark_cache_append(ctypes.addressof(c) if c else None, layer, starts, counts, parents, B, N, rows,
                                        pages, most, lengths, k, k_row, k_head, v, v_row, v_head, q, q_row, q_head,
                                        q_heads, out, out_row, out_head, inv, rotated, inter, qw, kw, eps, ws, ws_bytes,
                                        None)


def attend(c=None, layer=0, starts=None, counts=FAKE, parents=None, B=2, N=4, rows=8, pages=FAKE, most=5, lengths=FAKE,
           q=FAKE, q_row=1024, q_head=128, q_heads=8, scale=0.1, out=FAKE, out_row=1024, out_head=128, lse=None,
           ws=FAKE, ws_bytes=1 << 30):
    c = cache() if c is None else c
    return ds.lib().dspark_tree_attention(ctypes.addressof(c), layer, starts, counts, parents, B, N, rows, pages, most,
                                          lengths, q, q_row, q_head, q_heads, scale, out, out_row, out_head, lse, ws,
                                          ws_bytes, None)


def verify(p=FAKE, ld_p=1000, q=FAKE, ld_q=1000, dtype=F32, V=1000, tokens=FAKE, u=FAKE, starts=None, counts=None,
           parents=None, B=2, N=4, rows=8, accept=FAKE, path=FAKE, out=FAKE, n_out=FAKE, ws=FAKE, ws_bytes=256):
    return ds.lib().dspark_tree_verify(p, ld_p, q, ld_q, dtype, V, tokens, u, starts, counts, parents, B, N, rows,
                                       accept, path, out, n_out, ws, ws_bytes, None)


def keep(c=None, B=2, N=4, pages=FAKE, most=5, lengths=FAKE, path=FAKE, accept=FAKE, ws=FAKE, ws_bytes=256):
    c = cache() if c is None else c
    return ds.lib().dspark_cache_keep(ctypes.addressof(c), B, N, pages, most, lengths, path, accept, ws, ws_bytes, None)


BAD_CACHES = [dict(k=None), dict(v=FAKE + 8), dict(dtype=F32), dict(dtype=3), dict(layers=0), dict(pages=0),
              dict(page=0), dict(heads=0), dict(D=0), dict(layer_s=-8), dict(page_s=8196), dict(slot_s=100),
              dict(slot_s=0), dict(head_s=0), dict(page_s=0), dict(layer_s=0), dict(head_s=1 << 50)]
FAR_CACHES = [dict(page=24), dict(page=8, page_s=4096), dict(page=512, page_s=1 << 20, layer_s=1 << 24),
              dict(D=24, head_s=32), dict(D=272, head_s=272, slot_s=2048)]


@pytest.mark.parametrize("call", [append, attend, keep])
def test_caches_refused(call):
    for bad in BAD_CACHES:
        assert call(cache(**bad)) == INVALID, bad
    for far in FAR_CACHES:
        assert call(cache(**far)) == UNSUPPORTED, far


BAD_ROWS = [dict(B=-1), dict(N=0), dict(rows=-1), dict(rows=7), dict(starts=FAKE), dict(counts=FAKE + 2),
            dict(parents=FAKE + 1), dict(counts=None, starts=FAKE + 1), dict(ws=None), dict(ws=FAKE + 16),
            dict(ws_bytes=255)]
FAR_ROWS = [dict(B=65536, rows=1 << 20), dict(N=65, rows=130, parents=FAKE), dict(rows=1 << 30)]


@pytest.mark.parametrize("call", [append, attend, verify])
def test_rows_refused(call):
    for bad in BAD_ROWS:
        if call is verify and bad == dict(starts=FAKE):
            bad = dict(starts=FAKE, counts=FAKE)
        assert call(**bad) == INVALID, bad
    for far in FAR_ROWS:
        assert call(**far) == UNSUPPORTED, far


@pytest.mark.parametrize("call", [append, attend, keep])
def test_tables_refused(call):
    for bad in (dict(pages=None), dict(pages=FAKE + 2), dict(lengths=None), dict(lengths=FAKE + 1), dict(most=0)):
        assert call(**bad) == INVALID, bad
    assert call(most=(1 << 26) + 1) == UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(layer=-1), dict(layer=2), dict(k=None), dict(k=FAKE + 8), dict(k_row=513), dict(k_head=4), dict(v=FAKE + 2),
    dict(v_row=-8), dict(q=None), dict(out=None), dict(q=FAKE + 4), dict(q_row=1028), dict(out_row=1020),
    dict(out_head=64), dict(out_row=0), dict(out=FAKE, out_row=2048), dict(q_heads=0), dict(inv=FAKE + 4),
    dict(rotated=0), dict(rotated=144), dict(qw=FAKE + 8), dict(kw=FAKE + 4), dict(eps=-1.0), dict(eps=NAN),
    dict(eps=INF), dict(q=None, out=None, q_heads=0)])
def test_append_refuses(bad):
    assert append(**bad) == INVALID


def test_append_limits_and_nothing_to_do():
    assert append(rotated=24) == UNSUPPORTED
    assert append(q_heads=65537) == UNSUPPORTED
    assert append(B=0, rows=0, pages=None, lengths=None, k=None, v=None, q=None, out=None, qw=None) == OK
    assert append(B=0, rows=0, ws=None) == INVALID


@pytest.mark.parametrize("bad", [
    dict(layer=2), dict(q=None), dict(q=FAKE + 8), dict(q_row=12), dict(out=None), dict(out_head=100), dict(out_head=64),
    dict(out_row=0), dict(q_heads=6), dict(q_heads=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN),
    dict(scale=INF), dict(lse=FAKE + 2), dict(ws_bytes=1 << 20)])
def test_attention_refuses(bad):
    assert attend(**bad) == INVALID


def test_attention_limits_and_nothing_to_do():
    for D in (96, 256):
        assert attend(cache(D=D, head_s=256, slot_s=1024, page_s=1 << 14, layer_s=1 << 18), out_head=256, out_row=2048) == UNSUPPORTED
    assert attend(N=65, rows=130) == UNSUPPORTED
    assert attend(cache(heads=1024, slot_s=1 << 17, page_s=1 << 21, layer_s=1 << 25), q_heads=1024, most=1 << 26) == UNSUPPORTED
    assert attend(B=0, rows=0, pages=None, lengths=None, q=None, out=None) == OK
    size = ds.lib().dspark_tree_attention_workspace_bytes
    assert size(2, 4, 8, 4, 128) > 0
    for bad in ((-1, 4, 8, 4, 128), (2, 0, 8, 4, 128), (2, 65, 8, 4, 128), (2, 4, 6, 4, 128), (2, 4, 8, 0, 128), (2, 4, 8, 4, 96)):
        assert size(*bad) == 0, bad


@pytest.mark.parametrize("bad", [
    dict(p=None), dict(p=FAKE + 2), dict(dtype=3), dict(ld_p=999), dict(q=FAKE + 1), dict(ld_q=10), dict(V=0),
    dict(tokens=None), dict(u=FAKE + 2), dict(accept=None), dict(path=FAKE + 1), dict(out=None), dict(n_out=None)])
def test_verify_refuses(bad):
    assert verify(**bad) == INVALID


def test_verify_limits_and_nothing_to_do():
    assert verify(N=65, rows=130) == UNSUPPORTED
    assert verify(V=(1 << 30) + 8, ld_p=1 << 31, ld_q=1 << 31) == UNSUPPORTED
    assert verify(B=0, rows=0, p=None, q=None, tokens=None, u=None, accept=None) == OK


def test_keep_refuses():
    for bad in (dict(B=-1), dict(N=0), dict(path=None), dict(accept=FAKE + 2), dict(ws=None), dict(ws_bytes=0)):
        assert keep(**bad) == INVALID, bad
    assert keep(N=65) == UNSUPPORTED
    assert keep(B=65536) == UNSUPPORTED
    assert keep(B=0, pages=None, lengths=None, path=None, accept=None) == OK
