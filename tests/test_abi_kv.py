"""Host-side argument checks of include/spec_kv.h: bad input is refused before any CUDA call."""
import math

import pytest

from speculative_decoding_verification_33_gb300 import _lib

BAD, UNS, OK = _lib.SV_ERR_INVALID_ARG, _lib.SV_ERR_UNSUPPORTED, _lib.SV_OK
P = 1 << 20  # a pointer that nothing follows: every call below returns before a launch


def tables(**kw):
    a = dict(B=4, page_size=16, max_blocks=8, max_tokens=10, ctx=P, acc=P + 64, new=P + 128,
             table=P, held=P + 192, ring=P, ring_size=40, counters=P, o_ctx=P + 256,
             o_held=P + 320, o_counters=P + 64, o_kv=P + 384, o_status=P + 448, o_cu=P,
             o_slots=P, o_pos=P, o_seq=P)
    a.update(kw)
    return _lib.load().spec_block_tables(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(page_size=0), dict(page_size=24), dict(page_size=256), dict(max_blocks=0),
    dict(max_blocks=1 << 27), dict(max_tokens=-1), dict(ring_size=0), dict(ctx=0), dict(new=0),
    dict(table=0), dict(held=0), dict(ring=0), dict(counters=0), dict(o_ctx=0), dict(o_held=0),
    dict(o_counters=0), dict(o_counters=P), dict(o_kv=0), dict(o_status=0), dict(o_cu=0),
    dict(o_slots=0), dict(o_pos=0), dict(o_seq=0), dict(o_ctx=P), dict(o_held=P + 192),
    dict(o_kv=P + 64), dict(o_status=P + 128)])
def test_tables_refusals(kw):
    assert tables(**kw) == BAD


def test_tables_too_many_sequences():
    assert tables(B=8193) == UNS


def norm_rope(**kw):
    a = dict(T=3, hq=4, hk=2, D=64, rot=64, inter=0, dtype=1, q=P, qs=256, k=P, ks=128, wq=P, wk=P,
             pos=P, freq=P, eps=1e-6, oq=P + 65536, oqs=256, ok=P + 65536, oks=128)
    a.update(kw)
    return _lib.load().spec_qk_norm_rope(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(hq=0), dict(hk=-1), dict(D=0), dict(D=63), dict(rot=-2), dict(rot=63),
    dict(rot=66), dict(dtype=2), dict(q=0), dict(k=0), dict(qs=255), dict(ks=127), dict(pos=0),
    dict(freq=0), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(oq=0), dict(ok=0),
    dict(oqs=255), dict(oks=127), dict(oq=P, oqs=512), dict(ok=P, oks=256)])
def test_norm_rope_refusals(kw):
    assert norm_rope(**kw) == BAD


def test_norm_rope_sizes():
    assert norm_rope(D=514, rot=0, qs=4 * 514, oqs=4 * 514, ks=2 * 514, oks=2 * 514) == UNS
    assert norm_rope(T=0) == OK  # nothing to launch
    assert norm_rope(T=0, q=0, k=0, pos=0, freq=0, oq=0, ok=0) == OK


def append(**kw):
    a = dict(T=3, H=2, D=64, ps=16, pages=5, dtype=1, k=P, ks=128, v=P, vs=128, slots=P, gk=1.0,
             gv=1.0, cache=P, ok=P, ov=P)
    a.update(kw)
    return _lib.load().spec_kv4_append(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(D=0), dict(pages=0), dict(dtype=7), dict(k=0), dict(v=0),
    dict(slots=0), dict(cache=0), dict(ks=127), dict(vs=127), dict(ks=132), dict(k=P + 8),
    dict(v=P + 2), dict(cache=P + 8), dict(ok=P + 8), dict(ov=P + 8), dict(gk=0.0), dict(gv=-1.0),
    dict(gk=math.nan), dict(gv=math.inf)])
def test_append_refusals(kw):
    assert append(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(D=96, ks=192, vs=192), dict(D=256, ks=512, vs=512),
                                dict(ps=8), dict(ps=48), dict(ps=256)])
def test_append_sizes(kw):
    assert append(**kw) == UNS
    assert append(T=0) == OK


def attention(**kw):
    a = dict(B=2, T=3, hq=4, hk=2, D=64, ps=16, pages=5, blocks=4, q=P, qs=256, cache=P, table=P,
             lens=P, cu=P, scale=0.125, gk=1.0, gv=1.0, most=1, out=P, lse=P)
    a.update(kw)
    return _lib.load().spec_kv4_attention(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(T=-1), dict(hq=0), dict(hk=0), dict(hq=5), dict(D=0), dict(pages=0),
    dict(blocks=0), dict(blocks=1 << 27), dict(q=0), dict(cache=0), dict(table=0), dict(lens=0),
    dict(cu=0), dict(out=0), dict(qs=255), dict(qs=257), dict(q=P + 8), dict(cache=P + 4),
    dict(out=P + 8), dict(scale=math.nan), dict(gk=math.inf), dict(gv=math.nan), dict(most=-1)])
def test_attention_refusals(kw):
    assert attention(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(D=32, qs=128), dict(D=96, qs=384), dict(ps=0), dict(ps=20),
                                dict(hq=64, T=1 << 26, qs=4096)])
def test_attention_sizes(kw):
    assert attention(**kw) == UNS
    assert attention(T=0) == OK and attention(B=0) == OK


@pytest.mark.parametrize("ps,D,n", [(16, 64, 16 * 72), (128, 128, 128 * 144), (24, 64, 0),
                                    (16, 96, 0), (0, 128, 0), (-16, 64, 0)])
def test_page_bytes(ps, D, n):
    assert _lib.load().spec_kv4_page_bytes(ps, D) == n
