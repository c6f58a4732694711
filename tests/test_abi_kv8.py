"""Host-side argument checks of the 8-bit cache's and the prompt's entry points (include/spec_kv.h): bad
input is refused before any CUDA call."""
import math

import pytest

from speculative_decoding_verification_33_gb300 import _lib

BAD, UNS, OK = _lib.SV_ERR_INVALID_ARG, _lib.SV_ERR_UNSUPPORTED, _lib.SV_OK
P = 1 << 20  # a pointer that nothing follows: every call below returns before a launch


def append(**kw):
    a = dict(T=3, H=2, D=64, ps=16, pages=5, dtype=1, k=P, ks=128, v=P, vs=128, slots=P, cache=P, ok=P, ov=P)
    a.update(kw)
    return _lib.load().spec_kv8_append(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(D=0), dict(pages=0), dict(dtype=7), dict(k=0), dict(v=0),
    dict(slots=0), dict(cache=0), dict(ks=127), dict(vs=127), dict(ks=132), dict(k=P + 8),
    dict(v=P + 2), dict(cache=P + 8), dict(ok=P + 8), dict(ov=P + 8)])
def test_append_refusals(kw):
    assert append(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(D=96, ks=192, vs=192), dict(D=256, ks=512, vs=512),
                                dict(ps=8), dict(ps=48), dict(ps=256),
                                dict(H=32768, ks=64 * 32768, vs=64 * 32768)])
def test_append_sizes(kw):
    assert append(**kw) == UNS
    assert append(T=0) == OK


def attention(**kw):
    a = dict(B=2, T=3, hq=4, hk=2, D=64, ps=16, pages=5, blocks=4, q=P, qs=256, cache=P, table=P,
             lens=P, cu=P, scale=0.125, most=1, out=P, lse=P)
    a.update(kw)
    return _lib.load().spec_kv8_attention(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(T=-1), dict(hq=0), dict(hk=0), dict(hq=5), dict(D=0), dict(pages=0),
    dict(blocks=0), dict(blocks=1 << 27), dict(q=0), dict(cache=0), dict(table=0), dict(lens=0),
    dict(cu=0), dict(out=0), dict(qs=255), dict(qs=257), dict(q=P + 8), dict(cache=P + 4),
    dict(out=P + 8), dict(scale=math.nan), dict(scale=math.inf), dict(most=-1)])
def test_attention_refusals(kw):
    assert attention(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(D=32, qs=128), dict(D=96, qs=384), dict(ps=0), dict(ps=20),
                                dict(hq=64, T=1 << 26, qs=4096)])
def test_attention_sizes(kw):
    assert attention(**kw) == UNS
    assert attention(T=0) == OK and attention(B=0) == OK


def prompt(**kw):
    a = dict(B=2, T=3, hq=4, hk=2, D=64, q=P, qs=256, k=P, ks=128, v=P, vs=128, cu=P, scale=0.125, out=P, lse=P)
    a.update(kw)
    return _lib.load().spec_prompt_attention(*a.values(), 0)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(T=-1), dict(hq=0), dict(hk=0), dict(hq=5), dict(D=0), dict(q=0), dict(k=0), dict(v=0),
    dict(cu=0), dict(out=0), dict(qs=255), dict(ks=127), dict(vs=127), dict(qs=260), dict(ks=132), dict(vs=129),
    dict(q=P + 8), dict(k=P + 2), dict(v=P + 4), dict(out=P + 8), dict(scale=math.nan), dict(scale=-math.inf)])
def test_prompt_refusals(kw):
    assert prompt(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(D=32, qs=128, ks=64, vs=64), dict(D=96, qs=384, ks=192, vs=192),
                                dict(hq=129, hk=1, qs=129 * 64), dict(hq=64, T=1 << 26, qs=4096)])
def test_prompt_sizes(kw):
    assert prompt(**kw) == UNS
    assert prompt(T=0) == OK and prompt(B=0) == OK


@pytest.mark.parametrize("ps,D,n", [(16, 64, 16 * 129), (128, 128, 128 * 257), (24, 64, 0),
                                    (16, 96, 0), (0, 128, 0), (-16, 64, 0)])
def test_page_bytes(ps, D, n):
    assert _lib.load().spec_kv8_page_bytes(ps, D) == n
