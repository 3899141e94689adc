"""Refusals of the latent operators and of the step tables, without a GPU: the
C calls report bad arguments before anything is launched, and the binding names
the tensor that is wrong.  (The addresses below are never read.)"""
import ctypes

import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from paged_kv_cache_263_gb300 import build as pkv_build

A = 1 << 20     # any 256-byte aligned address
OK, INVALID, UNSUPPORTED = 0, 1, 3


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def _call(name, order, base, **change):
    args = dict(base, **change)
    return getattr(pkv.lib(), name)(*[args[k] for k in order])


STEP = dict(tables=A, mb=4, ctx=2 * A, new=3 * A, B=8, free=4 * A, nfree=8, nb=64, cu=5 * A, lens=6 * A, slots=7 * A,
            pos=8 * A, cap=32, totals=9 * A, stream=None)


@pytest.mark.parametrize("change", [
    dict(B=-1), dict(mb=0), dict(mb=1 << 28), dict(nfree=-1), dict(nb=0), dict(cap=-1), dict(nb=1 << 28),
    dict(tables=None), dict(ctx=None), dict(new=None), dict(free=None), dict(cu=None), dict(lens=None),
    dict(slots=None), dict(pos=None), dict(totals=None), dict(slots=7 * A + 4), dict(ctx=2 * A + 2),
    # overlaps: in place, an output over an input's tail, two outputs
    dict(lens=2 * A), dict(lens=3 * A + 28), dict(tables=4 * A - 124), dict(pos=7 * A + 252), dict(totals=5 * A + 32)])
def test_step_tables_refuses(change):
    assert _call("kv_build_step_tables", list(STEP), STEP, **change) == INVALID


WRITE = dict(lat=A, ls=512, rope=2 * A, rs=64, cache=3 * A, slots=4 * A, T=4, nb=8, stream=None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(nb=0), dict(lat=None), dict(rope=None), dict(cache=None), dict(slots=None), dict(ls=-8),
    dict(ls=516), dict(rs=65), dict(lat=A + 8), dict(rope=2 * A + 2), dict(cache=3 * A + 8), dict(slots=4 * A + 4)])
def test_latent_write_refuses(change):
    assert _call("reshape_and_cache_latent", list(WRITE), WRITE, **change) == INVALID


def test_latent_write_of_nothing():
    assert _call("reshape_and_cache_latent", list(WRITE), WRITE, T=0) == OK


ABS = dict(out=A, q=2 * A, cu=3 * A, lens=4 * A, B=4, R=4, cache=5 * A, tables=6 * A, mb=8, h=32, nb=64, scale=0.1,
           ws=7 * A, nbytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), INVALID), (dict(R=-1), INVALID), (dict(h=0), INVALID), (dict(h=129), UNSUPPORTED),
    (dict(mb=0), INVALID), (dict(nb=0), INVALID), (dict(mb=1 << 28), UNSUPPORTED), (dict(nb=1 << 28), UNSUPPORTED),
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(lens=None), INVALID), (dict(cache=None), INVALID),
    (dict(tables=None), INVALID), (dict(cu=None, R=5), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(out=A + 8), INVALID), (dict(q=2 * A + 2), INVALID), (dict(cache=5 * A + 4), INVALID),
    (dict(cu=3 * A + 2), INVALID), (dict(lens=4 * A + 1), INVALID)])
def test_absorbed_refuses(change, status):
    assert _call("paged_latent_attention", list(ABS), ABS, **change) == status


@pytest.mark.parametrize("change", [dict(ws=None, nbytes=0), dict(ws=7 * A + 16), dict(nbytes=-1)])
def test_absorbed_workspace_refusals(change):
    need = pkv.paged_latent_attention_workspace_size(4, 4, 32, 8)
    if need == 0:
        pytest.skip("these sizes need no workspace")
    if change.get("nbytes") == -1:
        change = dict(nbytes=need - 1)
    assert _call("paged_latent_attention", list(ABS), ABS, **change) == INVALID


def test_absorbed_of_nothing():
    assert _call("paged_latent_attention", list(ABS), ABS, B=0) == OK
    assert _call("paged_latent_attention", list(ABS), ABS, R=0) == OK


EXP = dict(out=A, q=2 * A, kv=3 * A, rope=4 * A, rs=64, cu_q=5 * A, cu_k=6 * A, B=4, R=64, K=64, h=32, scale=0.1,
           ws=7 * A, nbytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), INVALID), (dict(R=-1), INVALID), (dict(K=-1), INVALID), (dict(h=0), INVALID),
    (dict(h=129), UNSUPPORTED), (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(kv=None), INVALID),
    (dict(rope=None), INVALID), (dict(cu_q=None), INVALID), (dict(cu_k=None), INVALID), (dict(rs=56), INVALID),
    (dict(rs=68), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(out=A + 8), INVALID), (dict(q=2 * A + 8), INVALID), (dict(kv=3 * A + 2), INVALID),
    (dict(rope=4 * A + 8), INVALID), (dict(cu_q=5 * A + 2), INVALID), (dict(cu_k=6 * A + 1), INVALID)])
def test_expanded_refuses(change, status):
    assert _call("latent_prefill_attention", list(EXP), EXP, **change) == status


@pytest.mark.parametrize("change", [dict(ws=None, nbytes=0), dict(ws=7 * A + 16), dict(nbytes=-1)])
def test_expanded_workspace_refusals(change):
    need = pkv.latent_prefill_attention_workspace_size(4, 64, 32)
    if need == 0:
        pytest.skip("these sizes need no workspace")
    if change.get("nbytes") == -1:
        change = dict(nbytes=need - 1)
    assert _call("latent_prefill_attention", list(EXP), EXP, **change) == INVALID


def test_expanded_of_nothing():
    assert _call("latent_prefill_attention", list(EXP), EXP, B=0) == OK
    assert _call("latent_prefill_attention", list(EXP), EXP, R=0) == OK


def test_binding_names_a_tensor_that_is_not_on_a_gpu():
    z = torch.zeros
    i32, bf = torch.int32, torch.bfloat16
    with pytest.raises(ValueError, match="block_tables"):
        pkv.kv_build_step_tables(z(2, 4, dtype=i32), *[z(2, dtype=i32)] * 3, 8, *[z(2, dtype=i32)] * 5)
    with pytest.raises(ValueError, match="cache"):
        pkv.reshape_and_cache_latent(z(2, 512, dtype=bf), z(2, 64, dtype=bf), z(2, 16, 576, dtype=bf),
                                     z(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="q must be"):
        pkv.paged_latent_attention(z(1, 4, 512, dtype=bf), z(1, 4, 576, dtype=bf), z(2, 16, 576, dtype=bf),
                                   z(1, 2, dtype=i32), z(1, dtype=i32))
    with pytest.raises(ValueError, match="q must be"):
        pkv.latent_prefill_attention(z(1, 4, 128, dtype=bf), z(1, 4, 192, dtype=bf), z(1, 4, 256, dtype=bf),
                                     z(1, 64, dtype=bf), z(2, dtype=i32), z(2, dtype=i32))
    with pytest.raises(ValueError, match="required"):
        pkv.paged_latent_attention(None, None, None, None, None)
