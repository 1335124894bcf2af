"""Host-side argument checks of the page plan, the rotated write, the attention
with sinks and behind shared prefixes: they return before any launch, so fake
(never dereferenced) pointers are fine. No GPU."""
import math

import pytest

from draft_verify_sampling_spec_amd import binding as sb

A = 0x10000


def _plan(**kw):
    a = dict(table=A, refs=A, ctx=A, budgets=A, parents=A, prefix=A, B=4, T=6, page_size=64, max_pages=8,
             num_pages=40, window=0, sinks=0, starts=A, slots=A, positions=A, status=None, ws=A, ws_bytes=None)
    a.update(kw)
    need = sb.spec_verify_pages_plan_workspace_bytes(max(a["B"], 1), a["max_pages"], a["num_pages"])
    return sb.spec_verify_pages_plan(
        a["table"], a["refs"], a["ctx"], a["budgets"], a["parents"], a["prefix"], a["B"], a["T"], a["page_size"],
        a["max_pages"], a["num_pages"], a["window"], a["sinks"], a["starts"], a["slots"], a["positions"],
        a["status"], a["ws"], need if a["ws_bytes"] is None else a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0, table=None, refs=None, ctx=None, ws=None), sb.SV_OK),
    (dict(B=-1), sb.SV_ERR_ARG),
    (dict(B=sb.SV_MAX_BATCH + 1), sb.SV_ERR_ARG),
    (dict(T=0), sb.SV_ERR_ARG),
    (dict(T=sb.SV_MAX_CONTEXT + 1), sb.SV_ERR_ARG),
    (dict(window=-1), sb.SV_ERR_ARG),
    (dict(sinks=-1), sb.SV_ERR_ARG),
    (dict(page_size=48), sb.SV_ERR_ARG),
    (dict(page_size=16), sb.SV_ERR_ARG),
    (dict(max_pages=0), sb.SV_ERR_ARG),
    (dict(max_pages=sb.SV_MAX_CONTEXT // 64 + 1), sb.SV_ERR_ARG),
    (dict(num_pages=0), sb.SV_ERR_ARG),
    (dict(num_pages=1 << 25), sb.SV_ERR_ARG),
    (dict(table=None), sb.SV_ERR_NULL),
    (dict(refs=None), sb.SV_ERR_NULL),
    (dict(ctx=None), sb.SV_ERR_NULL),
    (dict(prefix=None), sb.SV_ERR_NULL),
    (dict(starts=None), sb.SV_ERR_NULL),
    (dict(slots=None), sb.SV_ERR_NULL),
    (dict(positions=None), sb.SV_ERR_NULL),
    (dict(ws=None), sb.SV_ERR_NULL),
    (dict(table=A + 2), sb.SV_ERR_ALIGN),
    (dict(budgets=A + 1), sb.SV_ERR_ALIGN),
    (dict(prefix=A + 3), sb.SV_ERR_ALIGN),
    (dict(status=A + 2), sb.SV_ERR_ALIGN),
    (dict(ws=A + 64), sb.SV_ERR_ALIGN),
    (dict(ws_bytes=8), sb.SV_ERR_ARG),
])
def test_plan_argument_checks(kw, code):
    assert _plan(**kw) == code


def test_plan_workspace():
    size = sb.spec_verify_pages_plan_workspace_bytes
    assert size(0, 8, 40) == 0 and size(4, 0, 40) == 0 and size(4, 8, 0) == 0
    assert size(sb.SV_MAX_BATCH + 1, 8, 40) == 0
    # Small tables need none; others list the pool's free pages.
    assert size(4, 8, 40) == 256 and size(512, 1024, 40) > 4 * 1024
    assert size(4, 8, 1 << 20) >= 4 << 20
    assert size(sb.SV_MAX_BATCH, 1 << 19, 1 << 26) < 1 << 29


def _rotated(**kw):
    a = dict(q=A, k=A, v=A, dtype=sb.SV_DTYPE_BF16, qs=1024, ks=256, vs=256, slots=A, positions=A, tokens=24,
             inv_freq=A, rot=128, inter=0, factor=1.0, qn=A, kn=A, nd=sb.SV_DTYPE_F32, eps=1e-6, q_heads=8,
             kv_heads=2, head_dim=128, page_size=64, num_pages=10, cache=A, out=A, ok=None, status=None)
    a.update(kw)
    return sb.spec_verify_cache_write_rotated(
        a["q"], a["k"], a["v"], a["dtype"], a["qs"], a["ks"], a["vs"], a["slots"], a["positions"], a["tokens"],
        a["inv_freq"], a["rot"], a["inter"], a["factor"], a["qn"], a["kn"], a["nd"], a["eps"], a["q_heads"],
        a["kv_heads"], a["head_dim"], a["page_size"], a["num_pages"], a["cache"], a["out"], a["ok"], a["status"],
        None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0, q=None, k=None, v=None, cache=None), sb.SV_OK),
    (dict(tokens=-1), sb.SV_ERR_ARG),
    (dict(tokens=1 << 31), sb.SV_ERR_ARG),
    (dict(q_heads=7), sb.SV_ERR_ARG),
    (dict(q_heads=1), sb.SV_ERR_ARG),
    (dict(kv_heads=0), sb.SV_ERR_ARG),
    (dict(q_heads=2 * sb.SV_MAX_HEADS, qs=1 << 20), sb.SV_ERR_ARG),
    (dict(head_dim=96), sb.SV_ERR_ARG),
    (dict(page_size=33), sb.SV_ERR_ARG),
    (dict(num_pages=0), sb.SV_ERR_ARG),
    (dict(num_pages=1 << 25), sb.SV_ERR_ARG),
    (dict(rot=8), sb.SV_ERR_ARG),
    (dict(rot=144), sb.SV_ERR_ARG),
    (dict(rot=-16), sb.SV_ERR_ARG),
    (dict(factor=math.nan), sb.SV_ERR_ARG),
    (dict(factor=math.inf), sb.SV_ERR_ARG),
    (dict(eps=-1.0), sb.SV_ERR_ARG),
    (dict(eps=math.nan), sb.SV_ERR_ARG),
    (dict(dtype=2), sb.SV_ERR_DTYPE),
    (dict(nd=5), sb.SV_ERR_DTYPE),
    (dict(nd=5, qn=None, kn=None, q=None), sb.SV_ERR_NULL),
    (dict(qs=1016), sb.SV_ERR_ARG),
    (dict(ks=248), sb.SV_ERR_ARG),
    (dict(vs=1 << 31), sb.SV_ERR_ARG),
    (dict(qs=1028), sb.SV_ERR_ALIGN),
    (dict(vs=258, dtype=sb.SV_DTYPE_F32), sb.SV_ERR_ALIGN),
    (dict(q=None), sb.SV_ERR_NULL),
    (dict(k=None), sb.SV_ERR_NULL),
    (dict(v=None), sb.SV_ERR_NULL),
    (dict(slots=None), sb.SV_ERR_NULL),
    (dict(positions=None), sb.SV_ERR_NULL),
    (dict(inv_freq=None), sb.SV_ERR_NULL),
    (dict(cache=None), sb.SV_ERR_NULL),
    (dict(out=None), sb.SV_ERR_NULL),
    (dict(q=A + 8), sb.SV_ERR_ALIGN),
    (dict(kn=A + 4), sb.SV_ERR_ALIGN),
    (dict(ok=A + 2), sb.SV_ERR_ALIGN),
    (dict(out=A + 8), sb.SV_ERR_ALIGN),
    (dict(slots=A + 1), sb.SV_ERR_ALIGN),
    (dict(inv_freq=A + 2), sb.SV_ERR_ALIGN),
    (dict(status=A + 2), sb.SV_ERR_ALIGN),
])
def test_rotated_write_argument_checks(kw, code):
    assert _rotated(**kw) == code


def _sinks(**kw):
    a = dict(q=A, qs=8 * 128, cache=A, page_table=A, ctx=A, budgets=A, B=4, K=4, q_heads=8, kv_heads=2, head_dim=128,
             page_size=64, max_pages=8, num_pages=16, scale=0.1, window=100, sinks=4, out=A, status=None, ws=A,
             ws_bytes=None)
    a.update(kw)
    need = sb.spec_verify_attention_sinks_workspace_bytes(max(a["B"], 1), a["K"], a["q_heads"], a["kv_heads"],
                                                          a["head_dim"], a["page_size"], a["max_pages"],
                                                          a["window"], a["sinks"])
    return sb.spec_verify_attention_sinks(
        a["q"], a["qs"], a["cache"], a["page_table"], a["ctx"], a["budgets"], a["B"], a["K"], a["q_heads"],
        a["kv_heads"], a["head_dim"], a["page_size"], a["max_pages"], a["num_pages"], a["scale"], a["window"],
        a["sinks"], a["out"], a["status"], a["ws"], need if a["ws_bytes"] is None else a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0, q=None, out=None, ws=None), sb.SV_OK),
    (dict(B=0, q=None, out=None, ws=None, window=0), sb.SV_OK),
    (dict(sinks=-1), sb.SV_ERR_ARG),
    (dict(window=-1), sb.SV_ERR_ARG),
    (dict(window=0, sinks=-1), sb.SV_ERR_ARG),
    (dict(K=sb.SV_MAX_K + 1), sb.SV_ERR_ARG),
    (dict(q_heads=7), sb.SV_ERR_ARG),
    (dict(num_pages=0), sb.SV_ERR_ARG),
    (dict(scale=math.nan), sb.SV_ERR_ARG),
    (dict(ws_bytes=0), sb.SV_ERR_ARG),
    (dict(q=None), sb.SV_ERR_NULL),
    (dict(ws=None), sb.SV_ERR_NULL),
    (dict(q=A + 8), sb.SV_ERR_ALIGN),
    (dict(ws=A + 16), sb.SV_ERR_ALIGN),
])
def test_attention_with_sinks_argument_checks(kw, code):
    assert _sinks(**kw) == code


def test_attention_with_sinks_workspace():
    size = sb.spec_verify_attention_sinks_workspace_bytes
    plain = sb.spec_verify_attention_workspace_bytes
    # Short spans are never split; sinks count among them.
    assert size(4, 4, 8, 2, 128, 64, 2048, 100, 4) == 256
    assert size(4, 4, 8, 2, 128, 64, 2048, 100, 5000) > 256
    assert size(4, 4, 8, 2, 128, 64, 2048, 0, 5000) == plain(4, 4, 8, 2, 128, 64, 2048, 0)
    assert size(4, 4, 8, 2, 128, 64, 2048, 100, -1) == 0 and size(0, 4, 8, 2, 128, 64, 2048, 100, 4) == 0
    assert size(4, 4, 8, 2, 128, 64, 2048, 2**31 - 1, 2**31 - 1) == plain(4, 4, 8, 2, 128, 64, 2048)


def _shared(**kw):
    a = dict(q=A, qs=8 * 128, cache=A, page_table=A, ctx=A, budgets=A, groups=A, lens=A, B=4, K=4, G=2, q_heads=8,
             kv_heads=2, head_dim=128, page_size=64, max_pages=8, num_pages=16, scale=0.1, out=A, status=None, ws=A,
             ws_bytes=None)
    a.update(kw)
    need = sb.spec_verify_attention_shared_workspace_bytes(max(a["B"], 1), a["K"], a["G"], a["q_heads"],
                                                           a["kv_heads"], a["head_dim"], a["page_size"],
                                                           a["max_pages"])
    return sb.spec_verify_attention_shared(
        a["q"], a["qs"], a["cache"], a["page_table"], a["ctx"], a["budgets"], a["groups"], a["lens"], a["B"], a["K"],
        a["G"], a["q_heads"], a["kv_heads"], a["head_dim"], a["page_size"], a["max_pages"], a["num_pages"],
        a["scale"], a["out"], a["status"], a["ws"], need if a["ws_bytes"] is None else a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0, q=None, out=None, ws=None, groups=None), sb.SV_OK),
    (dict(B=0, G=0, q=None, out=None, ws=None, groups=None), sb.SV_OK),
    (dict(G=-1), sb.SV_ERR_ARG),
    (dict(G=sb.SV_MAX_GROUPS + 1), sb.SV_ERR_ARG),
    (dict(K=-1), sb.SV_ERR_ARG),
    (dict(q_heads=7), sb.SV_ERR_ARG),
    (dict(head_dim=32), sb.SV_ERR_ARG),
    (dict(num_pages=0), sb.SV_ERR_ARG),
    (dict(scale=math.inf), sb.SV_ERR_ARG),
    (dict(ws_bytes=4096), sb.SV_ERR_ARG),
    (dict(qs=1016), sb.SV_ERR_ARG),
    (dict(q=None), sb.SV_ERR_NULL),
    (dict(groups=None), sb.SV_ERR_NULL),
    (dict(lens=None), sb.SV_ERR_NULL),
    (dict(ws=None), sb.SV_ERR_NULL),
    (dict(groups=A + 2), sb.SV_ERR_ALIGN),
    (dict(lens=A + 1), sb.SV_ERR_ALIGN),
    (dict(q=A + 8), sb.SV_ERR_ALIGN),
    (dict(ws=A + 16), sb.SV_ERR_ALIGN),
])
def test_attention_behind_shared_prefixes_argument_checks(kw, code):
    assert _shared(**kw) == code


def test_attention_behind_shared_prefixes_workspace():
    size = sb.spec_verify_attention_shared_workspace_bytes
    assert size(0, 4, 2, 8, 2, 128, 64, 8) == 0 and size(4, 4, -1, 8, 2, 128, 64, 8) == 0
    assert size(4, 4, sb.SV_MAX_GROUPS + 1, 8, 2, 128, 64, 8) == 0 and size(4, 4, 2, 8, 3, 128, 64, 8) == 0
    assert size(4, 4, 0, 8, 2, 128, 64, 8) == sb.spec_verify_attention_workspace_bytes(4, 4, 8, 2, 128, 64, 8)
    # At least one fp32 partial result of every row.
    assert size(128, 8, 1, 32, 8, 128, 64, 100) > 128 * 9 * 32 * 128 * 4
    assert size(sb.SV_MAX_BATCH, 32, 512, 256, 256, 256, 64, 1 << 18) > 1 << 35
