"""Host-side argument checks of the 4-bit cache, the blocks' attention and the
8-bit head: they return before any launch, so fake (never dereferenced)
pointers are fine. No GPU."""
import math

import pytest

from draft_verify_sampling_spec_amd import binding as sb

A = 0x10000


def _geometry(**kw):
    return {**dict(page_table=A, B=4, kv_heads=2, head_dim=128, page_size=64, max_pages=8,
                   num_pages=16, cache=A, out_status=None), **kw}


_BAD_GEOMETRY = [
    (dict(B=-1), sb.SV_ERR_ARG),
    (dict(B=sb.SV_MAX_BATCH + 1), sb.SV_ERR_ARG),
    (dict(kv_heads=0), sb.SV_ERR_ARG),
    (dict(kv_heads=sb.SV_MAX_HEADS + 1), sb.SV_ERR_ARG),
    (dict(head_dim=96), sb.SV_ERR_ARG),
    (dict(head_dim=512), sb.SV_ERR_ARG),
    (dict(page_size=16), sb.SV_ERR_ARG),
    (dict(page_size=96), sb.SV_ERR_ARG),
    (dict(page_size=2 * sb.SV_MAX_PAGE), sb.SV_ERR_ARG),
    (dict(max_pages=0), sb.SV_ERR_ARG),
    (dict(max_pages=sb.SV_MAX_CONTEXT // 64 + 1), sb.SV_ERR_ARG),
    (dict(num_pages=0), sb.SV_ERR_ARG),
    (dict(page_table=None), sb.SV_ERR_NULL),
    (dict(cache=None), sb.SV_ERR_NULL),
    (dict(cache=A + 8), sb.SV_ERR_ALIGN),
    (dict(page_table=A + 2), sb.SV_ERR_ALIGN),
    (dict(out_status=A + 1), sb.SV_ERR_ALIGN),
    (dict(B=0, page_table=None, cache=None), sb.SV_OK),
]


def _write(**kw):
    a = _geometry(keys=A, values=A, dtype=sb.SV_DTYPE_BF16, ks=256, vs=256, ctx=A, budgets=A, T=5)
    a.update(kw)
    return sb.spec_verify_cache_write(
        a["keys"], a["values"], a["dtype"], a["ks"], a["vs"], a["page_table"], a["ctx"],
        a["budgets"], a["B"], a["T"], a["kv_heads"], a["head_dim"], a["page_size"],
        a["max_pages"], a["num_pages"], a["cache"], a["out_status"], None)


@pytest.mark.parametrize("kw,code", _BAD_GEOMETRY + [
    (dict(T=-1), sb.SV_ERR_ARG),
    (dict(T=0, keys=None), sb.SV_OK),
    (dict(T=sb.SV_MAX_CONTEXT + 1), sb.SV_ERR_ARG),
    (dict(T=sb.SV_MAX_CONTEXT, kv_heads=8, ks=1024, vs=1024), sb.SV_ERR_ARG),
    (dict(dtype=2), sb.SV_ERR_DTYPE),
    (dict(ks=255), sb.SV_ERR_ARG),
    (dict(vs=248), sb.SV_ERR_ARG),
    (dict(ks=260), sb.SV_ERR_ALIGN),
    (dict(ks=258, dtype=sb.SV_DTYPE_F32), sb.SV_ERR_ALIGN),
    (dict(keys=None), sb.SV_ERR_NULL),
    (dict(values=None), sb.SV_ERR_NULL),
    (dict(ctx=None), sb.SV_ERR_NULL),
    (dict(keys=A + 8), sb.SV_ERR_ALIGN),
    (dict(values=A + 4), sb.SV_ERR_ALIGN),
    (dict(ctx=A + 2), sb.SV_ERR_ALIGN),
    (dict(budgets=A + 1), sb.SV_ERR_ALIGN),
])
def test_cache_write_argument_checks(kw, code):
    assert _write(**kw) == code


def _read(**kw):
    a = _geometry(starts=A, lens=A, T=5, dtype=sb.SV_DTYPE_F32, ok=A, ov=A)
    a.update(kw)
    return sb.spec_verify_cache_read(
        a["cache"], a["page_table"], a["starts"], a["lens"], a["B"], a["T"], a["kv_heads"],
        a["head_dim"], a["page_size"], a["max_pages"], a["num_pages"], a["dtype"], a["ok"],
        a["ov"], a["out_status"], None)


@pytest.mark.parametrize("kw,code", _BAD_GEOMETRY + [
    (dict(T=-1), sb.SV_ERR_ARG),
    (dict(T=0, lens=None), sb.SV_OK),
    (dict(T=sb.SV_MAX_CONTEXT, kv_heads=8), sb.SV_ERR_ARG),
    (dict(dtype=-1), sb.SV_ERR_DTYPE),
    (dict(lens=None), sb.SV_ERR_NULL),
    (dict(ok=None), sb.SV_ERR_NULL),
    (dict(ov=None), sb.SV_ERR_NULL),
    (dict(ok=A + 8), sb.SV_ERR_ALIGN),
    (dict(starts=A + 2), sb.SV_ERR_ALIGN),
    (dict(lens=A + 3), sb.SV_ERR_ALIGN),
])
def test_cache_read_argument_checks(kw, code):
    assert _read(**kw) == code


def _attend(**kw):
    a = _geometry(q=A, qs=8 * 128, ctx=A, budgets=A, K=4, q_heads=8, scale=0.1, window=0, out=A,
                  ws=A, ws_bytes=None)
    a.update(kw)
    need = sb.spec_verify_attention_workspace_bytes(max(a["B"], 1), a["K"], a["q_heads"],
                                                    a["kv_heads"], a["head_dim"], a["page_size"],
                                                    a["max_pages"], a["window"])
    return sb.spec_verify_attention(
        a["q"], a["qs"], a["cache"], a["page_table"], a["ctx"], a["budgets"], a["B"], a["K"],
        a["q_heads"], a["kv_heads"], a["head_dim"], a["page_size"], a["max_pages"],
        a["num_pages"], a["scale"], a["window"], a["out"], a["out_status"], a["ws"],
        need if a["ws_bytes"] is None else a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [c for c in _BAD_GEOMETRY if "B" not in c[0] or c[0]["B"] != 0] + [
    (dict(B=0, q=None, out=None, ws=None, page_table=None, cache=None), sb.SV_OK),
    (dict(K=-1), sb.SV_ERR_ARG),
    (dict(K=sb.SV_MAX_K + 1), sb.SV_ERR_ARG),
    (dict(q_heads=7), sb.SV_ERR_ARG),
    (dict(q_heads=1), sb.SV_ERR_ARG),
    (dict(q_heads=2 * sb.SV_MAX_HEADS, qs=1 << 20), sb.SV_ERR_ARG),
    (dict(scale=math.nan), sb.SV_ERR_ARG),
    (dict(scale=math.inf), sb.SV_ERR_ARG),
    (dict(window=-1), sb.SV_ERR_ARG),
    (dict(qs=8 * 128 - 8), sb.SV_ERR_ARG),
    (dict(qs=8 * 128 + 4), sb.SV_ERR_ALIGN),
    (dict(q=None), sb.SV_ERR_NULL),
    (dict(ctx=None), sb.SV_ERR_NULL),
    (dict(out=None), sb.SV_ERR_NULL),
    (dict(ws=None), sb.SV_ERR_NULL),
    (dict(q=A + 8), sb.SV_ERR_ALIGN),
    (dict(out=A + 8), sb.SV_ERR_ALIGN),
    (dict(ws=A + 16), sb.SV_ERR_ALIGN),
    (dict(ctx=A + 2), sb.SV_ERR_ALIGN),
    (dict(budgets=A + 2), sb.SV_ERR_ALIGN),
    (dict(ws_bytes=0), sb.SV_ERR_ARG),
])
def test_attention_argument_checks(kw, code):
    assert _attend(**kw) == code


def test_sizes():
    assert sb.spec_verify_cache_bytes(3, 2, 128, 64) == 3 * 2 * 2 * 34 * 128
    assert sb.spec_verify_cache_bytes(0, 2, 128, 64) == 0
    assert sb.spec_verify_cache_bytes(3, 2, 100, 64) == 0
    # Past 32 bits: 2^20 pages of 8 heads.
    assert sb.spec_verify_cache_bytes(1 << 20, 8, 128, 64) == (1 << 20) * 8 * 2 * 34 * 128
    assert sb.spec_verify_attention_workspace_bytes(0, 4, 8, 2, 128, 64, 8) == 0
    assert sb.spec_verify_attention_workspace_bytes(4, 4, 8, 3, 128, 64, 8) == 0
    one = sb.spec_verify_attention_workspace_bytes(1, 4, 8, 2, 128, 64, 2048)
    assert one >= 2 * 2 * 20 * 128 * 4          # split, two heads of 20 rows, fp32 partials
    # The most requests and heads need no more than the scratch of a few GiB.
    assert sb.spec_verify_attention_workspace_bytes(sb.SV_MAX_BATCH, 32, 256, 8, 128, 64, 2048) < 1 << 33


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), sb.SV_ERR_ARG),
    (dict(rows=sb.SV_MAX_VOCAB + 1), sb.SV_ERR_ARG),
    (dict(H=0), sb.SV_ERR_ARG),
    (dict(H=12), sb.SV_ERR_ARG),
    (dict(H=sb.SV_MAX_HIDDEN + 8), sb.SV_ERR_ARG),
    (dict(block=64), sb.SV_ERR_ARG),
    (dict(dtype=9), sb.SV_ERR_DTYPE),
    (dict(src=None), sb.SV_ERR_NULL),
    (dict(codes=None), sb.SV_ERR_NULL),
    (dict(scales=None), sb.SV_ERR_NULL),
    (dict(src=A + 8), sb.SV_ERR_ALIGN),
    (dict(codes=A + 8), sb.SV_ERR_ALIGN),
    (dict(rows=0, src=None, codes=None, scales=None), sb.SV_OK),
])
def test_head_quantize_argument_checks(kw, code):
    a = {**dict(src=A, dtype=sb.SV_DTYPE_BF16, rows=8, H=64, block=1, codes=A, scales=A), **kw}
    assert sb.spec_head_quantize(a["src"], a["dtype"], a["rows"], a["H"], a["block"], a["codes"],
                                 a["scales"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), sb.SV_ERR_ARG),
    (dict(R=sb.SV_MAX_VOCAB + 1), sb.SV_ERR_ARG),
    (dict(H=0), sb.SV_ERR_ARG),
    (dict(H=sb.SV_MAX_HIDDEN + 1), sb.SV_ERR_ARG),
    (dict(V=0), sb.SV_ERR_ARG),
    (dict(V=sb.SV_MAX_VOCAB + 1), sb.SV_ERR_ARG),
    (dict(dtype=3), sb.SV_ERR_DTYPE),
    (dict(hc=None), sb.SV_ERR_NULL),
    (dict(hs=None), sb.SV_ERR_NULL),
    (dict(wc=None), sb.SV_ERR_NULL),
    (dict(ws=None), sb.SV_ERR_NULL),
    (dict(out=None), sb.SV_ERR_NULL),
    (dict(hc=A + 8), sb.SV_ERR_ALIGN),
    (dict(wc=A + 4), sb.SV_ERR_ALIGN),
    (dict(out=A + 2), sb.SV_ERR_ALIGN),
    (dict(out=A + 1, dtype=sb.SV_DTYPE_BF16), sb.SV_ERR_ALIGN),
    (dict(R=0, hc=None, wc=None, out=None), sb.SV_OK),
])
def test_head_logits_argument_checks(kw, code):
    a = {**dict(hc=A, hs=A, wc=A, ws=A, R=4, H=128, V=100, dtype=sb.SV_DTYPE_F32, out=A), **kw}
    assert sb.spec_head_logits(a["hc"], a["hs"], a["wc"], a["ws"], a["R"], a["H"], a["V"],
                               a["dtype"], a["out"], None) == code
