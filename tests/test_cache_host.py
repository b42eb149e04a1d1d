"""Refusals of the 4-bit cache's entry points (no GPU): the C ABI returns its
status before anything is enqueued, the binding raises before it calls."""
import ctypes
import math

import pytest

import rejection_sampling_verify_12_amd as R

torch = pytest.importorskip("torch")
FAKE = 4096   # never dereferenced: every call below fails validation first


def cache(**kw):
    a = dict(data=FAKE, table=FAKE, pages=10, heads=2, page=64, dim=128, table_len=4)
    a.update(kw)
    return ctypes.byref(R.SpecCache(*a.values()))


BAD_CACHE = [dict(page=16), dict(page=48), dict(page=0), dict(page=512), dict(dim=96), dict(dim=0), dict(heads=0),
             dict(heads=-1), dict(pages=-1), dict(table_len=-1), dict(table_len=1 << 25), dict(data=None),
             dict(table=None), dict(data=FAKE + 8)]
BAD_CALL = [dict(B=-1), dict(n=0), dict(n=-3), dict(lag=2), dict(lag=-1), dict(B=1 << 13, n=1 << 12)]


def append(c=None, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=R.SPEC_BF16, ks=256, vs=256, len=None, lag=0, count=None, B=3, n=2, status=None,
             stream=None)
    a.update(kw)
    return R.load_library().spec_cache_append(cache(**(c or {})), *a.values())


def read(c=None, **kw):
    a = dict(len=None, lag=0, count=None, B=3, n=2, out_k=FAKE, out_v=FAKE, dtype=R.SPEC_BF16, status=None, stream=None)
    a.update(kw)
    return R.load_library().spec_cache_read(cache(**(c or {})), *a.values())


def attention(c=None, **kw):
    a = dict(q=FAKE, dtype=R.SPEC_BF16, qs=1024, heads_q=8, len=None, lag=0, count=None, B=3, n=2, scale=0.1, window=0,
             mask=None, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return R.load_library().spec_cache_attention(cache(**(c or {})), *a.values())


@pytest.mark.parametrize("call", [append, read, attention])
def test_bad_caches_and_sizes_are_refused(call):
    for c in BAD_CACHE:
        assert call(c) == R.SPEC_EINVAL, c
    for kw in BAD_CALL:
        assert call(**kw) == R.SPEC_EINVAL, kw
    assert call(dtype=2) == R.SPEC_EDTYPE
    assert call(dict(heads=1 << 24), n=1 << 10, B=4) == R.SPEC_EINVAL      # too many numbers
    assert call(dict(data=None, table=None), B=0) == R.SPEC_OK              # an empty batch is a no-op


def test_append_refuses():
    for kw in (dict(k=None), dict(v=None), dict(ks=-1), dict(vs=-1), dict(k=FAKE + 1), dict(v=FAKE + 2, dtype=R.SPEC_F32)):
        assert append(**kw) == R.SPEC_EINVAL, kw


def test_read_refuses():
    for kw in (dict(out_k=None), dict(out_v=None), dict(out_k=FAKE + 8), dict(out_v=FAKE + 2)):
        assert read(**kw) == R.SPEC_EINVAL, kw


def test_attention_refuses():
    for kw in (dict(q=None), dict(out=None), dict(qs=-1), dict(q=FAKE + 1), dict(out=FAKE + 8), dict(heads_q=0),
               dict(heads_q=3), dict(heads_q=1), dict(heads_q=-2), dict(scale=math.nan), dict(scale=math.inf), dict(scale=3.2e38),
               dict(window=-1), dict(n=65, mask=FAKE), dict(heads_q=1 << 30)):
        assert attention(**kw) == R.SPEC_EINVAL, kw
    assert attention(ws=None) == R.SPEC_EWORKSPACE
    assert attention(ws_bytes=8) == R.SPEC_EWORKSPACE


def test_size_queries():
    assert R.spec_cache_page_bytes(64, 128) == 64 * 136
    assert R.spec_cache_page_bytes(48, 128) == 0 and R.spec_cache_page_bytes(64, 80) == 0
    w = R.spec_cache_attention_workspace_bytes
    assert w(0, 1, 8, 8, 128) == 0 and w(-1, 1, 8, 8, 128) == 0 and w(2, 0, 8, 8, 128) == 0
    assert w(2, 1, 8, 3, 128) == 0 and w(2, 1, 8, 8, 96) == 0
    assert 0 < w(1, 1, 8, 8, 128) and w(1, 1, 8, 8, 128) % 256 == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_workspace_serves_every_smaller_call(dim):
    w = R.spec_cache_attention_workspace_bytes
    for heads, group in ((1, 1), (2, 5), (8, 4), (8, 16)):
        for n in (1, 2, 5, 9, 64, 700):
            sizes = [w(B, n, heads * group, heads, dim) for B in (1, 2, 3, 8, 64, 200)]
            assert sizes == sorted(sizes) and sizes[0] > 0
            big = w(64, n, heads * group, heads, dim)
            for m in {1, max(1, n // 3), n}:
                for g in {1, max(1, group // 2), group}:
                    for h in {1, heads}:
                        assert w(64, m, h * g, h, dim) <= big, (m, g, h)


def test_the_binding_refuses_before_it_calls():
    table = torch.zeros((2, 3), dtype=torch.int32)
    data = torch.zeros((4, 2, 64 * 136), dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        R.QuantCache(data, table, 64, 128)
    with pytest.raises(ValueError, match="page is"):
        R.QuantCache(data, table, 48, 128)
    with pytest.raises(ValueError, match="data is uint8"):
        R.QuantCache(data, table, 32, 128)
    with pytest.raises(ValueError, match="table is int32"):
        R.QuantCache(data, table.long(), 64, 128)


def test_token_strides():
    x = torch.zeros(3, 4, 5, 64)
    assert R._token_stride("k", x, 5, 64) == 320
    qkv = torch.zeros(3, 4, 9, 64)
    assert R._token_stride("k", qkv[:, :, 2:7], 5, 64) == 576
    assert R._token_stride("k", qkv[:, 1:2, 2:7], 5, 64) == 4 * 576      # one token each: the batch stride
    assert R._token_stride("k", qkv[1:2, 1:, 2:7], 5, 64) == 576
    for bad in (x.transpose(1, 2).contiguous().transpose(1, 2), x.transpose(2, 3).contiguous().transpose(2, 3),
                qkv[:, 1:3, 2:7], torch.zeros(4, 3, 5, 64).transpose(0, 1)):
        with pytest.raises(ValueError, match="side by side"):
            R._token_stride("k", bad, 5, 64)
    with pytest.raises(ValueError, match="got"):
        R._token_stride("k", x, 4, 64)
