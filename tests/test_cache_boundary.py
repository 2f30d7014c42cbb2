"""CPU tests of the paged cache's C ABI and binding: what each call refuses, with
which code, and what it hands to the library."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from scaled_dot_product_10_b200 import attn
from scaled_dot_product_10_b200.build import build
from test_binding_marshal import STREAM, FakeCuda, FakeLib, bf16, check_call, f32, u8

A = 0x10000  # addresses that no refused call follows


@pytest.fixture(scope="module")
def clib():
    build()
    return attn.load_library()


def cache_struct(**changes):
    f = dict(k_pages=A, v_pages=A, k_scale=A, v_scale=A, page_stride=16 * 2 * 128,
             token_stride=2 * 128, head_stride=128, num_pages=10, page_size=16, h_kv=2, d=128,
             type=1)
    f.update(changes)
    return attn._CacheStruct(**f)


APPEND = dict(k=A, v=A, q=A, q_out=A, page_table=A, seqlens_k=A, cu_seqlens=A, inv_freq=A, batch=3,
              max_pages=4, total=7, max_seqlen=5, h_q=4, k_stride=256, v_stride=256, q_stride=512,
              rotary_dim=64, interleaved=0, stream=None)
FWD = dict(q=A, o=A, lse=A, page_table=A, seqlens_k=A, cu_seqlens_q=A, batch=3, max_pages=4,
           total_q=7, max_seqlen_q=5, h_q=4, q_stride=512, causal=1, window_left=-1, scale=0.1,
           workspace=A, workspace_bytes=1 << 40, stream=None)

CACHE_RULES = [
    (dict(k_pages=None), attn.ATTN_ERR_INVALID), (dict(v_pages=None), attn.ATTN_ERR_INVALID),
    (dict(type=2), attn.ATTN_ERR_INVALID), (dict(type=0), attn.ATTN_ERR_INVALID),
    (dict(k_scale=None), attn.ATTN_ERR_INVALID), (dict(v_scale=None), attn.ATTN_ERR_INVALID),
    (dict(num_pages=0), attn.ATTN_ERR_INVALID), (dict(page_size=0), attn.ATTN_ERR_INVALID),
    (dict(page_size=12), attn.ATTN_ERR_INVALID), (dict(page_size=1 << 21), attn.ATTN_ERR_INVALID),
    (dict(h_kv=0), attn.ATTN_ERR_INVALID), (dict(h_kv=3), attn.ATTN_ERR_INVALID),
    (dict(d=64), attn.ATTN_ERR_UNSUPPORTED), (dict(d=0), attn.ATTN_ERR_INVALID),
    (dict(page_stride=0), attn.ATTN_ERR_INVALID), (dict(token_stride=-256), attn.ATTN_ERR_INVALID),
    (dict(head_stride=120), attn.ATTN_ERR_INVALID),
    (dict(page_stride=1 << 40), attn.ATTN_ERR_INVALID),
    (dict(k_pages=A + 8), attn.ATTN_ERR_ALIGN), (dict(v_pages=A + 1), attn.ATTN_ERR_ALIGN),
    (dict(k_scale=A + 2), attn.ATTN_ERR_ALIGN),
]
APPEND_RULES = [
    (dict(k=None), attn.ATTN_ERR_INVALID), (dict(v=None), attn.ATTN_ERR_INVALID),
    (dict(q=None), attn.ATTN_ERR_INVALID), (dict(q_out=None), attn.ATTN_ERR_INVALID),
    (dict(page_table=None), attn.ATTN_ERR_INVALID), (dict(seqlens_k=None), attn.ATTN_ERR_INVALID),
    (dict(inv_freq=None), attn.ATTN_ERR_INVALID), (dict(rotary_dim=0), attn.ATTN_ERR_INVALID),
    (dict(rotary_dim=24), attn.ATTN_ERR_INVALID), (dict(rotary_dim=144), attn.ATTN_ERR_INVALID),
    (dict(rotary_dim=-16), attn.ATTN_ERR_INVALID), (dict(interleaved=2), attn.ATTN_ERR_INVALID),
    (dict(batch=0), attn.ATTN_ERR_INVALID), (dict(max_pages=0), attn.ATTN_ERR_INVALID),
    (dict(total=0), attn.ATTN_ERR_INVALID), (dict(max_seqlen=0), attn.ATTN_ERR_INVALID),
    (dict(h_q=0), attn.ATTN_ERR_INVALID), (dict(h_q=5), attn.ATTN_ERR_INVALID),
    (dict(cu_seqlens=None), attn.ATTN_ERR_INVALID),  # 7 rows do not divide by 3
    (dict(k_stride=255), attn.ATTN_ERR_INVALID), (dict(v_stride=128), attn.ATTN_ERR_INVALID),
    (dict(q_stride=504), attn.ATTN_ERR_INVALID),
    (dict(batch=1 << 20, max_seqlen=1 << 30, total=1 << 30), attn.ATTN_ERR_INVALID),  # CTAs
    (dict(k=A + 8), attn.ATTN_ERR_ALIGN), (dict(q_out=A + 2), attn.ATTN_ERR_ALIGN),
    (dict(page_table=A + 1), attn.ATTN_ERR_ALIGN), (dict(cu_seqlens=A + 2), attn.ATTN_ERR_ALIGN),
    (dict(inv_freq=A + 2), attn.ATTN_ERR_ALIGN),
]
FWD_RULES = [
    (dict(q=None), attn.ATTN_ERR_INVALID), (dict(o=None), attn.ATTN_ERR_INVALID),
    (dict(lse=None), attn.ATTN_ERR_INVALID), (dict(workspace=None), attn.ATTN_ERR_INVALID),
    (dict(page_table=None), attn.ATTN_ERR_INVALID), (dict(batch=-1), attn.ATTN_ERR_INVALID),
    (dict(total_q=0), attn.ATTN_ERR_INVALID), (dict(max_seqlen_q=0), attn.ATTN_ERR_INVALID),
    (dict(h_q=3), attn.ATTN_ERR_INVALID), (dict(cu_seqlens_q=None), attn.ATTN_ERR_INVALID),
    (dict(scale=float("nan")), attn.ATTN_ERR_INVALID),
    (dict(scale=float("inf")), attn.ATTN_ERR_INVALID), (dict(causal=2), attn.ATTN_ERR_INVALID),
    (dict(window_left=-2), attn.ATTN_ERR_INVALID),
    (dict(window_left=4, causal=0), attn.ATTN_ERR_INVALID),
    (dict(q_stride=500), attn.ATTN_ERR_INVALID),
    (dict(total_q=1 << 30, max_seqlen_q=1 << 30), attn.ATTN_ERR_INVALID),  # 32-bit row numbers
    (dict(max_pages=1 << 27), attn.ATTN_ERR_INVALID),  # 2^31 keys of pages of 16
    (dict(q=A + 4), attn.ATTN_ERR_ALIGN), (dict(o=A + 8), attn.ATTN_ERR_ALIGN),
    (dict(lse=A + 2), attn.ATTN_ERR_ALIGN), (dict(workspace=A + 16), attn.ATTN_ERR_ALIGN),
]


def call(clib, name, args, cache):
    ref = None if cache is None else ctypes.addressof(cache)
    return getattr(clib, name)(ref, *args.values())


@pytest.mark.parametrize("changes,code", CACHE_RULES)
def test_cache_rules(clib, changes, code):
    c = cache_struct(**changes)
    assert call(clib, "attn_cache_append", APPEND, c) == code
    assert call(clib, "attn_fwd_cache", FWD, c) == code


def test_null_cache(clib):
    assert call(clib, "attn_cache_append", APPEND, None) == attn.ATTN_ERR_INVALID
    assert call(clib, "attn_fwd_cache", FWD, None) == attn.ATTN_ERR_INVALID


@pytest.mark.parametrize("changes,code", APPEND_RULES)
def test_append_rules(clib, changes, code):
    assert call(clib, "attn_cache_append", {**APPEND, **changes}, cache_struct()) == code


@pytest.mark.parametrize("changes,code", FWD_RULES)
def test_fwd_rules(clib, changes, code):
    assert call(clib, "attn_fwd_cache", {**FWD, **changes}, cache_struct()) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_valid_calls_fail_only_for_want_of_a_device(clib):
    for c in (cache_struct(), cache_struct(type=0, k_scale=None, v_scale=None),
              cache_struct(head_stride=16 * 128, token_stride=128)):
        assert call(clib, "attn_cache_append", APPEND, c) == attn.ATTN_ERR_CUDA
        assert call(clib, "attn_fwd_cache", FWD, c) == attn.ATTN_ERR_CUDA
    assert call(clib, "attn_cache_append",
                {**APPEND, **dict(q=None, q_out=None, q_stride=0, inv_freq=None, rotary_dim=0,
                                  total=6, cu_seqlens=None)}, cache_struct()) == attn.ATTN_ERR_CUDA
    assert clib.attn_fwd_cache_workspace_bytes(4, 2, 1) == 0


def test_workspace_of_bad_sizes(clib):
    for args in ((0, 1, 1), (4, 0, 1), (5, 2, 1), (4, 2, 0)):
        assert clib.attn_fwd_cache_workspace_bytes(*args) == 0


# ------------------------------------------------------------------ binding
@pytest.fixture
def lib(monkeypatch):
    import contextlib
    fake = FakeLib({"attn_fwd_cache_workspace_bytes": 4096})
    monkeypatch.setattr(attn, "load_library", lambda path=None: fake)
    monkeypatch.setattr(attn, "_on_device", lambda dev: contextlib.nullcontext())
    return fake


def i32(*values, index=0):
    return FakeCuda(torch.tensor(values, dtype=torch.int32), index)


def fp8(*shape, index=0):
    return FakeCuda(torch.zeros(shape, dtype=torch.float8_e4m3fn), index)


def pool(index=0):
    return fp8(6, 16, 2, 128, index=index), fp8(6, 16, 2, 128, index=index), \
        f32(6, 2, index=index), f32(6, 2, index=index)


def table(index=0):
    return FakeCuda(torch.zeros(3, 4, dtype=torch.int32), index)


def test_handle_fields():
    k, v, ks, vs = pool()
    s = attn.KVCache(k, v, ks, vs)._struct
    assert (s.k_pages, s.v_pages, s.k_scale, s.v_scale) == (k.data_ptr(), v.data_ptr(),
                                                            ks.data_ptr(), vs.data_ptr())
    assert (s.page_stride, s.token_stride, s.head_stride) == (16 * 256, 256, 128)
    assert (s.num_pages, s.page_size, s.h_kv, s.d, s.type) == (6, 16, 2, 128, 1)
    # heads before tokens, a BF16 slice of a wider pool
    w = torch.zeros(6, 2, 3, 16, 128, dtype=torch.bfloat16)
    views = [FakeCuda(w[:, i].permute(0, 2, 1, 3)) for i in range(2)]
    s = attn.KVCache(*views)._struct
    assert (s.page_stride, s.token_stride, s.head_stride) == (2 * 3 * 2048, 128, 2048)
    assert (s.k_scale, s.v_scale, s.h_kv, s.type) == (None, None, 3, 0)
    # a dimension of one has no stride
    one = [FakeCuda(torch.zeros(1, 8, 1, 128, dtype=torch.bfloat16).as_strided((1, 8, 1, 128),
                                                                               (7, 128, 3, 1)))
           for _ in range(2)]
    s = attn.KVCache(*one)._struct
    assert (s.page_stride, s.token_stride, s.head_stride) == (128, 128, 128)


@pytest.mark.parametrize("change", [
    lambda k, v, ks, vs: (k, bf16(6, 16, 2, 128), ks, vs),
    lambda k, v, ks, vs: (f32(6, 16, 2, 128), f32(6, 16, 2, 128), ks, vs),
    lambda k, v, ks, vs: (fp8(6, 16, 2, 64), fp8(6, 16, 2, 64), ks, vs),
    lambda k, v, ks, vs: (k, fp8(6, 16, 3, 128), ks, vs),
    lambda k, v, ks, vs: (k, FakeCuda(torch.zeros(6, 2, 16, 128).to(
        torch.float8_e4m3fn).permute(0, 2, 1, 3)), ks, vs),
    lambda k, v, ks, vs: (k, v, None, vs), lambda k, v, ks, vs: (k, v, ks, None),
    lambda k, v, ks, vs: (bf16(6, 16, 2, 128), bf16(6, 16, 2, 128), ks, vs),
    lambda k, v, ks, vs: (k, v, f32(6, 3), vs), lambda k, v, ks, vs: (k, v, ks, f32(6, 2, index=1)),
    lambda k, v, ks, vs: (k, fp8(6, 16, 2, 128, index=1), ks, vs),
    lambda k, v, ks, vs: (k, v, ks, FakeCuda(torch.zeros(6, 2, dtype=torch.float16))),
    lambda k, v, ks, vs: (k._t, v._t, ks._t, vs._t),
    lambda k, v, ks, vs: (fp8(0, 16, 2, 128), fp8(0, 16, 2, 128), f32(0, 2), f32(0, 2)),
])
def test_handle_refuses(change):
    with pytest.raises((ValueError, TypeError)):
        attn.KVCache(*change(*pool()))


def test_append_arguments(lib):
    cache = attn.KVCache(*pool())
    qkv = torch.zeros(7, 8, 128, dtype=torch.bfloat16)
    q, k, v = FakeCuda(qkv[:, :4]), FakeCuda(qkv[:, 4:6]), FakeCuda(qkv[:, 6:])
    t, sl, cu, inv = table(), i32(5, 6, 7), i32(0, 2, 4, 7), f32(32)
    out = bf16(7, 4, 128)
    got = attn.attn_cache_append(cache, k, v, t, sl, cu_seqlens=cu, max_seqlen=3, q=q, q_out=out,
                                 inv_freq=inv, interleaved=True, stream=STREAM)
    assert got is out
    want = dict(cache=cache._ref, k=k.data_ptr(), v=v.data_ptr(), q=q.data_ptr(),
                q_out=out.data_ptr(), page_table=t.data_ptr(), seqlens_k=sl.data_ptr(),
                cu_seqlens=cu.data_ptr(), inv_freq=inv.data_ptr(), batch=3, max_pages=4, total=7,
                max_seqlen=3, h_q=4, k_stride=1024, v_stride=1024, q_stride=1024, rotary_dim=64,
                interleaved=1, stream=STREAM)
    check_call(lib, "attn_cache_append", **want)
    assert attn.attn_cache_append(cache, k, v, t, sl, cu_seqlens=cu, stream=STREAM) is None
    check_call(lib, "attn_cache_append", **{**want, **dict(
        q=None, q_out=None, inv_freq=None, max_seqlen=7, h_q=2, q_stride=0, rotary_dim=0,
        interleaved=0)})


def test_fwd_arguments(lib):
    cache = attn.KVCache(*pool())
    q, t, sl, cu = bf16(7, 4, 128), table(), i32(5, 6, 7), i32(0, 2, 4, 7)
    o, lse, ws = bf16(7, 4, 128), f32(4, 7), u8(8192)
    assert attn.attn_fwd_cache(q, cache, t, sl, cu_seqlens_q=cu, max_seqlen_q=3, window_left=9,
                               scale=0.25, o=o, lse=lse, workspace=ws,
                               stream=STREAM) == (o, lse)
    want = dict(cache=cache._ref, q=q.data_ptr(), o=o.data_ptr(), lse=lse.data_ptr(),
                page_table=t.data_ptr(), seqlens_k=sl.data_ptr(), cu_seqlens_q=cu.data_ptr(),
                batch=3, max_pages=4, total_q=7, max_seqlen_q=3, h_q=4, q_stride=512, causal=1,
                window_left=9, scale=0.25, workspace=ws.data_ptr(), workspace_bytes=8192,
                stream=STREAM)
    check_call(lib, "attn_fwd_cache", **want)
    attn.attn_fwd_cache(q, cache, t, sl, cu_seqlens_q=cu, causal=False, o=o, lse=lse, workspace=ws,
                        stream=STREAM)
    check_call(lib, "attn_fwd_cache", **{**want, **dict(max_seqlen_q=7, window_left=-1, causal=0,
                                                        scale=1 / math.sqrt(128))})


def append_args(**changes):
    a = dict(k=bf16(6, 2, 128), v=bf16(6, 2, 128), page_table=table(), seqlens_k=i32(5, 6, 7),
             q=bf16(6, 4, 128), q_out=bf16(6, 4, 128), inv_freq=f32(32), stream=STREAM)
    a.update(changes)
    return a


@pytest.mark.parametrize("changes", [
    dict(k=f32(6, 2, 128)), dict(k=bf16(6, 3, 128)), dict(k=bf16(6, 2, 64)),
    dict(v=bf16(5, 2, 128)), dict(v=bf16(6, 2, 128, index=1)), dict(q=bf16(5, 4, 128)),
    dict(q=None), dict(q_out=bf16(6, 2, 128)), dict(q_out=f32(6, 4, 128)),
    dict(k=FakeCuda(torch.zeros(6, 128, 2, dtype=torch.bfloat16).transpose(1, 2))),
    dict(k=FakeCuda(torch.zeros(2, 6, 128, dtype=torch.bfloat16).transpose(0, 1))),
    dict(page_table=FakeCuda(torch.zeros(3, 4))), dict(page_table=i32(1, 2, 3)),
    dict(page_table=FakeCuda(torch.zeros(3, 8, dtype=torch.int32)[:, ::2])),
    dict(seqlens_k=i32(1, 2)), dict(seqlens_k=FakeCuda(torch.zeros(3, dtype=torch.int64))),
    dict(cu_seqlens=i32(0, 3, 6)), dict(inv_freq=FakeCuda(torch.zeros(32, dtype=torch.float64))),
    dict(inv_freq=f32(4, 8)), dict(inv_freq=f32(32, index=1)),
])
def test_append_refuses(lib, changes):
    with pytest.raises((ValueError, TypeError)):
        attn.attn_cache_append(attn.KVCache(*pool()), **append_args(**changes))
    assert not lib.calls


def test_cache_of_another_device(lib):
    with pytest.raises(ValueError, match="cache"):
        attn.attn_cache_append(attn.KVCache(*pool(1)), **append_args())
    with pytest.raises(ValueError, match="cache"):
        attn.attn_fwd_cache(bf16(3, 4, 128), attn.KVCache(*pool(1)), table(), i32(1, 2, 3))


@pytest.mark.parametrize("changes", [
    dict(q=f32(6, 4, 128)), dict(q=bf16(6, 4, 64)), dict(o=bf16(6, 2, 128)),
    dict(lse=f32(6, 4)), dict(cu_seqlens_q=i32(0, 1)), dict(workspace=u8(64, index=1)),
    dict(seqlens_k=i32(1, 2, 3, index=1)),
])
def test_fwd_refuses(lib, changes):
    args = dict(q=bf16(6, 4, 128), page_table=table(), seqlens_k=i32(5, 6, 7), o=bf16(6, 4, 128),
                lse=f32(4, 6), workspace=u8(4096), stream=STREAM)
    args.update(changes)
    with pytest.raises((ValueError, TypeError)):
        attn.attn_fwd_cache(args.pop("q"), attn.KVCache(*pool()), **args)
    assert all(name == "attn_fwd_cache_workspace_bytes" for name, _ in lib.calls)


def test_an_empty_batch_launches_nothing(lib):
    cache = attn.KVCache(*pool())
    t, sl = FakeCuda(torch.zeros(0, 4, dtype=torch.int32)), i32()
    o, lse = bf16(0, 4, 128), f32(4, 0)
    assert attn.attn_fwd_cache(bf16(0, 4, 128), cache, t, sl, o=o, lse=lse,
                               stream=STREAM) == (o, lse)
    assert attn.attn_cache_append(cache, bf16(0, 2, 128), bf16(0, 2, 128), t, sl, q=bf16(0, 4, 128),
                                  q_out=o, stream=STREAM) is o
    assert not lib.calls
