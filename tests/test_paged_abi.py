"""Host-side argument checks of the paged-cache entry points: each refused call
returns CIDER_ERR_INVALID_ARG with a message before any device is touched, so
this runs without a GPU."""
import ctypes

import pytest
import torch

import w8a8_activation_quantized_b200 as cider

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from w8a8_activation_quantized_b200._build import build_library
    build_library()
    return cider.lib()


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _cache(**kw):
    a = dict(k=64 * MB, v=128 * MB, dt=0, num_pages=64, page_size=16, H_kv=8, D=128, stride_page=16384, stride_head=2048,
             stride_token=128)
    a.update(kw)
    return cider._CACHE.pack(*a.values())


def _attend(lib, cache=None, **kw):
    a = dict(q=MB, ld_q=4096, T=4, H_q=32, cu=2 * MB, kv=3 * MB, B=3, table=4 * MB, ld_table=8, width=8, max_fresh=2,
             window=0, sinks=0, scale=0.1, out=5 * MB, ld_out=4096, ws=256 * MB, wsb=64 * MB)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.cider_paged_attention(c, _p(a["q"]), a["ld_q"], a["T"], a["H_q"], _p(a["cu"]), _p(a["kv"]),
                                     a["B"], _p(a["table"]), a["ld_table"], a["width"], a["max_fresh"], a["window"],
                                     a["sinks"], a["scale"], _p(a["out"]), a["ld_out"], _p(a["ws"]), a["wsb"], None)


BAD_CACHES = [dict(k=0), dict(v=0), dict(k=64 * MB + 8), dict(dt=2), dict(num_pages=0), dict(page_size=8), dict(page_size=48),
              dict(page_size=512), dict(num_pages=1 << 27), dict(H_kv=0), dict(D=96), dict(D=256), dict(stride_token=64),
              dict(stride_head=2052), dict(stride_page=2048), dict(stride_head=128), dict(stride_page=1 << 37),
              dict(stride_token=-128)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches_are_refused(lib, kw):
    assert _attend(lib, _cache(**kw)) == 1
    assert lib.cider_last_error()
    c = _cache(**kw)
    assert lib.cider_paged_append(c, _p(MB), 1024, _p(2 * MB), 1024, _p(3 * MB), 4, None) == 1


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(cu=None), dict(kv=None), dict(table=None), dict(ws=None), dict(q=MB + 2),
    dict(out=5 * MB + 8), dict(ws=256 * MB + 8), dict(cu=2 * MB + 2), dict(T=-1), dict(T=(1 << 28) + 1), dict(H_q=30),
    dict(H_q=0), dict(B=0), dict(B=4097), dict(ld_q=4088), dict(ld_q=4100), dict(ld_out=128), dict(width=0),
    dict(width=9), dict(width=(1 << 26) + 1, ld_table=1 << 27), dict(max_fresh=-1), dict(window=-1), dict(sinks=-1),
    dict(window=1 << 30), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_bad_attention_arguments_are_refused(lib, kw):
    assert _attend(lib, **kw) == 1
    assert lib.cider_last_error()
    if lib.cider_is_available():
        return
    assert _attend(lib) in (2, 3)  # good arguments get as far as the device


def test_token_major_and_degenerate_strides_are_taken(lib):
    if lib.cider_is_available():
        pytest.skip("a GPU is present: the call would be launched")
    assert _attend(lib, _cache(stride_token=1024, stride_head=128)) in (2, 3)
    assert _attend(lib, _cache(H_kv=1, stride_head=7, stride_page=2048), H_q=4, ld_q=512, ld_out=512) in (2, 3)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(ld_k=1016), dict(ld_v=1020), dict(k=None), dict(slots=None), dict(k=MB + 2),
                                dict(slots=3 * MB + 1), dict(k=64 * MB + 4096), dict(slots=128 * MB)])
def test_bad_append_arguments_are_refused(lib, kw):
    a = dict(k=MB, ld_k=1024, v=2 * MB, ld_v=1024, slots=3 * MB, T=4)
    a.update(kw)
    c = _cache()
    assert lib.cider_paged_append(c, _p(a["k"]), a["ld_k"], _p(a["v"]), a["ld_v"], _p(a["slots"]), a["T"],
                                  None) == 1
    assert lib.cider_last_error()


def test_append_refuses_one_buffer_for_k_and_v_and_takes_no_rows(lib):
    c = _cache(v=64 * MB)
    assert lib.cider_paged_append(c, _p(MB), 1024, _p(2 * MB), 1024, _p(3 * MB), 4, None) == 1
    c = _cache()
    assert lib.cider_paged_append(c, None, 0, None, 0, None, 0, None) == 0
    assert _attend(lib, T=0, q=None, out=None) == 0


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(B=4097), dict(num_free=-1), dict(num_pages=0), dict(page_size=20), dict(width=0), dict(ld_table=7),
    dict(rows=-1), dict(cached=None), dict(fresh=None), dict(free=None), dict(table=None), dict(cu=None), dict(kv=None),
    dict(slots=None), dict(taken=None), dict(cu=MB), dict(kv=6 * MB), dict(slots=4 * MB + 64), dict(taken=2 * MB),
    dict(cached=MB + 2), dict(taken=8 * MB + 1)])
def test_bad_tables_arguments_are_refused(lib, kw):
    a = dict(cached=MB, fresh=2 * MB, B=3, free=3 * MB, num_free=9, num_pages=64, page_size=16, table=4 * MB, ld_table=8,
             width=8, cu=5 * MB, kv=6 * MB, slots=7 * MB, rows=20, taken=8 * MB)
    if kw == dict(kv=6 * MB):
        kw = dict(kv=5 * MB + 4)  # inside cu_fresh
    a.update(kw)

    def call():
        return lib.cider_paged_tables(_p(a["cached"]), _p(a["fresh"]), a["B"], _p(a["free"]), a["num_free"], a["num_pages"],
                                      a["page_size"], _p(a["table"]), a["ld_table"], a["width"], _p(a["cu"]), _p(a["kv"]),
                                      _p(a["slots"]), a["rows"], _p(a["taken"]), None)
    assert call() == 1
    assert lib.cider_last_error()


def test_the_kernel_switch_is_checked(lib):
    assert lib.cider_test_set_paged_kernel(3) == 1 and lib.cider_test_set_paged_kernel(-1) == 1
    assert lib.cider_test_set_paged_kernel(0) == 0


def test_the_binding_refuses_what_the_abi_cannot_see():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    q = torch.zeros((3, 4, 64), dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    cases = [
        lambda: cider.cider_paged_attention(q, k, k[:2], t, i, i[:2]),                                # cache shapes
        lambda: cider.cider_paged_attention(q, k, k.bfloat16(), t, i, i[:2]),                         # cache dtypes
        lambda: cider.cider_paged_attention(q.bfloat16(), k, k, t, i, i[:2]),                         # q's dtype
        lambda: cider.cider_paged_attention(q[:, :, :32], k, k, t, i, i[:2]),                         # q's D
        lambda: cider.cider_paged_attention(q.transpose(0, 1), k, k, t, i, i[:2]),                    # q's rows not dense
        lambda: cider.cider_paged_attention(q, k, k, t.long(), i, i[:2]),                             # table dtype
        lambda: cider.cider_paged_attention(q, k, k, t[:1], i, i[:2]),                                # table rows
        lambda: cider.cider_paged_attention(q, k, k, t, i[:2], i[:2]),                                # cu_fresh length
        lambda: cider.cider_paged_attention(q, k, k, t, i.long(), i[:2]),                             # cu_fresh dtype
        lambda: cider.cider_paged_attention(q, k, k, t, i, i[:2], out=q[:2]),                         # out's shape
        lambda: cider.cider_paged_append(q, q, k, k.clone(), i),                                      # heads
        lambda: cider.cider_paged_append(q[:, :2], q[:, 2:], k, k.clone(), i[:2]),                    # rows
        lambda: cider.cider_paged_tables(i, i[:2], i, t, 16, 4, 3),                                   # lengths
        lambda: cider.cider_paged_tables(i[:2], i[:2], i.long(), t, 16, 4, 3),                        # free_pages dtype
    ]
    for n, c in enumerate(cases):
        with pytest.raises(ValueError):
            c()
            pytest.fail(f"case {n} was taken")


def test_a_scale_that_overflows_in_base_two_is_refused(lib):
    assert _attend(lib, scale=3.0e38) == 1  # finite, but 3e38 log2(e) is not
    assert b"log2" in lib.cider_last_error()
