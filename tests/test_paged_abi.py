"""Refusals of the paged cache's calls and of acceptance by sampling (host checks: nothing
is launched)."""
import ctypes

import pytest
import torch

import lossless_kv_compressed_b200 as vc
from lossless_kv_compressed_b200 import _lib

A = 1 << 20                                     # an aligned address that is never read
BAD, UNS = _lib.VC_ERR_INVALID, _lib.VC_ERR_UNSUPPORTED


def cache(**kw):
    c = _lib.PagedCacheStruct()
    c.type, c.B, c.Hkv, c.D, c.page, c.n_pages, c.max_pages = 0, 2, 2, 128, 64, 10, 4
    c.k = c.v = c.page_table = c.kv_len = A
    c.k_page_stride = c.v_page_stride = 2 * 64 * 128
    c.k_head_stride = c.v_head_stride = 64 * 128
    c.k_row_stride = c.v_row_stride = 128
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(type=3), BAD), (dict(type=-1), BAD), (dict(B=0), BAD), (dict(Hkv=0), BAD),
    (dict(n_pages=0), BAD), (dict(max_pages=0), BAD), (dict(D=96), UNS), (dict(D=256), UNS),
    (dict(page=8), UNS), (dict(page=48), UNS), (dict(page=512), UNS), (dict(B=70000), UNS),
    (dict(n_pages=1 << 25), UNS), (dict(max_pages=1 << 25), UNS), (dict(k=None), BAD),
    (dict(v=None), BAD), (dict(page_table=None), BAD), (dict(kv_len=None), BAD),
    (dict(k=A + 8), BAD), (dict(k_row_stride=0), BAD), (dict(v_head_stride=-128), BAD),
    (dict(k_page_stride=100), BAD), (dict(v_row_stride=4), BAD), (dict(type=1), BAD),
    (dict(type=2, k_scale=A), BAD), (dict(type=1, k_scale=A, v_scale=A + 4), BAD),
    (dict(type=1, k_scale=A, v_scale=A, k_row_stride=8), BAD),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(kw, status):
    L, c = vc.lib(), ctypes.byref(cache(**kw))
    assert L.vc_paged_write(c, A, 256, 128, A, 256, 128, 4, None, None) == status
    assert L.vc_last_error()
    assert L.vc_paged_read(c, 0, None, A, A, 8, None) == status
    assert L.vc_paged_attn(c, A, 1024, 128, 4, 8, None, 0, 0.0, 0, A, None, A, 1 << 40, None) == status
    assert L.vc_paged_attn_workspace_size(c, 4, 8, 0) == 0


def test_null_cache():
    L = vc.lib()
    assert L.vc_paged_write(None, A, 256, 128, A, 256, 128, 4, None, None) == BAD
    assert L.vc_paged_attn_workspace_size(None, 4, 8, 0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(N=3), BAD), (dict(N=-2), BAD), (dict(k=None), BAD), (dict(v=A + 2), BAD),
    (dict(kt=255), BAD), (dict(vh=-128), BAD), (dict(N=1 << 30), UNS), (dict(N=0), 0)])
def test_write_refusals(kw, status):
    a = dict(k=A, kt=256, kh=128, v=A, vt=256, vh=128, N=4)
    a.update(kw)
    assert vc.lib().vc_paged_write(ctypes.byref(cache()), *a.values(), None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(T=1 << 31), BAD), (dict(start=1 << 31), BAD), (dict(k=None), BAD),
    (dict(v=A + 8), BAD), (dict(T=0), 0)])
def test_read_refusals(kw, status):
    a = dict(start=0, starts=None, k=A, v=A, T=5)
    a.update(kw)
    assert vc.lib().vc_paged_read(ctypes.byref(cache()), *a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=7), BAD), (dict(Hq=0), BAD), (dict(N=3), BAD), (dict(N=-2), BAD), (dict(flags=1), BAD),
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(ws=None), BAD), (dict(q=A + 8), BAD),
    (dict(out=A + 4), BAD), (dict(ws=A + 1), BAD), (dict(qt=100), BAD), (dict(qh=-8), BAD),
    (dict(N=1 << 28), UNS), (dict(bytes=16), BAD), (dict(N=0), 0)])
def test_attention_refusals(kw, status):
    a = dict(q=A, qt=1024, qh=128, N=4, Hq=8, cu=None, max_q=0, scale=0.0, flags=0, out=A, lse=None,
             ws=A, bytes=1 << 40)
    a.update(kw)
    assert vc.lib().vc_paged_attn(ctypes.byref(cache()), *a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), BAD), (dict(n_q=0), BAD), (dict(V=0), BAD), (dict(B=70000), UNS),
    (dict(n_q=258), UNS), (dict(V=(1 << 31) - 1), UNS), (dict(flags=1), BAD), (dict(logits=None), BAD),
    (dict(u=None), BAD), (dict(commit=None), BAD), (dict(drafts=None), BAD), (dict(ws=None), BAD),
    (dict(logits=A + 4), BAD), (dict(ql=A + 4), BAD), (dict(ws=A + 8), BAD), (dict(bytes=8), BAD)])
def test_sample_refusals(kw, status):
    a = dict(logits=A, ql=None, drafts=A, u=A, T=None, n=None, B=2, n_q=3, V=100, flags=0, acc=A,
             commit=A, nc=A, err=None, ws=A, bytes=1 << 30)
    a.update(kw)
    assert vc.lib().vc_accept_sample(*a.values(), None) == status
    if status == UNS:
        assert vc.lib().vc_accept_sample_workspace_size(a["B"], a["n_q"], a["V"]) == 0


def test_python_checks():
    i32 = dict(dtype=torch.int32)
    pool, table, n = torch.zeros((2, 1, 16, 64)), torch.zeros((1, 1), **i32), torch.zeros(1, **i32)
    with pytest.raises(TypeError):
        vc.PagedCache(pool, pool, table, n)                     # float32 pages
    with pytest.raises(ValueError):
        vc.PagedCache(pool.bfloat16(), pool.bfloat16(), table, n)   # not on a GPU
    with pytest.raises(ValueError):
        vc.PagedCache(pool.bfloat16()[0], pool.bfloat16()[0], table, n)
    with pytest.raises(TypeError):
        vc.accept_sample(torch.zeros((1, 1, 5), dtype=torch.float64), None, torch.zeros((1, 1)))
    with pytest.raises(ValueError):
        vc.accept_sample_workspace_size(0, 1, 5)


@pytest.mark.parametrize("handle", [12345, 0])
def test_a_stream_given_as_a_number_is_one_of_the_calls_device(monkeypatch, handle):
    """A call's own tensors are made on that stream of the cache's device, not on a stream of the
    same number of the device that happens to be current."""
    from lossless_kv_compressed_b200 import api
    made = []

    class External:
        def __init__(self, ptr, device=None):
            self.cuda_stream, self.device = ptr, device

    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: made.append(s))
    api._on(handle, torch.device("cuda:1"))
    assert made[0].cuda_stream == handle and made[0].device == torch.device("cuda:1")
    own = External(7)
    api._on(own, torch.device("cuda:1"))
    assert made[1] is own


def test_sizes_past_32_bits_are_refused_not_wrapped():
    from lossless_kv_compressed_b200 import api
    big = 2 ** 32 + 4                                # 4 when taken modulo 2^32
    for sizes in ((big, 1, 5), (1, big, 5), (1, 1, big), (1, 1, 2 ** 31)):
        with pytest.raises(ValueError):
            vc.accept_sample_workspace_size(*sizes)
    cpu = torch.device("cpu")
    rows = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    assert api._new_rows(rows.expand(2 ** 31 - 1, 2, 64), "k", 64, cpu)[:2] == (2 ** 31 - 1, 2)
    with pytest.raises(ValueError):
        api._new_rows(rows.expand(big, 2, 64), "k", 64, cpu)
