"""Calls without a workspace of their own on streams that share a handle: every
thread's per-thread default stream, and streams made where others were
destroyed."""
import ctypes
import threading

import pytest
import torch

from attention_forward_gb300 import fa

pytestmark = pytest.mark.gpu
PER_THREAD = 2  # cudaStreamPerThread


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def make(B, H, Hkv, Sq, Skv, D, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return n(B, H, Sq, D), n(B, Hkv, Skv, D), n(B, Hkv, Skv, D)


def outputs(q, n):
    return [(torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float32, device="cuda"))
            for _ in range(n)]


def calls():
    """(function of (out, lse, stream), query) of calls that need a workspace."""
    a = make(1, 4, 1, 3, 5000, 128, 1)      # key ranges, merged
    b = make(1, 8, 8, 500, 900, 64, 2)      # documents
    ids = torch.arange(900, device="cuda").div(150, rounding_mode="floor").int()[None].contiguous()
    dq = ids[:, 400:].contiguous()
    Hkv, page, L = 2, 64, 6000
    per = -(-L // page)
    cache = fa.fa_cache_empty(per, Hkv, page, 128)
    table = torch.arange(per, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    k, v = make(1, 1, Hkv, 1, L, 128, 3)[1:]
    fa.fa_cache_write(k, v, cache, table)
    q = make(1, 16, 1, 1, 1, 128, 4)[0]
    length = torch.tensor([L], dtype=torch.int32, device="cuda")
    c = make(1, 2, 2, 1, 9000, 128, 5)      # fa_fwd: decode, split
    return [
        (lambda o, l, s: fa.fa_fwd_score(*a, causal=True, out=o, lse=l, stream=s), a[0]),
        (lambda o, l, s: fa.fa_fwd_score(*b, causal=True, doc_q=dq, doc_k=ids, out=o, lse=l,
                                         stream=s), b[0]),
        (lambda o, l, s: fa.fa_fwd_cache(q, cache, table, length, out=o, lse=l, stream=s), q),
        (lambda o, l, s: fa.fa_fwd(*c, out=o, lse=l, stream=s), c[0]),
    ]


def same(got, want):
    return torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_threads_on_their_per_thread_streams():
    todo = calls()
    want = []
    for f, q in todo:
        (o, l), = outputs(q, 1)
        f(o, l, None)
        want.append((o, l))
    torch.cuda.synchronize()
    n, threads_per_call = 60, 2
    jobs = [(i, outputs(todo[i][1], n)) for i in range(len(todo)) for _ in range(threads_per_call)]
    torch.cuda.synchronize()
    errors = []
    start = threading.Barrier(len(jobs))

    def work(i, outs):
        try:
            start.wait(60)
            for o, l in outs:
                todo[i][0](o, l, PER_THREAD)
            torch.cuda.ExternalStream(PER_THREAD).synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert fa.fa_get_device_status() == fa.FA_OK
    for i, outs in jobs:
        for got in outs:
            assert same(got, want[i]), f"call {i}"
    fa.fa_release_workspaces()


def test_a_new_stream_where_another_was_destroyed():
    """Its handle may be the old one's: its work does not share the old one's
    memory."""
    rt = torch.cuda.cudart()
    todo = calls()
    want = []
    for f, q in todo:
        (o, l), = outputs(q, 1)
        f(o, l, None)
        want.append((o, l))
    torch.cuda.synchronize()
    outs = [outputs(q, 24) for _, q in todo]
    torch.cuda.synchronize()
    fa.fa_release_workspaces()
    for n in range(24):
        handle = ctypes.c_void_p()
        assert int(rt.cudaStreamCreate(ctypes.addressof(handle))) == 0
        for i, (f, _) in enumerate(todo):
            f(*outs[i][n], handle.value)
        assert int(rt.cudaStreamDestroy(handle.value)) == 0  # its work may still run
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    for i in range(len(todo)):
        for got in outs[i]:
            assert same(got, want[i]), f"call {i}"
    fa.fa_release_workspaces()
