"""First calls of host threads: a thread that has not used the GPU yet leaves
what the library keeps for the device as it is."""
import threading

import pytest
import torch

from attention_forward_gb300 import fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def make(B, H, Hkv, Sq, Skv, D, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return n(B, H, Sq, D), n(B, Hkv, Skv, D), n(B, Hkv, Skv, D)


def calls():
    """(call of (out, lse, stream), query): split keys, the cache's parts, and
    kernels of fa_fwd that take a scheduler slot or the static scratch."""
    a = make(1, 4, 1, 3, 5000, 128, 1)
    b = make(1, 2, 2, 1, 9000, 128, 2)
    c = make(2, 8, 8, 600, 600, 64, 3)
    Hkv, page, L = 2, 64, 6000
    per = -(-L // page)
    cache = fa.fa_cache_empty(per, Hkv, page, 128)
    table = torch.arange(per, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    k, v = make(1, 1, Hkv, 1, L, 128, 4)[1:]
    fa.fa_cache_write(k, v, cache, table)
    q = make(1, 16, 1, 1, 1, 128, 5)[0]
    length = torch.tensor([L], dtype=torch.int32, device="cuda")
    return [
        (lambda o, l, s: fa.fa_fwd_score(*a, causal=True, out=o, lse=l, stream=s), a[0]),
        (lambda o, l, s: fa.fa_fwd_cache(q, cache, table, length, out=o, lse=l, stream=s), q),
        (lambda o, l, s: fa.fa_fwd(*b, out=o, lse=l, stream=s), b[0]),
        (lambda o, l, s: fa.fa_fwd(*c, causal=True, out=o, lse=l, stream=s), c[0]),
    ]


def outputs(q):
    return torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")


def reference(todo):
    want = []
    for f, q in todo:
        want.append(outputs(q))
        f(*want[-1], None)
    torch.cuda.synchronize()
    return want


def test_threads_one_after_the_other_share_the_streams_memory():
    """A workspace of 19 MB stays where it is, whoever calls."""
    fa.fa_release_workspaces()
    q, k, v = make(1, 16, 16, 256, 16384, 128, 6)
    assert fa.fa_score_workspace_bytes(1, 16, 16, 256, 16384, 128) > 1 << 24
    stream = torch.cuda.Stream()
    want, got = outputs(q), outputs(q)
    torch.cuda.synchronize()
    fa.fa_fwd_score(q, k, v, out=want[0], lse=want[1], stream=stream)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]

    def work():
        fa.fa_fwd_score(q, k, v, out=got[0], lse=got[1], stream=stream)

    for _ in range(12):
        got[0].zero_()
        torch.cuda.synchronize()
        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # less than one workspace: a thread's own resources are small
    assert free - torch.cuda.mem_get_info()[0] < 1 << 24
    fa.fa_release_workspaces()


def test_many_threads_first_calls_at_once():
    todo = calls()
    want = reference(todo)
    streams = [torch.cuda.Stream() for _ in range(12)]
    for _ in range(25):
        outs = [[outputs(q) for _, q in todo] for _ in streams]
        torch.cuda.synchronize()
        errors, start = [], threading.Barrier(len(streams))

        def work(n):
            try:
                start.wait(60)
                for i in range(len(todo)):
                    i = (i + n) % len(todo)
                    todo[i][0](*outs[n][i], streams[n])
            except Exception as e:  # noqa: BLE001
                errors.append(e)

        threads = [threading.Thread(target=work, args=(n,)) for n in range(len(streams))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not errors, errors
        assert fa.fa_get_device_status() == fa.FA_OK
        for n in range(len(streams)):
            for i, w in enumerate(want):
                assert torch.equal(outs[n][i][0], w[0]) and torch.equal(outs[n][i][1], w[1]), i
    fa.fa_release_workspaces()
