"""fa_fwd from several host threads on one stream: each call's launches stay
together, and none grows the workspace that another is about to launch with."""
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


def make(B, H, Sq, Skv, D, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return n(B, H, Sq, D), n(B, H, Skv, D), n(B, H, Skv, D)


def test_threads_on_one_stream():
    # a decode, a larger one, and a prefill with split keys: workspaces of
    # growing size
    data = [make(1, 2, 1, 5000, 128, 1), make(4, 8, 1, 20000, 64, 2), make(1, 2, 200, 9000, 128, 3)]
    for q, k, v in data:
        assert fa.fa_workspace_bytes(*q.shape[:3], k.shape[2], q.shape[3]) > 0
    stream = torch.cuda.Stream()
    outputs = lambda q: (torch.empty_like(q), torch.empty(q.shape[:3], device="cuda"))  # noqa: E731
    want = []
    for q, k, v in data:
        want.append(outputs(q))
        fa.fa_fwd(q, k, v, out=want[-1][0], lse=want[-1][1])
    torch.cuda.synchronize()
    for _ in range(6):
        fa.fa_release_workspaces()
        outs = [[outputs(q) for _ in range(30)] for q, _, _ in data for _ in range(2)]
        torch.cuda.synchronize()
        errors, start = [], threading.Barrier(len(outs))

        def work(n):
            try:
                start.wait(60)
                for o, lse in outs[n]:
                    fa.fa_fwd(*data[n // 2], out=o, lse=lse, stream=stream)
            except Exception as e:  # noqa: BLE001
                errors.append(e)

        threads = [threading.Thread(target=work, args=(n,)) for n in range(len(outs))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not errors, errors
        assert fa.fa_get_device_status() == fa.FA_OK
        for n, rows in enumerate(outs):
            for o, lse in rows:
                assert torch.equal(o, want[n // 2][0]) and torch.equal(lse, want[n // 2][1])
    fa.fa_release_workspaces()
