"""The score and cache calls captured next to nodes that are no kernels (copies
from and to the host, memsets) and where branches fork and join: they start
early only behind a kernel, and wait for everything before them."""
import pytest
import torch

from attention_forward_gb300 import fa

pytestmark = pytest.mark.gpu
B, H, Hkv, D, L, PAGE = 2, 8, 2, 128, 1500, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16()


class Server:
    """Buffers of a decode step over a cache, and a prompt's attention."""

    def __init__(self):
        per = -(-(L + 8) // PAGE)
        self.cache = fa.fa_cache_empty(B * per, Hkv, PAGE, D)
        self.table = torch.arange(B * per, dtype=torch.int32, device="cuda").flip(0).view(B, per).contiguous()
        self.length = torch.tensor([L, 700], dtype=torch.int32, device="cuda")
        k, v = rand(1, B, Hkv, L, D).cuda(), rand(2, B, Hkv, L, D).cuda()
        fa.fa_cache_write(k, v, self.cache, self.table)
        self.host = [torch.empty((B, n, 1, D), dtype=torch.bfloat16, pin_memory=True) for n in (H, Hkv, Hkv)]
        self.q, self.k, self.v = (torch.empty_like(t, device="cuda") for t in self.host)
        self.o, self.lse = torch.zeros_like(self.q), torch.zeros((B, H, 1), device="cuda")
        self.back = torch.zeros((B, H, 1, D), dtype=torch.bfloat16, pin_memory=True)
        self.part = [torch.zeros((B, Hkv, L, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.qp = rand(3, B, H, 40, D).cuda()
        self.op, self.lp = torch.zeros_like(self.qp), torch.zeros((B, H, 40), device="cuda")
        self.ids = torch.arange(L, device="cuda").div(200, rounding_mode="floor").int().expand(B, L).contiguous()
        self.dq = self.ids[:, L - 40:].contiguous()
        torch.cuda.synchronize()

    def inputs(self, seed):
        for n, t in enumerate(self.host):
            t.copy_(rand(10 * seed + n, *t.shape))

    def step(self):
        """Copies in, a token written, attention, the result copied out."""
        for d, h in zip((self.q, self.k, self.v), self.host):
            d.copy_(h, non_blocking=True)
        fa.fa_cache_write(self.k, self.v, self.cache, self.table, start=self.length)
        self.length.add_(1)
        fa.fa_fwd_cache(self.q, self.cache, self.table, self.length, softcap=30.0, out=self.o, lse=self.lse)
        self.back.copy_(self.o, non_blocking=True)

    def read_and_attend(self, side=None):
        """A memset, the cache read back, and attention over it with documents;
        the values read on another branch than the decode's attention."""
        main = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(main)
        with torch.cuda.stream(side or main):
            for t in self.part:
                t.zero_()
            fa.fa_cache_read(self.cache, self.table, out=self.part)
            fa.fa_fwd_score(self.qp, *self.part, causal=True, softcap=20.0, doc_q=self.dq, doc_k=self.ids,
                            out=self.op, lse=self.lp)
        fa.fa_fwd_cache(self.q, self.cache, self.table, self.length, out=self.o, lse=self.lse)
        if side is not None:
            main.wait_stream(side)
        # behind both branches: the key split's merge reads what they leave
        fa.fa_fwd_score(self.qp[:1], self.part[0][:1], self.part[1][:1], out=self.op[:1], lse=self.lp[:1])

    def outputs(self):
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_OK
        return [t.clone() for t in (self.o, self.lse, self.back, self.op, self.lp, *self.part,
                                    *self.cache, self.length)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.is_floating_point() else x,
                           y.view(torch.uint8) if y.is_floating_point() else y) for x, y in zip(a, b))


def test_copies_and_memsets_between_captured_calls():
    direct, replayed = Server(), Server()
    for s in (direct, replayed):
        s.inputs(0)
        s.step()
    assert same(direct.outputs(), replayed.outputs())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.step()
    for n in range(1, 6):
        direct.inputs(n)
        direct.step()
        replayed.inputs(n)
        graph.replay()
        assert same(direct.outputs(), replayed.outputs())


def test_branches_that_fork_and_join_in_a_capture():
    direct, replayed = Server(), Server()
    side = torch.cuda.Stream()
    for s in (direct, replayed):
        s.inputs(7)
        s.step()
        s.read_and_attend()
    want = direct.outputs()
    assert same(want, replayed.outputs())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.read_and_attend(side)
    for _ in range(5):
        for t in (replayed.op, replayed.lp, replayed.o, replayed.lse):
            t.zero_()
        graph.replay()
        assert same(want, replayed.outputs())
