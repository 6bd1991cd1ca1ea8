"""The calls on 16-bit pages and latent rows captured next to nodes that are no kernels
(copies from and to the host, memsets) and where branches fork and join: they start
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
    """Buffers of a decode step over a cache of keys and values and one of latent rows,
    and of a prompt's expanded attention."""

    def __init__(self):
        per = -(-(L + 8) // PAGE)
        self.cache = fa.fa_paged_empty(B * per, Hkv, PAGE, D)
        self.pages = fa.fa_latent_empty(B * per, PAGE)
        self.table = torch.arange(B * per, dtype=torch.int32, device="cuda").flip(0).view(B, per).contiguous()
        self.length = torch.tensor([L, 700], dtype=torch.int32, device="cuda")
        self.freqs = [torch.linspace(0.001, 1, n, device="cuda") for n in (D // 2, 32)]
        fa.fa_paged_write(rand(1, B, Hkv, L, D).cuda(), rand(2, B, Hkv, L, D).cuda(), self.cache, self.table)
        fa.fa_latent_write(rand(3, B, L, 512).cuda(), rand(4, B, L, 64).cuda(), self.pages, self.table)
        shapes = [(B, H, 1, D), (B, Hkv, 1, D), (B, Hkv, 1, D), (B, 1, 512), (B, 1, 64), (B, H, 1, 64)]
        self.host = [torch.empty(s, dtype=torch.bfloat16, pin_memory=True) for s in shapes]
        self.new = [torch.empty_like(t, device="cuda") for t in self.host]
        self.qr = torch.zeros((B, H, 1, D), dtype=torch.bfloat16, device="cuda")
        self.ql = rand(5, B, H, 1, 576).cuda()
        self.o, self.lse = torch.zeros_like(self.qr), torch.zeros((B, H, 1), device="cuda")
        self.ol = torch.zeros((B, H, 1, 512), dtype=torch.bfloat16, device="cuda")
        self.ll = torch.zeros_like(self.lse)
        self.back = torch.zeros((B, H, 1, 512), dtype=torch.bfloat16, pin_memory=True)
        self.part = [torch.zeros((B, L, n), dtype=torch.bfloat16, device="cuda") for n in (512, 64)]
        self.qe, self.kv = rand(6, B, H, 40, 192).cuda(), rand(7, B, H, L, 256).cuda()
        self.oe = torch.zeros((B, H, 40, 128), dtype=torch.bfloat16, device="cuda")
        self.le = torch.zeros((B, H, 40), device="cuda")
        torch.cuda.synchronize()

    def inputs(self, seed):
        for n, t in enumerate(self.host):
            t.copy_(rand(10 * seed + n, *t.shape))

    def step(self):
        """Copies in, a token written to both caches, attention over them, a result out."""
        for d, h in zip(self.new, self.host):
            d.copy_(h, non_blocking=True)
        q, k, v, c, r, qr = self.new
        fa.fa_paged_write(k, v, self.cache, self.table, self.length, freqs=self.freqs[0], q=q, q_out=self.qr)
        fa.fa_latent_write(c, r, self.pages, self.table, self.length, freqs=self.freqs[1], q_rope=qr, q=self.ql)
        self.length.add_(1)
        fa.fa_fwd_paged(self.qr, self.cache, self.table, self.length, out=self.o, lse=self.lse)
        fa.fa_fwd_latent(self.ql, self.pages, self.table, self.length, out=self.ol, lse=self.ll)
        self.back.copy_(self.ol, non_blocking=True)

    def read_and_attend(self, side=None):
        """A memset, the latent cache read back and expanded attention with what was read,
        on another branch than the decode's attention."""
        main = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(main)
        with torch.cuda.stream(side or main):
            for t in self.part:
                t.zero_()
            fa.fa_latent_read(self.pages, self.table, out=self.part)
            fa.fa_fwd_expanded(self.qe, self.kv, self.part[1], causal=True, out=self.oe, lse=self.le)
        fa.fa_fwd_paged(self.qr, self.cache, self.table, self.length, out=self.o, lse=self.lse)
        fa.fa_fwd_latent(self.ql, self.pages, self.table, self.length, out=self.ol, lse=self.ll)
        if side is not None:
            main.wait_stream(side)
        # behind both branches
        fa.fa_latent_write(*self.part, self.pages, self.table)
        fa.fa_fwd_expanded(self.qe[:1], self.kv[:1], self.part[1][:1], out=self.oe[:1], lse=self.le[:1])

    def outputs(self):
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_OK
        return [t.clone() for t in (self.o, self.lse, self.ol, self.ll, self.back, self.qr, self.ql, self.oe,
                                    self.le, *self.part, *self.cache, self.pages, self.length)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.is_floating_point() else x,
                           y.view(torch.uint8) if y.is_floating_point() else y) for x, y in zip(a, b))


def test_copies_between_captured_calls():
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
        for t in (replayed.oe, replayed.le, replayed.o, replayed.lse, replayed.ol, replayed.ll):
            t.zero_()
        graph.replay()
        assert same(want, replayed.outputs())
