"""The compiled calls of the 16-bit caches and latent attention: the same bits as the
ctypes path, taken for the plain call and left to it for everything else."""
import pytest
import torch

from attention_forward_gb300 import fa

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


class Inputs:
    def __init__(self, seed=1):
        g = torch.Generator("cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
        self.q, self.k, self.v = n(2, 4, 30, 64), n(2, 2, 30, 64), n(2, 2, 30, 64)
        self.cache = [n(8, 2, 16, 64), n(8, 2, 16, 64)]
        self.table = torch.arange(8, dtype=I32, device="cuda").view(2, 4)
        self.start = torch.tensor([5, 20], dtype=I32, device="cuda")
        self.count = torch.tensor([30, 7], dtype=I32, device="cuda")
        self.length = torch.tensor([60, 33], dtype=I32, device="cuda")
        self.freqs = torch.rand(32, generator=g, device="cuda")
        self.slopes = torch.rand(4, generator=g, device="cuda")
        self.c, self.r, self.qr = n(2, 30, 512), n(2, 30, 64), n(2, 4, 30, 64)
        self.wide, self.latent = n(2, 4, 30, 576), n(8, 16, 576)
        self.q192, self.kv = n(2, 4, 30, 192), n(2, 4, 30, 256)
        self.out = [torch.zeros_like(self.k), torch.zeros_like(self.k)]
        self.lout = [torch.zeros_like(self.c), torch.zeros_like(self.r)]
        self.turned = torch.zeros_like(self.q)


def calls(x):
    one = x.q[:, :, :1].contiguous()
    wide = x.wide[:, :, :1].contiguous()
    return {
        "paged_write": lambda: (fa.fa_paged_write(x.k, x.v, x.cache, x.table, x.start, x.count, x.freqs,
                                                  True, x.q, x.turned), *x.cache),
        "paged_read": lambda: fa.fa_paged_read(x.cache, x.table, x.start, x.count, x.out),
        "fwd_paged": lambda: fa.fa_fwd_paged(one, x.cache, x.table, x.length, None, 20.0, x.slopes),
        "latent_write": lambda: (fa.fa_latent_write(x.c, x.r, x.latent, x.table, x.start, x.count, x.freqs,
                                                    False, x.qr, x.wide), x.latent),
        "latent_read": lambda: fa.fa_latent_read(x.latent, x.table, x.start, x.count, x.lout),
        "fwd_latent": lambda: fa.fa_fwd_latent(wide, x.latent, x.table, x.length, 0.1),
        "fwd_expanded": lambda: fa.fa_fwd_expanded(x.q192, x.kv, x.r, True),
    }


NAMES = ["paged_write", "paged_read", "fwd_paged", "latent_write", "latent_read", "fwd_latent",
         "fwd_expanded"]


@pytest.mark.parametrize("name", NAMES)
def test_taken_for_the_plain_call_with_the_same_bits(name, monkeypatch):
    real = fa._load_native()
    taken = []

    class Watch:
        def __getattr__(self, n):
            def call(*a):
                got = getattr(real, n)(*a)
                taken.append(got is not NotImplemented)
                return got
            return call

    class Never:
        def __getattr__(self, n):
            return lambda *a: NotImplemented

    monkeypatch.setattr(fa, "_native", Watch())
    mine = [t.clone() for t in calls(Inputs())[name]()]
    assert taken == [True]
    monkeypatch.setattr(fa, "_native", Never())
    theirs = calls(Inputs())[name]()
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    for a, b in zip(mine, theirs):
        assert a.dtype is b.dtype and torch.equal(a, b)


def test_what_is_wrong_is_refused_by_name():
    x = Inputs()
    one, wide = x.q[:, :, :1].contiguous(), x.wide[:, :, :1].contiguous()
    half = [t.half() for t in x.cache]
    wrong = [
        lambda: fa.fa_fwd_paged(one.float(), x.cache, x.table, x.length),
        lambda: fa.fa_fwd_paged(one.transpose(1, 3), x.cache, x.table, x.length),
        lambda: fa.fa_fwd_paged(one, half, x.table, x.length),
        lambda: fa.fa_fwd_paged(one, x.cache[:1], x.table, x.length),
        lambda: fa.fa_fwd_paged(one, x.cache, x.table.long(), x.length),
        lambda: fa.fa_fwd_paged(one, x.cache, x.table, x.length[:1]),
        lambda: fa.fa_fwd_paged(one, x.cache, x.table, x.length.cpu()),
        lambda: fa.fa_fwd_paged(one, x.cache, x.table, None),
        lambda: fa.fa_fwd_paged(one, x.cache, x.table, x.length, slopes=x.slopes[:3]),
        lambda: fa.fa_paged_write(x.k, x.v[:, :1], x.cache, x.table),
        lambda: fa.fa_paged_write(x.k, x.v, x.cache, x.table, freqs=x.freqs.double()),
        lambda: fa.fa_paged_write(x.k, x.v, x.cache, x.table, q=x.q[:, :3].contiguous()),
        lambda: fa.fa_paged_write(x.k, x.v, x.cache, x.table, q_out=x.turned),
        lambda: fa.fa_paged_read(x.cache, x.table, out=[x.k, x.q]),
        lambda: fa.fa_latent_write(x.c, x.r, x.latent, x.table, freqs=x.freqs[:16]),
        lambda: fa.fa_latent_write(x.c, x.r, x.latent, x.table, q_rope=x.qr),
        lambda: fa.fa_latent_write(x.c, x.r[:, :3], x.latent, x.table),
        lambda: fa.fa_latent_read(x.latent, x.table, out=[x.r, x.c]),
        lambda: fa.fa_fwd_latent(x.q, x.latent, x.table, x.length),
        lambda: fa.fa_fwd_latent(wide, x.latent[..., :512], x.table, x.length),
        lambda: fa.fa_fwd_expanded(x.q192, x.kv, x.r[:1]),
        lambda: fa.fa_fwd_expanded(x.q192, x.q192, x.r),
        lambda: fa.fa_fwd_expanded(x.q192, x.kv[..., ::2], x.r),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fa.fa_fwd_paged(one, x.cache, x.table, x.length, softcap=-1.0),
                 lambda: fa.fa_fwd_paged(one, x.cache, x.table, x.length, scale=0.0),
                 lambda: fa.fa_paged_write(x.k, x.v, x.cache, x.table, freqs=x.freqs[:12].contiguous()),
                 lambda: fa.fa_fwd_latent(wide, x.latent, x.table, x.length, float("inf")),
                 lambda: fa.fa_fwd_expanded(x.q192, x.kv, x.r, scale=float("nan"))):
        with pytest.raises(fa.FAError):
            call()
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK


def test_plain_numbers_of_other_kinds_and_the_current_stream():
    x = Inputs()
    one = x.q[:, :, :1].contiguous()
    ref = fa.fa_fwd_paged(one, x.cache, x.table, x.length, scale=0.25, softcap=20.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = fa.fa_fwd_paged(one, tuple(x.cache), x.table, x.length, scale=torch.tensor(0.25), softcap=20)
    b = fa.fa_fwd_paged(torch.nn.Parameter(one), x.cache, x.table, x.length, scale=0.25, softcap=20.0)
    c = fa.fa_fwd_expanded(x.q192, x.kv, x.r, 1)
    d = fa.fa_fwd_expanded(x.q192, x.kv, x.r, True)
    torch.cuda.synchronize()
    for got, want in ((a, ref), (b, ref), (c, d)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not got[0].requires_grad


def test_pools_in_either_order_or_the_same():
    """One descriptor serves both pools in either order; K may be V."""
    x = Inputs()
    one = x.q[:, :, :1].contiguous()
    both = torch.stack([x.cache[1], x.cache[0]])
    ref = fa.fa_fwd_paged(one, x.cache, x.table, x.length)
    turned = fa.fa_fwd_paged(one, [both[1], both[0]], x.table, x.length)
    same = fa.fa_fwd_paged(one, [x.cache[0], x.cache[0]], x.table, x.length)
    again = fa.fa_fwd_paged(one, [x.cache[0], x.cache[0].clone()], x.table, x.length)
    torch.cuda.synchronize()
    for got, want in ((turned, ref), (same, again)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
