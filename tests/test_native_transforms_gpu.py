"""The calls of the 16-bit caches and latent attention under torch's function transforms,
whose tensors have no memory that a kernel could be given: each is refused with an
exception, and the process lives on.  In a process of its own, which a call that came
back without the interpreter's lock would end."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
TESTS = os.path.dirname(os.path.abspath(__file__))
TRANSFORMS = ["vmap", "grad", "jvp", "functionalize"]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def under(transform, call, x):
    """Whether call(x), x under the transform, raised."""
    import torch

    raised = []

    def body(y):
        try:
            call(y)
        except Exception:  # noqa: BLE001  (which one is torch's to say)
            raised.append(True)
        return y.float().sum()

    if transform == "vmap":
        torch.vmap(body)(torch.stack([x, x]))
    elif transform == "grad":
        torch.func.grad(body)(x)
    elif transform == "jvp":
        torch.func.jvp(body, (x,), (torch.ones_like(x),))
    else:
        torch.func.functionalize(body)(x)
    return raised == [True]


def child(transform):
    import torch

    import test_native_binding_gpu as plain
    from attention_forward_gb300 import fa

    x = plain.Inputs()
    one, wide = x.q[:, :, :1].contiguous(), x.wide[:, :, :1].contiguous()
    # each of a call's 16-bit tensors in turn
    calls = [
        (lambda k: fa.fa_paged_write(k, x.v, x.cache, x.table), x.k),
        (lambda v: fa.fa_paged_write(x.k, v, x.cache, x.table), x.v),
        (lambda q: fa.fa_paged_write(x.k, x.v, x.cache, x.table, q=q, q_out=x.turned), x.q),
        (lambda c: fa.fa_paged_write(x.k, x.v, [c, x.cache[1]], x.table), x.cache[0]),
        (lambda k: fa.fa_paged_read(x.cache, x.table, out=[k, x.out[1]]), x.out[0]),
        (lambda v: fa.fa_paged_read(x.cache, x.table, out=[x.out[0], v]), x.out[1]),
        (lambda q: fa.fa_fwd_paged(q, x.cache, x.table, x.length), one),
        (lambda c: fa.fa_fwd_paged(one, [x.cache[0], c], x.table, x.length), x.cache[1]),
        (lambda c: fa.fa_latent_write(c, x.r, x.latent, x.table), x.c),
        (lambda r: fa.fa_latent_write(x.c, r, x.latent, x.table), x.r),
        (lambda q: fa.fa_latent_write(x.c, x.r, x.latent, x.table, q_rope=q, q=x.wide), x.qr),
        (lambda c: fa.fa_latent_read(x.latent, x.table, out=[c, x.lout[1]]), x.lout[0]),
        (lambda r: fa.fa_latent_read(x.latent, x.table, out=[x.lout[0], r]), x.lout[1]),
        (lambda q: fa.fa_fwd_latent(q, x.latent, x.table, x.length), wide),
        (lambda c: fa.fa_fwd_latent(wide, c, x.table, x.length), x.latent),
        (lambda q: fa.fa_fwd_expanded(q, x.kv, x.r), x.q192),
        (lambda kv: fa.fa_fwd_expanded(x.q192, kv, x.r), x.kv),
        (lambda r: fa.fa_fwd_expanded(x.q192, x.kv, r), x.r),
    ]
    before = [t.clone() for t in (*x.cache, x.latent, *x.out, *x.lout, x.turned, x.wide)]
    for i, (call, t) in enumerate(calls):
        assert under(transform, call, t), f"call {i} was not refused"
    torch.cuda.synchronize()
    for a, b in zip(before, (*x.cache, x.latent, *x.out, *x.lout, x.turned, x.wide)):
        assert torch.equal(a, b)
    for name, call in plain.calls(x).items():
        assert call() is not None, name
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    print("alive")


def left_out():
    """Arguments that may be left out are not taken for that where they have no memory."""
    import torch

    import test_native_binding_gpu as plain
    from attention_forward_gb300 import fa

    x = plain.Inputs()
    one = x.q[:, :, :1].contiguous()
    four = fa.fa_cache_empty(8, 2, 16, 64)
    doc = torch.zeros((2, 30), dtype=torch.int32, device="cuda")
    calls = [
        (lambda q: fa.fa_paged_write(x.k, x.v, x.cache, x.table, q=q, q_out=q), x.q),
        (lambda s: fa.fa_paged_write(x.k, x.v, x.cache, x.table, s), x.start),
        (lambda n: fa.fa_paged_write(x.k, x.v, x.cache, x.table, None, n), x.count),
        (lambda f: fa.fa_paged_write(x.k, x.v, x.cache, x.table, freqs=f), x.freqs),
        (lambda s: fa.fa_paged_read(x.cache, x.table, s, None, x.out), x.start),
        (lambda n: fa.fa_paged_read(x.cache, x.table, None, n, x.out), x.count),
        (lambda s: fa.fa_fwd_paged(one, x.cache, x.table, x.length, slopes=s), x.slopes),
        (lambda s: fa.fa_latent_write(x.c, x.r, x.latent, x.table, s), x.start),
        (lambda n: fa.fa_latent_write(x.c, x.r, x.latent, x.table, None, n), x.count),
        (lambda f: fa.fa_latent_write(x.c, x.r, x.latent, x.table, freqs=f), x.freqs),
        (lambda q: fa.fa_latent_write(x.c, x.r, x.latent, x.table, q_rope=q, q=q),
         x.wide[..., :64].contiguous()),
        (lambda s: fa.fa_latent_read(x.latent, x.table, s, None, x.lout), x.start),
        (lambda n: fa.fa_latent_read(x.latent, x.table, None, n, x.lout), x.count),
        (lambda s: fa.fa_cache_write(x.k, x.v, four, x.table, s), x.start),
        (lambda n: fa.fa_cache_write(x.k, x.v, four, x.table, None, n), x.count),
        (lambda s: fa.fa_fwd_score(x.q, x.k, x.v, slopes=s), x.slopes),
        (lambda d: fa.fa_fwd_score(x.q, x.k, x.v, doc_q=d, doc_k=d), doc),
    ]
    kept = (*x.cache, x.latent, *x.out, *x.lout, *four)
    before = [t.clone() for t in kept]
    for i, (call, t) in enumerate(calls):
        assert under("functionalize", call, t), f"call {i} was not refused"
    torch.cuda.synchronize()
    for a, b in zip(before, kept):
        assert torch.equal(a, b)


def test_an_argument_without_memory_is_not_one_left_out():
    left_out()


@pytest.mark.parametrize("transform", TRANSFORMS)
def test_refused_with_an_exception(transform):
    r = subprocess.run([sys.executable, os.path.abspath(__file__), transform], cwd=os.path.dirname(TESTS),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "alive" in r.stdout, f"{r.returncode}\n{r.stdout}\n{r.stderr}"


if __name__ == "__main__":
    sys.path[:0] = [os.path.dirname(TESTS), TESTS]
    child(sys.argv[1])
