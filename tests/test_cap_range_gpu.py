"""Capped scores over the cap's whole range (1e-6 ... 1e6): small scores beside
ones at the cap, in the same tile, of other rows and of keys that no row sees.

Tolerances, fixed before the first run.  ops_ref.py bounds a capped score by
4e-7 of the cap; here each is bounded by its own size, which is what tells a
score of 3 under a cap of 1e6 from one that lost its digits to the cap:
  e_ij = 1.7e-6 |x_ij|    the polynomial (1.0e-6 of the value on [0, 0.5], 1.4e-6 for
                          three terms on [0, 0.145]) and four fp32 roundings
       + 2^-20 X_ij       X_ij = scale sum_d |q_id| |k_jd|: fp32 sums
       + 2^-20 cap        only where |x_ij| is past 0.14 of the cap: 2 cap / (1 +
                          e^2y), whose quotient is at most 1 and off by
                          2^-21.4: 2^-22 of the division, 2^-24 of the sum,
                          2^-24 and 2^-25.2 of the exponential and its argument
With e_i the largest over the row's visible keys: LSE e_i + 2^-20 + 2^-22 |LSE|,
O (p_step + 2 e_i + 2^-20) sum_j p_j |v_j| + p_step |O| + 2^-24 sum |v_j|, as in
ops_ref.py."""
import math

import pytest
import torch

from attention_forward_gb300 import fa
import ops_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def make(B, H, Hkv, Sq, Skv, D, dt, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dt])  # noqa: E731
    return n(B, H, Sq, D), n(B, Hkv, Skv, D), n(B, Hkv, Skv, D)


def expect(q, k, v, cap, seen, scale=None):
    """O, LSE in 64 bits and the bounds above; K of keys that a row does not see
    counts for nothing."""
    u = torch.finfo(q.dtype).eps / 2
    q, k, v = q.double(), k.double(), v.double()
    rep = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    scale = scale or q.shape[3] ** -0.5
    y = torch.einsum("bhid,bhjd->bhij", q, k) * scale
    big = torch.einsum("bhid,bhjd->bhij", q.abs(), k.abs()) * scale
    x = cap * torch.tanh(y / cap)
    e = 1.7e-6 * x.abs() + 2.0 ** -20 * big + torch.where(x.abs() > 0.14 * cap, 2.0 ** -20 * cap, 0.0)
    seen = seen.expand_as(x)
    e = torch.where(seen, e, 0.0).amax(-1)
    x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse.isfinite(), lse, 0.0)[..., None])
    o, a = p @ v, p @ v.abs()
    tol_o = (u + 2 * e + 2.0 ** -20)[..., None] * a + u * o.abs() + 2.0 ** -24 * v.abs().sum(2, keepdim=True)
    return o, lse, tol_o, e + 2.0 ** -20 + 2.0 ** -22 * torch.where(lse.isfinite(), lse.abs(), 0.0)


def run(q, k, v, **kw):
    o, lse = fa.fa_fwd_score(q, k, v, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    return o, lse


CAPS = [("bf16", 20.0), ("bf16", 50.0), ("fp16", 50.0), ("bf16", 1e4), ("fp16", 1e4), ("bf16", 1e5),
        ("bf16", 1e6)]
SHAPES = [(1, 4, 2, 1, 300), (1, 4, 2, 200, 300), (1, 80, 40, 513, 640)]
ids = lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else None  # noqa: E731


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt,cap", CAPS)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_masked_keys_at_the_cap_change_nothing(shape, dt, cap, D):
    """Keys of no document hold large finite values of the rows' sign: their
    scores leave the polynomial's range, and no row sees them."""
    q, k, v = make(*shape, D, dt, 1)
    q[..., 0] = q[..., 0].abs() + 0.5
    B, _, _, Sq, Skv = shape
    dq = torch.zeros((B, Sq), dtype=torch.int32, device="cuda")
    dk = torch.zeros((B, Skv), dtype=torch.int32, device="cuda")
    dk[:, 5::17] = -1
    dk[:, -40:] = -1
    kw = dict(softcap=cap, doc_q=dq, doc_k=dk)
    gone = dk[0] < 0
    k[:, :, gone] = 0.0
    ref = run(q, k, v, **kw)
    seen, _ = ops_ref.score_seen(Sq, Skv, False, None, dq, dk)
    ops_ref.check(*ref, expect(q, k, v, cap, seen))
    # scale q k: at least 0.5 * 6e4 / sqrt(D) in fp16
    k[:, :, gone, 0] = 6e4 if dt == "fp16" else 1e9
    for got, want in zip(run(q, k, v, **kw), ref):
        assert torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt,cap", CAPS)
@pytest.mark.parametrize("shape", SHAPES[1:], ids=ids)
def test_keys_behind_the_diagonal_at_the_cap_change_nothing(shape, dt, cap, D):
    q, k, v = make(*shape, D, dt, 2)
    q[..., 0] = q[..., 0].abs() + 0.5
    B, _, _, Sq, Skv = shape
    n = Sq - 30  # rows that do not see the last 30 keys
    k[:, :, -30:] = 0.0
    ref = run(q, k, v, causal=True, softcap=cap)
    seen, _ = ops_ref.score_seen(Sq, Skv, True)
    ops_ref.check(*ref, expect(q, k, v, cap, seen))
    k[:, :, -30:, 0] = 6e4 if dt == "fp16" else 1e9
    o, lse = run(q, k, v, causal=True, softcap=cap)
    assert torch.equal(o[:, :, :n], ref[0][:, :, :n]) and torch.equal(lse[:, :, :n], ref[1][:, :, :n])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dt,cap", CAPS)
def test_one_row_at_the_cap_beside_small_ones(dt, cap, bias, causal):
    """The row's own scores are at the cap, its neighbours' are not."""
    q, k, v = make(1, 4, 2, 300, 520, 128, dt, 3)
    q[..., 0] = 0.0
    for row in (0, 40, 163, 299):
        q[:, :, row, 0] = 250.0 if dt == "fp16" else 1e7
    k[..., 0] = 100.0 + k[..., 0].abs()
    s = torch.zeros(4, device="cuda") if bias else None  # the biased kernel's form
    o, lse = run(q, k, v, causal=causal, softcap=cap, slopes=s)
    seen, _ = ops_ref.score_seen(300, 520, causal)
    ops_ref.check(o, lse, expect(q, k, v, cap, seen))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("cap", [0.01, 1.0, 30.0, 60.0, 1e4, 1e6])
def test_scores_on_both_sides_of_where_the_forms_meet(cap, dt):
    """Scores spread over +- 2 caps (as far as the row's softmax lets them
    count): each row's largest lie anywhere in the range."""
    q, k, v = make(1, 2, 2, 200, 300, 64, dt, 4)
    q.zero_()
    k.zero_()
    q[..., 0] = torch.linspace(-1.0, 1.0, 200, device="cuda").to(q.dtype)
    k[..., 0] = torch.linspace(-1.0, 1.0, 300, device="cuda").to(q.dtype)
    o, lse = run(q, k, v, softcap=cap, scale=2 * cap)
    seen = torch.ones((1, 1, 200, 300), dtype=torch.bool, device="cuda")
    ops_ref.check(o, lse, expect(q, k, v, cap, seen, 2 * cap))


@pytest.mark.parametrize("scale,cap,mult", [
    (1e10, 1e6, 1e-5), (1e10, 50.0, 1e-5), (1e-10, 1e6, 1e5), (1e-14, 100.0, 1e7), (1e5, 1e5, 3e-3),
    (3e3, 1e-3, 1e-2), (1e37, 1e-6, 1e-15), (1e38, 1e6, 1e-17), (3e38, 1e-6, 1.0), (1e-37, 1e6, 1e18)])
def test_scales_far_from_one(scale, cap, mult):
    """Terms of the polynomial that fp32 would not hold; a query of zeros has
    scores of 0 whatever the scale."""
    q, k, v = make(1, 4, 2, 200, 300, 64, "bf16", 5)
    q, k = (q.float() * mult).bfloat16(), (k.float() * mult).bfloat16()
    q[:, :, 7] = 0.0
    if scale == 3e38:
        q.zero_()
    seen, _ = ops_ref.score_seen(200, 300, True)
    scale = torch.tensor(scale).item()
    o, lse = run(q, k, v, causal=True, softcap=cap, scale=scale)
    ops_ref.check(o, lse, expect(q, k, v, cap, seen, scale))
