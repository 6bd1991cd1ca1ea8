"""Plain 64-bit forms of the score-modified attention and of the 4-bit cache,
with the error that each output may have -- TEST INFRASTRUCTURE.

Tolerances, fixed before the first run.  u is half a step of the output type
(torch.finfo.eps / 2: bf16 2^-8, fp16 2^-11), A = sum_j p_j |v_j| per output
element.

attention(..., p_step=u):  |O - O64| <= (p_step + v_step) A  (P, and for the
cache V, rounded once to 16 bits) + u |O64| (the output's rounding) + d A +
2^-24 sum_j |v_j| / sum_j p'_j (probabilities in fp16's subnormal range; p'
are the probabilities against the reference maximum, whose sum is at least 1),
with d the relative error of a probability from fp32 work,
  d = 2 e + 2^-20,  e = 2^-20 X + 4e-7 cap + 2^-22 bias
where X bounds scale * sum_d |q_d| |k_d| (fp32 sums of at most 160 terms, each
step off by 2^-23 at most, and the scale's rounding), 4e-7 cap the tanh's two
fits and exponential, bias the largest slope * distance.  LSE: e + 2^-20 (its
own logarithm and sum) + 2^-22 |LSE|."""
import math

import torch


def attention(q, k, v, seen, scale, cap=0.0, slopes=None, distance=None, p_step=0.0, v_step=0.0,
              x_bound=None):
    """O, LSE in 64 bits and their bounds.  q [B, H, Sq, D]; k, v [B, Hkv, S,
    D]; seen broadcasts to [B, H, Sq, S]; distance to the same."""
    u = torch.finfo(q.dtype).eps / 2
    q, k, v = q.double(), k.double(), v.double()
    B, H, Sq, D = q.shape
    rep = H // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    x = torch.einsum("bhid,bhjd->bhij", q, k) * scale
    if x_bound is None:
        x_bound = (q.abs().sum(-1).amax() * k.abs().amax() * scale).item()
    bias = 0.0
    if cap:
        x = cap * torch.tanh(x / cap)
    if slopes is not None:
        b = slopes.double().view(1, -1, 1, 1) * distance
        bias = b.abs().amax().item()
        x = x - b
    x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse.isfinite(), lse, 0.0)[..., None])
    o, a = p @ v, p @ v.abs()
    e = 2.0 ** -20 * x_bound + 4e-7 * cap + 2.0 ** -22 * bias
    d = 2 * e + 2.0 ** -20
    tol_o = (p_step + v_step + d) * a + u * o.abs() + 2.0 ** -24 * v.abs().sum(2, keepdim=True)
    tol_l = e + 2.0 ** -20 + 2.0 ** -22 * torch.where(lse.isfinite(), lse.abs(), 0.0)
    return o, lse, tol_o, tol_l


def check(o, lse, ref):
    ro, rl, tol_o, tol_l = ref
    assert torch.equal(lse.isfinite(), rl.isfinite())
    assert torch.equal(lse == -math.inf, rl == -math.inf)
    fin = rl.isfinite()
    worst = ((lse.double() - rl)[fin].abs() / tol_l[fin]).amax().item() if fin.any() else 0.0
    assert worst <= 1, f"LSE off by {worst:.2f} of its bound"
    assert o.isfinite().all()
    assert (o[~fin] == 0).all(), "a row without keys is not 0"
    over = ((o.double() - ro).abs() / tol_o.clamp_min(1e-300))[fin]
    assert not fin.any() or over.amax().item() <= 1, f"O off by {over.amax().item():.2f} of its bound"


def score_seen(Sq, Skv, causal, prefix=None, doc_q=None, doc_k=None, device="cuda"):
    i = torch.arange(Sq, device=device)[:, None] + (Skv - Sq)
    j = torch.arange(Skv, device=device)[None]
    seen = torch.ones((1, 1, Sq, Skv), dtype=torch.bool, device=device)
    if causal:
        seen = (j <= i)[None, None]
        if prefix is not None:
            seen = seen | (j < prefix.view(-1, 1, 1, 1))
    if doc_q is not None:
        a, b = doc_q[:, None, :, None], doc_k[:, None, None, :]
        seen = seen & (a == b) & (a >= 0)
    return seen, (i - j).abs()


def quantise(x):
    """Codes by channel [..., D] and (scale, minimum) fp16 [..., D/32, 2] of
    rows x: the documented arithmetic, the floor decided in 64 bits."""
    x = x.float().clamp(-61440.0, 61440.0).unflatten(-1, (-1, 32))
    lo, hi = x.amin(-1), x.amax(-1)
    # through 64 bits: on a GPU torch divides by 15 as a product, an ulp off at times
    scale, least = ((hi - lo).double() / 15).float().half(), lo.half()
    s, z = scale.double()[..., None], least.double()[..., None]
    code = torch.floor((x.double() - z) / torch.where(s > 0, s, 1.0) + 0.5).clamp(0, 15)
    code = torch.where((s > 0) & ~torch.isnan(s), code, 0.0)
    return code.flatten(-2).to(torch.uint8), torch.stack([scale, least], -1)


def pack(codes):
    """Codes by channel [..., D] to the rows' bytes [..., D/2]."""
    D = codes.shape[-1]
    G = D // 32
    out = torch.zeros(codes.shape[:-1] + (D // 2,), dtype=torch.uint8, device=codes.device)
    for d in range(D):
        word, nib = G * (d % 32 // 8) + d // 32, d % 8
        out[..., 4 * word + nib // 2] |= codes[..., d] << (4 * (nib % 2))
    return out


def unpack(bytes_, params):
    """Values in 64 bits [..., D] of rows [..., D/2] with params [..., D/32, 2]."""
    D = bytes_.shape[-1] * 2
    G = D // 32
    out = torch.empty(bytes_.shape[:-1] + (D,), dtype=torch.float64, device=bytes_.device)
    p = params.double()
    for d in range(D):
        word, nib = G * (d % 32 // 8) + d // 32, d % 8
        code = (bytes_[..., 4 * word + nib // 2] >> (4 * (nib % 2))) & 15
        out[..., d] = code * p[..., d // 32, 0] + p[..., d // 32, 1]
    return out


def sequence(codes, params, table_row, length):
    """Tokens 0 ... length - 1 of one sequence, [Hkv, length, D] in 64 bits."""
    page = codes.shape[2]
    at = torch.arange(length, device=codes.device)
    pg = table_row[at // page].long()
    return unpack(codes[pg, :, at % page], params[pg, :, at % page]).transpose(0, 1)
