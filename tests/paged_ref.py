"""Plain 64-bit forms of the 16-bit paged caches' operators, with the error that
each output may have -- TEST INFRASTRUCTURE.

Tolerances, fixed before the first run.  u is half a step of the output's type
(torch.finfo.eps / 2: bf16 2^-8, fp16 2^-11).

rotate: the pair (x, y) at the angle a.  |out - out64| <= u |out64| + 2^-25 (fp16's
smallest step, halved) + 2^-20 (|x| + |y|): the angle in half turns is rounded to 24
bits (2^-25 pi), sine and cosine are off by 2^-23 at most, the products and the
difference by 3 2^-24, together 7e-7 < 2^-20.

attention: with A = sum_j p_j |v_j| per output element,
  |O - O64| <= (u + d + n 2^-23) A + u |O64| + 2^-24 sum_j |v_j|
u A: P rounded once to the type of V; n 2^-23: fp32 sums over the keys, 16 a step, n
= ceil(keys / 16) + 8 (the partials' merge); 2^-24 sum |v|: fp16 probabilities in
their subnormals (their sum is at least 1).  d = 2 e + 2^-20 is a probability's
relative error with e that of its score:
  e = D / 16 * 2^-23 X + 2^-22 |x| + 4e-7 cap + 2^-22 bias
X bounds scale * sum_d |q_d| |k_d|; the sums' steps are 16 channels wide, each off by
2^-23 of the partial sum; the scale's and log2(e)'s roundings are 2^-22 of the score;
4e-7 cap the tanh's fits, bias the largest slope * distance.
LSE: e + n 2^-23 + 2^-20 + 2^-22 |LSE|."""
import math

import torch


def rotate(x, at, freqs, interleaved):
    """x [..., S, D] in 64 bits, rows at positions `at` [S], and the outputs' bound."""
    u = torch.finfo(x.dtype).eps / 2
    y = x.double()
    half = freqs.numel()
    a = at.double()[:, None] * freqs.double()
    j = torch.arange(half, device=x.device)
    one, two = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    out, tol = y.clone(), torch.zeros_like(y)
    p, q = y[..., one], y[..., two]
    out[..., one] = p * a.cos() - q * a.sin()
    out[..., two] = q * a.cos() + p * a.sin()
    room = 2.0 ** -20 * (p.abs() + q.abs())
    tol[..., one] = room + u * out[..., one].abs() + 2.0 ** -25
    tol[..., two] = room + u * out[..., two].abs() + 2.0 ** -25
    return out, tol


def close(got, want, tol):
    over = (got.double() - want).abs() - tol
    assert not got.isnan().any() and over.amax().item() <= 0, f"off by {over.amax().item():.3g} more"


def sequence(pages, table_row, length):
    """Tokens 0 ... length - 1 of one sequence, [Hkv, length, D] (latent: [1, ...])."""
    if pages.dim() == 3:
        pages = pages[:, None]
    page = pages.shape[2]
    at = torch.arange(length, device=pages.device)
    return pages[table_row[at // page].long(), :, at % page].transpose(0, 1)


def attention(q, k, v, seen, scale, cap=0.0, slopes=None, distance=None):
    """(O, LSE, bounds of both) in 64 bits: q [B, H, Sq, D], k [B, Hkv, S, D], v [B,
    Hkv, S, Dv]; seen and distance broadcast to [B, H, Sq, S]."""
    u = torch.finfo(q.dtype).eps / 2
    D, keys = q.shape[-1], k.shape[2]
    q, k, v = q.double(), k.double(), v.double()
    rep = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    x = q @ k.transpose(2, 3) * scale
    X = (q.abs() @ k.abs().transpose(2, 3) * scale).amax(-1) if keys else q.sum(-1) * 0
    x_top = x.abs().amax(-1) if keys else X
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
    n = -(-keys // 16) + 8
    e = D / 16 * 2.0 ** -23 * X + 2.0 ** -22 * x_top + 4e-7 * cap + 2.0 ** -22 * bias
    d = (2 * e + 2.0 ** -20)[..., None]
    tol_o = (u + d + n * 2.0 ** -23) * a + u * o.abs() + 2.0 ** -24 * v.abs().sum(2, keepdim=True)
    tol_l = e + n * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * torch.where(lse.isfinite(), lse.abs(), 0.0)
    return o, lse, tol_o, tol_l


def newest(q, k_pages, v_pages, table, length, scale, cap=0.0, slopes=None):
    """attention() of the newest tokens over pages (v_pages None: the first 512 channels
    of k_pages' rows), sequence by sequence."""
    B, H, Sq, _ = q.shape
    outs = []
    for b in range(B):
        n = max(0, int(length[b]))
        k = sequence(k_pages, table[b], n)[None]
        v = k[..., :512] if v_pages is None else sequence(v_pages, table[b], n)[None]
        if n == 0:
            z = torch.zeros((1, H, Sq, v.shape[-1]), dtype=torch.float64, device=q.device)
            outs.append((z, torch.full((1, H, Sq), -math.inf, dtype=torch.float64, device=q.device),
                         z, z[..., 0]))
            continue
        i = torch.arange(Sq, device=q.device)[:, None] + (n - Sq)
        j = torch.arange(n, device=q.device)[None]
        outs.append(attention(q[b:b + 1], k, v, (j <= i)[None, None], scale, cap, slopes,
                              (i - j).abs()))
    return [torch.cat(x) for x in zip(*outs)]
