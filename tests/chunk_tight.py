"""A tight reference of chunk attention, for fp32 outputs.

As chunk_reference (values in f16, keys of requests of more than FINE tokens in
f16, else exact), but with errors added as what they are, independent and of
either sign, where that one bounds each by its largest.  Of a row with weights p:

* a key element that its fp32 sum of 512 products (off by 2^-18 at most: 32 steps of
  the tensor core's accumulator, 2^-23 of about 1 each) left on the other side of a
  border of f16's steps is off by a step, at most 2^-10 of it, with a chance of
  2^-18 / step: a variance of 2^-18 x 2^-10 |k|.  A score's variance v_t is scale^2
  times the sum of q^2 times that.  (Keys in 22 bits: (2^-22 k)^2.)
* the log-sum-exp moves by the sum of p_t times the scores' errors: variance
  sum p_t^2 v_t; six deviations, and fp32's roundings of scores (2^-20 of the sum of
  192 products, about 21 at a deviation, times the scale), exponentials, sums and
  the logarithm: 1e-5 + 2^-20 |lse|.
* the output moves by the sum of p_t (error of the score + rounding of the weight to
  f16, at most 2^-11, variance 2^-22 / 3) (v_t - out), and by p_t times the values'
  border crossings, 128 elements together: twice the root of their variances, and
  2^-23 of the output for each of L / 16 additions to fp32 accumulators (that cut
  off), twice for partial sums larger than the last.
"""
import torch

from tests.chunk_reference import FINE, LATENT, NOPE, latents, rows_of


def tight_reference(st, times=None):
    """[(rows, head, out, lse, tolerance of out's error in 2-norm, tolerance of lse)] for
    each request and head, fp64.  times: token weights of request 0 (1 where None), to
    plant a lost or doubled token."""
    parts, r0, dev = [], 0, st["q"].device
    for b, (L, n) in enumerate(zip(st["seq_h"], st["q_h"])):
        if n == 0 or L <= 0:
            r0 += n
            continue
        kv = latents(st, rows_of(st, b))
        last = L - n + torch.arange(n, device=dev)
        see = torch.arange(L, device=dev)[None, :] <= last[:, None]
        for h in range(st["H"]):
            up = kv[:, :LATENT] @ st["w"][256 * h:256 * h + 256].double().T
            f16 = up.float().to(torch.float16).double()
            nope, v = (up if L <= FINE else f16)[:, :NOPE], f16[:, NOPE:]
            q = st["q"][r0:r0 + n, h].double()
            s = st["scale"] * (q @ torch.cat([nope, kv[:, LATENT:]], 1).T)
            var = nope.abs() * 2.0 ** -28 if L > FINE else (nope * 2.0 ** -22) ** 2
            var = st["scale"] ** 2 * (q[:, :NOPE] ** 2 @ var.T)
            s = s.masked_fill(~see, -torch.inf)
            if times is not None and b == 0:
                s = s + torch.log(times.double())[None]
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - z[:, None])
            out = p @ v
            spread = (v ** 2).sum(1)[None] + (out ** 2).sum(1, keepdim=True)
            tol = 2 * ((p ** 2 * ((var + 2.0 ** -22 / 3) * spread + 2.0 ** -28 * v.abs().sum(1)[None])).sum(1)).sqrt()
            tol = tol + 2 * 2.0 ** -23 * (L / 16) * out.norm(dim=1)
            tol_lse = 6 * (p ** 2 * var).sum(1).sqrt() + 1e-5 + 2.0 ** -20 * z.abs()
            parts.append((slice(r0, r0 + n), h, out, z, tol, tol_lse))
        r0 += n
    return parts


def tight_check(got, got_lse, parts):
    assert got.dtype in (torch.float32, torch.float64)
    for rows, h, out, z, tol, tol_lse in parts:
        e = (got_lse[rows, h].double() - z).abs()
        assert (e <= tol_lse).all(), ("lse", h, float(e.max()), float(tol_lse.min()))
        e = (got[rows, h].double() - out).norm(dim=1)
        assert (e <= tol).all(), ("out", h, float((e / out.norm(dim=1)).max()), float((tol / out.norm(dim=1)).min()))
