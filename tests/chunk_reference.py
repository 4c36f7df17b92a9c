"""Inputs and the fp64 reference of chunk attention.

The reference rounds values to f16, and keys of requests of more than FINE
tokens, as the operator is documented to, and is exact otherwise.  What may
differ:

* the softmax weights, each rounded to f16 (half a step, 2^-11 of it), and the
  bf16 output (2^-8 of the value);
* keys and values that fp32 sums of 512 products left on the other side of a
  rounding border: a step, 2^-10 of the element.  About one in 500 does (an fp32
  error of 2^-20 on either side of a border, in steps of 2^-10), so six of a key's
  128 products may, and six of the values of a sum.  Keys of shorter requests:
  2^-22 of each product;
* fp32 sums of 192 products and of the weights: 1e-5 of the sum of magnitudes.
"""
import numpy as np
import torch

NOPE, ROPE, LATENT, KDIM, VDIM = 128, 64, 512, 576, 128
FINE = 1024


def owned(L, d, D, I):
    return (L // (D * I)) * I + min(max(L % (D * I) - d * I, 0), I)


def make(seq, q, H, bs=16, fp8=False, pow2=True, D=1, I=1, local=False, pad=0, seed=0, device="cuda", q_scale=1.5):
    g = torch.Generator(device=device).manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = len(seq)
    n = np.array([[-(-(owned(s, d, D, I) if local else s) // bs) for s in seq] for d in range(D if local else 1)])
    total, W = max(1, int(n.sum())), max(1, int(n.max()))
    perm = rng.permutation(total)
    table = np.full((n.shape[0], B, W), -1, np.int32)
    at = 0
    for d in range(n.shape[0]):
        for b in range(B):
            table[d, b, :n[d, b]] = perm[at:at + n[d, b]]
            at += n[d, b]
    x = torch.empty((total * bs, KDIM), dtype=torch.bfloat16, device=device).normal_(generator=g)
    st = dict(seq_h=list(seq), q_h=list(q), H=H, bs=bs, D=D, I=I, local=local, scale=0.0722, kv_scale=None,
              table=torch.from_numpy(table if local else table[0]).to(device),
              seq=torch.tensor(seq, dtype=torch.int32, device=device),
              qsl=torch.tensor(np.concatenate([[0], np.cumsum(q)]), dtype=torch.int32, device=device),
              T=sum(q) + pad, total=sum(max(0, s) for s in seq))
    if fp8:
        s = x.float().abs().amax(1) / 256
        s = torch.exp2(torch.ceil(torch.log2(s))) if pow2 else s
        st["cache"] = (x.float() / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(total, bs, KDIM)
        st["kv_scale"] = s.view(total, bs)
    else:
        st["cache"] = x.view(total, bs, KDIM)
    st["q"] = (q_scale * torch.empty((st["T"], H, NOPE + ROPE), device=device).normal_(generator=g)).to(torch.bfloat16)
    st["w"] = (torch.empty((H * 256, LATENT), device=device).normal_(generator=g) / 512 ** 0.5).to(torch.bfloat16)
    return st


def rows_of(st, b):
    """Cache rows (int64) of the positions of request b, -1 without a block."""
    p = np.arange(max(0, st["seq_h"][b]))
    table = st["table"].cpu().numpy().astype(np.int64)
    if st["local"]:
        j, row = p // (st["D"] * st["I"]) * st["I"] + p % st["I"], table[p // st["I"] % st["D"], b]
        blk = row[np.arange(len(p)), j // st["bs"]] if len(p) else np.zeros(0, np.int64)
    else:
        j, blk = p, table[b][p // st["bs"]]
    return np.where((blk >= 0) & (blk < st["cache"].shape[0]), blk * st["bs"] + j % st["bs"], -1)


def latents(st, rows):
    """fp64 values of cache rows; an FP8 code x scale rounded to bf16, as documented."""
    at = torch.from_numpy(np.maximum(rows, 0)).to(st["q"].device)
    flat = st["cache"].reshape(-1, KDIM)
    if st["kv_scale"] is None:
        return flat[at].double()
    return (flat[at].view(torch.float8_e4m3fn).float() * st["kv_scale"].reshape(-1)[at][:, None]).to(torch.bfloat16).double()


def reference(st, skip_requests=()):
    """(out, lse, tolerance of out, tolerance of lse) in fp64."""
    dev, H = st["q"].device, st["H"]
    out = torch.zeros((st["T"], H, VDIM), dtype=torch.float64, device=dev)
    lse = torch.full((st["T"], H), -torch.inf, dtype=torch.float64, device=dev)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    r0 = 0
    for b, (L, n) in enumerate(zip(st["seq_h"], st["q_h"])):
        rows = rows_of(st, b)
        if n == 0 or len(rows) == 0 or b in skip_requests:
            r0 += n
            continue
        kv = latents(st, rows)
        exists = torch.from_numpy(rows >= 0).to(dev)
        last = L - n + torch.arange(n, device=dev)
        see = (torch.arange(L, device=dev)[None, :] <= last[:, None]) & exists[None, :]
        for h in range(H):
            w = st["w"][256 * h:256 * h + 256].double()
            up = kv[:, :LATENT] @ w.T
            f16 = up.float().to(torch.float16).double()
            k, v = torch.cat([(up if L <= FINE else f16)[:, :NOPE], kv[:, LATENT:]], 1), f16[:, NOPE:]
            q = st["q"][r0:r0 + n, h].double()
            s = (st["scale"] * (q @ k.T)).masked_fill(~see, -torch.inf)
            z = torch.logsumexp(s, 1)
            some = see.any(1)
            p = torch.where(some[:, None], torch.exp(s - z[:, None]), torch.zeros_like(s))
            p = torch.where(see, p, torch.zeros_like(p))
            v0 = torch.where(exists[:, None], v, torch.zeros_like(v))
            size = p @ v0.abs()
            big = torch.nan_to_num(q.abs()).amax(1) * torch.nan_to_num(k.abs()).amax()
            ds = abs(st["scale"]) * ((6 * 2.0 ** -10 * big if L > FINE else 0.0) + 1e-5 * torch.nan_to_num(q.abs()) @ torch.nan_to_num(k.abs()).amax(0))
            peak = p.amax(1, keepdim=True) * torch.nan_to_num(v0.abs()).amax(0)[None]
            out[r0:r0 + n, h] = p @ v0
            lse[r0:r0 + n, h] = torch.where(some, z, torch.full_like(z, -torch.inf))
            tol[r0:r0 + n, h] = size * (2 * ds[:, None] + 2.0 ** -11 + 1e-5) + 6 * 2.0 ** -10 * peak
            tol_l[r0:r0 + n, h] = ds + 1e-5 * (1 + z.abs())
        r0 += n
    return out, lse, tol, tol_l


def check(got, got_lse, want):
    out, lse, tol, tol_l = want
    rounding = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    dead = lse == -torch.inf
    assert torch.equal(got_lse == -torch.inf, dead)
    assert (got[dead] == 0).all()
    nan = lse.isnan()
    assert torch.equal(got_lse.isnan(), nan) and got[nan].isnan().all()
    live = ~dead & ~nan
    e = (got.double() - out).abs()[live]
    assert (e <= (tol + rounding * (out.abs() + tol))[live]).all(), float(e.max())
    e = (got_lse.double() - lse).abs()[live]
    assert (e <= tol_l[live]).all(), float(e.max())
