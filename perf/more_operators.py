"""Cases of the operators around a prefill chunk of an MLA model on a paged
latent cache, in plain torch operations and through the library.

Three operators of one serving step:

* ``extend``  block tables and slot maps: the blocks that the step's new tokens
  need are taken from a free list on the device and entered in the requests'
  tables (one table or one per shard), and every new token gets its position
  and its cache slot;
* ``rope``    norm of the latent and position rotation of its rope part, written
  into the paged cache (bf16 or FP8 E4M3), with the rotated query;
* ``chunk``   causal attention of chunks of new tokens over the paged latent
  cache, keys and values projected up from the latents for each head.

``own`` selects the library's calls; otherwise ``run`` computes the same in
elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE, KDIM = 512, 64, 576
NOPE, VDIM = 128, 128
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
EPS = 1e-6
DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _extend(name, B, qlo, qhi, lo, hi, bs, D, I, local):
    return dict(name=name, op="extend", B=B, qlo=qlo, qhi=qhi, lo=lo, hi=hi, bs=bs, D=D, I=I, local=local)


def _rope(name, T, H, query, fp8, norm, pairs, top):
    return dict(name=name, op="rope", T=T, H=H, query=query, fp8=fp8, norm=norm, pairs=pairs, top=top, bs=64)


def _chunk(name, B, qlo, qhi, lo, hi, H, fp8, D, I, local, bs, pad):
    return dict(name=name, op="chunk", B=B, qlo=qlo, qhi=qhi, lo=lo, hi=hi, H=H, fp8=fp8, D=D, I=I, local=local,
                bs=bs, pad=pad)


def listed():
    return [
        # one request's decode step: latency
        _extend("extend_b1_q1", 1, 1, 1, 999, 999, 64, 1, 1, False),
        # the decode step of a large batch over eight shards with their own tables
        _extend("extend_b256_q1_d8_local", 256, 1, 1, 700, 33000, 64, 8, 1, True),
        # verification rows of many requests in small blocks
        _extend("extend_b515_q1to5", 515, 1, 5, 20, 9000, 16, 1, 1, False),
        # prefill chunks of seven requests over eight shards
        _extend("extend_b7_q2341_d8_i64_local", 7, 2341, 2341, 0, 20000, 64, 8, 64, True),
        # the decode step of one request, with the absorbed query: latency
        _rope("rope_t1_h128", 1, 128, "decode", False, True, True, 120000),
        # the decode step of a large batch into the fp8 cache
        _rope("rope_t256_h128_fp8", 256, 128, "decode", True, True, True, 120000),
        # a prefill chunk: the queries' rope parts and the cache rows, split halves
        _rope("rope_chunk_t4099_h128", 4099, 128, "pe", False, True, False, 33000),
        # a long prefill's cache rows alone, into the fp8 cache
        _rope("rope_prefill_t16381_fp8", 16381, 0, "none", True, True, True, 33000),
        # a short prompt on a tensor-parallel rank's heads: latency
        _chunk("chunk_b1_q9_h16", 1, 9, 9, 0, 0, 16, False, 1, 1, False, 16, 0),
        # chunked prefill of a few requests out of the fp8 cache
        _chunk("chunk_b4_q509_l8k_fp8", 4, 131, 509, 2900, 7700, 128, True, 1, 1, False, 64, 0),
        # decoding and prefilling requests in one step, eight shards with their own tables, padded rows
        _chunk("chunk_b12_mixed_h16_d8", 12, 1, 700, 450, 19000, 16, False, 8, 1, True, 64, 5),
        # a long prompt's last chunk, all heads: the tensor pipe's case
        _chunk("chunk_b1_q2048_l24k", 1, 2048, 2048, 21952, 21952, 128, False, 1, 1, False, 64, 0),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("extend", "rope", "chunk", "chunk"))
    if op == "extend":
        B = _logu(rng, 1, 600)
        qhi = _logu(rng, 1, max(2, 16000 // B))
        hi = _logu(rng, 1, min(32000, 4000000 // B))
        D = rng.choice((1, 2, 8))
        c = _extend("", B, max(1, qhi // rng.randint(1, 5)), qhi, rng.choice((0, hi // 3)), hi,
                    rng.choice((1, 16, 64)) if B * (hi + qhi) < 400000 and B * qhi < 5000 else 64, D, rng.choice((1, 3, 64)),
                    rng.random() < 0.5)
    elif op == "rope":
        query = rng.choice(("none", "decode", "pe"))
        H = 0 if query == "none" else rng.choice((1, 16, 33, 128))
        T = _logu(rng, 1, {"none": 16000, "decode": min(15000, 30000 // max(1, H)), "pe": min(16000, 480000 // max(1, H))}[query])
        c = _rope("", T, H, query, rng.random() < 0.5, rng.random() < 0.8, rng.random() < 0.5,
                  rng.choice((5000, 33000, 120000)))
    else:
        B = _logu(rng, 1, 16)
        H = rng.choice((1, 5, 16, 64, 128))
        qhi = _logu(rng, 1, 2048)
        # no more context than the listed cases have for so many rows
        most = min(32000.0, 24000.0 * 2048 * 128 / (max(qhi, 420) * H * B), 800000.0 / B)
        hi = _logu(rng, 1, max(2, most - qhi)) if most > qhi else rng.randint(0, 40)
        D = rng.choice((1, 1, 2, 8))
        c = _chunk("", B, max(1, qhi // rng.randint(1, 40)), qhi, rng.choice((0, hi // 4, hi)), hi, H,
                   rng.random() < 0.5, D, rng.choice((1, 3, 64)), D > 1 and rng.random() < 0.7,
                   rng.choice((1, 16, 64, 64)), rng.choice((0, 0, 3)))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case):
    """(context before the step, new rows) of each request: a fixed spread
    over the ranges, so that a case's work does not depend on the seed."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    ctx = [lo + (hi - lo) * ((7 * b + 3) % B) // max(1, B - 1) if B > 1 else hi for b in range(B)]
    q = [case["qlo"] + (case["qhi"] - case["qlo"]) * ((5 * b + B - 1) % B) // max(1, B - 1) if B > 1 else case["qhi"]
         for b in range(B)]
    return ctx, q


def _owned(L, d, D, I):
    """How many of the first L positions shard d owns."""
    full, rem = divmod(L, D * I)
    return full * I + min(max(rem - d * I, 0), I)


def _paged(seq, bs, D, I, local, rng):
    """Blocks in random order: (table, number of blocks); unused columns -1."""
    if local:
        n = [[-(-_owned(s, d, D, I) // bs) for s in seq] for d in range(D)]
    else:
        n = [[-(-s // bs) for s in seq]]
    n = np.asarray(n, dtype=np.int64)
    total, W = int(n.sum()), max(1, int(n.max(initial=0)))
    perm = rng.permutation(max(1, total)).astype(np.int32)
    first = np.concatenate([[0], np.cumsum(n.reshape(-1))])[:-1].reshape(n.shape)
    col = np.arange(W)
    live = col < n[..., None]
    table = np.where(live, perm[np.where(live, first[..., None] + col, 0)], -1).astype(np.int32)
    return (table if local else table[0]), max(1, total)


def _quantise(x):
    """FP8 E4M3 rows with power-of-two scales: the cache's format."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = e - (m == 0.5).to(e.dtype) - 8
    s = torch.ldexp(torch.ones_like(m), torch.where(m > 0, e, torch.zeros_like(e)))
    return (x / s[:, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = DEVICE
    seed = int(seed) & 0x7FFFFFFF
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    return {"extend": _prepare_extend, "rope": _prepare_rope, "chunk": _prepare_chunk}[case["op"]](case, g, rng, dev)


def _prepare_extend(case, g, rng, dev):
    ctx, q = _lengths(case)
    B, D, I, bs = case["B"], case["D"], case["I"], case["bs"]
    seq = [c + n for c, n in zip(ctx, q)]
    if B > 3:
        seq[3] = 0  # a slot of the batch that holds no request: its rows are padding
    old = [max(0, s - n) for s, n in zip(seq, q)]
    table, used = _paged(old, bs, D, I, case["local"], rng)
    # room for the new blocks, as a serving program sizes its tables
    wide = -(-max(seq) // bs) if not case["local"] else max(-(-_owned(s, d, D, I) // bs) for s in seq for d in range(D))
    grown = np.full(table.shape[:-1] + (wide + 3,), -1, dtype=np.int32)
    w = min(table.shape[-1], wide)
    grown[..., :w] = table[..., :w]
    need = sum(q) + B * D + 8
    free = (used + rng.permutation(need)).astype(np.int32)

    def on(x, t):
        return torch.tensor(np.asarray(x), dtype=t, device=dev)

    return dict(case=case, table=on(grown, torch.int32), seq=on(seq, torch.int32),
                qsl=on(np.concatenate([[0], np.cumsum(q)]), torch.int32), free=on(free, torch.int32),
                count=on([need - 3], torch.int32), left=on([0], torch.int32), T=int(sum(q)) + 2)


def _prepare_rope(case, g, rng, dev):
    T, H, bs, top = case["T"], case["H"], case["bs"], case["top"]
    x = torch.empty((T, KDIM), device=dev).normal_(generator=g)
    # the down projection's output: latent and rope part side by side
    kv = (2.5 * x).to(torch.bfloat16)
    nb = (T + 37 + bs - 1) // bs
    slots = torch.randperm(nb * bs, generator=g, device=dev)[:T]
    slots = torch.where(torch.arange(T, device=dev) % 16 == 15, torch.full_like(slots, -1), slots)
    i = torch.arange(ROPE // 2, device=dev, dtype=torch.float64)
    angle = torch.arange(top, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / ROPE)
    st = dict(case=case, kv_c=kv[:, :LATENT], k_pe=kv[:, LATENT:], slots=slots, num_slots=nb * bs,
              cos_sin=torch.cat([angle.cos(), angle.sin()], dim=1).float(),
              positions=torch.randint(0, top, (T,), generator=g, device=dev).to(torch.int32),
              weight=(1.0 + 0.2 * torch.empty(LATENT, device=dev).normal_(generator=g)).to(torch.bfloat16)
              if case["norm"] else None)
    if case["fp8"]:
        # one row past the cache takes what the plain form must not write
        codes = torch.zeros((nb * bs + 1, KDIM), dtype=torch.uint8, device=dev)
        scale = torch.ones(nb * bs + 1, device=dev)
        st.update(rows=codes, scales=scale, cache=codes[:nb * bs].view(nb, bs, KDIM), scale=scale[:nb * bs].view(nb, bs))
    else:
        rows = torch.zeros((nb * bs + 1, KDIM), dtype=torch.bfloat16, device=dev)
        st.update(rows=rows, cache=rows[:nb * bs].view(nb, bs, KDIM), scale=None)
    if case["query"] == "decode":
        # the transposed output of a per-head matmul, and a plain projection
        y = torch.empty((H, T, LATENT), dtype=torch.bfloat16, device=dev).normal_(generator=g)
        st["ql_nope"] = y.transpose(0, 1)
        st["q_pe"] = torch.empty((T, H, ROPE), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    elif case["query"] == "pe":
        # the query projection's output [T, H, 192]; the rotated parts go to the query that attends
        st["q_pe"] = torch.empty((T, H, NOPE + ROPE), dtype=torch.bfloat16, device=dev).normal_(generator=g)[..., NOPE:]
        st["q_out"] = torch.zeros((T, H, NOPE + ROPE), dtype=torch.bfloat16, device=dev)[..., NOPE:]
    return st


def _prepare_chunk(case, g, rng, dev):
    ctx, q = _lengths(case)
    H, bs = case["H"], case["bs"]
    seq = [c + n for c, n in zip(ctx, q)]
    table, nb = _paged(seq, bs, case["D"], case["I"], case["local"], rng)
    x = torch.empty((nb * bs, KDIM), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    # a request's first block draws more attention than the others
    first = torch.from_numpy(np.ascontiguousarray(table[0, :, 0] if case["local"] else table[:, 0])).to(dev).long()
    first = first[first >= 0]
    u = torch.cos(torch.arange(ROPE, device=dev, dtype=torch.float32) * 1.7)
    u = 6.0 * u / u.norm()
    x[first * bs, LATENT:] += u.to(torch.bfloat16)
    st = dict(case=case, seqs=seq, qs=q, scale=None, table=torch.from_numpy(table).to(dev),
              seq=torch.tensor(seq, dtype=torch.int32, device=dev),
              qsl=torch.tensor(np.concatenate([[0], np.cumsum(q)]), dtype=torch.int32, device=dev),
              T=sum(q) + case["pad"], total=sum(seq))
    if case["fp8"]:
        parts = [_quantise(c.float()) for c in x.split(1 << 18)]
        st["cache"] = torch.cat([p[0].view(torch.uint8) for p in parts]).view(nb, bs, KDIM)
        st["scale"] = torch.cat([p[1] for p in parts]).view(nb, bs)
    else:
        st["cache"] = x.view(nb, bs, KDIM)
    y = torch.empty((st["T"], H, NOPE + ROPE), dtype=torch.float32, device=dev).normal_(generator=g)
    y[..., NOPE:] += u
    st["q"] = (1.5 * y).to(torch.bfloat16)
    # the up projection's weight, a head's 128 key rows before its 128 value rows
    w = torch.empty((H * (NOPE + VDIM), LATENT), dtype=torch.float32, device=dev).normal_(generator=g)
    st["w"] = (w / math.sqrt(LATENT)).to(torch.bfloat16)
    if own:
        import mla_decode_context_gb300 as dcp
        st["packed"] = dcp.pack_kv_b(st["w"], H)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    return {"extend": _plain_extend, "rope": _plain_rope, "chunk": _plain_chunk}[op](st)


def _own(st, op):
    import mla_decode_context_gb300 as dcp
    c = st["case"]
    if op == "extend":
        pos, slots = dcp.cache_extend(st["table"], st["seq"], st["qsl"], st["free"], st["count"], st["T"], c["bs"],
                                      free_left=st["left"], D=c["D"], interleave=c["I"])
        return st["table"], pos, slots, st["left"]
    if op == "rope":
        q = dcp.norm_rope_cache(st["kv_c"], st["k_pe"], st["slots"], st["cache"], st["positions"], st["cos_sin"],
                                norm_weight=st["weight"], eps=EPS, ql_nope=st.get("ql_nope"), q_pe=st.get("q_pe"),
                                q_out=st.get("q_out"), interleaved=c["pairs"], kv_scale=st["scale"])
        out = () if q is None else (q,)
        return out + ((st["cache"].view(torch.float8_e4m3fn), st["scale"]) if c["fp8"] else (st["cache"],))
    return dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], st["packed"], scale=SCALE,
                               total_len=st["total"], kv_scale=st["scale"], D=c["D"], interleave=c["I"])


def _plain_extend(st):
    c = st["case"]
    D, I, bs, B = c["D"], c["I"], c["bs"], c["B"]
    dev = st["seq"].device
    seq, qsl = st["seq"].long(), st["qsl"].long()
    n = qsl[1:] - qsl[:-1]
    seq = seq.clamp(min=0)
    old = (seq - n).clamp(min=0)

    def blocks(x):  # blocks that a request's first x positions take in each table: [B] or [B, D]
        if not c["local"]:
            return (x + bs - 1) // bs
        x = x[:, None]
        own_ = x // (D * I) * I + (x % (D * I) - torch.arange(D, device=dev) * I).clamp(0, I)
        return (own_ + bs - 1) // bs

    table = st["table"]
    W = table.shape[-1]
    flat = table.view(-1, W) if not c["local"] else table.transpose(0, 1).reshape(-1, W)  # rows in order (b, d)
    b0, b1 = blocks(old).reshape(-1), blocks(seq).reshape(-1)
    take = b1 - b0
    end = take.cumsum(0)
    col = torch.arange(W, device=dev)
    new = (col >= b0[:, None]) & (col < b1[:, None])
    k = (end - take)[:, None] + col - b0[:, None]
    count = st["count"].long()
    at = count - 1 - k
    ids = torch.where(at >= 0, st["free"].long()[at.clamp(0, st["free"].numel() - 1)], torch.full_like(at, -1))
    flat = torch.where(new, ids, flat.long()).to(torch.int32)
    table.copy_(flat.view(B, D, W).transpose(0, 1) if c["local"] else flat.view(B, W))
    st["left"].copy_((count - end[-1]).clamp(min=0))

    t = torch.arange(st["T"], device=dev)
    b = (torch.searchsorted(qsl, t, right=True) - 1).clamp(0, B - 1)
    p = seq[b] - n[b] + t - qsl[b]
    ok = (t < qsl[-1]) & (seq[b] > 0) & (p >= 0)
    pc = p.clamp(min=0)
    d = pc // I % D
    if c["local"]:
        j = pc // (D * I) * I + pc % I
        blk = table[d, b, (j // bs).clamp(max=W - 1)].long()
    else:
        j = pc
        blk = table[b, (j // bs).clamp(max=W - 1)].long()
    none = torch.full_like(p, -1)
    slots = torch.where(ok & (blk >= 0), blk * bs + j % bs, none)
    return table, torch.where(ok, p, none).to(torch.int32), slots, st["left"]


def _rotate(x, cs, pairs):
    """x [..., 64] turned by the angles whose [cos | sin] are cs [..., 64]."""
    half = ROPE // 2
    c, s = cs[..., :half], cs[..., half:]
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :half], x[..., half:])
    u, v = a * c - b * s, b * c + a * s
    return torch.stack([u, v], dim=-1).flatten(-2) if pairs else torch.cat([u, v], dim=-1)


def _plain_rope(st):
    c = st["case"]
    cs = st["cos_sin"][st["positions"].long()]
    x = st["kv_c"].double()  # (the FP8 scale and codes lie next to borders)
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * st["weight"].double()
    row = torch.cat([x, _rotate(st["k_pe"].double(), cs.double(), c["pairs"])], dim=1)
    at = torch.where(st["slots"] >= 0, st["slots"], torch.full_like(st["slots"], st["num_slots"]))
    if c["fp8"]:
        m, e = torch.frexp(row.abs().amax(1))
        e = e - (m == 0.5).to(e.dtype) - 8  # the least e with max |x| <= 256 * 2^e
        s = torch.ldexp(torch.ones_like(m), torch.where(m > 0, e, torch.zeros_like(e)))
        st["rows"].index_copy_(0, at, (row / s[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8))
        st["scales"].index_copy_(0, at, s.float())
        out = (st["cache"].view(torch.float8_e4m3fn), st["scale"])
    else:
        st["rows"].index_copy_(0, at, row.float().to(torch.bfloat16))
        out = (st["cache"],)
    if c["query"] == "none":
        return out
    q = _rotate(st["q_pe"].float(), cs[:, None, :], c["pairs"]).to(torch.bfloat16)
    if c["query"] == "pe":
        st["q_out"].copy_(q)
        return (st["q_out"],) + out
    return (torch.cat([st["ql_nope"], q], dim=2),) + out


def _cache_rows(st, b, p):
    """Cache rows of positions p of request b."""
    c = st["case"]
    bs, D, I = c["bs"], c["D"], c["I"]
    if c["local"]:
        j = p // (D * I) * I + p % I
        return st["table"][p // I % D, b, j // bs].long() * bs + j % bs
    return st["table"][b, p // bs].long() * bs + p % bs


def _plain_chunk(st):
    c = st["case"]
    H, dev = c["H"], st["q"].device
    flat = st["cache"].view(-1, KDIM)
    out = torch.zeros((st["T"], H, VDIM), dtype=torch.bfloat16, device=dev)
    lse = torch.full((st["T"], H), -math.inf, device=dev)
    r0 = 0
    for b, (L, n) in enumerate(zip(st["seqs"], st["qs"])):
        p = torch.arange(L, device=dev)
        rows = _cache_rows(st, b, p)
        kv = flat[rows].float() if st["scale"] is None else \
            flat[rows].view(torch.float8_e4m3fn).float() * st["scale"].view(-1)[rows][:, None]
        last = L - n + torch.arange(n, device=dev)  # row i sees the positions up to its own
        hidden = p[None, :] > last[:, None]
        step = max(1, min(H, (1 << 30) // (n * L)))
        for h in range(0, H, step):
            w = st["w"].view(H, NOPE + VDIM, LATENT)[h:h + step].float()
            up = torch.matmul(kv[:, :LATENT], w.transpose(1, 2))  # [heads, L, 256]
            q = st["q"][r0:r0 + n, h:h + step].float().transpose(0, 1)
            s = torch.matmul(q[..., :NOPE], up[..., :NOPE].transpose(1, 2))
            s = (s + torch.matmul(q[..., NOPE:], kv[:, LATENT:].t())).mul_(SCALE)
            s.masked_fill_(hidden, -math.inf)
            m = s.amax(-1, keepdim=True)
            e = s.sub_(m).exp_()
            l = e.sum(-1, keepdim=True)
            o = torch.matmul(e, up[..., NOPE:]) / l
            out[r0:r0 + n, h:h + step] = o.transpose(0, 1).to(torch.bfloat16)
            lse[r0:r0 + n, h:h + step] = (m + l.log())[..., 0].t()
        r0 += n
    return out, lse


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "rope":
        T, H = case["T"], case["H"]
        live = T - T // 16
        q = {"none": 0, "decode": 4 * KDIM, "pe": 4 * ROPE}[case["query"]]
        return {"bytes": T * (2 * KDIM + 8 + 4 + 4 * ROPE + H * q) + live * (KDIM + 4 if case["fp8"] else 2 * KDIM),
                "flops": T * (4 * LATENT + 3 * ROPE * (1 + H))}
    ctx, q = _lengths(case)
    if case["op"] == "extend":
        bs, D, I = case["bs"], case["D"], case["I"]
        new = sum(-(-(c + n) // bs) - -(-c // bs) if not case["local"] else
                  sum(-(-_owned(c + n, d, D, I) // bs) - -(-_owned(c, d, D, I) // bs) for d in range(D))
                  for c, n in zip(ctx, q))
        return {"bytes": 8 * case["B"] + 8 * new + 12 * sum(q), "flops": sum(q)}
    H = case["H"]
    flops = 0
    for c, n in zip(ctx, q):
        pairs = n * c + n * (n + 1) // 2
        up = 2 * LATENT * (NOPE + VDIM)
        # keys and values projected up for each position, or queries and outputs taken to the latents' space
        flops += H * min(2 * (NOPE + ROPE + VDIM) * pairs + up * (c + n), 2 * (KDIM + LATENT) * pairs + up * n)
    T = sum(q) + case["pad"]
    return {"bytes": sum(c + n for c, n in zip(ctx, q)) * (KDIM + 4 if case["fp8"] else 2 * KDIM)
            + H * (NOPE + VDIM) * LATENT * 2 + T * H * (2 * (NOPE + ROPE) + 2 * VDIM + 4), "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "chunk":
        ctx, q = _lengths(case)
        if case["H"] * sum((c + n) * (640 * n + 262144) for c, n in zip(ctx, q)) > 7e12:
            return None
    st = prepare(case, seed)
    return {"extend": _exact_extend, "rope": _exact_rope, "chunk": _exact_chunk}[case["op"]](case, st)


def _exact_extend(case, st):
    bs, D, I = case["bs"], case["D"], case["I"]
    table = st["table"].cpu().numpy().copy()
    seq, qsl, free = (st[k].cpu().numpy() for k in ("seq", "qsl", "free"))
    left = int(st["count"][0])
    pos = np.full(st["T"], -1, dtype=np.int32)
    slots = np.full(st["T"], -1, dtype=np.int64)
    for b in range(case["B"]):
        n, L = int(qsl[b + 1] - qsl[b]), int(seq[b])
        if L <= 0:
            continue
        for d in range(D if case["local"] else 1):
            row = table[d, b] if case["local"] else table[b]
            have, want = ((_owned(x, d, D, I) if case["local"] else x) for x in (max(0, L - n), L))
            for col in range(-(-have // bs), -(-want // bs)):
                left -= 1
                row[col] = free[left]
        for i in range(n):
            p = L - n + i
            if p < 0:
                continue
            pos[qsl[b] + i] = p
            if case["local"]:
                j = p // (D * I) * I + p % I
                blk = table[p // I % D, b, j // bs]
            else:
                j, blk = p, table[b, p // bs]
            slots[qsl[b] + i] = int(blk) * bs + j % bs
    return table, pos, slots, np.array([left], dtype=np.int32)


def _exact_rope(case, st):
    x = st["kv_c"].double().cpu().numpy()
    if case["norm"]:
        x = x / np.sqrt(np.sum(x * x, 1, keepdims=True) / LATENT + EPS) * st["weight"].double().cpu().numpy()
    cs = st["cos_sin"].double().cpu().numpy()[st["positions"].cpu().numpy()]
    turn = cs[:, :ROPE // 2] + 1j * cs[:, ROPE // 2:]

    def rotated(y, turn):
        z = (y[..., 0::2] + 1j * y[..., 1::2] if case["pairs"] else y[..., :ROPE // 2] + 1j * y[..., ROPE // 2:]) * turn
        out = np.empty(y.shape)
        if case["pairs"]:
            out[..., 0::2], out[..., 1::2] = z.real, z.imag
        else:
            out[..., :ROPE // 2], out[..., ROPE // 2:] = z.real, z.imag
        return out

    row = np.concatenate([x, rotated(st["k_pe"].double().cpu().numpy(), turn)], 1)
    slots = st["slots"].cpu().numpy()
    live = slots >= 0
    shape = tuple(st["cache"].shape)
    if case["fp8"]:
        # every non-negative E4M3 value in order, its index being its code
        grid = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127])
        top = np.abs(row).max(1)
        s = np.where(top > 0, np.exp2(np.ceil(np.log2(np.where(top > 0, top, 1.0))) - 8), 1.0)
        s = np.where((top > 0) & (top > 256 * s), 2 * s, s)
        a = np.abs(row) / s[:, None]
        up = np.clip(np.searchsorted(grid, a, side="left"), 1, 126)
        mid = (grid[up] + grid[up - 1]) / 2
        code = np.where(a > mid, up, np.where(a < mid, up - 1, np.where(up % 2 == 0, up, up - 1)))
        codes, scales = np.zeros((st["num_slots"], KDIM)), np.ones(st["num_slots"])
        codes[slots[live]] = np.copysign(grid[code], row)[live]
        scales[slots[live]] = s[live]
        out = (codes.reshape(shape), scales.reshape(shape[:2]))
    else:
        rows = np.zeros((st["num_slots"], KDIM))
        rows[slots[live]] = row[live]
        out = (rows.reshape(shape),)
    if case["query"] == "none":
        return out
    q = rotated(st["q_pe"].double().cpu().numpy(), turn[:, None, :])
    if case["query"] == "decode":
        q = np.concatenate([st["ql_nope"].double().cpu().numpy(), q], 2)
    return (q,) + out


def _exact_chunk(case, st):
    H, bs, D, I = case["H"], case["bs"], case["D"], case["I"]
    dev = st["q"].device
    table = st["table"].cpu().numpy().astype(np.int64)
    qsl = st["qsl"].cpu().numpy()
    flat = st["cache"].reshape(-1, KDIM)
    out = torch.zeros((st["T"], H, VDIM), dtype=torch.float64, device=dev)
    lse = torch.full((st["T"], H), -math.inf, dtype=torch.float64, device=dev)
    for b in range(case["B"]):
        L, n = int(st["seq"][b]), int(qsl[b + 1] - qsl[b])
        pos = np.arange(L)
        if case["local"]:
            j = pos // (D * I) * I + pos % I
            at = table[pos // I % D, b, j // bs] * bs + j % bs
        else:
            at = table[b, pos // bs] * bs + pos % bs
        at = torch.from_numpy(at).to(dev)
        if st["scale"] is None:
            kv = flat[at].double()
        else:
            kv = flat[at].view(torch.float8_e4m3fn).double() * st["scale"].reshape(-1)[at][:, None].double()
        sees = torch.ones((n, L), dtype=torch.bool, device=dev).tril(L - n)
        for h in range(H):
            w = st["w"][h * (NOPE + VDIM):(h + 1) * (NOPE + VDIM)].double()
            k = torch.cat([kv[:, :LATENT] @ w[:NOPE].T, kv[:, LATENT:]], dim=1)
            v = kv[:, :LATENT] @ w[NOPE:].T
            s = SCALE * (st["q"][qsl[b]:qsl[b + 1], h].double() @ k.T)
            s = torch.where(sees, s, torch.full_like(s, -math.inf))
            z = torch.logsumexp(s, 1)
            lse[qsl[b]:qsl[b + 1], h] = z
            out[qsl[b]:qsl[b + 1], h] = torch.exp(s - z[:, None]) @ v
    return out, lse
