"""What is measured of the 4-bit latent cache: its write (append), its read
back, attention over the selected blocks of it and attention over all of it.

The cache holds a 512-wide latent row as 512 E2M1 codes (two to a byte, the
even dim in the low half) and 16 scale bytes, one for each group of 32 dims:
byte = e + 127, value = code value * 2^e.  A row's group exponents are the
smallest integers with max |x| <= 6 * 2^e, raised to within 15 of the row's
largest, which itself lies in [-50, 50].
"""
import math

import torch

own = False

LATENT, GROUPS, TOPK, POOL = 512, 16, 512, 4

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token for each of four sequences: a decode step's cache write
        {"name": "append step 4", "op": "append", "B": 4, "n_new": 1, "cap": 8192, "ragged": False},
        # a padded batch of prompts of up to 1536 tokens
        {"name": "append prompts 64x1536", "op": "append", "B": 64, "n_new": 1536, "cap": 1536,
         "ragged": True},
        # the rows of one selection of each sequence, out of 131072 cached tokens
        {"name": "read selection 4x2051", "op": "read", "B": 4, "m": 2051, "cap": 131072,
         "scattered": True},
        # the beginning of every sequence, of unequal lengths (an odd number of rows)
        {"name": "read prefix 16x8191", "op": "read", "B": 16, "m": 8191, "cap": 8192,
         "scattered": False},
        # decode, one sequence of 8192 tokens, 16 heads
        {"name": "sparse 1x8192 h16", "op": "sparse", "rows": 1, "n": 8192, "heads": 16,
         "shared": False, "ragged": False},
        # decode, four sequences of a million tokens, 64 heads
        {"name": "sparse 4x1M h64", "op": "sparse", "rows": 4, "n": 1048576, "heads": 64,
         "shared": False, "ragged": False},
        # decode, sixteen sequences of unequal lengths, 128 heads
        {"name": "sparse 16x128K h128", "op": "sparse", "rows": 16, "n": 131072, "heads": 128,
         "shared": False, "ragged": True},
        # a quarter of a 4096-token prefill chunk on a 131072-token cache
        {"name": "sparse chunk 1024 h64", "op": "sparse", "rows": 1024, "n": 131072, "heads": 64,
         "shared": True, "ragged": True},
        # attention over a short cache, one sequence
        {"name": "latent 1x515 h16", "op": "latent", "seqs": 1, "per_seq": 1, "n": 515, "heads": 16},
        # decode over short caches of unequal lengths
        {"name": "latent 64x1536 h64", "op": "latent", "seqs": 64, "per_seq": 1, "n": 1536,
         "heads": 64},
        # three draft tokens a sequence, 16 heads (a quarter of the layer's heads on each device)
        {"name": "latent 16x32K h16 x3", "op": "latent", "seqs": 16, "per_seq": 3, "n": 32768,
         "heads": 16},
        # decode over all of a million tokens of four sequences
        {"name": "latent 4x1M h64", "op": "latent", "seqs": 4, "per_seq": 1, "n": 1048576,
         "heads": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "sparse", "sparse", "latent", "latent"])
    if op == "append":
        B = _log(rng, 1, 64)
        n_new = _log(rng, 1, 98304 // B)
        return {"op": op, "B": B, "n_new": n_new, "cap": n_new + rng.randint(1, 2000),
                "ragged": rng.random() < 0.5}
    if op == "read":
        B = _log(rng, 1, 16)
        m = _log(rng, 1, 131056 // B)
        return {"op": op, "B": B, "m": m, "cap": max(m, _log(rng, 16, 131072)),
                "scattered": rng.random() < 0.5}
    heads = rng.choice([16, 32, 48, 64, 64, 80, 128])
    if op == "sparse":
        shared = rng.random() < 0.5
        rows = _log(rng, 1, 1024 * 64 // max(64, heads)) if shared else _log(rng, 1, 16)
        return {"op": op, "rows": rows, "n": _log(rng, 1, 131072 if shared or rows > 4 else 1048576),
                "heads": heads, "shared": shared, "ragged": rng.random() < 0.7}
    seqs = _log(rng, 1, 64)
    per_seq = rng.choice([1, 1, 2, 3, 4])
    most = 4 * 1048576 * 64 // (seqs * per_seq * heads)
    return {"op": op, "seqs": seqs, "per_seq": per_seq,
            "n": _log(rng, 1, min(1048576, 4 * 1048576 // seqs, most)), "heads": heads}


def work(case):
    op = case["op"]
    if op == "append":
        # a ragged batch holds 1 .. n_new rows a sequence
        rows = case["B"] * (0.5 * (case["n_new"] + 1) if case["ragged"] else case["n_new"])
        return {"bytes": rows * (1024 + 272 + 1024), "flops": rows * LATENT * 2}
    if op == "read":
        rows = case["B"] * case["m"]
        # rows behind a sequence's end (1 .. cap tokens) are zeros and read nothing
        read = rows if case["scattered"] else rows * (1 - 0.5 * case["m"] / case["cap"])
        return {"bytes": read * 272 + rows * 1024 + (rows * 8 if case["scattered"] else 0),
                "flops": rows * LATENT}
    H = case["heads"]
    if op == "sparse":
        n = case["n"] * (0.75 if case["ragged"] and not case["shared"] else 1.0)
        tok = min(n, TOPK * POOL + (1.5 if case["ragged"] else n % POOL))
        # a shared cache is read once, however many rows attend to the same token
        seen = min(case["rows"] * tok, case["n"]) if case["shared"] else case["rows"] * tok
        return {"bytes": seen * 272 + case["rows"] * (H * 2052 + TOPK * 4),
                "flops": case["rows"] * tok * H * LATENT * 4}
    rows, n = case["seqs"] * case["per_seq"], case["n"] * 0.75
    return {"bytes": case["seqs"] * n * 272 + rows * H * 2052, "flops": rows * n * H * LATENT * 4}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _cache(g, seqs, cap):
    """A filled cache: E2M1 codes with the frequencies of a normal variable whose
    group maximum is near 5, exponents that vary by group and by row."""
    dev = "cuda"
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=dev)
    u = (torch.arange(256, dtype=torch.float64, device=dev) + 0.5) / 256
    x = torch.erfinv(2 * u - 1) * math.sqrt(2.0) * 2.3
    lut = (torch.bucketize(x.abs(), edges) + 8 * (x < 0)).to(torch.uint8)
    codes = torch.empty(seqs, cap, LATENT // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(seqs, cap, GROUPS, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // (LATENT // 2))
    for b in range(seqs):
        for t0 in range(0, cap, step):
            t1 = min(cap, t0 + step)
            r = torch.randint(0, 256, (2, t1 - t0, LATENT // 2), generator=g, device=dev,
                              dtype=torch.uint8)
            codes[b, t0:t1] = lut[r[0].int()] | (lut[r[1].int()] << 4)
    row = torch.randint(125, 128, (seqs, cap, 1), generator=g, device=dev, dtype=torch.uint8)
    low = torch.randint(0, 8, (seqs, cap, GROUPS), generator=g, device=dev, dtype=torch.uint8)
    scales.copy_(row - (low > 3).to(torch.uint8) - (low > 6).to(torch.uint8))
    scales[..., 0:1] = row
    return codes, scales


def _query(g, rows, heads):
    # scaled by 1/sqrt(512), as the layer folds it into the query; the values of a
    # cached row have a spread of about 1/2 to 2
    q = torch.randn(rows, heads, LATENT, generator=g, device="cuda")
    return (q / math.sqrt(LATENT)).to(torch.bfloat16)


def prepare(case, seed):
    g, dev, op = _gen(seed), "cuda", case["op"]
    st = {"op": op}
    if op == "append":
        B, n_new, cap = case["B"], case["n_new"], case["cap"]
        x = torch.randn(B, n_new, LATENT, generator=g, device=dev)
        x *= torch.exp2(torch.randint(-3, 2, (1, 1, GROUPS), generator=g, device=dev)
                        .float()).repeat_interleave(32, -1)  # channels differ in spread
        x *= torch.exp2(torch.randn(B, n_new, 1, generator=g, device=dev) * 0.5)
        st["latent"] = x.to(torch.bfloat16)
        st["codes"], st["scales"] = _cache(g, B, cap)
        room = cap - n_new
        st["len"] = torch.randint(0, room + 1, (B,), generator=g, device=dev)
        st["n_add"] = (torch.randint(1, n_new + 1, (B,), generator=g, device=dev, dtype=torch.int32)
                       if case["ragged"] else None)
        st["stored"] = torch.zeros(B, n_new, LATENT, dtype=torch.bfloat16, device=dev)
    elif op == "read":
        B, m, cap = case["B"], case["m"], case["cap"]
        st["codes"], st["scales"] = _cache(g, B, cap)
        if case["scattered"]:
            st["n_vis"] = torch.full((B,), cap, dtype=torch.int64, device=dev)
            st["pos"] = torch.sort(torch.randint(0, cap, (B, m), generator=g, device=dev), -1)[0]
        else:
            st["n_vis"] = torch.randint(1, cap + 1, (B,), generator=g, device=dev)
            st["pos"] = None
        st["out"] = torch.empty(B, m, LATENT, dtype=torch.bfloat16, device=dev)
    elif op == "sparse":
        rows, n, H = case["rows"], case["n"], case["heads"]
        st["codes"], st["scales"] = _cache(g, 1 if case["shared"] else rows, n)
        if not case["ragged"]:
            n_vis = torch.full((rows,), n, dtype=torch.int64, device=dev)
        elif case["shared"]:  # a causal chunk: every row sees one token more
            n_vis = torch.clamp(torch.arange(n - rows + 1, n + 1, device=dev), min=1)
        else:
            n_vis = torch.randint((n + 1) // 2, n + 1, (rows,), generator=g, device=dev)
        st["n_vis"] = n_vis
        nblk = n_vis // POOL
        count = torch.clamp(nblk, max=TOPK)
        # distinct blocks spread over the row: one from each of `count` equal parts
        j = torch.arange(TOPK, device=dev)[None]
        c = torch.clamp(count, min=1)[:, None]
        lo, hi = j * nblk[:, None] // c, (j + 1) * nblk[:, None] // c
        pick = lo + (torch.rand(rows, TOPK, generator=g, device=dev) * (hi - lo)).long()
        st["idx"] = torch.where(j < count[:, None], pick, -1).to(torch.int32)
        st["count"] = count.to(torch.int32)
        st["q"] = _query(g, rows, H)
        st["seq_stride"] = 0 if case["shared"] else n * LATENT
    else:
        seqs, per, n, H = case["seqs"], case["per_seq"], case["n"], case["heads"]
        st["codes"], st["scales"] = _cache(g, seqs, n)
        last = torch.randint((n + 1) // 2, n + 1, (seqs, 1), generator=g, device=dev)
        st["n_vis"] = torch.clamp(last - torch.arange(per - 1, -1, -1, device=dev)[None],
                                  min=0).reshape(-1).contiguous()
        st["q"], st["per_seq"] = _query(g, seqs * per, H), per
    if op in ("sparse", "latent"):
        st["n"] = case["n"]
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(st["q"].shape[:2], device=dev)
        if own:  # the handle and the workspace a program keeps
            import long_context_decode_indexpool_b200 as spx
            st["d"] = spx.dims(case["heads"], 1.0)
            rows = st["q"].shape[0]
            need = (spx.spx_attn_fp4_workspace_size(st["d"], rows, st["n"]) if op == "sparse" else
                    spx.spx_latent_attn_fp4_workspace_size(st["d"], rows, st["per_seq"], st["n"]))
            st["ws"] = spx.workspace(need, dev)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    import long_context_decode_indexpool_b200 as spx
    op = st["op"]
    if op == "append":
        B, n_new = st["latent"].shape[:2]
        cap = st["codes"].shape[1]
        spx.spx_latent_append_fp4(B, st["latent"], n_new, st["n_add"], st["codes"], st["scales"],
                                  cap, st["len"], cap, st["stored"])
        return {"stored": st["stored"], "codes": st["codes"], "scales": st["scales"]}
    if op == "read":
        B, m = st["out"].shape[:2]
        spx.spx_latent_read_fp4(B, st["codes"], st["scales"], st["codes"].shape[1], st["pos"], m,
                                st["n_vis"], st["out"])
        return st["out"]
    rows = st["q"].shape[0]
    if op == "sparse":
        spx.spx_sparse_mla_attn_fp4(st["d"], rows, st["q"], st["codes"], st["scales"],
                                    st["seq_stride"], st["n"], st["idx"], st["count"], st["n_vis"],
                                    st["n"], st["out"], st["lse"], st["ws"])
    else:
        spx.spx_latent_attn_fp4(st["d"], rows, st["per_seq"], st["q"], st["codes"], st["scales"],
                                st["n"], st["n_vis"], st["n"], st["out"], st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _dequant(codes, scales):
    """fp32 rows [..., 512] of codes [..., 256] and scales [..., 16]."""
    v = torch.tensor(_VALUES, device=codes.device)
    v = torch.cat([v, -v])
    pair = torch.stack([v.repeat(16), v.repeat_interleave(16)], -1)  # value pair of a code byte
    x = pair[codes.int()].reshape(*codes.shape[:-1], GROUPS, 32)
    x = x * torch.exp2(scales.float() - 127.0)[..., None]
    return x.reshape(*codes.shape[:-1], LATENT)


def _attend(q, c, keep):
    """softmax attention of q [R, H, 512] over rows c [R or 1, T, 512], where keep [R, T]."""
    s = torch.matmul(q.float(), c.transpose(-1, -2))
    s = torch.where(keep[:, None], s, torch.full((), -math.inf, device=s.device))
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros((), device=s.device))
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, c) / torch.where(l > 0, l, torch.ones((), device=s.device))
    lse = (m + torch.log(l)).squeeze(-1)
    return out.to(torch.bfloat16), lse


def _plain(st):
    op = st["op"]
    if op == "append":
        x = st["latent"].float()
        B, n_new = x.shape[:2]
        g = x.reshape(B, n_new, GROUPS, 32)
        mant, exp = torch.frexp(g.abs().amax(-1))
        nat = torch.where(mant <= 0.75, exp - 3, exp - 2)
        nat = torch.where(mant == 0, torch.full_like(nat, -1000), nat)
        top = torch.clamp(nat.amax(-1, keepdim=True), -50, 50)
        e = torch.minimum(torch.maximum(nat, top - 15), top)
        a = torch.abs(g) * torch.exp2(-e.float())[..., None]
        c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
             + (a >= 3.5) + (a > 5.0))
        val = torch.tensor(_VALUES, device=x.device)[c.int()] * torch.exp2(e.float())[..., None]
        val = torch.copysign(val, g).reshape(B, n_new, LATENT).to(torch.bfloat16)
        c = (c | (torch.signbit(g).to(torch.uint8) << 3)).reshape(B, n_new, LATENT)
        byte = c[..., 0::2] | (c[..., 1::2] << 4)
        i = torch.arange(n_new, device=x.device)[None]
        at = (st["len"][:, None] + i)
        if st["n_add"] is None:
            b = torch.arange(B, device=x.device)[:, None].expand_as(at)
            st["codes"][b, at] = byte
            st["scales"][b, at] = (e + 127).to(torch.uint8)
            st["stored"].copy_(val)
        else:
            keep = i < st["n_add"][:, None]
            b = torch.arange(B, device=x.device)[:, None].expand_as(at)
            st["codes"][b[keep], at[keep]] = byte[keep]
            st["scales"][b[keep], at[keep]] = (e + 127).to(torch.uint8)[keep]
            st["stored"].copy_(torch.where(keep[..., None], val, st["stored"]))
        return {"stored": st["stored"], "codes": st["codes"], "scales": st["scales"]}
    if op == "read":
        B, m = st["out"].shape[:2]
        if st["pos"] is None:
            codes, scales = st["codes"][:, :m], st["scales"][:, :m]
            keep = torch.arange(m, device=codes.device)[None] < st["n_vis"][:, None]
        else:
            b = torch.arange(B, device=st["pos"].device)[:, None]
            codes, scales = st["codes"][b, st["pos"]], st["scales"][b, st["pos"]]
            keep = st["pos"] < st["n_vis"][:, None]
        x = _dequant(codes, scales)
        st["out"].copy_(torch.where(keep[..., None], x, torch.zeros((), device=x.device)))
        return st["out"]
    if op == "sparse":
        rows, dev = st["q"].shape[0], st["q"].device
        blk, n = st["idx"].long(), st["n_vis"][:, None]
        tok = (blk[..., None] * POOL + torch.arange(POOL, device=dev)).reshape(rows, -1)
        keep = (blk >= 0).repeat_interleave(POOL, -1)
        tail = n // POOL * POOL + torch.arange(POOL - 1, device=dev)[None]
        tok, keep = torch.cat([tok, tail], -1), torch.cat([keep, tail < n], -1)
        tok = torch.where(keep, tok, torch.zeros_like(tok))
        b = torch.arange(rows, device=dev)[:, None] if st["seq_stride"] else torch.zeros_like(n)
        c = _dequant(st["codes"][b, tok], st["scales"][b, tok])
        out, lse = _attend(st["q"], c, keep)
    else:
        per, (rows, H) = st["per_seq"], st["q"].shape[:2]
        c = _dequant(st["codes"], st["scales"])
        q = st["q"].reshape(rows // per, per * H, LATENT)
        s_keep = torch.arange(st["n"], device=q.device)[None] < st["n_vis"][:, None]
        keep = s_keep.reshape(rows // per, per, 1, -1).expand(-1, -1, H, -1)
        s = torch.matmul(q.float(), c.transpose(-1, -2)).reshape(rows // per, per, H, -1)
        s = torch.where(keep, s, torch.full((), -math.inf, device=s.device))
        m = s.amax(-1, keepdim=True)
        m = torch.where(torch.isfinite(m), m, torch.zeros((), device=s.device))
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        out = torch.matmul(p.reshape(rows // per, per * H, -1), c).reshape(rows, H, LATENT)
        l1 = l.reshape(rows, H, 1)
        out = (out / torch.where(l1 > 0, l1, torch.ones((), device=s.device))).to(torch.bfloat16)
        lse = (m + torch.log(l)).reshape(rows, H)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------
def _value64(nibble):
    """E2M1: sign, two exponent bits (bias 1), one fraction bit; exponent 0 is subnormal."""
    n = nibble.to(torch.int64)
    frac, ex = (n & 1).double(), (n >> 1) & 3
    mag = torch.where(ex == 0, frac * 0.5, (1.0 + 0.5 * frac) * torch.exp2(ex.double() - 1.0))
    return torch.where(n >= 8, -mag, mag)


def _rows64(codes, scales):
    x = torch.stack([_value64(codes & 15), _value64(codes >> 4)], -1)
    x = x.reshape(*codes.shape[:-1], GROUPS, 32)
    e = scales.to(torch.int64) - 127
    return torch.ldexp(x, e[..., None].double()).reshape(*codes.shape[:-1], LATENT)


def _softmax64(q, c, sees):
    """q [H, 512], c [T, 512] in fp64, sees [H, T] or None -> (out, lse)."""
    s = q @ c.T
    if sees is not None:
        s = s.masked_fill(~sees, -math.inf)
    lse = torch.logsumexp(s, -1)
    s -= torch.where(torch.isfinite(lse), lse, 0.0)[:, None]
    return s.exp_() @ c, lse


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "append":
        x = st["latent"].double()
        B, n_new = x.shape[:2]
        levels = torch.tensor(_VALUES, dtype=torch.float64, device=x.device)
        stored = st["stored"].double()
        for b in range(B):
            k = n_new if st["n_add"] is None else int(st["n_add"][b])
            g = x[b, :k].reshape(k, GROUPS, 32)
            big = g.abs().amax(-1)
            nat = torch.ceil(torch.log2(big / 6.0))  # fixed up below where log2 rounds
            nat = torch.where(big > 6.0 * torch.exp2(nat), nat + 1, nat)
            nat = torch.where(big <= 6.0 * torch.exp2(nat - 1), nat - 1, nat)
            top = nat.amax(-1, keepdim=True).clamp(-50, 50)
            step = torch.exp2(torch.maximum(nat, top - 15).minimum(top))[..., None]
            y = g / step
            d = (y.abs()[..., None] - levels).abs()
            near = d.amin(-1, keepdim=True)
            # of two levels equally near, the one with an even code
            c = torch.where(d == near, torch.arange(8, device=x.device) % 2, 9).argmin(-1)
            stored[b, :k] = (torch.copysign(levels[c], g) * step).reshape(k, LATENT)
        return {"stored": stored, "codes": None, "scales": None}
    if op == "read":
        B, m = st["out"].shape[:2]
        out = torch.zeros(B, m, LATENT, dtype=torch.float64, device="cuda")
        for b in range(B):
            if st["pos"] is None:
                k = min(m, int(st["n_vis"][b]))
                out[b, :k] = _rows64(st["codes"][b, :k], st["scales"][b, :k])
            else:
                out[b] = _rows64(st["codes"][b][st["pos"][b]], st["scales"][b][st["pos"][b]])
        return out
    q = st["q"].double()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    if op == "sparse":
        n_vis, count, idx = st["n_vis"].tolist(), st["count"].tolist(), st["idx"].long()
        four = torch.arange(POOL, device="cuda")
        for r in range(q.shape[0]):
            n, b = n_vis[r], r if st["seq_stride"] else 0
            pos = (idx[r, :count[r], None] * POOL + four).reshape(-1)
            pos = torch.cat([pos, torch.arange(n - n % POOL, n, device="cuda")])
            c = _rows64(st["codes"][b][pos], st["scales"][b][pos])
            out[r], lse[r] = _softmax64(q[r], c, None)
    else:
        per, H = st["per_seq"], case["heads"]
        n_vis = st["n_vis"].tolist()
        for b in range(case["seqs"]):
            rows = slice(b * per, b * per + per)
            n = max(n_vis[rows])
            c = _rows64(st["codes"][b, :n], st["scales"][b, :n])
            sees = torch.arange(n, device="cuda")[None] < st["n_vis"][rows, None]
            o, l = _softmax64(q[rows].reshape(per * H, LATENT), c, sees.repeat_interleave(H, 0))
            out[rows], lse[rows] = o.reshape(per, H, LATENT), l.reshape(per, H)
    return {"out": out, "lse": lse}
