"""The 8-bit latent cache (written, read back, attended to) and decode attention
over a prefix that the whole batch shares: cases, inputs, plain forms and
64-bit definitions.

One latent cache row is [latent (512) | rotary key (64)], as the decode
front-fold writes it. An 8-bit cache block of `bs` rows holds three planes:
E4M3 codes [bs, 512], rotary keys [bs, 64] in bf16, scales [bs] in fp32, padded
to a multiple of 128 bytes. Row j stands for [scale_j * code_j | rotary_j]
with scale_j the smallest power of two (exponent within [-64, 7]) that brings
the row's largest magnitude to at most 448.
"""
import math

import torch

own = False

RKV, DR = 512, 64
R = RKV + DR
D_N, D_V = 128, 128
SCALE = 1.0 / math.sqrt(D_N + DR)
K_MIN, K_MAX = -64, 7


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step's rows of a small batch: launch latency
        {"name": "write_step", "op": "write", "rows": 32, "bs": 64, "skip": False},
        # a prompt of 8192 tokens goes into the cache
        {"name": "write_prompt", "op": "write", "rows": 8192, "bs": 64, "skip": False},
        # a whole batch's prompts, some rows padding that is not written
        {"name": "write_batch", "op": "write", "rows": 131007, "bs": 128, "skip": True},
        # the rows of a cached prompt, for a prompt chunk that attends to them expanded
        {"name": "read_prompt", "op": "read", "rows": 8192, "bs": 64},
        # a batch of cached prompts
        {"name": "read_batch", "op": "read", "rows": 100003, "bs": 64},
        # one sequence of a few hundred rows: the latency of a single user's step
        {"name": "attn8_one_short", "op": "attn8", "heads": 16, "n": 1, "lo": 333, "hi": 333, "bs": 64},
        # the 16-head decode step: 32 sequences of 4096 rows
        {"name": "attn8_16h", "op": "attn8", "heads": 16, "n": 32, "lo": 4096, "hi": 4096, "bs": 64},
        # 128 heads, ragged lengths from 1024 to 16384 rows
        {"name": "attn8_128h_ragged", "op": "attn8", "heads": 128, "n": 64, "lo": 1024, "hi": 16384, "bs": 64},
        # a few chats over one system prompt of 2048 tokens, 16-bit cache
        {"name": "prefix_16h_few", "op": "prefix", "heads": 16, "n": 8, "prefix": 2048, "lo": 1, "hi": 300, "bs": 64,
         "fp8": False},
        # 64 sequences sampled from one prompt of 8192 tokens, 16-bit cache
        {"name": "prefix_16h", "op": "prefix", "heads": 16, "n": 64, "prefix": 8192, "lo": 1, "hi": 512, "bs": 64,
         "fp8": False},
        # the same for 128 heads and a long document
        {"name": "prefix_128h", "op": "prefix", "heads": 128, "n": 32, "prefix": 16384, "lo": 1, "hi": 1024, "bs": 64,
         "fp8": False},
        # a large batch over a long document in the 8-bit cache
        {"name": "prefix8_16h", "op": "prefix", "heads": 16, "n": 128, "prefix": 32767, "lo": 1, "hi": 512, "bs": 64,
         "fp8": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn8", "prefix"])
    bs = rng.choice([64, 64, 128, 192])
    if op == "write":
        return {"op": op, "rows": _log_int(rng, 1, 131007), "bs": bs, "skip": rng.random() < 0.5}
    if op == "read":
        return {"op": op, "rows": _log_int(rng, 1, 100003), "bs": bs}
    heads = rng.choice([16, 16, 128, 8, 24, 64])
    if op == "attn8":
        hi = _log_int(rng, 2, 16384)
        lo = rng.randint(1, hi)
        most = max(1, min(128, (64 * 8704 * 128) // (heads * (lo + hi))))
        return {"op": op, "heads": heads, "n": _log_int(rng, 1, most), "lo": lo, "hi": hi, "bs": bs}
    prefix = _log_int(rng, 100, 32767)
    hi = _log_int(rng, 2, 1024)
    most = max(1, min(128, (128 * 16 * 32767) // (heads * (prefix + hi))))
    return {"op": op, "heads": heads, "n": _log_int(rng, 1, most), "prefix": prefix, "lo": rng.randint(0, 1), "hi": hi,
            "bs": bs, "fp8": rng.random() < 0.5}


def _lens(case):
    """The sequences' own lengths: spread evenly over [lo, hi], shuffled by a fixed rule."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    if n == 1:
        return [hi]
    ls = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    step = next(s for s in (37, 41, 43) if math.gcd(s, n) == 1)
    return [ls[(i * step) % n] for i in range(n)]


def work(case):
    row16, row8 = R * 2, RKV + DR * 2 + 4
    if case["op"] in ("write", "read"):
        return {"bytes": case["rows"] * (row16 + row8 + 4), "flops": 0}
    heads, n, rows = case["heads"], case["n"], sum(_lens(case))
    row = row8 if case["op"] == "attn8" or case["fp8"] else row16
    prefix = case.get("prefix", 0)
    pairs = heads * (rows + n * prefix)          # (query row, key) pairs
    io = n * heads * (R + RKV) * 2
    if case["op"] == "attn8":
        io += n * heads * 4                      # log-sum-exp
    return {"bytes": (rows + prefix) * row + io, "flops": 2 * pairs * (R + RKV)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _plane_offsets(bs):
    pe = bs * RKV
    sc = pe + bs * DR * 2
    return pe, sc, -(-(sc + bs * 4) // 128) * 128


def _planes(cache, bs):
    """(codes [n_blocks, bs, 512] uint8, rotary [n_blocks, bs, 64] bf16, scales [n_blocks, bs] fp32), views of the cache."""
    pe, sc, _ = _plane_offsets(bs)
    return (cache[:, :pe].unflatten(1, (bs, RKV)), cache[:, pe:sc].view(torch.bfloat16).unflatten(1, (bs, DR)),
            cache[:, sc:sc + 4 * bs].view(torch.float32))


def _rows(gen, n, dev):
    """Latent rows as the normalised projection gives them: unit RMS, a few outlying
    channels, norms that differ between tokens; rotary keys of their own size."""
    x = torch.randn((n, R), generator=gen, device=dev)
    gain = torch.ones(R, device=dev)
    gain[torch.randint(0, RKV, (6,), generator=gen, device=dev)] = 8.0
    size = torch.exp2(torch.randint(-2, 2, (n, 1), generator=gen, device=dev).float() * 0.5)
    x = x * gain
    x[:, :RKV] *= size
    return x.to(torch.bfloat16)


def _quantise(rows):
    """(codes uint8 [n, 512], rotary [n, 64] bf16, scales [n] fp32) of bf16 rows, by the definition above."""
    lat = rows[:, :RKV].float()
    fine = torch.isfinite(lat)
    amax = torch.where(fine, lat.abs(), torch.zeros_like(lat)).amax(1)
    m, e = torch.frexp(amax)                     # amax = m 2^e with m in [0.5, 1); 448 = 0.875 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k.clamp(K_MIN, K_MAX), torch.zeros_like(k))
    scale = torch.ldexp(torch.ones_like(amax), k)
    x = (lat / scale[:, None]).clamp(-448.0, 448.0)
    x = torch.where(fine, x, torch.full_like(x, math.nan))
    return x.to(torch.float8_e4m3fn).view(torch.uint8), rows[:, RKV:], scale


def _store(cache, bs, slots, rows):
    codes, pe, scales = _planes(cache, bs)
    c, e, s = _quantise(rows)
    b, o = slots // bs, slots % bs
    codes[b, o], pe[b, o], scales[b, o] = c, e, s


def _layer(heads, bs, cache_dtype):
    """The handle that a serving program keeps; these operators read no weight of it."""
    from head_latent_attention_decode_b200 import workloads as wl
    from head_latent_attention_decode_b200.layer import MlaLayer
    import dataclasses
    s = dataclasses.replace(wl.V2LITE, n_heads=heads, block_size=bs)
    w = {k: torch.zeros(v, dtype=torch.bfloat16, device="cuda") for k, v in wl.weight_shapes(s).items()}
    w["kv_norm_w"] = torch.ones(RKV, device="cuda")
    return MlaLayer(s, w, cache_dtype=cache_dtype)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bs, op = case["bs"], case["op"]
    st = {"op": op, "bs": bs}
    if op in ("write", "read"):
        n = case["rows"]
        blocks = -(-n // bs) + 3
        order = torch.randperm(blocks, generator=gen, device=dev)
        pos = torch.arange(n, device=dev)
        slots = order[pos // bs] * bs + pos % bs
        rows = _rows(gen, n, dev)
        cache = torch.zeros((blocks, _plane_offsets(bs)[2]), dtype=torch.uint8, device=dev)
        if op == "read":
            _store(cache, bs, slots, rows)
            rows = torch.zeros_like(rows)
        elif case["skip"]:                       # every 16th row is padding
            slots = torch.where(pos % 16 == 15, torch.full_like(slots, -1), slots)
        st.update(rows=rows, cache=cache, slots=slots.int())
        if own:
            st["layer"] = _layer(16, bs, "fp8")
            st["ws"] = st["layer"].workspace(1, 1)
        return st
    heads, n, lens = case["heads"], case["n"], _lens(case)
    prefix = case.get("prefix", 0)
    fp8 = op == "attn8" or case["fp8"]
    npb, nb = -(-prefix // bs), [-(-x // bs) for x in lens]
    blocks = npb + sum(nb) + 3
    order = torch.randperm(blocks, generator=gen, device=dev).int()
    width = max(1, max(nb))
    cols = torch.arange(width, device=dev)
    nbt = torch.tensor(nb, device=dev)
    first = torch.cumsum(nbt, 0) - nbt + npb
    at = (first[:, None] + cols).clamp(max=blocks - 1)
    table = torch.where(cols < nbt[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32))
    rows = _rows(gen, blocks * bs, dev)
    if fp8:
        cache = torch.zeros((blocks, _plane_offsets(bs)[2]), dtype=torch.uint8, device=dev)
        _store(cache, bs, torch.arange(blocks * bs, device=dev), rows)
    else:
        cache = rows.view(blocks, 1, bs, R).clone()
    size = torch.exp2(torch.rand((1, heads, 1), generator=gen, device=dev) * 2.5 - 2.0)   # heads attend more or less sharply
    st.update(cache=cache, table=table, ctx=torch.tensor(lens, dtype=torch.int32, device=dev), max_ctx=max(1, max(lens)),
              prefix_len=prefix, prefix_table=order[:npb].contiguous(), fp8=fp8, heads=heads,
              q_abs=(torch.randn((n, heads, RKV), generator=gen, device=dev) * size).to(torch.bfloat16),
              q_pe=(torch.randn((n, heads, DR), generator=gen, device=dev) * size).to(torch.bfloat16))
    if own:
        st["layer"] = _layer(heads, bs, "fp8" if fp8 else None)
        st["ws"] = st["layer"].prefix_workspace(n, prefix, st["max_ctx"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    if st["op"] == "write":
        if own:
            st["layer"].cache_write(st["rows"], st["cache"], st["slots"])
        else:
            _plain_write(st)
        codes, pe, scales = _planes(st["cache"], st["bs"])
        return {"codes": codes.view(torch.float8_e4m3fn), "rotary": pe, "scales": scales}
    if st["op"] == "read":
        if own:
            return st["layer"].cache_read(st["cache"], st["slots"], st["rows"])
        return _plain_read(st)
    if own:
        kw = {"prefix_table": st["prefix_table"], "prefix_len": st["prefix_len"]} if st["prefix_len"] else {}
        o, lse = st["layer"].latent_attn(st["q_abs"], st["q_pe"], st["cache"], st["table"], st["ctx"], st["max_ctx"],
                                         want_lse=st["op"] == "attn8", **kw)
    else:
        o, lse = _plain_attn(st)
    return {"o": o, "lse": lse} if st["op"] == "attn8" else {"o": o}


def _plain_write(st):
    keep = st["slots"] >= 0
    _store(st["cache"], st["bs"], st["slots"][keep].long(), st["rows"][keep])


def _values(st, blk, off):
    """fp32 rows at (block, offset): the values an 8-bit row stands for, or a 16-bit row's own."""
    if st["cache"].dtype == torch.uint8:
        codes, pe, scales = _planes(st["cache"], st["bs"])
        lat = codes[blk, off].view(torch.float8_e4m3fn).float() * scales[blk, off][..., None]
        return torch.cat([lat, pe[blk, off].float()], -1)
    return st["cache"][blk, 0, off].float()


def _plain_read(st):
    s = st["slots"].long()
    return _values(st, s // st["bs"], s % st["bs"]).to(torch.bfloat16)


def _plain_attn(st):
    n, heads, bs = st["q_abs"].shape[0], st["heads"], st["bs"]
    q = torch.cat([st["q_abs"], st["q_pe"]], -1).float()
    pos = torch.arange(st["max_ctx"], device=q.device)
    live = pos < st["ctx"][:, None]                                       # [n, keys]
    blk = st["table"].long()[:, pos // bs].clamp(min=0)
    keys = torch.where(live[..., None], _values(st, blk, (pos % bs).expand_as(blk)), 0.0)   # [n, keys, 576]
    s = torch.matmul(q, keys.transpose(1, 2)) * SCALE
    s = torch.where(live[:, None], s, -math.inf)
    if st["prefix_len"]:
        pos = torch.arange(st["prefix_len"], device=q.device)
        shared = _values(st, st["prefix_table"].long()[pos // bs], pos % bs)   # [prefix, 576]
        s = torch.cat([torch.matmul(q.view(n * heads, R), shared.t()).view(n, heads, -1) * SCALE, s], -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    den = p.sum(-1, keepdim=True)
    at = st["prefix_len"]
    o = torch.matmul(p[..., at:], keys[..., :RKV])
    if at:
        o = o + torch.matmul(p[..., :at].reshape(n * heads, at), shared[:, :RKV]).view(n, heads, RKV)
    return (o / den).to(torch.bfloat16), (m + torch.log(den))[..., 0]


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    bs = st["bs"]
    _, _, size = _plane_offsets(bs)
    # a table of the 256 codes' values from the format: sign, 4 exponent bits (bias 7), 3 fraction bits
    value = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = math.nan if (e == 15 and f == 7) else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        value.append(-v if c & 128 else v)
    value = torch.tensor(value, dtype=torch.float64, device="cuda")
    if case["op"] == "write":
        flat = st["rows"].double()
        blocks = st["cache"].shape[0]
        codes = torch.zeros((blocks * bs, RKV), dtype=torch.float64, device="cuda")
        pe = torch.zeros((blocks * bs, DR), dtype=torch.float64, device="cuda")
        scales = torch.zeros(blocks * bs, dtype=torch.float64, device="cuda")
        positive = value[:127]                   # ascending
        middle = (positive[1:] + positive[:-1]) / 2
        for i in range(0, flat.shape[0], 16384):
            x, s = flat[i:i + 16384], st["slots"][i:i + 16384].long()
            x, s = x[s >= 0], s[s >= 0]
            top = x[:, :RKV].abs().amax(1)
            k = torch.full_like(top, K_MIN)
            for j in range(K_MIN, K_MAX):        # the smallest exponent whose 448 reaches the row's largest
                k += (top > 448.0 * 2.0 ** j) & (k == j)
            k = torch.where(top > 0, k, torch.zeros_like(k))
            u = x[:, :RKV] / torch.exp2(k)[:, None]
            a = u.abs().clamp(max=448.0)
            lo = torch.bucketize(a, middle, right=False)       # a tie goes to the lower neighbour here
            hi = torch.bucketize(a, middle, right=True)        # and to the upper one here: the even code wins
            lo = torch.where((lo != hi) & (lo % 2 == 1), hi, lo)
            codes[s] = torch.sign(u) * positive[lo]
            pe[s], scales[s] = x[:, RKV:], torch.exp2(k)
        return {"codes": codes.view(blocks, bs, RKV), "rotary": pe.view(blocks, bs, DR), "scales": scales.view(blocks, bs)}

    cache = st["cache"].reshape(-1)

    def rows_at(slots):
        if st["cache"].dtype != torch.uint8:
            return st["cache"].reshape(-1, R)[slots].double()
        start = (slots // bs) * size
        off = slots % bs
        at = (start + off * RKV)[:, None] + torch.arange(RKV, device="cuda")
        lat = value[cache[at].long()]
        at = (start + bs * RKV + off * DR * 2)[:, None] + torch.arange(DR * 2, device="cuda")
        pe = cache[at].contiguous().view(torch.bfloat16).double()
        at = (start + bs * (RKV + DR * 2) + off * 4)[:, None] + torch.arange(4, device="cuda")
        return torch.cat([lat * cache[at].contiguous().view(torch.float32).double(), pe], 1)

    if case["op"] == "read":
        return torch.cat([rows_at(s.long()) for s in st["slots"].split(16384)])
    n = case["n"]
    o, lse = [], []
    at = torch.arange(case.get("prefix", 0), device="cuda")
    shared = rows_at(st["prefix_table"].long()[at // bs] * bs + at % bs) if len(at) else None
    for t, length in enumerate(_lens(case)):
        at = torch.arange(length, device="cuda")
        keys = rows_at(st["table"][t].long()[at // bs] * bs + at % bs)
        if shared is not None:
            keys = torch.cat([shared, keys])
        q = torch.cat([st["q_abs"][t], st["q_pe"][t]], 1).double()
        z = q @ keys.t() / math.sqrt(D_N + DR)
        total = torch.logsumexp(z, 1)
        o.append(torch.exp(z - total[:, None]) @ keys[:, :RKV])
        lse.append(total)
    assert len(o) == n
    return {"o": torch.stack(o), "lse": torch.stack(lse)} if case["op"] == "attn8" else {"o": torch.stack(o)}
