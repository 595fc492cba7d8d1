"""Shared plumbing of the 8-bit cache and shared-prefix tests: small layers,
caches built row by row on the host, the fp64 definitions, and error bounds."""
import dataclasses
import functools

import numpy as np
import torch

from head_latent_attention_decode_b200 import workloads as wl
from oracle import latent_ref as lr

ACT = {"f32": torch.float32, "bf16": torch.bfloat16}
ESZ = {"f32": 4, "bf16": 2}


def shape_of(heads, bs, act="bf16", r_kv=512, d_r=64, q_lora=0, **kw):
    base = wl.V2LITE if act == "bf16" else wl.TINY
    return dataclasses.replace(base, hidden=256, n_heads=heads, q_lora_rank=q_lora, kv_lora_rank=r_kv, qk_rope=d_r,
                               block_size=bs, act_dtype=act, weight_dtype=act, **kw)


@functools.lru_cache(maxsize=None)
def _weights(shape):
    return wl.make_weights(shape, 11)


def layer_of(shape, fp8, sink=None, **kw):
    from head_latent_attention_decode_b200.build import build
    from head_latent_attention_decode_b200.layer import MlaLayer
    build()
    return MlaLayer(shape, _weights(shape), cache_dtype="fp8" if fp8 else None, attn_sink=sink, **kw)


def pack_block_rows(cache, shape, slot, codes, k, pe):
    """Row `slot` of a numpy uint8 cache [n_blocks, block bytes]; pe: act-dtype torch vector."""
    bs, r = shape.block_size, shape.kv_lora_rank
    po, so, _ = lr.block_layout(bs, r, shape.qk_rope, ESZ[shape.act_dtype])
    b, o = slot // bs, slot % bs
    cache[b, o * r:(o + 1) * r] = codes
    raw = pe.contiguous().view(torch.uint8).numpy()
    cache[b, po + o * raw.size: po + (o + 1) * raw.size] = raw
    cache[b, so + 4 * o: so + 4 * o + 4] = np.frombuffer(np.float32(2.0 ** k).tobytes(), np.uint8)


def pack_cache(shape, rows, slots, n_blocks, fill=0):
    """uint8 cache holding rows (act-dtype torch [n, R], latent first) at `slots`, by the definition."""
    _, _, size = lr.block_layout(shape.block_size, shape.kv_lora_rank, shape.qk_rope, ESZ[shape.act_dtype])
    cache = np.full((n_blocks, size), fill, np.uint8)
    lat = rows[:, :shape.kv_lora_rank].double().numpy()
    for t, s in enumerate(slots):
        if s >= 0:
            codes, k = lr.quantise_row(lat[t])
            pack_block_rows(cache, shape, int(s), codes, k, rows[t, shape.kv_lora_rank:])
    return cache


def row_values(shape, rows):
    """fp64 [n, R]: what the rows stand for once quantised."""
    r = shape.kv_lora_rank
    out = rows.double().numpy().copy()
    for t in range(out.shape[0]):
        codes, k = lr.quantise_row(out[t, :r])
        out[t, :r] = lr.E4M3[codes] * 2.0 ** k
    return out


def row_scales(shape, rows):
    """fp64 [n]: each row's scale once quantised."""
    lat = rows[:, :shape.kv_lora_rank].double().numpy()
    return np.array([2.0 ** lr.scale_exponent(x) for x in lat])


def tables(rng, lens, bs, prefix_len, spare=2):
    """Random physical blocks: (prefix table, block table [n, width] with -1 beyond, n_blocks)."""
    npb = -(-prefix_len // bs)
    nb = [-(-int(x) // bs) for x in lens]
    n_blocks = npb + sum(nb) + spare
    perm = rng.permutation(n_blocks).astype(np.int32)
    table = np.full((len(lens), max([1] + nb)), -1, np.int32)
    at = npb
    for t, m in enumerate(nb):
        table[t, :m] = perm[at:at + m]
        at += m
    return perm[:npb].copy(), table, n_blocks


class Case:
    """One attention call's inputs and its fp64 result."""

    def __init__(self, shape, lens, prefix_len=0, fp8=True, sink=False, seed=0, q_size=1.0, poison=True, rows=None):
        rng = np.random.default_rng(seed)
        self.shape, self.lens, self.prefix_len, self.fp8 = shape, list(lens), prefix_len, fp8
        act, bs, r, d = ACT[shape.act_dtype], shape.block_size, shape.kv_lora_rank, shape.qk_rope
        R, H, n = r + d, shape.n_heads, len(lens)
        self.ptable, self.table, self.n_blocks = tables(rng, lens, bs, prefix_len)
        total = self.n_blocks * bs
        if rows is None:
            rows = rng.standard_normal((total, R)) * 2.0 ** rng.integers(-3, 3, (total, 1))
        self.rows = torch.from_numpy(np.asarray(rows, np.float32)).to(act)
        used = [int(b) * bs + o for i, b in enumerate(self.ptable) for o in range(min(bs, prefix_len - i * bs))]
        for t, L in enumerate(lens):
            used += [int(self.table[t, j // bs]) * bs + j % bs for j in range(L)]
        self.used = np.array(sorted(set(used)), np.int64)
        if poison:   # rows that no sequence reaches hold NaN everywhere
            free = np.setdiff1d(np.arange(total), self.used)
            self.rows[torch.from_numpy(free)] = float("nan")
        self.q_abs = torch.from_numpy((rng.standard_normal((n, H, r)) * q_size).astype(np.float32)).to(act)
        self.q_pe = torch.from_numpy((rng.standard_normal((n, H, d)) * q_size).astype(np.float32)).to(act)
        self.sink = (rng.standard_normal(H) * 2).astype(np.float32) if sink else None
        self.scale = 1.0 / np.sqrt(shape.qk_nope + d)
        self.keys = row_values(shape, self.rows) if fp8 else self.rows.double().numpy()

    def key_slots(self, t):
        bs = self.shape.block_size
        return np.array([int(self.ptable[j // bs]) * bs + j % bs for j in range(self.prefix_len)]
                        + [int(self.table[t, j // bs]) * bs + j % bs for j in range(self.lens[t])], np.int64)

    def device_cache(self):
        s = self.shape
        if self.fp8:
            return torch.from_numpy(pack_cache(s, self.rows, np.arange(self.n_blocks * s.block_size), self.n_blocks)).cuda()
        return self.rows.view(self.n_blocks, 1, s.block_size, s.kv_row_dim).cuda()

    def layer(self, **kw):
        return layer_of(self.shape, self.fp8, sink=self.sink, **kw)

    def device_inputs(self):
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        return dict(q_abs=self.q_abs.cuda(), q_pe=self.q_pe.cuda(), kv_cache=self.device_cache(),
                    block_table=dev(self.table), context_lens=dev(np.array(self.lens, np.int32)),
                    max_context_len=max([1] + self.lens), prefix_table=dev(self.ptable) if self.prefix_len else None,
                    prefix_len=self.prefix_len)

    def oracle(self):
        """(o, lse, bound on |o error|, bound on |lse error|), from the formulas.

        The kernels' weights are p_j (1 + d_j): |d_j| <= e = e_score + e_p. A weighted mean whose
        weights are off by at most e is off by at most 2 e / (1 - e) sum_j p_j |c_j| (numerator and
        denominator each by e), and log sum p_j (1 + d_j) by at most e / (1 - e).
        e_score: |score error|. fp32 sums of r + d products, each at most half a step off and the
          sum in any order, 2 (r + d) 2^-24 sum |q_i c_i|; for a 16-bit act dtype the partial score
          that crosses between two CTAs in f16 adds 2^-11 of a half's score, and a query split in
          two E4M3 parts 2^-18 of its largest element per column, 2^-18 max|q| sum |c_i|.
        e_p: 16-bit: a probability in bf16, or in two E4M3 parts (2^-4 of 2^-4), 2^-8 either way.
          fp32 act: exponentials and sums, 64 2^-24.
        The two-part weights w_j = 2^8 p_j s_j / 2^R have an absolute floor besides: the second part's
        smallest step is 2^-9, so w_j is off by up to 2^-10 however light the key, p_j s_j by 2^-18 2^R.
        2^R is at most 2^6 of the largest of late, which forgets an octave every second tile:
        rec_t = max(largest p_i s_i of tile t, 2^-1/2 rec_(t-1)) over a pass's tiles of 128 keys (or
        2^-40 of the largest of all), so p_j s_j is off by up to 2^-12 rec_t. What it multiplies is the
        code, so o is off by up to the sum over tiles of 2^-12 rec_t sum_j |code_j|; the sums that
        normalise take the weights unrounded. o is then rounded once to its type.
    """
        s = self.shape
        r = s.kv_lora_rank
        o, lse, bo, bl = [], [], [], []
        for t in range(len(self.lens)):
            k = self.keys[self.key_slots(t)]
            c, pe = k[:, :r], k[:, r:]
            qa, qp = self.q_abs[t].double().numpy(), self.q_pe[t].double().numpy()
            x, ll, p = lr.latent_attention(qa, qp, c, pe, self.scale, self.sink)
            mag = (np.abs(qa) @ np.abs(c).T + np.abs(qp) @ np.abs(pe).T) * self.scale if len(k) else np.zeros_like(p)
            e = 2 * (r + s.qk_rope) * 2.0 ** -24 * mag
            floor = 0.0
            if s.act_dtype == "bf16":
                h = r // 2
                half = np.maximum(np.abs(qa[:, :h] @ c[:, :h].T), np.abs(qa[:, h:] @ c[:, h:].T))
                e = e + 2.0 ** -11 * (half + np.abs(qp @ pe.T)) * self.scale
                if self.fp8 and len(k):
                    e = e + 2.0 ** -18 * np.abs(qa).max(1)[:, None] * np.abs(c).sum(1)[None] * self.scale
                e = (e.max(1) if len(k) else np.zeros(len(p))) + 2.0 ** -8
                step = 2.0 ** -8
                if self.fp8 and len(k):
                    sc = row_scales(s, self.rows[torch.from_numpy(self.key_slots(t))])
                    code, ps = np.abs(c) / sc[:, None], p * sc
                    floor = 2.0 ** -50 * ps.max(1)[:, None] * code.sum(0)[None]
                    for a0, a1 in ((0, self.prefix_len), (self.prefix_len, len(k))):   # the passes' tiles
                        rec = np.zeros(len(ps))
                        for j in range(a0, a1, 128):
                            m = min(j + 128, a1)
                            rec = np.maximum(rec * 2.0 ** -0.5, ps[:, j:m].max(1))
                            floor = floor + 2.0 ** -12 * rec[:, None] * code[j:m].sum(0)[None]
            else:
                e = (e.max(1) if len(k) else np.zeros(len(p))) + 64 * 2.0 ** -24
                step = 2.0 ** -24
            assert (e < 0.5).all(), "inputs too sharp for the bound"
            a = p @ np.abs(c) if len(k) else np.zeros_like(x)
            o.append(x)
            lse.append(ll)
            bo.append((2 * (e / (1 - e))[:, None] * a + floor) * (1 + step) + step * np.abs(x) + 1e-30)
            bl.append(e / (1 - e) + 4 * 2.0 ** -24 * np.abs(np.where(np.isfinite(ll), ll, 0.0)) + 2.0 ** -22)
        return np.stack(o), np.stack(lse), np.stack(bo), np.stack(bl)


def check(case, o, lse, want=None):
    wo, wl_, bo, bl = want if want is not None else case.oracle()
    go = o.double().cpu().numpy()
    assert np.isfinite(go).all(), "non-finite outputs"
    worst = float((np.abs(go - wo) / bo).max())
    assert worst <= 1.0, f"o: {worst:.2f} of the bound"
    if lse is not None:
        gl = lse.double().cpu().numpy()
        fin = np.isfinite(wl_)
        assert (np.isfinite(gl) == fin).all() and (gl[~fin] == wl_[~fin]).all()
        wl = float((np.abs(gl[fin] - wl_[fin]) / bl[fin]).max()) if fin.any() else 0.0
        assert wl <= 1.0, f"lse: {wl:.2f} of the bound"
