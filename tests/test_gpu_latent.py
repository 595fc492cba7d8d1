"""GPU tests of the 8-bit latent cache (written, read back, attended to) and of
decode attention over a shared prefix, against the fp64 definitions in
oracle/latent_ref.py. Writing and reading are exact; the attention's bounds are
derived in latent_common.Case.oracle."""
import dataclasses

import numpy as np
import pytest
import torch

import head_latent_attention_decode_b200 as mla
from head_latent_attention_decode_b200 import workloads as wl
from oracle import latent_ref as lr
from oracle import mla_ref as ref

from latent_common import ACT, ESZ, Case, check, layer_of, pack_cache, row_scales, row_values, shape_of
from latent_common import _weights as weights_of

pytestmark = pytest.mark.gpu

SHAPES = {"latent512": dict(bs=64), "bs48": dict(bs=48), "small": dict(bs=16, r_kv=64, d_r=16),
          "odd_block": dict(bs=7, r_kv=96, d_r=8)}


def special_rows(shape, n, seed):
    """Rows of many sizes, with the values at which a quantiser can go wrong."""
    rng = np.random.default_rng(seed)
    r = shape.kv_lora_rank
    x = rng.standard_normal((n, shape.kv_row_dim)) * 2.0 ** rng.integers(-6, 6, (n, 1))
    rows = torch.from_numpy(x.astype(np.float32)).to(ACT[shape.act_dtype])
    lat = rows[:, :r]
    edge = [lambda v: v.zero_(), lambda v: v.fill_(448.0), lambda v: v.fill_(450.0), lambda v: v.mul_(1e-30),
            lambda v: v.mul_(1e30), lambda v: v[1:3].fill_(float("nan")), lambda v: v[:1].fill_(float("inf")),
            lambda v: v.fill_(-float("inf")), lambda v: v[5:6].fill_(57344.0), lambda v: v.fill_(1.75 * 2.0 ** -3),
            lambda v: v[:8].copy_(torch.tensor([17, 19, 21, 23, 25, 27, 29, 448.0])), lambda v: v.mul_(2.0 ** -90)]
    for i, f in enumerate(edge):
        if i < n:
            f(lat[i])
    return rows


def same_bytes(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.cpu().view(torch.uint8))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("n", [1, 13, 301])
def test_write_and_read_are_exact(name, act, n):
    shape = shape_of(4, act=act, **SHAPES[name])
    layer = layer_of(shape, True)
    rows = special_rows(shape, n, n)
    n_blocks = -(-n // shape.block_size) + 2
    rng = np.random.default_rng(n)
    slots = rng.permutation(n_blocks * shape.block_size)[:n].astype(np.int32)
    if n > 12:
        slots[12] = -1
    cache = layer.new_cache(n_blocks)
    cache.fill_(0xAB)
    layer.cache_write(rows.cuda(), cache, torch.from_numpy(slots).cuda())
    want = pack_cache(shape, rows, slots, n_blocks, fill=0xAB)
    got = cache.cpu().numpy()
    # E4M3 has two NaN codes and two zeros: the codes' values count, all other bytes are equal
    diff = got != want
    codes = np.zeros_like(diff)
    codes[:, :shape.block_size * shape.kv_lora_rank] = True
    assert not (diff & ~codes).any()
    a, b = lr.E4M3[got[codes]], lr.E4M3[want[codes]]
    assert np.array_equal(a, b, equal_nan=True)
    # back, with a repeated slot and one that is skipped
    back = np.concatenate([slots, slots[:1], [-5]]).astype(np.int32)
    out = torch.full((n + 2, shape.kv_row_dim), 7.0, dtype=ACT[act], device="cuda")
    layer.cache_read(cache, torch.from_numpy(back).cuda(), out)
    vals = row_values(shape, rows)
    vals[slots < 0] = 7.0
    vals = np.concatenate([vals, vals[:1], np.full((1, shape.kv_row_dim), 7.0)])
    assert np.array_equal(out.double().cpu().numpy(), vals, equal_nan=True)
    assert mla.mla_read_device_flag(layer.ws) == 0


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_row_copies_of_an_activation_dtype_cache(act):
    shape = shape_of(4, 16, act=act, r_kv=64, d_r=16)
    layer = layer_of(shape, False)
    rows = torch.randn(33, shape.kv_row_dim).to(ACT[act])
    slots = torch.randperm(64)[:33].int()
    cache = layer.new_cache(4)
    layer.cache_write(rows.cuda(), cache, slots.cuda())
    want = torch.zeros(64, shape.kv_row_dim, dtype=ACT[act])
    want[slots.long()] = rows
    assert same_bytes(cache.reshape(64, -1), want)
    assert same_bytes(layer.cache_read(cache, slots.cuda()), rows)


@pytest.mark.parametrize("fp8", [True, False])
def test_pe_first_rows(fp8):
    shape = shape_of(4, 16, r_kv=64, d_r=16)
    layer = layer_of(shape, fp8, row_layout=mla.MLA_ROW_PE_FIRST)
    rows = special_rows(shape, 5, 3)
    flipped = torch.cat([rows[:, 64:], rows[:, :64]], 1).contiguous().cuda()
    slots = torch.tensor([3, 1, 17, 30, 0], dtype=torch.int32, device="cuda")
    cache = layer.new_cache(2)
    layer.cache_write(flipped, cache, slots)
    want = row_values(shape, rows) if fp8 else rows.double().numpy()
    want = np.concatenate([want[:, 64:], want[:, :64]], 1)
    assert np.array_equal(layer.cache_read(cache, slots).double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("fp8", [True, False])
def test_slots_beyond_the_cache_are_flagged_and_left_out(fp8):
    shape = shape_of(4, 16, r_kv=64, d_r=16)
    layer = layer_of(shape, fp8)
    cache = layer.new_cache(2)
    before = cache.clone()
    rows = torch.randn(3, shape.kv_row_dim, device="cuda").bfloat16()
    slots = torch.tensor([32, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    layer.cache_write(rows, cache, slots)
    assert mla.mla_read_device_flag(layer.ws) == mla.MLA_FLAG_BAD_SLOT
    assert same_bytes(cache, before)
    mla.mla_clear_device_flag(layer.ws)
    out = torch.full_like(rows, 5.0)
    layer.cache_read(cache, slots, out)
    assert mla.mla_read_device_flag(layer.ws) == mla.MLA_FLAG_BAD_SLOT
    assert (out == 5.0).all()


ATTN = {
    # name: (heads, block size, own lengths, prefix length)
    "one_key": (16, 64, [1], 0),
    "ragged": (16, 64, [1, 63, 64, 65, 127, 128, 129, 300], 0),
    "long": (16, 64, [2111], 0),
    "blocks_of_16": (16, 16, [5, 200, 131], 0),
    "blocks_of_48": (16, 48, [1, 47, 49, 260], 0),
    "blocks_of_192": (16, 192, [191, 193, 500], 0),
    "blocks_of_24": (16, 24, [100, 30], 0),
    "one_head": (1, 64, [77, 400], 0),
    "24_heads": (24, 64, [300, 128, 1], 0),
    "40_heads": (40, 64, [150, 257], 0),
    "128_heads": (128, 64, [200, 65, 1], 0),
    "many_short": (16, 64, [1 + (7 * i) % 90 for i in range(160)], 0),
    "prefix_one_row": (16, 64, [0, 1, 70], 1),
    "prefix_only": (16, 64, [0, 0, 0], 130),
    "prefix": (16, 64, [0, 1, 5, 64, 100], 300),
    "prefix_blocks_of_16": (16, 16, [3, 40], 77),
    "prefix_24_heads": (24, 64, [10, 0, 129, 64, 64, 1, 2], 129),
    "prefix_128_heads": (128, 64, [10, 0, 129], 190),
    "prefix_5_heads": (5, 64, [i % 3 for i in range(67)], 64),
    "prefix_long": (16, 64, [100, 7], 1500),
    "prefix_odd_block": (8, 7, [20, 0, 9], 33),
    "128_heads_blocks_of_16": (128, 16, [33, 200], 50),
    "128_heads_long": (128, 64, [1500, 64], 0),
    "128_heads_many_tiles": (128, 64, [5000 - 61 * i for i in range(40)], 0),
    "80_heads": (80, 128, [70, 333], 140),
    "prefix_tiny": (8, 64, [3, 0], 700),
    "prefix_many_tiles": (16, 64, [1] * 40, 9000),
}


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("name", list(ATTN))
def test_latent_attention(name, fp8):
    heads, bs, lens, prefix = ATTN[name]
    case = Case(shape_of(heads, bs), lens, prefix, fp8, seed=len(name))
    layer = case.layer()
    o, lse = layer.latent_attn(want_lse=True, **case.device_inputs())
    torch.cuda.synchronize()
    assert mla.mla_read_device_flag(layer.ws) == 0
    check(case, o, lse)


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache32"])
@pytest.mark.parametrize("name", ["ragged", "prefix", "prefix_odd_block"])
def test_latent_attention_fp32(name, fp8):
    heads, bs, lens, prefix = ATTN[name]
    case = Case(shape_of(heads, bs, act="f32", r_kv=64, d_r=16), lens, prefix, fp8, seed=3)
    layer = case.layer()
    o, lse = layer.latent_attn(want_lse=True, **case.device_inputs())
    check(case, o, lse)


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("name", ["ragged", "prefix", "prefix_only", "128_heads", "prefix_128_heads"])
def test_attention_sink(name, fp8):
    heads, bs, lens, prefix = ATTN[name]
    case = Case(shape_of(heads, bs), lens, prefix, fp8, sink=True, seed=5)
    o, lse = case.layer().latent_attn(want_lse=True, **case.device_inputs())
    check(case, o, lse)


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("prefix", [0, 200])
def test_sharp_scores(fp8, prefix):
    # a few keys carry nearly everything, some of them late: the reference max moves by far
    case = Case(shape_of(16, 64), [400, 129], prefix, fp8, seed=9)
    for t in range(2):
        s = case.key_slots(t)
        for at in (5, len(s) // 2, len(s) - 1):
            case.rows[s[at], :64] = case.q_abs[t, at % 16, :64] * 3
    case.keys = row_values(case.shape, case.rows) if fp8 else case.rows.double().numpy()
    o, lse = case.layer().latent_attn(want_lse=True, **case.device_inputs())
    check(case, o, lse)


@pytest.mark.parametrize("heads,lens,prefix", [(128, [200, 64, 1], 0), (16, [100, 3, 0], 300), (64, [130, 70], 0)])
def test_rows_of_much_different_sizes_in_one_tile(heads, lens, prefix):
    # neighbouring rows 2^-20 to 2^3 of the usual size; below 2^-21 of a tile's largest scale the
    # values may be off by 2^-22 of it (weights add up to one, so o by no more)
    case = Case(shape_of(heads, 64), lens, prefix, True, seed=heads)
    size = np.random.default_rng(heads).integers(-20, 4, (len(case.rows), 1))
    case.rows[:, :512] *= torch.from_numpy(2.0 ** size).bfloat16()
    case.keys = row_values(case.shape, case.rows)
    o, lse = case.layer().latent_attn(want_lse=True, **case.device_inputs())
    wo, wl_, bo, bl = case.oracle()
    largest = row_scales(case.shape, case.rows[torch.from_numpy(case.used)]).max()
    check(case, o, lse, want=(wo, wl_, bo + 2.0 ** -22 * largest, bl))


@pytest.mark.parametrize("heads,lens,prefix,fp8", [(128, [700, 300, 64, 130], 0, True), (16, [100, 7, 0], 900, True),
                                                   (128, [200, 30], 400, False), (16, [64, 1, 90], 900, False)])
def test_the_lse_is_good_to_fp32(heads, lens, prefix, fp8):
    # Half of each score crosses between two CTAs in f16, off by d <= 2^-12 |half| scale, about 2^-12 4 =
    # 2^-10 here. The sums take that out to first order: d^2 / 2 = 2^-21 is left, and the weights'
    # own rounding times d, 2^-18 a key with either sign, over a hundred keys and more below 2^-21.
    # Together with the fp32 sums 2e-6 of an lse of about 6 at most; with the first order left in, 3e-5.
    case = Case(shape_of(heads, 64), lens, prefix, fp8, seed=17)
    size = 2.0 ** np.floor(np.log2(np.abs(case.rows[:, :512].float().numpy()).mean(1, keepdims=True) + 1e-30))
    size[~np.isfinite(size)] = 1.0
    case.rows[:, :512] /= torch.from_numpy(size).bfloat16()   # rows of one size, as a norm leaves them
    case.keys = row_values(case.shape, case.rows) if fp8 else case.rows.double().numpy()
    _, lse = case.layer().latent_attn(want_lse=True, **case.device_inputs())
    _, want, _, _ = case.oracle()
    got, keep = lse.double().cpu().numpy(), np.isfinite(want)
    assert (np.isfinite(got) == keep).all()
    assert np.linalg.norm(got[keep] - want[keep]) <= 2e-6 * np.linalg.norm(want[keep])


@pytest.mark.parametrize("heads,bs,lens,prefix,fp8", [
    (16, 16, [1 + i % 3 for i in range(800)], 0, True), (128, 64, [1 + i % 2 for i in range(300)], 0, True),
    (16, 64, [i % 3 for i in range(300)], 70, True), (16, 64, [i % 3 for i in range(300)], 70, False),
    (130, 64, [70, 3], 0, True), (130, 64, [70, 0], 100, True), (130, 64, [70, 0], 100, False),
], ids=["few_800", "heads_300", "prefix8_300", "prefix16_300", "130_heads", "prefix8_130_heads", "prefix16_130_heads"])
def test_more_tokens_than_a_pass_takes_and_more_heads_than_a_tile(heads, bs, lens, prefix, fp8):
    case = Case(shape_of(heads, bs), lens, prefix, fp8, seed=len(lens) + heads)
    layer = case.layer()
    o, lse = layer.latent_attn(want_lse=True, **case.device_inputs())
    assert mla.mla_read_device_flag(layer.ws) == 0
    check(case, o, lse)


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads", [16, 128])
def test_blocks_beyond_four_gigabytes(heads, fp8):
    case = Case(shape_of(heads, 64), [100, 64, 3], 130, fp8, seed=5)
    layer = case.layer()
    x = case.device_inputs()
    want, wl_ = layer.latent_attn(want_lse=True, **x)
    many = (1 << 32) // layer.block_bytes + 100
    big = layer.new_cache(many)
    at = many - case.n_blocks
    big[at:] = x["kv_cache"]
    move = lambda t: torch.where(t >= 0, t + at, t)  # noqa: E731
    o, lse = layer.latent_attn(want_lse=True, **dict(x, kv_cache=big, block_table=move(x["block_table"]),
                                                     prefix_table=move(x["prefix_table"])))
    assert mla.mla_read_device_flag(layer.ws) == 0
    assert same_bytes(o, want) and same_bytes(lse, wl_)
    # its last rows, written and read
    rows = case.rows[torch.from_numpy(case.used[:50])].cuda()
    slots = torch.arange(many * 64 - 50, many * 64, dtype=torch.int32, device="cuda")
    layer.cache_write(rows, big, slots)
    small = layer.new_cache(1)
    low = torch.arange(14, 64, dtype=torch.int32, device="cuda")
    layer.cache_write(rows, small, low)
    assert same_bytes(layer.cache_read(big, slots), layer.cache_read(small, low))


def test_a_graph_keeps_its_workspace_when_the_layer_needs_a_larger_one():
    case = Case(shape_of(16, 64), [30, 64], 40, True, seed=3)
    layer = case.layer()
    x = case.device_inputs()
    want, _ = layer.latent_attn(**x)
    o, g = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.latent_attn(o_lat=o, **x)
    held = layer.ws.data_ptr()
    layer.prefix_workspace(500, 4000, 4000)
    assert layer.ws.data_ptr() != held
    junk = [torch.full((layer.ws.numel() // 64,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert same_bytes(o, want) and all(bool((j == 255).all()) for j in junk)


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads", [4, 16, 40, 128])
def test_a_workspace_covers_every_smaller_call(heads, fp8):
    layer = layer_of(shape_of(heads, 64), fp8)
    sizes = [(n, p, c) for n in (1, 3, 40, 300) for p in (0, 1, 500) for c in (1, 100, 9000)]
    need = {s: mla.mla_prefix_workspace_bytes(layer.handle, *s) for s in sizes}
    for a in sizes:
        for b in sizes:
            if all(x <= y for x, y in zip(a, b)):
                assert need[a] <= need[b], (a, b)
    # and is accepted: short rows of a batch that was planned for long ones
    case = Case(shape_of(heads, 64), [3, 0, 70], 100, fp8, seed=1)
    x = case.device_inputs()
    ws = torch.empty(mla.mla_prefix_workspace_bytes(layer.handle, 40, 200, 9000), dtype=torch.uint8, device="cuda")
    mla.mla_workspace_init(ws)
    o, lse = torch.empty_like(x["q_abs"]), torch.empty(x["q_abs"].shape[:2], device="cuda")
    mla.mla_latent_attn(layer.handle, ws=ws, o_lat=o, lse=lse, **x)
    check(case, o, lse)


@pytest.mark.parametrize("prefix", [0, 2000])
def test_one_heavy_key_among_many_light_ones(prefix):
    # the first key has probability about 1/2, thousands of others share the rest
    n = 4000
    case = Case(shape_of(16, 64), [n - prefix], prefix, True, seed=2, q_size=0.05)
    s = case.key_slots(0)
    q = case.q_abs[0].double().mean(0)
    case.q_abs[0] = q.bfloat16()[None].expand(16, -1) + case.q_abs[0] * 0.1
    u = case.q_abs[0].double().mean(0)
    case.rows[s[0], :512] = (u / u.norm() ** 2 * np.log(n) / case.scale).bfloat16()
    case.keys = row_values(case.shape, case.rows)
    o, lse = case.layer().latent_attn(want_lse=True, **case.device_inputs())
    check(case, o, lse)


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads,bs,prefix", [(16, 64, 0), (16, 64, 100), (128, 64, 100), (4, 24, 50)])
def test_bad_lengths_and_blocks(heads, bs, prefix, fp8):
    lens = [50, 90, 70, 20]
    case = Case(shape_of(heads, bs), lens, prefix, fp8, seed=6)
    layer = case.layer()
    x = case.device_inputs()
    x["context_lens"] = torch.tensor([50, -3, 70, 2 ** 30], dtype=torch.int32, device="cuda")
    o, lse = layer.latent_attn(want_lse=True, **x)
    assert mla.mla_read_device_flag(layer.ws) == mla.MLA_FLAG_BAD_CONTEXT
    want = case.oracle()
    for t in (1, 3):
        want[0][t], want[1][t] = 0.0, -np.inf
    check(case, o, lse, want)
    mla.mla_clear_device_flag(layer.ws)
    # a block id out of range: its rows are left out
    x = case.device_inputs()
    bad = case.table.copy()
    for t, v in ((0, case.n_blocks), (2, -7)):
        bad[t, 0] = v
    x["block_table"] = torch.from_numpy(bad).cuda()
    o, lse = layer.latent_attn(want_lse=True, **x)
    assert mla.mla_read_device_flag(layer.ws) == mla.MLA_FLAG_BAD_BLOCK
    slots = case.key_slots
    case.key_slots = lambda t: np.delete(slots(t), np.arange(prefix, prefix + min(bs, lens[t]))) if t in (0, 2) else slots(t)
    check(case, o, lse)


def test_a_nan_row_stays_visible_and_a_zero_row_counts():
    case = Case(shape_of(16, 64), [200, 200], 0, True, seed=1)
    s = case.key_slots(0)
    case.rows[s[150], 7] = float("nan")
    case.rows[case.key_slots(1)[100], :512] = 0.0
    case.keys = row_values(case.shape, case.rows)
    o, _ = case.layer().latent_attn(**case.device_inputs())
    assert torch.isnan(o[0]).all()
    one = Case.__new__(Case)
    one.__dict__.update(case.__dict__)
    one.lens, one.q_abs, one.q_pe = [200], case.q_abs[1:], case.q_pe[1:]
    one.table = case.table[1:]
    check(one, o[1:], None)


def test_rows_never_written_count_as_zero_rows():
    shape = shape_of(16, 64)
    layer = layer_of(shape, True)
    cache = layer.new_cache(4)
    q = torch.randn(1, 16, 512, device="cuda").bfloat16()
    pe = torch.randn(1, 16, 64, device="cuda").bfloat16()
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    o, lse = layer.latent_attn(q, pe, cache, table, torch.tensor([100], dtype=torch.int32, device="cuda"), 100, want_lse=True)
    assert (o == 0).all()
    assert torch.allclose(lse, torch.full_like(lse, float(np.log(100.0))), atol=1e-5)


# ---------------------------------------------------------------------------
# the layer's own paths on an 8-bit cache
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["v2lite_bf16", "tiny_fp32", "v3_fp8"])
def test_front_folds_write_what_cache_write_would(name):
    w = wl.WORKLOADS[name]
    shape = dataclasses.replace(w.shape, hidden=512 if name == "v3_fp8" else w.shape.hidden,
                                n_heads=4, q_lora_rank=128 if name == "v3_fp8" else w.shape.q_lora_rank)
    from head_latent_attention_decode_b200.layer import MlaLayer
    weights = wl.make_weights(shape, 5)
    plain, quant = MlaLayer(shape, weights), MlaLayer(shape, weights, cache_dtype="fp8")
    n, act = 37, ACT[shape.act_dtype]
    x = torch.randn(n, shape.hidden, device="cuda").to(act)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 3
    cos, sin = plain.rope(pos)
    bs = shape.block_size
    n_blocks = n // bs + 2
    slots = torch.randperm(n_blocks * bs, device="cuda")[:n].int()
    slots[4] = -1
    rows16, got, want = plain.new_cache(n_blocks), quant.new_cache(n_blocks), quant.new_cache(n_blocks)
    for call in ("decode", "noalloc", "prefill"):
        for layer, cache in ((plain, rows16), (quant, got)):
            cache.zero_()
            if call == "decode":
                layer.decode_qkv(x, cos, sin, cache, slots)
            elif call == "noalloc":
                q_abs = torch.empty((n, shape.n_heads, shape.kv_lora_rank), dtype=act, device="cuda")
                q_pe = torch.empty((n, shape.n_heads, shape.qk_rope), dtype=act, device="cuda")
                mla.mla_decode_qkv_noalloc(layer.handle, x, cos, sin, cache, slots, q_abs, q_pe)
            else:
                layer.prefill(x, cos, sin, kv_cache=cache, slot_mapping=slots)
        want.zero_()
        keep = slots >= 0
        rows = rows16.reshape(n_blocks * bs, -1)[slots[keep].long()].contiguous()
        quant.cache_write(rows, want, slots[keep].contiguous())
        assert int((want != 0).sum()) > 0 and same_bytes(got, want), call
    assert mla.mla_read_device_flag(quant.ws) == 0


@pytest.mark.parametrize("heads", [16, 128])
def test_serving_a_batch_over_a_shared_prompt(heads):
    """Prefill a prompt into the 8-bit cache, read it back, decode a batch over it: the steps as a
    server runs them, against the same steps with the values read back into a 16-bit cache."""
    shape = dataclasses.replace(wl.V2LITE, hidden=512, n_heads=heads)
    from head_latent_attention_decode_b200.layer import MlaLayer
    weights = wl.make_weights(shape, 7)
    quant, plain = MlaLayer(shape, weights, cache_dtype="fp8"), MlaLayer(shape, weights)
    S, n, bs = 192, 5, 64
    perm = torch.randperm(3 + n + 1, device="cuda").int()
    ptable, own = perm[:3].contiguous(), perm[3:3 + n].view(n, 1).contiguous()
    n_blocks = perm.numel()
    cache = quant.new_cache(n_blocks)
    x = torch.randn(S, shape.hidden, device="cuda").bfloat16()
    cos, sin = quant.rope(torch.arange(S, dtype=torch.int32, device="cuda"))
    p = torch.arange(S, device="cuda")
    quant.prefill(x, cos, sin, kv_cache=cache, slot_mapping=(ptable[p // bs] * bs + p % bs).int())
    for step in range(3):
        h = torch.randn(n, shape.hidden, device="cuda").bfloat16()
        cos, sin = quant.rope(torch.full((n,), S + step, dtype=torch.int32, device="cuda"))
        q_abs, q_pe = quant.decode_qkv(h, cos, sin, cache, own[:, 0] * bs + step)
        ctx = torch.full((n,), step + 1, dtype=torch.int32, device="cuda")
        head = torch.empty((n, heads, shape.v_dim), dtype=torch.bfloat16, device="cuda")
        out = quant.decode_attn_prefix(q_abs, q_pe, cache, ptable, S, own, ctx, step + 1, head_out=head)
        # the whole context as one table per sequence, on both caches
        table = torch.cat([ptable[None].expand(n, 3), own], 1).contiguous()
        full = ctx + S
        one = quant.decode_attn(q_abs, q_pe, cache, table, full, S + step + 1)
        c16 = quant.cache_read(cache, torch.arange(n_blocks * bs, dtype=torch.int32, device="cuda"))
        want = plain.decode_attn(q_abs, q_pe, c16.view(n_blocks, 1, bs, -1), table, full, S + step + 1)
        scale = want.float().abs().max()
        for y in (out, one):   # as the decode path's own parity bound: 2e-2 of the largest
            assert ((y.float() - want.float()).abs().max() / scale) < 2e-2
        pre16 = plain.decode_attn_prefix(q_abs, q_pe, c16.view(n_blocks, 1, bs, -1), ptable, S, own, ctx, step + 1)
        assert ((pre16.float() - want.float()).abs().max() / scale) < 2e-2
        assert torch.isfinite(head.float()).all()
    for layer in (quant, plain):
        assert mla.mla_read_device_flag(layer.ws) == 0


def test_decode_attn_prefix_without_a_prefix_and_fp32():
    case = Case(shape_of(4, 16, act="f32", r_kv=64, d_r=16), [30, 70], 0, False, seed=4)
    layer = case.layer()
    x = case.device_inputs()
    a = layer.decode_attn(x["q_abs"], x["q_pe"], x["kv_cache"], x["block_table"], x["context_lens"], 70)
    b = layer.decode_attn_prefix(x["q_abs"], x["q_pe"], x["kv_cache"], None, 0, x["block_table"], x["context_lens"], 70)
    assert torch.allclose(a, b, rtol=1e-4, atol=1e-6)


def test_host_step_on_an_8bit_cache():
    shape = dataclasses.replace(wl.V2LITE, hidden=512)
    from head_latent_attention_decode_b200.layer import MlaLayer
    layer = MlaLayer(shape, wl.make_weights(shape, 3), cache_dtype="fp8")
    n, ctx = 3, 90
    cache = layer.new_cache(8)
    rows = torch.randn(8 * 64, shape.kv_row_dim, device="cuda").bfloat16()
    layer.cache_write(rows, cache, torch.arange(512, dtype=torch.int32, device="cuda"))
    table = torch.tensor([[0, 3], [5, 1], [2, 7]], dtype=torch.int32)
    lens = torch.full((n,), ctx, dtype=torch.int32)
    slots = table[:, 1] * 64 + (ctx - 1) % 64
    pos = lens - 1
    h = torch.randn(n, shape.hidden).bfloat16()
    ws = layer.workspace(n, ctx)
    stage = torch.empty(mla.mla_decode_step_host_bytes(layer.handle, n, 2), dtype=torch.uint8, device="cuda")
    out = torch.empty(n, shape.hidden).bfloat16()
    c2 = cache.clone()
    mla.mla_decode_step_host(layer.handle, h, pos, slots, table, lens, ctx, 10000.0, c2, out, stage, ws)
    torch.cuda.synchronize()
    cos, sin = layer.rope(pos.cuda())
    q_abs, q_pe = layer.decode_qkv(h.cuda(), cos, sin, cache, slots.cuda())
    want = layer.decode_attn(q_abs, q_pe, cache, table.cuda(), lens.cuda(), ctx)
    assert same_bytes(cache, c2) and same_bytes(out, want)


# ---------------------------------------------------------------------------
# streams, graphs, workspaces, refusals
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads", [16, 128])
def test_repeats_graphs_and_other_streams_give_the_same_bits(heads, fp8):
    case = Case(shape_of(heads, 64), [1, 200, 64, 0], 150, fp8, seed=8)
    layer = case.layer()
    x = case.device_inputs()
    want, wl_ = layer.latent_attn(want_lse=True, **x)
    check(case, want, wl_)
    for _ in range(3):
        o, lse = layer.latent_attn(want_lse=True, **x)
        same = same_bytes(o, want) and same_bytes(lse, wl_)
        assert same
    # a stream of its own with a workspace of its own, at the same time
    other = case.layer()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    outs = []
    for _ in range(4):
        outs.append(layer.latent_attn(**x)[0])
        with torch.cuda.stream(st):
            outs.append(other.latent_attn(**x)[0])
    torch.cuda.synchronize()
    same = [same_bytes(o, want) for o in outs]
    assert all(same)
    # two graphs that share a workspace, replayed in turn on changed inputs
    outs, graphs = [torch.empty_like(want) for _ in range(2)], []
    xs = [x, dict(x, q_abs=x["q_abs"].flip(0).contiguous(), q_pe=x["q_pe"].flip(0).contiguous(),
                  context_lens=x["context_lens"].flip(0).contiguous(), block_table=x["block_table"].flip(0).contiguous())]
    # (the schedule cuts the flipped batch at other rows, so its bits are those of its own eager call)
    wants = [want, layer.latent_attn(**xs[1])[0]]
    a, _, ba, _ = case.oracle()
    assert (np.abs(wants[1].flip(0).double().cpu().numpy() - a) <= ba).all()
    for y, o in zip(xs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.latent_attn(o_lat=o, **y)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        same = [same_bytes(o, y) for o, y in zip(outs, wants)]
        assert same == [True, True]
    assert mla.mla_read_device_flag(layer.ws) == 0


def test_cache_calls_in_a_graph():
    shape = shape_of(16, 64)
    layer = layer_of(shape, True)
    cache = layer.new_cache(3)
    rows = torch.randn(100, 576, device="cuda").bfloat16()
    slots = torch.randperm(192, device="cuda")[:100].int()
    out = torch.zeros_like(rows)
    layer.workspace(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.cache_write(rows, cache, slots)
        layer.cache_read(cache, slots, out)
    for seed in range(2):
        rows.copy_(torch.randn_like(rows))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), row_values(shape, rows.cpu()))


def test_refusals():
    shape = shape_of(16, 64)
    layer = layer_of(shape, True)
    L = mla.lib()
    h = layer.handle
    assert L.mla_set_cache_dtype(h, 9) == mla.MLA_ERR_INVALID_ARG
    assert L.mla_set_cache_dtype(h, mla.MLA_F32) == mla.MLA_ERR_UNSUPPORTED
    assert mla.mla_prefix_workspace_bytes(h, 1, -1, 1) == 0 and mla.mla_prefix_workspace_bytes(h, 1, 2 ** 30, 1) == 0
    case = Case(shape, [10, 20], 30, True, seed=0)
    x = case.device_inputs()
    ws = layer.prefix_workspace(2, 30, 20)
    o = torch.empty_like(x["q_abs"])
    kw = {k: v for k, v in x.items()}

    def status(**change):
        a = dict(kw, ws=ws, o_lat=o)
        a.update(change)
        with pytest.raises(mla.MlaError) as e:
            mla.mla_latent_attn(h, **a)
        return e.value.status

    assert status(prefix_len=-1) == mla.MLA_ERR_INVALID_ARG
    assert status(max_context_len=0) == mla.MLA_ERR_INVALID_ARG
    assert status(ws=ws[:1024]) == mla.MLA_ERR_WORKSPACE
    assert status(prefix_len=2 ** 30) == mla.MLA_ERR_UNSUPPORTED
    odd = torch.empty(x["kv_cache"].numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(x["kv_cache"].shape)
    assert status(kv_cache=odd) == mla.MLA_ERR_INVALID_ARG
    for bad in (dict(prefix_table=None), dict(q_pe=x["q_pe"][:1].contiguous()), dict(o_lat=o.float()),
                dict(context_lens=x["context_lens"].long()), dict(q_abs=x["q_abs"].transpose(0, 1)),
                dict(lse=torch.empty(2, 16, device="cuda").double()), dict(block_table=x["block_table"][:1].contiguous())):
        with pytest.raises(ValueError):
            mla.mla_latent_attn(h, **{**kw, "ws": ws, "o_lat": o, **bad})
    rows = torch.zeros(2, 576, device="cuda").bfloat16()
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mla.mla_cache_write(h, rows, x["kv_cache"], slots[:1].contiguous(), ws)
    with pytest.raises(ValueError):
        layer.cache_write(rows.float(), x["kv_cache"], slots)
    with pytest.raises(ValueError):
        layer.cache_write(rows, x["kv_cache"][:, :-128].contiguous(), slots)
    with pytest.raises(ValueError):
        layer.latent_attn(**dict(x, prefix_len=65))
    # nothing to do is no error
    mla.mla_cache_write(h, rows[:0], x["kv_cache"], slots[:0], ws)
    mla.mla_latent_attn(h, **dict(kw, q_abs=x["q_abs"][:0], q_pe=x["q_pe"][:0], block_table=x["block_table"][:0],
                                  context_lens=x["context_lens"][:0]), ws=ws, o_lat=o[:0])


def test_a_cache_of_the_other_kind_is_refused():
    shape = shape_of(16, 64)
    eight, full = layer_of(shape, True), layer_of(shape, False)
    c8, c16 = eight.new_cache(4), full.new_cache(4)
    hidden = torch.zeros(1, shape.hidden, device="cuda").bfloat16()
    cos, sin = full.rope(torch.zeros(1, dtype=torch.int32, device="cuda"))
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_abs, q_pe = full.decode_qkv(hidden, cos, sin, c16, slot)
    table, one = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for layer, cache in ((eight, c16), (full, c8)):
        for call in (lambda: layer.decode_qkv(hidden, cos, sin, cache, slot),
                     lambda: layer.decode_attn(q_abs, q_pe, cache, table, one, 1),
                     lambda: layer.prefill(hidden, cos, sin, kv_cache=cache, slot_mapping=slot),
                     lambda: layer.latent_attn(q_abs, q_pe, cache, table, one, 1),
                     lambda: layer.decode_attn_prefix(q_abs, q_pe, cache, table[0], 1, table, one, 1)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        eight.latent_attn(q_abs, q_pe, c8, table, one, 1, prefix_len=1)   # without a table


def test_block_bytes():
    for name, act in (("latent512", "bf16"), ("odd_block", "f32")):
        shape = shape_of(4, act=act, **SHAPES[name])
        _, _, size = lr.block_layout(shape.block_size, shape.kv_lora_rank, shape.qk_rope, ESZ[act])
        assert mla.mla_cache_block_bytes(layer_of(shape, True).handle) == size
        assert mla.mla_cache_block_bytes(layer_of(shape, False).handle) == shape.block_size * shape.kv_row_dim * ESZ[act]


# ---------------------------------------------------------------------------
# workspaces at any 16-byte boundary
# ---------------------------------------------------------------------------

def workspace_at(nbytes, offset):
    """A zeroed workspace `offset` bytes past a 256-byte boundary."""
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device="cuda")[offset:offset + nbytes]
    assert ws.data_ptr() % 256 == offset
    mla.mla_workspace_init(ws)
    return ws


@pytest.mark.parametrize("offset", [16, 48])
@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads,prefix", [(16, 0), (16, 100), (40, 0), (128, 0), (128, 100)])
def test_a_workspace_at_a_16_byte_boundary(heads, prefix, fp8, offset):
    case = Case(shape_of(heads, 64), [70, 3, 130], prefix, fp8, seed=heads)
    layer = case.layer()
    x = case.device_inputs()
    want, wl_ = layer.latent_attn(want_lse=True, **x)
    ws = workspace_at(mla.mla_prefix_workspace_bytes(layer.handle, 3, prefix, 130), offset)
    o, lse = torch.empty_like(want), torch.empty_like(wl_)
    mla.mla_latent_attn(layer.handle, ws=ws, o_lat=o, lse=lse, **x)
    assert same_bytes(o, want) and same_bytes(lse, wl_)
    if not prefix:   # the call that was there before
        args = [x[k] for k in ("q_abs", "q_pe", "kv_cache", "block_table", "context_lens", "max_context_len")]
        out = torch.empty(3, case.shape.hidden, dtype=torch.bfloat16, device="cuda")
        ws = workspace_at(mla.mla_workspace_bytes(layer.handle, 3, 130), offset)
        mla.mla_decode_attn(layer.handle, *args, out, ws)
        assert same_bytes(out, layer.decode_attn(*args))


def test_other_alignments_of_a_workspace_are_refused():
    case = Case(shape_of(16, 64), [10, 20], 30, True, seed=0)
    layer = case.layer()
    x = case.device_inputs()
    o = torch.empty_like(x["q_abs"])
    need = mla.mla_prefix_workspace_bytes(layer.handle, 2, 30, 20)
    ws = torch.zeros(need + 8, dtype=torch.uint8, device="cuda")[8:]
    args = [x[k] for k in ("q_abs", "q_pe", "kv_cache", "block_table", "context_lens", "max_context_len")]
    rows, slots = torch.zeros(1, 576, device="cuda").bfloat16(), torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda: mla.mla_latent_attn(layer.handle, ws=ws, o_lat=o, **x),
                 lambda: mla.mla_decode_attn(layer.handle, *args, torch.empty(2, 256, device="cuda").bfloat16(), ws),
                 lambda: mla.mla_cache_write(layer.handle, rows, x["kv_cache"], slots, ws[1:])):
        with pytest.raises(mla.MlaError) as e:
            call()
        assert e.value.status == mla.MLA_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# queries and outputs of another layer's shape or type
# ---------------------------------------------------------------------------

def test_queries_and_outputs_of_another_shape_or_type_are_refused():
    case = Case(shape_of(16, 64), [10, 20], 30, True, seed=0)
    layer, x = case.layer(), case.device_inputs()
    qa, qp = x["q_abs"], x["q_pe"]
    prefix = (x.pop("prefix_table"), x.pop("prefix_len"))
    rest = [x[k] for k in ("block_table", "context_lens", "max_context_len")]
    queries = [(qa[:, :8], qp[:, :8]), (qa[..., :256], qp), (qa, qp[..., :32]), (qa.float(), qp.float()),
               (qa.half(), qp.half()), (qa, qp.float()), (qa.flatten(1), qp.flatten(1)), (qa, qp[:1])]
    for a, b in queries:
        a, b = a.contiguous(), b.contiguous()
        with pytest.raises(ValueError):
            layer.latent_attn(a, b, x["kv_cache"], *rest, prefix_table=prefix[0], prefix_len=prefix[1])
        with pytest.raises(ValueError):
            layer.decode_attn_prefix(a, b, x["kv_cache"], *prefix, *rest)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    hidden, heads, dv = case.shape.hidden, case.shape.n_heads, case.shape.v_dim
    for bad in (dict(out=torch.empty(2, hidden // 2, **bf)), dict(out=torch.empty(1, hidden, **bf)),
                dict(out=torch.empty(2, hidden, device="cuda")), dict(head_out=torch.empty(2, heads // 2, dv, **bf)),
                dict(head_out=torch.empty(2, heads, dv // 2, **bf)), dict(head_out=torch.empty(1, heads, dv, **bf)),
                dict(head_out=torch.empty(2, heads, dv, device="cuda"))):
        with pytest.raises(ValueError):
            layer.decode_attn_prefix(qa, qp, x["kv_cache"], *prefix, *rest, **bad)
    # the binding, which does not know the layer, compares them with the query
    ws, out = layer.prefix_workspace(2, 30, 20), torch.empty(2, hidden, **bf)
    for bad in (dict(out=out[:1]), dict(out=out.float()), dict(head_out=torch.empty(2, 8, dv, **bf)),
                dict(head_out=torch.empty(2, heads, dv, device="cuda"))):
        kw = dict(out=out, head_out=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            mla.mla_decode_attn_prefix(layer.handle, qa, qp, x["kv_cache"], *prefix, *rest, kw["out"], ws, head_out=kw["head_out"])


# ---------------------------------------------------------------------------
# NaN and infinite scores
# ---------------------------------------------------------------------------

def dead_and_alive(case, layer, x, want, dead, lse=True):
    """The (sequence, head) pairs of `dead` give NaN, the others what they gave without it."""
    o, s = layer.latent_attn(want_lse=lse, **x)
    o, wo, wl_, bo, bl = o.double().cpu().numpy(), *want
    assert np.isnan(o[dead]).all()
    assert (np.abs(o - wo) <= bo)[~dead].all()
    if lse:
        s = s.double().cpu().numpy()
        assert np.isnan(s[dead]).all() and (np.abs(s - wl_) <= bl)[~dead].all()
    assert mla.mla_read_device_flag(layer.ws) == 0


NAN_ROUTES = [(16, 64, 0, True), (16, 64, 0, False), (16, 16, 0, True), (40, 64, 0, True), (40, 64, 0, False),
              (128, 64, 0, True), (128, 64, 0, False), (130, 64, 0, True), (16, 64, 70, True), (16, 64, 70, False),
              (4, 24, 0, True), (4, 24, 0, False)]


@pytest.mark.parametrize("last", [1, 65, 129, 257, 300])
@pytest.mark.parametrize("heads,bs,prefix,fp8", NAN_ROUTES)
def test_a_nan_in_the_newest_row_stays_visible(heads, bs, prefix, fp8, last):
    # alone in its tile for most lengths, so that no finite score stands beside it
    case = Case(shape_of(heads, bs), [last, 200, last], prefix, fp8, seed=last)
    want = case.oracle()
    case.rows[case.key_slots(0)[-1], 5] = float("nan")
    dead = np.zeros((3, heads), bool)
    dead[0] = True
    dead_and_alive(case, case.layer(), case.device_inputs(), want, dead)


@pytest.mark.parametrize("heads,n", [(4, 3), (16, 2), (16, 5), (128, 2)])
@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
def test_a_nan_in_the_last_row_of_a_prefix_stays_visible(heads, n, fp8):
    case = Case(shape_of(heads, 64), [3, 0, 70, 5, 0][:n], 129, fp8, seed=n)
    want = case.oracle()
    case.rows[case.key_slots(0)[128], 5] = float("nan")
    dead_and_alive(case, case.layer(), case.device_inputs(), want, np.ones((n, heads), bool))


@pytest.mark.parametrize("heads,bs,prefix,fp8", NAN_ROUTES)
def test_a_nan_in_a_query_head_spoils_that_head_alone(heads, bs, prefix, fp8):
    case = Case(shape_of(heads, bs), [1, 300, 129], prefix, fp8, seed=heads)
    want = case.oracle()
    x = case.device_inputs()
    dead = np.zeros((3, heads), bool)
    for t, h, c in ((0, heads - 1, 3), (1, 1, 300), (2, 0, 511)):
        x["q_abs"][t, h, c] = float("nan")
        dead[t, h] = True
    dead_and_alive(case, case.layer(), x, want, dead)


@pytest.mark.parametrize("heads,bs,prefix,fp8", NAN_ROUTES)
def test_infinite_rotary_keys(heads, bs, prefix, fp8):
    # score +inf where the query's entry is positive (NaN out), -inf where it is negative (the key has no weight)
    case = Case(shape_of(heads, bs), [129, 40, 1], prefix, fp8, seed=heads + 1)
    slots_of = [case.key_slots(t) for t in range(3)]
    slots, at = case.key_slots, {0: prefix + 128, 1: prefix + 7}
    case.lens, case.key_slots = [128, 39, 1], lambda t: np.delete(slots_of[t], at[t]) if t in at else slots_of[t]
    want = case.oracle()   # without those keys
    case.lens, case.key_slots = [129, 40, 1], slots
    for t, j in at.items():
        case.rows[slots_of[t][j], case.shape.kv_lora_rank + 2] = float("inf")
    dead = case.q_pe[:, :, 2].double().numpy() > 0
    dead[2] = False
    dead_and_alive(case, case.layer(), case.device_inputs(), want, dead, lse=False)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "plain"])
@pytest.mark.parametrize("heads", [16, 40])
def test_decode_attn_shows_a_nan_too(heads, fp8, act):
    small = dict(r_kv=64, d_r=16) if act == "f32" else {}
    case = Case(shape_of(heads, 64, act=act, **small), [3000, 200, 2049], 0, fp8, seed=heads)
    layer, x = case.layer(), case.device_inputs()
    args = lambda x: [x[k] for k in ("q_abs", "q_pe", "kv_cache", "block_table", "context_lens", "max_context_len")]  # noqa: E731
    head = torch.empty(3, heads, case.shape.v_dim, dtype=ACT[act], device="cuda")
    want = layer.decode_attn(*args(x), head_out=head)
    whole = head.clone()
    for t in (0, 2):   # among 951 other rows of its split, and alone in its tile
        case.rows[case.key_slots(t)[-1], 5] = float("nan")
    out = layer.decode_attn(*args(case.device_inputs()), head_out=head)
    assert torch.isnan(head[0::2]).all() and torch.isnan(out[0::2]).all()
    assert same_bytes(head[1], whole[1]) and same_bytes(out[1], want[1])


# ---------------------------------------------------------------------------
# the log-sum-exp on every route that returns one
# ---------------------------------------------------------------------------

LSE_ROUTES = {
    # name: (heads, own lengths, prefix, 8-bit)
    "16_heads_16bit": (16, [700, 300, 64, 130], 0, False),
    "5_heads_16bit": (5, [700, 300, 64, 130], 0, False),
    "32_heads_16bit": (32, [700, 300, 64, 130], 0, False),
    "40_heads_16bit": (40, [700, 300, 64, 130], 0, False),
    "128_heads_16bit": (128, [700, 300, 64, 130], 0, False),
    # ten sequences of up to 3840 rows are 600 tiles of 64: more than the prefix's launch takes along
    "16_heads_16bit_prefix_and_long_rows": (16, [3840] + [90] * 9, 100, False),
    "24_heads_16bit_prefix_and_long_rows": (24, [3840] + [90] * 9, 100, False),
    "16_heads_8bit": (16, [700, 300, 64, 130], 0, True),
    "40_heads_8bit": (40, [700, 300, 64, 130], 0, True),
    "130_heads_8bit": (130, [300, 130], 0, True),
    "4_heads_8bit_prefix": (4, [90, 64, 150], 700, True),
    "16_heads_8bit_prefix_and_long_rows": (16, [3840] + [90] * 9, 100, True),
}


@pytest.mark.parametrize("name", list(LSE_ROUTES))
def test_the_lse_is_good_to_fp32_on_every_route(name):
    # What is left is fp32: sums of 576 products, exponentials, sums of weights, all below 2^-20 of a
    # score of a few units; where partial scores cross in f16 and their first order is taken out, as in
    # test_the_lse_is_good_to_fp32, below 2^-20 over sixty keys and more. 2e-6 of an lse of about 5 is 10 times
    # that. Partials rounded to f16 leave 3e-5, row sums of weights rounded to bf16 2^-9 / sqrt(keys) / 5 = 5e-5.
    heads, lens, prefix, fp8 = LSE_ROUTES[name]
    case = Case(shape_of(heads, 64), lens, prefix, fp8, seed=23)
    size = 2.0 ** np.floor(np.log2(np.abs(case.rows[:, :512].float().numpy()).mean(1, keepdims=True) + 1e-30))
    size[~np.isfinite(size)] = 1.0
    case.rows[:, :512] /= torch.from_numpy(size).bfloat16()   # rows of one size, as a norm leaves them
    case.keys = row_values(case.shape, case.rows) if fp8 else case.rows.double().numpy()
    layer = case.layer()
    o, lse = layer.latent_attn(want_lse=True, **case.device_inputs())
    want = case.oracle()
    check(case, o, lse, want)
    err = lse.double().cpu().numpy() - want[1]
    assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(want[1])


# ---------------------------------------------------------------------------
# partial scores near f16's largest, and infinite ones
# ---------------------------------------------------------------------------

CORR_ROUTES = [(128, 0, True), (128, 0, False), (16, 150, True), (16, 150, False), (40, 100, False)]


@pytest.mark.parametrize("heads,prefix,fp8", CORR_ROUTES)
def test_the_lse_with_partial_scores_near_the_largest_of_f16(heads, prefix, fp8):
    # The halves of a score are near +-50000, where f16's steps are 32 (1.15 nat after the scale for half a
    # step), and cancel: a score of a few nats. One key, or one heavy key of many, holds nearly all the weight
    # (e^-40 elsewhere), so that its own rounding is all there is to take out: lse is its score.
    # fp32 sums of halves of 5e4 and their difference: 2^-24 512 5e4 scale = 0.11 at the worst, 2^-24 sqrt(512)
    # 5e4 scale = 5e-3 for products of either sign. Without the correction up to 1.15 and 0.6 on average.
    case = Case(shape_of(heads, 64), [1, 130], prefix, fp8, seed=3)
    rng = np.random.default_rng(7)
    q = np.sign(rng.standard_normal(512)) * 2.0 ** rng.integers(4, 6, 512)   # one direction for every head, but for
    q[500] = 0.0                                                             # a column that moves them to all places
    case.q_abs[:] = torch.from_numpy(q).bfloat16()                           # between two f16 values
    case.q_abs[:, :, 500] = torch.arange(heads).bfloat16()
    case.q_pe[:] = 0
    a = np.sign(q) * np.where(np.arange(512) < 256, 1.0, -1.0) * 8.0
    case.rows[:] = 0
    for t in range(2):
        for n, s in enumerate(case.key_slots(t)):
            row = np.zeros(576)
            if n == 0:
                row[:512] = a * rng.choice([0.875, 1.0, 1.125], 512)
                half = [float(q[:256] @ row[:256]), float(q[256:] @ row[256:512])]
                k = 300 + np.argmax(np.abs(q[300:]))     # bring the sum to about 200 (14 nats and more)
                row[k] += (200 - sum(half)) / q[k]
                row[500] = 1.0
            else:
                row[:512] = -np.sign(q) * 0.0625          # far below
            case.rows[s] = torch.from_numpy(row).bfloat16()
    case.keys = row_values(case.shape, case.rows) if fp8 else case.rows.double().numpy()
    o, lse = case.layer().latent_attn(want_lse=True, **case.device_inputs())
    lse = lse.double().cpu().numpy()
    for t in range(2):
        k = case.keys[case.key_slots(t)]
        _, want, p = lr.latent_attention(case.q_abs[t].double().numpy(), case.q_pe[t].double().numpy(), k[:, :512], k[:, 512:], case.scale)
        h = case.q_abs[t].double().numpy()
        h = np.abs([h[:, :256] @ k[0, :256], h[:, 256:] @ k[0, 256:512]])
        assert 3e4 < h.min() and h.max() < 65504 and p[:, 0].min() > 1 - 1e-9
        assert np.abs(h - np.float16(h)).max() * case.scale > 0.5
        assert np.isfinite(lse[t]).all() and np.abs(lse[t] - want).max() <= 0.02


@pytest.mark.parametrize("heads,bs,prefix,fp8", NAN_ROUTES)
def test_keys_that_an_infinite_score_takes_out(heads, bs, prefix, fp8):
    # -inf for every head: the row has no weight, in o and in the log-sum-exp
    case = Case(shape_of(heads, bs), [129, 40, 1], prefix, fp8, seed=heads + 2)
    case.q_pe[:, :, 2] = -case.q_pe[:, :, 2].abs() - 0.125
    slots_of = [case.key_slots(t) for t in range(3)]
    slots, at = case.key_slots, {0: prefix + 128, 1: prefix + 7}
    case.lens, case.key_slots = [128, 39, 1], lambda t: np.delete(slots_of[t], at[t]) if t in at else slots_of[t]
    want = case.oracle()   # without those keys
    case.lens, case.key_slots = [129, 40, 1], slots
    for t, j in at.items():
        case.rows[slots_of[t][j], case.shape.kv_lora_rank + 2] = float("inf")
    dead_and_alive(case, case.layer(), case.device_inputs(), want, np.zeros((3, heads), bool))


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads,prefix", [(128, 0), (40, 0), (16, 6400)])
def test_keys_that_an_infinite_score_takes_out_of_long_rows(heads, prefix, fp8):
    # several tiles to a cluster: the rotary keys of every second one belong to the CTA that sums the correction
    lens = [40] if prefix else [9600, 40]
    case = Case(shape_of(heads, 64), lens, prefix, fp8, seed=heads + 3)
    case.q_pe[:, :, 2] = -case.q_pe[:, :, 2].abs() - 0.125
    slots_of = [case.key_slots(t) for t in range(len(lens))]
    gone = np.arange(70, 64 * 12, 64)
    slots = case.key_slots
    if prefix:
        case.prefix_len -= len(gone)
    else:
        case.lens[0] -= len(gone)
    case.key_slots = lambda t: np.delete(slots_of[t], gone) if t == 0 else slots_of[t]
    want = case.oracle()   # without those keys
    case.lens, case.prefix_len, case.key_slots = lens, prefix, slots
    case.rows[slots_of[0][gone], case.shape.kv_lora_rank + 2] = float("inf")
    dead_and_alive(case, case.layer(), case.device_inputs(), want, np.zeros((len(lens), heads), bool))


# ---------------------------------------------------------------------------
# a layer's workspace: graphs that hold it, streams that share it, growth
# ---------------------------------------------------------------------------

def decode_layer(fp8, heads=16):
    from head_latent_attention_decode_b200.layer import MlaLayer
    shape = dataclasses.replace(wl.V2LITE, hidden=512, n_heads=heads)
    return MlaLayer(shape, wl.make_weights(shape, 3), cache_dtype="fp8" if fp8 else None)


def step_inputs(layer, n=3, ctx=90, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = layer.shape
    table = torch.randperm(2 * n, generator=g, device="cuda").int().view(n, 2)
    cache = layer.new_cache(2 * n)
    rows = torch.randn(2 * n * 64, shape.kv_row_dim, generator=g, device="cuda").bfloat16()
    layer.cache_write(rows, cache, torch.arange(2 * n * 64, dtype=torch.int32, device="cuda"))
    lens = torch.full((n,), ctx, dtype=torch.int32, device="cuda")
    cos, sin = layer.rope(lens - 1)
    h = torch.randn(n, shape.hidden, generator=g, device="cuda").bfloat16()
    slots = (table[:, (ctx - 1) // 64] * 64 + (ctx - 1) % 64).int()

    def step(out=None):
        q_abs, q_pe = layer.decode_qkv(h, cos, sin, cache, slots)
        return layer.decode_attn(q_abs, q_pe, cache, table, lens, ctx, out=out)

    return step


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("warm", [True, False])
def test_a_decode_step_in_a_graph_outlives_a_larger_workspace(fp8, warm):
    layer = decode_layer(fp8)
    want = step_inputs(decode_layer(fp8))()     # (another layer's, with a workspace of its own)
    step = step_inputs(layer)
    if warm:
        step()
    else:
        layer.ws = None                         # nothing but the captured calls has asked for one
    out, g = torch.empty_like(want), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(out)
    held = layer.ws.data_ptr() if warm else None
    layer.prefix_workspace(500, 4000, 4000)
    assert layer.ws.data_ptr() != held and mla.mla_read_device_flag(layer.ws) == 0
    junk = [torch.full((layer.ws.numel() // 64,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for _ in range(2):
        out.zero_()
        g.replay()
        assert same_bytes(step(), want)         # an eager call between replays
        torch.cuda.synchronize()
        assert same_bytes(out, want) and all(bool((j == 255).all()) for j in junk)


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads", [16, 128])
def test_two_streams_share_a_layer(heads, fp8):
    case = Case(shape_of(heads, 64), [1, 2000, 640, 0], 1500, fp8, seed=8)
    layer = case.layer()
    x = case.device_inputs()
    y = dict(x, q_abs=x["q_abs"].flip(1).contiguous(), q_pe=x["q_pe"].flip(1).contiguous())
    wants = [layer.latent_attn(want_lse=True, **z) for z in (x, y)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(layer.latent_attn(want_lse=True, **(x, y)[i % 2]))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(outs):
        assert same_bytes(o, wants[i % 2][0]) and same_bytes(lse, wants[i % 2][1]), i


def test_a_workspace_grows_while_another_stream_uses_it():
    case = Case(shape_of(16, 64), [2000, 900], 0, True, seed=2)
    layer = case.layer()
    x = case.device_inputs()
    want, _ = layer.latent_attn(**x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        outs = [layer.latent_attn(**x)[0] for _ in range(20)]
    old = layer.ws.numel()
    layer.prefix_workspace(400, 4000, 4000)
    junk = [torch.full((old,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]   # where the old one was, if free
    torch.cuda.synchronize()
    assert all([same_bytes(o, want) for o in outs]) and all(bool((j == 255).all()) for j in junk)


def test_the_device_flag_survives_a_larger_workspace():
    shape = shape_of(16, 64)
    layer = layer_of(shape, True)
    rows, slot = torch.zeros(1, 576, device="cuda").bfloat16(), torch.tensor([999], dtype=torch.int32, device="cuda")
    layer.cache_write(rows, layer.new_cache(1), slot)
    small = layer.ws
    layer.prefix_workspace(300, 4000, 4000)
    assert layer.ws is not small and mla.mla_read_device_flag(layer.ws) == mla.MLA_FLAG_BAD_SLOT
    mla.mla_clear_device_flag(layer.ws)
    assert mla.mla_read_device_flag(layer.ws) == 0


# ---------------------------------------------------------------------------
# what a workspace holds
# ---------------------------------------------------------------------------

def misaligned(t):
    """The same values at an address that is a multiple of an element alone."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    buf.copy_(t)
    assert buf.data_ptr() % 16 and buf.is_contiguous()
    return buf


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads,lens,prefix,aligned", [
    (16, [1, 200, 64], 0, True), (16, [1, 200, 64], 0, False), (16, [0, 3, 70], 150, True), (16, [0, 3, 70], 150, False),
    (128, [300, 64], 0, True), (128, [300, 64], 0, False), (128, [10, 0], 190, True), (128, [10, 0], 190, False),
    (40, [2111], 0, False), (1, [5], 0, False), (16, [i % 3 + 1 for i in range(900)], 0, False),
    (128, [i % 2 + 1 for i in range(300)], 5, False), (130, [70, 3], 40, True), (130, [70, 3], 40, False)])
def test_calls_stay_within_the_workspace_they_asked_for(heads, lens, prefix, aligned, fp8):
    case = Case(shape_of(heads, 64), lens, prefix, fp8, seed=heads)
    layer, x = case.layer(), case.device_inputs()
    if not aligned:
        x["q_abs"], x["q_pe"] = misaligned(x["q_abs"]), misaligned(x["q_pe"])
    n, ctx = len(lens), max(1, *lens)
    need = mla.mla_prefix_workspace_bytes(layer.handle, n, prefix, ctx)
    want = case.oracle()
    for lse in (True, False):
        buf = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        ws = buf[:need]
        mla.mla_workspace_init(ws)
        o = torch.empty(x["q_abs"].shape, dtype=torch.bfloat16, device="cuda")
        s = torch.empty(x["q_abs"].shape[:2], device="cuda") if lse else None
        mla.mla_latent_attn(layer.handle, ws=ws, o_lat=o, lse=s, **x)
        check(case, o, s, want)
        assert bool((buf[need:] == 0x5A).all()) and mla.mla_read_device_flag(ws) == 0
    if prefix == 0:
        need = mla.mla_workspace_bytes(layer.handle, n, ctx)
        buf = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        mla.mla_workspace_init(buf[:need])
        out = torch.empty(n, case.shape.hidden, dtype=torch.bfloat16, device="cuda")
        head = torch.empty(n, heads, case.shape.v_dim, dtype=torch.bfloat16, device="cuda")
        args = [x[k] for k in ("q_abs", "q_pe", "kv_cache", "block_table", "context_lens", "max_context_len")]
        mla.mla_decode_attn(layer.handle, *args, out, buf[:need], head_out=head)
        assert bool((buf[need:] == 0x5A).all()) and mla.mla_read_device_flag(buf[:need]) == 0
        _, w_uv = ref.split_wkv_b(ref.weights_fp64(weights_of(case.shape))["wkv_b"], heads, case.shape.qk_nope, case.shape.v_dim)
        exact = np.einsum("thr,hrd->thd", want[0], w_uv)
        assert np.abs(head.double().cpu().numpy() - exact).max() <= 2e-2 * np.abs(exact).max()


def test_workspaces_are_no_larger_than_their_kernels_need():
    size = lambda layer, *a: mla.mla_prefix_workspace_bytes(layer.handle, *a)  # noqa: E731
    plain = lambda layer, *a: mla.mla_workspace_bytes(layer.handle, *a)  # noqa: E731
    eight, full = layer_of(shape_of(128, 64), True), layer_of(shape_of(128, 64), False)
    # split partials of 128 rows of 2 KB and their sums: 74 SM pairs and 64 sequences; beside them a step's own buffers
    assert plain(eight, 64, 16384) < 138 * 128 * 2100 + (60 << 20)
    assert size(eight, 64, 0, 16384) == plain(eight, 64, 16384)
    # a prompt, which attends to no cache, asks for no more than on the other cache
    assert plain(eight, 8192, 1) <= plain(full, 8192, 1)
    # a prefix adds its own partials alone
    assert size(full, 64, 8192, 16384) <= plain(full, 64, 16384) + 202 * 128 * 2100
    assert size(eight, 64, 8192, 16384) <= plain(eight, 64, 16384) + 64 * 128 * 2100 + (1 << 20)


# ---------------------------------------------------------------------------
# light keys behind heavy ones
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bs", [64, 16])
def test_light_keys_behind_heavy_ones_keep_their_weight(bs):
    # As many sequences as SMs, so that each CTA has one of 28 tiles of 128 keys. Two tiles of every eight begin
    # with a heavy key; the others have a weight of 2^-15.1 of it, 1.2 % of the sum together. All values share a
    # mean, so that o is that mean whatever the weights, if o and the sum count the same keys: half a step of the
    # heavy key's weight, 2^-8, of the light ones', 2^-4 of 1.2 %, and of o's type, 2^-8 at the worst: 0.0085 in all.
    # Without the light keys o is 0.012 short.
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    shape = shape_of(16, bs)
    layer = layer_of(shape, True)
    n, L = sms, 28 * 128
    g = torch.Generator(device="cuda").manual_seed(1)
    mean = torch.rand(512, generator=g, device="cuda") * 0.4 + 0.55
    mean[0] = 1.0
    mean *= torch.where(torch.rand(512, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    rows = torch.zeros(L, 576, device="cuda")
    rows[:, :512] = mean * (1 + 0.02 * torch.randn(L, 512, generator=g, device="cuda").clamp(-3, 3))
    tile = torch.arange(L, device="cuda") // 128
    heavy = (torch.arange(L, device="cuda") % 128 == 0) & (tile // 2 % 4 == 0)
    rows[:, 512] = torch.where(heavy, 18.125, -0.048)
    cache = layer.new_cache(L // bs)
    slots = torch.arange(L, dtype=torch.int32, device="cuda")
    layer.cache_write(rows.bfloat16(), cache, slots)
    q_abs, q_pe = torch.zeros(n, 16, 512, device="cuda").bfloat16(), torch.zeros(n, 16, 64, device="cuda").bfloat16()
    q_pe[:, :, 0] = 8.0
    table = torch.arange(L // bs, dtype=torch.int32, device="cuda").expand(n, -1).contiguous()
    o, lse = layer.latent_attn(q_abs, q_pe, cache, table, torch.full((n,), L, dtype=torch.int32, device="cuda"), L, want_lse=True)
    keys = layer.cache_read(cache, slots).double()
    s = 8.0 * keys[:, 512] / np.sqrt(192.0)
    p = torch.softmax(s, 0)
    light = float(p[~heavy].sum())
    assert 0.0115 < light < 0.013 and float(p[~heavy].max() / p[heavy].max()) < 2.0 ** -15
    want = p @ keys[:, :512]
    short = (1 - o.double() / want).mean(-1)   # the rounding of single values averages out over the columns
    assert float(short.abs().max()) <= 0.0085
    assert float((lse.double() - torch.logsumexp(s, 0)).abs().max()) <= 1e-5


# ---------------------------------------------------------------------------
# the serving calls against fp64, and errors on average
# ---------------------------------------------------------------------------

def off_by(got, want):
    """(the error's size, its part along the result), both relative to the result's size."""
    d = got.double().cpu().numpy() - want
    return np.linalg.norm(d) / np.linalg.norm(want), abs((d * want).sum()) / (want * want).sum()


def steps_shape(weights, heads, bs=64):
    if weights == "fp8":
        return dataclasses.replace(wl.V3_FP8, hidden=512, n_heads=heads, q_lora_rank=128, block_size=bs)
    return shape_of(heads, bs)


@pytest.mark.parametrize("weights", ["fp8", "bf16"])
@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads,n,prefix", [(16, 3, 0), (16, 3, 150), (16, 1, 700), (40, 5, 70), (128, 3, 0), (128, 3, 150),
                                            (16, 140, 70), (16, 300, 5)])
def test_decode_calls_against_fp64(weights, heads, n, prefix, fp8):
    # o_lat within its bound (Case.oracle; rounded to f16 or bf16), then sums of 512 and heads * 128 products in
    # fp32 and a rounding to 16 bits after each: 2^-8 of the value at most. On average (the roundings of weights,
    # o_lat, head_out and out are independent, each at most 2^-8 / sqrt(3) of the value in the mean square) half of 2^-7;
    # along the result they cancel.
    shape = steps_shape(weights, heads)
    case = Case(shape, [(37 * i) % 260 + 1 for i in range(n)], prefix, fp8, seed=n)
    layer, x = case.layer(), case.device_inputs()
    W = ref.weights_fp64(weights_of(shape))
    _, w_uv = ref.split_wkv_b(W["wkv_b"], heads, shape.qk_nope, shape.v_dim)
    o, _, bo, _ = case.oracle()
    want = np.einsum("thr,hrd->thd", o, w_uv)
    bh = np.einsum("thr,hrd->thd", bo + 2.0 ** -14 * np.abs(o), np.abs(w_uv)) + 2.0 ** -8 * np.abs(want)
    final = want.reshape(n, -1) @ W["wo"]
    bf = bh.reshape(n, -1) @ np.abs(W["wo"]) + 2.0 ** -12 * np.abs(want).reshape(n, -1) @ np.abs(W["wo"]) + 2.0 ** -8 * np.abs(final)
    act = dict(device="cuda", dtype=torch.bfloat16)
    table = [x[k] for k in ("block_table", "context_lens", "max_context_len")]
    for head in (torch.empty(n, heads, shape.v_dim, **act), None):   # with FP8 weights, without head_out: kept in f16
        if prefix:
            out = layer.decode_attn_prefix(x["q_abs"], x["q_pe"], x["kv_cache"], x["prefix_table"], prefix, *table, head_out=head)
        else:
            out = layer.decode_attn(x["q_abs"], x["q_pe"], x["kv_cache"], *table, head_out=head)
        for got, w, b in ((head, want, bh), (out, final, bf)):
            if got is not None:
                assert (np.abs(got.double().cpu().numpy() - w) <= b).all()
                size, along = off_by(got, w)
                assert size <= 2.0 ** -7 and along <= 1e-3, (size, along)
    assert mla.mla_read_device_flag(layer.ws) == 0


@pytest.mark.parametrize("fp8", [True, False], ids=["cache8", "cache16"])
@pytest.mark.parametrize("heads,bs,lens,prefix", [
    (16, 64, [700, 300, 512, 130], 0), (16, 16, [700, 300, 130], 0), (40, 64, [700, 300], 0), (128, 64, [700, 300, 64], 0),
    (16, 64, [100, 70, 200], 900), (4, 64, [90, 200], 700), (128, 64, [70, 200], 500), (130, 64, [300, 90], 100),
    (16, 24, [200, 90], 100)])
def test_errors_on_average(heads, bs, lens, prefix, fp8):
    # o is rounded once to bf16 (at most 2^-8 / sqrt(3) = 2.3e-3 in the mean square, 1.7e-3 for values spread evenly),
    # after weights rounded to bf16, f16 or two E4M3 parts and scores with a half rounded to f16 (2^-12 of a few
    # units), each of whose errors averages out over a hundred keys and more: 3e-3 in all, and along the result,
    # where nothing is left but a steady bias, 3e-4.
    case = Case(shape_of(heads, bs), lens, prefix, fp8, seed=heads + bs)
    size = 2.0 ** np.floor(np.log2(np.abs(case.rows[:, :512].float().numpy()).mean(1, keepdims=True) + 1e-30))
    size[~np.isfinite(size)] = 1.0
    case.rows[:, :512] /= torch.from_numpy(size).bfloat16()   # rows of one size, as a norm leaves them
    case.keys = row_values(case.shape, case.rows) if fp8 else case.rows.double().numpy()
    want = case.oracle()[0]
    for lse in (True, False):
        o, _ = case.layer().latent_attn(want_lse=lse, **case.device_inputs())
        size, along = off_by(o, want)
        assert size <= 3e-3 and along <= 3e-4, (size, along)


def test_a_prefix_at_more_heads_than_the_head_major_list_holds():
    # 256 blocks of 128 query rows of one token: one more than fit beside the sequence's own entry
    heads, prefix, own = 128 * 255 + 64, 70, 3
    shape = dataclasses.replace(wl.V2LITE, hidden=64, n_heads=heads, qk_nope=8, v_dim=32, block_size=64)
    weights = {k: torch.zeros(v, dtype=torch.bfloat16, device="cuda") for k, v in wl.weight_shapes(shape).items()}
    weights["kv_norm_w"] = torch.ones(512, device="cuda")
    from head_latent_attention_decode_b200.layer import MlaLayer
    layer = MlaLayer(shape, weights, cache_dtype="fp8")
    del weights
    cache = layer.new_cache(3)
    slots = torch.arange(192, dtype=torch.int32, device="cuda")
    layer.cache_write(torch.randn(192, 576, device="cuda").bfloat16(), cache, slots)
    q = torch.randn(1, heads, 576, device="cuda").bfloat16()
    args = (cache, torch.tensor([[2]], dtype=torch.int32, device="cuda"), torch.tensor([own], dtype=torch.int32, device="cuda"), own)
    o, lse = layer.latent_attn(q[..., :512].contiguous(), q[..., 512:].contiguous(), *args, want_lse=True,
                               prefix_table=torch.tensor([0, 1], dtype=torch.int32, device="cuda"), prefix_len=prefix)
    keys = layer.cache_read(cache, slots).double()[torch.cat([torch.arange(prefix), torch.arange(128, 128 + own)]).cuda()]
    s = q[0].double() @ keys.T / np.sqrt(72.0)
    want = torch.softmax(s, 1) @ keys[:, :512]
    assert float((o[0].double() - want).norm() / want.norm()) <= 2.0 ** -7
    assert float((lse[0].double() - torch.logsumexp(s, 1)).abs().max()) <= 1e-4
    assert mla.mla_read_device_flag(layer.ws) == 0
