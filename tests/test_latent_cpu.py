"""Host-side tests of the 8-bit cache and shared-prefix attention: the fp64
definitions against torch and literal loops, and the refusals that need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import head_latent_attention_decode_b200 as mla
from head_latent_attention_decode_b200 import build as mla_build
from oracle import latent_ref as lr

P = 4096


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.lib()


def test_codes_match_torch_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(want), np.isnan(lr.E4M3)) and np.isnan(lr.E4M3).sum() == 2
    ok = ~np.isnan(want)
    assert np.array_equal(want[ok], lr.E4M3[ok])


def test_rounding_matches_torch_on_every_bf16():
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x)].clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = lr.e4m3_round(x.double().numpy())
    assert np.array_equal(lr.E4M3[want], lr.E4M3[got])


def test_rounding_of_what_is_not_finite_or_too_large():
    got = lr.e4m3_round(np.array([np.inf, -np.inf, np.nan, 449.0, -1e30]))
    assert list(got) == [0x7F, 0x7F, 0x7F, 126, 254]


@pytest.mark.parametrize("amax,k", [(448.0, 0), (448.5, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.7501, -7),
                                    (448.0 * 128, 7), (1e30, 7), (1e-30, -64), (0.0, 0)])
def test_scale_exponent(amax, k):
    row = np.array([amax / 3, -amax, math.inf, math.nan])
    assert lr.scale_exponent(row) == k


def test_quantisation_error_is_within_half_a_step():
    rng = np.random.default_rng(0)
    for size in (1e-12, 1.0, 3e4):
        x = rng.standard_normal(512) * size
        codes, k = lr.quantise_row(x)
        v = lr.E4M3[codes] * 2.0 ** k
        assert (np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (k - 10))).all() or k == lr.K_MAX


def test_attention_against_literal_loops():
    rng = np.random.default_rng(1)
    q, qp, c, pe = (rng.standard_normal(s) for s in ((2, 8), (2, 4), (5, 8), (5, 4)))
    o, lse, p = lr.latent_attention(q, qp, c, pe, 0.3)
    for h in range(2):
        s = [0.3 * (sum(q[h, i] * c[j, i] for i in range(8)) + sum(qp[h, i] * pe[j, i] for i in range(4))) for j in range(5)]
        den = sum(math.exp(v) for v in s)
        assert abs(lse[h] - math.log(den)) < 1e-12
        for i in range(8):
            assert abs(o[h, i] - sum(math.exp(s[j]) / den * c[j, i] for j in range(5))) < 1e-12
    # a set of keys is the lse-weighted mean of its parts
    a, la, _ = lr.latent_attention(q, qp, c[:2], pe[:2], 0.3)
    b, lb, _ = lr.latent_attention(q, qp, c[2:], pe[2:], 0.3)
    w = np.exp(la - np.logaddexp(la, lb))[:, None]
    assert np.allclose(w * a + (1 - w) * b, o, atol=1e-12) and np.allclose(np.logaddexp(la, lb), lse)


def test_attention_without_keys():
    o, lse, _ = lr.latent_attention(np.ones((3, 4)), np.ones((3, 2)), np.zeros((0, 4)), np.zeros((0, 2)), 1.0)
    assert (o == 0).all() and (lse == -np.inf).all()
    o, lse, _ = lr.latent_attention(np.ones((1, 4)), np.ones((1, 2)), np.zeros((0, 4)), np.zeros((0, 2)), 1.0, sink=[0.7])
    assert (o == 0).all() and lse[0] == np.float64(0.7)


def test_calls_reject_a_null_handle(lib):
    bad = mla.MLA_ERR_INVALID_ARG
    assert lib.mla_set_cache_dtype(None, mla.MLA_FP8_E4M3_ROW) == bad
    assert lib.mla_cache_block_bytes(None) == 0
    assert lib.mla_cache_write(None, P, 1, P, 1, P, P, 256, None) == bad
    assert lib.mla_cache_read(None, P, 1, P, 1, P, P, 256, None) == bad
    assert lib.mla_prefix_workspace_bytes(None, 1, 1, 1) == 0
    assert lib.mla_latent_attn(None, P, P, P, 1, None, 0, P, 1, P, 1, 1, P, None, P, 1 << 20, None) == bad
    assert lib.mla_decode_attn_prefix(None, P, P, P, 1, None, 0, P, 1, P, 1, 1, P, None, P, 1 << 20, None) == bad


def test_binding_refuses_host_and_mismatched_tensors(lib):
    x = torch.zeros((2, 576), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.mla_cache_write(0, x, x, i, x)
    with pytest.raises(ValueError):
        mla.mla_cache_read(0, x, i, x, x)
    q = torch.zeros((2, 4, 512), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.mla_latent_attn(0, q, q, x, i.view(2, 1), i, 1, q, x)
    with pytest.raises(ValueError):
        mla.mla_decode_attn_prefix(0, q, q, x, i, 2, i.view(2, 1), i, 1, x, x)


def test_new_dtype_is_no_weight_or_activation_type(lib):
    from head_latent_attention_decode_b200 import workloads as wl
    c = mla.make_config(wl.TINY)
    c.weight_dtype = mla.MLA_FP8_E4M3_ROW
    assert mla.mla_weights_bytes(c) == 0
    c = mla.make_config(wl.TINY)
    c.act_dtype = mla.MLA_FP8_E4M3_ROW
    assert mla.mla_weights_bytes(c) == 0
    assert ctypes.sizeof(mla.mla_config) == 15 * 4


def test_the_layer_refuses_queries_and_outputs_of_another_shape_or_type():
    from types import SimpleNamespace
    from head_latent_attention_decode_b200.layer import MlaLayer
    layer = MlaLayer.__new__(MlaLayer)   # the checks read the shape and the type alone
    layer.shape, layer.act = SimpleNamespace(n_heads=4, kv_lora_rank=64, qk_rope=16, hidden=32, v_dim=8), torch.bfloat16
    q, p = torch.zeros(2, 4, 64).bfloat16(), torch.zeros(2, 4, 16).bfloat16()
    layer._check_query(q, p)
    for a, b in ((q[:, :2], p[:, :2]), (q[..., :32], p), (q, p[..., :8]), (q, p[:1]), (q.float(), p.float()), (q.flatten(1), p)):
        with pytest.raises(ValueError):
            layer._check_query(a, b)
    out, head = torch.zeros(2, 32).bfloat16(), torch.zeros(2, 4, 8).bfloat16()
    layer._check_out(2, out, None)
    layer._check_out(2, out, head)
    for a, b in ((out[:1], None), (out[:, :16], None), (out.float(), None), (out, head[:1]), (out, head[..., :4]), (out, head.float())):
        with pytest.raises(ValueError):
            layer._check_out(2, a, b)
