"""Host side of the norm-and-rotation calls: argument checks of the C ABI and
the Python helpers, and the rotary frequencies (no GPU needed)."""
import math

import pytest
import torch

import exact_attention_11_gb300 as fa
from exact_attention_11_gb300 import _build

NULL, P = None, 4096   # a 16-byte-aligned fake address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


FWD = dict(q=P, k=P, q_weight=P, k_weight=P, positions=P, inv_freq=P, q_out=P, k_out=P,
           num_tokens=0, num_heads=4, num_kv_heads=2, d=128, rot_dim=64, interleaved=0,
           q_stride=512, k_stride=256, eps=1e-6, mscale=1.0)
BAD = [
    (dict(), 0),                                  # no tokens: nothing to do
    (dict(q_weight=NULL, k_weight=NULL), 0),
    (dict(rot_dim=0, inv_freq=NULL), 0),
    (dict(rot_dim=128, interleaved=1), 0),
    (dict(q=NULL), -1),
    (dict(k=NULL), -1),
    (dict(positions=NULL), -1),
    (dict(inv_freq=NULL), -1),
    (dict(num_tokens=-1), -1),
    (dict(num_heads=0), -1),
    (dict(num_kv_heads=0), -1),
    (dict(eps=-1.0), -1),
    (dict(eps=math.nan), -1),
    (dict(mscale=math.inf), -1),
    (dict(rot_dim=-16), -1),
    (dict(rot_dim=144), -1),                      # more than the head
    (dict(rot_dim=40), -2),                       # not a multiple of 16
    (dict(d=96, rot_dim=32), -2),
    (dict(num_heads=70000, q_stride=70000 * 128), -2),
    (dict(q=P + 8), -3),
    (dict(k_weight=P + 2), -3),
    (dict(positions=P + 2), -3),
    (dict(inv_freq=P + 4), -3),
    (dict(q_stride=511), -1),                     # does not cover the heads
    (dict(k_stride=260), -3),                     # rows not 16-byte aligned
]


@pytest.mark.parametrize("change,expect", BAD)
def test_forward_checks(lib, change, expect):
    a = {**FWD, **change}
    for name in ("fa_qk_norm_rope", "fa_qk_norm_rope_f16"):
        assert getattr(lib, name)(*a.values(), None) == expect
    if change != dict(k_stride=260):              # 260 fp32 values are 65 * 16 bytes
        assert lib.fa_qk_norm_rope_fp32(*a.values(), None) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(q_out=NULL), -1), (dict(k_out=NULL), -1), (dict(q_out=P + 4), -3)])
def test_forward_output_checks(lib, change, expect):
    assert lib.fa_qk_norm_rope(*{**FWD, **change}.values(), None) == expect


CACHE = dict(q=P, k=P, v=P, q_weight=P, k_weight=P, positions=P, inv_freq=P, slots=P, q_out=P,
             k_cache=P, v_cache=P, num_tokens=0, num_heads=4, num_kv_heads=2, head_size=128,
             block_size=16, num_blocks=8, rot_dim=64, interleaved=0, q_stride=512, k_stride=256,
             v_stride=256, eps=1e-6, mscale=1.0)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0), (dict(v=NULL), -1), (dict(slots=NULL), -1), (dict(k_cache=NULL), -1),
    (dict(v_cache=NULL), -1), (dict(num_blocks=-1), -1), (dict(head_size=64), -2),
    (dict(block_size=32), -2), (dict(v_cache=P + 2), -3), (dict(slots=P + 4), -3),
    (dict(v_stride=255), -1), (dict(v_stride=257), -3)])
def test_cache_checks(lib, change, expect):
    assert lib.fa_qk_norm_rope_cache(*{**CACHE, **change}.values(), None) == expect


BWD = dict(dq_out=P, dk_out=P, q=P, k=P, q_weight=NULL, k_weight=NULL, positions=P, inv_freq=P,
           dq=P, dk=P, dq_weight=NULL, dk_weight=NULL, num_tokens=0, num_heads=4, num_kv_heads=2,
           d=128, rot_dim=64, interleaved=0, q_stride=512, k_stride=256, eps=1e-6, mscale=1.0,
           workspace=NULL, workspace_bytes=0)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0), (dict(dq_out=NULL), -1), (dict(dk=NULL), -1),
    (dict(q_weight=P), -1),                        # a weight without its gradient
    (dict(dk_weight=P), -1),                       # a gradient without its weight
    (dict(q_weight=P, dq_weight=P, num_tokens=5), -1),                       # no workspace
    (dict(q_weight=P, dq_weight=P, num_tokens=5, workspace=P, workspace_bytes=64), -1),
    (dict(q_weight=P, dq_weight=P, num_tokens=5, workspace=P + 4, workspace_bytes=1 << 30), -3),
    (dict(dk=P + 4), -3), (dict(dq_weight=P + 2, q_weight=P), -3)])
def test_backward_checks(lib, change, expect):
    for name in ("fa_qk_norm_rope_backward", "fa_qk_norm_rope_backward_f16",
                 "fa_qk_norm_rope_backward_fp32"):
        assert getattr(lib, name)(*{**BWD, **change}.values(), None) == expect


def test_workspace_sizes(lib):
    size = fa.fa_qk_norm_rope_backward_workspace_bytes
    assert size(-1, 128) == 0
    assert size(1, 128) == 2 * 128 * 4
    assert size(1 << 20, 64) == size(1 << 30, 64)      # bounded by the grid


def test_helpers_refuse_inconsistent_tensors(lib):
    q, k = torch.zeros(3, 4, 128), torch.zeros(3, 2, 128)
    pos, freq = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):      # not on a GPU
        fa.qk_norm_rope(q, k, pos, freq)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q.int(), k.int(), pos, freq)


def test_frequencies():
    plain, m = fa.rope_frequencies(64, 10000.0)
    assert m == 1.0 and plain.dtype == torch.float64 and plain.shape == (32,)
    assert plain[0] == 1.0 and math.isclose(plain[1].item(), 10000.0 ** (-1 / 32))
    linear, m = fa.rope_frequencies(64, scaling="linear", factor=4.0)
    assert m == 1.0 and torch.equal(linear, plain / 4.0)
    ntk, _ = fa.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[-1].item(), plain[-1].item() / 4.0, rel_tol=1e-12)
    yarn, m = fa.rope_frequencies(64, scaling="yarn", factor=4.0, original_context=4096)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1.0)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(yarn[turns >= 32], plain[turns >= 32])
    assert torch.allclose(yarn[turns <= 1], plain[turns <= 1] / 4.0, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (yarn[between] < plain[between]).all()
    assert (yarn[between] > plain[between] / 4.0).all()
    assert fa.rope_frequencies(0)[0].numel() == 0
    for bad in (dict(rot_dim=3), dict(rot_dim=64, scaling="other"), dict(rot_dim=64, factor=0.5)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**bad)


def test_frequencies_refuse_an_empty_ramp():
    for bad in (dict(beta_slow=32.0), dict(original_context=0)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(64, scaling="yarn", factor=4.0, **bad)


@pytest.mark.parametrize("rot,base,context,factor,beta_slow,beta_fast,first,last", [
    (128, 10000.0, 4096, 4.0, 1.0, 32.0, 20, 46),      # 20.9 and 45.03 before rounding
    (64, 10000.0, 4096, 16.0, 1.0, 32.0, 10, 23),      # 10.5, 22.5
    (128, 1e6, 32768, 4.0, 1.0, 32.0, 23, 40),         # 23.6, 39.6
    (64, 10000.0, 100, 2.0, 1.0, 32.0, 0, 10),         # clamped: no frequency turns 32 times
    (64, 10000.0, 1 << 30, 2.0, 1.0, 32.0, 53, 63),    # 53.8, 65.9 (clamped at rot_dim - 1)
])
def test_yarn_ramps_over_the_index(rot, base, context, factor, beta_slow, beta_fast, first, last):
    """Frequency i keeps its value up to `first`, is divided from `last` on and goes from
    one to the other linearly in i between them, as models trained with YaRN have it.
    (The bounds' comments give rot_dim ln(context / 2 pi beta) / 2 ln base.)"""
    got, m = fa.rope_frequencies(rot, base, scaling="yarn", factor=factor,
                                 original_context=context, beta_slow=beta_slow,
                                 beta_fast=beta_fast)
    for i, f in enumerate(got.tolist()):
        plain = base ** (-2.0 * i / rot)
        divided = min(max((i - first) / (last - first), 0.0), 1.0)
        assert math.isclose(f, plain * (1.0 - divided + divided / factor), rel_tol=1e-14)
    assert math.isclose(m, 0.1 * math.log(factor) + 1.0)


def test_yarn_by_turns():
    """The ramp that is linear in a frequency's turns over the original context."""
    got, _ = fa.rope_frequencies(64, scaling="yarn", factor=4.0, ramp="turns")
    for i, f in enumerate(got.tolist()):
        plain = 10000.0 ** (-2.0 * i / 64)
        keep = min(max((4096 * plain / (2 * math.pi) - 1.0) / 31.0, 0.0), 1.0)
        assert math.isclose(f, plain * (keep + (1.0 - keep) / 4.0), rel_tol=1e-14)
    for bad in (dict(ramp="other"), dict(beta_slow=0.0)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(64, scaling="yarn", factor=4.0, **bad)
