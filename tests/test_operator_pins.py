"""The oracle's 8-bit blocks, balance loss and router gradients against closed
forms, torch's own e4m3 type and differences; and every refusal of their
entry points that the host can check (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import routed_expert_ffn_03_amd as moe
from routed_expert_ffn_03_amd.build import LIB

FAKE = 0x100000        # 16- and 256-byte aligned, never dereferenced


# ------------------------------------------------------------ oracle

def test_e4m3_table_is_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oracle.e4m3_to_f64(codes), want)


def test_e4m3_rounding_is_nearest_even():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 2.0 ** -6, [0.0, -0.0, 448.0, -448.0]])
    table = oracle.e4m3_to_f64(np.arange(0x7F))
    v = np.concatenate([v, (table[1:] + table[:-1]) / 2, -(table[1:] + table[:-1]) / 2])       # every tie
    v = v.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(oracle.f64_to_e4m3(v), want)
    assert oracle.f64_to_e4m3(np.array([np.nan, np.inf, -np.inf])).tolist() == [0x7F] * 3


def test_block_scale_is_the_least_power_of_two():
    assert oracle.fp8_block_scale(0.0) == 1.0
    assert oracle.fp8_block_scale(448.0) == 1.0
    assert oracle.fp8_block_scale(449.0) == 2.0
    assert oracle.fp8_block_scale(224.0) == 0.5
    assert oracle.fp8_block_scale(1e-40) == 2.0 ** -126
    for top in np.random.default_rng(1).lognormal(0, 20, 200):
        s = oracle.fp8_block_scale(top)
        assert np.log2(s) == round(np.log2(s)) and top <= 448 * s and (top > 448 * s / 2 or s == 2.0 ** -126)


def test_quantised_values_are_within_half_a_step():
    # half an e4m3 step: 2^-4 of the value, 2^-10 of the scale below the normal range
    v = np.random.default_rng(2).standard_normal((256, 256)) * np.exp(np.random.default_rng(3).standard_normal((256, 1)))
    for br in (1, 128):
        q, s = oracle.quantize_fp8(v, br)
        s_full = np.repeat(np.repeat(s, br, 0), 128, 1)
        assert np.all(np.abs(oracle.fp8_values(q, s) - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s_full))


def test_uniform_router_loss_is_coef():
    T, E, k = 12, 6, 2
    ids = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    for groups in (1, 2, 4):
        b = oracle.balance_loss(np.zeros((T, E)), ids, groups, 0.25)
        assert abs(b["loss"] - 0.25) < 1e-15
        assert b["counts"].sum() == T * k
    # everything on one expert: p = 1 there, so the loss is coef * E / k * 1 (k = 1)
    l = np.zeros((T, E)); l[:, 3] = 200.0
    assert abs(oracle.balance_loss(l, np.full((T, 1), 3), 1, 0.5)["loss"] - 0.5 * E) < 1e-12


def test_router_gradient_matches_differences():
    rng = np.random.default_rng(4)
    T, E, k, G = 12, 7, 3, 3
    l = rng.standard_normal((T, E))
    mask = rng.random(T) > 0.3
    mask[4:8] = False                                         # an empty group
    ids, w = oracle.route_topk(l.astype(np.float32), k)
    l = l.astype(np.float32).astype(np.float64)
    target = rng.standard_normal((T, k))
    fixed = oracle.balance_loss(l, ids, G, 0.7, mask)

    def total(x):
        b = oracle.balance_loss(x, ids, G, 0.7, mask)
        s = np.take_along_axis(x, ids.astype(np.int64), 1)
        gate = np.exp(s - s.max(1, keepdims=True))
        gate /= gate.sum(1, keepdims=True)
        return 1.3 * b["loss"] + float((gate * target).sum())

    got = oracle.route_backward(l, ids, w, target, fixed, 1.3, mask)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(l); d[t, e] = h
            num = (total(l + d) - total(l - d)) / (2 * h)
            assert abs(num - got[t, e]) < 1e-8, (t, e)       # O(h^2) + rounding 1e-16 / h


def test_combine_gradient_matches_differences():
    rng = np.random.default_rng(5)
    T, k, H = 4, 2, 8
    Y, w = rng.standard_normal((T * k, H)), rng.random((T, k))
    p2s = rng.permutation(T * k)
    d_out = rng.standard_normal((T, H))
    dY, dw = oracle.combine_backward(d_out, Y, w, p2s, k)
    f = lambda Y, w: float((oracle.combine(Y, w, p2s, k) * d_out).sum())
    h = 1e-4                                                  # f is linear in each: differences are exact up to rounding
    for i in range(T * k):
        for c in range(H):
            d = np.zeros_like(Y); d[i, c] = h
            assert abs((f(Y + d, w) - f(Y - d, w)) / (2 * h) - dY[i, c]) < 1e-10
    for t in range(T):
        for j in range(k):
            d = np.zeros_like(w); d[t, j] = h
            assert abs((f(Y, w + d) - f(Y, w - d)) / (2 * h) - dw[t, j]) < 1e-10


# ------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(LIB):
        pytest.skip("library not built")
    return moe.lib()


def test_fp8_workspace_size(L):
    r = lambda v: (v + 255) // 256 * 256
    T, E, k, H, I = 100, 16, 2, 512, 384
    lists = L.moe_workspace_size(T, E, k, H, I, 0) - r(T * k * I * 2)       # (T k < 224: the same lists)
    want = lists + r(T * k * I) + r(T * k * (I // 128) * 4) + r(T * H) + r(T * (H // 128) * 4) + r(T * k * (H // 128) * 4)
    assert L.moe_workspace_size(T, E, k, H, I, 4) == want
    assert L.moe_workspace_size(T, E, k, H, I + 64, 4) == 0
    assert L.moe_workspace_size(T, E, k, H, I, 3) == 0


def test_fp8_ffn_rejects(L):
    def call(**kw):
        a = dict(x=FAKE, wfmt=4, wg=FAKE, wu=FAKE, wd=FAKE, sg=FAKE, su=FAKE, sd=FAKE, off=FAKE, sp=FAKE, T=64, E=16,
                 k=2, H=256, I=128, thr=32, y=FAKE, ws=FAKE, wsb=1 << 40, s=None)
        a.update(kw)
        return L.moe_grouped_ffn(*a.values())
    for key in ("x", "wg", "wu", "wd", "sg", "su", "sd", "off", "sp", "y"):
        assert call(**{key: None}) == moe.MOE_ERR_INVALID_ARG, key
    for key in ("x", "wg", "wu", "wd", "y"):
        assert call(**{key: FAKE + 8}) == moe.MOE_ERR_INVALID_ARG, key
    for key in ("sg", "su", "sd"):
        assert call(**{key: FAKE + 2}) == moe.MOE_ERR_INVALID_ARG, key
    assert call(H=128) == moe.MOE_ERR_UNSUPPORTED
    assert call(I=192) == moe.MOE_ERR_UNSUPPORTED
    assert call(ws=None) == moe.MOE_ERR_WORKSPACE
    assert call(wsb=1024) == moe.MOE_ERR_WORKSPACE
    F = FAKE
    gu = [F, 4, F, F, F, F, F, 64, 16, 2, 256, 128, 32, F, 1 << 40, None]
    for i in (4, 5):
        bad = list(gu); bad[i] = None
        assert L.moe_ffn_gate_up(*bad) == moe.MOE_ERR_INVALID_ARG
    dn = [4, F, F, 64, 16, 2, 256, 128, 32, F, F, 1 << 40, None]
    for i, v in ((2, None), (1, F + 4), (9, F + 4)):
        bad = list(dn); bad[i] = v
        assert L.moe_ffn_down(*bad) == moe.MOE_ERR_INVALID_ARG
    na = [F, 4, F, F, F, F, F, F, F, F, 64, 16, 2, 256, 128, 32, F, None]
    for i, v in ((5, None), (6, None), (7, None), (2, F + 1), (16, F + 8)):
        bad = list(na); bad[i] = v
        assert L.moe_grouped_ffn_noalloc(*bad) == moe.MOE_ERR_INVALID_ARG


def test_quantize_rejects(L):
    call = lambda src=FAKE, mats=1, rows=128, cols=128, br=1, codes=FAKE, scales=FAKE: L.moe_quantize_fp8(
        src, ctypes.c_int64(mats), rows, cols, br, codes, scales, None)
    for kw in (dict(src=None), dict(codes=None), dict(scales=None), dict(mats=0), dict(mats=-1), dict(rows=0),
               dict(cols=0), dict(src=FAKE + 8), dict(codes=FAKE + 4), dict(scales=FAKE + 2)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(br=64), dict(br=0), dict(cols=120), dict(rows=100, br=128), dict(mats=1 << 40),
               dict(mats=1 << 62), dict(rows=1 << 30, cols=1 << 30)):
        assert call(**kw) == moe.MOE_ERR_UNSUPPORTED, kw


def test_balance_rejects(L):
    names = ("l", "ids", "mask", "T", "E", "k", "G", "coef", "c", "p", "s", "loss", "ws", "wsb", "st")
    def call(**kw):
        a = dict(l=FAKE, ids=FAKE, mask=None, T=64, E=16, k=2, G=1, coef=ctypes.c_float(1.0), c=FAKE, p=FAKE, s=FAKE,
                 loss=FAKE, ws=FAKE, wsb=1 << 40, st=None)
        a.update(kw)
        return L.moe_balance_loss(*[a[n] for n in names])
    for key in ("l", "ids", "c", "p", "s", "loss"):
        assert call(**{key: None}) == moe.MOE_ERR_INVALID_ARG, key
    for kw in (dict(T=0), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(G=0), dict(G=3), dict(G=128),
               dict(G=-1), dict(ws=FAKE + 16), dict(T=1 << 30, k=2)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert call(ws=None) == moe.MOE_ERR_WORKSPACE
    assert call(wsb=moe.moe_balance_workspace_size(64, 16, 1) - 1) == moe.MOE_ERR_WORKSPACE
    assert call(T=1 << 25, G=1 << 25, k=1) == moe.MOE_ERR_UNSUPPORTED        # 2^25 blocks of tokens
    assert moe.moe_balance_workspace_size(64, 16, 3) == 0
    assert moe.moe_balance_workspace_size(64, 1025, 1) == 0


def test_route_backward_rejects(L):
    names = ("l", "ids", "w", "dw", "c", "s", "dl", "mask", "T", "E", "k", "G", "out", "st")
    def call(**kw):
        a = dict(l=FAKE, ids=FAKE, w=FAKE, dw=FAKE, c=FAKE, s=FAKE, dl=FAKE, mask=None, T=64, E=16, k=2, G=1,
                 out=FAKE, st=None)
        a.update(kw)
        return L.moe_route_backward(*[a[n] for n in names])
    for kw in (dict(out=None), dict(dw=None, c=None, s=None, dl=None), dict(c=None), dict(s=None), dict(dl=None),
               dict(l=None), dict(ids=None), dict(w=None), dict(T=0), dict(E=1025), dict(k=17), dict(G=5), dict(G=0)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw


def test_combine_backward_rejects(L):
    names = ("do", "y", "w", "p", "T", "k", "H", "dy", "dw", "st")
    def call(**kw):
        a = dict(do=FAKE, y=FAKE, w=FAKE, p=FAKE, T=4, k=2, H=64, dy=FAKE, dw=FAKE, st=None)
        a.update(kw)
        return L.moe_combine_backward(*[a[n] for n in names])
    for kw in (dict(do=None), dict(p=None), dict(dy=None, dw=None), dict(w=None), dict(y=None), dict(T=0), dict(k=0),
               dict(k=33), dict(H=0), dict(do=FAKE + 4), dict(y=FAKE + 8), dict(dy=FAKE + 8), dict(T=1 << 30)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert call(H=60) == moe.MOE_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_types():
    f = torch.zeros
    with pytest.raises(ValueError):
        moe.moe_quantize_fp8(f(2, 128, dtype=torch.bfloat16), f(2, 128, dtype=torch.uint8), f(2, 1))
    with pytest.raises(ValueError):
        moe.moe_balance_loss(f(4, 8), f(4, 2, dtype=torch.int32), f(1, 8, dtype=torch.int32), f(1, 8), f(1), f(1),
                             f(1024, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_route_backward(f(4, 8), f(4, 2, dtype=torch.int32), f(4, 2), f(4, 8), d_topk_w=f(4, 2))
    with pytest.raises(ValueError):
        moe.moe_combine_backward(f(4, 8), f(8, 8, dtype=torch.float16), f(4, 2), f(8, dtype=torch.int32),
                                 d_topk_w=f(4, 2))
