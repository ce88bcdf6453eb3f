"""The 8-bit experts, the quantiser, the balance loss and the gradients at the
ends of their ranges on the GPU: offsets past 32 bits, the largest expert and
slot counts, M-tile borders, many tokens per wave, calls on two streams at
once, weights of zero and of negative scale.

Where a problem is too large for the float64 oracle its last part is compared,
bit for bit, with the same values as a small problem of their own.
"""
import numpy as np
import pytest
import torch

import oracle
import routed_expert_ffn_03_amd as moe
from tests import test_gpu_fp8 as F8
from tests import test_gpu_router_grad as RG
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
FP8 = moe.MOE_WFMT_FP8_B128


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_quantize_past_2_31_values():
    _cuda()
    rows = (1 << 24) + 3
    src = torch.randn(1 << 16, 128, device="cuda").to(torch.bfloat16).repeat(257, 1)[:rows].contiguous()
    codes = torch.full((rows, 128), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 1), -1.0, device="cuda")
    moe.moe_quantize_fp8(src, codes, scales)
    c, s = torch.empty((1 << 16, 128), dtype=torch.uint8, device="cuda"), torch.empty((1 << 16, 1), device="cuda")
    moe.moe_quantize_fp8(src[:1 << 16], c, s)
    torch.cuda.synchronize()
    for lo in range(0, rows, 1 << 16):
        n = min(1 << 16, rows - lo)
        assert torch.equal(codes[lo:lo + n], c[:n]) and torch.equal(scales[lo:lo + n], s[:n]), lo


@pytest.mark.parametrize("T,k", [(4, 2), (90, 2)])
def test_experts_past_2_32_bytes_of_weights(T, k):
    """The last of 700 experts (5.9 GB a matrix) against the same experts as a layer of four."""
    _cuda()
    E, H, I, last = 700, 4096, 2048, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    def codes(*s):
        return torch.empty(s, dtype=torch.uint8, device="cuda").random_(0, 0x60, generator=g)
    big = {"gate": codes(E, I, H), "up": codes(E, I, H), "down": codes(E, H, I)}
    for n, (r, c) in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
        big[n + "_scale"] = (torch.rand(E, r // 128, c // 128, device="cuda", generator=g) - 0.5) * 2.0 ** -9
    small = {n: t[E - last:].clone() for n, t in big.items()}
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    lg = torch.randn(T, last, device="cuda", generator=g)
    b, s = moe.MoELayerBuffers(T, E, k, H, I, FP8), moe.MoELayerBuffers(T, last, k, H, I, FP8)
    want = s.forward(lg, x, small)
    got = b.forward(torch.cat([torch.full((T, E - last), -50.0, device="cuda"), lg], 1), x, big)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and want.abs().max() > 0
    assert torch.equal(b.y_sorted, s.y_sorted) and torch.equal(got, want)


@pytest.mark.parametrize("thr", [1, 1000])
def test_ffn_1024_experts_32_slots(thr):
    _cuda()
    T, E, k, H, I = 20, 1024, 32, 256, 128
    logits, x, W = F8.make_case(T, E, k, H, I, 17)
    ref = F8.reference(logits, x, W, k)
    F8.check(F8.run_ffn(logits, x, W, k, thr)[0], ref, f"thr {thr}", thr)


@pytest.mark.parametrize("T", [223, 224, 225, 449])
def test_ffn_m_tile_borders(T):
    """One live expert: its list fills, or spills over, M-tiles of 224 rows."""
    _cuda()
    E, k, H, I = 3, 1, 256, 128
    logits, x, W = F8.make_case(T, E, k, H, I, T, 1)
    F8.check(F8.run_ffn(logits, x, W, k, 32)[0], F8.reference(logits, x, W, k), f"{T} rows", 32)


def test_zero_rows_and_signed_scales():
    _cuda()
    T, E, k, H, I = 70, 4, 2, 256, 256
    logits, x, W = F8.make_case(T, E, k, H, I, 4)
    x[::3] = 0
    for n in ("gate_scale", "up_scale", "down_scale"):
        W[n][:, 0] *= -1
        W[n][1] = 0
    ref = F8.reference(logits, x, W, k)
    for thr in (1, 1000):
        b, _ = F8.run_ffn(logits, x, W, k, thr)
        F8.check(b, ref, f"thr {thr}", thr)
        y, sp = b.y_sorted.cpu(), b.sorted_pair.cpu().numpy()
        assert (y[torch.from_numpy((sp // k) % 3 == 0)] == 0).all()


def test_two_streams_at_once():
    _cuda()
    T, E, k, H, I = 120, 8, 2, 512, 256
    logits, x, W = F8.make_case(T, E, k, H, I, 31)
    dw = F8.dev_weights(W)
    lg = [torch.from_numpy(np.roll(logits, i, 1).copy()).cuda() for i in range(2)]
    xs = [x.cuda(), x.flip(0).contiguous().cuda()]
    seq = [moe.MoELayerBuffers(T, E, k, H, I, FP8) for _ in range(2)]
    grads = [moe.RouterGradBuffers(b, groups=2) for b in seq]
    d_out = torch.randn(T, H, device="cuda")
    one = torch.ones(1, device="cuda")
    def step(i, stream=None):
        seq[i].forward(lg[i], xs[i], dw, stream=stream)
        grads[i].balance_loss(lg[i], 0.1, stream=stream)
        grads[i].backward(lg[i], d_out, one, stream=stream)
    want = []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (seq[i].out, grads[i].loss, grads[i].d_logits)])
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for b, g in zip(seq, grads):
            b.out.fill_(5.0)
            g.d_logits.fill_(5.0)
        torch.cuda.synchronize()
        for i in range(2):
            step(i, st[i])
        torch.cuda.synchronize()
        for i in range(2):
            for a, c in zip((seq[i].out, grads[i].loss, grads[i].d_logits), want[i]):
                assert torch.equal(a, c), i


@pytest.mark.parametrize("T,E,k", [(1, 6, 2), (37, 6, 2), (300, 5, 3)])
def test_captured_whole_call_replays(T, E, k):
    """moe_grouped_ffn in a graph, on other inputs at each replay, against its phases one by one."""
    _cuda()
    H, I = 256, 384
    dw = F8.dev_weights(F8.make_case(T, E, k, H, I, 77)[2])
    w = (dw["gate"], dw["up"], dw["down"])
    kw = dict(s_gate=dw["gate_scale"], s_up=dw["up_scale"], s_down=dw["down_scale"], wfmt=FP8)
    b = moe.MoELayerBuffers(T, E, k, H, I, FP8)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    off, sp = torch.zeros_like(b.expert_offsets), torch.zeros_like(b.sorted_pair)
    y, ws = torch.empty_like(b.y_sorted), torch.full_like(b.workspace, 0xFF)
    graph = None
    for seed in range(4):
        logits, xs, _ = F8.make_case(T, E, k, H, I, 200 + seed, 1 + seed if seed + 1 >= k else None)
        x.copy_(xs)
        b.workspace.fill_(0xFF)
        b.forward(torch.from_numpy(logits).cuda(), x, dw)
        off.copy_(b.expert_offsets)
        sp.copy_(b.sorted_pair)
        torch.cuda.synchronize()
        if graph is None:
            moe.moe_grouped_ffn(x, *w, off, sp, k, y, ws, **kw)
            torch.cuda.synchronize()
            assert torch.equal(y, b.y_sorted)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                moe.moe_grouped_ffn(x, *w, off, sp, k, y, ws, **kw)
        for _ in range(2):
            y.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, b.y_sorted), seed


@pytest.mark.parametrize("T,E,k,G,mask_kind", [(40002, 20, 2, 6, "some"), (30000, 70, 4, 7500, None),
                                               (5000, 8, 2, 5000, "some")])
def test_many_tokens_and_many_groups(T, E, k, G, mask_kind):
    """Waves with many tokens, groups that begin inside a wave's run, a group for each token."""
    _cuda()
    say(f"[balance] T={T} E={E} k={k} G={G} mask={mask_kind}")
    a = RG.make(T, E, k, T + E, mask_kind)
    RG.check(RG.run(*a, G, 0.3, 1.7), *a, G, 0.3, 1.7)


def test_balance_past_2_31_logits():
    """The last group of 2.2 million tokens against the same tokens alone (other sums, so by their rounding)."""
    _cuda()
    E, k, L, G = 1024, 2, 1000, 2200
    T = L * G
    g = torch.Generator(device="cuda").manual_seed(2)
    lg = torch.zeros(T, E, device="cuda")
    tail = torch.randn(L, E, device="cuda", generator=g)
    lg[-L:] = tail
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    ids[:, 1] = E - 1
    ids[-L:] = tail.topk(k, 1).indices.to(torch.int32)
    def run(lg, ids, G):
        T = lg.shape[0]
        o = [torch.full((G, E), -1, dtype=torch.int32, device="cuda"), torch.full((G, E), -1.0, device="cuda"),
             torch.full((G,), -1.0, device="cuda"), torch.full((1,), -1.0, device="cuda")]
        ws = torch.empty(moe.moe_balance_workspace_size(T, E, G), dtype=torch.uint8, device="cuda")
        moe.moe_balance_loss(lg, ids, *o, ws, coef=1.0)
        d = torch.full((T, E), 9.0, device="cuda")
        moe.moe_route_backward(lg, ids, torch.empty(T, k, device="cuda"), d, expert_counts=o[0], group_scale=o[2],
                               d_loss=torch.full((1,), float(G), device="cuda"))
        torch.cuda.synchronize()
        return *o, d
    counts, prob, scale, loss, d = run(lg, ids, G)
    c1, p1, s1, l1, d1 = run(tail, ids[-L:].contiguous(), 1)
    assert torch.equal(counts[-1:], c1) and (counts[:-1, 0] == L).all() and (counts[:-1, E - 1] == L).all()
    assert (counts[:-1, 1:E - 1] == 0).all()
    # sums of at most 1,000 terms each to within 1,000 half units, twice
    assert torch.allclose(prob[-1:], p1, rtol=1000 * 2.0 ** -23, atol=0)
    assert torch.allclose(prob[:-1], torch.full_like(prob[:-1], 1 / E), rtol=1000 * 2.0 ** -23, atol=0)
    # d_loss = G undoes the mean over groups: the gradient's factors differ by 4 roundings, its difference of
    # like terms by those of either term, below max(p) of a token times the largest b
    lim = 64 * 2.0 ** -24 * float(torch.softmax(tail, 1).max()) * float(c1.max() * s1)
    assert float((d[-L:] - d1).abs().max()) <= lim
    # uniform logits: d = (b_e - mean b) / E
    b = float(scale[0]) * G * L
    want = torch.full((E,), -2 * b / E / E, device="cuda")
    want[0] += b / E
    want[E - 1] += b / E
    for lo in range(0, T - L, 500 * L):
        n = min(500 * L, T - L - lo)
        assert float((d[lo:lo + n] - want).abs().max()) <= 64 * 2.0 ** -24 * b / E, lo


def test_combine_backward_past_2_31_values():
    _cuda()
    T, k, H, n = 70000, 8, 4096, 100
    g = torch.Generator(device="cuda").manual_seed(3)
    y = torch.empty(T * k, H, dtype=torch.float16, device="cuda").normal_(generator=g)
    w = torch.rand(T, k, device="cuda", generator=g)
    go = torch.empty(T, H, device="cuda").normal_(generator=g)
    p2s = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).contiguous()
    dy, dw = torch.full_like(y, 9.0), torch.full((T, k), 9.0, device="cuda")
    moe.moe_combine_backward(go, y, w, p2s, dy, dw)
    for t0 in (0, T - n):                                   # rows at the end and at the start of y
        idx = p2s[t0 * k:(t0 + n) * k].long()
        sy, sdy, sdw = y[idx].contiguous(), torch.empty(n * k, H, dtype=torch.float16, device="cuda"), torch.empty(
            n, k, device="cuda")
        moe.moe_combine_backward(go[t0:t0 + n], sy, w[t0:t0 + n], torch.arange(n * k, dtype=torch.int32, device="cuda"),
                                 sdy, sdw)
        torch.cuda.synchronize()
        assert torch.equal(dy[idx], sdy) and torch.equal(dw[t0:t0 + n], sdw)


def test_combine_backward_more_tokens_than_blocks():
    _cuda()
    T, H = (1 << 20) + 77, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    y = torch.randn(T, H, device="cuda", generator=g).half()
    w, go = torch.rand(T, 1, device="cuda", generator=g), torch.randn(T, H, device="cuda", generator=g)
    p2s = torch.randperm(T, device="cuda", generator=g).to(torch.int32)
    dy, dw = torch.full_like(y, 9.0), torch.full((T, 1), 9.0, device="cuda")
    moe.moe_combine_backward(go, y, w, p2s, dy, dw)
    torch.cuda.synchronize()
    i = p2s.long()
    ref = w.double() * go.double()
    # fp16 rounding 2^-11 (2^-25 below the normal range), perhaps of a product rounded to fp32
    assert ((dy[i].double() - ref).abs() <= 2.0 ** -11 * 1.001 * ref.abs() + 2.0 ** -25).all()
    terms = go.double() * y[i].double()
    assert ((dw[:, 0].double() - terms.sum(1)).abs() <= 18 * 2.0 ** -24 * terms.abs().sum(1)).all()
