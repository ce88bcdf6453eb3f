"""The 8-bit experts on the GPU: codes and scales bit for bit, the grouped FFN
element by element against the float64 oracle, every kernel path (streaming
and MFMA tiles), the decode, captured and allocation-free forms.

Error bound of one element of y, from the arithmetic (u = 2^-24, fp32):
  * the e4m3 MFMA of the M-tiles adds the products of eight consecutive k with
    each term cut 13 bits below the largest product of the eight (measured: next
    to 2^16 a term of 2^3 is kept, 2^2 lost), and such octets in fp32: an octet
    is off by at most 8 2^-13 of its largest product.  (The streaming kernel
    multiplies the codes as fp16 and loses nothing there.)  The octets' sums (at
    most K / 8 additions) and the scaling (K / 128 fmas, two products) add 2 u
    each:
      |g - g*| <= sum_octets 2^-10 max|xq wg| + (K / 8 + K / 128 + 4) 2 u sum|xq||wg| =: dg
  * a = silu(g) u: |silu'| <= 1.1, and the fp32 silu and product are good to
    8 u of |a| (reciprocal and exponential of 1 ulp, three roundings; the
    exponential's argument error |g| u enters as |a| |g| u)
      da = 1.1 dg |u| + (|silu(g)| + 1.1 dg) du + (8 + 2 |g|) 2 u |a|
  * a's code is the oracle's unless a* is within da of a rounding border; then
    it may be the neighbour, a step of at most 2^-3 |a| or 2^-9 of the scale.
    (The scale itself is the same unless the block's maximum is within da of
    448 s: then a's code may be off by a step of the doubled scale.)
  * y: the ambiguous steps through |wd|, the same sum bound as above, and one
    rounding to fp16: 2^-11 |y| (2^-25 below the normal range).
That is a worst case.  All rows together are held to what the errors' spread
gives (norm_bound): an error of r rms relative to g puts 2 sqrt(2) r / 0.09 of
a's codes (steps of 2^-4 .. 2^-3, rms 0.09 of the value) on the other side, of
n codes up to m + 4 sqrt(m) + 4 about the mean m; each changes y by 0.09 of its
share, so y's norm by 0.09 sqrt(flips / n).  M-tiles: the cut terms are off by
2^-13 / sqrt(3) of an octet's largest product, r = 5e-5 and 1.6e-3 of the codes;
streaming: at most 64 additions' roundings and the exponential's, r = 1e-6 and
3e-5 of them.  Twice that, for codes of uneven size, and fp16's 2^-11.
"""
import numpy as np
import pytest
import torch

import oracle
import routed_expert_ffn_03_amd as moe
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
FP8 = moe.MOE_WFMT_FP8_B128
U = 2.0 ** -24


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bf16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)


# ------------------------------------------------------------ quantiser

def _quant_case(kind, shape, rng):
    v = rng.standard_normal(shape).astype(np.float32)
    if kind == "wide":
        v *= np.exp(rng.uniform(-60, 60, (*shape[:-1], 1))).astype(np.float32)
    elif kind == "edge":                    # maxima on and next to 448 * 2^e, zero and tiny blocks
        flat = v.reshape(-1, 128)
        for i in range(flat.shape[0]):
            top = [448.0, 450.0, 446.0, 224.0, 0.0, 1e-39, 2.0 ** -126, 3.3e38][i % 8]
            flat[i] = 0 if top == 0 else np.clip(flat[i] / 8, -1, 1) * top
            flat[i, i % 128] = -top
    elif kind == "bad":
        flat = v.reshape(-1, 128)
        flat[0, 5] = np.nan
        flat[-1, 7] = np.inf
        flat[len(flat) // 2, 9] = -np.inf
        if len(flat) > 3:
            flat[2] = np.nan                    # not one finite value
    return v


@pytest.mark.parametrize("kind", ["normal", "wide", "edge", "bad"])
@pytest.mark.parametrize("shape,br", [((1, 128), 1), ((3, 384), 1), ((1001, 256), 1), ((2, 5, 128), 1),
                                      ((128, 128), 128), ((256, 384), 128), ((3, 128, 256), 128)])
def test_quantize_is_bit_exact(kind, shape, br):
    _cuda()
    say(f"[quant] {kind} {shape} block_rows={br}")
    rng = np.random.default_rng(abs(hash((len(kind), shape, br))) % 1000)
    src = bf16(_quant_case(kind, shape, rng))
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty((*shape[:-2], shape[-2] // br, shape[-1] // 128), device="cuda")
    moe.moe_quantize_fp8(src.cuda(), codes, scales, block_rows=br)
    v = src.double().numpy().reshape(-1, *shape[-2:])
    got_c, got_s = codes.cpu().numpy().reshape(v.shape), scales.cpu().numpy().reshape(len(v), -1, shape[-1] // 128)
    for i in range(len(v)):
        c, s = oracle.quantize_fp8(v[i], br)
        np.testing.assert_array_equal(got_s[i].astype(np.float64), s)
        nan = (c & 0x7F) == 0x7F
        np.testing.assert_array_equal((got_c[i] & 0x7F) == 0x7F, nan)
        np.testing.assert_array_equal(got_c[i][~nan], c[~nan])


# ------------------------------------------------------------ grouped FFN

def _weights(E, N, K, rng, spread=0.5):
    codes = oracle.f64_to_e4m3(np.clip(rng.standard_normal((E, N, K)) * 100, -448, 448))
    scales = (2e-4 * (1 + spread * (2 * rng.random((E, N // 128, K // 128)) - 1))).astype(np.float32)
    return codes, scales


def make_case(T, E, k, H, I, seed, live=None):
    """Random layer of e4m3 experts; only the first `live` experts are ever picked."""
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if live is not None:
        logits[:, live:] -= 100
    x = bf16(rng.standard_normal((T, H)) * np.exp(0.5 * rng.standard_normal(H)))
    W = {}
    for n, (N, K) in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
        W[n], W[n + "_scale"] = _weights(E, N, K, rng)
    return logits, x, W


def dev_weights(W):
    return {n: torch.from_numpy(a).cuda() for n, a in W.items()}


def sum_error(x, w):
    """Bound of the e4m3 product sums x w^T (module docstring), x and w values with their scales."""
    K = x.shape[1]
    ax, aw = np.abs(x), np.abs(w)
    d = (K / 8 + K / 128 + 4) * 2 * U * (ax @ aw.T)
    for o in range(0, K, 8):
        for r in range(0, len(x), 64):
            d[r:r + 64] += 2.0 ** -10 * np.max(ax[r:r + 64, None, o:o + 8] * aw[None, :, o:o + 8], axis=2)
    return d


def rows_reference(rows, wg, wu, wd):
    """Oracle y of one expert's quantised rows and the bound of each element (module docstring)."""
    H, I = wg.shape[1], wg.shape[0]
    y, a, aq = oracle.fp8_expert_ffn(rows, wg, wu, wd)
    g, u = rows @ wg.T, rows @ wu.T
    dg, du = sum_error(rows, wg), sum_error(rows, wu)
    da = 1.1 * dg * np.abs(u) + (np.abs(oracle.silu(g)) + 1.1 * dg) * du + (8 + 2 * np.abs(g)) * 2 * U * np.abs(a)
    step = np.zeros_like(a)                         # how far aq may be from the oracle's
    for r in range(a.shape[0]):
        for b in range(I // 128):
            c = slice(128 * b, 128 * b + 128)
            top = np.max(np.abs(a[r, c]))
            near = da[r, c][np.argmax(np.abs(a[r, c]))]
            scales = {oracle.fp8_block_scale(max(top - near, 0)), oracle.fp8_block_scale(top),
                      oracle.fp8_block_scale(top + near)}
            for q in scales:                        # every code that a within da may get
                for d in (-1, 1):
                    z = np.clip((a[r, c] + d * da[r, c]) / q, -448, 448)
                    v = oracle.e4m3_to_f64(oracle.f64_to_e4m3(z)) * q
                    step[r, c] = np.maximum(step[r, c], np.abs(v - aq[r, c]))
    bound = step @ np.abs(wd).T + sum_error(np.abs(aq) + step, wd)
    return y, bound * (1 + 2.0 ** -11) + 2.0 ** -11 * np.abs(y) + 2.0 ** -25


def reference(logits, x, W, k):
    """Oracle y and its per-element bound for every sorted row, and the routing."""
    T, E = logits.shape
    ids, w = oracle.route_topk(logits, k)
    _, off, sp, p2s = oracle.permute(ids, E)
    xv = x.double().numpy()
    xq = oracle.fp8_values(*oracle.quantize_fp8(xv, 1))
    H = xv.shape[1]
    Y, bound = np.zeros((T * k, H)), np.zeros((T * k, H))
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi == lo:
            continue
        m = (oracle.fp8_values(W[n][e], W[n + "_scale"][e].astype(np.float64)) for n in ("gate", "up", "down"))
        Y[lo:hi], bound[lo:hi] = rows_reference(xq[np.asarray(sp[lo:hi]) // k], *m)
    return Y, bound, w, ids, off, sp, p2s


def run_ffn(logits, x, W, k, thr, dw=None):
    T, E = logits.shape
    H, I = x.shape[1], W["gate"].shape[1]
    b = moe.MoELayerBuffers(T, E, k, H, I, FP8)
    b.y_sorted.fill_(7.0)
    b.workspace.fill_(0xFF)                         # whatever an earlier call left behind
    out = b.forward(torch.from_numpy(logits).cuda(), x.cuda(), dw or dev_weights(W), fat_threshold=thr)
    torch.cuda.synchronize()
    return b, out


def norm_bound(n, tiles):
    m = (1.6e-3 if tiles else 3e-5) * n
    return 2 * 0.09 * np.sqrt((m + 4 * np.sqrt(m) + 4) / n) + 2.0 ** -11


def check(b, ref, what, thr):
    Y, bound = ref[0], ref[1]
    got = b.y_sorted.double().cpu().numpy()
    ratio = np.abs(got - Y) / bound
    norm = np.linalg.norm(got - Y) / np.linalg.norm(Y)
    say(f"   {what}: worst error / bound {ratio.max():.3f}, norm {norm:.2e}, rel max {oracle.rel_max_err(got, Y):.2e}")
    assert np.isfinite(got).all() and ratio.max() <= 1.0, what
    assert norm <= norm_bound(len(Y) * b.I, thr <= len(Y)), what


CASES = [(1, 4, 2, 256, 128, None), (3, 4, 4, 256, 128, None), (5, 16, 3, 512, 384, None), (31, 3, 1, 256, 128, 1),
         (32, 3, 1, 256, 128, 1), (33, 3, 2, 256, 256, 2), (64, 16, 2, 256, 128, None), (70, 8, 2, 512, 128, 5),
         (130, 4, 2, 256, 384, None), (257, 5, 2, 256, 128, 2), (300, 6, 2, 768, 256, 3)]


@pytest.mark.parametrize("T,E,k,H,I,live", CASES)
def test_ffn_matches_the_oracle(T, E, k, H, I, live):
    _cuda()
    logits, x, W = make_case(T, E, k, H, I, T + H, live)
    ref = reference(logits, x, W, k)
    dw = dev_weights(W)
    for thr in (1, 8, 32, 10 ** 6):
        say(f"[fp8] T={T} E={E} k={k} H={H} I={I} live={live} thr={thr}")
        b, out = run_ffn(logits, x, W, k, thr, dw)
        check(b, ref, f"thr {thr}", thr)
        Yk = b.y_sorted.double().cpu().numpy()
        want = oracle.combine(Yk, ref[2], ref[6], k)
        # fp32 fma over k terms, gate weights within 2e-6
        lim = (k * U * 2 + 2e-6) * oracle.combine(np.abs(Yk), np.ones_like(ref[2]), ref[6], k) + 1e-30
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= lim)


@pytest.mark.parametrize("T,E,k,H,I", [(4, 384, 8, 4096, 2048), (65, 24, 4, 2304, 1408), (1500, 12, 6, 1024, 640)])
def test_ffn_paths_agree_on_larger_layers(T, E, k, H, I):
    """All-streaming, all-MFMA and mixed plans agree; sampled rows of each within the oracle's bound."""
    _cuda()
    say(f"[fp8 large] T={T} E={E} k={k} H={H} I={I}")
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = {}
    for n, (N, K) in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
        src = (torch.randn(E, N, K, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
        w[n] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
        w[n + "_scale"] = torch.empty(E, N // 128, K // 128, device="cuda")
        moe.moe_quantize_fp8(src, w[n], w[n + "_scale"], block_rows=128)
        del src
    ys = []
    for thr in (32, 1, 10 ** 6):
        b = moe.MoELayerBuffers(T, E, k, H, I, FP8)
        b.forward(logits, x, w, fat_threshold=thr)
        ys.append(b.y_sorted.double().cpu().numpy())
    ids = b.topk_ids.cpu().numpy()
    off, sp = b.expert_offsets.cpu().numpy(), b.sorted_pair.cpu().numpy()
    assert (ids < E).all()
    rng = np.random.default_rng(T)
    rows = rng.choice(T * k, 12, replace=False)
    xn = x.double().cpu().numpy()
    for r in rows:
        e = int(np.searchsorted(off, r, side="right") - 1)
        xq = oracle.fp8_values(*oracle.quantize_fp8(xn[sp[r] // k][None], 1))
        m = [oracle.fp8_values(w[n][e].view(torch.uint8).cpu().numpy(), w[n + "_scale"][e].double().cpu().numpy())
             for n in ("gate", "up", "down")]
        y, bound = rows_reference(xq, *m)
        for got in ys:
            assert np.all(np.abs(got[r] - y[0]) <= bound[0]), r
    # every row: each path is within norm_bound of the values, so two are within twice that
    for y in ys[1:]:
        assert np.linalg.norm(y - ys[0]) <= 2 * norm_bound(T * k * I, True) * np.linalg.norm(ys[0])


def test_bad_values_stay_in_their_rows():
    _cuda()
    T, E, k, H, I = 40, 4, 2, 256, 128
    logits, x, W = make_case(T, E, k, H, I, 11)
    x[3, 17] = float("nan")
    x[9, 200] = float("inf")
    x[12] = 0
    for thr in (1, 10 ** 6):
        b, out = run_ffn(logits, x, W, k, thr)
        bad = set(torch.nonzero(~torch.isfinite(out).all(1)).reshape(-1).tolist())
        assert bad == {3, 9}, (thr, bad)
        rows = b.pair_to_sorted.view(T, k)[12].long()
        assert (b.y_sorted[rows] == 0).all()


def test_noalloc_and_another_stream_give_the_same_bits():
    _cuda()
    T, E, k, H, I = 300, 8, 2, 512, 256
    logits, x, W = make_case(T, E, k, H, I, 5)
    dw = dev_weights(W)
    b, _ = run_ffn(logits, x, W, k, 32, dw)
    ref = b.y_sorted.clone()
    kw = dict(s_gate=dw["gate_scale"], s_up=dw["up_scale"], s_down=dw["down_scale"], wfmt=FP8)
    y = torch.full_like(ref, 7.0)
    moe.moe_grouped_ffn_noalloc(x.cuda(), dw["gate"], dw["up"], dw["down"], b.expert_offsets, b.sorted_pair, k, y, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, ref)
    s = torch.cuda.Stream()
    y2 = torch.full_like(ref, 7.0)
    ws = torch.empty_like(b.workspace)
    xd = x.cuda()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_grouped_ffn(xd, dw["gate"], dw["up"], dw["down"], b.expert_offsets, b.sorted_pair, k, y2, ws, stream=s, **kw)
    s.synchronize()
    assert torch.equal(y2, ref)


@pytest.mark.parametrize("T", [1, 4, 80])
def test_captured_layer_replays(T):
    """A captured layer call on changing inputs, with eager work between the replays."""
    _cuda()
    E, k, H, I = 12, 3, 512, 256
    dw = dev_weights(make_case(T, E, k, H, I, 21)[2])
    b, e = (moe.MoELayerBuffers(T, E, k, H, I, FP8) for _ in range(2))
    lg, xs = torch.empty(T, E, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    for seed in (0, 1, 2, 3):
        l, x, _ = make_case(T, E, k, H, I, 100 + seed)
        lg.copy_(torch.from_numpy(l))
        xs.copy_(x)
        if seed == 0:
            st = torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                b.forward(lg, xs, dw)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                b.forward(lg, xs, dw)
        b.out.fill_(3.0)
        graph.replay()
        want = e.forward(lg, xs, dw)
        torch.cuda.synchronize()
        assert torch.equal(b.out, want), seed


def test_single_phases_equal_the_whole():
    _cuda()
    T, E, k, H, I = 90, 6, 2, 256, 256
    logits, x, W = make_case(T, E, k, H, I, 8)
    dw = dev_weights(W)
    b, _ = run_ffn(logits, x, W, k, 32, dw)
    ref = b.y_sorted.clone()
    xd = x.cuda()
    moe.moe_ffn_plan(b.expert_offsets, T, k, H, I, b.workspace, wfmt=FP8)
    for _ in range(2):                              # a phase may run again on one plan
        moe.moe_ffn_gate_up(xd, dw["gate"], dw["up"], b.sorted_pair, E, k, b.workspace, s_gate=dw["gate_scale"],
                            s_up=dw["up_scale"], wfmt=FP8)
    b.y_sorted.fill_(1.0)
    moe.moe_ffn_down(dw["down"], T, E, k, I, b.y_sorted, b.workspace, s_down=dw["down_scale"], wfmt=FP8)
    torch.cuda.synchronize()
    assert torch.equal(b.y_sorted, ref)


def test_binding_refuses_wrong_scales_and_codes():
    _cuda()
    T, E, k, H, I = 8, 4, 2, 256, 128
    logits, x, W = make_case(T, E, k, H, I, 1)
    dw = dev_weights(W)
    b, _ = run_ffn(logits, x, W, k, 32, dw)
    def call(**kw):
        a = dict(dw); a.update(kw)
        moe.moe_grouped_ffn(x.cuda(), a["gate"], a["up"], a["down"], b.expert_offsets, b.sorted_pair, k, b.y_sorted,
                            b.workspace, s_gate=a["gate_scale"], s_up=a["up_scale"], s_down=a["down_scale"], wfmt=FP8)
    for kw in (dict(gate_scale=dw["gate_scale"].half()), dict(up_scale=dw["up_scale"][:, :, :1].contiguous()),
               dict(down=dw["down"].float()), dict(down_scale=None), dict(up=dw["up"][:2].contiguous()),
               dict(gate=dw["gate"].transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)
