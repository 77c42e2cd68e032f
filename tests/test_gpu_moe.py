"""The experts' feed-forward block against the oracle: routing, rows quantised
through a list, grouped products, combination, and all of them in a row."""

import numpy as np
import pytest
import torch

from oracle import iq_oracle as O
from oracle import moe_oracle as X

pytestmark = pytest.mark.gpu


def _iq():
    from fp4_fp8_quant_gb300 import iq
    return iq


def dev(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).cuda()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def bf16(rng, shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def weights(rng, G, N, K):
    """Codes of normal values and block scales over 2^8."""
    codes = O.round_to_e4m3_codes(np.clip(rng.standard_normal((G, N, K)) * 64, -448, 448)).astype(np.uint8)
    return codes, rng.integers(112, 120, (G, -(-N // 128), K // 128)).astype(np.uint8)


def rows(rng, M, K):
    """Random codes and packed scale words of M rows."""
    codes = O.round_to_e4m3_codes(np.clip(rng.standard_normal((M, K)) * 64, -448, 448)).astype(np.uint8)
    words = np.zeros((-(-K // 512), (M + 3) // 4 * 4, 4), np.uint8)
    for b in range(K // 128):
        words[b // 4, :M, b % 4] = rng.integers(116, 124, M)
    return codes, words.view(np.int32)[:, :, 0]


def grouped_bound(out, mag, K):
    """Largest allowed |kernel - exact|: the result is rounded to BF16, at most
    2^-8 of it; a float32 sum of K exact products, each addition truncated, is off
    by at most K 2^-23 of the sum of their magnitudes (mag; gated it already
    carries the derivatives of silu(g) u); gated, exp, quotient and products are
    off by less than 2^-16."""
    return (2.0 ** -8 + 2.0 ** -16) * np.abs(out) + K * 2.0 ** -23 * mag + 1e-30


def check_grouped(got, x, words, w, w_sf, row_start, gated, before):
    want, mag, there = X.grouped(x, words, w, w_sf, row_start, gated)
    err = np.abs(f64(got) - want)
    bad = ~(err <= grouped_bound(want, mag, x.shape[1])) & there[:, None]
    assert not bad.any(), (np.argwhere(bad)[:5], err[bad][:5], want[bad][:5])
    assert torch.equal(got.cpu()[~torch.from_numpy(there)], before[~torch.from_numpy(there)])


def run_grouped(x, words, w, w_sf, row_start, gated, ld_pad=0):
    n = w.shape[1] // 2 if gated else w.shape[1]
    before = torch.full((x.shape[0], n + ld_pad), 7.0, dtype=torch.bfloat16)
    out = before.cuda()
    _iq().grouped_gemm(dev(x), dev(words), dev(w), dev(w_sf), dev(np.asarray(row_start, np.int32)), gated=gated,
                       out=out[:, :n] if ld_pad else out)
    torch.cuda.synchronize()
    if ld_pad:
        assert torch.equal(out[:, n:].cpu(), before[:, n:])
    check_grouped(out[:, :n], x, words, w, w_sf, row_start, gated, before[:, :n])
    assert _iq().device_status() == 0


SHAPES = [
    # K, N, gated, rows per group
    (128, 8, False, [1]),
    (128, 256, True, [1]),
    (256, 128, False, [3]),
    (512, 256, False, [16, 0, 17]),
    (640, 384, False, [0, 1, 0, 31, 0]),
    (1536, 512, True, [5, 33, 0, 1]),
    (384, 520, False, [100, 225, 7]),
    (1280, 768, True, [224, 225]),
    (896, 1544, False, [449, 2, 300]),
    (2048, 256, False, [700]),
    (256, 4096, False, [1] * 40),
    (256, 512, True, [13] * 33),
    (2304, 1544, False, [1, 0, 2]),              # cut between pairs: a workspace and a join
    (4224, 768, True, [40, 3]),
    (5248, 2048, False, [230, 256, 90]),
    (2432, 256, True, [1] * 500),
]


@pytest.mark.parametrize("K,N,gated,counts", SHAPES)
def test_grouped(cuda_device, K, N, gated, counts):
    rng = np.random.default_rng(K + N + sum(counts))
    M = sum(counts)
    run_grouped(*rows(rng, M, K), *weights(rng, len(counts), N, K), np.concatenate([[0], np.cumsum(counts)]), gated)


def test_grouped_rows_of_no_group(cuda_device):
    """Rows before the first and behind the last group, and a wider output."""
    rng = np.random.default_rng(1)
    x, words = rows(rng, 77, 256)
    run_grouped(x, words, *weights(rng, 3, 136, 256), [5, 20, 20, 61], False, ld_pad=24)


@pytest.mark.parametrize("row_start", [[0, 0, 0], [-9, 4, 1000], [40, 10, 50], [60, 60, 60], [7, -1, 2]])
def test_grouped_row_start_outside_its_range(cuda_device, row_start):
    rng = np.random.default_rng(2)
    run_grouped(*rows(rng, 50, 128), *weights(rng, 2, 128, 128), row_start, False)


def test_grouped_many_groups(cuda_device):
    """1024 groups, most of them empty, the first and the last among the others."""
    rng = np.random.default_rng(3)
    counts = np.zeros(1024, int)
    counts[[0, 31, 32, 500, 511, 512, 1022, 1023]] = [1, 2, 3, 18, 1, 40, 2, 5]
    M = counts.sum()
    run_grouped(*rows(rng, M, 128), *weights(rng, 1024, 128, 128), np.concatenate([[0], np.cumsum(counts)]), False)


LOGITS = [(1, 2, 1), (1, 256, 8), (3, 33, 5), (32, 64, 8), (33, 64, 6), (200, 7, 7), (130, 300, 3), (129, 1024, 32),
          (700, 513, 2), (513, 1, 1), (1000, 512, 8), (2048, 6, 2), (2049, 6, 2), (9001, 34, 3), (64, 1024, 4), (255, 40, 32),
          (256, 1000, 5), (257, 70, 6), (16385, 5, 2), (16, 64, 8), (17, 64, 8), (128, 65, 3), (512, 256, 8), (1024, 8, 4),
          (1025, 9, 4), (2048, 40, 4), (513, 40, 4), (5, 1024, 32), (16, 600, 1), (3, 500, 9), (4900, 260, 3), (1024, 128, 8), (1025, 64, 6), (1000, 3, 2), (1300, 1, 1)]


def check_route(got, logits, k, score, normalize, scale):
    w, experts, slots, rows_, start = X.route(f64(logits), k, score, normalize, scale)
    for name, a, b in (("experts", got.experts, experts), ("slots", got.slots, slots), ("rows", got.rows, rows_),
                       ("row_start", got.row_start, start)):
        assert np.array_equal(a.cpu().numpy(), b), name
    # exp within 2 units, sums of up to 1024 positive terms over 32 lanes within
    # 40 roundings, division and products: below 64 * 2^-24 of the weight; exp
    # of a rounded difference |d| < 32: 2 * 2^-24 |d| more.
    assert np.all(np.abs(f64(got.weights) - w) <= 128 * 2.0 ** -24 * np.abs(w) + 1e-37)


@pytest.mark.parametrize("T,E,k", LOGITS)
@pytest.mark.parametrize("score,normalize,dtype", [("softmax", False, torch.float32), ("softmax", True, torch.bfloat16),
                                                   ("sigmoid", True, torch.float32), ("sigmoid", False, torch.bfloat16)])
def test_route(cuda_device, T, E, k, score, normalize, dtype):
    rng = np.random.default_rng(T * 7 + E + k)
    l = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32)).to(dtype)
    if T > 2:                                     # ties, and the same row throughout
        l[1] = l[1].round()
        l[2] = 0.5
    pad = torch.zeros((T, E + 3), dtype=dtype)
    pad[:, :E] = l
    got = _iq().moe_route(dev(pad)[:, :E], k, score=score, normalize=normalize, scale=1.5)
    check_route(got, l, k, score, normalize, 1.5)


@pytest.mark.parametrize("score,normalize", [("softmax", False), ("softmax", True), ("sigmoid", True), ("sigmoid", False)])
def test_route_masked_logits(cuda_device, score, normalize):
    """-inf, the lowest value, NaN and signed zeros; a row that leaves nothing."""
    l = torch.zeros((70, 9))
    l[0] = -np.inf
    l[1] = torch.tensor([-np.inf, 1, -np.inf, 2, -np.inf, -np.inf, 0, -np.inf, -np.inf])
    l[2] = torch.tensor([0.0, -0.0, 0.0, -0.0, -1, -1, -1, -1, -1])
    l[3] = torch.finfo(torch.float32).min
    l[4] = torch.tensor([np.nan, 3, np.nan, 3, 1, np.nan, np.nan, np.nan, np.nan])
    l[5] = torch.tensor([-np.inf] * 8 + [torch.finfo(torch.float32).min])
    l[6] = torch.tensor([np.nan] * 9)
    got = _iq().moe_route(dev(l), 4, score=score, normalize=normalize)
    check_route(got, l, 4, score, normalize, 1.0)


def test_route_without_tokens(cuda_device):
    got = _iq().moe_route(torch.empty((0, 8), device="cuda"), 2)
    assert got.row_start.cpu().tolist() == [0] * 9 and got.weights.shape == (0, 2) and got.rows.shape == (0,)


@pytest.mark.parametrize("K,M", [(128, 1), (640, 7), (1536, 130), (7168, 33)])
def test_quantised_rows_of_a_list(cuda_device, K, M):
    """The codes and scales of the listed rows are the quantizer's own; rows
    outside are zeros."""
    iq = _iq()
    rng = np.random.default_rng(K + M)
    x = dev(bf16(rng, (20, K), 3.0))
    idx = rng.integers(-3, 24, M).astype(np.int32)
    inside = (idx >= 0) & (idx < 20)
    gathered = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    gathered[dev(inside)] = x[dev(idx[inside].astype(np.int64))]
    y, s = iq.fp8_quant_1x128_ue8m0(x, rows=dev(idx))
    want, ws = iq.fp8_quant_1x128_ue8m0(gathered)
    assert torch.equal(y, want) and torch.equal(s, ws)


@pytest.mark.parametrize("T,k,N,add", [(1, 1, 8, False), (1, 8, 7168, True), (5, 3, 1032, True), (300, 9, 136, False),
                                       (64, 20, 2048, True)])
def test_combine(cuda_device, T, k, N, add):
    rng = np.random.default_rng(T + k + N)
    S = T * k
    y = bf16(rng, (S, N + 8))
    slots = rng.permutation(S).reshape(T, k).astype(np.int32)
    slots[0, 0] = -1 if T > 1 else slots[0, 0]
    if T > 2:
        slots[1, 0], slots[2, 0] = S, slots[2, -1]            # past the end; the same slot twice
    w = rng.uniform(-1, 1, (T, k)).astype(np.float32)
    a = bf16(rng, (T, N)) if add else None
    got = _iq().moe_combine(dev(y)[:, :N], dev(slots), dev(w), add=None if a is None else dev(a))
    want, mag = X.combine(f64(y[:, :N]), slots, w, None if a is None else f64(a))
    # k + 1 float32 additions of exact products (fused), one rounding to BF16
    assert np.all(np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -24 * mag + 1e-30)


def test_combine_into_what_is_added(cuda_device):
    rng = np.random.default_rng(9)
    y, a = bf16(rng, (6, 64)), bf16(rng, (3, 64))
    slots, w = np.arange(6, dtype=np.int32).reshape(3, 2), np.ones((3, 2), np.float32)
    want = _iq().moe_combine(dev(y), dev(slots), dev(w), add=dev(a))
    acc = dev(a)
    assert _iq().moe_combine(dev(y), dev(slots), dev(w), add=acc, out=acc) is acc and torch.equal(acc, want)


def moe_block(iq, x, logits, k, wu, wu_sf, wd, wd_sf, add):
    r = iq.moe_route(logits, k, normalize=True)
    xq, xs = iq.fp8_quant_1x128_ue8m0(x, rows=r.rows)
    h = iq.grouped_gemm(xq, xs, wu, wu_sf, r.row_start, gated=True)
    hq, hs = iq.fp8_quant_1x128_ue8m0(h)
    y = iq.grouped_gemm(hq, hs, wd, wd_sf, r.row_start)
    return r, h, y, iq.moe_combine(y, r.slots, r.weights, add=add)


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (37, 8, 3), (150, 6, 2)])
def test_a_feed_forward_block(cuda_device, T, E, k):
    """Route, quantise, up, quantise, down, combine: each step against the
    oracle on what the step before gave."""
    iq = _iq()
    rng = np.random.default_rng(T)
    K, I = 384, 256
    x, add = bf16(rng, (T, K)), bf16(rng, (T, K))
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    wu, wu_sf = weights(rng, E, 2 * I, K)
    wd, wd_sf = weights(rng, E, K, I)
    wd_sf -= 8
    wu_sf -= 4
    args = [dev(a) for a in (x, logits)] + [k] + [dev(a) for a in (wu, wu_sf, wd, wd_sf, add)]
    r, h, y, out = moe_block(iq, *args)
    torch.cuda.synchronize()
    check_route(r, logits, k, "softmax", True, 1.0)
    start, none = r.row_start.cpu().numpy(), torch.zeros(0)
    bits = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)
    xq, xw = O.fp8_quant_1x128_ue8m0(bits(x[r.rows.cpu().long()].contiguous()))
    check_grouped(h, xq, xw, wu, wu_sf, start, True, h.cpu())
    hq, hw = O.fp8_quant_1x128_ue8m0(bits(h))
    check_grouped(y, hq, hw, wd, wd_sf, start, False, y.cpu())
    want, mag = X.combine(f64(y), r.slots.cpu().numpy(), r.weights.cpu().numpy(), f64(add))
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -24 * mag + 1e-30)
    # captured and replayed on other rows
    graph = torch.cuda.CUDAGraph()
    x2 = dev(bf16(rng, (T, K)))
    with torch.cuda.graph(graph):
        _, _, _, out_g = moe_block(iq, *args)
    args[0].copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_g, moe_block(iq, *args)[3])
    assert iq.device_status() == 0


def test_gates_far_below_zero(cuda_device):
    """gate * up where gate times up, before the sigmoid, is no float32 any more."""
    x = np.zeros((3, 128), np.uint8)
    x[:, 0] = 0x38                                              # 1
    words = np.zeros((1, 4), np.int32)
    words.view(np.uint8)[0, ::4] = 127
    w = np.zeros((1, 256, 128), np.uint8)
    g = np.array([-448, -224, -100, -88, -40, -20, -1, 0, 1, 20, 448], np.float64)
    w[0, :len(g), 0] = O.round_to_e4m3_codes(g)
    w[0, 128:, 0] = O.round_to_e4m3_codes(np.where(np.arange(128) % 2, -1.0, 1.0))
    for up in (127, 247):                                       # 1, 2^120
        w_sf = np.array([[[128], [up]]], np.uint8)              # gates twice their codes
        if up == 247:                                           # and none whose product overflows
            w[0, 128 + 8:, 0] = 0
        run_grouped(x, words, w, w_sf, [0, 3], True)


@pytest.mark.parametrize("K,gated", [(384, False), (4224, True)])
def test_what_stands_in_rows_of_no_group_goes_nowhere(cuda_device, K, gated):
    rng = np.random.default_rng(K)
    M, start = 90, [3, 20, 20, 37, 80]
    x, words = rows(rng, M, K)
    w, w_sf = weights(rng, 4, 512, K)
    clean = run_again(x, words, w, w_sf, start, gated)
    none = np.ones(M, bool)
    none[start[0]:start[-1]] = False
    x[none] = 0x7F                                              # NaN, and NaN scales
    words[:, :M][:, none] = -1
    w[1], w_sf[1] = 0x7F, 255                                   # the empty group's
    assert torch.equal(run_again(x, words, w, w_sf, start, gated)[3:80], clean[3:80])


def run_again(x, words, w, w_sf, start, gated):
    return _iq().grouped_gemm(dev(x), dev(words), dev(w), dev(w_sf), dev(np.asarray(start, np.int32)), gated=gated).cpu()


def test_grouped_on_two_streams_at_once_and_replayed(cuda_device):
    """Products that are cut between pairs, so that workspaces are used: on two
    streams at a time, and from a graph on other rows and other bounds."""
    iq = _iq()
    rng = np.random.default_rng(11)
    K, N = 5248, 1544
    w, w_sf = weights(rng, 3, N, K)
    gw, gsf = dev(w), dev(w_sf)
    x, words = rows(rng, 200, K)
    starts = [np.array(s, np.int32) for s in ([0, 70, 71, 200], [0, 9, 150, 151])]
    gx, gwords, gs = dev(x), dev(words), [dev(s) for s in starts]
    assert iq.grouped_gemm_workspace_bytes(200, K) > 0
    torch.cuda.synchronize()
    outs = [[], []]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for i, s in enumerate(streams):
            outs[i].append(iq.grouped_gemm(gx, gwords, gw, gsf, gs[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        n = starts[i][-1]
        check_grouped(outs[i][0], x, words, w, w_sf, starts[i], False, outs[i][0].cpu())
        assert all(torch.equal(o[:n], outs[i][0][:n]) for o in outs[i])
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros((200, N), dtype=torch.bfloat16, device="cuda")
    with torch.cuda.graph(graph):
        iq.grouped_gemm(gx, gwords, gw, gsf, gs[0], out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, outs[0][0])
    gs[0].copy_(gs[1])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:151], outs[1][0][:151]) and torch.equal(out[151:], outs[0][0][151:])
    assert iq.device_status() == 0


@pytest.mark.parametrize("T", [20, 100, 2100, 16400])
def test_route_and_combine_on_another_stream_and_replayed(cuda_device, T):
    iq = _iq()
    rng = np.random.default_rng(T)
    E, k = 40, 4
    l, y = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)) for s in ((2, T, E), (T * k, 72)))
    y = y.to(torch.bfloat16)
    gl, gy = dev(l[0]), dev(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r = iq.moe_route(gl, k, score="sigmoid", normalize=True, stream=side)
    c = iq.moe_combine(gy, r.slots, r.weights, stream=side)
    side.synchronize()
    check_route(r, l[0], k, "sigmoid", True, 1.0)
    want, mag = X.combine(f64(y), r.slots.cpu().numpy(), r.weights.cpu().numpy())
    assert np.all(np.abs(f64(c) - want) <= 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -24 * mag + 1e-30)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = iq.moe_route(gl, k, score="sigmoid", normalize=True)
        c = iq.moe_combine(gy, r.slots, r.weights)
    gl.copy_(l[1])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        check_route(r, l[1], k, "sigmoid", True, 1.0)
        assert torch.equal(c, iq.moe_combine(gy, r.slots, r.weights))


def test_offsets_past_32_bits(cuda_device):
    """Rows, results, weights and combined rows further apart than 2^32 bytes."""
    iq = _iq()
    rng = np.random.default_rng(12)
    M, K, N, far = 40, 256, 136, (1 << 27) + 64                 # 40 rows: 5 GB of bytes, 10 of BF16
    x, words = rows(rng, M, K)
    w, w_sf = weights(rng, 1, N, K)
    buf = torch.empty((M * far,), dtype=torch.uint8, device="cuda").view(M, far)
    buf[:, :K] = dev(x)
    out = torch.empty((M * far,), dtype=torch.bfloat16, device="cuda").view(M, far)[:, :N]
    got = iq.grouped_gemm(buf[:, :K], dev(words), dev(w), dev(w_sf), dev(np.array([0, M], np.int32)), out=out)
    check_grouped(got.contiguous(), x, words, w, w_sf, [0, M], False, got.contiguous().cpu())
    slots = np.array([[M - 1, 0], [1, M - 1]], np.int32)
    weight = rng.uniform(-1, 1, (2, 2)).astype(np.float32)
    c = iq.moe_combine(out, dev(slots), dev(weight))
    want, mag = X.combine(f64(got.contiguous()), slots, weight)
    assert np.all(np.abs(f64(c) - want) <= 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -24 * mag + 1e-30)
    src = out.as_strided((M, 128), (far // 2, 1))               # rows 2^27 bytes apart
    src.copy_(dev(bf16(rng, (M, 128))))
    idx = dev(np.array([M - 1, 0, M - 1], np.int32))
    y, s = iq.fp8_quant_1x128_ue8m0(src, rows=idx)
    want_y, want_s = iq.fp8_quant_1x128_ue8m0(src[idx.long()].contiguous())
    assert torch.equal(y, want_y) and torch.equal(s, want_s)
    del buf, out, got, src
    G, N, K = 640, 1024, 7168                                   # 4.7 GB of weights, the last group's tested
    wide = torch.zeros((G, N, K), dtype=torch.uint8, device="cuda")
    sf = torch.full((G, N // 128, K // 128), 100, dtype=torch.uint8, device="cuda")
    w, w_sf = weights(rng, 1, N, K)
    wide[-1], sf[-1] = dev(w[0]), dev(w_sf[0])
    x, words = rows(rng, 5, K)
    start = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    start[-1] = 5
    for gated in (False, True):
        got = iq.grouped_gemm(dev(x), dev(words), wide, sf, start, gated=gated)
        check_grouped(got, x, words, w, w_sf, [0, 5], gated, got.cpu())
    assert iq.device_status() == 0


@pytest.mark.parametrize("K,ldx", [(512, 520), (1152, 1152), (2176, 2304)])
def test_quantised_rows_all_of_one(cuda_device, K, ldx):
    """A list that names one row throughout, and one that names none; more rows than
    a block's, K that ends inside a warp's columns, a wider input and output."""
    iq = _iq()
    rng = np.random.default_rng(K)
    x = dev(bf16(rng, (5, ldx), 3.0))[:, :K]
    want, ws = iq.fp8_quant_1x128_ue8m0(x[3:4].contiguous())
    none, ns = iq.fp8_quant_1x128_ue8m0(torch.zeros((1, K), dtype=torch.bfloat16, device="cuda"))
    for M in (4, 1027):
        y = torch.zeros((M, K + 16), dtype=torch.uint8, device="cuda")
        _, s = iq.fp8_quant_1x128_ue8m0(x, y[:, :K], rows=torch.full((M,), 3, dtype=torch.int32, device="cuda"))
        assert torch.equal(y[:, :K], want.expand(M, K)) and torch.equal(s[:, :M], ws[:, :1].expand(-1, M)) and not y[:, K:].any()
        y, s = iq.fp8_quant_1x128_ue8m0(x, rows=torch.full((M,), 5, dtype=torch.int32, device="cuda"))
        assert torch.equal(y, none.expand(M, K)) and torch.equal(s[:, :M], ns[:, :1].expand(-1, M))


@pytest.mark.parametrize("inference", [False, True])
def test_results_in_one_allocation_are_tensors_of_their_own(cuda_device, inference):
    """Routing and quantised rows: shapes, types and places that do not overlap,
    written in place one by one, usable by autograd and outliving each other."""
    iq = _iq()
    rng = np.random.default_rng(13)
    l, x = dev(rng.standard_normal((6, 5)).astype(np.float32)), dev(bf16(rng, (6, 256)))
    with torch.inference_mode(inference):
        r = iq.moe_route(l, 2)
        y, sf = iq.fp8_quant_1x128_ue8m0(x, rows=r.rows)
        parts = [*r, y, sf]
        copies = [t.clone() for t in parts]
        assert [t.dtype for t in parts] == [torch.float32] + [torch.int32] * 4 + [torch.uint8, torch.int32]
        assert all(t.is_contiguous() and t.is_inference() == inference for t in parts)
        for group in (parts[:5], parts[5:]):
            spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in group)
            assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])) and all(a % 256 == 0 for a, _ in spans)
        for i, t in enumerate(parts):
            t.fill_(0)
            assert all(torch.equal(u, c) for u, c in list(zip(parts, copies))[i + 1:])
    if not inference:
        w = iq.moe_route(l, 2).weights.requires_grad_()      # the others are gone
        junk = torch.full((4096,), -1, dtype=torch.int32, device="cuda")
        (w * 2).sum().backward()
        assert torch.equal(w.detach(), copies[0]) and torch.equal(w.grad, torch.full_like(copies[0], 2)) and junk.min() == -1


@pytest.mark.parametrize("K", [2560, 4096])
def test_grouped_one_workspace_for_all_sizes(cuda_device, K):
    """One of the size for the most rows serves calls that are cut, that could be
    and that never are; the last kind takes none at all."""
    iq = _iq()
    rng = np.random.default_rng(K)
    w, w_sf = (dev(v) for v in weights(rng, 2, 264, K))
    ws = torch.empty(iq.grouped_gemm_workspace_bytes(600, K), dtype=torch.uint8, device="cuda")
    for M in (1, 40, 200, 256, 600):
        x, words = (dev(v) for v in rows(rng, M, K))
        start = dev(np.array([0, M // 3, M], np.int32))
        want = iq.grouped_gemm(x, words, w, w_sf, start)
        assert torch.equal(iq.grouped_gemm(x, words, w, w_sf, start, workspace=ws), want)
        if M >= 256:                                            # 10 and 16 steps, and a cut costs 17
            out = torch.zeros_like(want)
            stream = torch.cuda.current_stream().cuda_stream
            assert iq.lib().iq_grouped_gemm(x.data_ptr(), K, words.data_ptr(), M, K, w.data_ptr(), w_sf.data_ptr(), 2, 264,
                                            start.data_ptr(), 0, out.data_ptr(), 264, None, 0, stream) == 0
            assert torch.equal(out, want)
    assert iq.device_status() == 0


def test_route_one_workspace_for_all_sizes(cuda_device):
    """One of the size for 4000 tokens on both sides of where blocks get larger."""
    iq = _iq()
    rng = np.random.default_rng(14)
    ws = torch.empty(iq.moe_route_workspace_bytes(4000, 256), dtype=torch.uint8, device="cuda")
    for T in (4000, 2049, 2048, 1100, 129, 3):
        l = torch.from_numpy(rng.standard_normal((T, 256)).astype(np.float32))
        check_route(iq.moe_route(dev(l), 8, workspace=ws), l, 8, "softmax", False, 1.0)


def test_quantised_rows_of_very_many_columns(cuda_device):
    """More pairs of scale words than a launch's second dimension has blocks."""
    iq = _iq()
    K = 1024 * 65535 + 1024 + 128
    x = torch.randn((2, K), generator=torch.Generator(device="cuda").manual_seed(15), device="cuda").to(torch.bfloat16)
    want, ws = iq.fp8_quant_1x128_ue8m0(x)
    y, s = iq.fp8_quant_1x128_ue8m0(x, rows=torch.tensor([1, 2, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(y[::2], want.flip(0)) and not y[1].any()
    assert torch.equal(s[:, 0], ws[:, 1]) and torch.equal(s[:, 2], ws[:, 0])


@pytest.mark.parametrize("normalize", [False, True])
def test_route_scores_far_below_zero(cuda_device, normalize):
    """Sigmoid scores that are denormal float32 numbers or less, and their shares."""
    rng = np.random.default_rng(16)
    top = np.array([-30, -39.9, -40.1, -79.9, -80.1, -87, -89, -95, -103, -104, -110, -300, -744, -1000, -1e30], np.float32)
    l = torch.from_numpy((top[:, None] - rng.uniform(0, 5, (len(top), 12)) * (top[:, None] > -744)).astype(np.float32))
    l[:, 3] = torch.from_numpy(top)
    got = _iq().moe_route(dev(l), 4, score="sigmoid", normalize=normalize)
    check_route(got, l, 4, "sigmoid", normalize, 1.0)
    w = f64(got.weights)
    if normalize:                                               # exp(744) is no 64-bit number, so the score is 0
        assert np.allclose(w[:12].sum(axis=1), 1, rtol=1e-6) and not w[12:].any()
    else:                                                       # the smallest float32 is 2^-149
        want = X.route(f64(l), 4, "sigmoid", False)[0]
        assert np.all(np.abs(w - want) <= 128 * 2.0 ** -24 * want + 2.0 ** -149)


def whole_numbers(gen, shape, bits):
    """E4M3 codes of -2 .. 2 and UE8M0 bytes of 1 and 2 (times 2^bits), on the GPU."""
    codes = torch.randint(-2, 3, shape, generator=gen, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    scales = (*shape[:-1], shape[-1] // 128) if len(shape) == 2 else (shape[0], -(-shape[1] // 128), shape[2] // 128)
    return codes, torch.randint(127, 129, scales, generator=gen, device="cuda", dtype=torch.uint8) + bits


CUT = [
    # K, N, gated, rows per group; with 76 CTA pairs
    (2560, 136, False, [1, 0, 2]),                                             # 2 tiles of 16 rows, all of it cut
    (4736, 256, True, [250, 256]),                                             # 256 rows wide, an odd number of K-blocks
    (4608, 264, False, [512]),
    (7168, 2048, True, [300, 0, 17, 256, 1000, 0, 5, 640, 33, 2000, 0]),       # 76 of 168 tiles whole, the rest cut from inside a group
    (7168, 2040, False, [300, 0, 17, 256, 1000, 0, 5, 640, 33, 2000, 0]),
    (7168, 512, True, [1] * 100 + [0] * 20 + [30] * 20),                       # 152 of 240 whole
    (7168, 1544, False, [40] * 90),                                            # 532 of 630 whole
]


@pytest.mark.parametrize("K,N,gated,counts", CUT)
def test_grouped_cut_tiles_hold_whole_numbers(cuda_device, K, N, gated, counts):
    """Products whose float32 sums are exact, so that the rounding to BF16 is all that
    may show: a K-block left out, taken twice or joined to another tile does.  Gates
    are 0 or at least 128 away from it, where silu is 0 or the gate itself."""
    iq = _iq()
    gen = torch.Generator(device="cuda").manual_seed(K + N)
    M, G = sum(counts), len(counts)
    start = np.concatenate([[0], np.cumsum(counts)])
    x, xs = whole_numbers(gen, (M, K), 0)
    words = torch.zeros((-(-K // 512), (M + 3) // 4 * 4, 4), dtype=torch.uint8, device="cuda")
    for b in range(K // 128):
        words[b // 4, :M, b % 4] = xs[:, b]
    w, w_sf = whole_numbers(gen, (G, N, K), 0)
    if gated:
        w_sf[:, :N // 256] += 7
    ws = torch.zeros(iq.grouped_gemm_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    n_out = N // 2 if gated else N
    out = torch.full((M, n_out), 7.0, dtype=torch.bfloat16, device="cuda")
    iq.grouped_gemm(x, words.view(torch.int32)[:, :, 0], w, w_sf, dev(start.astype(np.int32)), gated=gated, out=out, workspace=ws)
    value = lambda c, s: c.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127)
    xv = value(x.view(M, K // 128, 128), xs[:, :, None]).view(M, K)
    for g in range(G):
        if counts[g] == 0:
            continue
        f = w_sf[g].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        y = xv[start[g]:start[g + 1]] @ value(w[g], f).t()
        if gated:
            y = (y[:, :n_out].clamp_min(0).float() * y[:, n_out:].float())
        assert torch.equal(out[start[g]:start[g + 1]], y.to(torch.bfloat16)), g
    # The workspace ends in a header of two int4 per pair; the first word says that
    # its last tile goes on in the next pair.
    heads = ws[-2 * 80 * 16:].view(torch.int32).view(80, 8)
    assert (heads[:, 0] == 1).any() and iq.device_status() == 0
