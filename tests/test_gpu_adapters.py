"""Low-rank adapters of many requests against the oracle."""

import numpy as np
import pytest
import torch

from oracle import moe_oracle as X

pytestmark = pytest.mark.gpu


def _iq():
    from fp4_fp8_quant_gb300 import iq
    return iq


def bf16(rng, shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def inputs(rng, T, K, N, r, A):
    return dict(x=bf16(rng, (T, K)), base=bf16(rng, (T, N)), a=bf16(rng, (A, r, K), K ** -0.5), b=bf16(rng, (A, N, r)),
                scale=torch.from_numpy(rng.uniform(-2, 2, A).astype(np.float32)))


def check(got, d, row_start, used, before=None, use_base=True):
    """Float32 sums of K and then of rank exact products (additions truncated):
    (K + rank) 2^-23 of the sum of magnitudes; A x times scale rounded to
    float32 and split into two BF16 terms: 2^-16 of it; the result rounded to
    BF16: 2^-8 of it."""
    want, mag, there = X.adapters(f64(d["x"]), f64(d["base"]) if use_base else None, f64(d["a"]), f64(d["b"]),
                                  d["scale"].numpy(), row_start, used)
    K, r = d["x"].shape[1], d["a"].shape[1]
    err = np.abs(f64(got) - want)
    bad = ~(err <= 2.0 ** -8 * np.abs(want) + ((K + r + 8) * 2.0 ** -23 + 2.0 ** -16) * mag + 1e-30) & there[:, None]
    assert not bad.any(), (np.argwhere(bad)[:5], err[bad][:5], want[bad][:5])
    if before is not None:
        keep = torch.from_numpy(~there)
        assert torch.equal(got.cpu()[keep], before[keep])


def call(d, row_start, used, **kw):
    iq = _iq()
    g = {k: v.cuda() for k, v in d.items()}
    kw = {"base": g["base"]} | kw
    return iq.adapters(g["x"], kw.pop("base"), g["a"], g["b"], g["scale"],
                       torch.tensor(np.asarray(row_start), dtype=torch.int32, device="cuda"),
                       torch.tensor(np.asarray(used), dtype=torch.int32, device="cuda"), **kw)


CASES = [
    # K, N, rank, adapters, lengths, adapter of each request
    (8, 8, 8, 1, [1], [0]),
    (64, 128, 16, 2, [1], [1]),
    (136, 72, 24, 3, [2, 1], [2, 0]),
    (256, 136, 64, 2, [17, 0, 16], [0, 1, 1]),
    (1536, 264, 16, 4, [1, 1, 1, 1, 1], [3, 3, -1, 0, 3]),
    (520, 520, 72, 2, [127, 129, 1], [1, 0, 0]),
    (1064, 1032, 128, 3, [5, 300, 0, 33], [0, 2, 1, -1]),
    (448, 2048, 40, 2, [128, 128, 128], [0, 0, 1]),
    (7168, 512, 32, 64, [1] * 64, [(7 * i) % 48 for i in range(64)]),
    (2048, 136, 8, 2, [900], [1]),
    (64, 64, 16, 9, [1, 0, 2] * 300, [(i // 3) % 10 - 1 for i in range(900)]),
    (64, 72, 8, 5, [(3 * i) % 4 for i in range(32)], [(i // 2) % 6 - 1 for i in range(32)]),
    (64, 72, 8, 5, [(3 * i) % 4 for i in range(33)], [(i // 2) % 6 - 1 for i in range(33)]),
    (64, 72, 8, 5, [(3 * i) % 4 for i in range(192)], [(i // 2) % 6 - 1 for i in range(192)]),
    (64, 72, 8, 5, [(3 * i) % 4 for i in range(193)], [(i // 2) % 6 - 1 for i in range(193)]),
    (64, 72, 8, 5, [(3 * i) % 4 for i in range(320)], [(i // 2) % 6 - 1 for i in range(320)]),
    (64, 72, 8, 5, [(3 * i) % 4 for i in range(321)], [(i // 2) % 6 - 1 for i in range(321)]),
    (64, 72, 8, 5, [(3 * i) % 4 for i in range(1024)], [(i // 2) % 6 - 1 for i in range(1024)]),
]


@pytest.mark.parametrize("K,N,r,A,lengths,used", CASES)
def test_adapters(cuda_device, K, N, r, A, lengths, used):
    rng = np.random.default_rng(K + N + r)
    start = np.concatenate([[0], np.cumsum(lengths)])
    d = inputs(rng, int(start[-1]), K, N, r, A)
    check(call(d, start, used), d, start, used)
    assert _iq().device_status() == 0


def test_adapters_without_base_and_in_place(cuda_device):
    rng = np.random.default_rng(1)
    d = inputs(rng, 70, 128, 96, 16, 3)
    start, used = [0, 30, 31, 70], [1, 7, 2]                    # 7: none
    check(call(d, start, used, base=None), d, start, used, use_base=False)
    acc = d["base"].cuda()
    got = call(d, start, used, base=acc, out=acc)
    assert got is acc
    check(got, d, start, used)


def test_adapters_rows_of_no_request_and_wider_tensors(cuda_device):
    rng = np.random.default_rng(2)
    d = inputs(rng, 90, 136, 88, 24, 2)
    start, used = [7, 40, 40, 77], [1, 0, 0]
    wide = torch.full((90, 104), 5.0, dtype=torch.bfloat16)
    out = wide.cuda()
    x, base = torch.zeros((90, 200), dtype=torch.bfloat16), torch.zeros((90, 96), dtype=torch.bfloat16)
    x[:, 8:144], base[:, 8:] = d["x"], d["base"]
    iq = _iq()
    got = iq.adapters(x.cuda()[:, 8:144], base.cuda()[:, 8:], d["a"].cuda(), d["b"].cuda(), d["scale"].cuda(),
                      torch.tensor(start, dtype=torch.int32, device="cuda"),
                      torch.tensor(used, dtype=torch.int32, device="cuda"), out=out[:, 8:96])
    check(got, d, start, used, before=wide[:, 8:96])
    assert torch.equal(out[:, :8].cpu(), wide[:, :8]) and torch.equal(out[:, 96:].cpu(), wide[:, 96:])


@pytest.mark.parametrize("start", [[-5, 10, 400], [60, 20, 64], [0, 0, 0], [200, 300, 400], [0, 50, 0], [0, 64, 0]])
def test_adapters_row_start_outside_its_range(cuda_device, start):
    rng = np.random.default_rng(3)
    d = inputs(rng, 64, 128, 64, 16, 2)
    before = torch.full((64, 64), 9.0, dtype=torch.bfloat16)
    check(call(d, start, [0, 1], out=before.cuda()), d, start, [0, 1], before=before)


def test_adapters_on_another_stream_and_in_a_graph(cuda_device):
    iq = _iq()
    rng = np.random.default_rng(4)
    d = inputs(rng, 40, 256, 128, 16, 2)
    start, used = [0, 1, 40], [0, 1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(d, start, used, stream=side)
    side.synchronize()
    check(got, d, start, used)
    g = {k: v.cuda() for k, v in d.items()}
    rs, ad = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (start, used))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = iq.adapters(g["x"], g["base"], g["a"], g["b"], g["scale"], rs, ad)
    d["x"] = bf16(rng, (40, 256))
    g["x"].copy_(d["x"])
    ad.copy_(torch.tensor([1, -1]))
    graph.replay()
    torch.cuda.synchronize()
    check(out, d, start, [1, -1])
    assert iq.device_status() == 0


def test_adapters_beside_a_shared_projection(cuda_device):
    """Quantise, project with one shared weight, add the requests' adapters."""
    iq = _iq()
    rng = np.random.default_rng(5)
    T, K, N = 50, 512, 256
    d = inputs(rng, T, K, N, 32, 3)
    w = torch.from_numpy(rng.integers(0, 0x70, (1, N, K)).astype(np.uint8)).cuda()
    w_sf = torch.full((1, 2, 4), 110, dtype=torch.uint8, device="cuda")
    whole = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    xq, xs = iq.fp8_quant_1x128_ue8m0(d["x"].cuda())
    d["base"] = iq.grouped_gemm(xq, xs, w, w_sf, whole).cpu()
    start, used = [0, 20, 21, 50], [2, -1, 0]
    check(call(d, start, used), d, start, used)


def test_adapters_of_rows_given_to_many_requests(cuda_device):
    """A row_start that falls again and again: a row belongs to the first request
    that has it, and the parts' place in the workspace is that of the rows."""
    rng = np.random.default_rng(6)
    d = inputs(rng, 64, 128, 64, 16, 3)
    start, used = [0, 40] + [0, 64] * 200, [i % 3 for i in range(401)]
    check(call(d, start, used), d, start, used)
    assert _iq().device_status() == 0


def test_adapters_nan_stays_where_it_is(cuda_device):
    """NaN in rows of no request, in rows of another request, behind a row's end
    and in adapters that nobody uses."""
    rng = np.random.default_rng(7)
    T, K, N, r = 60, 136, 88, 24
    d = inputs(rng, T, K, N, r, 3)
    start, used = [2, 20, 33, 34, 50], [1, 0, -1, 0]
    wide = torch.full((T, K + 56), float("nan"), dtype=torch.bfloat16)
    wide[:, :K] = d["x"]
    for t in (d["a"], d["b"], d["scale"]):
        t[2] = float("nan")
    poisoned = list(range(2)) + list(range(50, T)) + [25, 33]    # 25: of the request of adapter 0; 33: without
    wide[poisoned] = float("nan")
    d["base"][poisoned[:-1]] = float("nan")
    g = {k: v.cuda() for k, v in d.items()}
    got = _iq().adapters(wide.cuda()[:, :K], g["base"], g["a"], g["b"], g["scale"],
                         *(torch.tensor(v, dtype=torch.int32, device="cuda") for v in (start, used)))
    assert torch.isnan(got[25]).all() and torch.equal(got[33].cpu(), d["base"][33])
    keep = [t for t in range(2, 50) if t != 25]
    clean = {**d, "base": torch.where(torch.isnan(d["base"]), torch.zeros_like(d["base"]), d["base"])}
    clean["x"] = d["x"].clone()
    for name in ("a", "b", "scale"):
        clean[name] = torch.nan_to_num(d[name])
    want, mag, _ = X.adapters(f64(clean["x"]), f64(clean["base"]), f64(clean["a"]), f64(clean["b"]), clean["scale"].numpy(), start, used)
    bound = 2.0 ** -8 * np.abs(want) + ((K + r + 8) * 2.0 ** -23 + 2.0 ** -16) * mag + 1e-30
    assert np.all((np.abs(f64(got) - want) <= bound)[keep])


def test_adapters_on_two_streams_at_once(cuda_device):
    iq = _iq()
    rng = np.random.default_rng(8)
    d = inputs(rng, 300, 1536, 1032, 64, 4)
    g = {k: v.cuda() for k, v in d.items()}
    cases = [([0, 100, 101, 300], [0, 1, 2]), ([0, 3, 290, 300], [3, 3, 1])]
    ints = [[torch.tensor(v, dtype=torch.int32, device="cuda") for v in c] for c in cases]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            outs[i].append(iq.adapters(g["x"], g["base"], g["a"], g["b"], g["scale"], *ints[i], stream=s))
    torch.cuda.synchronize()
    for i, (start, used) in enumerate(cases):
        check(outs[i][0], d, start, used)
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])
    assert iq.device_status() == 0


def test_adapters_offsets_past_32_bits(cuda_device):
    """Rows further than 2^32 bytes apart."""
    rng = np.random.default_rng(9)
    T, K, N, far = 40, 136, 136, 1 << 26
    d = inputs(rng, T, K, N, 16, 2)
    x, base, out = (torch.empty((T * far,), dtype=torch.bfloat16, device="cuda").view(T, far)[:, :136] for _ in range(3))
    x.copy_(d["x"].cuda())
    base.copy_(d["base"].cuda())
    start, used = [0, 39, 40], [1, 0]
    g = {k: v.cuda() for k, v in d.items()}
    got = _iq().adapters(x, base, g["a"], g["b"], g["scale"], *(torch.tensor(v, dtype=torch.int32, device="cuda") for v in (start, used)), out=out)
    check(got.contiguous(), d, start, used)


def whole_numbers(rng, lengths, K, N, r, A):
    """Inputs whose every sum is a whole number: A x has 24 significant bits (three
    digits of 2^16, 2^8 and 1 in each row of A, at places anywhere along K, and small
    numbers elsewhere that cancel), neighbouring rows of A differ by a few units, and
    B takes their differences, so that what is left of the 24 bits is a number that
    BF16 holds.  base cancels part of it."""
    T = int(sum(lengths))
    place = rng.permutation(K)
    digits, rest = place[:3], place[3:]
    a = np.zeros((A, r, K))
    half = rest[:len(rest) // 2 * 2].reshape(-1, 2)
    small = rng.integers(-3, 4, (A, r, len(half)))
    a[:, :, half[:, 0]], a[:, :, half[:, 1]] = small, -small
    pairs = r // 2
    for i, low in ((0, 64), (1, 128), (2, 110)):             # below 2^23
        a[:, 0::2, digits[i]] = rng.integers(-low, low + 1, (A, pairs))
        a[:, 1::2, digits[i]] = a[:, 0::2, digits[i]]
    a[:, 1::2, digits[2]] += rng.integers(-9, 10, (A, pairs))
    x = np.ones((T, K))
    x[:, digits] = [2.0 ** 16, 2.0 ** 8, 1.0]
    x *= rng.choice([1.0, -1.0, 0.5], (T, 1))
    b = np.zeros((A, N, r))
    pick = rng.integers(-1, 2, (A, N, pairs)) * (rng.random((A, N, pairs)) < 4 / pairs)
    b[:, :, 0::2], b[:, :, 1::2] = pick, -pick
    base = rng.integers(-20, 21, (T, N))
    to = lambda v: torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)
    d = dict(x=to(x), base=to(base), a=to(a), b=to(b), scale=torch.from_numpy(rng.choice([1.0, -1.0, 2.0], A).astype(np.float32)))
    assert all(np.array_equal(f64(d[k]), v) for k, v in (("x", x), ("base", base), ("a", a), ("b", b)))
    return d


EXACT = [
    (8, 8, 8, 1, [1], [0]),
    (520, 136, 24, 3, [5, 0, 33, 16], [2, 1, 0, 2]),
    (1536, 264, 16, 4, [1, 1, 1, 1, 1], [3, 3, -1, 0, 3]),
    (1536, 520, 64, 2, [127, 129, 1], [1, 0, 0]),
    (1064, 1032, 128, 3, [5, 300, 0, 33], [0, 2, 1, -1]),
    (2048, 256, 72, 40, [1] * 40, list(range(40))),
]


@pytest.mark.parametrize("K,N,r,A,lengths,used", EXACT)
def test_adapters_keep_all_bits_of_a_x(cuda_device, K, N, r, A, lengths, used):
    """Float32 sums of these inputs are exact, so nothing but the rounding to BF16 may
    show; of A x held in 16 bits most results are off by whole numbers."""
    rng = np.random.default_rng(K + r)
    d = whole_numbers(rng, lengths, K, N, r, A)
    start = np.concatenate([[0], np.cumsum(lengths)])
    want, _, _ = X.adapters(f64(d["x"]), f64(d["base"]), f64(d["a"]), f64(d["b"]), d["scale"].numpy(), start, used)
    got = call(d, start, used)
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))
    assert _iq().device_status() == 0


def test_adapters_infinities(cuda_device):
    """What the definition gives: an infinite A x is an infinity, or NaN where B
    makes both signs or a zero of it, in its own row alone; a value beyond the largest
    BF16 counts in full; neither depends on the rank's padding."""
    inf = float("inf")
    T, K, N, r = 7, 72, 40, 8
    rng = np.random.default_rng(10)
    d = inputs(rng, T, K, N, r, 2)
    d["scale"] = torch.tensor([1.0, -1.0])
    d["x"][:, :2] = 0                                          # places 0 and 1 of x make row values of their own
    d["a"][:, :, 0] = d["a"][:, 1::2, 1] = 1
    d["a"][:, 0::2, 1] = -1
    d["b"][:, 8:16] = d["b"][:, 8:16].abs()
    d["b"][:, 24:32, 0::2], d["b"][:, 24:32, 1::2] = d["b"][:, 24:32, 0::2].abs(), -d["b"][:, 24:32, 1::2].abs()
    d["b"][:, 16, 3] = 0
    d["x"][1, 0], d["x"][2, 0], d["x"][3, 1], d["x"][4, 1] = inf, -inf, inf, -inf
    d["x"][5] = 0
    d["x"][5, 0], d["x"][5, 1] = 2.0 ** 120 * 255, 2.0 ** 119   # their sum rounds to a BF16 infinity
    d["b"] *= 2.0 ** -20
    start, used = [0, 4, 7], [1, 0]
    with np.errstate(invalid="ignore"):
        want, mag, _ = X.adapters(f64(d["x"]), f64(d["base"]), f64(d["a"]), f64(d["b"]), d["scale"].numpy(), start, used)
    got = f64(call(d, start, used))
    plain = np.isfinite(want)
    assert np.isinf(want[1:5]).any(axis=1).all() and np.isnan(want[1:5]).any(axis=1).all() and plain[[0, 5, 6]].all()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    bound = 2.0 ** -8 * np.abs(want) + (K + r + 8) * 2.0 ** -23 * mag + 1e-30
    assert np.all(np.abs(got[plain] - want[plain]) <= bound[plain])


def test_adapters_sums_of_few_rows_are_not_one_long_chain(cuda_device):
    """Each addition of the MMA truncates, half a unit of the running sum on the mean, at
    most 2^-24 of it, so a sum of positive numbers is off to one side by up to n 2^-25
    after n MMAs.  64 tiles of 56 steps over 152 CTAs: runs of 24 steps, 192 MMAs, in
    four chains of 48.  (One chain of 192, emulated: 56 * 2^-24.)"""
    rng = np.random.default_rng(17)
    T, K, r = 64, 7168, 64
    pos = lambda *s: torch.from_numpy(rng.uniform(0.5, 1.5, s).astype(np.float32)).to(torch.bfloat16)
    d = dict(x=pos(T, K), a=pos(T, r, K) * 2.0 ** -12, b=torch.eye(r, dtype=torch.bfloat16).repeat(T, 1, 1), scale=torch.ones(T))
    v = np.einsum("tk,trk->tr", f64(d["x"]), f64(d["a"]))
    d["base"] = -torch.from_numpy(v).to(torch.bfloat16)         # what is left shows the sum's lower bits
    got = f64(call(d, np.arange(T + 1), np.arange(T)))
    off = (got - (v + f64(d["base"]))) / v
    assert abs(off.mean()) <= (48 + 2) * 2.0 ** -25 and np.abs(off).max() <= 2.0 ** -16
