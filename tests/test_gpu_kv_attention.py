"""The attention over the 8-bit cache against the oracle, with the bound of
tests/kv_cases.py."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from tests.kv_cases import attention_bound, bf16, dev, gaussian_cache, make_batch, make_cache

pytestmark = pytest.mark.gpu


def _iq():
    from fp4_fp8_quant_gb300 import iq
    return iq


def _gpu_cache(kc, vc):
    return _iq().KVCache(dev(kc["codes"]), dev(vc["codes"]), dev(kc["sf"]), dev(vc["sf"]))


def _check(got, kc, vc, q, batch, scale, indices=None):
    out, mag, top, dot = K.attention(kc, vc, q, batch, scale, indices)
    err = np.abs(got.double().cpu().numpy() - out)
    bound = attention_bound(out, mag, top, dot)
    worst = np.unravel_index(np.argmax(err / bound), err.shape)
    assert np.all(err <= bound), f"at {worst}: error {err[worst]:.3g}, allowed {bound[worst]:.3g}, exact {out[worst]:.3g}"
    assert _iq().device_status() == 0


def _indices(rng, batch, k, lists="random"):
    """Positions per row in any order, some of them invalid."""
    T = int(batch[1][-1])
    idx = np.full((T, k), -1, np.int32)
    for t, b, pos in K.rows_of(batch):
        if lists == "empty" and t % 2 == 0:
            continue
        n = min(k, max(pos + 1, 0))
        pick = rng.permutation(max(pos + 1, 0))[:n]
        if lists == "sorted":
            idx[t, :n] = np.sort(pick)
        else:
            idx[t, rng.permutation(k)[:n]] = pick
            if n < k:                                    # a position the row may not see
                idx[t, np.argmax(idx[t] < 0)] = pos + 1 + int(rng.integers(0, 1000))
    return idx


BATCHES = [
    ([1], [1]),                                           # one token, one key
    ([1, 1, 1, 1], [1, 127, 128, 129]),                   # decode around a tile
    ([1, 0, 1], [700, 5, 16]),                            # a sequence without rows
    ([3, 2, 1], [3, 2, 300]),                             # short prompts
    ([37, 130], [200, 130]),                              # chunks, one behind a prefix
    ([5], [3]),                                           # more rows than positions: two rows see nothing
]


@pytest.mark.parametrize("new,kv_len", BATCHES)
@pytest.mark.parametrize("H,G,page,D", [(1, 1, 16, 128), (2, 8, 64, 128), (1, 64, 64, 128), (3, 5, 32, 64),
                                        (2, 16, 128, 64), (1, 100, 16, 64), (1, 33, 128, 128)])
def test_attention_matches_oracle(cuda_device, new, kv_len, H, G, page, D):
    rng = np.random.default_rng(len(new) * 100 + H * G)
    batch, P = make_batch(rng, new, kv_len, page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    q, qt = bf16(rng, (int(batch[1][-1]), H * G, D), 2.0)
    got = _iq().kv_attention(_gpu_cache(kc, vc), dev(qt), *map(dev, batch))
    _check(got, kc, vc, q, batch, D ** -0.5)


@pytest.mark.parametrize("new,kv_len", BATCHES)
@pytest.mark.parametrize("H,G,page,D,k,lists", [(1, 64, 64, 128, 128, "sorted"), (1, 8, 16, 128, 1, "random"),
                                                (2, 16, 128, 64, 37, "random"), (1, 64, 32, 128, 300, "empty"),
                                                (1, 3, 64, 64, 129, "sorted")])
def test_attention_over_selected_keys_matches_oracle(cuda_device, new, kv_len, H, G, page, D, k, lists):
    rng = np.random.default_rng(len(new) * 100 + H * G + k)
    batch, P = make_batch(rng, new, kv_len, page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    q, qt = bf16(rng, (int(batch[1][-1]), H * G, D), 2.0)
    idx = _indices(rng, batch, k, lists)
    got = _iq().kv_attention_topk(_gpu_cache(kc, vc), dev(qt), dev(idx), *map(dev, batch))
    _check(got, kc, vc, q, batch, D ** -0.5, idx)


@pytest.mark.parametrize("D", [64, 128])
def test_all_code_magnitudes_and_scales(cuda_device, D):
    """Codes of every magnitude under scales spread over 2^7 within a sequence;
    query rows that differ by 2^20 in magnitude."""
    rng = np.random.default_rng(D)
    page, H, G = 16, 2, 6
    batch, P = make_batch(rng, [1, 9], [333, 140], page)
    kc, vc = make_cache(rng, P, H, page, D, 112, 119), make_cache(rng, P, H, page, D, 108, 130)
    q, qt = bf16(rng, (10, H * G, D), np.exp2(rng.integers(-22, -1, (10, H * G, 1)).astype(float)))
    got = _iq().kv_attention(_gpu_cache(kc, vc), dev(qt), *map(dev, batch))
    _check(got, kc, vc, q, batch, D ** -0.5)


def test_sharp_and_flat_softmax(cuda_device):
    """One key far ahead of all others late in the row (the running maximum
    jumps), and rows without any preference."""
    rng = np.random.default_rng(4)
    page, H, G, D, n = 64, 1, 4, 128, 1500
    batch, P = make_batch(rng, [2], [n], page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    q, qt = bf16(rng, (2, G, D), 2.0)
    K1, _ = K.gather(kc, batch[0], 0, np.array([1300, 20]))
    qt[0, 1] = torch.from_numpy(K1[0, 0] * 20).to(torch.bfloat16)
    qt[0, 2] = torch.from_numpy(K1[1, 0] * 20).to(torch.bfloat16)
    qt[1, 0] = 0
    q = qt.to(torch.float64).numpy()
    got = _iq().kv_attention(_gpu_cache(kc, vc), dev(qt), *map(dev, batch))
    _check(got, kc, vc, q, batch, D ** -0.5)


@pytest.mark.parametrize("scale", [0.0, 1e-3, -0.1, 3.0])
def test_scales(cuda_device, scale):
    rng = np.random.default_rng(11)
    batch, P = make_batch(rng, [4], [260], 64)
    kc, vc = gaussian_cache(rng, P, 2, 64, 128), gaussian_cache(rng, P, 2, 64, 128)
    q, qt = bf16(rng, (4, 6, 128))
    got = _iq().kv_attention(_gpu_cache(kc, vc), dev(qt), *map(dev, batch), scale=scale)
    _check(got, kc, vc, q, batch, scale)


def test_bytes_behind_the_sequence_do_not_matter(cuda_device):
    """Slots past kv_len and unused pages hold NaN codes, their scales 255, and
    the table's unused entries are outside the pool."""
    rng = np.random.default_rng(12)
    page, H, G, D = 64, 2, 8, 128
    new, kv_len = [1, 3, 20], [130, 67, 20]
    batch, P = make_batch(rng, new, kv_len, page)
    batch[0][batch[0] < 0] = 1 << 30
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    used = np.zeros((P, page), bool)
    for b, n in enumerate(kv_len):
        for s in range(n):
            used[batch[0][b, s // page], s % page] = True
    for c in (kc, vc):
        c["codes"] = np.where(used[:, None, :, None], c["codes"], np.uint8(0x7F))
        c["sf"] = np.where(used.any(axis=1)[:, None], c["sf"], np.uint8(255))
    q, qt = bf16(rng, (24, H * G, D), 2.0)
    cache = _gpu_cache(kc, vc)
    _check(_iq().kv_attention(cache, dev(qt), *map(dev, batch)), kc, vc, q, batch, D ** -0.5)
    idx = _indices(rng, batch, 150)
    _check(_iq().kv_attention_topk(cache, dev(qt), dev(idx), *map(dev, batch)), kc, vc, q, batch, D ** -0.5, idx)


def test_pages_outside_the_pool_are_not_seen(cuda_device):
    rng = np.random.default_rng(13)
    page, H, G, D = 16, 1, 8, 64
    batch, P = make_batch(rng, [2, 4], [200, 90], page)
    batch[0][0, 3], batch[0][0, 7], batch[0][1, 0] = -7, P, 1 << 30
    batch = (np.ascontiguousarray(batch[0][:, :12]), batch[1], batch[2])     # positions 192.. have no entry
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    q, qt = bf16(rng, (6, H * G, D), 2.0)
    cache = _gpu_cache(kc, vc)
    _check(_iq().kv_attention(cache, dev(qt), *map(dev, batch)), kc, vc, q, batch, D ** -0.5)
    idx = _indices(rng, batch, 60)
    _check(_iq().kv_attention_topk(cache, dev(qt), dev(idx), *map(dev, batch)), kc, vc, q, batch, D ** -0.5, idx)


def test_strided_rows(cuda_device):
    """q as a slice of a wider projection, out as rows of a wider tensor whose
    other columns stay as they are, indices and table with row strides."""
    rng = np.random.default_rng(14)
    page, H, G, D, T = 64, 2, 4, 128, 9
    batch, P = make_batch(rng, [T], [300], page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    f, ft = bf16(rng, (T, 3 * H * G, D))
    fd = dev(ft)
    out = torch.full((T, 2 * H * G, D), 5.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.full((1, batch[0].shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :-3] = dev(batch[0])
    cache = _gpu_cache(kc, vc)
    sl = slice(H * G, 2 * H * G)
    _iq().kv_attention(cache, fd[:, sl], wide[:, :-3], dev(batch[1]), dev(batch[2]), out=out[:, sl])
    _check(out[:, sl], kc, vc, f[:, sl], batch, D ** -0.5)
    assert torch.all(out[:, :H * G] == 5.0)
    idx = _indices(rng, batch, 40)
    wi = torch.full((T, 47), 3, dtype=torch.int32, device="cuda")
    wi[:, :40] = dev(idx)
    got = _iq().kv_attention_topk(cache, fd[:, sl], wi[:, :40], wide[:, :-3], dev(batch[1]), dev(batch[2]))
    _check(got, kc, vc, f[:, sl], batch, D ** -0.5, idx)


def test_long_sequence_is_split_and_joined(cuda_device):
    """20011 keys, one row: the long axis is worked on by many blocks."""
    rng = np.random.default_rng(15)
    page, H, G, D, n = 128, 1, 8, 128, 20011
    batch, P = make_batch(rng, [1], [n], page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    q, qt = bf16(rng, (1, G, D), 2.0)
    got = _iq().kv_attention(_gpu_cache(kc, vc), dev(qt), *map(dev, batch))
    _check(got, kc, vc, q, batch, D ** -0.5)


def test_offsets_past_32_bits(cuda_device):
    """Pages more than 2^32 bytes into the pool."""
    rng = np.random.default_rng(16)
    page, D, H, G = 128, 128, 8, 4
    P = (1 << 32) // (H * page * D) + 4
    small = gaussian_cache(rng, 3, H, page, D), gaussian_cache(rng, 3, H, page, D)
    cache = _iq().KVCache.empty(P, H, page, D)
    cache.k_codes[P - 3:] = dev(small[0]["codes"])
    cache.v_codes[P - 3:] = dev(small[1]["codes"])
    cache.k_sf[P - 3:] = dev(small[0]["sf"])
    cache.v_sf[P - 3:] = dev(small[1]["sf"])
    q, qt = bf16(rng, (2, H * G, D), 2.0)
    sb = (np.array([[2, 0, 1]], np.int32), np.array([0, 2], np.int32), np.array([301], np.int32))
    batch = (sb[0] + P - 3, sb[1], sb[2])
    got = _iq().kv_attention(cache, dev(qt), *map(dev, batch))
    _check(got, *small, q, sb, D ** -0.5)
    idx = _indices(rng, sb, 200)
    got = _iq().kv_attention_topk(cache, dev(qt), dev(idx), *map(dev, batch))
    _check(got, *small, q, sb, D ** -0.5, idx)


def _larger_case():
    rng = np.random.default_rng(17)
    page, H, G, D = 64, 4, 8, 128
    batch, P = make_batch(rng, [1, 300, 1, 64], [4000, 900, 33, 1500], page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    _, qt = bf16(rng, (366, H * G, D), 2.0)
    idx = _indices(rng, batch, 500, "sorted")
    return _gpu_cache(kc, vc), dev(qt), dev(idx), [dev(a) for a in batch]


def test_same_bits_every_time_and_with_any_workspace_contents(cuda_device):
    cache, q, idx, batch = _larger_case()
    need = _iq().kv_attention_workspace_bytes(q.shape[0], q.shape[1], cache.kv_heads, cache.head_dim)
    first = _iq().kv_attention(cache, q, *batch), _iq().kv_attention_topk(cache, q, idx, *batch)
    for fill in (0, 0xFF, 0x5A):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(_iq().kv_attention(cache, q, *batch, workspace=ws), first[0])
        assert torch.equal(_iq().kv_attention_topk(cache, q, idx, *batch, workspace=ws), first[1])


def test_in_a_graph_and_on_other_streams(cuda_device):
    """Captured calls give the same bits, also after the lengths grow; the
    workspace of a call on a side stream is not handed out again too early."""
    cache, q, idx, batch = _larger_case()
    want = _iq().kv_attention(cache, q, *batch), _iq().kv_attention_topk(cache, q, idx, *batch)
    need = _iq().kv_attention_workspace_bytes(q.shape[0], q.shape[1], cache.kv_heads, cache.head_dim)
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    length = batch[2].clone()
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            _iq().kv_attention(cache, q, batch[0], batch[1], length, out=out, workspace=ws)
    length.copy_(torch.clamp(length - 5, min=1))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _iq().kv_attention(cache, q, batch[0], batch[1], length))
    length.copy_(batch[2])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    st.wait_stream(torch.cuda.current_stream())
    results = []
    for _ in range(5):
        results.append(_iq().kv_attention(cache, q, *batch, stream=st))
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xFF)     # the current stream's allocations
        results.append(_iq().kv_attention_topk(cache, q, idx, *batch, stream=st))
    torch.cuda.synchronize()
    for i, r in enumerate(results):
        assert torch.equal(r, want[i % 2])


def test_write_attend_chain_without_synchronisation(cuda_device):
    """Decode steps: write the new token, attend, on one stream; every step's
    result against the oracle."""
    rng = np.random.default_rng(18)
    page, H, G, D, B, steps = 16, 2, 8, 128, 3, 6
    (table, _, _), P = make_batch(rng, [1] * B, [60, 33, 16 + steps], page)
    kc, vc = gaussian_cache(rng, P, H, page, D), gaussian_cache(rng, P, H, page, D)
    cache, tab, rs = _gpu_cache(kc, vc), dev(table), dev(np.arange(B + 1, dtype=np.int32))
    todo = []
    for i in range(steps):
        n = np.array([60, 33, 16 + steps], np.int32) - steps + 1 + i
        k, kt = bf16(rng, (B, H, D), 1.0 + i)
        v, vt = bf16(rng, (B, H, D), 1.0 + i)
        q, qt = bf16(rng, (B, H * G, D))
        todo.append((n, k, v, q, dev(kt), dev(vt), dev(qt), dev(n)))
    torch.cuda.synchronize()
    outs = []
    for n, k, v, q, kd, vd, qd, nd in todo:
        _iq().kv_cache_write(cache, kd, vd, tab, rs, nd)
        outs.append(_iq().kv_attention(cache, qd, tab, rs, nd))
    for (n, k, v, q, *_), got in zip(todo, outs):
        batch = (table, np.arange(B + 1), n)
        kc, vc = K.write(kc, k, batch), K.write(vc, v, batch)
        _check(got, kc, vc, q, batch, D ** -0.5)


def test_indexer_selection_to_attention(cuda_device):
    """The indexer's scores and top-k feed the sparse attention: the whole
    selection path of a small causal prompt."""
    from fp4_fp8_quant_gb300 import workloads as W
    iq = _iq()
    rng = np.random.default_rng(19)
    T, k, page, G, D = 150, 64, 64, 16, 128
    batch, P = make_batch(rng, [T], [T], page)
    kc, vc = gaussian_cache(rng, P, 1, page, D), gaussian_cache(rng, P, 1, page, D)
    q, qt = bf16(rng, (T, G, D), 2.0)
    arrays = [dev(a) for a in W.indexer_inputs(T, T, seed=3, causal=True)]
    logits = iq.indexer_logits(*arrays)
    idx = iq.indexer_topk(logits, arrays[5], k)
    got = iq.kv_attention_topk(_gpu_cache(kc, vc), dev(qt), idx, *map(dev, batch))
    _check(got, kc, vc, q, batch, D ** -0.5, idx.cpu().numpy())
