"""Multi-token attention where it can go wrong: what must not reach a row, long
batches, references that move, bad inputs, captured calls, large pools.

The bounds are those of test_gpu_extend.py.
"""
import numpy as np
import pytest

from oracle.extend import visible
from paged_kv_cache_163_gb300 import workloads as wl

from test_gpu_extend import PAIRS, check, run
from test_gpu_gather import fill
from test_gpu_rope import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def capi():
    from paged_kv_cache_163_gb300 import capi as c
    c.load()
    return c


@pytest.fixture(scope="module")
def workspace(capi):
    return {d: torch.zeros(capi.paged_attention_extend_workspace_bytes(d), dtype=torch.uint8, device="cuda")
            for d in (64, 128)}


def poison(cache, tables, bs, tokens, b, cache_dtype, value, column=None):
    """Every KV head's K and V of some tokens of sequence b (of V only one column, when given)."""
    k, v, ks, vs = cache
    for t in tokens:
        blk, off = int(tables[b, t // bs]), t % bs
        if cache_dtype in ("f16", "bf16"):
            if column is None:
                k[blk, :, off] = value
                v[blk, :, off] = value
            else:
                v[blk, :, off, column] = value
        else:
            ks[blk, :, off] = value
            vs[blk, :, off] = value
            if cache_dtype.startswith("fp8"):
                k[blk, :, off].view(torch.uint8).fill_(0x7F)
                v[blk, :, off].view(torch.uint8).fill_(0x7F)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_dtype,cache_dtype", PAIRS)
@pytest.mark.parametrize("lens,news,hq,hkv,window,sinks,bad", [
    ([300], [170], 4, 2, 0, 0, [220, 221, 260]),            # ahead of the first rows
    ([700, 50], [5, 50], 8, 2, 100, 3, [3, 597, 698]),  # behind some windows, ahead of some rows; rows split
    ([5000], [300], 4, 1, 1000, 0, [3701, 3750, 4900]),      # an item over several CTAs
])
def test_invisible_values_do_not_reach_a_row(capi, workspace, value, d, q_dtype, cache_dtype, lens, news, hq, hkv,
                                             window, sinks, bad):
    bs = 16
    cache, tables, model = fill(capi, lens, hkv, d, q_dtype, cache_dtype, bs, 5)
    poison(cache, tables, bs, bad, 0, cache_dtype, value)
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    rng = np.random.default_rng(2)
    q = wl.round_to(rng.standard_normal((int(starts[-1]), hq, d)).astype(np.float32), q_dtype)
    scale = float(np.float32(1.0) / np.sqrt(np.float32(d)))
    o = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    capi.paged_attention_extend(o, dev(q, q_dtype), *cache, dev(tables), dev(np.array(lens, np.int32)), dev(starts),
                                scale, workspace[d], window=window, sinks=sinks, cache_dtype=cache_dtype)
    got = o.double().cpu().numpy()
    for b, (L, n) in enumerate(zip(lens, news)):
        K, V = model.gather(tables[b], L)
        see = visible(L, n, window, sinks)
        sees_bad = see[:, bad].any(1) if b == 0 else np.zeros(n, bool)
        assert not sees_bad.all() and (b or sees_bad.any())
        rows = got[starts[b]:starts[b + 1]]
        # a row that sees one: its score or its weighted value is no number
        assert np.all(~np.isfinite(rows[sees_bad]).all(-1))
        # the rest, run by run of rows so that the oracle's rows keep their positions
        for i in np.flatnonzero(~sees_bad)[::7]:
            check(rows[i:i + 1], q[starts[b] + i:starts[b] + i + 1], K[:L - n + i + 1], V[:L - n + i + 1], scale,
                  window, sinks, q_dtype, cache_dtype, False)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_an_infinite_element_stays_in_its_column(capi, workspace, dtype):
    """V holds one infinity: rows that see it have it in that column, the others' columns are the formula's."""
    cache, tables, model = fill(capi, [400], 2, 128, dtype, dtype, 16, 6)
    poison(cache, tables, 16, [250], 0, dtype, float("inf"), column=77)
    n, hq = 300, 4
    q = wl.round_to(np.random.default_rng(3).standard_normal((n, hq, 128)).astype(np.float32), dtype)
    o = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    capi.paged_attention_extend(o, dev(q, dtype), *cache, dev(tables), dev(np.array([400], np.int32)),
                                dev(np.array([0, n], np.int32)), 0.05, workspace[128], cache_dtype=dtype)
    got = o.double().cpu().numpy()
    K, V = model.gather(tables[0], 400)
    sees = np.arange(n) + 100 >= 250
    assert np.all(np.isposinf(got[sees][:, :, 77]))
    got[sees, :, 77] = 0.0
    V = V.copy()
    col = V[:, :, 77].copy()
    V[:, :, 77] = 0.0
    zeroed = got.copy()
    zeroed[:, :, 77] = 0.0
    check(zeroed, q, K, V, 0.05, 0, 0, dtype, dtype, False)
    V[:, :, 77] = col
    check(got[:150], q[:150], K[:250], V[:250], 0.05, 0, 0, dtype, dtype, False)


@pytest.mark.parametrize("q_dtype,cache_dtype", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "fp8_e4m3"), ("f16", "int8")])
@pytest.mark.parametrize("seqs,longest,hq,hkv,window", [(31, 400, 8, 2, 0), (32, 200, 4, 4, 60), (33, 300, 8, 1, 0),
                                                        (200, 90, 2, 1, 33), (1024, 40, 2, 2, 0)])
def test_many_sequences(capi, workspace, q_dtype, cache_dtype, seqs, longest, hq, hkv, window):
    rng = np.random.default_rng(seqs)
    lens = [int(x) for x in rng.integers(0, longest, seqs)]
    news = [int(min(L + 2, rng.choice([0, 1, 1, 1, 4, 37]))) for L in lens]
    run(capi, workspace, lens, news, hq, hkv, 64, q_dtype, cache_dtype, 16, window, 2 if window else 0, seed=seqs)


@pytest.mark.parametrize("q_dtype,cache_dtype", PAIRS)
def test_references_that_move(capi, workspace, q_dtype, cache_dtype):
    """Scores of many hundreds that grow along the sequence: references, sums and O change units again and again."""
    lens, news, hq, hkv, d, bs = [900, 600], [130, 3], 4, 2, 128, 16
    cache, tables, model = fill(capi, lens, hkv, d, q_dtype, cache_dtype, bs, 9)
    rng = np.random.default_rng(4)
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    q = wl.round_to(30 * rng.standard_normal((int(starts[-1]), hq, d)).astype(np.float32), q_dtype)
    # later tokens' keys are larger: the maximum moves step by step
    for b, L in enumerate(lens):
        p = np.arange(L)
        x = rng.standard_normal((2, L, hkv, d)).astype(np.float32)
        x[0] *= (p / 100 + 0.05)[:, None, None]
        x[1] *= np.exp2(rng.integers(-6, 6, (L, 1, 1)))
        x = wl.round_to(x.astype(np.float32), q_dtype)
        slots = (tables[b, p // bs] * bs + p % bs).astype(np.int32)
        capi.paged_kv_append(dev(x[0], q_dtype), dev(x[1], q_dtype), dev(slots), *cache, cache_dtype=cache_dtype)
        model.write(slots, x[0], x[1])
    for window in (0, 200):
        o = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
        capi.paged_attention_extend(o, dev(q, q_dtype), *cache, dev(tables), dev(np.array(lens, np.int32)),
                                    dev(starts), 0.3, workspace[d], window=window, cache_dtype=cache_dtype)
        got = o.double().cpu().numpy()
        for b, L in enumerate(lens):
            K, V = model.gather(tables[b], L)
            check(got[starts[b]:starts[b + 1]], q[starts[b]:starts[b + 1]], K, V, 0.3, window, 0, q_dtype, cache_dtype,
                  False)


@pytest.mark.parametrize("cache_dtype", ["bf16", "fp8_e4m3"])
def test_repeated_calls_give_the_same_bits(capi, workspace, cache_dtype):
    """Rows split over CTAs and tiles, read by atomically counted merges: no order of arrival shows."""
    for lens, news, hq, hkv in [([6000, 300, 2500], [1, 1, 4], 8, 2), ([4000, 900], [700, 300], 4, 1)]:
        cache, tables, _ = fill(capi, lens, hkv, 128, "bf16", cache_dtype, 16, 1)
        starts = dev(np.concatenate(([0], np.cumsum(news))).astype(np.int32))
        q = torch.randn((sum(news), hq, 128), device="cuda").bfloat16()
        n, t = dev(np.array(lens, np.int32)), dev(tables)
        first = None
        for _ in range(30):
            o = torch.zeros_like(q)
            capi.paged_attention_extend(o, q, *cache, t, n, starts, 0.09, workspace[128], cache_dtype=cache_dtype)
            first = o if first is None else first
            assert torch.equal(o, first)


@pytest.mark.parametrize("cache_dtype", ["bf16", "fp8_e4m3_int4"])
def test_bad_entries_are_reported_and_bounded(capi, workspace, cache_dtype):
    lens, news, hq, hkv, d, bs = [150, 90, 64], [20, 90, 3], 4, 2, 128, 16
    cache, tables, model = fill(capi, lens, hkv, d, "bf16", cache_dtype, bs, 8)
    q = wl.round_to(np.random.default_rng(8).standard_normal((sum(news), hq, d)).astype(np.float32), "bf16")
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(tables=tables, lens=lens, starts=starts, window=0):
        err.zero_()
        o = torch.full(q.shape, 7.0, device="cuda")
        capi.paged_attention_extend(o, dev(q, "bf16"), *cache, dev(tables), dev(np.array(lens, np.int32)), dev(starts),
                                    0.09, workspace[d], window=window, d_error=err, cache_dtype=cache_dtype)
        return o.double().cpu().numpy(), int(err.item())

    def others(got, bad):
        for b, (L, n) in enumerate(zip(lens, news)):
            if b != bad:
                rows = slice(starts[b], starts[b + 1])
                check(got[rows], q[rows], *model.gather(tables[b], L), 0.09, 0, 0, "bf16", cache_dtype, False)

    got, bits = call()
    assert bits == 0
    others(got, -1)
    for bad in (-5, len(model.k), 1 << 30):                 # a block id outside the pool
        t = tables.copy()
        t[1, 2] = bad
        got, bits = call(tables=t)
        assert bits == capi.DEVERR_BAD_BLOCK
        others(got, 1)
        K, V = (x.copy() for x in model.gather(tables[1], lens[1]))
        K[2 * bs:3 * bs] = 0
        V[2 * bs:3 * bs] = 0
        rows = slice(starts[1], starts[2])
        check(got[rows], q[rows], K, V, 0.09, 0, 0, "bf16", cache_dtype, False)
    for bad in (-1, tables.shape[1] * bs + 1, 2 ** 31 - 1):  # a length outside the table
        n = list(lens)
        n[0] = bad
        got, bits = call(lens=n)
        assert bits == capi.DEVERR_BAD_CONTEXT_LEN
        assert np.all(got[:news[0]] == 0.0)
        others(got, 0)
    for s in ([0, 20, 110, 114], [-1, 20, 110, 113], [0, 20, 2 ** 31 - 1, 113], [0, -2 ** 31, 110, 113]):
        got, bits = call(starts=np.array(s, np.int32))      # rows outside q
        assert bits == capi.DEVERR_BAD_CONTEXT_LEN
    got, bits = call()
    assert bits == 0
    others(got, -1)


@pytest.mark.parametrize("cache_dtype", ["f16", "fp8_e5m2"])
def test_captured_on_another_stream_and_replayed(capi, cache_dtype):
    """One graph of two calls on one workspace; lengths, tables and queries change between replays."""
    lens, hq, hkv, d, bs = [1500, 40, 777], 8, 2, 128, 16
    cache, tables, model = fill(capi, lens, hkv, d, "f16", cache_dtype, bs, 12)
    news = [4, 40, 100]
    ws = torch.zeros(capi.paged_attention_extend_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    q_d = torch.zeros((sum(news), hq, d), dtype=torch.float16, device="cuda")
    n_d, s_d, t_d = dev(np.array(lens, np.int32)), dev(starts), dev(tables)
    a, b = (torch.zeros(q_d.shape, device="cuda") for _ in range(2))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        def both():
            capi.paged_attention_extend(a, q_d, *cache, t_d, n_d, s_d, 0.1, ws, cache_dtype=cache_dtype)
            capi.paged_attention_extend(b, q_d, *cache, t_d, n_d, s_d, 0.1, ws, window=64, sinks=4,
                                        cache_dtype=cache_dtype)
        both()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            both()
        for trial, ls in enumerate((lens, [1400, 40, 700], [1, 39, 100], lens)):
            q = wl.round_to(np.random.default_rng(trial).standard_normal(q_d.shape).astype(np.float32), "f16")
            q_d.copy_(dev(q, "f16"))
            n_d.copy_(dev(np.array(ls, np.int32)))
            graph.replay()
            stream.synchronize()
            for o, window, sinks in ((a, 0, 0), (b, 64, 4)):
                got = o.double().cpu().numpy()
                for i, (L, n) in enumerate(zip(ls, news)):
                    skip = max(n - L, 0)
                    rows = slice(starts[i] + skip, starts[i + 1])
                    assert np.all(got[starts[i]:starts[i] + skip] == 0)
                    check(got[rows], q[rows], *model.gather(tables[i], L), 0.1, window, sinks, "f16", cache_dtype, False)


@pytest.mark.parametrize("q_dtype,cache_dtype", [("bf16", "bf16"), ("f16", "int8"), ("bf16", "fp8_e4m3_int4")])
def test_a_pool_beyond_32_bit_offsets(capi, workspace, q_dtype, cache_dtype):
    """Sequences at the end of a pool whose element offsets pass 2^32 (codes: their bytes pass 2^31)."""
    lens, news, hq, hkv, d, bs = [333, 70], [50, 1], 16, 8, 128, 16
    cache, tables, model = fill(capi, lens, hkv, d, q_dtype, cache_dtype, bs, 4)
    small = cache[0].shape[0]
    nb = (1 << 32) // (hkv * bs * d) + small if cache_dtype == "bf16" else (1 << 31) // (hkv * bs * d) + 2 * small
    big = []
    for x in cache[:2]:
        y = torch.empty((nb, *x.shape[1:]), dtype=x.dtype, device="cuda")
        y[nb - small:] = x
        big.append(y)
    if cache[2] is not None:
        both = torch.empty((nb, hkv, 2, bs), device="cuda")
        both[nb - small:, :, 0] = cache[2]
        both[nb - small:, :, 1] = cache[3]
        big += [both[:, :, 0], both[:, :, 1]]
    else:
        big += [None, None]
    q = wl.round_to(np.random.default_rng(1).standard_normal((sum(news), hq, d)).astype(np.float32), q_dtype)
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    o = torch.zeros(q.shape, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.paged_attention_extend(o, dev(q, q_dtype), *big, dev(np.where(tables >= 0, tables + nb - small, tables)),
                                dev(np.array(lens, np.int32)), dev(starts), 0.09, workspace[d], d_error=err,
                                cache_dtype=cache_dtype)
    assert int(err.item()) == 0
    got = o.double().cpu().numpy()
    for b, L in enumerate(lens):
        rows = slice(starts[b], starts[b + 1])
        check(got[rows], q[rows], *model.gather(tables[b], L), 0.09, 0, 0, q_dtype, cache_dtype, False)
