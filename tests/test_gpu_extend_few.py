"""Multi-token attention with few query rows a KV head: single and drafted tokens.

Batches whose average is few rows run on a kernel of their own, whatever the
single sequences bring.  Bounds as in test_gpu_extend.py.
"""
import numpy as np
import pytest

from oracle.extend import visible
from paged_kv_cache_163_gb300 import workloads as wl

from test_gpu_extend import PAIRS, check, run
from test_gpu_extend_edges import poison
from test_gpu_gather import fill
from test_gpu_rope import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from paged_kv_cache_163_gb300 import capi as c
    c.load()
    return c


@pytest.fixture(scope="module")
def workspace(capi):
    return {d: torch.zeros(capi.paged_attention_extend_workspace_bytes(d), dtype=torch.uint8, device="cuda")
            for d in (64, 128)}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_dtype,cache_dtype", PAIRS)
@pytest.mark.parametrize("lens,news,hq,hkv,bs,window,sinks", [
    ([900, 17, 16, 15, 1, 0, 130], [1, 1, 1, 1, 1, 1, 1], 8, 2, 16, 0, 0),      # single tokens
    ([260, 500, 33], [5, 1, 8], 8, 2, 16, 0, 0),                                # drafted ones, 32 rows at most
    ([400, 129], [1, 1], 16, 1, 32, 0, 0),                                      # 16 heads a KV head
    ([100 + 7 * i for i in range(31)] + [150], [1] * 31 + [100], 2, 2, 16, 0, 0),  # and a prompt: rows in many passes
    ([300 - 6 * i for i in range(40)], [1] * 39 + [9], 4, 4, 16, 70, 5),        # more than 32 sequences
    ([2, 3, 0, 40], [4, 3, 2, 1], 2, 1, 32, 0, 0),                              # more queries than tokens
    ([1000, 800], [1, 2], 4, 1, 16, 1, 0),                                      # nothing but itself
    ([1000, 90], [2, 2], 4, 2, 16, 33, 20),
])
def test_few_rows(capi, workspace, d, q_dtype, cache_dtype, lens, news, hq, hkv, bs, window, sinks):
    run(capi, workspace, lens, news, hq, hkv, d, q_dtype, cache_dtype, bs, window, sinks, seed=len(lens) + d)


@pytest.mark.parametrize("q_dtype,cache_dtype", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "fp8_e4m3"), ("f16", "int8"),
                                                 ("f16", "fp8_e4m3_int4"), ("bf16", "fp8_e5m2")])
@pytest.mark.parametrize("lens,news,hq,hkv", [([20000], [1], 4, 1), ([7000, 100], [2, 2], 4, 1), ([9000, 9000, 3000], [1, 1, 1], 8, 4)])
def test_few_rows_of_long_contexts(capi, workspace, q_dtype, cache_dtype, lens, news, hq, hkv):
    """Items cut over many CTAs, and whole ones; the same bits every time."""
    o = run(capi, workspace, lens, news, hq, hkv, 128, q_dtype, cache_dtype, 16, 0, 0, "32", seed=11)
    for _ in range(3):
        assert torch.equal(o, run(capi, workspace, lens, news, hq, hkv, 128, q_dtype, cache_dtype, 16, 0, 0, "32", seed=11))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_dtype,cache_dtype", PAIRS)
def test_invisible_values_do_not_reach_few_rows(capi, workspace, value, d, q_dtype, cache_dtype):
    lens, news, hq, hkv, window, sinks, bs = [700, 300, 40], [4, 1, 1], 4, 2, 100, 3, 16
    bad = [3, 500, 597, 698]              # of the first sequence: seen by none, none, its first row, its last two
    cache, tables, model = fill(capi, lens, hkv, d, q_dtype, cache_dtype, bs, 15)
    poison(cache, tables, bs, bad, 0, cache_dtype, value)
    poison(cache, tables, bs, [4, 150, 199], 1, cache_dtype, value)   # its row sees 0 .. 2 and 200 .. 299
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    q = wl.round_to(np.random.default_rng(2).standard_normal((int(starts[-1]), hq, d)).astype(np.float32), q_dtype)
    o = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    capi.paged_attention_extend(o, dev(q, q_dtype), *cache, dev(tables), dev(np.array(lens, np.int32)), dev(starts),
                                0.1, workspace[d], window=window, sinks=sinks, cache_dtype=cache_dtype)
    got = o.double().cpu().numpy()
    for b, (L, n) in enumerate(zip(lens, news)):
        K, V = model.gather(tables[b], L)
        sees_bad = visible(L, n, window, sinks)[:, bad].any(1) if b == 0 else np.zeros(n, bool)
        for i in range(n):
            row = slice(starts[b] + i, starts[b] + i + 1)
            if sees_bad[i]:
                assert not np.isfinite(got[row]).any()
            else:
                end = L - n + i + 1
                check(got[row], q[row], K[:end], V[:end], 0.1, window, sinks, q_dtype, cache_dtype, False)
        assert b or list(sees_bad) == [True, False, True, True]


@pytest.mark.parametrize("q_dtype,cache_dtype", PAIRS)
def test_few_rows_with_references_that_move(capi, workspace, q_dtype, cache_dtype):
    """Scores of hundreds that grow along the sequence, V scales over twelve binades."""
    lens, news, hq, hkv, d, bs = [900, 600], [3, 1], 4, 2, 128, 16
    cache, tables, model = fill(capi, lens, hkv, d, q_dtype, cache_dtype, bs, 9)
    rng = np.random.default_rng(4)
    q = wl.round_to(30 * rng.standard_normal((4, hq, d)).astype(np.float32), q_dtype)
    for b, L in enumerate(lens):
        p = np.arange(L)
        x = rng.standard_normal((2, L, hkv, d)).astype(np.float32)
        x[0] *= (p / 100 + 0.05)[:, None, None]
        x[1] *= np.exp2(rng.integers(-6, 6, (L, 1, 1)))
        x = wl.round_to(x.astype(np.float32), q_dtype)
        slots = (tables[b, p // bs] * bs + p % bs).astype(np.int32)
        capi.paged_kv_append(dev(x[0], q_dtype), dev(x[1], q_dtype), dev(slots), *cache, cache_dtype=cache_dtype)
        model.write(slots, x[0], x[1])
    o = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    capi.paged_attention_extend(o, dev(q, q_dtype), *cache, dev(tables), dev(np.array(lens, np.int32)),
                                dev(np.array([0, 3, 4], np.int32)), 0.3, workspace[d], cache_dtype=cache_dtype)
    got = o.double().cpu().numpy()
    check(got[:3], q[:3], *model.gather(tables[0], lens[0]), 0.3, 0, 0, q_dtype, cache_dtype, False)
    check(got[3:], q[3:], *model.gather(tables[1], lens[1]), 0.3, 0, 0, q_dtype, cache_dtype, False)


@pytest.mark.parametrize("q_dtype,cache_dtype", [("bf16", "bf16"), ("f16", "fp8_e4m3")])
def test_one_token_is_what_decode_computes(capi, workspace, q_dtype, cache_dtype):
    """The single-token form and the decode call lie within the same bound of the same formula."""
    lens, hq, hkv, d = [1500, 33, 400], 8, 2, 128
    cache, tables, model = fill(capi, lens, hkv, d, q_dtype, cache_dtype, 16, 21)
    x = wl.round_to(np.random.default_rng(7).standard_normal((3, hq, d)).astype(np.float32), q_dtype)
    q = dev(x, q_dtype)
    one, ref = (torch.zeros(q.shape, device="cuda") for _ in range(2))
    n, t = dev(np.array(lens, np.int32)), dev(tables)
    capi.paged_attention_extend(one, q, *cache, t, n, dev(np.arange(4, dtype=np.int32)), 0.09, workspace[d],
                                cache_dtype=cache_dtype)
    ws = torch.zeros(capi.paged_attention_workspace_bytes(3, hq, hkv, d, q_dtype, cache_dtype), dtype=torch.uint8,
                     device="cuda")
    capi.paged_attention_decode(ref, q, *cache, t, n, max(lens), 0.09, ws, cache_dtype=cache_dtype)
    for out in (one, ref):
        got = out.double().cpu().numpy()
        for b, L in enumerate(lens):
            check(got[b:b + 1], x[b:b + 1], *model.gather(tables[b], L), 0.09, 0, 0, q_dtype, cache_dtype, False)
