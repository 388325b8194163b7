"""GPU parity of multi-token attention over the paged cache, against the fp64 definition.

Tolerances, from roundings counted before the first run.  The fp32 result of
a row is a mean of V rows with weights P / l.  P is rounded once to the
operand type (half a step: bf16 keeps 8 significant bits, so its spacing is
2^-7 of the binade's base and half of it 2^-8 of the value at most; f16 keeps
11, 2^-11: u = 2^-8 over bf16 caches, 2^-11 otherwise), so a row is off by at most u * mean|V| (weights P / l); every other step is fp32:
the scores' dot products of D terms (each rounded, 2^-24 * D * |q|.|k|), the
exponent's argument and 2^x (2^-22), sums of up to L terms.  These add at
most a relative error of e32 = scale * D * max|q|.|k| * 2^-23 + 2^-19 of
mean|V|.  A 16-bit output adds half a step of the result.

An f16 P below 2^-14 is subnormal: its half step is 2^-25 whatever its value
(the row's reference is one of its scores, so l >= 1 in the same unit).  That
adds at most 2^-25 sum|V| <= 2^-25 L max|V|.  Over a coded cache V becomes an
f16 operand, code x f16(scale / unit): two more roundings of 2^-11 each.
"""
import numpy as np
import pytest

from oracle.extend import extend_attention, visible
from paged_kv_cache_163_gb300 import workloads as wl

from test_gpu_gather import fill
from test_gpu_rope import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PAIRS = [("f16", "f16"), ("bf16", "bf16"), ("bf16", "fp8_e4m3"), ("f16", "fp8_e4m3"), ("bf16", "fp8_e5m2"),
         ("f16", "fp8_e5m2"), ("f16", "int8"), ("bf16", "int8"), ("f16", "fp8_e4m3_int4"), ("bf16", "fp8_e4m3_int4")]
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def capi():
    from paged_kv_cache_163_gb300 import capi as c
    c.load()
    return c


@pytest.fixture(scope="module")
def workspace(capi):
    return {d: torch.zeros(capi.paged_attention_extend_workspace_bytes(d), dtype=torch.uint8, device="cuda")
            for d in (64, 128)}


def check(got, q, K, V, scale, window, sinks, q_dtype, cache_dtype, out16):
    """Every row of one sequence within the bound of its own P, V and scores."""
    want = extend_attention(q, K, V, scale, window, sinks)
    n, hq, d = q.shape
    if n == 0 or len(K) == 0:
        assert np.all(got == 0.0)
        return
    L, hkv, _ = K.shape
    see = visible(L, n, window, sinks)
    u = HALF_STEP["bf16" if cache_dtype == "bf16" else "f16"]
    G = hq // hkv
    # tokens that no row sees have no part in the bounds (0 x NaN of an unwritten one is NaN)
    K, V = (np.where(see.any(0)[:, None, None], x, 0.0) for x in (K, V))
    for h in range(hq):
        k, v = K[:, h // G], V[:, h // G]
        s = np.where(see, scale * (q[:, h].astype(np.float64) @ k.T), -np.inf)
        top = s.max(-1, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(top), top, 0))
        l = p.sum(-1, keepdims=True)
        mean = (p / np.where(l > 0, l, 1)) @ np.abs(v)
        dots = abs(scale) * np.max(np.where(see, np.abs(q[:, h]).astype(np.float64) @ np.abs(k).T, 0), -1, keepdims=True)
        if cache_dtype not in ("f16", "bf16"):
            u = 3.01 * 2.0 ** -11
        tol = (u + dots * d * 2.0 ** -23 + 2.0 ** -19) * mean
        if cache_dtype != "bf16":
            tol = tol + 2.0 ** -25 * L * np.abs(v).max()
        if out16:
            tol = tol + HALF_STEP[q_dtype] * (np.abs(want[:, h]) + tol) + 2.0 ** -25
        off = np.abs(got[:, h] - want[:, h])
        assert np.all(np.isfinite(got[:, h]))
        assert np.all(off <= tol), (h, float((off / np.maximum(tol, 1e-300)).max()), np.argwhere(off > tol)[:4].tolist())


def run(capi, ws, lens, news, hq, hkv, d, q_dtype, cache_dtype, bs, window, sinks, out="16", seed=0, scale=None,
        poison_tables=True):
    rng = np.random.default_rng(seed)
    cache, tables, model = fill(capi, lens, hkv, d, q_dtype, cache_dtype, bs, seed)
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    total = int(starts[-1])
    q = wl.round_to(rng.standard_normal((total, hq, d)).astype(np.float32), q_dtype)
    if poison_tables and window:       # blocks that nobody sees may be gone from the table
        tables = tables.copy()
        for b, (L, n) in enumerate(zip(lens, news)):
            if n:
                seen = visible(L, min(n, L), window, sinks).any(0) if L else np.zeros(0, bool)
                for i in range(-(-L // bs)):
                    if not seen[i * bs:(i + 1) * bs].any():
                        tables[b, i] = 1 << 30
    scale = float(np.float32(1.0) / np.sqrt(np.float32(d))) if scale is None else scale
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[q_dtype]
    o = torch.full((total + 3, hq, d), 7.0, dtype=torch.float32 if out == "32" else dt, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd = torch.cat((dev(q, q_dtype), torch.zeros((3, hq, d), dtype=dt, device="cuda")))
    capi.paged_attention_extend(o, qd, *cache, dev(tables), dev(np.array(lens, np.int32)), dev(starts), scale, ws[d],
                                window=window, sinks=sinks, d_error=err, cache_dtype=cache_dtype)
    assert capi.pkv_read_device_error(err) == 0
    assert torch.all(o[total:] == 7.0)
    got = o.double().cpu().numpy()
    for b, (L, n) in enumerate(zip(lens, news)):
        K, V = model.gather(np.where(tables[b] < (1 << 30), tables[b], 0), L)
        rows = slice(starts[b], starts[b + 1])
        if n > L:                      # queries before the first token see nothing
            assert np.all(got[starts[b]:starts[b] + n - L] == 0.0)
            rows = slice(starts[b] + n - L, starts[b + 1])
        check(got[rows], q[rows], K, V, scale, window, sinks, q_dtype, cache_dtype, out == "16")
    return o


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_dtype,cache_dtype", PAIRS)
def test_one_step_each_type(capi, workspace, d, q_dtype, cache_dtype):
    """One item, one 128-token step or less: every type."""
    run(capi, workspace, [40], [3], 4, 1, d, q_dtype, cache_dtype, 16, 0, 0, "32", seed=1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_dtype,cache_dtype", PAIRS)
@pytest.mark.parametrize("lens,news,hq,hkv,bs,window,sinks", [
    ([1], [1], 1, 1, 16, 0, 0),
    ([1, 17, 33, 100], [1, 1, 1, 1], 8, 2, 16, 0, 0),
    ([300, 0, 129, 128, 127], [300, 0, 70, 1, 127], 4, 2, 32, 0, 0),
    ([500, 260], [500, 31], 8, 8, 16, 0, 0),
    ([700, 90, 411], [90, 90, 5], 16, 2, 16, 130, 0),
    ([700, 90, 411], [90, 90, 1], 16, 1, 32, 37, 21),
    ([1000, 333], [600, 1], 2, 2, 16, 1, 3),
    ([20, 5], [33, 5], 4, 4, 16, 0, 0),
])
def test_shapes(capi, workspace, d, q_dtype, cache_dtype, lens, news, hq, hkv, bs, window, sinks):
    run(capi, workspace, lens, news, hq, hkv, d, q_dtype, cache_dtype, bs, window, sinks, seed=len(lens) + hq)


@pytest.mark.parametrize("q_dtype,cache_dtype", [("bf16", "bf16"), ("bf16", "fp8_e4m3"), ("f16", "fp8_e4m3_int4")])
@pytest.mark.parametrize("lens,news,window,sinks", [([5000, 1234], [1, 1], 0, 0), ([9000], [5], 4096, 4),
                                                    ([3100, 2900, 40], [260, 2, 40], 0, 0)])
def test_long_contexts_are_split_and_merged(capi, workspace, q_dtype, cache_dtype, lens, news, window, sinks):
    o = run(capi, workspace, lens, news, 8, 2, 128, q_dtype, cache_dtype, 16, window, sinks, "32", seed=7)
    # the counters are left at zero: the same call on the same workspace gives the same bits
    again = run(capi, workspace, lens, news, 8, 2, 128, q_dtype, cache_dtype, 16, window, sinks, "32", seed=7)
    assert torch.equal(o, again)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.5])
@pytest.mark.parametrize("q_dtype,cache_dtype", [("f16", "f16"), ("bf16", "int8")])
def test_scales(capi, workspace, scale, q_dtype, cache_dtype):
    run(capi, workspace, [200, 31], [9, 31], 4, 2, 64, q_dtype, cache_dtype, 16, 50, 5, "32", seed=3, scale=scale)
