"""GPU parity of the cache read-back: values bit for bit, rows in place, errors reported and skipped."""
import numpy as np
import pytest

from oracle.cache import PagedCacheModel
from paged_kv_cache_163_gb300 import workloads as wl

from helpers import oracle_bits
from test_gpu_rope import bits16, dev, empty_cache

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from paged_kv_cache_163_gb300 import capi as c
    c.load()
    return c


def fill(capi, lens, hkv, d, in_dtype, cache_dtype, bs, seed):
    """A written cache of sequences over a shuffled pool: tensors, tables, oracle rows per sequence."""
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 2
    order = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), max(need + [1])), -1, np.int32)
    model = PagedCacheModel(nb, hkv, d, cache_dtype, block_size=bs)
    cache = empty_cache(nb, hkv, bs, d, cache_dtype)
    at = 0
    for b, n in enumerate(lens):
        tables[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        if not n:
            continue
        x = rng.standard_normal((2, n, hkv, d)).astype(np.float32)
        x *= np.where(rng.random(x.shape) < 0.01, 20, 1).astype(np.float32)
        x = wl.round_to(x, in_dtype)
        p = np.arange(n)
        slots = (tables[b, p // bs] * bs + p % bs).astype(np.int32)
        capi.paged_kv_append(dev(x[0], in_dtype), dev(x[1], in_dtype), dev(slots), *cache, cache_dtype=cache_dtype)
        model.write(slots, x[0], x[1])
    return cache, tables, model


def once_rounded(x64, dtype):
    """fp64 products of an exact code and an fp32 scale -> fp32 (one rounding) -> the output type."""
    y = x64.astype(np.float32)
    return y if dtype == "f32" else wl.round_to(y, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cache_dtype,in_dtype", [("f16", "f16"), ("bf16", "bf16"), ("fp8_e4m3", "bf16"),
                                                  ("fp8_e5m2", "f16"), ("int8", "bf16"), ("fp8_e4m3_int4", "f16")])
@pytest.mark.parametrize("lens,hkv,bs,tails", [([1], 1, 16, False), ([100, 0, 33, 1, 16, 17], 2, 16, True),
                                               ([300, 47], 8, 32, True), ([0, 0, 5], 3, 32, False)])
def test_gather_bit_exact(capi, d, cache_dtype, in_dtype, lens, hkv, bs, tails):
    cache, tables, model = fill(capi, lens, hkv, d, in_dtype, cache_dtype, bs, d + len(lens))
    rng = np.random.default_rng(3)
    first = np.array([rng.integers(0, n + 1) if tails and n else 0 for n in lens], np.int32)
    count = np.array(lens) - first
    lead, more = 2, 3                                  # rows before and behind the sequences stay as they were
    starts = np.concatenate(([0], np.cumsum(count))).astype(np.int32) + lead
    total = int(starts[-1]) + more
    for out in ["f32"] + ([cache_dtype] if cache_dtype in ("f16", "bf16") else ["f16", "bf16"]):
        dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[out]
        k, v = (torch.full((total, hkv, d), 7.0, dtype=dt, device="cuda") for _ in range(2))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        capi.paged_kv_gather(k, v, *cache, dev(tables), dev(np.array(lens, np.int32)), dev(starts),
                             token_starts=dev(first) if tails else None, d_error=err, cache_dtype=cache_dtype)
        assert capi.pkv_read_device_error(err) == 0
        for got, which in ((k, 0), (v, 1)):
            assert torch.all(got[:lead] == 7.0) and torch.all(got[total - more:] == 7.0)
            for b, n in enumerate(lens):
                want = once_rounded(model.gather(tables[b], n)[which][first[b]:], out)
                rows = got[starts[b]:starts[b + 1]]
                if out == "f32":
                    assert np.array_equal(rows.cpu().numpy(), want)
                else:
                    assert np.array_equal(bits16(rows), oracle_bits(want, out))


def test_gather_reports_and_skips(capi):
    cache, tables, _ = fill(capi, [40, 40, 40], 2, 64, "f16", "f16", 16, 1)
    tables[1, 1] = 99999
    starts = dev(np.array([0, 40, 80, 125], np.int32))   # five rows more than sequence 2 holds
    k, v = (torch.full((125, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.paged_kv_gather(k, v, *cache, dev(tables), dev(np.array([40, 40, 40], np.int32)), starts, d_error=err)
    assert capi.pkv_read_device_error(err) == capi.DEVERR_BAD_BLOCK | capi.DEVERR_BAD_CONTEXT_LEN
    untouched = (k == 7.0).all(-1).all(-1).nonzero()[:, 0].tolist()
    assert untouched == list(range(56, 72)) + list(range(120, 125))


def test_gather_many_sequences_and_fewer_rows_than_named(capi):
    """A batch at the limit, most sequences empty; rows past the outputs' end are not written."""
    rng = np.random.default_rng(9)
    lens = np.zeros(1024, np.int64)
    lens[rng.integers(0, 1024, 40)] = rng.integers(1, 50, 40)
    cache, tables, model = fill(capi, lens.tolist(), 1, 64, "bf16", "fp8_e4m3", 16, 2)
    starts = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    n = int(starts[-1]) - 11
    k, v = (torch.empty((n, 1, 64), dtype=torch.float32, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.paged_kv_gather(k, v, *cache, dev(tables), dev(lens.astype(np.int32)), dev(starts), d_error=err)
    assert capi.pkv_read_device_error(err) == 0
    want = np.concatenate([model.gather(tables[b], int(m))[1] for b, m in enumerate(lens) if m])[:n]
    assert np.array_equal(v.cpu().numpy(), want.astype(np.float32))
