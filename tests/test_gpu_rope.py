"""GPU parity of the rotary table and of the rotating append.

The append is compared bit for bit: its fp32 operations are fixed, so the
rotated queries, the 16-bit cache rows and the codes and scales of coded
caches equal the oracle's on the same fp32 table.  Against fp64 the rotation
is off by at most the rounding of two products and one sum.
"""
import numpy as np
import pytest

from oracle import rope
from oracle.cache import PagedCacheModel
from paged_kv_cache_163_gb300 import workloads as wl
from paged_kv_cache_163_gb300.capi import SCALED_CACHES, v_row_elems

from helpers import cache_bits, oracle_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PAIRS = [("f16", "f16"), ("bf16", "bf16"), ("bf16", "fp8_e4m3"), ("f16", "fp8_e4m3"), ("bf16", "fp8_e5m2"),
         ("f16", "int8"), ("bf16", "int8"), ("f16", "fp8_e4m3_int4")]


@pytest.fixture(scope="module")
def capi():
    from paged_kv_cache_163_gb300 import capi as c
    c.load()
    return c


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to({"f16": torch.float16, "bf16": torch.bfloat16}[dtype])


def empty_cache(nb, hkv, bs, d, cache_dtype):
    from paged_kv_cache_163_gb300.engine import torch_dtype
    kc = torch.empty((nb, hkv, bs, d), dtype=torch_dtype(cache_dtype), device="cuda")
    vc = torch.empty((nb, hkv, bs, v_row_elems(cache_dtype, d)), dtype=kc.dtype, device="cuda")
    kc.view(torch.uint8).fill_(0xFF)
    vc.view(torch.uint8).fill_(0xFF)
    if cache_dtype not in SCALED_CACHES:
        return kc, vc, None, None
    both = torch.full((nb, hkv, 2, bs), float("nan"), device="cuda")
    return kc, vc, both[:, :, 0], both[:, :, 1]


def compare(kc, vc, ks, vs, model, cache_dtype):
    filled = model.filled
    for got, want, part in ((kc, model.k, model.k_type), (vc, model.v, model.v_type)):
        g = cache_bits(got).transpose(0, 2, 1, 3)
        w = want.transpose(0, 2, 1, 3)[filled]
        assert np.array_equal(g[filled], oracle_bits(w, part) if part in ("f16", "bf16") else w)
        assert np.all(g[~filled] == (0xFFFF if part in ("f16", "bf16") else 0xFF))  # slots not named stay as they were
    if ks is not None:
        for got, want in ((ks, model.k_scale), (vs, model.v_scale)):
            assert np.array_equal(got.cpu().numpy().transpose(0, 2, 1)[filled], want.transpose(0, 2, 1)[filled])


def bits16(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("in_dtype,cache_dtype", PAIRS)
@pytest.mark.parametrize("t,hq,hkv,rot,interleaved,bs", [
    (1, 8, 2, 64, False, 16), (5, 32, 8, 64, True, 32), (37, 1, 1, 16, False, 16), (700, 6, 3, 48, False, 16),
    (640, 32, 8, 32, True, 16), (3, 0, 4, 64, False, 32)])
def test_append_rope_bit_exact(capi, d, in_dtype, cache_dtype, t, hq, hkv, rot, interleaved, bs):
    rot = rot * d // 64 if rot != 48 else 48
    rng = np.random.default_rng(t + d + rot)
    nb = -(-t // bs) + 3
    x = rng.standard_normal((t, hq + 2 * hkv, d)).astype(np.float32)
    x *= rng.uniform(1e-3, 30, x.shape[:2] + (1,)).astype(np.float32)
    if t > 4:
        x[3, hq] = 0.0                                   # an all-zero key
    x = wl.round_to(x, in_dtype)
    maxp = 5000
    cos, sin = (a.astype(np.float32) for a in rope.table(maxp, rot, base=10000.0))
    pos = rng.integers(0, maxp, t).astype(np.int32)
    pos[0] = maxp - 1
    slots = rng.permutation(nb * bs)[:t].astype(np.int32)
    slots[2::23] = -1
    rows = dev(x, in_dtype)                              # one projection's output: q, k, v side by side
    q, k, v = rows.split((hq, hkv, hkv), 1)
    q_out = torch.empty((t, hq, d), dtype=rows.dtype, device="cuda")
    kc, vc, ks, vs = empty_cache(nb, hkv, bs, d, cache_dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs = dev(np.stack((cos, sin), 1))
    capi.paged_kv_append_rope(q_out if hq else None, q if hq else None, k, v, dev(pos), dev(slots), cs, kc, vc, ks, vs,
                              interleaved=interleaved, d_error=err, cache_dtype=cache_dtype)
    assert capi.pkv_read_device_error(err) == 0
    y = rope.rotate(x[:, :hq + hkv], cos[pos], sin[pos], rot, interleaved)
    if hq:
        assert np.array_equal(bits16(q_out), oracle_bits(wl.round_to(y[:, :hq], in_dtype), in_dtype))
    model = PagedCacheModel(nb, hkv, d, cache_dtype, block_size=bs)
    yk = y[:, hq:]
    model.write(slots, wl.round_to(yk, in_dtype) if cache_dtype == in_dtype else yk, x[:, hq + hkv:])
    compare(kc, vc, ks, vs, model, cache_dtype)
    # against fp64 on the same table: two products and a sum, each rounded by 2^-24
    y64 = rope.rotate(x[:, :hq + hkv].astype(np.float64), cos[pos], sin[pos], rot, interleaved)
    size = rope.rotate(np.abs(x[:, :hq + hkv]).astype(np.float64), np.abs(cos[pos]), -np.abs(sin[pos]), rot, interleaved)
    size = np.maximum(np.abs(size), rope.rotate(np.abs(x[:, :hq + hkv]).astype(np.float64), np.abs(cos[pos]),
                                                np.abs(sin[pos]), rot, interleaved))
    assert np.all(np.abs(y - y64) <= size * 2.1 * 2.0 ** -24 + 1e-44)


def test_queries_in_place_and_no_fused_rounding(capi):
    """q_out = q; the result does not depend on where it is written."""
    rng = np.random.default_rng(5)
    t, hq, hkv, d = 19, 8, 2, 128
    x = wl.round_to(rng.standard_normal((t, hq + 2 * hkv, d)).astype(np.float32), "bf16")
    cos, sin = (a.astype(np.float32) for a in rope.table(64, d))
    pos = rng.integers(0, 64, t).astype(np.int32)
    q, k, v = dev(x[:, :hq], "bf16"), dev(x[:, hq:hq + hkv], "bf16"), dev(x[:, hq + hkv:], "bf16")
    kc, vc, ks, vs = empty_cache(2, hkv, 16, d, "int8")
    cs = dev(np.stack((cos, sin), 1))
    out = torch.empty_like(q)
    args = (k, v, dev(pos), torch.arange(t, dtype=torch.int32, device="cuda"), cs, kc, vc, ks, vs)
    capi.paged_kv_append_rope(out, q, *args, cache_dtype="int8")
    capi.paged_kv_append_rope(q, q, *args, cache_dtype="int8")
    assert torch.equal(out, q)


def test_bad_positions_and_slots_are_reported_and_skipped(capi):
    t, hq, hkv, d, nb = 6, 2, 1, 64, 2
    rows = torch.ones((t, hq + 2 * hkv, d), dtype=torch.float16, device="cuda")
    q, k, v = rows.split((hq, hkv, hkv), 1)
    cs = dev(np.stack([a.astype(np.float32) for a in rope.table(8, 64)], 1))
    kc, vc, _, _ = empty_cache(nb, hkv, 16, d, "f16")
    q_out = torch.full((t, hq, d), 7.0, dtype=torch.float16, device="cuda")
    pos = dev(np.array([0, -1, 8, 3, 4, 5], np.int32))
    slots = dev(np.array([0, 1, 2, nb * 16, -1, 5], np.int32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.paged_kv_append_rope(q_out, q, k, v, pos, slots, cs, kc, vc, d_error=err)
    assert capi.pkv_read_device_error(err) == capi.DEVERR_BAD_POSITION | capi.DEVERR_BAD_SLOT
    assert torch.all(q_out[1:3] == 7.0) and not torch.any(q_out[3:] == 7.0)
    written = (kc[:, 0].view(torch.int16).reshape(nb * 16, d)[:, 0] != -1).nonzero()[:, 0].tolist()
    assert written == [0, 5]


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
                                dict(scaling="ntk", factor=8.0),
                                dict(scaling="by_parts", factor=16.0, original_max=4096, slow_turns=1.0, fast_turns=32.0)])
@pytest.mark.parametrize("rot", [16, 64, 96, 128])
def test_table_matches_fp64(capi, kw, rot):
    maxp = 20011
    t = torch.empty((maxp, 2, rot // 2), dtype=torch.float32, device="cuda")
    capi.pkv_rope_table(t, **kw)
    cos, sin = rope.table(maxp, rot, **kw)
    mag = 0.1 * np.log(kw["factor"]) + 1.0 if kw.get("scaling") == "by_parts" else 1.0
    # one rounding to fp32 (2^-24 of a value up to mag) and the fp64 angle's own error
    # (a few units of 2^-53 of angles up to maxp)
    tol = mag * (2.0 ** -24 + maxp * 8 * 2.0 ** -53) * 1.001
    got = t.cpu().numpy().astype(np.float64)
    assert np.max(np.abs(got[:, 0] - cos)) <= tol and np.max(np.abs(got[:, 1] - sin)) <= tol
