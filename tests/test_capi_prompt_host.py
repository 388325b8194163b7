"""CPU tests of what the calls for many tokens of a sequence refuse, at the C ABI and in the Python binding.

Every call here is refused by its argument checks, before anything reaches a GPU.
"""
import ctypes as C
import os

import pytest

from paged_kv_cache_163_gb300 import build, capi

torch = pytest.importorskip("torch")
F32, F16, BF16 = (capi.DTYPE_NAMES[n] for n in ("f32", "f16", "bf16"))
E4M3, INT8 = capi.DTYPE_NAMES["fp8_e4m3"], capi.DTYPE_NAMES["int8"]
A = 0x10000                 # an aligned address that nobody reads
INVALID, UNSUPPORTED, WORKSPACE = -1, -4, -6


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(capi.LIB_PATH):
        build.build()
    return capi.load()


def refused(lib, fn, args, status, word, **change):
    assert not set(change) - set(args), change
    assert getattr(lib, fn)(*{**args, **change}.values()) == status, change
    assert word in lib.pkv_last_error().decode(), (change, lib.pkv_last_error())


ROPE_TABLE = dict(cos_sin=A, max_positions=8, rot_dim=64, base=1e4, scaling=0, factor=1.0, original_max=0,
                  slow_turns=1.0, fast_turns=32.0, magnitude=0.0, stream=None)


@pytest.mark.parametrize("change,word", [
    (dict(max_positions=-1), "rot_dim"), (dict(rot_dim=0), "rot_dim"), (dict(rot_dim=24), "rot_dim"),
    (dict(rot_dim=144), "rot_dim"), (dict(scaling=9), "scaling"), (dict(base=1.0), "base"),
    (dict(base=float("nan")), "base"), (dict(base=float("inf")), "base"), (dict(magnitude=-1.0), "magnitude"),
    (dict(scaling=1, factor=0.5), "factor"), (dict(scaling=2, factor=float("inf")), "factor"),
    (dict(scaling=3, factor=4.0), "original_max"), (dict(scaling=3, factor=4.0, original_max=64, slow_turns=32.0), "slow"),
    (dict(cos_sin=None), "NULL"), (dict(cos_sin=A + 4), "misaligned"),
])
def test_rope_table(lib, change, word):
    refused(lib, "pkv_rope_table", ROPE_TABLE, INVALID, word, **change)


POOL = dict(k_cache=A << 20, v_cache=A << 21, cache_dtype=BF16, k_scale=None, v_scale=None)
APPEND = dict(q_out=A, q=A << 4, k=A << 8, v=A << 12, in_dtype=BF16, q_stride=512, k_stride=128, v_stride=128, tokens=4,
              hq=8, hkv=2, d=64, positions=A, slots=A, cos_sin=A, max_positions=8, rot_dim=64, interleaved=0,
              **POOL, num_blocks=4, block_size=16, d_error=None, stream=None)
GATHER = dict(k_out=A, v_out=A << 4, out_dtype=BF16, num_rows=8, **POOL, tables=A, max_blocks=4, token_starts=None,
              lens=A, starts=A, num_seqs=2, hkv=2, d=64, num_blocks=4, block_size=16, d_error=None, stream=None)
EXTEND = dict(out=A, out_dtype=F32, q=A << 4, q_dtype=BF16, num_queries=8, **POOL, tables=A, max_blocks=4, lens=A,
              starts=A, num_seqs=2, hq=8, hkv=2, d=64, num_blocks=4, block_size=16, scale=0.1, window=0, sinks=0,
              workspace=A, workspace_bytes=0, d_error=None, stream=None)


@pytest.mark.parametrize("fn,args", [("paged_kv_append_rope", APPEND), ("paged_kv_gather", GATHER),
                                     ("paged_attention_extend", EXTEND)])
@pytest.mark.parametrize("change,status,word", [
    (dict(hkv=0), INVALID, "sizes"), (dict(num_blocks=0), INVALID, "sizes"),
    (dict(block_size=8), UNSUPPORTED, "block_size"), (dict(block_size=64), UNSUPPORTED, "block_size"),
    (dict(d=96), UNSUPPORTED, "head_dim"), (dict(d=256), UNSUPPORTED, "head_dim"),
    (dict(cache_dtype=F32), INVALID, "cache dtype"), (dict(cache_dtype=99), INVALID, "cache dtype"),
    (dict(num_blocks=1 << 27, hkv=2), UNSUPPORTED, "2^31"), (dict(k_cache=None), INVALID, "cache"),
    (dict(v_cache=(A << 21) + 8), INVALID, "cache"), (dict(cache_dtype=E4M3), INVALID, "scale"),
    (dict(cache_dtype=E4M3, k_scale=A, v_scale=A), INVALID, "scale"),
    (dict(cache_dtype=INT8, k_scale=A + 4, v_scale=A + 68), INVALID, "scale"),
])
def test_pools(lib, fn, args, change, status, word):
    refused(lib, fn, args, status, word, **change)


@pytest.mark.parametrize("change,status,word", [
    (dict(tokens=-1), INVALID, "sizes"), (dict(hq=-1), INVALID, "sizes"), (dict(in_dtype=F32), INVALID, "F16 or BF16"),
    (dict(in_dtype=F16), UNSUPPORTED, "match"), (dict(rot_dim=80), UNSUPPORTED, "rot_dim"),
    (dict(rot_dim=8), UNSUPPORTED, "rot_dim"), (dict(q_stride=504), INVALID, "stride"),
    (dict(q_stride=516), INVALID, "stride"), (dict(k_stride=120), INVALID, "stride"),
    (dict(v_stride=132), INVALID, "stride"), (dict(k=None), INVALID, "NULL"), (dict(v=(A << 12) + 2), INVALID, "misaligned"),
    (dict(positions=None), INVALID, "NULL"), (dict(slots=None), INVALID, "NULL"), (dict(cos_sin=None), INVALID, "NULL"),
    (dict(q=None), INVALID, "NULL"), (dict(q_out=None), INVALID, "NULL"), (dict(q=A + 16), INVALID, "overlaps"),
    (dict(q=A, q_stride=768), INVALID, "overlaps"), (dict(k=A + 256), INVALID, "overlaps"),
    (dict(v=A), INVALID, "overlaps"),
])
def test_append_rope(lib, change, status, word):
    refused(lib, "paged_kv_append_rope", APPEND, status, word, **change)


@pytest.mark.parametrize("change,status,word", [
    (dict(num_rows=-1), INVALID, "sizes"), (dict(max_blocks=-1), INVALID, "sizes"),
    (dict(num_seqs=-1), UNSUPPORTED, "num_seqs"), (dict(num_seqs=1025), UNSUPPORTED, "num_seqs"),
    (dict(out_dtype=E4M3), INVALID, "out_dtype"), (dict(out_dtype=F16), UNSUPPORTED, "own type"),
    (dict(k_out=None), INVALID, "NULL"), (dict(v_out=A + 8), INVALID, "misaligned"), (dict(tables=None), INVALID, "NULL"),
    (dict(lens=None), INVALID, "NULL"), (dict(starts=None), INVALID, "NULL"),
])
def test_gather(lib, change, status, word):
    refused(lib, "paged_kv_gather", GATHER, status, word, **change)


@pytest.mark.parametrize("change,status,word", [
    (dict(num_queries=-1), INVALID, "sizes"), (dict(max_blocks=-1), INVALID, "sizes"),
    (dict(num_seqs=1025), UNSUPPORTED, "num_seqs"), (dict(num_seqs=-1), UNSUPPORTED, "num_seqs"),
    (dict(hq=0), INVALID, "num_q_heads"), (dict(hq=7), INVALID, "num_q_heads"), (dict(hq=6), UNSUPPORTED, "1, 2, 4, 8"),
    (dict(hq=64), UNSUPPORTED, "1, 2, 4, 8"), (dict(q_dtype=F16), UNSUPPORTED, "pair"), (dict(q_dtype=F32), UNSUPPORTED, "pair"),
    (dict(out_dtype=F16), UNSUPPORTED, "out_dtype"), (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"), (dict(window=-1), INVALID, "window"), (dict(sinks=-1), INVALID, "sinks"),
    (dict(num_queries=1 << 29), UNSUPPORTED, "too many"), (dict(max_blocks=1 << 27), UNSUPPORTED, "too many"),
    (dict(out=None), INVALID, "NULL"), (dict(q=(A << 4) + 2), INVALID, "misaligned"), (dict(tables=None), INVALID, "NULL"),
    (dict(lens=None), INVALID, "NULL"), (dict(starts=None), INVALID, "NULL"), (dict(workspace=None), INVALID, "NULL"),
    (dict(out=A << 4), INVALID, "overlaps"), (dict(out=(A << 4) - 64), INVALID, "overlaps"),
])
def test_extend(lib, change, status, word):
    refused(lib, "paged_attention_extend", EXTEND, status, word, **change)


def test_workspace_bytes(lib):
    n = C.c_size_t()
    assert lib.paged_attention_extend_workspace_bytes(96, C.byref(n)) == UNSUPPORTED
    assert lib.paged_attention_extend_workspace_bytes(128, None) == INVALID


def test_calls_with_nothing_to_do_return(lib):
    """Empty calls are no errors and launch nothing."""
    for fn, args, change in (("paged_kv_append_rope", APPEND, dict(tokens=0)), ("paged_kv_gather", GATHER, dict(num_rows=0)),
                             ("paged_kv_gather", GATHER, dict(num_seqs=0)),
                             ("paged_attention_extend", EXTEND, dict(num_queries=0)),
                             ("paged_attention_extend", EXTEND, dict(num_seqs=0)),
                             ("pkv_rope_table", ROPE_TABLE, dict(max_positions=0))):
        assert getattr(lib, fn)(*{**args, **change}.values()) == 0


def test_the_binding_wants_gpu_tensors():
    """Host tensors are refused by name instead of being read as device pointers."""
    z = torch.zeros
    k = z((4, 2, 64), dtype=torch.bfloat16)
    pool = z((4, 2, 16, 64), dtype=torch.bfloat16)
    i = z(4, dtype=torch.int32)
    with pytest.raises(capi.PkvError, match="cos_sin"):
        capi.pkv_rope_table(z((8, 2, 32)))
    with pytest.raises(capi.PkvError, match="k"):
        capi.paged_kv_append_rope(None, None, k, k, i, i, z((8, 2, 32)), pool, pool)
    with pytest.raises(capi.PkvError, match="k_out"):
        capi.paged_kv_gather(k, k, pool, pool, None, None, i.view(2, 2), i[:2], i[:3])
    with pytest.raises(capi.PkvError, match="q"):
        capi.paged_attention_extend(k, k, pool, pool, None, None, i.view(2, 2), i[:2], i[:3], 1.0, z(8))
