"""The engine's prompts, chunks, drafted tokens and read-backs: rotation, cache write, attention and gather together.

Expected values come from the oracle: rows rotated in fp32 on the engine's
table, quantised by the cache model, attended in fp64.  Bounds as in
test_gpu_extend.py.
"""
import numpy as np
import pytest

from oracle import rope
from oracle.cache import PagedCacheModel
from paged_kv_cache_163_gb300 import capi, workloads as wl
from paged_kv_cache_163_gb300.engine import PagedKVCache

from helpers import oracle_bits
from test_gpu_extend import check
from test_gpu_gather import once_rounded
from test_gpu_rope import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
LAYERS, HKV, G, D = 2, 2, 4, 64


class Mirror:
    """Every sequence's rows as the cache should hold them, layer by layer."""

    def __init__(self, cache, q_dtype, cos_sin, interleaved):
        self.cache, self.q_dtype, self.cs, self.interleaved = cache, q_dtype, cos_sin, interleaved
        self.rows = {}

    def fork(self, a, b):
        self.cache.fork(a, b)
        self.rows[b] = [[x.copy() for x in r] for r in self.rows[a]]

    def turn(self, x, pos):
        if self.cs is None:
            return x
        return rope.rotate(x, self.cs[pos, 0], self.cs[pos, 1], 2 * self.cs.shape[2], self.interleaved)

    def kv(self, seq, layer):
        """K and V [L, Hkv, D] in fp64 as stored."""
        k, v = self.rows[seq][layer]
        n = max(len(k), 1)
        model = PagedCacheModel(-(-n // 16), HKV, D, self.cache.cache_dtype)
        model.write(np.arange(len(k)), k, v)
        return model.gather(np.arange(-(-n // 16)), len(k))

    def extend(self, seqs, counts, seed, scale=0.11, window=0, sinks=0, by_layer=False):
        rng = np.random.default_rng(seed)
        total = sum(counts)
        fused = wl.round_to(rng.standard_normal((LAYERS, total, (G + 2) * HKV, D)).astype(np.float32), self.q_dtype)
        q, k, v = dev(fused, self.q_dtype).split((G * HKV, HKV, HKV), 2)
        before = [len(self.rows.setdefault(s, [[np.zeros((0, HKV, D), np.float32)] * 2 for _ in range(LAYERS)])[0][0])
                  for s in seqs]
        if by_layer:                  # a model's way: a layer's rows come after the attention of the one before
            ext = self.cache.begin(seqs, counts)
            out = torch.stack([self.cache.extend_layer(
                ext, l, k[l], v[l], q[l], scale, torch.empty(q[l].shape, dtype=torch.float32, device="cuda"), window, sinks)
                for l in range(LAYERS)])
        else:
            out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
            assert self.cache.extend(seqs, counts, k, v, q, scale, out, window, sinks) is out
        got = out.double().cpu().numpy()
        at = 0
        for s, n, L0 in zip(seqs, counts, before):
            pos = np.arange(L0, L0 + n)
            for l in range(LAYERS):
                x = fused[l, at:at + n]
                y = self.turn(x[:, :(G + 1) * HKV], pos)
                yk = y[:, G * HKV:]
                stored = wl.round_to(yk, self.q_dtype) if self.cache.cache_dtype == self.q_dtype else yk
                r = self.rows[s][l]
                self.rows[s][l] = [np.concatenate((r[0], stored)), np.concatenate((r[1], x[:, (G + 1) * HKV:]))]
                check(got[l, at:at + n], wl.round_to(y[:, :G * HKV], self.q_dtype), *self.kv(s, l), scale, window, sinks,
                      self.q_dtype, self.cache.cache_dtype, False)
            assert self.cache.seq_len(s) == L0 + n
            at += n


@pytest.mark.parametrize("q_dtype,cache_dtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8_e4m3"), ("f16", "int8"),
                                                 ("bf16", "fp8_e4m3_int4")])
@pytest.mark.parametrize("rotary", ["none", "half", "interleaved"])
def test_prompts_chunks_drafts_forks_and_readback(q_dtype, cache_dtype, rotary):
    cache = PagedKVCache(num_layers=LAYERS, num_blocks=120, num_kv_heads=HKV, head_dim=D, cache_dtype=cache_dtype,
                         poison=True)
    if rotary != "none":
        cache.use_rope(700, rot_dim=D if rotary == "half" else 32, interleaved=rotary == "interleaved", base=5000.0)
    m = Mirror(cache, q_dtype, None if rotary == "none" else cache._rope.cpu().numpy(), rotary == "interleaved")
    for s in (3, 8):
        cache.create(s)
    m.extend([3, 8], [150, 17], 1)                          # two prompts
    m.extend([8, 3], [200, 1], 2, by_layer=True)            # a chunk of one beside a single token of the other
    m.fork(3, 5)
    m.extend([5, 3, 8], [4, 5, 0], 3)                       # drafted tokens on a shared last block: copied on write
    assert cache.cow_pairs
    m.extend([3, 5, 8], [1, 1, 1], 4, window=40, sinks=3)   # a step, windowed
    m.extend([5], [300], 5, window=64, by_layer=True)
    k, v, starts = cache.gather([8, 5], first=[0, 37])
    assert k.dtype == (torch.bfloat16 if cache.k_scale is not None else cache.k.dtype)
    name = "bf16" if k.dtype == torch.bfloat16 else "f16"
    for i, (s, first) in enumerate(((8, 0), (5, 37))):
        rows = slice(int(starts[i]), int(starts[i + 1]))
        for l in range(LAYERS):
            for got, want in zip((k, v), m.kv(s, l)):
                bits = got[l, rows].view(torch.int16).cpu().numpy().view(np.uint16)
                assert np.array_equal(bits, oracle_bits(once_rounded(want[first:], name), name))
    assert cache.check() == 0


def test_prefix_hit_then_the_rest_of_the_prompt():
    """An admitted prompt's mapped tokens are attended without being written again."""
    cache = PagedKVCache(num_layers=LAYERS, num_blocks=64, num_kv_heads=HKV, head_dim=D, cache_dtype="bf16", poison=True)
    cache.enable_prefix_cache(7)
    cache.use_rope(400)
    m = Mirror(cache, "bf16", cache._rope.cpu().numpy(), False)
    tokens = list(range(100, 230))
    assert cache.admit(1, tokens) == 0
    m.extend([1], [130], 1)
    cache.commit(1, tokens)
    got = cache.admit(2, tokens[:100] + [7] * 50)
    assert got == 96
    m.rows[2] = [[x[:got].copy() for x in r] for r in m.rows[1]]
    m.extend([2], [150 - got], 2)
    assert cache.check() == 0


def test_refusals_change_nothing():
    cache = PagedKVCache(num_layers=1, num_blocks=8, num_kv_heads=HKV, head_dim=D, cache_dtype="bf16")
    cache.use_rope(100)
    cache.create(1)
    cache.create(2)

    def rows(n, heads, d=D, dtype=torch.bfloat16):
        return torch.zeros((n, heads, d), dtype=dtype, device="cuda")

    cache.extend([1], [20], rows(20, HKV), rows(20, HKV), rows(20, HKV * G))
    with pytest.raises(ValueError):
        cache.begin([1, 1], [1, 1])
    with pytest.raises(ValueError):
        cache.begin([1, 2], [1])
    with pytest.raises(ValueError):
        cache.begin([1], [-1])
    with pytest.raises(ValueError):
        cache.begin([1], [81])                       # position 100
    with pytest.raises(ValueError):
        cache.extend([1], [3], rows(2, HKV), rows(3, HKV), rows(3, HKV * G))
    with pytest.raises(ValueError):
        cache.extend([1], [3], rows(3, HKV), rows(3, HKV), rows(3, 6))
    with pytest.raises(ValueError):
        cache.extend([1], [3], *(rows(3, h, dtype=torch.float16) for h in (HKV, HKV, HKV * G)))
    with pytest.raises(ValueError):
        cache.extend([1], [3], rows(3, HKV), rows(3, HKV), rows(3, HKV * G), out=rows(3, HKV))
    for bad in (dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
                dict(out=torch.zeros(3 * HKV * G * D + 1, device="cuda")[1:].view(3, HKV * G, D))):
        with pytest.raises(ValueError):
            cache.extend([1], [3], rows(3, HKV), rows(3, HKV), rows(3, HKV * G), **bad)
    with pytest.raises(capi.NoBlocksError):
        cache.begin([1, 2], [70, 70])
    with pytest.raises(ValueError):
        cache.gather([1], first=[21])
    assert cache.seq_len(1) == 20 and cache.seq_len(2) == 0
    ext = cache.begin([1], [2])
    for bad in ((rows(2, HKV), rows(2, HKV), rows(3, 8)), (rows(2, HKV, 32), rows(2, HKV), rows(2, 8)),
                (rows(2, HKV), rows(2, HKV, dtype=torch.float16), rows(2, 8)), (rows(2, HKV).cpu(), rows(2, HKV), rows(2, 8))):
        with pytest.raises(ValueError):
            cache.extend_layer(ext, 0, *bad)
    with pytest.raises(ValueError):
        cache.extend_layer(ext, 0, rows(2, HKV), rows(2, HKV), rows(2, 6))
    out = cache.extend_layer(ext, 0, rows(2, HKV), rows(2, HKV), rows(2, 8))
    assert out.shape == (2, 8, D) and cache.check() == 0
    k, v, starts = cache.gather([])
    assert k.shape[1] == 0 and list(starts) == [0]
    assert cache.extend([1, 2], [0, 0], rows(0, HKV), rows(0, HKV), rows(0, 8)).shape == (0, 8, D)


def test_on_a_stream_of_its_own():
    cache = PagedKVCache(num_layers=1, num_blocks=40, num_kv_heads=HKV, head_dim=D, cache_dtype="fp8_e5m2")
    base = PagedKVCache(num_layers=1, num_blocks=40, num_kv_heads=HKV, head_dim=D, cache_dtype="fp8_e5m2")
    torch.manual_seed(0)
    x = torch.randn((300, (G + 2) * HKV, D), device="cuda").bfloat16()
    q, k, v = x.split((G * HKV, HKV, HKV), 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    outs = []
    for c, s in ((base, None), (cache, stream)):
        c.create(0)
        c.use_rope(400, stream=s)
        outs.append((c.extend([0], [300], k, v, q, stream=s), c.gather([0], stream=s)[0]))
    stream.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("rotary", [False, True])
def test_rows_laid_out_in_any_way(rotary):
    """Transposed, broadcast, misaligned and strided rows give what dense ones give."""
    torch.manual_seed(3)
    n = 37
    q = torch.randn((n, HKV * G, D), device="cuda").bfloat16()
    kv = torch.randn((1, HKV, D), device="cuda").bfloat16().expand(n, HKV, D)

    def transposed(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    def misaligned(t):
        x = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        x.copy_(t)
        return x

    def slices(t):
        return torch.cat((t, t), 1)[:, t.shape[1]:]

    outs = []
    for lay in (torch.Tensor.contiguous, lambda t: t, transposed, misaligned, slices):
        c = PagedKVCache(num_layers=1, num_blocks=8, num_kv_heads=HKV, head_dim=D, cache_dtype="bf16", poison=True)
        if rotary:
            c.use_rope(64)
        c.create(0)
        outs.append(c.extend([0], [n], lay(kv), lay(kv), lay(q)))
        assert c.check() == 0
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
