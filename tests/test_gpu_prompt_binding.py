"""The binding of the prompt-side calls: native and Python argument checks pass and refuse the same."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from paged_kv_cache_163_gb300 import capi as c
    c.load()
    return c


@pytest.fixture(params=["native", "python"])
def side(request, capi, monkeypatch):
    if request.param == "native":
        assert capi._native_calls() is not None
    else:
        monkeypatch.setattr(capi, "_native", None)
    return request.param


def arguments(capi, cache_dtype):
    """Positional and keyword arguments of each call, by name, over one small pool."""
    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    torch.manual_seed(1)
    coded = cache_dtype != "bf16"
    pool = (4, 2, 16, 64)
    k, v = ((torch.zeros(pool, dtype=torch.uint8, device="cuda") if coded else
             torch.zeros(pool, dtype=torch.bfloat16, device="cuda")) for _ in range(2))
    sc = torch.zeros((4, 2, 2, 16), device="cuda")
    ks, vs = (sc[:, :, 0], sc[:, :, 1]) if coded else (None, None)
    rows = torch.randn((5, 12, 64), device="cuda").bfloat16()
    q, kn, vn = rows.split((8, 2, 2), 1)
    cs = torch.zeros((16, 2, 32), device="cuda")
    capi.pkv_rope_table(cs)
    err = ints(0)
    append = dict(q_out=torch.zeros((5, 8, 64), device="cuda").bfloat16(), q=q, k=kn, v=vn, positions=ints(0, 1, 2, 3, 4),
                  slot_mapping=ints(16, 17, 18, 19, 20), cos_sin=cs, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs,
                  interleaved=False, d_error=err, cache_dtype=cache_dtype)
    tables, lens = ints(1, 3).view(1, 2), ints(5)
    gather = dict(k_out=torch.zeros((5, 2, 64), device="cuda"), v_out=torch.zeros((5, 2, 64), device="cuda"), k_cache=k,
                  v_cache=v, k_scale=ks, v_scale=vs, block_tables=tables, context_lens=lens, out_starts=ints(0, 5),
                  token_starts=ints(0), d_error=err, cache_dtype=cache_dtype)
    ws = torch.zeros(capi.paged_attention_extend_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    extend = dict(out=torch.zeros((5, 8, 64), device="cuda"), q=append["q_out"], k_cache=k, v_cache=v, k_scale=ks,
                  v_scale=vs, block_tables=tables, context_lens=lens, query_starts=ints(0, 5), scale=0.125, workspace=ws,
                  window=0, sinks=0, d_error=err, cache_dtype=cache_dtype)
    return {"paged_kv_append_rope": append, "paged_kv_gather": gather, "paged_attention_extend": extend}


@pytest.mark.parametrize("cache_dtype", ["bf16", "fp8_e4m3"])
def test_both_sides_compute_the_same(capi, cache_dtype, monkeypatch):
    results = []
    for native in (True, False):
        if native:
            assert capi._native_calls() is not None
        else:
            monkeypatch.setattr(capi, "_native", None)
        args = arguments(capi, cache_dtype)
        for name, kw in args.items():
            before = capi.pkv_launch_count()
            getattr(capi, name)(**kw)
            assert capi.pkv_launch_count() == before + 1
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        getattr(capi, "paged_kv_gather")(**{**args["paged_kv_gather"], "stream": stream})
        stream.synchronize()
        torch.cuda.synchronize()
        results.append([args["paged_kv_append_rope"]["q_out"], args["paged_kv_gather"]["k_out"],
                        args["paged_kv_gather"]["v_out"], args["paged_attention_extend"]["out"]])
    for a, b in zip(*results):
        assert torch.equal(a, b) and bool(a.abs().sum() > 0)


TENSORS = {"paged_kv_append_rope": ["q_out", "q", "k", "v", "positions", "slot_mapping", "cos_sin", "k_cache", "v_cache",
                                    "k_scale", "v_scale", "d_error"],
           "paged_kv_gather": ["k_out", "v_out", "k_cache", "v_cache", "k_scale", "v_scale", "block_tables",
                               "context_lens", "out_starts", "token_starts", "d_error"],
           "paged_attention_extend": ["out", "q", "k_cache", "v_cache", "k_scale", "v_scale", "block_tables",
                                      "context_lens", "query_starts", "workspace", "d_error"]}


@pytest.mark.parametrize("name", sorted(TENSORS))
@pytest.mark.parametrize("wrong", ["host", "type", "rows", "strided"])
def test_wrong_tensors_are_refused(capi, side, name, wrong):
    """Each tensor argument in turn: on the host, of another type, one row short, not dense; nothing is launched."""
    for arg in TENSORS[name]:
        kw = arguments(capi, "fp8_e4m3")[name]
        t = kw[arg]
        if wrong == "host":
            bad = t.cpu()
        elif wrong == "type":
            if arg == "workspace":
                continue                                     # any type's bytes do
            bad = t.double()
        elif wrong == "rows":
            if arg in ("k_cache", "cos_sin", "workspace"):
                continue                                     # their size is the call's to know
            bad = t[:-1] if t.dim() else t
        else:
            if arg in ("q", "k", "v", "k_scale", "v_scale", "d_error") or t.dim() == 1 and t.numel() == 1:
                continue                                     # may be strided, or have one element
            bad = torch.stack((t, t), -1)[..., 0]
        before = capi.pkv_launch_count()
        with pytest.raises((capi.PkvError, ValueError)) as e:
            getattr(capi, name)(**{**kw, arg: bad})
        assert capi.pkv_launch_count() == before
        assert name in str(e.value)


def test_wrong_sizes_are_refused_by_the_library(capi, side):
    args = arguments(capi, "bf16")
    for name, change, word in (("paged_attention_extend", dict(scale=float("nan")), "scale"),
                               ("paged_attention_extend", dict(window=-1), "window"),
                               ("paged_attention_extend", dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                                "workspace"),
                               ("paged_kv_gather", dict(k_out=torch.zeros((5, 2, 64), device="cuda").half(),
                                                        v_out=torch.zeros((5, 2, 64), device="cuda").half()), "own type"),
                               ("paged_kv_append_rope", dict(cos_sin=torch.zeros((4, 2, 36), device="cuda")), "rot_dim")):
        with pytest.raises(capi.PkvError, match=word):
            getattr(capi, name)(**{**args[name], **change})


def test_numbers_of_other_kinds_are_taken(capi, side):
    """NumPy integers and floats, None for the cache's type, raw stream handles."""
    args = arguments(capi, "bf16")
    a = args["paged_kv_append_rope"]
    capi.paged_kv_append_rope(**{**a, "cache_dtype": None, "interleaved": np.bool_(False),
                                 "stream": torch.cuda.current_stream().cuda_stream})
    e = args["paged_attention_extend"]
    capi.paged_attention_extend(**{**e, "scale": np.float32(0.125), "window": np.int64(3), "sinks": np.int32(1)})
    want = torch.zeros_like(e["out"])
    capi.paged_attention_extend(**{**e, "out": want, "window": 3, "sinks": 1})
    assert torch.equal(want, e["out"])
