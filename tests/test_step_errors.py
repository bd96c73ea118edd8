"""Host-side refusals of the step operators (planning, norm + rotation + cache
write, attention of several new tokens): each is returned before anything is
enqueued, so stand-in addresses that nothing reads serve and no GPU is
needed.  And the binding's refusals of tensors.  CPU only."""

import pytest
import torch

from paged_kv_cache_124_gb300 import api

L = api._lib
A = 0x100000            # a 256-byte-aligned stand-in address (never dereferenced)


def multi(fp8=False, **kw):
    a = dict(out=2 * A, out_dtype=api.PA_DTYPE_BF16, q=A, k=A, v=A, tables=A, start=A, ctx=A, mask=None, block_size=16,
             scale=0.088, k_scale=0.01, v_scale=0.01, hq=32, hkv=8, d=128, num_seqs=4, tokens=16, most=4, max_blocks=8,
             num_blocks=64, max_ctx=128, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    scales = (a["k_scale"], a["v_scale"]) if fp8 else ()
    fn = L.pa_decode_multi_fp8 if fp8 else L.pa_decode_multi
    return fn(a["out"], a["out_dtype"], a["q"], a["k"], a["v"], a["tables"], a["start"], a["ctx"], a["mask"],
              a["block_size"], a["scale"], *scales, a["hq"], a["hkv"], a["d"], a["num_seqs"], a["tokens"], a["most"],
              a["max_blocks"], a["num_blocks"], a["max_ctx"], a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("kw,want", [
    (dict(num_seqs=0), api.PA_OK),
    (dict(tokens=0), api.PA_OK),
    (dict(num_seqs=-1), api.PA_ERR_INVALID_ARG),
    (dict(tokens=-1), api.PA_ERR_INVALID_ARG),
    (dict(most=0), api.PA_ERR_INVALID_ARG),
    (dict(max_ctx=-1), api.PA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), api.PA_ERR_INVALID_ARG),
    (dict(out_dtype=5), api.PA_ERR_INVALID_ARG),
    (dict(out=None), api.PA_ERR_INVALID_ARG),
    (dict(start=None), api.PA_ERR_INVALID_ARG),
    (dict(out=A), api.PA_ERR_INVALID_ARG),                        # in place of q
    (dict(block_size=64), api.PA_ERR_UNSUPPORTED),
    (dict(d=96), api.PA_ERR_UNSUPPORTED),
    (dict(hq=12), api.PA_ERR_UNSUPPORTED),
    (dict(hq=24), api.PA_ERR_UNSUPPORTED),                        # G = 3
    (dict(hq=256), api.PA_ERR_UNSUPPORTED),                       # G = 32
    (dict(mask=A, most=65), api.PA_ERR_UNSUPPORTED),              # a mask word has 64 bits
    (dict(num_blocks=1 << 30), api.PA_ERR_UNSUPPORTED),           # rows past 31 bits
    (dict(q=A + 8), api.PA_ERR_MISALIGNED),
    (dict(mask=A + 4), api.PA_ERR_MISALIGNED),
    (dict(ws=None), api.PA_ERR_WORKSPACE),
    (dict(ws=A + 16), api.PA_ERR_WORKSPACE),
])
def test_multi_host_checks(fp8, kw, want):
    assert multi(fp8, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(d=64), api.PA_ERR_UNSUPPORTED),
    (dict(k_scale=0.0), api.PA_ERR_INVALID_ARG),
    (dict(v_scale=float("inf")), api.PA_ERR_INVALID_ARG),
    (dict(v_scale=float("nan")), api.PA_ERR_INVALID_ARG),
])
def test_multi_fp8_host_checks(kw, want):
    assert multi(True, **kw) == want


def rope(fp8=False, **kw):
    a = dict(q_out=A, kc=A, vc=A, q=A, k=A, v=A, qs=4096, ks=1024, vs=1024, qw=A, kw=A, eps=1e-6, cs=A, maxpos=100,
             rot=128, inter=0, pos=A, slots=A, tokens=4, hq=32, hkv=8, d=128, block_size=16, num_blocks=64,
             k_scale=0.01, v_scale=0.01)
    a.update(kw)
    args = [a[n] for n in ("q_out", "kc", "vc", "q", "k", "v", "qs", "ks", "vs", "qw", "kw", "eps", "cs", "maxpos",
                           "rot", "inter", "pos", "slots", "tokens", "hq", "hkv", "d", "block_size", "num_blocks")]
    if fp8:
        return L.pa_qk_norm_rope_cache_fp8(*args, a["k_scale"], a["v_scale"], None, None)
    return L.pa_qk_norm_rope_cache(*args, None, None)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), api.PA_OK),
    (dict(tokens=-1), api.PA_ERR_INVALID_ARG),
    (dict(maxpos=0), api.PA_ERR_INVALID_ARG),
    (dict(eps=-1.0), api.PA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), api.PA_ERR_INVALID_ARG),
    (dict(eps=float("inf")), api.PA_ERR_INVALID_ARG),
    (dict(qw=None), api.PA_ERR_INVALID_ARG),                      # one gain without the other
    (dict(kw=None), api.PA_ERR_INVALID_ARG),
    (dict(cs=None), api.PA_ERR_INVALID_ARG),
    (dict(qs=4088), api.PA_ERR_INVALID_ARG),                      # tokens would overlap
    (dict(rot=0), api.PA_ERR_UNSUPPORTED),
    (dict(rot=24), api.PA_ERR_UNSUPPORTED),
    (dict(rot=144), api.PA_ERR_UNSUPPORTED),
    (dict(d=80), api.PA_ERR_UNSUPPORTED),
    (dict(block_size=4), api.PA_ERR_UNSUPPORTED),
    (dict(tokens=1 << 26), api.PA_ERR_UNSUPPORTED),               # rows past 31 bits
    (dict(qs=4100), api.PA_ERR_MISALIGNED),
    (dict(k=A + 2), api.PA_ERR_MISALIGNED),
    (dict(cs=A + 4), api.PA_ERR_MISALIGNED),
    (dict(slots=A + 4), api.PA_ERR_MISALIGNED),
])
def test_rope_host_checks(fp8, kw, want):
    assert rope(fp8, **kw) == want


def test_rope_fp8_scales():
    assert rope(True, k_scale=0.0) == rope(True, v_scale=float("inf")) == api.PA_ERR_INVALID_ARG


def plan(**kw):
    a = dict(tables=A, ctx=A, start=A, pos=A, slots=A, rows=A, new=A, lens=A, row_tables=A, row_blocks=A, free=A,
             count=A, capacity=10, seqs=4, num_rows=8, max_blocks=16, tokens=9, block_size=16, num_blocks=64)
    a.update(kw)
    return L.pa_plan_step(*[a[n] for n in ("tables", "ctx", "start", "pos", "slots", "rows", "new", "lens",
                                           "row_tables", "row_blocks", "free", "count", "capacity", "seqs", "num_rows",
                                           "max_blocks", "tokens", "block_size", "num_blocks")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(seqs=-1), api.PA_ERR_INVALID_ARG),
    (dict(tokens=-1), api.PA_ERR_INVALID_ARG),
    (dict(capacity=-1), api.PA_ERR_INVALID_ARG),
    (dict(num_rows=0), api.PA_ERR_INVALID_ARG),
    (dict(block_size=12), api.PA_ERR_UNSUPPORTED),
    (dict(seqs=8193), api.PA_ERR_UNSUPPORTED),
    (dict(num_rows=(1 << 18) + 1), api.PA_ERR_UNSUPPORTED),
    (dict(max_blocks=1 << 28), api.PA_ERR_UNSUPPORTED),
    (dict(start=None), api.PA_ERR_INVALID_ARG),
    (dict(rows=None), api.PA_ERR_INVALID_ARG),
    (dict(slots=None), api.PA_ERR_INVALID_ARG),
    (dict(count=None), api.PA_ERR_INVALID_ARG),                   # a list without its count
    (dict(row_tables=A + 4), api.PA_ERR_MISALIGNED),
    (dict(slots=A + 4), api.PA_ERR_MISALIGNED),
    (dict(new=A + 2), api.PA_ERR_MISALIGNED),
])
def test_plan_host_checks(kw, want):
    assert plan(**kw) == want


def release(**kw):
    a = dict(rows=A, n=3, row_tables=A, row_blocks=A, num_rows=8, max_blocks=16, free=A, count=A, capacity=10)
    a.update(kw)
    return L.pa_release_rows(*[a[n] for n in ("rows", "n", "row_tables", "row_blocks", "num_rows", "max_blocks", "free",
                                              "count", "capacity")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), api.PA_OK),
    (dict(n=-1), api.PA_ERR_INVALID_ARG),
    (dict(n=8193), api.PA_ERR_UNSUPPORTED),
    (dict(free=None), api.PA_ERR_INVALID_ARG),
    (dict(rows=A + 2), api.PA_ERR_MISALIGNED),
])
def test_release_host_checks(kw, want):
    assert release(**kw) == want


def test_workspace_size_of_nothing_is_zero():
    f = L.pa_decode_multi_workspace_size
    assert f(0, 32, 8, 128) == f(4, 32, 0, 128) == f(4, 4, 8, 128) == f(4, 32, 8, 0) == 0


def test_binding_refuses_host_tensors_before_any_call(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.pa_plan_step(z(2, 4), z(2), z(3), z(5), z(5, dt=torch.int64), z(2), z(2), z(8), z(8, 4), z(8), None, None,
                         16, 64, stream=0)
    with pytest.raises(TypeError, match="block_tables must be torch.int32, got torch.int64"):
        api.pa_plan_step(z(2, 4, dt=torch.int64), z(2), z(3), z(5), z(5, dt=torch.int64), z(2), z(2), z(8), z(8, 4), z(8),
                         None, None, 16, 64, stream=0)
    with pytest.raises(TypeError, match="seq_rows must be a torch.Tensor"):
        api.pa_plan_step(z(2, 4), z(2), z(3), z(5), z(5, dt=torch.int64), [0, 1], z(2), z(8), z(8, 4), z(8), None, None,
                         16, 64, stream=0)
    with pytest.raises(ValueError, match="row_tables must have 2 dimensions"):
        api.pa_release_rows(z(2), z(8), z(8), z(9), z(1), stream=0)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="go together"):
        api.pa_qk_norm_rope_cache(b(1, 4, 64), b(2, 2, 16, 64), b(2, 2, 16, 64), b(1, 4, 64), b(1, 2, 64), b(1, 2, 64),
                                  z(1), z(1, dt=torch.int64), z(9, 64, dt=torch.float32), k_scale=0.1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.pa_decode_multi(b(1, 4, 64), b(1, 4, 64), b(2, 2, 16, 64), b(2, 2, 16, 64), z(1, 3), z(2), z(1), 1, 16,
                            0.125, 4, 2, 64, 48, workspace=z(16, dt=torch.uint8), stream=0)


def test_rope_table_is_the_angles_cosines_and_sines():
    t = api.rope_table(1000, 64, base=500000.0, device="cpu")
    assert t.shape == (1000, 64) and t.dtype == torch.float32
    angle = torch.tensor(999.0, dtype=torch.float64) * 500000.0 ** (-2 * 31 / 64.0)
    assert t[999, 31] == angle.cos().float() and t[999, 63] == angle.sin().float()


class _Handle:
    """A stream object of another library: its handle alone."""

    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


@pytest.mark.parametrize("given,used", [
    (None, "current"), (0x5000, 0x5000), (_Handle(0x6000), 0x6000), (0, "default"), (1, "default"), (_Handle(0), "default"),
])
def test_a_workspace_of_the_calls_own_comes_from_the_streams_pool(monkeypatch, given, used):
    """Memory of another stream's pool could still be in use there when the call writes it."""
    current, seen = ["current"], []

    class use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(api, "_current_handle", lambda dev: 77)
    monkeypatch.setattr(api, "decode_multi_workspace", lambda *a: seen.append(current[-1]) or torch.zeros(16))
    monkeypatch.setattr(api._step_calls, "decode_multi", lambda *a: seen.append(a[-1]) or api.PA_OK)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    assert api.pa_decode_multi(q, q, q, q, q, q, q, 1, 16, 0.125, 4, 2, 64, 48, stream=given) == api.PA_OK
    handle = 77 if given is None else getattr(given, "cuda_stream", given)
    assert seen == [used, handle] and current == ["current"]


def test_a_workspace_of_its_own_is_refused_on_the_per_thread_stream(monkeypatch):
    """One handle for a stream of every thread: no pool is ordered with it."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="per-thread"):
        api.pa_decode_multi(*[None] * 7, 1, 16, 0.125, 4, 2, 64, 48, stream=2)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_rope_in_place_of_a_strided_q_is_refused(fp8):
    assert rope(fp8, qs=6144) == api.PA_ERR_INVALID_ARG
    assert rope(fp8, qs=6144, tokens=0) == api.PA_OK


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("name", ["tables", "start", "ctx"])
def test_multi_takes_aligned_lengths_and_tables_only(fp8, name):
    assert multi(fp8, **{name: A + 2}) == api.PA_ERR_MISALIGNED
