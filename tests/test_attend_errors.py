"""Host-side refusals of the shaped attention, of rotation by several axes and
of the block-scaled appends: each is returned before anything is enqueued, so
stand-in addresses that nothing reads serve and no GPU is needed.  And the
binding's refusals of tensors.  CPU only."""

import ctypes

import pytest
import torch

from paged_kv_cache_124_gb300 import api

L = api._lib
A = 0x100000            # a 256-byte-aligned stand-in address (never dereferenced)
INF, NAN = float("inf"), float("nan")


def attend(scaled=False, **kw):
    a = dict(out=2 * A, out_dtype=api.PA_DTYPE_BF16, q=A, k=A, v=A, ks=A, vs=A, tables=A, start=A, ctx=A, visible=None, slopes=None,
             cap=0.0, block_size=16, scale=0.088, hq=32, hkv=8, d=128, num_seqs=4, tokens=16, most=4, max_blocks=8, num_blocks=64,
             max_ctx=128, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    scales = (a["ks"], a["vs"]) if scaled else ()
    fn = L.pa_attend_scaled if scaled else L.pa_attend
    return fn(a["out"], a["out_dtype"], a["q"], a["k"], a["v"], *scales, a["tables"], a["start"], a["ctx"], a["visible"], a["slopes"],
              a["cap"], a["block_size"], a["scale"], a["hq"], a["hkv"], a["d"], a["num_seqs"], a["tokens"], a["most"],
              a["max_blocks"], a["num_blocks"], a["max_ctx"], a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("most", [4, 700], ids=["few", "many"])
@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("kw,want", [
    (dict(num_seqs=0), api.PA_OK),
    (dict(tokens=0), api.PA_OK),
    (dict(num_seqs=-1), api.PA_ERR_INVALID_ARG),
    (dict(tokens=-1), api.PA_ERR_INVALID_ARG),
    (dict(most=0), api.PA_ERR_INVALID_ARG),
    (dict(max_ctx=-1), api.PA_ERR_INVALID_ARG),
    (dict(scale=NAN), api.PA_ERR_INVALID_ARG),
    (dict(scale=INF), api.PA_ERR_INVALID_ARG),
    (dict(cap=-1.0), api.PA_ERR_INVALID_ARG),
    (dict(cap=NAN), api.PA_ERR_INVALID_ARG),
    (dict(cap=INF), api.PA_ERR_INVALID_ARG),
    (dict(out_dtype=5), api.PA_ERR_INVALID_ARG),
    (dict(out=None), api.PA_ERR_INVALID_ARG),
    (dict(ctx=None), api.PA_ERR_INVALID_ARG),
    (dict(out=A), api.PA_ERR_INVALID_ARG),                        # in place of q
    (dict(block_size=64), api.PA_ERR_UNSUPPORTED),
    (dict(d=96), api.PA_ERR_UNSUPPORTED),
    (dict(hq=12), api.PA_ERR_UNSUPPORTED),
    (dict(hq=24), api.PA_ERR_UNSUPPORTED),                        # G = 3
    (dict(hq=256), api.PA_ERR_UNSUPPORTED),                       # G = 32
    (dict(num_blocks=1 << 30), api.PA_ERR_UNSUPPORTED),           # rows past 31 bits
    (dict(q=A + 8), api.PA_ERR_MISALIGNED),
    (dict(visible=A + 4), api.PA_ERR_MISALIGNED),
    (dict(slopes=A + 2), api.PA_ERR_MISALIGNED),
    (dict(tables=A + 2), api.PA_ERR_MISALIGNED),
    (dict(ws=None), api.PA_ERR_WORKSPACE),
    (dict(ws=A + 16), api.PA_ERR_WORKSPACE),
])
def test_attend_host_checks(most, scaled, kw, want):
    assert attend(scaled, **dict(dict(most=most), **kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(d=64), api.PA_ERR_UNSUPPORTED),
    (dict(ks=None), api.PA_ERR_INVALID_ARG),
    (dict(vs=None), api.PA_ERR_INVALID_ARG),
])
def test_scaled_attend_host_checks(kw, want):
    assert attend(True, **kw) == want


def test_attend_workspace_size_of_nothing_is_zero():
    f = L.pa_attend_workspace_size
    good = [2, 4, 8, 16, 32, 8, 128, 0]
    for i in range(7):
        bad = list(good)
        bad[i] = 0
        assert f(*bad) == 0
    assert f(2, 4, 8, 16, 4, 8, 128, 0) == 0


def axes_of(*x):
    return (ctypes.c_int8 * 64)(*x)


def mrope(kind="bf16", **kw):
    a = dict(q_out=A, kc=A, vc=A, ks_=A, vs_=A, q=A, k=A, v=A, qs=4096, ks=1024, vs=1024, qw=A, kw=A, eps=1e-6, cs=A, maxpos=100,
             rot=128, inter=0, pos=A, num=3, axes=axes_of(0, 1, 2), slots=A, tokens=4, hq=32, hkv=8, d=128, block_size=16,
             num_blocks=64)
    a.update(kw)
    if a["axes"] is not None:
        a["axes"] = ctypes.cast(a["axes"], ctypes.c_void_p)
    names = ["q_out", "kc", "vc"] + (["ks_", "vs_"] if kind == "scaled" else []) + [
        "q", "k", "v", "qs", "ks", "vs", "qw", "kw", "eps", "cs", "maxpos", "rot", "inter", "pos", "num", "axes", "slots", "tokens",
        "hq", "hkv", "d", "block_size", "num_blocks"]
    args = [a[n] for n in names]
    if kind == "fp8":
        return L.pa_qk_norm_mrope_cache_fp8(*args, 0.1, 0.1, None, None)
    return (L.pa_qk_norm_rope_cache_scaled if kind == "scaled" else L.pa_qk_norm_mrope_cache)(*args, None, None)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "scaled"])
@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), api.PA_OK),
    (dict(tokens=-1), api.PA_ERR_INVALID_ARG),
    (dict(num=-1), api.PA_ERR_INVALID_ARG),
    (dict(num=5), api.PA_ERR_UNSUPPORTED),
    (dict(axes=None), api.PA_ERR_INVALID_ARG),
    (dict(axes=axes_of(0, 3)), api.PA_ERR_INVALID_ARG),           # an axis that is not there
    (dict(axes=axes_of(0, -1)), api.PA_ERR_INVALID_ARG),
    (dict(maxpos=0), api.PA_ERR_INVALID_ARG),
    (dict(eps=-1.0), api.PA_ERR_INVALID_ARG),
    (dict(eps=NAN), api.PA_ERR_INVALID_ARG),
    (dict(qw=None), api.PA_ERR_INVALID_ARG),                      # one gain without the other
    (dict(cs=None), api.PA_ERR_INVALID_ARG),
    (dict(pos=None), api.PA_ERR_INVALID_ARG),
    (dict(q_out=None), api.PA_ERR_INVALID_ARG),
    (dict(hq=0), api.PA_ERR_INVALID_ARG),
    (dict(qs=4088), api.PA_ERR_INVALID_ARG),                      # tokens would overlap
    (dict(qs=6144), api.PA_ERR_INVALID_ARG),                      # in place of a strided q
    (dict(rot=0), api.PA_ERR_UNSUPPORTED),
    (dict(rot=24), api.PA_ERR_UNSUPPORTED),
    (dict(rot=144), api.PA_ERR_UNSUPPORTED),
    (dict(d=80), api.PA_ERR_UNSUPPORTED),
    (dict(block_size=4), api.PA_ERR_UNSUPPORTED),
    (dict(tokens=1 << 26), api.PA_ERR_UNSUPPORTED),               # rows past 31 bits
    (dict(ks=1028), api.PA_ERR_MISALIGNED),
    (dict(k=A + 2), api.PA_ERR_MISALIGNED),
    (dict(pos=A + 2), api.PA_ERR_MISALIGNED),
    (dict(slots=A + 4), api.PA_ERR_MISALIGNED),
])
def test_mrope_host_checks(kind, kw, want):
    assert mrope(kind, **kw) == want


def test_mrope_needs_axes_and_scaled_scales():
    assert mrope("bf16", num=0) == mrope("fp8", num=0) == api.PA_ERR_INVALID_ARG
    assert mrope("scaled", ks_=None) == mrope("scaled", vs_=None) == api.PA_ERR_INVALID_ARG


def append(**kw):
    a = dict(kc=A, vc=A, ks_=A, vs_=A, k=A, v=A, ks=1024, vs=1024, slots=A, tokens=4, hkv=8, d=128, block_size=16, num_blocks=64)
    a.update(kw)
    return L.pa_reshape_and_cache_scaled(*[a[n] for n in ("kc", "vc", "ks_", "vs_", "k", "v", "ks", "vs", "slots", "tokens", "hkv", "d",
                                                          "block_size", "num_blocks")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), api.PA_OK),
    (dict(tokens=-1), api.PA_ERR_INVALID_ARG),
    (dict(hkv=0), api.PA_ERR_INVALID_ARG),
    (dict(num_blocks=0), api.PA_ERR_INVALID_ARG),
    (dict(vc=None), api.PA_ERR_INVALID_ARG),
    (dict(ks_=None), api.PA_ERR_INVALID_ARG),
    (dict(slots=None), api.PA_ERR_INVALID_ARG),
    (dict(ks=1016), api.PA_ERR_INVALID_ARG),
    (dict(d=32), api.PA_ERR_UNSUPPORTED),
    (dict(block_size=64), api.PA_ERR_UNSUPPORTED),
    (dict(vs=1028), api.PA_ERR_MISALIGNED),
    (dict(v=A + 8), api.PA_ERR_MISALIGNED),
])
def test_append_host_checks(kw, want):
    assert append(**kw) == want


def test_rope_axes():
    assert list(api.rope_axes([2, 1, 3])) == [0, 0, 1, 2, 2, 2]
    assert list(api.rope_axes([2, 1, 3], interleaved=True)) == [0, 1, 2, 0, 2, 2]
    for bad in ([], [1, -1]):
        with pytest.raises(ValueError):
            api.rope_axes(bad)


def test_binding_refuses_tensors_before_any_call(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    b = lambda *s: z(*s, dt=torch.bfloat16)  # noqa: E731
    u = lambda *s: z(*s, dt=torch.uint8)  # noqa: E731
    args = (b(1, 4, 64), b(1, 4, 64), b(2, 2, 16, 64), b(2, 2, 16, 64), z(1, 3), z(2), z(1), 1, 16, 0.125, 4, 2, 64, 48)
    with pytest.raises(ValueError, match="go together"):
        api.pa_attend(*args, k_scales=u(2, 2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.pa_attend(*args, workspace=u(16), stream=0)
    with pytest.raises(TypeError, match="axes must be"):
        api.pa_qk_norm_mrope_cache(*[None] * 6, None, None, None, None, stream=0)
    with pytest.raises(TypeError, match="k_scales and v_scales"):
        api.pa_qk_norm_rope_cache_scaled(*[None] * 11, stream=0)
    with pytest.raises(ValueError, match="go together"):
        api.pa_qk_norm_mrope_cache(*[None] * 6, None, [0], None, None, k_scale=0.1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.pa_reshape_and_cache_scaled(u(2, 2, 16, 64), u(2, 2, 16, 64), u(2, 2), u(2, 2), b(1, 2, 64), b(1, 2, 64),
                                        z(1, dt=torch.int64), stream=0)


def test_refusals_name_the_call_that_was_made(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)  # noqa: E731
    b = lambda *s: z(*s, dt=torch.bfloat16)  # noqa: E731
    rope = (b(1, 4, 64), b(1, 2, 64), b(1, 2, 64), z(2, 1, dt=torch.int32))
    with pytest.raises(ValueError, match="^pa_qk_norm_rope_cache_scaled: "):
        api.pa_qk_norm_rope_cache_scaled(b(1, 4, 64), z(2, 2, 16, 64), z(2, 2, 16, 64), z(2, 2), z(2, 2), *rope,
                                         z(1, dt=torch.int64), z(9, 64, dt=torch.float32), axes=[0] * 32, stream=0)
    with pytest.raises(ValueError, match="^pa_qk_norm_mrope_cache: "):
        api.pa_qk_norm_mrope_cache(b(1, 4, 64), b(2, 2, 16, 64), b(2, 2, 16, 64), *rope, [0] * 32, z(1, dt=torch.int64),
                                   z(9, 64, dt=torch.float32), stream=0)


class _Handle:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


@pytest.mark.parametrize("given,used", [(None, "current"), (0x5000, 0x5000), (_Handle(0x6000), 0x6000), (0, "default")])
def test_a_workspace_of_the_calls_own_comes_from_the_streams_pool(monkeypatch, given, used):
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
    monkeypatch.setattr(api, "attend_workspace", lambda *a: seen.append(current[-1]) or torch.zeros(16))
    monkeypatch.setattr(api._step_calls, "attend", lambda *a: seen.append(a[-1]) or api.PA_OK)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    assert api.pa_attend(q, q, q, q, q, q, q, 1, 16, 0.125, 4, 2, 64, 48, stream=given) == api.PA_OK
    assert seen == [used, 77 if given is None else getattr(given, "cuda_stream", given)] and current == ["current"]
