"""CPU tests of the operators around the recurrence: the fp64 oracle's gradients against central differences of its
forward definitions, the frequency tables, and the refusals of the C ABI (before anything touches a device)."""
import math
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from kda_gated_delta_chunk_amd import _lib
from oracle import layers as ol

ROOT = Path(__file__).resolve().parent.parent
INVALID, UNSUP, WS_SMALL = 1, 2, 3
A = 1 << 20  # a 16-byte aligned address that is never read


def _rand(*shape, seed=0, std=1.0):
    return std * torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


# ------------------------------------------------------------------------------------------ the oracle's gradients
def _differences(f, x, h=1e-5):
    """Central differences of the scalar f in every entry of x (O(h^2) = 1e-10 of the third derivative, plus the
    rounding 1e-16 |f| / h = 1e-11 |f|)."""
    out = torch.zeros_like(x)
    flat, o = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = f()
        flat[i] = keep - h
        o[i] = (up - f()) / (2 * h)
        flat[i] = keep
    return out


@pytest.mark.parametrize("cu", [None, [0, 2, 2, 5]])
def test_hd_gradients_against_differences(cu):
    B, T, H, Hk, K, V = 1, 5, 4, 2, 3, 2
    N = B if cu is None else len(cu) - 1
    cu = None if cu is None else torch.tensor(cu)
    q, k, v = _rand(B, T, Hk, K, seed=1), _rand(B, T, Hk, K, seed=2), _rand(B, T, H, V, seed=3)
    g, S0 = -_rand(B, T, H, seed=4).exp(), _rand(N, H, K, V, seed=5)
    do, dS = _rand(B, T, H, V, seed=6), _rand(N, H, K, V, seed=7)

    def loss():
        o, S = ol.hd_forward(q, k, v, g, S0, cu, 0.7)
        return float((o * do).sum() + (S * dS).sum())

    grads = ol.hd_backward(q, k, v, g, do, S0, dS, cu, 0.7)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dS0", S0)):
        assert torch.allclose(grads[name], _differences(loss, x), atol=1e-7, rtol=1e-7), name


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("gate", [True, False])
def test_norm_gradients_against_differences(center, gate):
    x, w, b = _rand(3, 2, 5, seed=1), _rand(2, 5, seed=2), _rand(2, 5, seed=3)
    z, dy = (_rand(3, 2, 5, seed=4) if gate else None), _rand(3, 2, 5, seed=5)

    def loss():
        return float((ol.norm_forward(x, w, b, z, 1e-3, center) * dy).sum())

    grads = ol.norm_backward(dy, x, w, b, z, 1e-3, center)
    for name, p in (("dx", x), ("dweight", w), ("dbias", b), ("do_gate", z)):
        if p is not None:
            assert torch.allclose(grads[name], _differences(loss, p), atol=1e-7, rtol=1e-7), name


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_orthogonal_and_its_inverse_the_gradient(layout):
    x, dy = _rand(7, 2, 10, seed=1), _rand(7, 2, 10, seed=2)
    f, pos = kda.rotary_freqs(6, device="cpu"), torch.arange(7) * 1000003
    y = ol.rotate(x, f, pos, layout)
    assert torch.allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-12)
    assert torch.allclose(ol.rotate(y, f, pos, layout, inverse=True), x, atol=1e-12)
    # <dy, rotate x> = <rotate back dy, x>
    assert torch.allclose((dy * y).sum(), (ol.rotate(dy, f, pos, layout, inverse=True) * x).sum(), rtol=1e-12)
    # a pair turns by the difference of two positions: scores depend on distances only
    a, b = ol.rotate(x, f, pos, layout), ol.rotate(x, f, pos + 12345, layout)
    assert torch.allclose(a[0, 0] @ a[3, 0], b[0, 0] @ b[3, 0], atol=1e-9)


def test_rotary_freqs():
    f = kda.rotary_freqs(8, base=100.0, device="cpu")
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75],
                                                                       dtype=torch.float64), rtol=1e-15)
    assert torch.equal(kda.rotary_freqs(8, scaling="linear", factor=4.0, device="cpu"),
                       kda.rotary_freqs(8, device="cpu") / 4)
    p = kda.rotary_freqs(64, scaling="by_parts", factor=8.0, original_context=4096, device="cpu")
    f = kda.rotary_freqs(64, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(p[turns >= 32], f[turns >= 32]) and torch.allclose(p[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    assert bool(((p <= f) & (p >= f / 8)).all()) and bool((p[1:] < p[:-1]).all())
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=0.0), dict(rot_dim=8, factor=-1.0),
                dict(rot_dim=8, scaling="dynamic"), dict(rot_dim=8, scaling="by_parts")):
        with pytest.raises(ValueError):
            kda.rotary_freqs(**bad, device="cpu")


# ------------------------------------------------------------------------------------------ refusals of the C ABI
M = 1 << 24  # ranges in the calls below are smaller


def _hd_fwd(**kw):
    a = dict(q=A, k=A + M, v=A + 2 * M, g=A + 3 * M, S0=None, cu=None, B=1, T=64, H=4, Hk=2, K=32, V=64, N=1, io=1,
             decay=0, scale=1.0, o=A + 4 * M, Sf=A + 5 * M, ws=A + 6 * M, wsb=1 << 40, stream=None)
    a.update(kw)
    return _lib.load().kda_hd_chunk_fwd(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(g=None), INVALID), (dict(o=None), INVALID),
    (dict(k=A + M + 8), INVALID), (dict(S0=A + 7 * M + 4), INVALID), (dict(cu=A + 7 * M + 2), INVALID),
    (dict(g=A + 3 * M + 1), INVALID), (dict(g=A + 3 * M + 2, decay=1), INVALID),
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID), (dict(Hk=3), INVALID),
    (dict(Hk=8), INVALID), (dict(N=2), INVALID), (dict(B=2, N=2, cu=A + 7 * M), INVALID),
    (dict(io=2), INVALID), (dict(decay=2), INVALID), (dict(decay=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(T=1 << 31), INVALID), (dict(T=1 << 30, B=1 << 30, N=1 << 30), INVALID),
    (dict(o=A), INVALID), (dict(o=A + M + 16), INVALID),  # overlaps an input, also in part
    (dict(S0=A + 7 * M, Sf=A + 7 * M), INVALID), (dict(ws=A + 2 * M), INVALID), (dict(Sf=A + 4 * M), INVALID),
    (dict(K=48), UNSUP), (dict(V=256), UNSUP),
    (dict(ws=None), WS_SMALL), (dict(wsb=10), WS_SMALL), (dict(wsb=100, cu=A + 7 * M, N=3), WS_SMALL),
])
def test_hd_chunk_fwd_rejects(kw, expect):
    assert _hd_fwd(**kw) == expect


def _hd_bwd(**kw):
    a = dict(q=A, k=A + M, v=A + 2 * M, g=A + 3 * M, S0=None, cu=None, do=A + 4 * M, dS=None, B=1, T=64, H=4, Hk=2,
             K=32, V=64, N=1, io=1, decay=0, scale=1.0, dq=A + 5 * M, dk=A + 6 * M, dv=A + 7 * M, dg=A + 8 * M,
             dS0=A + 9 * M, ws=A + 10 * M, wsb=1 << 40, stream=None)
    a.update(kw)
    return _lib.load().kda_hd_chunk_bwd(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(do=None), INVALID), (dict(dq=None), INVALID), (dict(dv=A + 7 * M + 2), INVALID),
    (dict(dg=A + 8 * M + 1), INVALID), (dict(dq=A + 6 * M), INVALID), (dict(dv=A + 4 * M), INVALID),
    (dict(dg=A + 3 * M), INVALID), (dict(dS=A + 9 * M), INVALID), (dict(Hk=3), INVALID), (dict(N=4), INVALID),
    (dict(decay=1), UNSUP), (dict(K=16), UNSUP), (dict(wsb=256), WS_SMALL), (dict(ws=None), WS_SMALL),
])
def test_hd_chunk_bwd_rejects(kw, expect):
    assert _hd_bwd(**kw) == expect


def _hd_dec(**kw):
    a = dict(q=A, k=A + M, v=A + 2 * M, g=A + 3 * M, S=A + 4 * M, o=A + 5 * M, N=4, H=4, Hk=2, K=32, V=64, io=1,
             decay=0, scale=1.0, stream=None)
    a.update(kw)
    return _lib.load().kda_hd_decode_step(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(S=None), INVALID), (dict(v=A + 2 * M + 2), INVALID), (dict(S=A + 2 * M), INVALID), (dict(o=A + 4 * M), INVALID),
    (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=3), INVALID), (dict(io=5), INVALID), (dict(decay=3), INVALID),
    (dict(N=1 << 30, H=4), INVALID), (dict(K=256), UNSUP), (dict(V=16), UNSUP), (dict(N=0, S=None, q=None), 0),
])
def test_hd_decode_rejects(kw, expect):
    assert _hd_dec(**kw) == expect


def test_hd_workspace_bytes():
    w = kda.hd_workspace_bytes
    assert w(1, 64, 4, 32, 64, 1, Hk=2) > 0 and w(1, 64, 4, 48, 64, 1) == 0 and w(1, 64, 4, 32, 64, 2) == 0
    assert w(1, 64, 4, 32, 64, 1, Hk=3) == 0 and w(1, 0, 4, 32, 64, 1) > 0
    # few heads over many tokens: segments, each with a state
    assert w(1, 1 << 20, 1, 128, 128, 1) >= 128 * 128 * 4 * 2
    assert w(1, 1 << 20, 1, 128, 128, 1, packed=True) > 0
    b = kda.hd_bwd_workspace_bytes
    assert b(1, 64, 4, 32, 64, 1) > 0 and b(1, 64, 4, 32, 60, 1) == 0
    assert b(1, 4096, 8, 128, 128, 1, Hk=4) > b(1, 4096, 8, 128, 128, 1)  # dq and dk per head, before their sums


def _rot(**kw):
    a = dict(q=A, k=A + M, f=A + 2 * M, pos=A + 3 * M, qo=A + 4 * M, ko=A + 5 * M, n=8, T=8, Hq=4, Hk=2, D=64, R=32,
             io=1, layout=0, inv=0, scale=1.0, stream=None)
    a.update(kw)
    return _lib.load().kda_rotary(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(f=None), INVALID), (dict(k=None), INVALID), (dict(ko=None), INVALID),
    (dict(q=A + 2), INVALID), (dict(f=A + 2 * M + 4), INVALID), (dict(pos=A + 3 * M + 2), INVALID),
    (dict(R=31), INVALID), (dict(R=66), INVALID), (dict(R=0), INVALID), (dict(D=0, R=0), INVALID), (dict(n=-1), INVALID),
    (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID), (dict(layout=2), INVALID), (dict(inv=2), INVALID),
    (dict(io=9), INVALID), (dict(scale=float("nan")), INVALID), (dict(pos=None, T=0), INVALID),
    (dict(qo=A + 64), INVALID),               # overlaps q without being q
    (dict(qo=A + M), INVALID),                # is k
    (dict(ko=A + 4 * M), INVALID),            # both results in one place
    (dict(qo=A + 3 * M), INVALID), (dict(D=514, R=32), UNSUP), (dict(n=0, q=None), 0),
])
def test_rotary_rejects(kw, expect):
    assert _rot(**kw) == expect


def _nf(**kw):
    a = dict(x=A, w=A + M, b=A + 2 * M, z=A + 3 * M, y=A + 4 * M, rows=6, G=3, C=33, eps=1e-5, center=1, io=1, stream=None)
    a.update(kw)
    return _lib.load().kda_layer_norm_fwd(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=A + 2), INVALID), (dict(w=A + M + 4), INVALID),
    (dict(y=A), INVALID), (dict(y=A + 3 * M), INVALID), (dict(rows=7), INVALID), (dict(rows=-3), INVALID),
    (dict(G=0), INVALID), (dict(C=0), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(center=2), INVALID), (dict(io=4), INVALID), (dict(C=16385), UNSUP),
    (dict(rows=0, x=None), 0),
])
def test_layer_norm_fwd_rejects(kw, expect):
    assert _nf(**kw) == expect


def _nb(**kw):
    a = dict(dy=A, x=A + M, w=A + 2 * M, b=A + 3 * M, z=A + 4 * M, dx=A + 5 * M, dw=A + 6 * M, db=A + 7 * M, dz=A + 8 * M,
             rows=6, G=3, C=33, eps=1e-5, center=1, io=1, ws=A + 9 * M, wsb=1 << 40, stream=None)
    a.update(kw)
    return _lib.load().kda_layer_norm_bwd(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dz=None), INVALID), (dict(dx=A), INVALID),
    (dict(dx=A + M), INVALID), (dict(dw=A + 7 * M), INVALID), (dict(dz=A + 4 * M), INVALID), (dict(rows=5), INVALID),
    (dict(ws=A + 5 * M), INVALID), (dict(wsb=8), WS_SMALL), (dict(ws=None), WS_SMALL), (dict(C=20000), UNSUP),
])
def test_layer_norm_bwd_rejects(kw, expect):
    assert _nb(**kw) == expect


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 3, 32)
    for f in (lambda: kda.hd_decode_step(x, x, x, torch.zeros(2, 3), torch.zeros(2, 3, 32, 32)),
              lambda: kda.hd_chunk_fwd(x[None], x[None], x[None], torch.zeros(1, 2, 3)),
              lambda: kda.rotary(x, torch.zeros(4, dtype=torch.float64)), lambda: kda.layer_norm_fwd(x),
              lambda: kda.layer_norm_bwd(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(TypeError):
        kda.layer_norm_fwd(x.half())


# ------------------------------------------------------------------------------------------ host code under ASan
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANGXX = "/opt/rocm/lib/llvm/bin/clang++"


@pytest.mark.timeout(900)
@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX) and shutil.which("g++")),
                    reason="needs hipcc and ROCm clang++")
def test_layer_abi_under_address_sanitizer(tmp_path):
    """The layer operators' host code instrumented (-Xarch_host), their kernels as usual; the driver calls every entry
    point with rejected arguments, sweeps the workspace queries and, without a GPU, stops valid calls at the device
    check."""
    csrc = ROOT / "kda_gated_delta_chunk_amd" / "csrc"
    sources = ["kda_layer_api.hip", "kda_hd.hip", "kda_hd_fwd.hip", "kda_hd_grad_bf16.hip", "kda_hd_grad_fp32.hip",
               "kda_hd_decode.hip", "kda_rotary.hip", "kda_norm.hip"]
    flags = ["-O1", "-g", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Wno-unused-command-line-argument",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = [tmp_path / (s.rsplit(".", 1)[0] + ".o") for s in sources]
    cmds = [[HIPCC, *flags, "-c", str(csrc / s), "-o", str(o)] for s, o in zip(sources, objs)]
    main_o = tmp_path / "main.o"
    cmds.append([CLANGXX, "-O1", "-g", "-std=c++17", "-fsanitize=address", "-fno-omit-frame-pointer",
                 "-c", str(ROOT / "tests" / "sanitize" / "layers_main.cpp"), "-o", str(main_o)])

    def run(cmd, env=None):
        r = subprocess.run(list(map(str, cmd)), stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, env=env,
                           timeout=600)
        assert r.returncode == 0, "%s\n%s" % (" ".join(map(str, cmd)), r.stdout[-4000:])
        return r.stdout

    with ThreadPoolExecutor(max_workers=4) as ex:
        list(ex.map(run, cmds))
    exe = tmp_path / "layers_asan"
    run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", str(main_o), *map(str, objs), "-o", str(exe)])
    # with a GPU valid calls would run, on addresses that are none
    out = run([str(exe)] + ["refusals"] * (torch.cuda.device_count() > 0), env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1"))
    assert "all checks passed" in out
