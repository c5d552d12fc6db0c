"""CPU tests of the gated delta rule with one decay per head, the rotary positions with several axes and the checkpoints
in 8 bits: the fp64 oracle against central differences and against other oracles, and the refusals of the C ABI (before
anything touches a device)."""
import os
import shutil
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

import pytest
import torch

import kda_gated_delta_chunk_amd as kda
import oracle
from kda_gated_delta_chunk_amd import _lib
from oracle import delta as od
from oracle import layers as ol
from tests.test_layers_cpu import _differences, _rand
from tests.test_sanitizers_cpu import CLANGXX, HIPCC, _run

ROOT = Path(__file__).resolve().parent.parent
INVALID, UNSUP, WS_SMALL = 1, 2, 3
A = 1 << 20  # a 16-byte aligned address that is never read


# ------------------------------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("cu", [None, [0, 2, 2, 5]])
def test_gd_gradients_against_differences(cu):
    B, T, H, Hk, K, V = 1, 5, 4, 2, 3, 2
    N = B if cu is None else len(cu) - 1
    cu = None if cu is None else torch.tensor(cu)
    q, k, v = _rand(B, T, Hk, K, seed=1), _rand(B, T, Hk, K, seed=2, std=0.6), _rand(B, T, H, V, seed=3)
    g, beta = -_rand(B, T, H, seed=4).exp(), torch.sigmoid(_rand(B, T, H, seed=8))
    S0, do, dS = _rand(N, H, K, V, seed=5), _rand(B, T, H, V, seed=6), _rand(N, H, K, V, seed=7)

    def loss():
        o, S = od.gd_forward(q, k, v, g, beta, S0, cu, 0.7)
        return float((o * do).sum() + (S * dS).sum())

    grads = od.gd_backward(q, k, v, g, beta, do, S0, dS, cu, 0.7)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta), ("dS0", S0)):
        assert torch.allclose(grads[name], _differences(loss, x), atol=1e-7, rtol=1e-7), name


def test_gd_is_kda_with_one_decay_for_all_channels():
    """The C oracle of the recurrence with a decay per channel, given the same number for every channel."""
    B, T, H, K, V = 2, 37, 3, 16, 8
    q, k, v = _rand(B, T, H, K, seed=11), _rand(B, T, H, K, seed=12, std=0.25), _rand(B, T, H, V, seed=13)
    g, beta, S0 = -_rand(B, T, H, seed=14).exp(), torch.sigmoid(_rand(B, T, H, seed=15)), _rand(B, H, K, V, seed=16)
    # inputs that the C oracle takes in fp32: the same numbers on both sides
    q, k, v, g, beta, S0 = (x.float() for x in (q, k, v, g, beta, S0))
    o, S = od.gd_forward(q, k, v, g, beta, S0)
    ro, rS = oracle.chunk_fwd(q, k, v, g[..., None].expand(B, T, H, K).contiguous(), beta, S0=S0)
    assert torch.allclose(o, torch.as_tensor(ro).double(), atol=1e-12, rtol=1e-12)
    assert torch.allclose(S, torch.as_tensor(rS).double(), atol=1e-12, rtol=1e-12)


def test_gd_without_writing_strength_only_decays():
    q, k, v = _rand(1, 6, 1, 4, seed=21), _rand(1, 6, 1, 4, seed=22), _rand(1, 6, 1, 4, seed=23)
    g, S0 = -_rand(1, 6, 1, seed=24).exp(), _rand(1, 1, 4, 4, seed=25)
    o, S = od.gd_forward(q, k, v, g, torch.zeros_like(g), S0)
    assert torch.allclose(S, torch.exp(g.sum()) * S0, atol=1e-14)
    z = S0 * torch.exp(g[0, :3].sum())
    assert torch.allclose(o[0, 2, 0], (q[0, 2, 0][:, None] * z[0, 0]).sum(0), atol=1e-14)


def test_gd_recalls_what_was_written():
    """beta = 1 and keys of length one: reading with the key just written gives its value, whatever was there."""
    k = torch.nn.functional.normalize(_rand(1, 9, 1, 6, seed=31), dim=-1)
    v, S0 = _rand(1, 9, 1, 5, seed=32), _rand(1, 1, 6, 5, seed=33)
    o, _ = od.gd_forward(k, k, v, torch.zeros(1, 9, 1), torch.ones(1, 9, 1), S0)
    assert torch.allclose(o, v, atol=1e-13)


def test_axes_of_one_are_the_plain_rotation():
    x, freqs = _rand(2, 5, 3, 12, seed=41), kda.rotary_freqs(8, device="cpu")
    pos = torch.arange(10).reshape(2, 5) * 7 - 11
    for layout in ("half", "interleaved"):
        a = ol.rotate(x, freqs, pos, layout, inverse=True, scale=1.5)
        b = ol.rotate_axes(x, freqs, torch.zeros(4, dtype=torch.int32), pos[None], layout, inverse=True, scale=1.5)
        assert torch.allclose(a, b, atol=1e-13)


def test_sections():
    assert kda.rotary_sections([2, 3, 1], device="cpu").tolist() == [0, 0, 1, 1, 1, 2]
    assert kda.rotary_sections([2, 3, 1], "turns", device="cpu").tolist() == [0, 1, 2, 0, 1, 1]
    assert kda.rotary_sections([0, 2], "turns", device="cpu").tolist() == [1, 1]
    for bad in ([], [0, 0], [-1, 2]):
        with pytest.raises(ValueError):
            kda.rotary_sections(bad, device="cpu")
    with pytest.raises(ValueError):
        kda.rotary_sections([1], "rows", device="cpu")


def test_saved_values_are_within_half_a_step():
    x = _rand(7, 300, seed=51).float()
    x[2, :128] = 0.0
    codes, scales = ol.save8(x)
    assert scales.shape == (7, 3) and float(scales[2, 0]) == 0.0 and bool((codes[2, :128] == 0).all())
    step = scales.repeat_interleave(128, dim=1)[:, :300]
    assert bool(((ol.restore8(codes, scales) - x.double()).abs() <= step * 0.5 * (1 + 1e-12)).all())
    assert int(codes.abs().max()) == 127


# ------------------------------------------------------------------------------------------ refusals
def _fwd(lib, **kw):
    a = dict(q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, S0=0, cu=0, B=1, T=64, H=4, Hk=2, K=32, V=64, N=1, io=1, gates=1,
             scale=1.0, o=6 * A, S=7 * A, ws=8 * A, wsb=1 << 19)
    a.update(kw)
    return lib.kda_gd_chunk_fwd(*(a[n] for n in ("q", "k", "v", "g", "beta", "S0", "cu", "B", "T", "H", "Hk", "K", "V", "N",
                                                 "io", "gates", "scale", "o", "S", "ws", "wsb")), None)


def _bwd(lib, **kw):
    a = dict(q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, S0=0, cu=0, do=6 * A, dS=0, B=1, T=64, H=4, Hk=2, K=32, V=64, N=1,
             io=1, gates=1, scale=1.0, dq=7 * A, dk=8 * A, dv=9 * A, dg=10 * A, dbeta=11 * A, dS0=12 * A, ws=16 * A,
             wsb=1 << 23)
    a.update(kw)
    return lib.kda_gd_chunk_bwd(*(a[n] for n in ("q", "k", "v", "g", "beta", "S0", "cu", "do", "dS", "B", "T", "H", "Hk",
                                                 "K", "V", "N", "io", "gates", "scale", "dq", "dk", "dv", "dg", "dbeta",
                                                 "dS0", "ws", "wsb")), None)


def _step(lib, **kw):
    a = dict(q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, S=6 * A, o=7 * A, N=3, H=4, Hk=2, K=32, V=64, io=1, gates=1,
             scale=1.0)
    a.update(kw)
    return lib.kda_gd_decode_step(*(a[n] for n in ("q", "k", "v", "g", "beta", "S", "o", "N", "H", "Hk", "K", "V", "io",
                                                   "gates", "scale")), None)


BAD = [(dict(q=0), INVALID), (dict(g=0), INVALID), (dict(beta=0), INVALID), (dict(q=A + 8), INVALID),
       (dict(g=4 * A + 1), INVALID), (dict(beta=5 * A + 2, gates=0), INVALID), (dict(H=3), INVALID), (dict(Hk=0), INVALID),
       (dict(K=48), UNSUP), (dict(V=256), UNSUP), (dict(io=2), INVALID), (dict(io=0, gates=1), INVALID),
       (dict(gates=2), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID)]
BAD_CHUNKED = [(dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(N=2), INVALID),
               (dict(B=2, cu=20 * A), INVALID), (dict(cu=20 * A + 2), INVALID), (dict(H=1 << 16, Hk=1 << 16), INVALID),
               (dict(N=1 << 26, cu=20 * A), INVALID), (dict(ws=0), WS_SMALL), (dict(wsb=16), WS_SMALL), (dict(S0=7 * A), INVALID)]


@pytest.mark.parametrize("kw,status", BAD + BAD_CHUNKED + [(dict(o=0), INVALID), (dict(o=A), INVALID),
                                                           (dict(S=3 * A), INVALID), (dict(S=8 * A), INVALID)])
def test_fwd_refusals(kw, status):
    assert _fwd(_lib.load(), **kw) == status


@pytest.mark.parametrize("kw,status", BAD + BAD_CHUNKED + [
    (dict(do=0), INVALID), (dict(dq=0), INVALID), (dict(dg=0), INVALID), (dict(dbeta=0), INVALID), (dict(dv=6 * A), INVALID),
    (dict(dbeta=10 * A), INVALID), (dict(dS0=16 * A), INVALID), (dict(dS=12 * A), INVALID), (dict(dg=10 * A + 1), INVALID)])
def test_bwd_refusals(kw, status):
    assert _bwd(_lib.load(), **kw) == status


@pytest.mark.parametrize("kw,status", BAD + [(dict(N=-1), INVALID), (dict(N=1 << 27), INVALID), (dict(S=0), INVALID),
                                             (dict(o=3 * A), INVALID), (dict(S=A), INVALID), (dict(N=0, q=0), 0)])
def test_decode_refusals(kw, status):
    assert _step(_lib.load(), **kw) == status


def _axes(lib, **kw):
    a = dict(q=A, k=2 * A, f=3 * A, axes=4 * A, pos=5 * A, qo=6 * A, ko=7 * A, tokens=8, n=3, Hq=4, Hk=2, D=64, R=32, io=1,
             layout=0, inverse=0, scale=1.0)
    a.update(kw)
    return lib.kda_rotary_axes(*(a[n] for n in ("q", "k", "f", "axes", "pos", "qo", "ko", "tokens", "n", "Hq", "Hk", "D", "R",
                                                "io", "layout", "inverse", "scale")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), INVALID), (dict(axes=0), INVALID), (dict(pos=0), INVALID), (dict(f=0), INVALID), (dict(k=0), INVALID),
    (dict(n=0), INVALID), (dict(n=17), UNSUP), (dict(R=0), INVALID), (dict(R=33), INVALID), (dict(R=66), INVALID),
    (dict(D=1024, R=32), UNSUP), (dict(io=3), INVALID), (dict(layout=2), INVALID), (dict(inverse=2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(tokens=-1), INVALID), (dict(axes=4 * A + 2), INVALID), (dict(pos=6 * A), INVALID),
    (dict(qo=2 * A), INVALID), (dict(axes=7 * A), INVALID), (dict(tokens=0, q=0), 0), (dict(Hq=1 << 21), INVALID)])
def test_axes_refusals(kw, status):
    assert _axes(_lib.load(), **kw) == status


@pytest.mark.parametrize("fn", ["save", "restore"])
@pytest.mark.parametrize("kw,status", [
    (dict(x=0), INVALID), (dict(codes=0), INVALID), (dict(scales=0), INVALID), (dict(x=A + 2), INVALID),
    (dict(codes=2 * A + 4), INVALID), (dict(scales=3 * A + 2), INVALID), (dict(rows=-1), INVALID), (dict(C=0), INVALID),
    (dict(io=2), INVALID), (dict(codes=A), INVALID), (dict(scales=A), INVALID), (dict(rows=1 << 60, C=1 << 20), INVALID),
    (dict(rows=0, x=0), 0)])
def test_checkpoint_refusals(fn, kw, status):
    a = dict(x=A, codes=2 * A, scales=3 * A, rows=4, C=300, io=1)
    a.update(kw)
    first = (a["x"], a["codes"], a["scales"]) if fn == "save" else (a["codes"], a["scales"], a["x"])
    assert getattr(_lib.load(), "kda_checkpoint8_" + fn)(*first, a["rows"], a["C"], a["io"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=0), INVALID), (dict(scales=0), INVALID), (dict(dy=0), INVALID), (dict(dx=0), INVALID),
    (dict(scales=3 * A + 1), INVALID), (dict(dx=2 * A), INVALID), (dict(dweight=3 * A), INVALID), (dict(rows=7), INVALID),
    (dict(C=16385), UNSUP), (dict(eps=0.0), INVALID), (dict(gate=20 * A, dgate=0), INVALID), (dict(wsb=16), WS_SMALL),
    (dict(center=2), INVALID), (dict(io=5), INVALID)])
def test_norm_from_a_checkpoint_refusals(kw, status):
    a = dict(dy=A, codes=2 * A, scales=3 * A, weight=4 * A, bias=0, gate=0, dx=5 * A, dweight=6 * A, dbias=0, dgate=0,
             rows=6, groups=3, C=96, eps=1e-5, center=1, io=1, ws=8 * A, wsb=1 << 22)
    a.update(kw)
    assert _lib.load().kda_layer_norm_bwd_checkpoint8(*(a[n] for n in (
        "dy", "codes", "scales", "weight", "bias", "gate", "dx", "dweight", "dbias", "dgate", "rows", "groups", "C", "eps",
        "center", "io", "ws", "wsb")), None) == status


def test_workspace_queries():
    lib = _lib.load()
    for fn in (lib.kda_gd_chunk_fwd_workspace_bytes, lib.kda_gd_chunk_bwd_workspace_bytes):
        assert fn(1, 64, 4, 2, 32, 64, 1, 0, 1) > 0
        assert fn(1, 64, 4, 3, 32, 64, 1, 0, 1) == 0 and fn(1, 64, 4, 2, 40, 64, 1, 0, 1) == 0
        assert fn(1, 64, 4, 2, 32, 64, 1, 0, 2) == 0 and fn(2, 64, 4, 2, 32, 64, 2, 1, 1) == 0
        assert fn(1, 64, 4, 2, 32, 64, 3, 1, 1) >= fn(1, 64, 4, 2, 32, 64, 1, 1, 1) > 0
        assert fn(1, 0, 4, 2, 32, 64, 1, 0, 1) > 0
    assert kda.gd_workspace_bytes(1, 64, 4, 32, 64, 1, Hk=2) == lib.kda_gd_chunk_fwd_workspace_bytes(1, 64, 4, 2, 32, 64, 1, 0, 1)
    assert kda.gd_bwd_workspace_bytes(1, 64, 4, 32, 64, 1) == lib.kda_gd_chunk_bwd_workspace_bytes(1, 64, 4, 4, 32, 64, 1, 0, 1)


def test_host_tensors_are_refused():
    x, g = torch.zeros(1, 4, 2, 32), torch.zeros(1, 4, 2)
    for call in (lambda: kda.gd_chunk_fwd(x, x, x, g, g), lambda: kda.gd_chunk_bwd(x, x, x, g, g, x),
                 lambda: kda.gd_decode_step(x[0], x[0], x[0], g[0], g[0], torch.zeros(4, 2, 32, 32)),
                 lambda: kda.rotary_axes(x, kda.rotary_freqs(8, device="cpu"), torch.zeros(4, dtype=torch.int32),
                                         torch.zeros(1, 1, 4, dtype=torch.int32)),
                 lambda: kda.checkpoint8(x),
                 lambda: kda.restore8(kda.Checkpoint8(x.to(torch.int8), torch.zeros(1, 4, 2, 1), torch.float32)),
                 lambda: kda.layer_norm_bwd(x, kda.Checkpoint8(x.to(torch.int8), torch.zeros(1, 4, 2, 1), torch.float32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ------------------------------------------------------------------------------------------ host code under a sanitizer
@pytest.mark.timeout(900)
@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)) or shutil.which("gcc") is None,
                    reason="needs hipcc and ROCm clang++")
def test_host_code_under_address_sanitizer(tmp_path):
    csrc = ROOT / "kda_gated_delta_chunk_amd" / "csrc"
    sources = ["kda_gd_api.hip", "kda_gd.hip", "kda_gd_state.hip", "kda_gd_grad_bf16.hip", "kda_gd_grad_gates.hip",
               "kda_gd_grad_fp32.hip", "kda_gd_decode.hip", "kda_ckpt_api.hip", "kda_ckpt.hip", "kda_layer_api.hip",
               "kda_hd.hip", "kda_hd_fwd.hip", "kda_hd_grad_bf16.hip", "kda_hd_grad_fp32.hip", "kda_hd_decode.hip",
               "kda_rotary.hip", "kda_norm.hip"]
    flags = ["-O1", "-g", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Wno-unused-command-line-argument",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = [tmp_path / (s.rsplit(".", 1)[0] + ".o") for s in sources]
    cmds = [[HIPCC, *flags, "-c", str(csrc / s), "-o", str(o)] for s, o in zip(sources, objs)]
    main_o = tmp_path / "main.o"
    cmds.append([CLANGXX, "-O1", "-g", "-std=c++17", "-fsanitize=address", "-fno-omit-frame-pointer",
                 "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-c", str(ROOT / "tests" / "sanitize" / "delta_main.cpp"),
                 "-o", str(main_o)])
    with ThreadPoolExecutor(max_workers=8) as ex:
        list(ex.map(_run, cmds))
    exe = tmp_path / "delta_asan"
    _run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", str(main_o), *map(str, objs), "-o", str(exe)])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")  # the HIP runtime keeps its allocations
    out = _run([str(exe)] + (["gpu"] if torch.cuda.is_available() else []), env=env)
    assert "all checks passed" in out
