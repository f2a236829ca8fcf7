"""The 8-bit serving entries on the host: argument checks that return before any
device work, workspace queries, and the oracle's own identities.  No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import post_int4_weight_gptq_b200 as piq
from oracle import serving as S
from post_int4_weight_gptq_b200 import build as piq_build

FAKE = ctypes.c_void_p(1 << 12)   # aligned and never read
BAD = ctypes.c_void_p((1 << 12) + 4)


@pytest.fixture(scope="module")
def lib():
    piq_build.build()
    return piq.load_library()


def quantize(lib, X=FAKE, dtype=0, rows=4, cols=64, ldx=64, codes=FAKE, ldc=64, scales=FAKE):
    return lib.piq_int8_quantize_rows(X, dtype, rows, cols, ldx, codes, ldc, scales, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(cols=60, ldx=64), dict(cols=0),
    dict(ldx=56), dict(ldx=68), dict(ldc=56), dict(ldc=68), dict(X=None), dict(X=BAD),
    dict(codes=None), dict(codes=BAD), dict(scales=None), dict(cols=(1 << 20) + 8,
                                                             ldx=1 << 21, ldc=1 << 21)])
def test_quantize_rows_refuses(lib, kw):
    assert quantize(lib, **kw) == piq.PIQ_ERR_INVALID_ARG


def test_quantize_no_rows_is_nothing(lib):
    assert quantize(lib, rows=0, X=None, codes=None, scales=None) == piq.PIQ_OK


def linear(lib, X=FAKE, dtype=0, tokens=40, inp=64, ldx=64, W=FAKE, out=32, ldw=64, ws=FAKE,
           bias=None, Y=FAKE, ldy=32, status=None, work=FAKE, nbytes=1 << 20):
    return lib.piq_int8_linear(X, dtype, tokens, inp, ldx, W, out, ldw, ws, bias, Y, ldy, status,
                               work, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=5), dict(tokens=-1), dict(inp=0), dict(inp=60), dict(inp=131072, ldx=131072,
                                                                   ldw=131072),
    dict(out=0), dict(out=(1 << 24) + 1, ldy=1 << 25), dict(ldx=56), dict(ldx=68), dict(ldw=48),
    dict(ldw=72), dict(ldy=31), dict(X=None), dict(X=BAD), dict(W=None), dict(W=BAD),
    dict(ws=None), dict(Y=None), dict(work=None), dict(work=BAD),
    dict(status=ctypes.c_void_p(4098))])
def test_linear_refuses(lib, kw):
    assert linear(lib, **kw) == piq.PIQ_ERR_INVALID_ARG


def test_linear_workspace(lib):
    assert linear(lib, nbytes=0) == piq.PIQ_ERR_WORKSPACE_TOO_SMALL
    assert linear(lib, tokens=0, X=None, Y=None, work=None) == piq.PIQ_OK
    a, b = piq.int8_linear_workspace_bytes(40, 32, 64), piq.int8_linear_workspace_bytes(400, 32, 64)
    assert 0 < a <= b
    # one token runs as one kernel without a workspace; a long one, or more, do not
    assert piq.int8_linear_workspace_bytes(1, 32, 16384) == 0
    assert piq.int8_linear_workspace_bytes(1, 32, 16392) > 0
    assert piq.int8_linear_workspace_bytes(2, 32, 64) > 0
    out = ctypes.c_size_t()
    assert lib.piq_int8_linear_workspace_bytes(4, 32, 60, ctypes.byref(out)) < 0
    assert lib.piq_int8_linear_workspace_bytes(4, 32, 64, None) < 0


CACHE = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pages=3, heads=2, dim=64, block=16)
BATCH = dict(cu=FAKE, lens=FAKE, batch=2, table=FAKE, width=4, ldt=4, status=None)
BAD_CACHE = [dict(kc=None), dict(vc=BAD), dict(ks=None), dict(vs=ctypes.c_void_p(4098)),
             dict(pages=0), dict(heads=0), dict(heads=1025), dict(dim=96), dict(block=24),
             dict(block=256), dict(cu=None), dict(lens=None), dict(batch=0), dict(batch=65536),
             dict(table=None), dict(width=0), dict(ldt=3), dict(status=ctypes.c_void_p(4098))]


def append(lib, k=FAKE, v=FAKE, dtype=0, tokens=4, ldk=128, ldv=128, **kw):
    a = {**CACHE, **BATCH, **kw}
    return lib.piq_kv8_append(k, v, dtype, tokens, ldk, ldv, a["cu"], a["lens"], a["batch"],
                              a["table"], a["width"], a["ldt"], a["kc"], a["vc"], a["ks"],
                              a["vs"], a["pages"], a["heads"], a["dim"], a["block"], a["status"],
                              None)


def read(lib, k=FAKE, v=FAKE, dtype=0, rows=4, ldk=128, ldv=128, **kw):
    a = {**CACHE, **BATCH, **kw}
    return lib.piq_kv8_read(a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["heads"], a["dim"],
                            a["block"], a["cu"], a["lens"], a["batch"], a["table"], a["width"],
                            a["ldt"], rows, k, v, dtype, ldk, ldv, a["status"], None)


def attention(lib, q=FAKE, dtype=0, tokens=4, ldq=256, qheads=4, scale=0.1, window=0, max_new=2,
              max_len=64, out=FAKE, ldo=256, lse=None, work=FAKE, nbytes=1 << 30, **kw):
    a = {**CACHE, **BATCH, **kw}
    return lib.piq_kv8_attention(q, dtype, tokens, ldq, qheads, a["cu"], a["lens"], a["batch"],
                                 a["table"], a["width"], a["ldt"], a["kc"], a["vc"], a["ks"],
                                 a["vs"], a["pages"], a["heads"], a["dim"], a["block"], scale,
                                 window, max_new, max_len, out, ldo, lse, a["status"], work,
                                 nbytes, None)


@pytest.mark.parametrize("call", [append, read, attention])
@pytest.mark.parametrize("kw", BAD_CACHE)
def test_cache_entries_refuse(lib, call, kw):
    assert call(lib, **kw) == piq.PIQ_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [append, read])
@pytest.mark.parametrize("kw", [dict(dtype=3), dict(k=None), dict(v=BAD), dict(ldk=120),
                                dict(ldv=132)])
def test_append_and_read_refuse(lib, call, kw):
    assert call(lib, **kw) == piq.PIQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(q=None), dict(q=BAD), dict(out=BAD), dict(ldq=248), dict(ldo=260),
    dict(qheads=3), dict(qheads=1), dict(qheads=1024, ldq=1 << 17, ldo=1 << 17),
    dict(tokens=-1), dict(max_new=-1), dict(max_len=-1), dict(max_len=(1 << 26) + 1),
    dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(work=None),
    dict(work=BAD), dict(lse=ctypes.c_void_p(4098))])
def test_attention_refuses(lib, kw):
    assert attention(lib, **kw) == piq.PIQ_ERR_INVALID_ARG


def test_nothing_to_do_is_no_error(lib):
    assert append(lib, tokens=0, k=None, v=None) == piq.PIQ_OK
    assert read(lib, rows=0, k=None, v=None) == piq.PIQ_OK
    assert attention(lib, tokens=0, q=None, out=None, work=None) == piq.PIQ_OK


def test_attention_workspace(lib):
    assert attention(lib, nbytes=0) == piq.PIQ_ERR_WORKSPACE_TOO_SMALL
    small = piq.kv8_attention_workspace_bytes(1, 8, 2, 128, 1, 1, 1000)
    big = piq.kv8_attention_workspace_bytes(1, 8, 2, 128, 1, 1, 100000)
    assert 256 <= small <= big
    out = ctypes.c_size_t()
    assert lib.piq_kv8_attention_workspace_bytes(1, 7, 2, 128, 1, 1, 10, 0,
                                                 ctypes.byref(out)) < 0


@pytest.mark.parametrize("fault,code", [("timeout", piq.PIQ_ERR_TIMEOUT), ("oom", piq.PIQ_ERR_CUDA)])
def test_injected_faults(lib, monkeypatch, fault, code):
    monkeypatch.setenv("PIQ_FAULT", fault)
    for call in (quantize, linear, append, read, attention):
        assert call(lib) == code


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, s = torch.zeros(32, 64, dtype=torch.int8), torch.ones(32)
    with pytest.raises(TypeError):
        piq.int8_quantize_rows(x)
    with pytest.raises(TypeError):
        piq.int8_linear(x, w, s)
    cache = piq.kv8_cache(3, 2, 64, 16, device="cpu")
    cu, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 3, dtype=torch.int32)
    kv = torch.zeros(0, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        piq.kv8_append(cache, kv, kv, cu, lens, table)
    with pytest.raises(TypeError):
        piq.kv8_read(cache, cu, lens, table, 0)
    with pytest.raises(TypeError):
        piq.kv8_attention(cache, kv, cu, lens, table, 1, 1)


# ------------------------------------------------------------------ the oracle itself
def test_oracle_codes_are_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.normal(0, 3, (20, 200)).astype(np.float32)
    codes, scales = S.quantize_rows_ref(x)
    step = scales.astype(np.float64)[:, None]
    # half a step, and the two float32 roundings of x * (1 / scale), each 2^-24 of at most 127
    assert (np.abs(codes * step - x) <= step * (0.5 + 127 * 2.0 ** -23)).all()
    assert (np.abs(codes).max(1) == 127).all()


def test_oracle_append_in_pieces_bounds_every_value():
    rng = np.random.default_rng(1)
    c = S.Kv8Ref(8, 2, 64, 16)
    table, x = [[3, 5, 1, 7]], rng.normal(0, 1, (2, 50, 2, 64)).astype(np.float32)
    at = 0
    for n in (1, 1, 20, 3, 25):
        c.append(x[:, at:at + n], [0, n], [at], table)
        at += n
    for which in range(2):
        got = c.tokens(which, 0, 0, 50, table)
        for j in range(4):
            sl = slice(16 * j, min(50, 16 * j + 16))
            s = c.scale[which][table[0][j]].astype(np.float64)
            amax = np.abs(x[which, sl]).max((0, 2))
            assert np.allclose(s, amax / 127, rtol=2.0 ** -22)   # the block's own largest value
            # a value is rounded once when written and once each time the scale grows
            assert (np.abs(got[sl] - x[which, sl]) <= 5 * 0.5001 * s[None, :, None]).all()


def test_oracle_attention_against_a_plain_softmax():
    rng = np.random.default_rng(2)
    c = S.Kv8Ref(4, 1, 64, 16)
    x = rng.normal(0, 1, (2, 20, 1, 64)).astype(np.float32)
    c.append(x, [0, 20], [0], [[2, 0]])
    q = rng.normal(0, 1, (3, 2, 64))
    out, lse, _, _ = S.attention_ref(c, q, [0, 3], [20], [[2, 0]], 0.125)
    k, v = c.tokens(0, 0, 0, 20, [[2, 0]])[:, 0], c.tokens(1, 0, 0, 20, [[2, 0]])[:, 0]
    for i in range(3):
        s = q[i] @ k[:18 + i].T * 0.125
        p = np.exp(s)
        assert np.allclose(out[i], p @ v[:18 + i] / p.sum(1, keepdims=True), rtol=1e-12)
        assert np.allclose(lse[i], np.log(p.sum(1)), rtol=1e-12)


def test_wait_limit(lib):
    assert lib.piq_serving_wait_limit(10 ** 10 + 1) == piq.PIQ_ERR_INVALID_ARG
    for ns in (1, 10 ** 10, 0):
        piq.serving_wait_limit(ns)


def test_attention_heads_up_to_the_limit(lib):
    assert piq.kv8_attention_workspace_bytes(1, 256 * 1024, 1024, 64, 1, 1, 1000) >= 256
    assert piq.kv8_attention_workspace_bytes(4, 65536, 1024, 128, 3, 2, 100000) >= 256
    with pytest.raises(piq.PiqError):
        piq.kv8_attention_workspace_bytes(1, 257 * 1024, 1024, 64, 1, 1, 1000)
    with pytest.raises(piq.PiqError):   # tokens * heads
        piq.kv8_attention_workspace_bytes(1 << 13, 256 * 1024, 1024, 64, 1, 1, 1000)


def test_binding_is_rebuilt_for_another_torch_or_python(monkeypatch, tmp_path):
    import subprocess
    built = []

    def compile_(cmd, **kw):
        built.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("binding")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(piq_build.subprocess, "run", compile_)
    monkeypatch.setattr(piq_build, "SERVE", str(tmp_path / "piq_serve.so"))
    monkeypatch.setattr(piq_build, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(piq_build, "SERVE_FOR", str(tmp_path / "obj" / "piq_serve.for"))
    piq_build.build_serve()
    piq_build.build_serve()
    assert len(built) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    piq_build.build_serve()
    piq_build.build_serve()
    assert len(built) == 2
    monkeypatch.setattr(piq_build.sys, "version", "4.0")
    piq_build.build_serve()
    assert len(built) == 3
    (tmp_path / "obj" / "piq_serve.for").unlink()    # nobody knows what it was built for
    piq_build.build_serve()
    assert len(built) == 4
