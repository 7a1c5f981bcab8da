"""Host-side checks of the serving entry points: what gptq_serve.h declares is exported and bound,
and bad arguments are refused before the device is touched (no GPU needed)."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import post_weight_quantization_06_b200 as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(256)   # never dereferenced: every case below fails validation first
Q = ctypes.c_void_p(257)


def test_header_exports_and_binding_agree():
    src = open(os.path.join(ROOT, "include", "gptq_serve.h")).read()
    declared = sorted(set(re.findall(r"GPTQ_API\s+[\w\s\*]+?\b(gptq_\w+)\s*\(", src)))
    assert declared == sorted(g.EXPORTED_SERVE)
    out = subprocess.run(["nm", "-D", "--defined-only", g.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = set(re.findall(r"\sT\s+(\w+)$", out, re.M))
    for name in declared:
        assert name in exported and callable(getattr(g, name))
    assert f"GPTQ_F16 = {g.GPTQ_F16}" in src
    assert f"#define GPTQ_FP8_BLOCK {g.GPTQ_FP8_BLOCK}" in src
    assert f"#define GPTQ_CACHE_UNCLAIMED {g.GPTQ_CACHE_UNCLAIMED}" in src
    for name in ("INT4", "INT8", "E4M3"):
        assert f"GPTQ_CACHE_{name} = {getattr(g, 'GPTQ_CACHE_' + name)}" in src


def refused(fn, args, expect=-1):
    before = g.gptq_launch_count()
    assert getattr(g._lib, fn)(*args) == expect
    assert g.gptq_launch_count() == before


QUANT = dict(X=P, dt=0, rows=4, cols=200, ldx=200, br=1, codes=P, ldc=208, scales=P, s=None)


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(codes=None), dict(scales=None), dict(dt=3), dict(dt=-1), dict(rows=-1),
    dict(cols=-1), dict(ldx=199), dict(ldc=199), dict(br=2), dict(br=0), dict(rows=1 << 31),
    dict(cols=1 << 31, ldx=1 << 31, ldc=1 << 31), dict(rows=1 << 30, cols=1024, ldx=1024, ldc=1024)])
def test_quantize_refuses(kw):
    refused("gptq_fp8_quantize", {**QUANT, **kw}.values())


def test_quantize_of_nothing():
    refused("gptq_fp8_quantize", {**QUANT, "X": None, "rows": 0}.values(), 0)
    refused("gptq_fp8_quantize", {**QUANT, "codes": None, "cols": 0, "ldx": 0}.values(), 0)


MM = dict(A=P, lda=208, sA=P, B=P, ldb=208, sB=P, m=4, n=8, k=200, Y=P, dt=0, ldy=8, s=None)


@pytest.mark.parametrize("kw", [
    dict(A=None), dict(B=None), dict(sA=None), dict(sB=None), dict(Y=None), dict(dt=5), dict(m=-1),
    dict(n=-2), dict(k=-1), dict(lda=200), dict(ldb=216), dict(lda=192), dict(ldy=7), dict(A=Q),
    dict(B=Q), dict(m=1 << 31), dict(n=1 << 31, ldy=1 << 31),
    dict(k=1 << 31, lda=1 << 31, ldb=1 << 31)])
def test_matmul_refuses(kw):
    refused("gptq_fp8_matmul", {**MM, **kw}.values())


def test_matmul_of_nothing():
    refused("gptq_fp8_matmul", {**MM, "m": 0, "A": None, "Y": None}.values(), 0)
    refused("gptq_fp8_matmul", {**MM, "n": 0}.values(), 0)


WRITE = dict(K=P, kt=128, kh=64, V=P, vt=128, vh=64, dt=0, tokens=3, heads=2, dim=64, slots=P, n=10,
             fmt=1, group=0, ck=P, sk=P, zk=P, cv=P, sv=P, zv=P, claims=P, s=None)


@pytest.mark.parametrize("kw", [
    dict(K=None), dict(slots=None), dict(ck=None), dict(sk=None), dict(zk=None), dict(cv=None),
    dict(sv=None), dict(zv=None), dict(dt=3), dict(tokens=-1), dict(heads=0), dict(dim=0),
    dict(dim=60), dict(dim=4), dict(fmt=3), dict(fmt=-1), dict(group=-8), dict(group=12),
    dict(group=48), dict(group=128), dict(dim=2048), dict(heads=1025), dict(n=-1), dict(ck=Q),
    dict(cv=Q), dict(tokens=513, claims=None), dict(tokens=1 << 31)])
def test_write_refuses(kw):
    refused("gptq_cache_write", {**WRITE, **kw}.values())


READ = dict(slots=P, tokens=3, n=10, heads=2, dim=64, fmt=1, group=0, ck=P, sk=P, zk=P, cv=P, sv=P,
            zv=P, K=P, kt=128, kh=64, V=P, vt=128, vh=64, dt=0, s=None)


@pytest.mark.parametrize("kw", [
    dict(K=None), dict(slots=None), dict(ck=None), dict(zv=None), dict(dt=9), dict(dim=20),
    dict(group=24), dict(fmt=7), dict(ck=Q), dict(kt=127), dict(kh=63), dict(kt=0), dict(vt=-128),
    dict(vh=0), dict(heads=2000)])
def test_read_refuses(kw):
    refused("gptq_cache_read", {**READ, **kw}.values())


def test_cache_calls_of_nothing_and_transposed_rows():
    refused("gptq_cache_write", {**WRITE, "tokens": 0, "K": None, "slots": None}.values(), 0)
    refused("gptq_cache_read", {**READ, "tokens": 0, "K": None}.values(), 0)
    # heads outermost is fine for three tokens (64 apart, heads 192), but not with heads 191 apart
    refused("gptq_cache_read", {**READ, "kt": 64, "kh": 191}.values())


def test_binding_refuses_host_tensors_types_and_shapes():
    f8 = torch.float8_e4m3fn
    X, codes, scales = torch.zeros(4, 256), torch.zeros(4, 256).to(f8), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="current device"):
        g.gptq_fp8_quantize(X, 1, codes, scales)
    with pytest.raises(TypeError):
        g.gptq_fp8_quantize(X, 1, X, scales)
    with pytest.raises(ValueError, match="block_rows"):
        g.fp8_quantize(X, block_rows=64)
    with pytest.raises(ValueError, match="scales"):
        g.gptq_fp8_quantize(X, 128, codes, scales)
    with pytest.raises(ValueError, match="shape of X"):
        g.gptq_fp8_quantize(X, 1, codes[:3], scales)
    with pytest.raises(ValueError, match="same number of columns"):
        g.gptq_fp8_matmul(codes, scales, codes[:, :128], scales[:1], torch.zeros(4, 4))
    with pytest.raises(ValueError, match="sB"):
        g.gptq_fp8_matmul(codes, scales, codes, scales, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="current device"):
        g.gptq_fp8_matmul(codes, scales, codes, scales[:1], torch.zeros(4, 4))
    K, at = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    c = g.kv_cache(10, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="current device"):
        g.cache_write(c, K, K, at)
    with pytest.raises(TypeError, match="slots"):
        g.cache_write(c, K, K, at.int())
    with pytest.raises(ValueError, match="slots"):
        g.cache_write(c, K, K, at[:2])
    with pytest.raises(ValueError, match="shape of K"):
        g.cache_write(c, K, K[:2], at)
    with pytest.raises(TypeError, match="V"):
        g.cache_write(c, K, K.bfloat16(), at)
    with pytest.raises(ValueError, match="codes"):
        g.cache_write(c, K[..., :32], None, at)
    with pytest.raises(ValueError, match="contiguous"):
        g.cache_write(c, torch.zeros(3, 2, 128)[..., ::2], None, at)
    for kw in (dict(group_size=48), dict(group_size=12), dict(fmt=4)):
        with pytest.raises(ValueError):
            g.kv_cache(10, 2, 64, device="cpu", **kw)
    with pytest.raises(ValueError):
        g.kv_cache(10, 2, 60, device="cpu")


R = ctypes.c_void_p(258)   # a multiple of 2 only


@pytest.mark.parametrize("kw", [dict(X=Q), dict(X=R, dt=1), dict(scales=R)])
def test_quantize_refuses_addresses_no_element_starts_at(kw):
    refused("gptq_fp8_quantize", {**QUANT, **kw}.values())


@pytest.mark.parametrize("kw", [dict(Y=Q), dict(Y=R, dt=1), dict(sA=R), dict(sB=Q),
                                dict(lda=1 << 41), dict(ldb=1 << 40)])
def test_matmul_refuses_addresses_and_pitches_out_of_range(kw):
    refused("gptq_fp8_matmul", {**MM, **kw}.values())


@pytest.mark.parametrize("kw", [dict(K=Q), dict(V=R, dt=1), dict(slots=R), dict(sk=R), dict(sv=Q),
                                dict(claims=R)])
def test_write_refuses_addresses_no_element_starts_at(kw):
    refused("gptq_cache_write", {**WRITE, **kw}.values())


@pytest.mark.parametrize("kw", [dict(K=R, dt=1), dict(V=Q), dict(slots=R), dict(sk=Q)])
def test_read_refuses_addresses_no_element_starts_at(kw):
    refused("gptq_cache_read", {**READ, **kw}.values())


def test_cache_scales_are_fp32_whatever_the_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.bfloat16)
    try:
        c = g.kv_cache(4, 2, 64, device="cpu")
    finally:
        torch.set_default_dtype(before)
    assert c["scales_k"].dtype == c["scales_v"].dtype == torch.float32


def test_binding_refuses_a_cache_that_lacks_an_array():
    K, at = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    c = g.kv_cache(10, 2, 64, device="cpu", values=False)
    with pytest.raises(ValueError, match="lacks"):
        g.cache_write(c, K, K, at)
    with pytest.raises(ValueError, match="lacks"):
        g.cache_read(c, at, out=(K, K))
    with pytest.raises(ValueError, match="lacks"):
        g.cache_write({**c, "zeros_k": None}, K, None, at)
    with pytest.raises(ValueError, match="lacks"):
        g.cache_write({**c, "scales_k": None}, K, None, at)


@pytest.mark.parametrize("fmt", [19, 16 - 1, 32, 33, 16 + 32, -16])
def test_read_refuses_formats_it_does_not_know(fmt):
    refused("gptq_cache_read", {**READ, "fmt": fmt}.values())


def test_clearing_belongs_to_reading():
    src = open(os.path.join(ROOT, "include", "gptq_serve.h")).read()
    assert f"#define GPTQ_CACHE_CLEAR {g.GPTQ_CACHE_CLEAR}" in src
    refused("gptq_cache_write", {**WRITE, "fmt": 1 + g.GPTQ_CACHE_CLEAR}.values())
    refused("gptq_cache_read", {**READ, "fmt": 1 + g.GPTQ_CACHE_CLEAR, "tokens": 0, "K": None}.values(), 0)
    refused("gptq_cache_read", {**READ, "fmt": 1 + g.GPTQ_CACHE_CLEAR, "zk": None}.values())


@pytest.mark.parametrize("kt,kh", [(1 << 62, 1 << 62), (1 << 62, 1 << 61), ((1 << 63) - 1, (1 << 63) - 1)])
def test_read_refuses_strides_whose_products_pass_64_bits(kt, kh):
    refused("gptq_cache_read", {**READ, "kt": kt, "kh": kh}.values())
    refused("gptq_cache_read", {**READ, "heads": 4, "V": None, "kt": kt, "kh": kh}.values())


def test_binding_refuses_a_cache_without_codes_of_keys():
    K, at = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    c = {**g.kv_cache(10, 2, 64, device="cpu"), "codes_k": None}
    for call in (lambda: g.cache_write(c, K, K, at), lambda: g.cache_read(c, at),
                 lambda: g.cache_read(c, at, out=(K, K))):
        with pytest.raises(ValueError, match="lacks"):
            call()


@pytest.mark.parametrize("device,want", [(0, 0), (1, 1), ("cpu", "cpu"), (None, "cuda")])
def test_a_cache_lies_on_the_device_that_was_named(monkeypatch, device, want):
    seen, zeros = [], torch.zeros

    def on_the_host(*shape, device=None, **kw):
        seen.append(device)
        return zeros(*shape, **kw)
    monkeypatch.setattr(torch, "zeros", on_the_host)
    g.kv_cache(4, 2, 64, device=device)
    assert seen and all(type(d) is type(want) and d == want for d in seen)


@pytest.mark.parametrize("heads,dim,group", [(0, 64, 0), (-1, 64, 0), (512, 256, 0), (1025, 64, 32)])
def test_no_cache_is_made_that_the_calls_would_refuse(heads, dim, group):
    with pytest.raises(ValueError, match="heads"):
        g.kv_cache(4, heads, dim, group_size=group, device="cpu")
    refused("gptq_cache_write", {**WRITE, "heads": heads, "dim": dim, "group": group}.values())
    refused("gptq_cache_read", {**READ, "heads": heads, "dim": dim, "group": group, "kt": 1 << 20,
                                "kh": dim, "vt": 1 << 20, "vh": dim}.values())
    assert g.kv_cache(1, 65536 // dim, dim, group_size=group, device="cpu")["codes_k"].shape[1] == 65536 // dim


def test_the_package_imports_where_torch_has_no_cuda():
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import post_weight_quantization_06_b200 as g
try:
    g.fp8_quantize(torch.zeros(4, 256))
except ValueError as e:
    assert "current device" in str(e)
    print("ok")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.stdout.strip() == "ok", out.stderr[-2000:]


@pytest.mark.parametrize("t,h", [(1 << 62, 64), (-(1 << 62), 64), (64, 1 << 60), (1 << 59, 1 << 59),
                                 (-(1 << 63), 0), ((1 << 63) - 1, -(1 << 63))])
def test_write_refuses_strides_whose_products_pass_64_bits(t, h):
    refused("gptq_cache_write", {**WRITE, "kt": t, "kh": h}.values())
    refused("gptq_cache_write", {**WRITE, "vt": t, "vh": h}.values())
