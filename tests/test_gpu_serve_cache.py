"""The quantized cache on the GPU against the 64-bit oracle: codes, scales and zero-points equal,
values read back within a half step of their type (and one of fp32, where they are computed)."""
import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BITS = {0: 4, 1: 8, 2: None}   # by format


@pytest.fixture(scope="module")
def g():
    import post_weight_quantization_06_b200 as lib
    return lib


def np64(t):
    return t.detach().double().cpu().numpy()


def rows(t, h, d, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, d, generator=gen) * torch.exp(torch.randn(1, h, d, generator=gen))
    return x.to(DT[dtype]).to(DEV)


def slots_of(t, n, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randperm(n, generator=gen)[:t].to(DEV)


def check_arrays(cache, which, X, at, fmt, group):
    """The cache's rows `at` hold what the oracle makes of X (fp64)."""
    q = serve.cache_quantize(X, BITS[fmt], group)
    codes = cache["codes_" + which][at].cpu().numpy()
    want = serve.pack4(q["codes"]) if BITS[fmt] == 4 else q["codes"]
    assert np.array_equal(cache["scales_" + which][at].cpu().numpy(), q["scales"], equal_nan=True)
    if BITS[fmt]:
        assert np.array_equal(cache["zeros_" + which][at].cpu().numpy(), q["zeros"])
    else:   # either sign of NaN
        nan = (want & 127) == 127
        codes, want = np.where(nan, codes & 127, codes), np.where(nan, want & 127, want)
    assert np.array_equal(codes, want)
    return q["values"]


def check_values(y, want, dtype):
    got = np64(y)
    eps = torch.finfo(DT[dtype]).eps / 2
    bound = np.abs(want) * (2.0 ** -24 + eps * (1 + 2.0 ** -24)) + torch.finfo(DT[dtype]).tiny
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= bound[ok]).all()


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t,h,d,group", [(1, 1, 8, 0), (1, 8, 128, 0), (3, 2, 64, 16), (5, 3, 96, 0),
                                         (64, 8, 128, 64), (7, 1, 40, 8), (33, 4, 80, 40),
                                         (6, 2, 512, 0), (4, 1, 1024, 0), (600, 2, 128, 32)])
def test_write_and_read_equal_the_oracle(g, fmt, dtype, t, h, d, group):
    n = t + 37
    K, V = rows(t, h, d, dtype, 1), rows(t, h, d, dtype, 2)
    at = slots_of(t, n, t)
    c = g.kv_cache(n, h, d, fmt=fmt, group_size=group)
    g.cache_write(c, K, V, at)
    k, v = g.cache_read(c, at, dtype=DT[dtype])
    g.gptq_sync_status()
    check_values(k, check_arrays(c, "k", np64(K), at, fmt, group), dtype)
    check_values(v, check_arrays(c, "v", np64(V), at, fmt, group), dtype)
    # the other slots are as they were, and the scratch is zero again
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[at] = False
    for p in ("k", "v"):
        assert (c["codes_" + p][rest] == 0).all() and (c["scales_" + p][rest] == 0).all()
    assert (c["claims"] == 0).all()


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_zero_symmetric_tiny_and_huge_groups(g, fmt):
    X = torch.zeros(8, 1, 64)
    X[1, 0, :] = torch.linspace(-1, 1, 64)          # a zero-point between two numbers
    X[2, 0, :] = torch.linspace(0.5, 2, 64)         # the grid still holds zero
    X[3, 0, :] = -torch.linspace(0.5, 2, 64)
    X[4, 0, :] = torch.linspace(-1e-44, 2e-44, 64)
    X[5, 0, :] = torch.linspace(-1.5e38, 1.5e38, 64)
    X[6, 0, 3] = 1e-3
    X[7, 0, :] = torch.arange(64) - 31.5
    for dt in ("fp32", "bf16"):
        x = X.to(DT[dt]).to(DEV)
        c = g.kv_cache(8, 1, 64, fmt=fmt, values=False)
        at = torch.arange(8, device=DEV)
        g.cache_write(c, x, None, at)
        k, v = g.cache_read(c, at, dtype=torch.float32)
        g.gptq_sync_status()
        assert v is None
        check_values(k, check_arrays(c, "k", np64(x), at, fmt, 0), "fp32")


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite_is_reported_unless_skipped(g, fmt, bad):
    K, V = rows(6, 2, 64, "bf16", 1), rows(6, 2, 64, "bf16", 2)
    K[2, 1, 40] = bad
    at = torch.tensor([5, 1, 7, 2, 0, 6], device=DEV)
    c = g.kv_cache(8, 2, 64, fmt=fmt, group_size=32)
    g.cache_write(c, K, V, at)
    st, info = g.gptq_sync_status(raise_on_error=False)
    assert st == g.GPTQ_ERR_NONFINITE and info == 2
    k, _ = g.cache_read(c, at, dtype=torch.float32)
    g.gptq_sync_status()
    check_values(k, check_arrays(c, "k", np64(K), at, fmt, 32), "fp32")
    nan = torch.isnan(k)
    want = torch.zeros_like(nan)
    want[2, 1, 32:] = True
    if BITS[fmt] is None:
        want[2, 1, 32:] = False
        want[2, 1, 40] = True
    assert torch.equal(nan, want)
    # the same token, skipped
    at[2] = -1
    g.cache_write(c, K, V, at)
    g.gptq_sync_status()


def test_range_beyond_fp32_is_reported(g):
    K = torch.zeros(1, 1, 8, device=DEV)
    K[0, 0, 0], K[0, 0, 1] = 3e38, -3e38
    c = g.kv_cache(1, 1, 8, fmt=g.GPTQ_CACHE_INT8, values=False)
    at = torch.zeros(1, dtype=torch.int64, device=DEV)
    g.cache_write(c, K, None, at)
    st, info = g.gptq_sync_status(raise_on_error=False)
    assert st == g.GPTQ_ERR_NONFINITE and info == 0
    assert torch.isnan(g.cache_read(c, at, dtype=torch.float32)[0]).all()


@pytest.mark.parametrize("t", [20, 513, 3000])
def test_padding_and_slots_out_of_range(g, t):
    h, d, n = 2, 64, t
    K, V = rows(t, h, d, "bf16", 1), rows(t, h, d, "bf16", 2)
    at = slots_of(t, n, 4)
    skip = torch.arange(t, device=DEV) % 3 == 1
    at[skip] = -1 - at[skip]
    c = g.kv_cache(n, h, d, fmt=g.GPTQ_CACHE_INT8)
    g.cache_write(c, K, V, at)
    g.gptq_sync_status()
    live = ~skip
    want = check_arrays(c, "k", np64(K[live]), at[live], 1, 0)
    outk = torch.full((t, h, d), 9.0, device=DEV)
    outv = outk.clone()
    args = [c[f] for f in ("codes_k", "scales_k", "zeros_k", "codes_v", "scales_v", "zeros_v")]
    g.gptq_cache_read(at, 1, 0, *args, outk, outv)
    g.gptq_sync_status()
    assert (outk[skip] == 9).all() and (outv[skip] == 9).all()
    check_values(outk[live], want, "fp32")
    # a slot behind the end: reported, its token skipped, the others done
    far = at.clone()
    far[6] = n
    before = {k: v.clone() for k, v in c.items() if torch.is_tensor(v)}
    g.cache_write(c, K, V, far)
    st, info = g.gptq_sync_status(raise_on_error=False)
    assert st == g.GPTQ_ERR_ARG and info == 6
    assert all(torch.equal(before[k], c[k]) for k in before)
    outk.fill_(9.0)
    g.gptq_cache_read(far, 1, 0, *args, outk, outv)
    st, info = g.gptq_sync_status(raise_on_error=False)
    assert st == g.GPTQ_ERR_ARG and info == 6
    assert (outk[6] == 9).all()


@pytest.mark.parametrize("t", [2, 100, 512, 513, 5000])
def test_of_tokens_with_the_same_slot_the_last_stays(g, t):
    h, d, n = 2, 64, max(1, t // 3)
    K, V = rows(t, h, d, "bf16", 1), rows(t, h, d, "bf16", 2)
    gen = torch.Generator().manual_seed(t)
    at = torch.randint(0, n, (t,), generator=gen).to(DEV)
    c = g.kv_cache(n, h, d, fmt=g.GPTQ_CACHE_INT4, group_size=32)
    for _ in range(3):
        g.cache_write(c, K, V, at)
    g.gptq_sync_status()
    last = {int(s): i for i, s in enumerate(at.tolist())}
    slots = torch.tensor(sorted(last), device=DEV)
    src = torch.tensor([last[s] for s in sorted(last)], device=DEV)
    check_arrays(c, "k", np64(K[src]), slots, 0, 32)
    check_arrays(c, "v", np64(V[src]), slots, 0, 32)
    assert (c["claims"] == 0).all()


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("shift", [0, 1])
def test_views_of_a_fused_projection_and_transposed_outputs(g, fmt, shift):
    t, h, d = 50, 3, 64
    gen = torch.Generator().manual_seed(3)
    buf = torch.randn(t * 9 * d + shift, generator=gen).to(torch.bfloat16).to(DEV)
    qkv = buf[shift:].view(t, 9, d)      # shift 1: no row is 16-byte aligned
    K, V = qkv[:, 3:6], qkv[:, 6:]
    at = slots_of(t, 64, 8)
    c = g.kv_cache(64, h, d, fmt=fmt)
    g.cache_write(c, K, V, at)
    outk = torch.zeros(h, t, d, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    outv = torch.zeros(t, h, d + 1, dtype=torch.bfloat16, device=DEV)[..., :d]
    args = [c[f] for f in ("codes_k", "scales_k", "zeros_k", "codes_v", "scales_v", "zeros_v")]
    g.gptq_cache_read(at, fmt, 0, *args, outk, outv)
    g.gptq_sync_status()
    check_values(outk, check_arrays(c, "k", np64(K), at, fmt, 0), "bf16")
    check_values(outv, check_arrays(c, "v", np64(V), at, fmt, 0), "bf16")


def test_a_cache_beyond_32_bit_offsets(g):
    """4.5 GB of codes a plane: the last slots lie behind 2^32 bytes."""
    h, d = 16, 256
    n = (1 << 32) // (h * d) + 65536
    c = g.kv_cache(n, h, d, fmt=g.GPTQ_CACHE_INT8, values=False)
    at = torch.tensor([n - 1, 0, n - 2, (1 << 31) // (h * d), (1 << 32) // (h * d)], device=DEV)
    K = rows(5, h, d, "bf16", 6)
    g.cache_write(c, K, None, at)
    k, _ = g.cache_read(c, at, dtype=torch.float32)
    g.gptq_sync_status()
    check_values(k, check_arrays(c, "k", np64(K), at, 1, 0), "fp32")


def test_reading_a_slot_many_times_and_none(g):
    K = rows(4, 2, 64, "bf16", 6)
    c = g.kv_cache(4, 2, 64, fmt=g.GPTQ_CACHE_E4M3)
    g.cache_write(c, K, K, torch.arange(4, device=DEV))
    at = torch.tensor([2] * 700, device=DEV)
    k, v = g.cache_read(c, at)
    assert torch.equal(k, k[:1].expand_as(k)) and torch.equal(k, v)
    before = g.gptq_launch_count()
    g.cache_write(c, K[:0], K[:0], at[:0])
    assert g.cache_read(c, at[:0])[0].shape == (0, 2, 64)
    assert g.gptq_launch_count() == before
    g.gptq_sync_status()


@pytest.mark.parametrize("t", [16, 2000])
def test_two_streams_and_a_captured_step(g, t):
    h, d = 4, 128
    n = 2 * t
    perm = slots_of(n, n, 5)
    a, b = perm[:t].clone(), perm[t:].clone()
    Ka, Kb = rows(t, h, d, "bf16", 1), rows(t, h, d, "bf16", 2)
    c = g.kv_cache(n, h, d, fmt=g.GPTQ_CACHE_INT4, group_size=64)
    args = [c[f] for f in ("codes_k", "scales_k", "zeros_k", "codes_v", "scales_v", "zeros_v")]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):   # two calls at once on one cache, other slots
        g.gptq_cache_write(Ka, Ka, a, 0, 64, *args, c["claims"], stream=s1)
        g.gptq_cache_write(Kb, Kb, b, 0, 64, *args, c["claims"], stream=s2)
    torch.cuda.synchronize()
    check_arrays(c, "k", np64(Ka), a, 0, 64)
    check_arrays(c, "v", np64(Kb), b, 0, 64)
    k, v = torch.zeros_like(Ka), torch.zeros_like(Ka)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gptq_cache_write(Ka, Ka, a, 0, 64, *args, c["claims"])
        g.gptq_cache_read(a, 0, 64, *args, k, v)
    for seed in (21, 22):
        Ka.copy_(rows(t, h, d, "bf16", seed))
        a.copy_(slots_of(t, n, seed))
        graph.replay()
        torch.cuda.synchronize()
        want = check_arrays(c, "k", np64(Ka), a, 0, 64)
        check_values(k, want, "bf16")
        check_values(v, want, "bf16")
    assert (c["claims"] == 0).all()
    g.gptq_sync_status()


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_projection_into_the_cache_and_back(g, fmt):
    """A decode step's use of all four: activations and a K/V weight in 8 bits, their product, its
    rows into the cache, read back. Against the oracle on the same codes and products."""
    from test_gpu_serve_fp8 import judge, raw
    t, hidden, h, d = 37, 640, 4, 64
    X = rows(t, 1, hidden, "bf16", 1).view(t, hidden)
    W = 0.02 * rows(2 * h * d, 1, hidden, "fp32", 2).view(2 * h * d, hidden)
    A, sA = g.fp8_quantize(X)
    B, sB = g.fp8_quantize(W, block_rows=128)
    Y = g.fp8_matmul(A, sA, B, sB)
    kv = Y.view(t, 2 * h, d)
    c = g.kv_cache(64, h, d, fmt=fmt)
    at = slots_of(t, 64, 3)
    g.cache_write(c, kv[:, :h], kv[:, h:], at)
    k, v = g.cache_read(c, at)
    g.gptq_sync_status()
    assert np.array_equal(raw(A), serve.fp8_quantize(np64(X), 1)[0])
    assert np.array_equal(raw(B), serve.fp8_quantize(np64(W), 128)[0])
    judge(Y, A, sA, B, sB, "bf16")
    check_values(k, check_arrays(c, "k", np64(kv[:, :h]), at, fmt, 0), "bf16")
    check_values(v, check_arrays(c, "v", np64(kv[:, h:]), at, fmt, 0), "bf16")


def test_reading_into_tensors_of_the_caller(g):
    c = g.kv_cache(40, 2, 64, fmt=g.GPTQ_CACHE_INT8, group_size=32)
    K, V = rows(40, 2, 64, "bf16", 8), rows(40, 2, 64, "bf16", 9)
    g.cache_write(c, K, V, torch.arange(40, device=DEV))
    at = slots_of(20, 40, 3)
    at[::3] = -1
    fresh = g.cache_read(c, at)
    buf = torch.full((20, 2, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)   # K and V side by side
    k, v = g.cache_read(c, at, out=(buf[:, 0], buf[:, 1]))
    g.gptq_sync_status()
    assert k.data_ptr() == buf.data_ptr()
    kept = at >= 0
    for got, want in zip((k, v), fresh):
        assert torch.equal(got[kept], want[kept])
        assert (got[~kept] == 7).all() and (want[~kept] == 0).all()


@pytest.mark.parametrize("fmt,dim,group", [(0, 72, 24), (1, 128, 32), (2, 80, 0)])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pitch", [0, 8, 3])   # heads that follow each other, apart, and unaligned
def test_clearing_the_rows_without_a_slot(g, fmt, dim, group, dtype, pitch):
    c = g.kv_cache(30, 3, dim, fmt=fmt, group_size=group)
    K = rows(30, 3, dim, "fp32", 4)
    g.cache_write(c, K, K, torch.arange(30, device=DEV))
    g.gptq_sync_status()
    at = slots_of(20, 30, 5)
    at[::3], at[1] = -1, -(1 << 40)
    fresh = g.cache_read(c, at, dtype=DT[dtype])
    buf = torch.full((2, 20, 3, dim + pitch), 7.0, dtype=DT[dtype], device=DEV)
    args = [c[n] for n in ("codes_k", "scales_k", "zeros_k", "codes_v", "scales_v", "zeros_v")]
    g.gptq_cache_read(at, fmt + g.GPTQ_CACHE_CLEAR, group, *args, buf[0, ..., :dim], buf[1, ..., :dim])
    g.gptq_sync_status()
    kept = at >= 0
    for got, want in zip(buf, fresh):
        assert (got[..., dim:] == 7).all()
        assert torch.equal(got[..., :dim], want)
        assert (want[~kept] == 0).all() and (want[kept] != 0).any()
    at[4] = 30   # behind the last slot: zero as well, and reported
    k, _ = g.cache_read(c, at, dtype=DT[dtype])
    with pytest.raises(g.GptqError):
        g.gptq_sync_status()
    assert (k[4] == 0).all() and torch.equal(k[5:], fresh[0][5:])


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("dim,group", [(128, 32), (72, 24)])
def test_values_are_rounded_to_fp32_and_then_to_the_output(g, fmt, dim, group):
    n = 500
    c = g.kv_cache(n, 4, dim, fmt=fmt, group_size=group)
    at = torch.arange(n, device=DEV)
    g.cache_write(c, rows(n, 4, dim, "fp32", 1), rows(n, 4, dim, "fp32", 2), at)
    wide = g.cache_read(c, at, dtype=torch.float32)
    for dtype in ("bf16", "fp16"):
        for got, want in zip(g.cache_read(c, at, dtype=DT[dtype]), wide):
            assert torch.equal(got, want.to(DT[dtype]))
    q = serve.cache_quantize(np64(rows(n, 4, dim, "fp32", 1)), BITS[fmt], group)
    assert np.array_equal(wide[0].cpu().numpy(), q["values"].astype(np.float32))
    g.gptq_sync_status()


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,h,d,group", [(3000, 16, 80, 0), (1100, 16, 80, 0), (9000, 4, 96, 0),
                                         (2000, 8, 192, 0), (3000, 8, 80, 40), (40000, 1, 40, 0)])
def test_long_writes_of_heads_that_are_no_power_of_two(g, fmt, dtype, t, h, d, group):
    """Both widths of a lane, and calls that end inside a CTA; every 97th token against the oracle."""
    K, V = rows(t, h, d, dtype, 1), rows(t, h, d, dtype, 2)
    at = slots_of(t, t + 5, 7)
    at[::5] = -1
    c = g.kv_cache(t + 5, h, d, fmt=fmt, group_size=group)
    g.cache_write(c, K, V, at)
    g.gptq_sync_status()
    some = torch.arange(1, t, 97, device=DEV)
    some = torch.cat([some, torch.tensor([t - 1], device=DEV)])
    some = some[at[some] >= 0]
    check_arrays(c, "k", np64(K[some]), at[some], fmt, group)
    check_arrays(c, "v", np64(V[some]), at[some], fmt, group)
    assert (c["claims"] == 0).all()
