"""Host checks of the MXFP4 experts and of the orthogonalised update: sizes,
refusals before anything is enqueued, and the 64-bit references themselves.
No kernel is launched (these run without a GPU)."""
import ctypes

import numpy as np
import pytest

import mixture_experts_layer_logit_amd as moe
import _mx_ref as ref

FAKE = 1 << 20  # an aligned, never dereferenced address
BIG = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


def status(fn, *args):
    return getattr(moe.load(), fn)(*args)


def prob(**kw):
    a = dict(T=64, d=256, E=8, k=2, F=384, act="swiglu")
    a.update(kw)
    return moe.problem(a.pop("T"), a.pop("d"), a.pop("E"), a.pop("k"), a.pop("F"), **a)


# ---------------------------------------------------------------- the references
def test_reference_codes():
    v = np.array([0.25, 0.250001, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 6.0, -0.0, -0.75, -2.6])
    assert list(ref.encode(v)) == [0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 8, 10, 13]
    assert np.array_equal(ref.encode(ref.TABLE), np.arange(16))
    q, e = ref.quantise(np.concatenate([ref.TABLE, ref.TABLE])[None])
    assert e[0, 0] == 0 and list(q[0, :8]) == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert np.array_equal(ref.widen(q, e)[0, :16], ref.TABLE)


def test_reference_scales():
    for a, e in ((0.0, 0), (6.0, 0), (6.0001, 1), (3.0, -1), (3.1, 0), (2.0 ** -200, -127), (1.0, -2), (3.4e38, 126)):
        assert ref.exponent(a) == e
    for a in np.exp(np.random.default_rng(1).uniform(-60, 60, 2000)):
        e = int(ref.exponent(a))
        assert 3 * 2.0 ** e < a <= 6 * 2.0 ** e


def test_reference_half_steps():
    v = np.random.default_rng(3).uniform(-6, 6, 20000)
    d = np.abs(ref.TABLE[ref.encode(v)] - v)
    assert np.all(d <= ref.half_step(np.abs(v), 1.0))
    assert d.max() > 0.99


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (5, 5), (7, 30), (33, 8)])
def test_reference_orthogonal(shape):
    u = np.random.default_rng(4).standard_normal(shape)
    a, b = ref.orthogonal(u, 5), ref.orthogonal_by_products(u, 5)
    assert np.allclose(a, b, rtol=0, atol=1e-9)
    s = np.linalg.svd(ref.orthogonal(u, 8), compute_uv=False)
    assert s.max() < 1.21 and s.min() > 0.6
    assert np.all(ref.orthogonal(np.zeros(shape), 5) == 0)


def test_reference_momentum():
    g, m = np.array([1.0, -2.0]), np.array([4.0, 8.0])
    assert np.array_equal(ref.momentum(g, m, 0.5, False)[1], [3.0, 2.0])
    assert np.array_equal(ref.momentum(g, m, 0.5, True)[1], [2.5, -1.0])


# ---------------------------------------------------------------- refusals
@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), INVALID), (dict(dt=-1), INVALID), (dict(rows=-1), INVALID), (dict(K=16), UNSUPPORTED), (dict(K=48), UNSUPPORTED),
    (dict(K=0), UNSUPPORTED), (dict(K=65536 + 32), UNSUPPORTED), (dict(rows=1 << 36), UNSUPPORTED), (dict(wide=None), INVALID),
    (dict(wide=FAKE + 8), INVALID), (dict(codes=None), INVALID), (dict(codes=FAKE + 8), INVALID), (dict(scales=None), INVALID)])
def test_quantise_refusals(kw, want):
    a = dict(wide=FAKE, dt=moe.MOE_BF16, rows=8, K=64, codes=FAKE, scales=FAKE)
    a.update(kw)
    assert status("moe_quantize_mxfp4", a["wide"], a["dt"], a["rows"], a["K"], a["codes"], a["scales"], None) == want
    assert moe.load().moe_last_error()
    assert status("moe_dequantize_mxfp4", a["codes"], a["scales"], a["rows"], a["K"], a["wide"], a["dt"], None) == want


def test_no_rows():
    assert status("moe_quantize_mxfp4", None, 0, 0, 32, None, None, None) == moe.MOE_OK
    assert status("moe_dequantize_mxfp4", None, None, 0, 32, None, 1, None) == moe.MOE_OK
    p = prob(T=0)
    assert status("moe_expert_up_mxfp4", ctypes.byref(p), *[None] * 9, 0, None) == moe.MOE_OK
    assert status("moe_expert_down_mxfp4", ctypes.byref(p), *[None] * 7, 0, None) == moe.MOE_OK
    assert status("moe_forward_mxfp4", ctypes.byref(p), *[None] * 11, 0, None) == moe.MOE_OK
    assert status("moe_orthogonalize", None, 0, None, 0.9, 0, 0, 8, 8, 5, None, None, 0, None) == moe.MOE_OK


@pytest.mark.parametrize("kw,want", [(dict(dtype="f32"), UNSUPPORTED), (dict(d=320), UNSUPPORTED), (dict(F=448), UNSUPPORTED),
                                     (dict(k=9, E=16), UNSUPPORTED), (dict(T=-1), INVALID)])
def test_problem_refusals(kw, want):
    p, n = prob(**kw), ctypes.c_size_t()
    assert status("moe_mxfp4_workspace_size", ctypes.byref(p), ctypes.byref(n)) == want
    assert status("moe_expert_up_mxfp4", ctypes.byref(p), *[FAKE] * 8, None, 0, None) == want
    assert status("moe_expert_down_mxfp4", ctypes.byref(p), *[FAKE] * 6, None, 0, None) == want
    assert status("moe_forward_mxfp4", ctypes.byref(p), *[FAKE] * 8, None, None, FAKE, BIG, None) == want
    assert b"FP8" not in moe.load().moe_last_error()


def test_workspace_sizes_need_their_result():
    assert status("moe_mxfp4_workspace_size", ctypes.byref(prob()), None) == INVALID
    assert status("moe_orthogonalize_workspace_size", 1, 8, 8, None) == INVALID


@pytest.mark.parametrize("at,bad,want", [(0, None, INVALID), (0, FAKE + 8, INVALID), (1, None, INVALID), (1, FAKE + 2, INVALID),
                                         (2, FAKE + 2, INVALID), (3, None, INVALID), (4, FAKE + 8, INVALID), (5, None, INVALID),
                                         (5, FAKE + 1, INVALID), (6, None, INVALID), (7, FAKE + 2, INVALID), (8, FAKE + 8, INVALID),
                                         (9, 16, WORKSPACE)])
def test_up_refusals(at, bad, want):
    a = [FAKE] * 9 + [BIG]
    a[at] = bad
    assert status("moe_expert_up_mxfp4", ctypes.byref(prob()), *a, None) == want
    assert moe.load().moe_last_error()


@pytest.mark.parametrize("at,bad,want", [(0, None, INVALID), (0, FAKE + 8, INVALID), (1, None, INVALID), (1, FAKE + 2, INVALID),
                                         (2, None, INVALID), (3, FAKE + 8, INVALID), (4, FAKE + 2, INVALID), (5, None, INVALID),
                                         (5, FAKE + 2, INVALID), (6, FAKE + 8, INVALID), (7, 16, WORKSPACE)])
def test_down_refusals(at, bad, want):
    a = [FAKE] * 7 + [BIG]
    a[at] = bad
    assert status("moe_expert_down_mxfp4", ctypes.byref(prob()), *a, None) == want


@pytest.mark.parametrize("at,bad,want", [(0, None, INVALID), (1, FAKE + 8, INVALID), (2, FAKE + 2, INVALID), (3, None, INVALID),
                                         (4, FAKE + 2, INVALID), (5, None, INVALID), (6, None, INVALID), (7, None, INVALID),
                                         (8, FAKE + 2, INVALID), (10, None, INVALID), (11, 64, WORKSPACE)])
def test_layer_refusals(at, bad, want):
    a = [FAKE] * 8 + [None, None, FAKE, BIG]
    a[at] = bad
    assert status("moe_forward_mxfp4", ctypes.byref(prob()), *a, None) == want


def test_layer_with_given_logits_needs_them():
    a = [FAKE, None, None] + [FAKE] * 5 + [None, None, FAKE, BIG]
    assert status("moe_forward_mxfp4", ctypes.byref(prob()), *a, None) == INVALID


def test_gather_beyond_32_bits_is_refused():
    p = prob(T=1 << 24, d=512, E=8, k=1)
    assert status("moe_expert_up_mxfp4", ctypes.byref(p), *[FAKE] * 8, None, 0, None) == UNSUPPORTED
    assert status("moe_forward_mxfp4", ctypes.byref(p), *[FAKE] * 8, None, None, FAKE, BIG, None) == UNSUPPORTED


ORTH = dict(grad=FAKE, dt=moe.MOE_F32, mom=FAKE, beta=0.95, nesterov=1, count=2, rows=24, cols=40, steps=5, out=FAKE, ws=FAKE, size=BIG)


@pytest.mark.parametrize("kw,want", [
    (dict(grad=None), INVALID), (dict(grad=FAKE + 2), INVALID), (dict(grad=FAKE + 1, dt=1), INVALID), (dict(dt=2), INVALID),
    (dict(mom=FAKE + 2), INVALID), (dict(mom=None), INVALID), (dict(beta=float("nan")), INVALID), (dict(beta=float("inf")), INVALID),
    (dict(nesterov=2), INVALID), (dict(count=-1), INVALID), (dict(count=40000), UNSUPPORTED), (dict(rows=0), INVALID),
    (dict(cols=-3), INVALID), (dict(rows=65537), UNSUPPORTED), (dict(rows=32768, cols=32768), UNSUPPORTED),
    (dict(rows=16384, cols=32768, count=4096), UNSUPPORTED), (dict(steps=0), INVALID), (dict(steps=65), UNSUPPORTED),
    (dict(out=None), INVALID), (dict(out=FAKE + 1), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 8), INVALID),
    (dict(size=64), WORKSPACE)])
def test_orthogonalize_refusals(kw, want):
    a = dict(ORTH, **kw)
    assert status("moe_orthogonalize", a["grad"], a["dt"], a["mom"], a["beta"], a["nesterov"], a["count"], a["rows"], a["cols"],
                  a["steps"], a["out"], a["ws"], a["size"], None) == want
    assert moe.load().moe_last_error()


def test_orthogonalize_workspace_covers_every_orientation():
    for count, rows, cols in ((3, 65, 100), (3, 100, 65), (2, 4096, 14336), (1, 65, 65536), (1, 1, 1), (3, 7, 100), (5, 64, 64),
                              (1, 1, 65536), (32768, 8, 16)):
        n = moe.moe_orthogonalize_workspace_size(count, rows, cols)
        # X in both orientations (one of them twice) and its remainder, and the two square
        # products, all of them fp16
        assert n >= count * (8 * rows * cols + 4 * min(rows, cols) ** 2)
        assert n == moe.moe_orthogonalize_workspace_size(count, cols, rows)


# ------------------------------------------------- the binding: element types, sizes, devices
def calls(torch):
    """Arguments of the right types and sizes for every entry point, on the host:
    nothing that is refused reads them."""
    T, d, E, k, F = 64, 256, 8, 2, 384

    def u8(*shape):
        return torch.zeros(*shape, dtype=torch.uint8)

    def i32(*shape):
        return torch.zeros(*shape, dtype=torch.int32)

    def bf(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16)

    w1, s1, w2, s2 = u8(E, 2 * F, d // 2), u8(E, 2 * F, d // 32), u8(E, d, F // 2), u8(E, d, F // 32)
    hq, hs = u8(T * k, F // 2), u8(T * k, F // 32)
    return {
        "moe_quantize_mxfp4": dict(src=bf(T, d), codes=u8(T, d // 2), scales=u8(T, d // 32)),
        "moe_dequantize_mxfp4": dict(codes=u8(T, d // 2), scales=u8(T, d // 32), dst=bf(T, d)),
        "moe_expert_up_mxfp4": dict(p=prob(), aq=u8(T, d // 2), a_scale=u8(T, d // 32), src_token=i32(T * k), offsets=i32(E + 1),
                                    W1q=w1, w1s=s1, hq=hq, hs=hs),
        "moe_expert_down_mxfp4": dict(p=prob(), hq=hq, hs=hs, offsets=i32(E + 1), W2q=w2, w2s=s2, y_perm=bf(T * k, d)),
        "moe_forward_mxfp4": dict(p=prob(), x=bf(T, d), Wg=bf(E, d), bg=torch.zeros(E), W1q=w1, w1s=s1, W2q=w2, w2s=s2,
                                  y=bf(T, d), logits=torch.zeros(T, E),
                                  info=dict(topk_idx=i32(T, k), topk_w=torch.zeros(T, k), counts=i32(E), offsets=i32(E + 1),
                                            slot=i32(T, k), src_token=i32(T * k))),
        "moe_orthogonalize": dict(grad=torch.zeros(2, 24, 40), out=bf(2, 24, 40), momentum=torch.zeros(2, 24, 40), ws=u8(16))}


TYPES = [("moe_quantize_mxfp4", "src", "float16"), ("moe_quantize_mxfp4", "codes", "float32"), ("moe_quantize_mxfp4", "scales", "float32"),
         ("moe_dequantize_mxfp4", "dst", "float16"), ("moe_dequantize_mxfp4", "codes", "int32"), ("moe_dequantize_mxfp4", "scales", "bfloat16"),
         ("moe_expert_up_mxfp4", "aq", "float8_e4m3fn"), ("moe_expert_up_mxfp4", "a_scale", "float32"),
         ("moe_expert_up_mxfp4", "src_token", "int64"), ("moe_expert_up_mxfp4", "offsets", "int64"), ("moe_expert_up_mxfp4", "W1q", "bfloat16"),
         ("moe_expert_up_mxfp4", "w1s", "float32"), ("moe_expert_up_mxfp4", "hq", "bfloat16"), ("moe_expert_up_mxfp4", "hs", "float32"),
         ("moe_expert_down_mxfp4", "hq", "float8_e4m3fn"), ("moe_expert_down_mxfp4", "hs", "float16"), ("moe_expert_down_mxfp4", "offsets", "float32"),
         ("moe_expert_down_mxfp4", "W2q", "float32"), ("moe_expert_down_mxfp4", "w2s", "float32"), ("moe_expert_down_mxfp4", "y_perm", "float32"),
         ("moe_forward_mxfp4", "x", "float32"), ("moe_forward_mxfp4", "Wg", "float32"), ("moe_forward_mxfp4", "bg", "bfloat16"),
         ("moe_forward_mxfp4", "W1q", "float8_e4m3fn"), ("moe_forward_mxfp4", "w1s", "float32"), ("moe_forward_mxfp4", "W2q", "bfloat16"),
         ("moe_forward_mxfp4", "w2s", "float32"), ("moe_forward_mxfp4", "y", "float16"), ("moe_forward_mxfp4", "logits", "bfloat16"),
         ("moe_forward_mxfp4", "topk_idx", "int64"), ("moe_forward_mxfp4", "topk_w", "bfloat16"),
         ("moe_orthogonalize", "grad", "float16"), ("moe_orthogonalize", "out", "float32"), ("moe_orthogonalize", "momentum", "bfloat16")]


@pytest.mark.parametrize("fn,name,dtype", TYPES)
def test_bindings_refuse_other_element_types(fn, name, dtype):
    torch = pytest.importorskip("torch")
    a = calls(torch)[fn]
    holder = a if name in a else a["info"]
    holder[name] = torch.zeros(holder[name].shape).to(getattr(torch, dtype))
    with pytest.raises(TypeError, match=name):
        getattr(moe, fn)(**a, stream=0)


def sizes():
    torch = pytest.importorskip("torch")
    for fn, a in calls(torch).items():
        for name, t in {**a, **a.get("info", {})}.items():
            if torch.is_tensor(t) and name not in ("src", "dst", "grad", "ws"):
                yield fn, name


@pytest.mark.parametrize("fn,name", list(sizes()))
def test_bindings_refuse_tensors_that_are_too_small(fn, name):
    torch = pytest.importorskip("torch")
    a = calls(torch)[fn]
    holder = a if name in a else a["info"]
    holder[name] = holder[name].new_zeros(holder[name].numel() - 1)
    with pytest.raises(ValueError, match=name):
        getattr(moe, fn)(**a, stream=0)


@pytest.mark.parametrize("fn", list(calls(pytest.importorskip("torch"))))
def test_bindings_refuse_host_tensors(fn):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="GPU"):
        getattr(moe, fn)(**calls(torch)[fn], stream=0)


@pytest.mark.parametrize("fn", list(calls(pytest.importorskip("torch"))))
def test_bindings_as_a_process_first_call(fn, monkeypatch):
    """Before any call has looked up the element types."""
    torch = pytest.importorskip("torch")
    for name in ("_f32", "_i32", "_bf16", "_codes"):
        monkeypatch.setattr(moe, name, None)
    monkeypatch.setattr(moe, "_packed", ())
    monkeypatch.setattr(moe, "_device", None)
    monkeypatch.setattr(moe, "_src_types", {})
    monkeypatch.setattr(moe, "_scale_types", {})
    with pytest.raises(ValueError, match="GPU"):
        getattr(moe, fn)(**calls(torch)[fn], stream=0)


def test_bindings_pass_plain_addresses():
    """Plain addresses reach the library, which refuses the workspace or the address."""
    torch = pytest.importorskip("torch")
    for fn, a in calls(torch).items():
        if "p" not in a:
            continue
        a = {n: FAKE if torch.is_tensor(t) else None if n == "info" else t for n, t in a.items()}
        a["W1q" if "W1q" in a else "W2q"] = FAKE + 8
        with pytest.raises(moe.MoeError, match="W[12]"):
            getattr(moe, fn)(**a, stream=0)


def test_orthogonalize_binding_shapes():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="grad"):
        moe.moe_orthogonalize(torch.zeros(8), torch.zeros(8).bfloat16(), stream=0)


def test_reference_update_error_goes_by_the_matrix_and_the_steps():
    """The fp16 roundings' emulation: what they cost usual gradients at 5 steps they exceed
    where singular values are equal and in longer runs."""
    def error(u, steps):
        want = ref.orthogonal_by_products(u, steps)
        return np.linalg.norm(ref.orthogonal_fp16(u, steps) - want) / np.linalg.norm(want)

    g = np.random.default_rng(9)
    normal, equal = g.standard_normal((100, 140)), np.kron(np.eye(4), np.ones((25, 35)))
    assert error(normal, 5) <= 1.5e-3 < error(normal, 14) <= 2e-2
    assert 1.5e-3 < error(np.eye(300, 1000), 5) <= 1.2e-2
    assert 3e-3 < error(equal, 5) <= 1.2e-2 and error(equal, 8) <= 3e-2


@pytest.mark.parametrize("count,rows,cols", [(5000, 8, 65536), (2000, 65536, 16), (32768, 8, 16), (8192, 64, 1024), (1500, 33, 4096)])
def test_orthogonalize_workspace_of_few_rows_stays_small(count, rows, cols):
    """Up to 64 rows the usual steps read the gradient twice and keep sums of its small side,
    no copies of the batch; those of longer runs are taken in parts of 1 GiB, with at most
    64 MiB of partial tiles."""
    n = moe.moe_orthogonalize_workspace_size(count, rows, cols)
    mt = -(-min(rows, cols) // 16)  # tiles of 16: fp64 on and below the diagonal, fp32 all of them
    small = count * (mt * (mt + 1) // 2 * 2048 + mt * mt * 1024 + 8) + (1 << 20)
    assert n <= max(1088 << 20, small), f"{n / 2 ** 20:.0f} MiB"
    # a single matrix of such rows fits as ever
    assert moe.moe_orthogonalize_workspace_size(1, rows, cols) <= 320 << 20


@pytest.mark.parametrize("name", ["out", "momentum"])
@pytest.mark.parametrize("shape", [(2, 40, 24), (24, 2, 40), (2, 960), (1920,), (3, 24, 40)])
def test_orthogonalize_refuses_other_shapes(name, shape):
    """As many values in another order, which would be filled as if they were grad's, or more."""
    torch = pytest.importorskip("torch")
    a = calls(torch)["moe_orthogonalize"]
    a[name] = a[name].new_zeros(shape)
    with pytest.raises(ValueError, match=name):
        moe.moe_orthogonalize(**a, stream=0)


def test_orthogonalize_takes_a_batch_of_one_either_way():
    torch = pytest.importorskip("torch")
    g = torch.zeros(24, 40)
    with pytest.raises(ValueError, match="GPU"):  # past the shapes, to the next check
        moe.moe_orthogonalize(g, g[None].bfloat16(), momentum=g[None].clone(), stream=0)


class Handle:
    """A stream of GPU 0."""
    device_index, cuda_stream = 0, 0x1000


@pytest.mark.parametrize("fn", list(calls(pytest.importorskip("torch"))))
@pytest.mark.parametrize("stream", [None, 0, Handle()], ids=["none", "null", "stream"])
def test_bindings_refuse_tensors_of_another_gpu(fn, stream, monkeypatch):
    """The current GPU is 0, the tensors are on GPU 1: without a stream, on the null stream and on
    a stream of GPU 0 the kernels would run on GPU 0 and read addresses of GPU 1."""
    torch = pytest.importorskip("torch")

    class OnGpu1(torch.Tensor):
        def get_device(self):
            return 1

    def place(v):
        return {n: place(t) for n, t in v.items()} if isinstance(v, dict) else v.as_subclass(OnGpu1) if torch.is_tensor(v) else v

    moe._fill_packed()
    monkeypatch.setattr(moe, "_device", lambda: 0)
    monkeypatch.setattr(moe, "load", lambda: pytest.fail("reached the library"))
    a = place(calls(torch)[fn])
    with pytest.raises(ValueError, match="on GPU 1, not on GPU 0"):
        getattr(moe, fn)(**a, stream=stream)
    # a bare handle's GPU is not known: the tensors have to agree with each other
    moe._on_gpu(0x1000, [t for t in a.values() if torch.is_tensor(t)])
