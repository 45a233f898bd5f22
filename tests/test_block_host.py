"""Host checks of the block-scaled FP8 experts and of the balance loss: sizes,
refusals before anything is enqueued, and the 64-bit references themselves.
No kernel is launched (these run without a GPU)."""
import ctypes

import numpy as np
import pytest

import mixture_experts_layer_logit_amd as moe
import _block_ref as ref

FAKE = 1 << 20  # an aligned, never dereferenced address
BIG = 1 << 40


def status(fn, *args):
    return getattr(moe.load(), fn)(*args)


def prob(**kw):
    a = dict(T=64, d=256, E=8, k=2, F=384, act="swiglu")
    a.update(kw)
    return moe.problem(a.pop("T"), a.pop("d"), a.pop("E"), a.pop("k"), a.pop("F"), **a)


# ---------------------------------------------------------------- the references
def test_reference_codes():
    assert ref.POS[126] == 448 and ref.POS[1] == 2.0 ** -9 and len(ref.POS) == 127
    assert list(ref.encode(np.array([1.0625, 1.1875, 448.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10]))) == [
        0x38, 0x3A, 0x7E, 0x80, 0x00, 0x02]
    try:
        import torch
    except ImportError:
        return
    v = np.random.default_rng(0).standard_normal(100000) * 20
    t = torch.from_numpy(v).float()
    assert np.array_equal(ref.encode(t.double().numpy()), t.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_scales():
    for a, e in ((0.0, 0), (448.0, 0), (448.0001, 1), (224.0, -1), (224.5, 0), (2.0 ** -200, -127), (1.0, -8)):
        assert ref.exponent(a) == e
    for a in np.exp(np.random.default_rng(1).uniform(-60, 60, 2000)):
        e = int(ref.exponent(a))
        assert a <= 448 * 2.0 ** e and a > 224 * 2.0 ** e


def test_reference_gradient_by_differences():
    g = np.random.default_rng(2)
    z, idx = g.standard_normal((6, 4)), g.integers(0, 4, (6, 2))
    off = np.array([0, 2, 2, 5])
    for norm in (False, True):
        _, _, dz, _ = ref.balance(z, idx, off, 0.6, 0.2, norm, 1.7)
        assert np.all(np.isnan(dz[5]))
        for t in range(5):
            for e in range(4):
                l = []
                for s in (1e-5, -1e-5):
                    zz = z.copy()
                    zz[t, e] += s
                    v = ref.balance(zz, idx, off, 0, 0, norm, 1.7)[1]
                    l.append(0.6 * v[0] + 0.2 * v[1])
                assert abs((l[0] - l[1]) / 2e-5 - dz[t, e]) < 1e-8


# ---------------------------------------------------------------- refusals
def quantise(src=FAKE, dt=moe.MOE_BF16, rows=8, K=256, br=1, codes=FAKE, scales=FAKE, kind=moe.MOE_SCALE_E8M0):
    return status("moe_quantize_fp8_block", src, dt, rows, K, br, codes, scales, kind, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), moe.MOE_ERR_INVALID_ARG), (dict(kind=2), moe.MOE_ERR_INVALID_ARG), (dict(kind=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(br=0), moe.MOE_ERR_INVALID_ARG), (dict(br=64), moe.MOE_ERR_INVALID_ARG), (dict(rows=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(K=64), moe.MOE_ERR_UNSUPPORTED), (dict(K=192), moe.MOE_ERR_UNSUPPORTED), (dict(K=65536 + 128), moe.MOE_ERR_UNSUPPORTED),
    (dict(rows=1 << 31), moe.MOE_ERR_UNSUPPORTED), (dict(rows=(1 << 31) - 1, K=65536), moe.MOE_ERR_UNSUPPORTED),
    (dict(src=None), moe.MOE_ERR_INVALID_ARG), (dict(src=FAKE + 8), moe.MOE_ERR_INVALID_ARG),
    (dict(codes=None), moe.MOE_ERR_INVALID_ARG), (dict(codes=FAKE + 8), moe.MOE_ERR_INVALID_ARG),
    (dict(scales=None), moe.MOE_ERR_INVALID_ARG),
    (dict(scales=FAKE + 2, kind=moe.MOE_SCALE_F32), moe.MOE_ERR_INVALID_ARG)])
def test_quantise_refusals(kw, want):
    assert quantise(**kw) == want
    assert moe.load().moe_last_error()


def test_quantise_of_no_rows():
    assert quantise(rows=0, src=None, codes=None, scales=None) == moe.MOE_OK


@pytest.mark.parametrize("kw,want", [(dict(dtype="f32"), moe.MOE_ERR_UNSUPPORTED), (dict(d=320), moe.MOE_ERR_UNSUPPORTED),
                                     (dict(F=448), moe.MOE_ERR_UNSUPPORTED), (dict(k=9, E=16), moe.MOE_ERR_UNSUPPORTED),
                                     (dict(T=-1), moe.MOE_ERR_INVALID_ARG)])
def test_layer_problem_refusals(kw, want):
    p = prob(**kw)
    n = ctypes.c_size_t()
    assert status("moe_fp8_block_workspace_size", ctypes.byref(p), ctypes.byref(n)) == want
    assert status("moe_expert_up_fp8_block", ctypes.byref(p), *[FAKE] * 6, 0, FAKE, FAKE, None, 0, None) == want
    assert status("moe_expert_down_fp8_block", ctypes.byref(p), *[FAKE] * 5, 0, FAKE, None, 0, None) == want
    assert status("moe_forward_fp8_block", ctypes.byref(p), *[FAKE] * 7, 0, FAKE, None, None, FAKE, BIG, None) == want


def test_workspace_size_needs_its_result():
    assert status("moe_fp8_block_workspace_size", ctypes.byref(prob()), None) == moe.MOE_ERR_INVALID_ARG
    assert status("moe_balance_workspace_size", ctypes.byref(prob()), 1, None) == moe.MOE_ERR_INVALID_ARG


UP = dict(aq=FAKE, as_=FAKE, src=FAKE, off=FAKE, w=FAKE, ws=FAKE, kind=0, hq=FAKE, hs=FAKE, work=None, n=0)


@pytest.mark.parametrize("kw,want", [
    (dict(aq=None), 1), (dict(aq=FAKE + 4), 1), (dict(as_=None), 1), (dict(src=FAKE + 2), 1), (dict(off=None), 1),
    (dict(off=FAKE + 1), 1), (dict(w=None), 1), (dict(w=FAKE + 8), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 1, kind=1), 1), (dict(kind=7), 1), (dict(hq=None), 1), (dict(hq=FAKE + 8), 1), (dict(hs=None), 1),
    (dict(work=FAKE, n=16), 3), (dict(work=FAKE + 8, n=BIG), 1)])
def test_up_refusals(kw, want):
    a = dict(UP, **kw)
    assert status("moe_expert_up_fp8_block", ctypes.byref(prob()), a["aq"], a["as_"], a["src"], a["off"], a["w"], a["ws"],
                  a["kind"], a["hq"], a["hs"], a["work"], a["n"], None) == want
    assert moe.load().moe_last_error()


def test_gather_beyond_32_bits_is_refused():
    p = prob(T=1 << 24, d=256, E=8, k=1)
    assert status("moe_expert_up_fp8_block", ctypes.byref(p), *[FAKE] * 6, 0, FAKE, FAKE, None, 0, None) == moe.MOE_ERR_UNSUPPORTED
    assert status("moe_forward_fp8_block", ctypes.byref(p), *[FAKE] * 7, 0, FAKE, None, None, FAKE, BIG, None) == moe.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("at,bad,want", [(0, None, 1), (0, FAKE + 8, 1), (1, None, 1), (2, None, 1), (2, FAKE + 1, 1),
                                         (3, FAKE + 8, 1), (4, None, 1), (5, 5, 1), (6, None, 1), (6, FAKE + 2, 1)])
def test_down_refusals(at, bad, want):
    a = [FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE]
    a[at] = bad
    assert status("moe_expert_down_fp8_block", ctypes.byref(prob()), *a, None, 0, None) == want


@pytest.mark.parametrize("at,bad,want", [(0, None, 1), (1, FAKE + 8, 1), (2, FAKE + 2, 1), (3, None, 1), (4, None, 1),
                                         (5, None, 1), (6, None, 1), (7, 3, 1), (8, None, 1), (9, FAKE + 2, 1),
                                         (11, None, 1), (12, 64, 3)])
def test_layer_refusals(at, bad, want):
    a = [FAKE] * 7 + [0, FAKE, None, None, FAKE, BIG]
    a[at] = bad
    assert status("moe_forward_fp8_block", ctypes.byref(prob()), *a, None) == want


def test_layer_with_given_logits_needs_them():
    a = [FAKE, None, None] + [FAKE] * 4 + [0, FAKE, None, None, FAKE, BIG]
    assert status("moe_forward_fp8_block", ctypes.byref(prob()), *a, None) == moe.MOE_ERR_INVALID_ARG


def test_binding_checks_scale_types():
    torch = pytest.importorskip("torch")
    p = prob()
    f, b, h = torch.zeros(4), torch.zeros(4, dtype=torch.uint8), torch.zeros(4, dtype=torch.float16)
    with pytest.raises(TypeError):
        moe.moe_quantize_fp8_block(torch.zeros(2, 128), b, h, stream=0)
    with pytest.raises(TypeError):
        moe.moe_expert_up_fp8_block(p, b, f, None, b, b, b, b, b, stream=0)
    with pytest.raises(TypeError):
        moe.moe_expert_down_fp8_block(p, b, b, b, b, h, b, stream=0)
    with pytest.raises(TypeError):
        moe.moe_forward_fp8_block(p, b, None, None, b, b, b, f, b, stream=0)


BAL = dict(logits=FAKE, idx=FAKE, off=FAKE, n=3, a=0.1, z=0.1, counts=FAKE, losses=FAKE, dz=FAKE, ws=FAKE, size=BIG)


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), 1), (dict(logits=FAKE + 2), 1), (dict(idx=None), 1), (dict(off=None), 1), (dict(off=FAKE + 1), 1),
    (dict(n=0), 1), (dict(n=-4), 1), (dict(n=(1 << 20) + 1), 2), (dict(a=float("nan")), 1), (dict(z=float("inf")), 1),
    (dict(counts=None), 1), (dict(losses=None), 1), (dict(dz=FAKE + 2), 1), (dict(ws=None), 1), (dict(size=8), 3)])
def test_balance_refusals(kw, want):
    b = dict(BAL, **kw)
    assert status("moe_balance_loss", ctypes.byref(prob()), b["logits"], b["idx"], b["off"], b["n"], b["a"], b["z"],
                  b["counts"], b["losses"], b["dz"], b["ws"], b["size"], None) == want
    assert moe.load().moe_last_error()


def test_binding_checks_the_offsets_type():
    torch = pytest.importorskip("torch")
    f, i = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        moe.moe_balance_loss(prob(), f, f, i, f, f, None, stream=0)


def test_balance_counts_beyond_32_bits_are_refused():
    n = ctypes.c_size_t()
    assert status("moe_balance_workspace_size", ctypes.byref(prob(E=1024, k=2)), 1 << 21, ctypes.byref(n)) == 2
    assert status("moe_balance_workspace_size", ctypes.byref(prob(E=1024, k=2)), 1 << 20, ctypes.byref(n)) == 0


# ------------------------------------------------- the binding: element types and sizes
def balance_args(torch):
    """A call of 64 tokens, 8 experts, 2 choices and 2 sequences, on the host: nothing
    that is refused reads it."""
    return dict(logits=torch.zeros(64, 8), topk_idx=torch.zeros(64, 2, dtype=torch.int32),
                seq_offsets=torch.zeros(3, dtype=torch.int32), counts=torch.zeros(2, 8, dtype=torch.int32),
                losses=torch.zeros(2), dlogits=torch.zeros(64, 8))


@pytest.mark.parametrize("name,dtype", [
    ("topk_idx", "int64"),       # what torch.topk returns
    ("topk_idx", "float32"), ("seq_offsets", "float32"), ("seq_offsets", "int64"), ("logits", "bfloat16"),
    ("logits", "float64"), ("dlogits", "bfloat16"), ("dlogits", "float16"), ("counts", "int64"), ("counts", "float32"),
    ("losses", "float64"), ("losses", "int32")])
def test_balance_binding_refuses_other_element_types(name, dtype):
    torch = pytest.importorskip("torch")
    a = balance_args(torch)
    a[name] = a[name].to(getattr(torch, dtype))
    with pytest.raises(TypeError, match=name):
        moe.moe_balance_loss(prob(), **a, stream=0)


@pytest.mark.parametrize("name,shape", [("logits", (63, 8)), ("topk_idx", (64, 1)), ("counts", (1, 8)), ("losses", (1,)),
                                        ("dlogits", (64, 7))])
def test_balance_binding_refuses_tensors_that_are_too_small(name, shape):
    torch = pytest.importorskip("torch")
    a = balance_args(torch)
    a[name] = a[name].new_zeros(shape)
    with pytest.raises(ValueError, match=name):
        moe.moe_balance_loss(prob(), **a, stream=0)


def test_balance_binding_passes_what_fits():
    """Larger buffers, no gradient and plain addresses reach the library (which
    refuses the missing workspace)."""
    torch = pytest.importorskip("torch")
    a = balance_args(torch)
    for change in (dict(), dict(dlogits=None), dict(counts=torch.zeros(5, 8, dtype=torch.int32), losses=torch.zeros(7)),
                   dict(logits=FAKE, topk_idx=FAKE, counts=FAKE, losses=FAKE, dlogits=FAKE)):
        with pytest.raises(moe.MoeError) as err:
            moe.moe_balance_loss(prob(), **dict(a, **change), stream=0)
        assert err.value.status == moe.MOE_ERR_WORKSPACE


def fp8_block_calls(torch):
    """Arguments of the right types and sizes for every block FP8 entry point, on the
    host: nothing that is refused reads them."""
    T, d, E, k, F = 64, 256, 8, 2, 384

    def u8(*shape):
        return torch.zeros(*shape, dtype=torch.uint8)

    def i32(*shape):
        return torch.zeros(*shape, dtype=torch.int32)

    def bf(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16)

    w1, s1, w2, s2 = u8(E, 2 * F, d), u8(E, 2 * F // 128, d // 128), u8(E, d, F), u8(E, d // 128, F // 128)
    return {
        "moe_quantize_fp8_block": dict(src=bf(T, d), codes=u8(T, d), scales=u8(T, d // 128)),
        "moe_expert_up_fp8_block": dict(p=prob(), aq=u8(T, d), a_scale=u8(T, d // 128), src_token=i32(T * k), offsets=i32(E + 1),
                                        W1q=w1, w1s=s1, hq=u8(T * k, F), hs=u8(T * k, F // 128)),
        "moe_expert_down_fp8_block": dict(p=prob(), hq=u8(T * k, F), hs=u8(T * k, F // 128), offsets=i32(E + 1), W2q=w2, w2s=s2,
                                          y_perm=bf(T * k, d)),
        "moe_forward_fp8_block": dict(p=prob(), x=bf(T, d), Wg=bf(E, d), bg=torch.zeros(E), W1q=w1, w1s=s1, W2q=w2, w2s=s2,
                                      y=bf(T, d), logits=torch.zeros(T, E),
                                      info=dict(topk_idx=i32(T, k), topk_w=torch.zeros(T, k), counts=i32(E), offsets=i32(E + 1),
                                                slot=i32(T, k), src_token=i32(T * k)))}


@pytest.mark.parametrize("fn,name,dtype", [
    ("moe_quantize_fp8_block", "codes", "float32"), ("moe_quantize_fp8_block", "codes", "float8_e4m3fnuz"),
    ("moe_expert_up_fp8_block", "aq", "bfloat16"), ("moe_expert_up_fp8_block", "aq", "float8_e5m2"),
    ("moe_expert_up_fp8_block", "src_token", "int64"), ("moe_expert_up_fp8_block", "offsets", "int64"),
    ("moe_expert_up_fp8_block", "W1q", "bfloat16"), ("moe_expert_up_fp8_block", "hq", "bfloat16"),
    ("moe_expert_down_fp8_block", "hq", "bfloat16"), ("moe_expert_down_fp8_block", "offsets", "float32"),
    ("moe_expert_down_fp8_block", "W2q", "float32"), ("moe_expert_down_fp8_block", "y_perm", "float32"),
    ("moe_expert_down_fp8_block", "y_perm", "float16"),
    ("moe_forward_fp8_block", "x", "float16"), ("moe_forward_fp8_block", "x", "float32"),
    ("moe_forward_fp8_block", "Wg", "float32"), ("moe_forward_fp8_block", "bg", "bfloat16"),
    ("moe_forward_fp8_block", "W1q", "bfloat16"), ("moe_forward_fp8_block", "W2q", "bfloat16"),
    ("moe_forward_fp8_block", "y", "float16"), ("moe_forward_fp8_block", "logits", "bfloat16"),
    ("moe_forward_fp8_block", "topk_idx", "int64"), ("moe_forward_fp8_block", "topk_w", "bfloat16"),
    ("moe_forward_fp8_block", "src_token", "int64")])
def test_block_bindings_refuse_other_element_types(fn, name, dtype):
    torch = pytest.importorskip("torch")
    a = fp8_block_calls(torch)[fn]
    holder = a if name in a else a["info"]
    holder[name] = torch.zeros(holder[name].shape).to(getattr(torch, dtype))
    with pytest.raises(TypeError, match=name):
        getattr(moe, fn)(**a, stream=0)


@pytest.mark.parametrize("fn,name,shape", [
    ("moe_quantize_fp8_block", "codes", (63, 256)), ("moe_quantize_fp8_block", "scales", (64, 1)),
    ("moe_forward_fp8_block", "x", (63, 256)), ("moe_forward_fp8_block", "y", (63, 256)),
    ("moe_forward_fp8_block", "logits", (64, 7)), ("moe_forward_fp8_block", "topk_idx", (64, 1)),
    ("moe_forward_fp8_block", "offsets", (8,))])
def test_block_bindings_refuse_tensors_that_are_too_small(fn, name, shape):
    torch = pytest.importorskip("torch")
    a = fp8_block_calls(torch)[fn]
    holder = a if name in a else a["info"]
    holder[name] = holder[name].new_zeros(shape)
    with pytest.raises(ValueError, match=name):
        getattr(moe, fn)(**a, stream=0)


@pytest.mark.parametrize("block_rows,scales", [(1, 7 * 2), (128, 2)])
def test_quantiser_sizes_count_the_blocks(block_rows, scales):
    """7 rows of 256 values: enough scales pass on to the library (which refuses
    the odd address), one fewer does not."""
    torch = pytest.importorskip("torch")
    src, codes = torch.zeros(8, 256)[1:].bfloat16(), torch.zeros(7 * 256 + 8, dtype=torch.uint8)[8:]
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_fp8_block(src, codes, torch.zeros(scales, dtype=torch.uint8), block_rows=block_rows, stream=0)
    with pytest.raises(ValueError, match="scales"):
        moe.moe_quantize_fp8_block(src, codes, torch.zeros(scales - 1, dtype=torch.uint8), block_rows=block_rows, stream=0)


def test_block_bindings_pass_what_fits():
    """Codes as float8_e4m3fn, scales as float8_e8m0fnu, larger buffers and plain
    addresses reach the library, which refuses the workspace."""
    torch = pytest.importorskip("torch")
    a = fp8_block_calls(torch)
    small = torch.zeros(16, dtype=torch.uint8)
    for bad in (None, FAKE + 8):
        with pytest.raises(moe.MoeError, match="codes"):
            moe.moe_quantize_fp8_block(**dict(a["moe_quantize_fp8_block"], codes=bad), stream=0)
    for fn in ("moe_expert_up_fp8_block", "moe_expert_down_fp8_block", "moe_forward_fp8_block"):
        plain, typed = dict(a[fn]), dict(a[fn])
        for n, t in a[fn].items():
            if torch.is_tensor(t) and t.dtype is torch.uint8:
                typed[n] = t.view(torch.float8_e8m0fnu if n in ("a_scale", "hs", "w1s", "w2s") else torch.float8_e4m3fn)
            elif torch.is_tensor(t):
                plain[n] = FAKE
        for call in (a[fn], plain, typed, dict(a[fn], **({"y": torch.zeros(65, 256).bfloat16()} if "y" in a[fn] else {}))):
            with pytest.raises(moe.MoeError) as err:
                getattr(moe, fn)(**call, ws=small, stream=0)
            assert err.value.status == moe.MOE_ERR_WORKSPACE
