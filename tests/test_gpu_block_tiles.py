"""The block-scaled FP8 products on every tile and epilogue that a call can reach,
whole and split along K, and with rotated slices (K 4096): the expert layers from
ragged segments, and the layer, whose down projection leaves fp32 rows.  References
in 64 bits (tests/_block_ref.py), the bounds those of tests/test_gpu_block_fp8.py."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_logit_amd as moe
import _block_ref as ref
import test_gpu_block_fp8 as base

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BLK = ref.BLK
dev = base.dev


def stack(g, E, n, K, f32):
    """Random codes and scales of E matrices [n][K]."""
    codes = g.integers(0, 0x60, (E, n, K), dtype=np.uint8) | (g.integers(0, 2, (E, n, K), dtype=np.uint8) << 7)
    if f32:
        return codes, (0.01 * (0.5 + g.random((E, n // BLK, K // BLK)))).astype(np.float32)
    return codes, g.integers(117, 123, (E, n // BLK, K // BLK), dtype=np.uint8)


def numbers(codes, scales):
    s = scales.astype(np.float64)
    return ref.widen_matrix(codes, s if scales.dtype == np.float32 else np.exp2(s - 127))


def rows_of(total, parts):
    """Segments of about total / parts rows, ragged by up to 8 either way."""
    n = np.full(parts, total // parts) + (np.arange(parts) * 5 % 17 - 8) * (parts > 1)
    n[-1] += total - n.sum()
    return n


# kind, experts, rows in all, K, columns of the output.  On 256 CUs:
SHAPES = [
    # 64 x 128 tiles, rotated slices, 8 parts
    ("down", 2, 33, 4096, 384), ("relu", 2, 33, 4096, 384),
    # 64 x 256: a tail of a few tiles in 4 and 8 parts; SwiGLU rotated
    ("down", 13, 1144, 2048, 2560), ("down", 13, 1144, 4096, 2560), ("relu", 13, 1144, 4096, 2560),
    ("swiglu", 2, 33, 4096, 384),
    # 96 x 256
    ("down", 7, 1050, 2048, 4864), ("down", 7, 1050, 4096, 4864), ("relu", 7, 1050, 4096, 4864),
    ("swiglu", 7, 1050, 2048, 2432), ("swiglu", 7, 1050, 4096, 2432),
    # 128 x 256: E8M0 scales, all tiles in one round; fp32 scales, split
    ("down", 1, 2100, 2048, 3840), ("relu", 1, 2100, 2048, 3840),
    ("down", 2, 2100, 2048, 4352), ("relu", 2, 2100, 2048, 4352),
    # 256 x 256 (128 x 256 with fp32 scales), split
    ("down", 2, 2100, 2048, 7680), ("relu", 2, 2100, 2048, 7680),
]


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_products(shape, f32):
    kind, E, total, K, N = shape
    print(f"[block tiles] {shape} f32={f32}", flush=True)
    g = base.gen(total + K + N)
    up = kind != "down"
    p = moe.problem(total, K if up else N, E, 1, N if up else K, act="swiglu" if kind == "swiglu" else "relu")
    off = np.concatenate([[0], np.cumsum(rows_of(total, E))]).astype(np.int32)
    assert np.all(np.diff(off) > 0) and off[-1] == total
    W, s = stack(g, E, 2 * N if kind == "swiglu" else N, K, f32)
    aq, ae = ref.quantise(g.standard_normal((total, K)) * np.exp(g.standard_normal((total, 1))))
    a = ref.widen_rows(aq, ae)
    src = g.permutation(total).astype(np.int32)
    dA, dS, dW, dw, dO = dev(aq), dev((ae + 127).astype(np.uint8)), dev(W), dev(s), dev(off)

    def call(ws):
        if up:
            out = torch.full((total, N), 0x5A, dtype=torch.uint8, device="cuda")
            hs = torch.full((total, N // BLK), 77, dtype=torch.uint8, device="cuda")
            moe.moe_expert_up_fp8_block(p, dA, dS, dev(src), dO, dW, dw, out, hs, ws=ws)
            torch.cuda.synchronize()
            return out.cpu().numpy(), hs.cpu().numpy()
        y = torch.full((total, N), 3.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_down_fp8_block(p, dA, dS, dO, dW, dw, y, ws=ws)
        torch.cuda.synchronize()
        return (y.double().cpu().numpy(),)

    ws = torch.empty(moe.moe_fp8_block_workspace_size(p), dtype=torch.uint8, device="cuda")
    whole, split, again = call(None), call(ws.fill_(0)), call(ws.fill_(0xFF))
    assert all(np.array_equal(x, y) for x, y in zip(split, again))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        w = numbers(W[e], s[e])
        if up:
            h, dh = ref.hidden(a[src[r]], w, "swiglu" if kind == "swiglu" else "relu", N)
        else:
            v, dv = ref.product(a[r], w)
        for name, got in (("whole", whole), ("split", split)):
            what = f"expert {e}, {name}"
            if up:
                ref.check_quantised(got[0][r], got[1][r].astype(np.int64) - 127, h, dh, what)
                continue
            over = np.abs(got[0][r] - v) - (dv + ref.U8 * (np.abs(v) + dv))
            assert np.all(over <= 0), f"{what}: {over.max():.3e} beyond the bound"
            # half a bf16 step evenly: U8 / sqrt(3) in the root mean square
            assert np.linalg.norm(got[0][r] - v) <= 0.6 * ref.U8 * np.linalg.norm(v), f"{what}: in the norm"


# tokens, width, experts, k, F.  The down projection (K = F, columns = width) on 256 CUs:
LAYERS = [
    (520, 2560, 13, 1, 2048),    # 64 x 256, whole
    (1144, 2560, 13, 1, 2048),   # 64 x 256, split
    (1050, 7168, 7, 1, 2048),    # 96 x 256, whole (its last round is too full to split)
    (1050, 4864, 7, 1, 2048),    # 96 x 256, split
    (2100, 3840, 1, 1, 2048),    # 128 x 256, whole
    (1050, 4352, 2, 2, 2048),    # 256 x 256, whole; fp32 scales: 128 x 256, split
    (1050, 7680, 2, 2, 2048),    # 256 x 256, split; fp32 scales: 128 x 256, split
]


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "-".join(map(str, s)))
def test_layer_on_wide_tiles(shape, f32):
    """Given logits spread the tokens evenly; the hidden codes are those of the
    public steps (the same kernels on the same inputs), so that y is held to the
    fp32 rows of the down projection and one rounding."""
    T, d, E, k, F = shape
    print(f"[block layer tiles] {shape} f32={f32}", flush=True)
    g = base.gen(T + d)
    p = moe.problem(T, d, E, k, F, act="relu")
    W1, s1 = stack(g, E, F, d, f32)
    W2, s2 = stack(g, E, d, F, f32)
    x, _ = base.bf16(g.standard_normal((T, d)))
    z = g.standard_normal((T, E)).astype(np.float32) * 0.1
    z[np.arange(T), np.arange(T) % E] += 3.0
    dW1, d1, dW2, d2, dz = dev(W1), dev(s1), dev(W2), dev(s2), dev(z)
    info = {"topk_idx": torch.empty(T, k, dtype=torch.int32, device="cuda"),
            "topk_w": torch.empty(T, k, dtype=torch.float32, device="cuda"),
            "offsets": torch.empty(E + 1, dtype=torch.int32, device="cuda"),
            "slot": torch.empty(T, k, dtype=torch.int32, device="cuda"),
            "src_token": torch.empty(T * k, dtype=torch.int32, device="cuda")}
    ws = torch.empty(moe.moe_fp8_block_workspace_size(p), dtype=torch.uint8, device="cuda")
    got = []
    for fill in (0, 0xFF):
        y = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        moe.moe_forward_fp8_block(p, x, None, None, dW1, d1, dW2, d2, y, logits=dz, info=info, ws=ws.fill_(fill))
        torch.cuda.synchronize()
        got.append(y.double().cpu().numpy())
    assert np.array_equal(*got)
    i = {n: t.cpu().numpy() for n, t in info.items()}
    xq = torch.empty(T, d, dtype=torch.uint8, device="cuda")
    xs = torch.empty(T, d // BLK, dtype=torch.uint8, device="cuda")
    hq = torch.empty(T * k, F, dtype=torch.uint8, device="cuda")
    hs = torch.empty(T * k, F // BLK, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_fp8_block(x, xq, xs)
    moe.moe_expert_up_fp8_block(p, xq, xs, info["src_token"], info["offsets"], dW1, d1, hq, hs, ws=ws)
    torch.cuda.synchronize()
    h = ref.widen_rows(hq.cpu().numpy(), hs.cpu().numpy().astype(np.int64) - 127)
    want, bound = np.zeros((T, d)), np.zeros((T, d))
    for e in range(E):
        r = np.arange(i["offsets"][e], i["offsets"][e + 1])
        v, dv = ref.product(h[r], numbers(W2[e], s2[e]))
        t, j = np.nonzero(i["topk_idx"] == e)
        at, w = i["slot"][t, j] - r[0], i["topk_w"][t, j].astype(np.float64)[:, None]
        np.add.at(want, t, w * v[at])
        # the combine: a product and an addition for each of at most 2 choices
        np.add.at(bound, t, w * (dv[at] + 4 * ref.U24 * (np.abs(v[at]) + dv[at])))
    over = np.abs(got[0] - want) - (bound + ref.U8 * (np.abs(want) + bound))
    assert np.all(over <= 0), f"{over.max():.3e} beyond the bound"
    assert np.linalg.norm(got[0] - want) <= 0.6 * ref.U8 * np.linalg.norm(want)


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("shape", [(70, 256, 8, 5, 256, "relu", False, 0.0), (41, 384, 9, 8, 256, "swiglu", True, 0.8),
                                   (33, 256, 4, 4, 128, "relu", False, 1.0)], ids=lambda s: "-".join(map(str, s)))
def test_layer_of_many_choices(shape, f32):
    """Four to eight choices a token, some of them dropped."""
    base.test_layer(shape, f32)


@pytest.mark.parametrize("shape", [(9, 384, 2, 1, 256, "relu", "even"), (300, 384, 2, 1, 256, "swiglu", "even")],
                         ids=lambda s: "-".join(map(str, s)))
def test_the_outermost_e8m0_scales(shape):
    """Bytes 0 and 254 on either side, whose products stay in range."""
    c = base.Case(*shape, False)
    c.xs[:, 0], c.xs[:, 1], c.xs[:, 2] = 0, 254, 100
    c.x = ref.widen_rows(c.xq, c.xs.astype(np.int64) - 127)
    c.s1[:, :, 0], c.s1[:, :, 1], c.s1[:, :, 2] = 250, 0, 140
    c.hs[:, 0], c.hs[:, 1] = 0, 254
    c.h = ref.widen_rows(c.hq, c.hs.astype(np.int64) - 127)
    c.s2[:, :, 0], c.s2[:, :, 1] = 254, 0
    for e in range(c.E):
        c.w1[e] = ref.widen_matrix(c.W1[e], np.exp2(c.s1[e].astype(np.float64) - 127))
        c.w2[e] = ref.widen_matrix(c.W2[e], np.exp2(c.s2[e].astype(np.float64) - 127))
    c.check_up(*c.up())
    c.check_down(c.down())


@pytest.mark.parametrize("shape", [(9, 640, 2, 1, 640, "relu", "even"), (300, 640, 2, 1, 640, "swiglu", "even")],
                         ids=lambda s: "-".join(map(str, s)))
def test_fp32_scales_of_every_kind(shape):
    """Negative, zero, subnormal, tiny and large weight scales."""
    c = base.Case(*shape, True)
    for s in (c.s1, c.s2):
        s[:, :, 0] *= -1
        s[:, :, 1] = 0
        s[:, :, 2] = 1e-40
        s[:, ::2, 3] *= 2.0 ** 20
        s[:, 1::2, 3] *= 2.0 ** -30
    for e in range(c.E):
        c.w1[e] = ref.widen_matrix(c.W1[e], c.s1[e])
        c.w2[e] = ref.widen_matrix(c.W2[e], c.s2[e])
    c.check_up(*c.up())
    c.check_down(c.down())
