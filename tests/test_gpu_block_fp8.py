"""FP8 experts scaled by blocks of 128, through the C ABI, against 64-bit
references (tests/_block_ref.py): the quantiser bit for bit, the expert layers
within bounds derived from the number of fp32 roundings and half a step of the
stored type, the layer against its own steps bit for bit and against the
64-bit layer, graph replays, other streams, and rows that have to stay as they
were."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_logit_amd as moe
import _block_ref as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BLK = 128


def gen(seed):
    return np.random.Generator(np.random.PCG64(seed))


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    """float array -> (bf16 CUDA tensor, its values in float64)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def weights(g, E, n, K, f32):
    """Codes, scales and the numbers they stand for, of one expert stack."""
    w = g.standard_normal((E, n, K)) * 0.05 * np.exp(g.standard_normal((E, n // BLK, 1, K // BLK, 1)) * 0.5).repeat(
        BLK, 2).repeat(BLK, 4).reshape(E, n, K)
    codes = np.empty((E, n, K), np.uint8)
    scales = np.empty((E, n // BLK, K // BLK), np.float32 if f32 else np.uint8)
    wide = np.empty((E, n, K))
    for e in range(E):
        if f32:  # any fp32 number: no power of two
            top = np.abs(w[e].reshape(n // BLK, BLK, K // BLK, BLK)).max(axis=(1, 3))
            s = (top / 448 * 1.01).astype(np.float32)
            codes[e] = ref.encode(w[e] / np.repeat(np.repeat(s.astype(np.float64), BLK, 0), BLK, 1))
            scales[e] = s
        else:
            codes[e], x = ref.quantise(w[e], BLK)
            s = np.exp2(x.astype(np.float64))
            scales[e] = x + 127
        wide[e] = ref.widen_matrix(codes[e], s)
    return codes, scales, wide


def segments(g, T, E, k, how):
    """Token of each permuted row and the segment borders."""
    if how == "one":       # every token's first choice on one expert, the others' segments empty
        idx = np.zeros((T, k), np.int64) + np.arange(k)[None, :]
    else:
        bias = -2.0 * np.log(1 + np.arange(E)) if how == "skew" else np.zeros(E)
        idx = np.argsort(-(g.standard_normal((T, E)) + bias), axis=1)[:, :k]
    flat = idx.reshape(-1)
    order = np.argsort(flat, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    return (order // k).astype(np.int32), off.astype(np.int32)


# ---------------------------------------------------------------- the quantiser
def edge_rows(K, rows, rng, dtype):
    """Rows with blocks of zeros, of one value on a scale's border and just past
    it, tiny and subnormal values, signed zeros and a lone outlier."""
    v = rng.standard_normal((rows, K)).astype(np.float32)
    for b in range(K // BLK):
        s = slice(b * BLK, (b + 1) * BLK)
        for r in range(rows):
            kind = (r * 7 + b) % 9
            if kind == 0:
                v[r, s] = 0.0
            elif kind == 1:
                v[r, s.start] = 448.0 * 2.0 ** (r % 5)
            elif kind == 2:
                v[r, s.start] = np.nextafter(np.float32(448), np.float32(1e9)) if dtype == "f32" else 450.0
            elif kind == 3:
                v[r, s] *= np.float32(2.0 ** -126)
            elif kind == 4:
                v[r, s] = np.float32(2.0 ** -133) * np.where(np.arange(BLK) % 3 == 0, -1, 1)
            elif kind == 5:
                v[r, s] = -0.0
                v[r, s.start + 5] = 1.0625  # a tie between two codes
            elif kind == 6:
                v[r, s] = 2.0 ** -9 * np.arange(BLK) / 4
            elif kind == 7:
                v[r, s] *= np.float32(2.0 ** 100)
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("rows,K,block_rows", [(1, 128, 1), (7, 384, 1), (33, 4096, 1), (1000, 640, 1), (1, 128, 128),
                                               (127, 256, 128), (129, 384, 128), (640, 1408, 128)])
def test_quantise_bit_exact(dtype, scale, rows, K, block_rows):
    print(f"[quantise block] {dtype} {scale} rows={rows} K={K} block_rows={block_rows}", flush=True)
    v = edge_rows(K, rows, gen(rows + K), dtype)
    src, wide = bf16(v) if dtype == "bf16" else (dev(v), v.astype(np.float64))
    codes = torch.full((rows, K), 0xA5, dtype=torch.uint8, device="cuda")
    nb = -(-rows // block_rows)
    scales = torch.zeros(nb, K // BLK, dtype=torch.uint8 if scale == "e8m0" else torch.float32, device="cuda")
    moe.moe_quantize_fp8_block(src, codes, scales, block_rows=block_rows)
    torch.cuda.synchronize()
    q, e = ref.quantise(wide, block_rows)
    want = (e + 127).astype(np.uint8) if scale == "e8m0" else np.exp2(e.astype(np.float64)).astype(np.float32)
    assert np.array_equal(scales.cpu().numpy(), want)
    assert np.array_equal(codes.cpu().numpy(), q)


# ---------------------------------------------------------------- the expert layers
# (T, d, E, k, F, act, how): one token; few rows; empty experts; one K block;
# widths that end inside a 256-column tile; segments that end inside a tile and
# on its border; K from 2048 on (split); many rows per expert
SHAPES = [
    (1, 128, 1, 1, 128, "relu", "even"),
    (1, 256, 8, 2, 384, "swiglu", "even"),
    (5, 384, 3, 3, 128, "swiglu", "even"),
    (17, 640, 7, 2, 640, "relu", "skew"),
    (64, 256, 4, 1, 256, "swiglu", "one"),
    (33, 2176, 5, 2, 384, "swiglu", "skew"),
    (100, 384, 6, 2, 2304, "relu", "even"),
    (300, 512, 2, 2, 384, "swiglu", "even"),
    (513, 384, 3, 2, 640, "relu", "skew"),
    (700, 256, 2, 1, 512, "swiglu", "one"),
    (260, 2304, 2, 2, 2176, "swiglu", "skew"),
    # ReLU and the down projection on few tiles (64 x 128), with a K split and
    # several tiles a segment; then too many of those: 64 rows, 96, 96 although
    # there are many, 128 and 256 (up or down); 256 rows with a K split
    (40, 2304, 3, 2, 384, "relu", "even"),
    (400, 256, 3, 2, 1152, "relu", "skew"),
    (1400, 128, 20, 1, 2560, "relu", "even"),
    (1400, 2560, 20, 1, 128, "relu", "even"),
    (2100, 128, 30, 1, 2560, "relu", "skew"),
    (2100, 2560, 30, 1, 128, "swiglu", "even"),
    (600, 128, 3, 1, 5632, "relu", "even"),
    (600, 5632, 3, 1, 128, "relu", "skew"),
    (1280, 128, 1, 1, 2560, "swiglu", "even"),
    (1280, 5120, 1, 1, 128, "relu", "even"),
    (1500, 128, 3, 1, 5632, "relu", "even"),
    (1500, 5632, 3, 1, 128, "relu", "skew"),
    (1500, 128, 3, 1, 2560, "swiglu", "skew"),
    (2100, 2048, 1, 1, 2048, "relu", "even"),
    (2200, 2048, 1, 1, 4096, "swiglu", "even"),
]


class Case:
    def __init__(self, T, d, E, k, F, act, how, f32, seed=0):
        g = gen(seed + T * 1000 + d + F)
        self.T, self.d, self.E, self.k, self.F, self.act = T, d, E, k, F, act
        n1 = 2 * F if act == "swiglu" else F
        self.p = moe.problem(T, d, E, k, F, act=act)
        self.src, self.off = segments(g, T, E, k, how)
        self.W1, self.s1, self.w1 = weights(g, E, n1, d, f32)
        self.W2, self.s2, self.w2 = weights(g, E, d, F, f32)
        x = g.standard_normal((T, d)) * np.exp(g.standard_normal((T, 1)))
        self.xq, xe = ref.quantise(x)
        self.xs = (xe + 127).astype(np.uint8)
        self.x = ref.widen_rows(self.xq, xe)
        h = np.maximum(g.standard_normal((T * k, F)), -0.5)
        self.hq, he = ref.quantise(h)
        self.hs = (he + 127).astype(np.uint8)
        self.h = ref.widen_rows(self.hq, he)

    def up(self, gather=True, ws=None, rows=None, stream=None):
        rows = rows or self.T * self.k
        hq = torch.full((rows, self.F), 0x5A, dtype=torch.uint8, device="cuda")
        hs = torch.full((rows, self.F // BLK), 77, dtype=torch.uint8, device="cuda")
        a, s = (self.xq, self.xs) if gather else (self.xq[self.src], self.xs[self.src])
        moe.moe_expert_up_fp8_block(self.p, dev(a), dev(s), dev(self.src) if gather else None, dev(self.off),
                                    dev(self.W1), dev(self.s1), hq, hs, ws=ws, stream=stream)
        torch.cuda.synchronize()
        return hq.cpu().numpy(), hs.cpu().numpy()

    def down(self, ws=None):
        y = torch.full((self.T * self.k, self.d), 3.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_down_fp8_block(self.p, dev(self.hq), dev(self.hs), dev(self.off), dev(self.W2), dev(self.s2), y,
                                      ws=ws)
        torch.cuda.synchronize()
        return y.double().cpu().numpy()

    def workspace(self, fill):
        ws = torch.empty(moe.moe_fp8_block_workspace_size(self.p), dtype=torch.uint8, device="cuda")
        return ws.fill_(fill)

    def check_up(self, hq, hs):
        for e in range(self.E):
            r = slice(self.off[e], self.off[e + 1])
            if r.start == r.stop:
                continue
            h, dh = ref.hidden(self.x[self.src[r]], self.w1[e], self.act, self.F)
            ref.check_quantised(hq[r], hs[r].astype(np.int64) - 127, h, dh, f"expert {e}")

    def check_down(self, y):
        for e in range(self.E):
            r = slice(self.off[e], self.off[e + 1])
            if r.start == r.stop:
                continue
            v, dv = ref.product(self.h[r], self.w2[e])
            over = np.abs(y[r] - v) - (dv + ref.U8 * (np.abs(v) + dv))
            assert np.all(over <= 0), f"expert {e}: {over.max():.3e} beyond the bound"
            # bf16 rounds evenly within half a step of at most U8 |v|: U8 / sqrt(3)
            # = 0.577 U8 in the root mean square; the sums add about 2^-13.8
            assert np.linalg.norm(y[r] - v) <= 0.6 * ref.U8 * np.linalg.norm(v), f"expert {e}: in the norm"


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_up(shape, f32):
    print(f"[block up] {shape} f32={f32}", flush=True)
    c = Case(*shape, f32)
    for gather in (True, False):
        c.check_up(*c.up(gather))
    a, b = c.up(ws=c.workspace(0)), c.up(ws=c.workspace(0xFF))
    c.check_up(*a)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_down(shape, f32):
    print(f"[block down] {shape} f32={f32}", flush=True)
    c = Case(*shape, f32)
    c.check_down(c.down())
    a, b = c.down(c.workspace(0)), c.down(c.workspace(0xFF))
    c.check_down(a)
    assert np.array_equal(a, b)


@pytest.mark.parametrize("d", [22016, 32768])
def test_down_with_fp32_scales_on_many_columns(d):
    """fp32 scales from K 2048 on with more than two 64 x 128 tiles a CU: 64 rows
    and 96."""
    T, F = 130, 2048
    g = gen(d)
    hq, he = ref.quantise(g.standard_normal((T, F)))
    w = g.integers(0, 0x60, (1, d, F)).astype(np.uint8) | g.integers(0, 2, (1, d, F)).astype(np.uint8) << 7
    s = (0.01 * (0.5 + g.random((1, d // BLK, F // BLK)))).astype(np.float32)
    y = torch.full((T, d), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_down_fp8_block(moe.problem(T, d, 1, 1, F), dev(hq), dev((he + 127).astype(np.uint8)),
                                  dev(np.array([0, T], np.int32)), dev(w), dev(s), y)
    torch.cuda.synchronize()
    v, dv = ref.product(ref.widen_rows(hq, he), ref.widen_matrix(w[0], s[0]))
    y = y.double().cpu().numpy()
    assert np.all(np.abs(y - v) <= dv + ref.U8 * (np.abs(v) + dv))
    assert np.linalg.norm(y - v) <= 0.6 * ref.U8 * np.linalg.norm(v)


def test_rows_behind_the_last_segment_stay():
    c = Case(200, 256, 4, 2, 384, "swiglu", "even", False)
    c.off = np.minimum(c.off, 333).astype(np.int32)  # the capacity clip leaves fewer than T*k rows
    P = int(c.off[-1])
    hq, hs = c.up()
    c.check_up(hq, hs)
    assert np.all(hq[P:] == 0x5A) and np.all(hs[P:] == 77)
    y = c.down()
    c.check_down(y)
    assert np.all(y[P:] == 3.0)


def test_no_rows_at_all():
    c = Case(40, 256, 4, 1, 256, "relu", "even", False)
    c.off = np.zeros(5, np.int32)
    hq, hs = c.up(ws=c.workspace(0xFF))
    assert np.all(hq == 0x5A) and np.all(hs == 77)
    assert np.all(c.down(c.workspace(0xFF)) == 3.0)


def test_scales_at_the_ends_of_their_range():
    """E8M0 bytes near both ends whose products stay in range, and zero blocks."""
    c = Case(9, 384, 2, 1, 128, "relu", "even", False)
    c.xs[:, 0], c.xs[:, 1] = 20, 230
    c.x = ref.widen_rows(c.xq, c.xs.astype(np.int64) - 127)
    c.s1[:, :, 0], c.s1[:, :, 1] = 234, 24
    c.xq[:, 2 * BLK:] = 0
    c.x[:, 2 * BLK:] = 0
    for e in range(2):
        c.w1[e] = ref.widen_matrix(c.W1[e], np.exp2(c.s1[e].astype(np.float64) - 127))
    c.check_up(*c.up())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_and_infinity_to_quantise(dtype, block_rows):
    """A NaN becomes a NaN code and leaves its block as a zero would; an infinity
    becomes a NaN code."""
    rows, K = 140, 384
    v = gen(5).standard_normal((rows, K)).astype(np.float32)
    v[[2, 131], [7, 130]] = 0
    bad = v.copy()
    bad[2, 7], bad[131, 130] = np.nan, -np.nan
    bad[9, 256:] = np.nan
    v[9, 256:] = 0
    out = []
    for values in (v, bad, np.where(np.isnan(bad), np.inf, bad)):
        src = bf16(values)[0] if dtype == "bf16" else dev(values)
        codes = torch.full((rows, K), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(-(-rows // block_rows), K // BLK, dtype=torch.uint8, device="cuda")
        moe.moe_quantize_fp8_block(src, codes, scales, block_rows=block_rows)
        torch.cuda.synchronize()
        out.append((codes.cpu().numpy(), scales.cpu().numpy()))
    at = np.isnan(bad)
    (c0, s0), (c1, s1), (c2, _) = out
    assert np.array_equal(s1, s0) and np.array_equal(c1[~at], c0[~at])
    assert np.all((c1[at] & 0x7F) == 0x7F) and np.all((c2[at] & 0x7F) == 0x7F)


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("shape", [(40, 256, 3, 2, 384, "relu", "even"), (40, 256, 3, 2, 384, "swiglu", "even"),
                                   (600, 256, 2, 1, 384, "relu", "even"), (33, 2176, 5, 2, 384, "relu", "skew")],
                         ids=lambda s: "-".join(map(str, s)))
def test_nan_codes_reach_their_rows_and_no_other(shape, f32):
    c = Case(*shape, f32)
    clean_h, clean_y = c.up(ws=c.workspace(0)), c.down(c.workspace(0))
    tok = int(c.src[c.off[-1] // 2])
    rows = np.zeros(c.T * c.k, bool)
    rows[: c.off[-1]] = c.src[: c.off[-1]] == tok
    c.xq[tok, 5] = 0x7F
    c.hq[rows, 140] = 0xFF
    (hq, hs), y = c.up(ws=c.workspace(0)), c.down(c.workspace(0))
    assert np.all((hq[rows] & 0x7F) == 0x7F) and np.all(np.isnan(y[rows]))
    assert np.array_equal(hq[~rows], clean_h[0][~rows]) and np.array_equal(hs[~rows], clean_h[1][~rows])
    assert np.array_equal(y[~rows], clean_y[~rows])


def test_strided_tensor_is_refused():
    c = Case(4, 256, 2, 1, 256, "relu", "even", False)
    x = dev(c.xq).repeat(1, 2)[:, :256]
    with pytest.raises(ValueError):
        moe.moe_expert_up_fp8_block(c.p, x, dev(c.xs), dev(c.src), dev(c.off), dev(c.W1), dev(c.s1), dev(c.hq),
                                    dev(c.hs))


# ---------------------------------------------------------------- the layer
LAYERS = [  # T, d, E, k, F, act, normalize, cf
    (1, 256, 4, 2, 128, "swiglu", False, 0.0),
    (37, 384, 6, 2, 384, "relu", True, 0.0),
    (300, 256, 4, 2, 384, "swiglu", True, 1.0),
    (512, 512, 2, 1, 256, "swiglu", False, 0.7),
    (90, 2048, 3, 3, 2176, "swiglu", False, 0.0),
]


class Layer:
    def __init__(self, T, d, E, k, F, act, normalize, cf, f32=False, seed=5):
        g = gen(seed + T)
        self.T, self.d, self.E, self.k, self.F, self.act = T, d, E, k, F, act
        self.p = moe.problem(T, d, E, k, F, act=act, normalize=normalize, cf=cf)
        n1 = 2 * F if act == "swiglu" else F
        W1, s1, self.w1 = weights(g, E, n1, d, f32)
        W2, s2, self.w2 = weights(g, E, d, F, f32)
        self.W1, self.s1, self.W2, self.s2 = dev(W1), dev(s1), dev(W2), dev(s2)
        self.x, self.xw = bf16(g.standard_normal((T, d)))
        self.x2, _ = bf16(g.standard_normal((T, d)))
        self.Wg, _ = bf16(g.standard_normal((E, d)) / np.sqrt(d))
        self.bg = dev((g.standard_normal(E) * 0.3).astype(np.float32))
        self.ws = torch.empty(moe.moe_fp8_block_workspace_size(self.p), dtype=torch.uint8, device="cuda")
        self.info = {"topk_idx": torch.empty(T, k, dtype=torch.int32, device="cuda"),
                     "topk_w": torch.empty(T, k, dtype=torch.float32, device="cuda"),
                     "counts": torch.empty(E, dtype=torch.int32, device="cuda"),
                     "offsets": torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                     "slot": torch.empty(T, k, dtype=torch.int32, device="cuda"),
                     "src_token": torch.empty(T * k, dtype=torch.int32, device="cuda")}
        self.logits = torch.empty(T, E, dtype=torch.float32, device="cuda")
        self.y = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, stream=None, info=True):
        moe.moe_forward_fp8_block(self.p, self.x, self.Wg, self.bg, self.W1, self.s1, self.W2, self.s2, self.y,
                                  logits=self.logits, info=self.info if info else None, ws=self.ws, stream=stream)

    def bits(self):
        torch.cuda.synchronize()
        return self.y.view(torch.int16).cpu().numpy().copy()


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "-".join(map(str, s)))
def test_layer(shape, f32):
    print(f"[block layer] {shape} f32={f32}", flush=True)
    L = Layer(*shape, f32=f32)
    L.ws.fill_(0xFF)
    L.run()
    got = L.bits()
    T, d, E, k, F, act = shape[:6]
    i = {n: t.cpu().numpy() for n, t in L.info.items()}
    # the steps, one by one, on buffers of their own
    xq = torch.empty(T, d, dtype=torch.uint8, device="cuda")
    xs = torch.empty(T, d // BLK, dtype=torch.uint8, device="cuda")
    hq = torch.empty(T * k, F, dtype=torch.uint8, device="cuda")
    hs = torch.empty(T * k, F // BLK, dtype=torch.uint8, device="cuda")
    yp = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(L.y)
    moe.moe_quantize_fp8_block(L.x, xq, xs)
    moe.moe_expert_up_fp8_block(L.p, xq, xs, L.info["src_token"], L.info["offsets"], L.W1, L.s1, hq, hs, ws=L.ws)
    moe.moe_expert_down_fp8_block(L.p, hq, hs, L.info["offsets"], L.W2, L.s2, yp, ws=L.ws)
    moe.moe_combine(L.p, yp, L.info["slot"], L.info["topk_w"], y)
    torch.cuda.synchronize()
    # the same but for the steps' bf16 rows: a half step of each of them
    rows, w = yp.double().cpu().numpy(), i["topk_w"].astype(np.float64)
    size = sum(np.where(i["slot"][:, j:j + 1] >= 0, w[:, j:j + 1] * np.abs(rows[i["slot"][:, j]]), 0) for j in range(k))
    off = np.abs(y.double().cpu().numpy() - L.y.double().cpu().numpy())
    assert np.all(off <= 1.01 * ref.U8 * size + 2.02 * ref.U8 * np.abs(L.y.double().cpu().numpy()) + 1e-30)
    L.run(info=False)
    assert np.array_equal(got, L.bits())
    # 64 bits, from the routing of the call (tested on its own)
    q, e = ref.quantise(L.xw)
    x = ref.widen_rows(q, e)
    want, bound = np.zeros((T, d)), np.zeros((T, d))
    for ex in range(E):
        rows = np.arange(i["offsets"][ex], i["offsets"][ex + 1])
        if len(rows) == 0:
            continue
        tok = i["src_token"][rows]
        h, away = ref.code_slack(*ref.hidden(x[tok], L.w1[ex], act, F))
        v, dv = ref.product(h, L.w2[ex])
        dv = dv * 1.25 + away @ np.abs(L.w2[ex]).T  # 1.25: |h| moved by at most a step of 2^-3
        t, j = np.nonzero(np.isin(i["slot"], rows) & (i["topk_idx"] == ex))
        at = i["slot"][t, j] - rows[0]
        w = i["topk_w"][t, j].astype(np.float64)[:, None]
        np.add.at(want, t, w * v[at])
        np.add.at(bound, t, np.abs(w) * (dv[at] + 8 * ref.U24 * np.abs(v[at])))
    bound = bound + ref.U8 * (np.abs(want) + bound)
    over = np.abs(L.y.double().cpu().numpy() - want) - bound
    assert np.all(over <= 0), f"{over.max():.3e} beyond the bound"
    dropped = np.all(i["slot"] < 0, axis=1)
    assert np.all(got[dropped] == 0)


def test_layer_given_logits_and_no_tokens():
    L = Layer(50, 256, 4, 2, 256, "relu", False, 0.0)
    L.run()
    a = L.bits()
    L.y.fill_(7.0)
    moe.moe_forward_fp8_block(L.p, L.x, None, None, L.W1, L.s1, L.W2, L.s2, L.y, logits=L.logits, ws=L.ws)
    assert np.array_equal(a, L.bits())
    p0 = moe.problem(0, 256, 4, 2, 256)
    moe.moe_forward_fp8_block(p0, None, None, None, None, L.s1, None, L.s2, None)


def test_graphs_that_share_a_workspace():
    """Two captured layers on one workspace, replayed in turn with eager calls
    and new inputs between: every replay equals an eager call bit for bit."""
    A = Layer(70, 256, 4, 2, 384, "swiglu", True, 1.0)
    B = Layer(70, 256, 4, 2, 384, "swiglu", True, 1.0, f32=True, seed=9)
    B.ws = A.ws
    graphs = []
    for L in (A, B):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.run(s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            L.run(s)
        graphs.append(g)
    torch.cuda.synchronize()
    for rep in range(3):
        want = []
        for L in (A, B):
            L.run()
            want.append(L.bits())
            L.y.fill_(float("nan"))
        A.ws.fill_(0xFF)
        for L, g, w in zip((A, B), graphs, want):
            g.replay()
            assert np.array_equal(L.bits(), w), f"replay {rep}"
        for L in (A, B):
            L.x, L.x2 = L.x, L.x2.clone()
            keep = L.x.clone()
            L.x.copy_(L.x2)
            L.x2.copy_(keep)


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with a workspace of its own."""
    layers = [Layer(120, 384, 4, 2, 640, "swiglu", False, 0.0, seed=s) for s in (1, 2)]
    want = []
    for L in layers:
        L.run()
        want.append(L.bits())
        L.y.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for L, s in zip(layers, streams):
            L.run(s)
    for L, w in zip(layers, want):
        assert np.array_equal(L.bits(), w)


def test_training_step_then_serving():
    """As a user chains them: fp32 weights are quantised by blocks, the layer
    runs on them, and the balance loss of the batch's sequences gives the
    gradient of its logits."""
    g = gen(77)
    T, d, E, k, F = 96, 256, 4, 2, 384
    p = moe.problem(T, d, E, k, F, act="swiglu")
    L = Layer(T, d, E, k, F, "swiglu", False, 0.0)
    w1 = (g.standard_normal((E, 2 * F, d)) * 0.05).astype(np.float32)
    w2 = (g.standard_normal((E, d, F)) * 0.05).astype(np.float32)
    for name, w in (("1", w1), ("2", w2)):
        rows, K = w.shape[0] * w.shape[1], w.shape[2]
        codes = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
        scales = torch.empty(E, w.shape[1] // BLK, K // BLK, dtype=torch.uint8, device="cuda")
        moe.moe_quantize_fp8_block(dev(w.reshape(rows, K)), codes.view(rows, K), scales.view(rows // BLK, -1),
                                   block_rows=128)
        setattr(L, "W" + name, codes)
        setattr(L, "s" + name, scales)
    L.run()
    y = L.y.double().cpu().numpy()
    off = np.array([0, 31, 31, 80], np.int32)
    counts = torch.empty(3, E, dtype=torch.int32, device="cuda")
    losses = torch.empty(2, device="cuda")
    dz = torch.full((T, E), 9.0, device="cuda")
    ws = torch.empty(moe.moe_balance_workspace_size(p, 3), dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(p, L.logits, L.info["topk_idx"], dev(off), counts, losses, dz, 0.01, 0.001, ws)
    torch.cuda.synchronize()
    c, l, want, bound = ref.balance(L.logits.cpu().numpy(), L.info["topk_idx"].cpu().numpy(), off, 0.01, 0.001)
    assert np.array_equal(counts.cpu().numpy(), c)
    got = dz.cpu().numpy()
    assert np.all(got[80:] == 9.0) and np.all(np.abs(got[:80] - want[:80]) <= bound[:80])
    # the layer's output is near the one of the unquantised weights: codes are
    # off by at most 2^-4 relative (or 2^-10 of a block's scale), so the rows
    # agree to a few per cent
    i = {n: t.cpu().numpy() for n, t in L.info.items()}
    full = np.zeros((T, d))
    for e in range(E):
        rows = np.arange(i["offsets"][e], i["offsets"][e + 1])
        h, _ = ref.hidden(L.xw[i["src_token"][rows]], w1[e].astype(np.float64), "swiglu", F)
        v = h @ w2[e].astype(np.float64).T
        t, j = np.nonzero(i["topk_idx"] == e)
        np.add.at(full, t, i["topk_w"][t, j][:, None] * v[i["slot"][t, j] - rows[0]])
    assert np.linalg.norm(y - full) <= 4 * ref.U4 * np.linalg.norm(full)
