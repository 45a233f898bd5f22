"""MXFP4 experts through the C ABI against 64-bit references (tests/_mx_ref.py):
quantiser and its inverse bit for bit, the expert layers within bounds derived from
the number of fp32 roundings and half a step of the stored type, the layer against
its own steps and against the 64-bit layer, graph replays, other streams, and rows
that have to stay as they were."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_logit_amd as moe
import _mx_ref as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BLK = 32


def gen(seed):
    return np.random.Generator(np.random.PCG64(seed))


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    """float array -> (bf16 CUDA tensor, its values in float64)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def quantised(v):
    """Codes and scale bytes of v, and the values they stand for."""
    q, e = ref.quantise(v)
    return q, (e + 127).astype(np.uint8), ref.widen(q, e)


def weights(g, E, n, K):
    return quantised(g.standard_normal((E, n, K)) * 0.05 * np.exp(g.standard_normal((E, n, K // BLK)) * 0.7).repeat(BLK, 2))


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
    """Rows with blocks of zeros, of one value on a scale's border and just past it,
    of ties between codes, tiny and subnormal values, signed zeros, large values."""
    v = rng.standard_normal((rows, K)).astype(np.float32)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    for b in range(K // BLK):
        s = slice(b * BLK, (b + 1) * BLK)
        for r in range(rows):
            kind = (r * 7 + b) % 9
            if kind == 0:
                v[r, s] = 0.0
            elif kind == 1:
                v[r, s.start] = 6.0 * 2.0 ** (r % 5)
            elif kind == 2:
                v[r, s.start] = np.nextafter(np.float32(6), np.float32(1e9)) if dtype == "f32" else 6.03125
            elif kind == 3:
                v[r, s] *= np.float32(2.0 ** -126)
            elif kind == 4:
                v[r, s] = np.float32(2.0 ** -133) * np.where(np.arange(BLK) % 3 == 0, -1, 1)
            elif kind == 5:
                v[r, s] = -0.0
                v[r, s.start + 5] = 1.0625
            elif kind == 6:
                v[r, s] = np.tile(ties, 4) * np.where(np.arange(BLK) % 2 == 0, -1, 1) * np.float32(2.0 ** (r % 7 - 3))
            elif kind == 7:
                v[r, s] *= np.float32(2.0 ** 100)
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (7, 96), (33, 4096), (1000, 160), (3, 65536), (129, 1408)])
def test_quantise_bit_exact_and_back(dtype, rows, K):
    print(f"[mxfp4 quantise] {dtype} rows={rows} K={K}", flush=True)
    v = edge_rows(K, rows, gen(rows + K), dtype)
    src, wide = bf16(v) if dtype == "bf16" else (dev(v), v.astype(np.float64))
    codes = torch.full((rows * K // 2 + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * K // BLK + 3,), 77, dtype=torch.uint8, device="cuda")  # at an odd address
    moe.moe_quantize_mxfp4(src, codes, scales[1:])
    back = {}
    for t in (torch.float32, torch.bfloat16):
        back[t] = torch.full((rows, K), 5.0, dtype=t, device="cuda")
        moe.moe_dequantize_mxfp4(codes, scales[1:], back[t])
    torch.cuda.synchronize()
    q, e = ref.quantise(wide)
    s = scales.cpu().numpy()
    assert np.array_equal(s[1:-2].reshape(rows, -1), (e + 127).astype(np.uint8)) and s[0] == s[-1] == s[-2] == 77
    c = codes.cpu().numpy()
    assert np.array_equal(c[:-16].reshape(rows, -1), q) and np.all(c[-16:] == 0xA5)
    for t, b in back.items():
        assert np.array_equal(b.double().cpu().numpy(), ref.widen(q, e)), t


def test_every_code_and_scale_back():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :256]
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    for t in (torch.float32, torch.bfloat16):
        out = torch.empty(256, 512, dtype=t, device="cuda")
        moe.moe_dequantize_mxfp4(dev(codes), dev(scales), out)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        want = ref.widen(codes, scales.astype(np.float64) - 127)
        want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)  # 4 and 6 times 2^127, 4 and 6 times 2^126
        assert np.all(np.isnan(got[255]))
        assert np.array_equal(got[:255], want[:255])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [np.nan, -np.nan, np.inf, -np.inf])
def test_nan_and_infinity_to_quantise(dtype, bad):
    """They make their own block NaN and change no other."""
    rows, K = 50, 320
    v = gen(5).standard_normal((rows, K)).astype(np.float32)
    hit = np.zeros((rows, K // BLK), bool)
    w = v.copy()
    for r, c in ((0, 0), (17, 31), (17, 32), (49, 319)):
        w[r, c] = bad
        hit[r, c // BLK] = True
    outs = []
    for a in (v, w):
        src = bf16(a)[0] if dtype == "bf16" else dev(a)
        codes = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(rows, K // BLK, dtype=torch.uint8, device="cuda")
        back = torch.empty(rows, K, device="cuda")
        moe.moe_quantize_mxfp4(src, codes, scales)
        moe.moe_dequantize_mxfp4(codes, scales, back)
        torch.cuda.synchronize()
        outs.append((scales.cpu().numpy(), back.cpu().numpy().reshape(rows, -1, BLK)))
    assert np.all(outs[1][0][hit] == 255) and np.all(np.isnan(outs[1][1][hit]))
    assert np.array_equal(outs[0][0][~hit], outs[1][0][~hit]) and np.array_equal(outs[0][1][~hit], outs[1][1][~hit])


def test_no_rows_to_quantise():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    u = torch.empty(0, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(e, u, u)
    moe.moe_dequantize_mxfp4(u, u, e)


# ---------------------------------------------------------------- the expert layers
# (T, d, E, k, F, act, how): one token; few rows; empty experts; widths that end inside a
# tile and inside a slice of K (odd multiples of 128); segments that end inside a tile and
# on its border; K long enough to be split; many rows per expert; many tiles
SHAPES = [
    (1, 128, 1, 1, 128, "relu", "even"),
    (1, 256, 8, 2, 384, "swiglu", "even"),
    (5, 384, 3, 3, 128, "swiglu", "even"),
    (17, 640, 7, 2, 640, "relu", "skew"),
    (64, 256, 4, 1, 256, "swiglu", "one"),
    (33, 2176, 5, 2, 384, "swiglu", "skew"),
    (33, 4224, 2, 2, 384, "relu", "even"),
    (100, 384, 6, 2, 2304, "relu", "even"),
    (300, 512, 2, 2, 384, "swiglu", "even"),
    (513, 384, 3, 2, 640, "relu", "skew"),
    (700, 256, 2, 1, 512, "swiglu", "one"),
    (260, 2304, 2, 2, 2176, "swiglu", "skew"),
    (40, 4352, 3, 2, 384, "relu", "even"),
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
    # both tile shapes with each epilogue, whole and with the last round split along K,
    # most of them with half a slice at the end; as many experts as there may be
    (40, 5760, 1, 1, 128, "swiglu", "even"),
    (60, 5760, 3, 1, 384, "relu", "skew"),
    (700, 1152, 5, 1, 4224, "swiglu", "even"),
    (150, 8320, 1, 1, 2560, "swiglu", "even"),
    (150, 12416, 1, 1, 4224, "relu", "even"),
    (3300, 1152, 1, 1, 2560, "relu", "even"),
    (700, 128, 1024, 1, 128, "swiglu", "even"),
    (3, 256, 1024, 8, 128, "relu", "even"),
]


class Case:
    def __init__(self, T, d, E, k, F, act, how, seed=0):
        g = gen(seed + T * 1000 + d + F)
        self.T, self.d, self.E, self.k, self.F, self.act = T, d, E, k, F, act
        n1 = 2 * F if act == "swiglu" else F
        self.p = moe.problem(T, d, E, k, F, act=act)
        self.src, self.off = segments(g, T, E, k, how)
        self.W1, self.s1, self.w1 = weights(g, E, n1, d)
        self.W2, self.s2, self.w2 = weights(g, E, d, F)
        self.xq, self.xs, self.x = quantised(g.standard_normal((T, d)) * np.exp(g.standard_normal((T, 1))))
        self.hq, self.hs, self.h = quantised(np.maximum(g.standard_normal((T * k, F)), -0.5))

    def up(self, gather=True, ws=None, stream=None):
        rows = self.T * self.k
        hq = torch.full((rows, self.F // 2), 0x5A, dtype=torch.uint8, device="cuda")
        hs = torch.full((rows, self.F // BLK), 77, dtype=torch.uint8, device="cuda")
        a, s = (self.xq, self.xs) if gather else (self.xq[self.src], self.xs[self.src])
        moe.moe_expert_up_mxfp4(self.p, dev(a), dev(s), dev(self.src) if gather else None, dev(self.off),
                                dev(self.W1), dev(self.s1), hq, hs, ws=ws, stream=stream)
        torch.cuda.synchronize()
        return hq.cpu().numpy(), hs.cpu().numpy()

    def down(self, ws=None):
        y = torch.full((self.T * self.k, self.d), 3.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_down_mxfp4(self.p, dev(self.hq), dev(self.hs), dev(self.off), dev(self.W2), dev(self.s2), y, ws=ws)
        torch.cuda.synchronize()
        return y.double().cpu().numpy()

    def workspace(self, fill):
        ws = torch.empty(moe.moe_mxfp4_workspace_size(self.p), dtype=torch.uint8, device="cuda")
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
            # bf16 rounds evenly within half a step of at most U8 |v|, so the error's square
            # is U8^2 / 3 sum v^2 in the mean, with a deviation of at most U8^2 sqrt(4/45 sum
            # v^4) (a uniform number's square: mean 1/3, variance 4/45); five of them, and
            # 2^-13 of the norm for the sums
            mean, dev = np.sum(v ** 2) / 3, np.sqrt(4 / 45 * np.sum(v ** 4))
            size = ref.U8 * np.sqrt(mean + 5 * dev) + 2.0 ** -13 * np.linalg.norm(v)
            assert np.linalg.norm(y[r] - v) <= size, f"expert {e}: in the norm"


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_up(shape):
    print(f"[mxfp4 up] {shape}", flush=True)
    c = Case(*shape)
    for gather in (True, False):
        c.check_up(*c.up(gather))
    a, b = c.up(ws=c.workspace(0)), c.up(ws=c.workspace(0xFF))
    c.check_up(*a)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_down(shape):
    print(f"[mxfp4 down] {shape}", flush=True)
    c = Case(*shape)
    c.check_down(c.down())
    a, b = c.down(c.workspace(0)), c.down(c.workspace(0xFF))
    c.check_down(a)
    assert np.array_equal(a, b)


def test_rows_behind_the_last_segment_stay():
    c = Case(200, 256, 4, 2, 384, "swiglu", "even")
    c.off = np.minimum(c.off, 333).astype(np.int32)  # the capacity clip leaves fewer than T*k rows
    P = int(c.off[-1])
    hq, hs = c.up()
    c.check_up(hq, hs)
    assert np.all(hq[P:] == 0x5A) and np.all(hs[P:] == 77)
    y = c.down()
    c.check_down(y)
    assert np.all(y[P:] == 3.0)


def test_no_rows_at_all():
    c = Case(40, 256, 4, 1, 256, "relu", "even")
    c.off = np.zeros(5, np.int32)
    hq, hs = c.up(ws=c.workspace(0xFF))
    assert np.all(hq == 0x5A) and np.all(hs == 77)
    assert np.all(c.down(c.workspace(0xFF)) == 3.0)


def test_offsets_and_tokens_out_of_range_stay_in_bounds():
    """Unspecified results of the rows concerned; nothing else is written."""
    c = Case(40, 256, 4, 1, 256, "relu", "even")
    want = c.up()
    c.off = np.array([0, 1 << 30, -5, 60, 40], np.int32)
    c.src = c.src.copy()
    c.src[::7] = 1 << 29
    c.src[3] = -1
    c.up(ws=c.workspace(0))
    c.down(c.workspace(0))
    c = Case(40, 256, 4, 1, 256, "relu", "even")
    assert np.array_equal(c.up()[0], want[0])


def test_scales_at_the_ends_of_their_range():
    """E8M0 bytes near both ends whose products stay in range, and zero blocks."""
    c = Case(9, 384, 2, 1, 128, "relu", "even")
    c.xs[:, 0], c.xs[:, 1], c.xs[:, 5] = 20, 230, 254
    c.s1[:, :, 0], c.s1[:, :, 1], c.s1[:, :, 5] = 234, 24, 0
    c.xq[:, 6 * 16:] = 0
    c.x = ref.widen(c.xq, c.xs.astype(np.int64) - 127)
    c.w1 = ref.widen(c.W1, c.s1.astype(np.int64) - 127)
    c.check_up(*c.up())


@pytest.mark.parametrize("shape", [(40, 256, 3, 2, 384, "relu", "even"), (40, 256, 3, 2, 384, "swiglu", "even"),
                                   (600, 256, 2, 1, 384, "relu", "even"), (33, 2176, 5, 2, 384, "relu", "skew")],
                         ids=lambda s: "-".join(map(str, s)))
def test_nan_scales_reach_their_rows_and_no_other(shape):
    c = Case(*shape)
    clean_h, clean_y = c.up(ws=c.workspace(0)), c.down(c.workspace(0))
    tok = int(c.src[c.off[-1] // 2])
    rows = np.zeros(c.T * c.k, bool)
    rows[: c.off[-1]] = c.src[: c.off[-1]] == tok
    c.xs[tok, c.d // BLK - 1] = 255
    c.hs[rows, 3] = 255
    (hq, hs), y = c.up(ws=c.workspace(0)), c.down(c.workspace(0))
    assert np.all(hs[rows] == 255) and np.all(np.isnan(y[rows]))
    assert np.array_equal(hq[~rows], clean_h[0][~rows]) and np.array_equal(hs[~rows], clean_h[1][~rows])
    assert np.array_equal(y[~rows], clean_y[~rows])


def test_nan_weights_reach_their_columns_and_no_other():
    c = Case(70, 256, 2, 1, 384, "relu", "even")
    clean_h, clean_y = c.up(ws=c.workspace(0)), c.down(c.workspace(0))
    c.s1[1, 37, 2] = 255
    c.s2[0, 200, 11] = 255
    (hq, hs), y = c.up(ws=c.workspace(0)), c.down(c.workspace(0))
    lo = int(c.off[1])
    block = np.zeros((70, 384 // BLK), bool)
    block[lo:, 1] = True  # column 37's block of every row of expert 1
    assert np.all(hs[block] == 255) and np.array_equal(hs[~block], clean_h[1][~block])
    assert np.all(np.isnan(y[:lo, 200]))
    y[:lo, 200] = clean_y[:lo, 200]
    assert np.array_equal(y, clean_y)


def test_strided_tensor_is_refused():
    c = Case(4, 256, 2, 1, 256, "relu", "even")
    x = dev(c.xq).repeat(1, 2)[:, :128]
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_expert_up_mxfp4(c.p, x, dev(c.xs), dev(c.src), dev(c.off), dev(c.W1), dev(c.s1), dev(c.hq), dev(c.hs))


# ---------------------------------------------------------------- the layer
LAYERS = [  # T, d, E, k, F, act, normalize, cf
    (1, 256, 4, 2, 128, "swiglu", False, 0.0),
    (37, 384, 6, 2, 384, "relu", True, 0.0),
    (300, 256, 4, 2, 384, "swiglu", True, 1.0),
    (512, 512, 2, 1, 256, "swiglu", False, 0.7),
    (90, 2048, 3, 3, 2176, "swiglu", False, 0.0),
    (40, 256, 2, 1, 5760, "relu", False, 0.0),
    (2600, 2560, 1, 1, 1152, "relu", False, 0.0),
    (300, 2560, 1, 1, 8320, "relu", False, 0.0),
]


class Layer:
    def __init__(self, T, d, E, k, F, act, normalize, cf, seed=5):
        g = gen(seed + T)
        self.T, self.d, self.E, self.k, self.F, self.act = T, d, E, k, F, act
        self.p = moe.problem(T, d, E, k, F, act=act, normalize=normalize, cf=cf)
        n1 = 2 * F if act == "swiglu" else F
        W1, s1, self.w1 = weights(g, E, n1, d)
        W2, s2, self.w2 = weights(g, E, d, F)
        self.W1, self.s1, self.W2, self.s2 = dev(W1), dev(s1), dev(W2), dev(s2)
        self.x, self.xw = bf16(g.standard_normal((T, d)))
        self.x2, _ = bf16(g.standard_normal((T, d)))
        self.Wg, _ = bf16(g.standard_normal((E, d)) / np.sqrt(d))
        self.bg = dev((g.standard_normal(E) * 0.3).astype(np.float32))
        self.ws = torch.empty(moe.moe_mxfp4_workspace_size(self.p), dtype=torch.uint8, device="cuda")
        self.info = {"topk_idx": torch.empty(T, k, dtype=torch.int32, device="cuda"),
                     "topk_w": torch.empty(T, k, dtype=torch.float32, device="cuda"),
                     "counts": torch.empty(E, dtype=torch.int32, device="cuda"),
                     "offsets": torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                     "slot": torch.empty(T, k, dtype=torch.int32, device="cuda"),
                     "src_token": torch.empty(T * k, dtype=torch.int32, device="cuda")}
        self.logits = torch.empty(T, E, dtype=torch.float32, device="cuda")
        self.y = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, stream=None, info=True):
        moe.moe_forward_mxfp4(self.p, self.x, self.Wg, self.bg, self.W1, self.s1, self.W2, self.s2, self.y,
                              logits=self.logits, info=self.info if info else None, ws=self.ws, stream=stream)

    def bits(self):
        torch.cuda.synchronize()
        return self.y.view(torch.int16).cpu().numpy().copy()


@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "-".join(map(str, s)))
def test_layer(shape):
    print(f"[mxfp4 layer] {shape}", flush=True)
    L = Layer(*shape)
    L.ws.fill_(0xFF)
    L.run()
    got = L.bits()
    T, d, E, k, F, act = shape[:6]
    i = {n: t.cpu().numpy() for n, t in L.info.items()}
    # the steps, one by one, on buffers of their own
    xq = torch.empty(T, d // 2, dtype=torch.uint8, device="cuda")
    xs = torch.empty(T, d // BLK, dtype=torch.uint8, device="cuda")
    hq = torch.empty(T * k, F // 2, dtype=torch.uint8, device="cuda")
    hs = torch.empty(T * k, F // BLK, dtype=torch.uint8, device="cuda")
    yp = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(L.y)
    moe.moe_quantize_mxfp4(L.x, xq, xs)
    moe.moe_expert_up_mxfp4(L.p, xq, xs, L.info["src_token"], L.info["offsets"], L.W1, L.s1, hq, hs, ws=L.ws)
    moe.moe_expert_down_mxfp4(L.p, hq, hs, L.info["offsets"], L.W2, L.s2, yp, ws=L.ws)
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
    x = ref.widen(*ref.quantise(L.xw))
    want, bound = np.zeros((T, d)), np.zeros((T, d))
    for ex in range(E):
        rows = np.arange(i["offsets"][ex], i["offsets"][ex + 1])
        if len(rows) == 0:
            continue
        tok = i["src_token"][rows]
        h, away = ref.code_slack(*ref.hidden(x[tok], L.w1[ex], act, F))
        v, dv = ref.product(h, L.w2[ex])
        dv = dv * 1.5 + away @ np.abs(L.w2[ex]).T  # 1.5: |h| moved by at most a step of half its value
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
    moe.moe_forward_mxfp4(L.p, L.x, None, None, L.W1, L.s1, L.W2, L.s2, L.y, logits=L.logits, ws=L.ws)
    assert np.array_equal(a, L.bits())
    moe.moe_forward_mxfp4(moe.problem(0, 256, 4, 2, 256), None, None, None, None, None, None, None, None)


def test_graphs_that_share_a_workspace():
    """Two captured layers on one workspace, replayed in turn with eager calls and
    new inputs between: every replay equals an eager call bit for bit."""
    A = Layer(70, 256, 4, 2, 384, "swiglu", True, 1.0)
    B = Layer(70, 256, 4, 2, 384, "swiglu", True, 1.0, seed=9)
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
    """As a user chains them: the layer's backward gives the experts' gradients, their
    orthogonalised updates change the fp32 weights, those are quantised, and the layer
    runs on them."""
    g = gen(77)
    T, d, E, k, F = 160, 256, 4, 2, 384
    p = moe.problem(T, d, E, k, F, act="swiglu")
    L = Layer(T, d, E, k, F, "swiglu", False, 0.0)
    w = {"1": dev((g.standard_normal((E, 2 * F, d)) * 0.05).astype(np.float32)),
         "2": dev((g.standard_normal((E, d, F)) * 0.05).astype(np.float32))}
    b = {n: t.to(torch.bfloat16) for n, t in w.items()}
    saved = {"u": torch.empty(T * k, 2 * F, dtype=torch.bfloat16, device="cuda"),
             "h": torch.empty(T * k, F, dtype=torch.bfloat16, device="cuda"),
             "y_perm": torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")}
    ws = torch.empty(moe.moe_workspace_size(p), dtype=torch.uint8, device="cuda")
    moe.moe_forward_train(p, L.x, L.Wg, L.bg, b["1"], b["2"], L.y, L.logits, L.info, saved, ws)
    dy, _ = bf16(g.standard_normal((T, d)))
    grad = {"1": torch.empty_like(w["1"]), "2": torch.empty_like(w["2"])}
    bws = torch.empty(moe.moe_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    moe.moe_backward(p, dy, L.x, L.Wg, b["1"], b["2"], L.logits, L.info, saved, torch.empty_like(L.x),
                     torch.empty(E, d, device="cuda"), torch.empty(E, device="cuda"), grad["1"], grad["2"], bws)
    for n in "12":
        # the gate and up projections are matrices of their own
        G = grad[n].view(2 * E, F, d) if n == "1" else grad[n]
        mom = torch.zeros_like(G)
        out = torch.empty(G.shape, dtype=torch.bfloat16, device="cuda")
        ows = torch.empty(moe.moe_orthogonalize_workspace_size(*G.shape), dtype=torch.uint8, device="cuda")
        moe.moe_orthogonalize(G, out, momentum=mom, beta=0.95, nesterov=True, steps=5, ws=ows)
        torch.cuda.synchronize()
        assert torch.equal(mom, G)
        for i in range(G.shape[0]):
            want = ref.orthogonal(1.95 * G[i].double().cpu().numpy(), 5)
            o = out[i].double().cpu().numpy()
            # few tokens: the gradient's rank is at most theirs; see test_gpu_orthogonalize.py
            assert np.linalg.norm(o - want) <= (4e-3 + 0.6 * ref.U8) * np.linalg.norm(want)
        w[n] -= 0.02 * out.view(w[n].shape).float()
        codes = torch.empty(*w[n].shape[:-1], w[n].shape[-1] // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(*w[n].shape[:-1], w[n].shape[-1] // BLK, dtype=torch.uint8, device="cuda")
        moe.moe_quantize_mxfp4(w[n], codes, scales)
        setattr(L, "W" + n, codes)
        setattr(L, "s" + n, scales)
    L.run()
    y = L.y.double().cpu().numpy()
    # the layer on the updated weights without their quantisation: codes are off by at
    # most 1/4 of their value's power of two (or 1/4 of the block's scale), which over
    # many terms leaves the rows' norms within a third
    i = {n: t.cpu().numpy() for n, t in L.info.items()}
    full = np.zeros((T, d))
    for e in range(E):
        rows = np.arange(i["offsets"][e], i["offsets"][e + 1])
        h, _ = ref.hidden(L.xw[i["src_token"][rows]], w["1"][e].double().cpu().numpy(), "swiglu", F)
        v = h @ w["2"][e].double().cpu().numpy().T
        t, j = np.nonzero(i["topk_idx"] == e)
        np.add.at(full, t, i["topk_w"][t, j][:, None] * v[i["slot"][t, j] - rows[0]])
    assert np.linalg.norm(y - full) <= 0.34 * np.linalg.norm(full)


# ---------------------------------------------------------------- offsets that pass 32 bits
def big_ints(n):
    return torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(n % 1000))


@pytest.fixture
def roomy():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_quantise_more_than_2_32_values(roomy):
    """Rows behind the first 2^32 values get what they get by themselves."""
    K, rows = 4096, (1 << 20) + 77
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(rows, K // BLK, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(x, q, s)
    for at in (0, 1 << 19, rows - 100):
        tq, ts = torch.empty_like(q[:100]), torch.empty_like(s[:100])
        moe.moe_quantize_mxfp4(x[at:at + 100], tq, ts)
        assert torch.equal(tq, q[at:at + 100]) and torch.equal(ts, s[at:at + 100]), at
    moe.moe_dequantize_mxfp4(q, s, x)
    for at in (0, 1 << 19, rows - 100):
        back = torch.empty(100, K, dtype=torch.bfloat16, device="cuda")
        moe.moe_dequantize_mxfp4(q[at:at + 100], s[at:at + 100], back)
        assert torch.equal(back, x[at:at + 100]), at


def test_weights_of_more_than_4_gib(roomy):
    """Both layers' last expert lies behind the first 4 GiB of codes; 64 of each layer's
    columns, from all over, against 64-bit products."""
    T, d, F, E = 9, 16384, 8192, 65
    g = gen(65)
    off = dev(np.array([0, 4] + [4] * (E - 2) + [T], np.int32))  # the first and the last
    xq, xs, x = quantised(g.standard_normal((T, d)))
    hq, hs, h = quantised(np.maximum(g.standard_normal((T, F)), -0.5))
    src = dev(np.arange(T, dtype=np.int32))
    cols = np.sort(g.choice(F // BLK, 2, replace=False))
    hidden = np.concatenate([np.arange(c * BLK, (c + 1) * BLK) for c in cols])
    rows_of = dict(up=np.concatenate([hidden, F + hidden]), down=np.sort(g.choice(d, 64, replace=False)))
    W, sc = {}, {}
    for name, n, K in (("up", 2 * F, d), ("down", d, F)):
        W[name] = big_ints(E * n * K // 2).view(E, n, K // 2)
        sc[name] = (big_ints(E * n * K // BLK).view(E, n, K // BLK) % 5) + 118
    assert min(W["up"].numel(), W["down"].numel()) > 1 << 32

    def picked(name, e):
        at = torch.from_numpy(rows_of[name]).cuda()
        q, s = W[name][e].index_select(0, at).cpu().numpy(), sc[name][e].index_select(0, at).cpu().numpy()
        return ref.widen(q, s.astype(np.int64) - 127)

    p = moe.problem(T, d, E, 1, F, act="swiglu")
    ws = torch.empty(moe.moe_mxfp4_workspace_size(p), dtype=torch.uint8, device="cuda")
    oq = torch.zeros(T, F // 2, dtype=torch.uint8, device="cuda")
    os_ = torch.zeros(T, F // BLK, dtype=torch.uint8, device="cuda")
    y = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_up_mxfp4(p, dev(xq), dev(xs), src, off, W["up"], sc["up"], oq, os_, ws=ws)
    moe.moe_expert_down_mxfp4(p, dev(hq), dev(hs), off, W["down"], sc["down"], y, ws=ws)
    torch.cuda.synchronize()
    for e, r in ((0, slice(0, 4)), (E - 1, slice(4, T))):
        v, dv = ref.hidden(x[r], picked("up", e), "swiglu", 2 * BLK)
        codes = oq[r].cpu().numpy().reshape(-1, F // BLK, BLK // 2)[:, cols].reshape(-1, BLK)
        ref.check_quantised(codes, os_[r].cpu().numpy()[:, cols].astype(np.int64) - 127, v, dv, f"up, expert {e}")
        v, dv = ref.product(h[r], picked("down", e))
        over = np.abs(y[r].double().cpu().numpy()[:, rows_of["down"]] - v) - (dv + ref.U8 * (np.abs(v) + dv))
        assert np.all(over <= 0), f"down, expert {e}"


# ---------------------------------------------------------------- malformed segments write nothing else
class Guarded:
    """A tensor in the middle of a larger one of a known pattern."""
    EDGE = 1 << 16

    def __init__(self, *shape, dtype=torch.uint8):
        n = int(np.prod(shape))
        size = torch.empty(0, dtype=dtype).element_size()
        self.all = torch.full((n * size + 2 * self.EDGE,), 0x5A, dtype=torch.uint8, device="cuda")
        self.mid = self.all[self.EDGE:self.EDGE + n * size]
        self.t = self.mid.view(dtype).view(*shape)

    def edges_stay(self):
        return bool(torch.all(self.all[:self.EDGE] == 0x5A)) and bool(torch.all(self.all[self.EDGE + self.mid.numel():] == 0x5A))

    def rows(self):
        """Rows as bytes."""
        return self.mid.view(self.t.shape[0], -1).cpu().numpy()


def clamped_rows(off, rows):
    """The rows of every segment, its borders clamped into [0, rows] and its end not in front of its start."""
    held = np.zeros(rows, bool)
    for e in range(len(off) - 1):
        lo = min(max(int(off[e]), 0), rows)
        held[lo:min(max(int(off[e + 1]), lo), rows)] = True
    return held


@pytest.mark.parametrize("shape", [(40, 256, 4, 1, 256, "relu"), (40, 256, 4, 1, 384, "swiglu"), (300, 5632, 4, 2, 384, "relu"),
                                   (700, 256, 4, 1, 2304, "swiglu")], ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("off", [[0, 1 << 30, -5, 60, 40], [-7, 3, 3, 1 << 30, -(1 << 30)], [11, 5, 17, 17, 23], [-1, -1, -1, -1, -1],
                                 [1 << 30, 1 << 30, 1 << 30, 1 << 30, 1 << 30]], ids=lambda o: "_".join(map(str, o)))
@pytest.mark.parametrize("ws", [False, True])
def test_malformed_segments_write_their_clamped_rows_only(shape, off, ws):
    """Tokens and segments that no routing gives: outputs and workspace lie between guards, rows
    outside every clamped segment keep what they held, and a row of one valid segment and a
    valid token is as in a call without the others."""
    print(f"[mxfp4 malformed] {shape} {off} {ws}", flush=True)
    T, d, E, k, F, act = shape
    c = Case(T, d, E, k, F, act, "even")
    rows = T * k
    src = c.src.copy()
    src[::7], src[3], src[5] = 1 << 29, -1, T
    off = np.array(off, np.int32)
    hq, hs, y = Guarded(rows, F // 2), Guarded(rows, F // BLK), Guarded(rows, d, dtype=torch.bfloat16)
    space = Guarded(moe.moe_mxfp4_workspace_size(c.p)) if ws else None
    moe.moe_expert_up_mxfp4(c.p, dev(c.xq), dev(c.xs), dev(src), dev(off), dev(c.W1), dev(c.s1), hq.t, hs.t, ws=space and space.t)
    moe.moe_expert_down_mxfp4(c.p, dev(c.hq), dev(c.hs), dev(off), dev(c.W2), dev(c.s2), y.t, ws=space and space.t)
    torch.cuda.synchronize()
    held = clamped_rows(off, rows)
    for name, g in dict(hq=hq, hs=hs, y=y).items():
        assert g.edges_stay(), f"{name}: written outside"
        assert np.all(g.rows()[~held] == 0x5A), f"{name}: a row outside every segment"
    assert space is None or space.edges_stay(), "workspace: written outside"
    # [11, 5, 17, 17, 23]: 5 .. 16 of expert 1 and 17 .. 22 of expert 3 are segments like any
    if list(off) == [11, 5, 17, 17, 23]:
        c.off = np.array([5, 5, 17, 17, 23], np.int32)
        good = (src >= 0) & (src < T) & held
        want_q, want_s = c.up(ws=c.workspace(0) if ws else None)
        assert np.array_equal(hq.rows()[good], want_q[good]) and np.array_equal(hs.rows()[good], want_s[good])
        c.check_down(y.t.double().cpu().numpy())


def test_negative_gates():
    """silu of gates down to -87 within (1.3 |u| + 8) 2^-24 of it: the exponent's rounding grows with
    |u|.  A gate is the sum of two codes whose scales lie at most 2^6 apart and an up value one
    code, so both are exact."""
    T, d, F = 400, 128, 128
    g = gen(41)
    p = moe.problem(T, d, 1, 1, F, act="swiglu")
    codes, e = np.zeros((T, d), np.uint8), np.zeros((T, d // BLK), np.int64)
    e[:, 0] = g.integers(-4, 4, T)
    e[:, 1] = e[:, 0] - g.integers(0, 4, T)
    codes[:, 0], codes[:, 32], codes[:, 64] = g.integers(1, 8, T), g.integers(0, 8, T), 2
    W, we = np.zeros((1, 2 * F, d), np.uint8), np.zeros((1, 2 * F, d // BLK), np.int64)
    W[0, :F, 0] = W[0, :F, 32] = 10  # -1
    W[0, F:, 64] = g.integers(0, 16, F)
    u = -(ref.POS[codes[:, 0]] * np.exp2(e[:, 0]) + ref.POS[codes[:, 32]] * np.exp2(e[:, 1]))
    keep = u > -87
    assert np.count_nonzero(keep) > 300 and u[keep].min() < -60
    h = (u / (1 + np.exp(-u)))[:, None] * ref.TABLE[W[0, F:, 64]][None, :]
    hq = torch.empty(T, F // 2, dtype=torch.uint8, device="cuda")
    hs = torch.empty(T, F // BLK, dtype=torch.uint8, device="cuda")
    moe.moe_expert_up_mxfp4(p, dev(ref.pack(codes)), dev((e + 127).astype(np.uint8)), None, dev(np.array([0, T], np.int32)), dev(ref.pack(W)),
                            dev((we + 127).astype(np.uint8)), hq, hs)
    torch.cuda.synchronize()
    dh = (1.3 * np.abs(u) + 8)[:, None] * ref.U24 * np.abs(h)
    ref.check_quantised(hq.cpu().numpy()[keep], hs.cpu().numpy()[keep].astype(np.int64) - 127, h[keep], dh[keep], "negative gates")
