"""Low-rank adapters beside packed projections, the gated activation with 8-bit
checkpoints, and the packed projection's input gradient, against plain fp64
forms of their formulas.

Tolerances.  A sum of n fp32 terms in any order is within n 2^-23 of its terms'
magnitudes when every addition is off by one unit in the last place (a tensor
core may truncate); rounding a result to type t is off by eps(t) / 2."""
import numpy as np
import pytest
import torch

from w8_a8_quantized_b200 import aq

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(autouse=True)
def _no_kernel_errors():
    yield
    aq.check_all_workspaces()


def half_step(t):
    return torch.finfo(t).eps / 2


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def assert_within(got, ref, tol, what=""):
    got, err = got.double(), (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; first at {i}: got "
                             f"{got[i].item()!r}, want {ref[i].item()!r} +- {tol[i].item() if tol.dim() else tol!r}")


# ------------------------------------------------------------------ adapters

class LoraCase:
    def __init__(self, M, N, K, ranks, ids, seed=0, scales=None, pad=0):
        g = rng(seed)
        self.M, self.N, self.K, self.ranks = M, N, K, ranks
        self.scales = scales or [0.5 + 0.25 * l for l in range(len(ranks))]
        R = sum(ranks)
        self.a, self.bt = normal(g, R, K, scale=K ** -0.5), normal(g, R, N, scale=0.1)
        self.x, self.dy = normal(g, M, K + pad)[:, :K], normal(g, M, N + pad, scale=0.01)[:, :N]
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
        assert self.ids.numel() == M
        self.ad = aq.Adapters(self.a, self.bt, ranks, self.scales)
        self.off = np.concatenate([[0], np.cumsum(ranks)])

    def each(self):
        """(adapter's rows, its tokens, scale) of every adapter that a token has."""
        for l, r in enumerate(self.ranks):
            at = (self.ids == l).nonzero().reshape(-1)
            yield slice(int(self.off[l]), int(self.off[l + 1])), at, float(np.float32(self.scales[l])), r

    def forward(self):
        """S and the adapters' part in fp64, with bounds on their errors."""
        d = torch.float64
        s = torch.zeros(self.M, max(self.ranks), dtype=d, device="cuda")
        out = torch.zeros(self.M, self.N, dtype=d, device="cuda")
        ts, to = torch.zeros_like(s), torch.zeros_like(out)
        for rows, at, c, r in self.each():
            if r == 0 or at.numel() == 0:
                continue
            x, a, b = self.x[at].to(d), self.a[rows].to(d), self.bt[rows].to(d)
            s[at, :r] = c * (x @ a.t())
            ts[at, :r] = abs(c) * (self.K + 4) * U * (x.abs() @ a.t().abs())
            out[at] = s[at, :r] @ b
            to[at] = ts[at, :r] @ b.abs() + (3 * r + 8) * U * ((s[at, :r].abs() + ts[at, :r]) @ b.abs())
        return s, out, ts, to


def mixed_ids(M, L, seed, none=0.2):
    g = np.random.default_rng(seed)
    ids = g.integers(0, L, M)
    ids[g.random(M) < none] = -1
    return ids.tolist()


def segment_ids(M, L, seed):
    g = np.random.default_rng(seed)
    cuts = np.sort(g.integers(0, M + 1, L - 1))
    return np.searchsorted(cuts, np.arange(M), side="right").tolist()


LORA = [  # M, N, K, ranks, ids
    (1, 64, 128, [4], [0]),
    (1, 1024, 2560, [16, 8], [1]),
    (1, 136, 72, [1], [0]),
    (2, 128, 128, [3, 0, 7], [1, 2]),
    (5, 200, 328, [1, 64, 17], [2, 2, -1, 0, 1]),
    (64, 640, 1536, [5, 33, 64, 8, 16, 9], mixed_ids(64, 6, 1)),
    (64, 256, 384, [2 + i % 9 for i in range(64)], list(range(63, -1, -1))),
    (63, 128, 256, [8, 8], [7, -5] + mixed_ids(61, 2, 2)),
    (65, 328, 1032, [16], [0] * 65),
    (200, 512, 640, [12, 70, 1], segment_ids(200, 3, 3)),
    (130, 264, 520, [256, 130], mixed_ids(130, 2, 4)),
    (1000, 1024, 4096, [16, 64, 8, 31], segment_ids(1000, 4, 5)),
    (333, 2048, 896, [24, 40], mixed_ids(333, 2, 6, none=0.5)),
    (77, 128, 128, [9], [-1] * 77),
    # decode beyond one cluster's columns, beyond one stage of rows, and beyond the decode kernel's widest input
    (3, 17408, 264, [33, 200], [1, 0, 1]),
    (9, 520, 40960, [5, 24], mixed_ids(9, 2, 10)),
    (2, 128, 41024, [12], [0, 0]),
    # many column blocks per tile, tiles of one adapter, of several and of none
    (2000, 8192, 256, [16, 40, 33], [0] * 500 + [-1] * 700 + segment_ids(300, 3, 7) + [2] * 60 + [-1] * 10 + [1] * 430),
    (1300, 4096, 4104, [64, 3, 17, 50, 8], segment_ids(1000, 5, 8) + mixed_ids(300, 5, 9)),
]


@pytest.mark.parametrize("case", range(len(LORA)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lora_apply(case, dtype):
    c = LoraCase(*LORA[case], seed=case, pad=8 * (case % 3))
    y = normal(rng(100 + case), c.M, c.N + 8, dtype=dtype)[:, :c.N]
    s64, d64, ts, td = c.forward()
    s = torch.full((c.M, max(c.ranks)), float("nan"), device="cuda")
    out = aq.aq_lora_apply(c.ad, c.x, c.ids, y, s=s)
    assert out.dtype == dtype
    assert_within(s, s64, ts, "s")
    ref = y.double() + d64
    assert_within(out, ref, td + 2 * U * (y.double().abs() + d64.abs()) + half_step(dtype) * (ref.abs() + td), "out")
    # without an adapter: y itself
    none = [m for m in range(c.M) if not 0 <= c.ids[m].item() < len(c.ranks) or c.ranks[c.ids[m].item()] == 0]
    assert torch.equal(out[none], y[none]) and not s[none].any()
    # the same bits again, in place, and into rows of another pitch that are otherwise left alone
    assert torch.equal(aq.aq_lora_apply(c.ad, c.x, c.ids, y), out)
    wide = torch.full((c.M + 3, c.N + 16), 7.0, dtype=dtype, device="cuda")
    aq.aq_lora_apply(c.ad, c.x, c.ids, y, out=wide)
    assert torch.equal(wide[:c.M, :c.N], out) and bool((wide[c.M:] == 7).all()) and bool((wide[:, c.N:] == 7).all())
    z = y.clone(memory_format=torch.contiguous_format)
    assert aq.aq_lora_apply(c.ad, c.x, c.ids, z, out=z) is z and torch.equal(z, out)
    # the adapters' part alone
    alone = aq.aq_lora_apply(c.ad, c.x, c.ids, out_dtype=dtype)
    assert_within(alone, d64, td + half_step(dtype) * (d64.abs() + td), "alone")


def test_lora_products_keep_all_bits():
    """A_l picks single activations, so S is exact and only the second product's
    few roundings are left: a lost term of S (2^-9 of it) would show."""
    M, N, K, r = 70, 256, 512, 16
    c = LoraCase(M, N, K, [r, r], segment_ids(M, 2, 9), seed=9, scales=[1 / 3, 0.7])
    c.a.zero_()
    for l in range(2):
        c.a[l * r + torch.arange(r), 31 * torch.arange(r) + l] = 1.0
    s64 = torch.zeros(M, r, dtype=torch.float64, device="cuda")
    for l in range(2):
        at = c.ids == l
        s64[at] = (c.x[at][:, 31 * torch.arange(r) + l].float() * np.float32(c.scales[l])).double()
    d64 = torch.stack([s64[m] @ c.bt[c.ids[m] * r:(c.ids[m] + 1) * r].double() for m in range(M)])
    mag = torch.stack([s64[m].abs() @ c.bt[c.ids[m] * r:(c.ids[m] + 1) * r].double().abs() for m in range(M)])
    s = torch.empty(M, r, device="cuda")
    out = aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    assert torch.equal(s.double(), s64)
    assert_within(out, d64, (3 * r + 2) * U * mag)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_lora_foreign_infinities_stay_out(bad):
    M, N, K = 70, 128, 256
    ids = [m % 3 for m in range(M)]
    c = LoraCase(M, N, K, [8, 5, 12], ids, seed=11)
    s0 = torch.empty(M, 12, device="cuda")
    out0 = aq.aq_lora_apply(c.ad, c.x, c.ids, s=s0)
    da0, db0, dx0 = aq.aq_lora_backward(c.ad, c.dy, c.ids, s0, c.x)
    ok = c.ids != 1
    # adapter 1's weights and tokens
    c.a[8:13] = bad
    c.bt[8:13, ::2] = bad
    c.x[c.ids == 1] = bad
    c.dy[c.ids == 1, ::3] = bad
    s = torch.empty_like(s0)
    out = aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    assert torch.equal(out[ok], out0[ok]) and torch.equal(s[ok], s0[ok])
    assert not torch.isfinite(out[~ok]).all()
    da, db, dx = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x)
    keep = [i for i in range(25) if not 8 <= i < 13]
    assert torch.equal(da[keep], da0[keep]) and torch.equal(db[keep], db0[keep]) and torch.equal(dx[ok], dx0[ok])


def test_lora_odd_tables_stay_in_bounds():
    """Offsets outside the table are clamped, ids outside it have no adapter."""
    c = LoraCase(40, 64, 128, [4, 4], [i % 2 for i in range(40)], seed=12)
    want = aq.aq_lora_apply(c.ad, c.x, c.ids)
    c.ad.off.copy_(torch.tensor([0, 4, 2 ** 31 - 1], dtype=torch.int32))  # last adapter: clamped to the table's end
    assert torch.equal(aq.aq_lora_apply(c.ad, c.x, c.ids), want)
    c.ad.off.copy_(torch.tensor([-7, 4, 8], dtype=torch.int32))
    assert torch.equal(aq.aq_lora_apply(c.ad, c.x, c.ids), want)
    c.ids.copy_(torch.tensor([2 ** 31 - 1, -2 ** 31] * 20, dtype=torch.int32))
    assert not aq.aq_lora_apply(c.ad, c.x, c.ids).any()


def backward_reference(c, s, x, add):
    """Gradients and error bounds in fp64; x fp64 [M][K]."""
    d = torch.float64
    R = sum(c.ranks)
    da, db = torch.zeros(R, c.K, dtype=d, device="cuda"), torch.zeros(R, c.N, dtype=d, device="cuda")
    ta, tb = torch.zeros_like(da), torch.zeros_like(db)
    dx, tx = add.to(d).clone(), torch.zeros(c.M, c.K, dtype=d, device="cuda")
    for rows, at, sc, r in c.each():
        if r == 0 or at.numel() == 0:
            continue
        dy, b, a, xx, ss = c.dy[at].to(d), c.bt[rows].to(d), c.a[rows].to(d), x[at], s[at, :r].to(d)
        t = sc * (dy @ b.t())
        tt = abs(sc) * (c.N + 4) * U * (dy.abs() @ b.t().abs())
        n = 3 * at.numel() + 24
        da[rows], ta[rows] = t.t() @ xx, tt.t() @ xx.abs() + n * U * ((t.abs() + tt).t() @ xx.abs())
        db[rows], tb[rows] = ss.t() @ dy, n * U * (ss.t().abs() @ dy.abs())
        dx[at] += t @ a
        tx[at] = tt @ a.abs() + (3 * r + 8) * U * ((t.abs() + tt) @ a.abs())
    return (da, ta), (db, tb), (dx, tx)


@pytest.mark.parametrize("case", range(len(LORA)))
@pytest.mark.parametrize("codes", [False, True])
def test_lora_backward(case, codes):
    c = LoraCase(*LORA[case], seed=50 + case, pad=16 * (case % 2))
    if codes and c.K % 16:
        pytest.skip("codes come 16 at a time: refused (see the refusals)")
    dtype = torch.float32 if case % 2 else torch.bfloat16
    s = torch.empty(c.M, max(c.ranks), device="cuda")
    aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    x, sx, x64 = c.x, None, c.x.double()
    if codes:
        x, sx = aq.aq_quant_act(c.x.contiguous())
        x64 = x.double() * sx.double()[:, None]
    add = normal(rng(case), c.M, c.K + 16, scale=0.01, dtype=dtype)[:, :c.K]
    (da64, ta), (db64, tb), (dx64, tx) = backward_reference(c, s, x64, add)
    da, db, dx = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, x, sx=sx, add=add)
    assert da.dtype == db.dtype == torch.float32 and dx.dtype == dtype
    assert_within(da, da64, ta, "da")
    assert_within(db, db64, tb, "dbt")
    assert_within(dx, dx64, tx + 2 * U * dx64.abs() + 2 * U * add.double().abs() + half_step(dtype) * (dx64.abs() + tx),
                  "dx")
    again = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, x, sx=sx, add=add)
    assert all(torch.equal(p, q) for p, q in zip(again, (da, db, dx)))
    z = add.clone(memory_format=torch.contiguous_format)
    assert aq.aq_lora_backward(c.ad, c.dy, c.ids, s, x, sx=sx, add=z, dx=z)[2] is z and torch.equal(z, dx)
    none = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, x, sx=sx, want_dx=False)
    assert none[2] is None and torch.equal(none[0], da) and torch.equal(none[1], db)


def test_lora_gradients_against_differences():
    """The loss sum(out * dy) is linear in A and in B: its difference for a step in
    one entry is the gradient, up to fp32 rounding of the outputs."""
    M, N, K = 90, 128, 192
    c = LoraCase(M, N, K, [6, 3], segment_ids(M, 2, 21), seed=21)
    s = torch.empty(M, 6, device="cuda")
    out0 = aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    da, db, dx = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x, dx_dtype=torch.float32)
    for table, grad, r, k in ((c.a, da, 2, 77), (c.a, da, 7, 191), (c.bt, db, 0, 5), (c.bt, db, 8, 127)):
        old = table[r, k].clone()
        table[r, k] = old + 4.0
        step = (table[r, k].double() - old.double()).item()
        out1 = aq.aq_lora_apply(c.ad, c.x, c.ids)
        diff = ((out1.double() - out0.double()) * c.dy.double()).sum() / step
        # each output is off by at most K 2^-23 of its terms' size on both sides
        mag = ((out1.double().abs() + out0.double().abs()) * c.dy.double().abs()).sum() / abs(step)
        assert abs(diff - grad[r, k].double()) <= 64 * K * U * mag
        table[r, k] = old
    # the input: moving x[m][k] by a power of two
    for m, k in ((0, 3), (89, 100)):
        old = c.x[m, k].clone()
        c.x[m, k] = old + 8.0
        step = (c.x[m, k].double() - old.double()).item()
        out1 = aq.aq_lora_apply(c.ad, c.x, c.ids)
        diff = ((out1.double() - out0.double()) * c.dy.double()).sum() / step
        mag = ((out1.double().abs() + out0.double().abs()) * c.dy.double().abs()).sum() / abs(step)
        assert abs(diff - dx[m, k].double()) <= 64 * K * U * mag
        c.x[m, k] = old


@pytest.mark.parametrize("M", [13, 70, 300])
@pytest.mark.parametrize("ranks", [[8, 5], [8, 90]])
def test_lora_padded_batch(M, ranks):
    """Tokens without an adapter may hold anything: NaN in their activations, gradients
    and products leave the others' results as they are, bit for bit."""
    N, K = 264, 320
    ids = np.array(segment_ids(M, 2, M))
    ids[np.random.default_rng(M).random(M) < 0.3] = -1
    ids[-5:] = -1
    c = LoraCase(M, N, K, ranks, ids.tolist(), seed=M)
    s = torch.empty(M, max(ranks), device="cuda")
    out0 = aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    want = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x)
    pad = c.ids == -1
    c.x[pad], c.dy[pad] = float("nan"), float("nan")
    out = aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    assert torch.equal(out, out0) and not s[pad].any()
    s[pad] = float("nan")
    got = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x)
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and not got[2][pad].any()


SIZES = [  # M, N, K, ranks, ids: the smallest and the longest axes, the most adapters
    (1, 8, 8, [1], [0]),
    (70, 8, 8, [1, 2], [m % 2 for m in range(70)]),
    (70, 8, 16, [3], [0] * 70),
    (1, 1 << 20, 1 << 20, [2], [0]),
    (66, 8, 1 << 20, [1, 2], segment_ids(66, 2, 1)),
    (66, 1 << 20, 16, [2, 1], segment_ids(66, 2, 2)),
    (100, 64, 48, [1] * 16383, [(m * m * 163) % 16383 for m in range(100)]),
    (1500, 136, 64, [1 + l % 3 for l in range(500)], mixed_ids(1500, 500, 11)),
    (66100, 64, 80, [3, 5, 2], segment_ids(66100, 3, 3)),
    # three of twelve tiles have two to four adapters; 5 tokens and as many adapters
    (1500, 4096, 2048, [16, 8, 30, 24, 12, 5], [0] * 140 + [1] * 20 + [2] * 30 + [3] * 500 + [4] * 500 + [5] * 310),
    (5, 192, 1152, [16 + l for l in range(35)], [3, 17, 34, 9, 3]),
]


@pytest.mark.parametrize("case", range(len(SIZES)))
def test_lora_extreme_sizes(case):
    c = LoraCase(*SIZES[case], seed=70 + case, scales=[0.5 + (l % 7) / 8 for l in range(len(SIZES[case][3]))])
    s64, d64, ts, td = c.forward()
    s = torch.empty(c.M, max(c.ranks), device="cuda")
    out = aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    assert_within(s, s64, ts, "s")
    assert_within(out, d64, td + 2 * U * d64.abs() + half_step(torch.float32) * (d64.abs() + td), "out")
    x, sx, x64 = c.x, None, c.x.double()
    if c.K % 16 == 0:
        x, sx = aq.aq_quant_act(c.x.contiguous())
        x64 = x.double() * sx.double()[:, None]
    add = torch.zeros(c.M, c.K, device="cuda")
    (da64, ta), (db64, tb), (dx64, tx) = backward_reference(c, s, x64, add)
    da = torch.full((sum(c.ranks), c.K), float("nan"), device="cuda")
    db = torch.full((sum(c.ranks), c.N), float("nan"), device="cuda")
    _, _, dx = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, x, sx=sx, add=add, da=da, dbt=db)
    assert_within(da, da64, ta, "da")
    assert_within(db, db64, tb, "dbt")
    assert_within(dx, dx64, tx + 2 * U * dx64.abs() + half_step(torch.float32) * (dx64.abs() + tx), "dx")


@pytest.mark.parametrize("M", [3, 70])
def test_rows_past_32_bit_offsets(M):
    """Pitches so long that the last row lies more than 2^31 elements on."""
    N = K = 256
    pitch = (1 << 31) // (M - 1) // 16 * 16 + 64
    wide = lambda dtype: torch.empty(pitch * (M - 1) + K, dtype=dtype, device="cuda").as_strided((M, K), (pitch, 1))  # noqa: E731

    def moved(t, dtype=None):
        w = wide(dtype or t.dtype)
        w.copy_(t)
        return w

    ids = [m % 2 for m in range(M)]
    for ranks in ([8, 5], [8, 90]):
        c = LoraCase(M, N, K, ranks, ids, seed=M)
        y = normal(rng(M), M, N)
        s = torch.empty(M, max(ranks), device="cuda")
        want = aq.aq_lora_apply(c.ad, c.x, c.ids, y, s=s)
        wx, wy, wo = moved(c.x), moved(y), wide(y.dtype)
        assert torch.equal(aq.aq_lora_apply(c.ad, wx, c.ids, wy, out=wo), want)
        want = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x, add=y)
        wy.copy_(y)
        got = aq.aq_lora_backward(c.ad, moved(c.dy), c.ids, s, wx, add=wy, dx=wo)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        del wx, wy, wo, got
    w, _ = packed(N, K, 128, 0.5, 7)
    dy = normal(rng(8), M, N)
    want = aq.aq_linear_backward(w, dy, add=y)
    assert torch.equal(aq.aq_linear_backward(w, moved(dy), add=moved(y), out=wide(y.dtype)), want)
    want = aq.aq_silu_mul_quant(dy, y, keep=True)
    got = aq.aq_silu_mul_quant(moved(dy), moved(y), keep=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    want = aq.aq_silu_mul_backward(c.x, *want[2:])
    got = aq.aq_silu_mul_backward(moved(c.x), *got[2:], dgate=wide(y.dtype), dup=wide(y.dtype))
    assert all(torch.equal(p, q) for p, q in zip(got, want))


# ------------------------------------------------------------------ gated activation

def codes64(v, width):
    """The quantization rule in fp64 on the host, `width` features per scale."""
    M, F = v.shape
    q, s = np.empty((M, F), np.int8), np.empty((M, -(-F // width)), np.float32)
    for j in range(s.shape[1]):
        part = v[:, j * width:(j + 1) * width]
        sc = np.maximum(np.abs(part).max(1, keepdims=True) * (1.0 / 127.0), 1e-12)
        q[:, j * width:(j + 1) * width] = np.clip(np.rint(part / sc), -127, 127)
        with np.errstate(over="ignore"):
            s[:, j] = sc[:, 0].astype(np.float32)
    return q, s


def host(t):
    return t.double().cpu().numpy()


def gated64(g, u):
    with np.errstate(over="ignore"):
        return g * (1.0 / (1.0 + np.exp(-g))) * u


GATED = [(1, 16), (3, 48), (2, 128), (17, 144), (5, 1104), (64, 2048), (33, 9728), (7, 14336), (2, 17408), (2, 40000),
         (1, 65536)]


@pytest.mark.parametrize("M,F", GATED)
@pytest.mark.parametrize("keep", [False, True])
def test_gated_codes_are_exact(M, F, keep):
    g = rng(M * F)
    gate, up = normal(g, M, F + 8, scale=2.0)[:, :F], normal(g, M, F + 24)[:, :F]
    gate[:, ::37] *= 20
    if M > 2:
        gate[1], up[2] = 0, 0
    got = aq.aq_silu_mul_quant(gate, up, keep=keep)
    h = gated64(host(gate), host(up))
    hq, sh = codes64(h, F)
    assert np.array_equal(got[0].cpu().numpy(), hq)
    assert np.array_equal(got[1].cpu().numpy(), sh[:, 0])
    if keep:
        for q, s, v in ((got[2], got[3], gate), (got[4], got[5], up)):
            rq, rs = codes64(host(v), 128)
            assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    else:
        assert len(got) == 2


def test_gated_extreme_values():
    """Rows that fp32 alone cannot carry: huge and tiny products, gates far below the
    range of exp, one value among zeros; and a row of infinities beside a fine one."""
    F = 256
    g = rng(5)
    gate, up = normal(g, 10, F, scale=3.0), normal(g, 10, F)
    gate[0], up[0] = normal(g, F, scale=1e20), normal(g, F, scale=1e25)
    gate[1] = normal(g, F, scale=200.0)
    gate[2] = -normal(g, F).abs() * 30 - 70
    up[2] = normal(g, F, scale=1e37)
    up[3] = normal(g, F, scale=1e-38)
    gate[4], up[4] = 0, 0
    gate[4, 77], up[4, 77] = -3.5, 11.0
    gate[5] = -normal(g, F).abs() - 100
    up[6] = normal(g, F, scale=1e-14)
    gate[7] = 1.0          # every element the row's maximum
    up[7] = 2.0
    gate[8, 3], up[9, 200] = float("inf"), float("nan")
    fine = list(range(8))
    hq, sh, gq, gs, uq, us = aq.aq_silu_mul_quant(gate, up, keep=True)
    rq, rs = codes64(gated64(host(gate[fine]), host(up[fine])), F)
    assert np.array_equal(hq[fine].cpu().numpy(), rq)
    assert np.array_equal(sh[fine].cpu().numpy(), rs[:, 0])
    rq, rs = codes64(host(gate[fine]), 128)
    assert np.array_equal(gq[fine].cpu().numpy(), rq) and np.array_equal(gs[fine].cpu().numpy(), rs)


def test_gated_ties_round_to_even():
    """silu(g) = g / 2 at g = 0 only; ties of the final quotient come from u: g a large
    gate (silu(g) = g in fp64 from 40 on) and products that are half-integers of the scale."""
    F = 16
    gate = torch.full((1, F), 64.0, device="cuda", dtype=torch.bfloat16)
    want = [127.0, 2.5, -2.5, 3.5, 0.5, 1.5, -0.5, -126.5, 4.5, -127.0, 0.0, 100.5, 99.5, -1.5, 7.5, 8.5]
    up = torch.tensor([want], device="cuda", dtype=torch.bfloat16)
    hq, sh = aq.aq_silu_mul_quant(gate, up)
    rq, rs = codes64(gated64(host(gate), host(up)), F)
    assert sh.item() == 64.0 and np.array_equal(hq.cpu().numpy(), rq)
    assert list(rq[0]) == [127, 2, -2, 4, 0, 2, 0, -126, 4, -127, 0, 100, 100, -2, 8, 8]


@pytest.mark.parametrize("exponent", [0, -20, 30, -33, -34, -40])
def test_gated_checkpoints_of_every_ratio(exponent):
    """Every bf16 mantissa as a group's largest with every value from it down to 2^-9 of
    it: among them all quotients that are half-integers.  2^-33 and less: around the
    scale's floor and below it."""
    rest = np.concatenate([np.arange(128, 256) * 2.0 ** -d for d in range(10)])
    groups = []
    for a in range(128, 256):
        x = rest[rest <= a]
        x = np.concatenate([x, np.full(-len(x) % 126, float(a))]).reshape(-1, 126)
        x[:, ::3] *= -1
        groups.append(np.concatenate([np.full((len(x), 1), -float(a)), x, np.full((len(x), 1), a / 2)], 1))
    v = np.concatenate(groups) * 2.0 ** (exponent - 7)
    v = np.concatenate([v, np.zeros((-len(v) % 16, 128))]).reshape(-1, 16 * 128)
    gate = torch.from_numpy(v).to("cuda").to(torch.bfloat16)
    assert np.array_equal(host(gate), v)
    _, _, gq, gs, uq, us = aq.aq_silu_mul_quant(gate, -gate, keep=True)
    rq, rs = codes64(v, 128)
    assert np.array_equal(gq.cpu().numpy(), rq) and np.array_equal(gs.cpu().numpy(), rs)
    assert np.array_equal(uq.cpu().numpy(), -rq) and np.array_equal(us.cpu().numpy(), rs)


@pytest.mark.parametrize("M,F", GATED)
def test_gated_backward(M, F):
    g = rng(7 * M + F)
    gate, up = normal(g, M, F, scale=3.0), normal(g, M, F)
    gate[:, ::29] *= 30
    dh = normal(g, M, F + 16, scale=0.1)[:, :F]
    _, _, gq, gs, uq, us = aq.aq_silu_mul_quant(gate, up, keep=True)
    dg, du = aq.aq_silu_mul_backward(dh, gq, gs, uq, us)
    cols = torch.arange(F, device="cuda") // 128
    # the checkpoint's value is one fp32 product
    g64, u64 = (gq.float() * gs[:, cols]).double(), (uq.float() * us[:, cols]).double()
    p, d = torch.sigmoid(g64), dh.double()
    f = lambda z: z * torch.sigmoid(z)  # noqa: E731
    rg, ru = d * u64 * (p + g64 * p * (1 - p)), d * g64 * p
    # p within 8 2^-24 relative, 1 - p within 8 2^-24 absolute, a handful of products
    half = half_step(torch.bfloat16)
    assert_within(dg, rg, half * rg.abs() + (d * u64 * p).abs() * (g64.abs() + 2) * 16 * 2 ** -24 + 1e-38, "dgate")
    assert_within(du, ru, half * ru.abs() + ru.abs() * 16 * 2 ** -24 + 1e-38, "dup")
    # against central differences of the formula in fp64 (step h: h^2 / 6 of a third derivative below 1)
    h = 1e-4
    num = (f(g64 + h) - f(g64 - h)) / (2 * h) * d * u64
    assert_within(dg, num, half * num.abs() + (d * u64).abs() * 1e-6 + (d * u64 * p).abs() * (g64.abs() + 2) * 2e-6 + 1e-38)
    # strided outputs, rows beyond left alone
    wide = torch.full((2, M + 1, F + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    aq.aq_silu_mul_backward(dh, gq, gs, uq, us, dgate=wide[0], dup=wide[1])
    assert torch.equal(wide[0, :M, :F], dg) and torch.equal(wide[1, :M, :F], du)
    assert bool((wide[:, M:] == 7).all()) and bool((wide[:, :, F:] == 7).all())


# ------------------------------------------------------------------ input gradient of a packed projection

def packed(N, K, bN, frac8, seed):
    g = rng(seed)
    R, C = N // bN, K // 128
    pmap = torch.ones(R * C, dtype=torch.uint8, device="cuda")
    pmap[torch.randperm(R * C, generator=g, device="cuda")[: round(frac8 * R * C)]] = 0
    pmap = pmap.view(R, C)
    codes = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int16)
    int4 = pmap.bool().repeat_interleave(bN, 0).repeat_interleave(128, 1)
    codes = torch.where(int4, (codes & 15) - 8, codes).to(torch.int8)
    scales = (torch.rand((N, C), generator=g, device="cuda") * 9e-3 + 1e-3).to(torch.float16)
    w = (codes.double().view(N, C, 128) * scales.double()[:, :, None]).view(N, K)
    return aq.aq_pack(codes, scales, pmap, bN, 128), w


BACK = [(1, 64, 128, 64, 0.0), (1, 128, 128, 128, 1.0), (3, 192, 384, 64, 0.5), (16, 640, 256, 128, 0.5),
        (33, 1088, 640, 64, 0.25), (64, 256, 2560, 128, 0.5), (77, 1088, 2560, 64, 0.5), (128, 128, 256, 128, 0.0),
        (129, 384, 512, 128, 0.25), (200, 2048, 384, 128, 1.0), (257, 320, 896, 64, 0.5), (500, 1024, 1280, 128, 0.5),
        (1111, 704, 640, 64, 0.25), (2, 14336, 256, 128, 0.5), (900, 2048, 2176, 128, 0.5), (513, 4864, 2560, 128, 0.25),
        (1030, 2560, 9728, 64, 0.5), (1500, 2560, 4096, 128, 0.5), (2048, 2560, 9728, 128, 0.5), (6000, 512, 640, 64, 0.5)]


@pytest.mark.parametrize("M,N,K,bN,frac8", BACK)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_backward(M, N, K, bN, frac8, dtype):
    w, w64 = packed(N, K, bN, frac8, N + K + M)
    g = rng(M)
    dy = normal(g, M, N + 8, scale=0.01)[:, :N]
    add = normal(g, M, K + 8, scale=0.01, dtype=dtype)[:, :K]
    # weights rounded to bf16, products exact, fp32 sums, one rounding
    tol = (half_step(torch.bfloat16) + (N + 8) * U) * (dy.double().abs() @ w64.abs())
    ref = dy.double() @ w64
    got = aq.aq_linear_backward(w, dy, out_dtype=dtype)
    assert got.dtype == dtype
    assert_within(got, ref, tol + half_step(dtype) * (ref.abs() + tol))
    assert torch.equal(aq.aq_linear_backward(w, dy, out_dtype=dtype), got)
    ref = ref + add.double()
    both = aq.aq_linear_backward(w, dy, add=add)
    assert_within(both, ref, tol + half_step(dtype) * (ref.abs() + tol) + 2 * U * add.double().abs())
    wide = torch.full((M + 2, K + 16), 7.0, dtype=dtype, device="cuda")
    aq.aq_linear_backward(w, dy, out=wide)
    assert torch.equal(wide[:M, :K], got) and bool((wide[M:] == 7).all()) and bool((wide[:, K:] == 7).all())
    z = add.clone(memory_format=torch.contiguous_format)
    assert aq.aq_linear_backward(w, dy, add=z, out=z) is z and torch.equal(z, both)


@pytest.mark.parametrize("N,K,bN,frac8", [(256, 384, 128, 0.5), (192, 256, 64, 0.5), (128, 128, 64, 0.0)])
def test_linear_backward_reads_every_weight(N, K, bN, frac8):
    """dy = the identity: dx is the weight matrix, each entry off by its rounding alone."""
    w, w64 = packed(N, K, bN, frac8, N)
    got = aq.aq_linear_backward(w, torch.eye(N, device="cuda", dtype=torch.bfloat16), out_dtype=torch.float32)
    assert_within(got, w64, half_step(torch.bfloat16) * w64.abs())
    assert torch.equal(aq.aq_linear_backward(w, torch.eye(N, device="cuda", dtype=torch.bfloat16)),
                       w64.to(torch.bfloat16))


def test_linear_backward_infinite_rows_stay_out():
    w, _ = packed(256, 256, 128, 0.5, 3)
    dy = normal(rng(3), 150, 256)
    want = aq.aq_linear_backward(w, dy)
    dy[7], dy[149, 3] = float("inf"), float("nan")
    got = aq.aq_linear_backward(w, dy)
    ok = [m for m in range(150) if m not in (7, 149)]
    assert torch.equal(got[ok], want[ok]) and not torch.isfinite(got[149].float()).any()


# ------------------------------------------------------------------ graphs, streams, a whole block

class Block:
    """A gated MLP block over packed projections with adapters on all three, its
    forward pass and its backward pass."""

    def __init__(self, M, H, F, ids, seed=0, L=2):
        g = rng(seed)
        self.M, self.H, self.F = M, H, F
        self.w = {n: packed(*((H, F) if n == "down" else (F, H)), 128 if n != "up" else 64, 0.5, seed + i)
                  for i, n in enumerate(("gate", "up", "down"))}
        self.ranks = [6 + 5 * l for l in range(L)]
        R = sum(self.ranks)
        self.ad = {}
        for n in ("gate", "up", "down"):
            N, K = (H, F) if n == "down" else (F, H)
            self.ad[n] = aq.Adapters(normal(g, R, K, scale=K ** -0.5), normal(g, R, N, scale=0.05), self.ranks,
                                     [1.0 + l for l in range(L)])
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
        self.x, self.dy = normal(g, M, H, scale=0.3), normal(g, M, H, scale=0.01)

    def linear(self, n, x, xq, sx):
        s = torch.empty(self.M, max(self.ranks), device="cuda")
        y = aq.aq_linear_prefill(self.w[n][0], xq, sx, out_dtype=torch.bfloat16)
        return aq.aq_lora_apply(self.ad[n], x, self.ids, y, s=s), s

    def step(self):
        xq, sx = aq.aq_quant_act(self.x)
        gate, s_gate = self.linear("gate", self.x, xq, sx)
        up, s_up = self.linear("up", self.x, xq, sx)
        hq, sh, gq, gs, uq, us = aq.aq_silu_mul_quant(gate, up, keep=True)
        h = (hq.float() * sh[:, None]).to(torch.bfloat16)
        y, s_down = self.linear("down", h, hq, sh)
        grads = {}
        dh = aq.aq_linear_backward(self.w["down"][0], self.dy)
        da, db, dh = aq.aq_lora_backward(self.ad["down"], self.dy, self.ids, s_down, hq, sx=sh, add=dh)
        grads["down"] = (da, db)
        dgate, dup = aq.aq_silu_mul_backward(dh, gq, gs, uq, us)
        dx = aq.aq_linear_backward(self.w["gate"][0], dgate, out_dtype=torch.float32)
        dx = aq.aq_linear_backward(self.w["up"][0], dup, add=dx, out=dx)
        for n, d, s in (("gate", dgate, s_gate), ("up", dup, s_up)):
            da, db, dx = aq.aq_lora_backward(self.ad[n], d, self.ids, s, xq, sx=sx, add=dx, dx=dx)
            grads[n] = (da, db)
        flat = [y, dx] + [t for n in ("gate", "up", "down") for t in grads[n]]
        return flat, (xq, sx, hq, sh)

    def reference(self, kept):
        """The same block in fp64 on the codes that the step used: every projection
        sees its codes, as the packed layer does; adapters see the same activations."""
        xq, sx, hq, sh = (t.double() for t in kept)
        off = np.concatenate([[0], np.cumsum(self.ranks)])

        def delta(n, grads=None, dy=None, x=None):
            ad, out = self.ad[n], []
            for l in range(len(self.ranks)):
                rows, at = slice(int(off[l]), int(off[l + 1])), (self.ids == l).double()[:, None]
                out.append((ad.a[rows].double(), ad.bt[rows].double(), ad.scales[l], at, rows))
            return out

        def fwd(n, base, x):
            return base @ self.w[n][1].t() + sum(c * at * (x @ a.t() @ b) for a, b, c, at, _ in delta(n))

        def bwd(n, dy, x):
            da, db = torch.zeros_like(self.ad[n].a, dtype=torch.float64), torch.zeros_like(self.ad[n].bt, dtype=torch.float64)
            dx = dy @ self.w[n][1]
            for a, b, c, at, rows in delta(n):
                t = c * at * (dy @ b.t())
                da[rows], db[rows] = t.t() @ x, (c * at * (x @ a.t())).t() @ dy
                dx = dx + t @ a
            return da, db, dx

        x64, x8, h8 = self.x.double(), xq * sx[:, None], hq * sh[:, None]
        gate, up = fwd("gate", x8, x64), fwd("up", x8, x64)
        y = fwd("down", h8, h8)
        da_d, db_d, dh = bwd("down", self.dy.double(), h8)
        p = torch.sigmoid(gate)
        dgate, dup = dh * up * (p + gate * p * (1 - p)), dh * gate * p
        da_g, db_g, dx_g = bwd("gate", dgate, x8)
        da_u, db_u, dx_u = bwd("up", dup, x8)
        return [y, dx_g + dx_u, da_g, db_g, da_u, db_u, da_d, db_d]


@pytest.mark.parametrize("M,H,F,ids", [(9, 256, 512, mixed_ids(9, 2, 1)), (200, 512, 1408, segment_ids(200, 2, 2))])
def test_block_forward_and_backward(M, H, F, ids):
    """Norm-wise: the forward output is off by the bf16 roundings of the projections'
    outputs and the codes' input; a gradient passes at most four bf16 roundings (2^-8
    each), the 8-bit checkpoints of gate and up (half a step of 1 / 127 of the
    largest of 128, below 2% of the norm for normal values) and, for B, S of the
    unquantized activations: 6% in all."""
    b = Block(M, H, F, ids, seed=M)
    got, kept = b.step()
    for i, (x, ref) in enumerate(zip(got, b.reference(kept))):
        err = (x.double() - ref).norm() / ref.norm()
        assert err <= (0.01 if i == 0 else 0.06), (i, err.item())


def test_block_step_in_a_graph():
    """Captured and replayed on new inputs, beside an eager step on another stream."""
    b = Block(130, 256, 640, segment_ids(130, 2, 4), seed=4)
    b.step()  # kernels loaded, attributes set
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = b.step()
    other = Block(70, 256, 512, mixed_ids(70, 2, 5), seed=5)
    want_other, _ = other.step()
    for seed in (40, 41):
        b.x.copy_(normal(rng(seed), b.M, b.H, scale=0.3))
        b.dy.copy_(normal(rng(seed + 10), b.M, b.H, scale=0.01))
        b.ids.copy_(torch.tensor(mixed_ids(b.M, 2, seed), dtype=torch.int32))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph.replay()
        with torch.cuda.stream(side):
            got_other, _ = other.step()
        torch.cuda.synchronize()
        want, _ = b.step()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.equal(p, q) for p, q in zip(got_other, want_other))


def test_two_graphs_replayed_at_once():
    blocks = [Block(66 + 64 * i, 256, 512, mixed_ids(66 + 64 * i, 2, i), seed=20 + i) for i in range(2)]
    want = [b.step()[0] for b in blocks]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in blocks]
    for b in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.step()[0])
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, w))


def test_two_threads_on_one_stream():
    """Calls of two threads may take turns between one call's launches."""
    import threading
    blocks = [Block(66 + 64 * i, 256, 512, mixed_ids(66 + 64 * i, 2, i), seed=30 + i) for i in range(2)]
    want = [b.step()[0] for b in blocks]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, barrier = [[] for _ in blocks], threading.Barrier(2)

    def run(i):
        with torch.cuda.stream(stream):
            barrier.wait(30)
            for _ in range(20):
                got[i].append(blocks[i].step()[0])

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert len(g) == 20 and all(torch.equal(p, q) for o in g for p, q in zip(o, w))


@pytest.mark.parametrize("M,N,K", [(1500, 2560, 4096), (1030, 2560, 9728), (2048, 9728, 2560), (2048, 2560, 9728)])
def test_linear_backward_in_graphs_on_two_streams(M, N, K):
    """Captured and replayed on new gradients, beside eager calls of another stream and an
    adapter's backward pass of a third."""
    w, _ = packed(N, K, 128, 0.5, 1)
    dy, other = normal(rng(1), M, N), normal(rng(2), M, N)
    aq.aq_linear_backward(w, dy)
    want_other = aq.aq_linear_backward(w, other)
    c = LoraCase(300, 512, 640, [12, 40], segment_ids(300, 2, 6), seed=6)
    s = torch.empty(300, 40, device="cuda")
    aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    want_lora = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = aq.aq_linear_backward(w, dy)
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    for seed in (3, 4):
        dy.copy_(normal(rng(seed), M, N))
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
            with torch.cuda.stream(side):
                got_other = aq.aq_linear_backward(w, other)
            with torch.cuda.stream(third):
                got_lora = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x)
        torch.cuda.synchronize()
        assert torch.equal(got, aq.aq_linear_backward(w, dy)) and torch.equal(got_other, want_other)
        assert all(torch.equal(p, q) for p, q in zip(got_lora, want_lora))
