"""Calls of the adapter, gated-activation and input-gradient entries at the edges of what
they document: buffers beside and over one another, captured calls and their workspaces,
waits that give up, long sums."""
import time

import pytest
import torch

from test_gpu_adapters import (LoraCase, U, _no_kernel_errors, assert_within, mixed_ids, normal, packed,  # noqa: F401
                               rng, segment_ids)
from w8_a8_quantized_b200 import aq

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ buffers

@pytest.mark.parametrize("M", [9, 300])
def test_rows_side_by_side_in_one_buffer(M):
    """Inputs and outputs as column ranges of one buffer give the bits of separate tensors."""
    N, K, F = 256, 384, 512
    c = LoraCase(M, N, K, [8, 24], mixed_ids(M, 2, M), seed=M)
    s = torch.empty(M, 24, device="cuda")
    y = normal(rng(1), M, N)
    want = aq.aq_lora_apply(c.ad, c.x, c.ids, y, s=s)
    buf = torch.zeros(M, K + 2 * N + K, dtype=torch.bfloat16, device="cuda")
    x, y2, out, dx = buf[:, :K], buf[:, K:K + N], buf[:, K + N:K + 2 * N], buf[:, K + 2 * N:]
    x.copy_(c.x), y2.copy_(y)
    assert torch.equal(aq.aq_lora_apply(c.ad, x, c.ids, y2, out=out), want)
    dy = y2.copy_(c.dy)
    want = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x)
    got = aq.aq_lora_backward(c.ad, dy, c.ids, s, x, dx=dx)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    w, _ = packed(N, K, 128, 0.5, 2)
    assert torch.equal(aq.aq_linear_backward(w, dy, out=dx), aq.aq_linear_backward(w, c.dy))
    both = normal(rng(3), M, 2 * F)
    kept = aq.aq_silu_mul_quant(both[:, :F], both[:, F:], keep=True)
    want = aq.aq_silu_mul_quant(both[:, :F].contiguous(), both[:, F:].contiguous(), keep=True)
    assert all(torch.equal(p, q) for p, q in zip(kept, want))
    grads = torch.zeros(M, 3 * F, dtype=torch.bfloat16, device="cuda")
    grads[:, 2 * F:] = normal(rng(4), M, F, scale=0.01)
    want = aq.aq_silu_mul_backward(grads[:, 2 * F:].contiguous(), *kept[2:])
    got = aq.aq_silu_mul_backward(grads[:, 2 * F:], *kept[2:], dgate=grads[:, :F], dup=grads[:, F:2 * F])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("M,F", [(1, 16), (77, 9728), (300, 1104), (33, 40000)])
def test_gated_backward_in_place(M, F):
    gate, up, dh = (normal(rng(i), M, F) for i in range(3))
    kept = aq.aq_silu_mul_quant(gate, up, keep=True)[2:]
    want = aq.aq_silu_mul_backward(dh, *kept)
    for i, name in enumerate(("dgate", "dup")):
        d = dh.clone()
        got = aq.aq_silu_mul_backward(d, *kept, **{name: d})
        assert got[i] is d and all(torch.equal(p, q) for p, q in zip(got, want))


def test_outputs_over_inputs_are_refused():
    M, N = 130, 256
    c = LoraCase(M, N, N, [8], segment_ids(M, 1, 1), seed=5)
    s = torch.empty(M, 8, device="cuda")
    aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    w, _ = packed(N, N, 128, 0.5, 2)
    dy, x = c.dy.clone(), c.x.clone()
    for call in (lambda: aq.aq_lora_backward(c.ad, dy, c.ids, s, x, add=dy, dx=dy),
                 lambda: aq.aq_lora_backward(c.ad, dy, c.ids, s, x, dx=dy),
                 lambda: aq.aq_lora_backward(c.ad, dy, c.ids, s, x, dx=x),
                 lambda: aq.aq_linear_backward(w, dy, add=dy, out=dy),
                 lambda: aq.aq_linear_backward(w, dy, out=dy),
                 lambda: aq.aq_lora_apply(c.ad, x, c.ids, out=x)):
        with pytest.raises(aq.AqError):
            call()
    assert torch.equal(dy, c.dy) and torch.equal(x, c.x)


# ------------------------------------------------------------------ input gradient

SUMS = [(1, 128, 256, 128), (33, 1088, 640, 64), (64, 4864, 384, 128), (77, 1088, 2560, 64), (129, 384, 512, 128),
        (200, 14336, 256, 128), (257, 2560, 896, 64), (1030, 2560, 9728, 64), (2048, 9728, 1280, 128),
        (700, 4096, 14336, 128)]


@pytest.mark.parametrize("N,K,bN,frac8", [(256, 384, 128, 0.5), (192, 256, 64, 0.5), (128, 128, 64, 1.0)])
def test_linear_backward_takes_the_weights_as_asked(N, K, bN, frac8):
    """dy = the identity: dx is the weight matrix, exact or rounded once."""
    w, w64 = packed(N, K, bN, frac8, N)
    eye = torch.eye(N, device="cuda", dtype=torch.bfloat16)
    rounded = w64.to(torch.bfloat16)
    for out_dtype, weights, want in ((torch.float32, None, w64), (torch.float32, torch.float32, w64),
                                     (torch.float32, torch.bfloat16, rounded.double()), (torch.bfloat16, None, rounded),
                                     (torch.bfloat16, torch.bfloat16, rounded), (torch.bfloat16, torch.float32, rounded)):
        got = aq.aq_linear_backward(w, eye, out_dtype=out_dtype, weights=weights)
        assert got.dtype == out_dtype and torch.equal(got.to(want.dtype), want), (out_dtype, weights)
    with pytest.raises(TypeError):
        aq.aq_linear_backward(w, eye, weights=torch.float16)


@pytest.mark.parametrize("M,N,K,bN", SUMS)
def test_linear_backward_keeps_fp32(M, N, K, bN):
    """A sum of 512 rows takes 96 additions in tensor memory, each off by 2^-23 of the partial
    sum at most, whose norm grows with the root of its terms: 64 2^-23 of the norm, and one
    rounding for each 512 rows and for `add` (weights rounded to bf16 are off by 1.6e-3)."""
    w, w64 = packed(N, K, bN, 0.5, N + K + M)
    dy = normal(rng(M), M, N, scale=0.01)
    add = torch.randn(M, K, generator=rng(M + 1), device="cuda") * 0.01
    ref = dy.double() @ w64
    tol = (64 + N // 512 + 2) * U
    got = aq.aq_linear_backward(w, dy, out_dtype=torch.float32)
    assert (got.double() - ref).norm() <= tol * ref.norm()
    assert torch.equal(aq.aq_linear_backward(w, dy, out_dtype=torch.float32), got)
    both = aq.aq_linear_backward(w, dy, add=add)
    assert (both.double() - ref - add.double()).norm() <= tol * (ref.norm() + add.double().norm())
    z = add.clone()
    assert aq.aq_linear_backward(w, dy, add=z, out=z) is z and torch.equal(z, both)
    wide = torch.full((M + 2, K + 16), 7.0, device="cuda")
    aq.aq_linear_backward(w, dy, out=wide)
    assert torch.equal(wide[:M, :K], got) and bool((wide[M:] == 7).all()) and bool((wide[:, K:] == 7).all())
    # exact weights and sums in tensor memory alone for a bf16 result: its own rounding, after 3N / 16 additions
    got16 = aq.aq_linear_backward(w, dy, weights=torch.float32)
    own = (ref.to(torch.bfloat16).double() - ref).norm()
    assert (got16.double() - ref).norm() <= own * 1.01 + 3 * N / 16 * U * ref.norm()


def whole_numbers(N, K, bN, frac8, seed):
    """Packed weights that are whole multiples of 2^-4, 8 bits wide at most, and their values."""
    g = rng(seed)
    R, C = N // bN, K // 128
    pmap = torch.ones(R * C, dtype=torch.uint8, device="cuda")
    pmap[torch.randperm(R * C, generator=g, device="cuda")[: round(frac8 * R * C)]] = 0
    pmap = pmap.view(R, C)
    codes = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int16)
    int4 = pmap.bool().repeat_interleave(bN, 0).repeat_interleave(128, 1)
    codes = torch.where(int4, (codes & 15) - 8, codes).to(torch.int8)
    scales = 2.0 ** torch.randint(-4, -2, (N, C), generator=g, device="cuda")
    w = (codes.double().view(N, C, 128) * scales.double()[:, :, None]).view(N, K)
    return aq.aq_pack(codes, scales.to(torch.float16), pmap, bN, 128), w


@pytest.mark.parametrize("M,N,K,bN", SUMS + [(2, 14336, 256, 128), (16, 4864, 256, 128), (900, 2048, 2176, 128),
                                             (513, 4864, 2560, 128), (1500, 2560, 4096, 128), (2048, 2560, 9728, 128),
                                             (6000, 512, 640, 64), (4096, 14336, 512, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weights", [torch.bfloat16, torch.float32])
def test_linear_backward_sums_every_row(M, N, K, bN, dtype, weights):
    """Weights of 8 bits times dy in -2 .. 2: every sum is a whole multiple of 2^-4 below 2^24
    of them (2 x 256 x 14336 < 2^23), so fp32 holds it in any order and the result is exact: a
    step, a row or an entry that is left out or taken twice shows."""
    w, w64 = whole_numbers(N, K, bN, 0.5, N + K + M)
    dy = torch.randint(-2, 3, (M, N), generator=rng(M), device="cuda").to(torch.bfloat16)
    add = torch.randint(-64, 65, (M, K), generator=rng(M + 1), device="cuda").to(dtype)
    ref = dy.double() @ w64
    assert torch.equal(aq.aq_linear_backward(w, dy, out_dtype=dtype, weights=weights), ref.to(dtype))
    assert torch.equal(aq.aq_linear_backward(w, dy, add=add, weights=weights), (ref + add.double()).to(dtype))


@pytest.mark.parametrize("M", [150, 1100])
def test_exact_weights_keep_infinite_rows_apart(M):
    w, _ = packed(1024, 2560, 128, 0.5, 3)
    dy = normal(rng(3), M, 1024)
    want = aq.aq_linear_backward(w, dy, out_dtype=torch.float32)
    dy[7], dy[M - 1, 3] = float("inf"), float("nan")
    got = aq.aq_linear_backward(w, dy, out_dtype=torch.float32)
    ok = [m for m in range(M) if m not in (7, M - 1)]
    assert torch.equal(got[ok], want[ok])
    assert not torch.isfinite(got[[7, M - 1]]).any()


# ------------------------------------------------------------------ waits that give up

WAIT_NS = 20_000_000


def gave_up(ws, codes, t0):
    rc, info = aq.aq_workspace_status(ws)  # synchronizes
    assert rc == -7 and info in codes, (rc, info)
    assert time.monotonic() - t0 < 5.0
    assert not ws[:256].any()


@pytest.mark.parametrize("M,N,K,dtype", [
    (64, 1024, 256, torch.bfloat16), (300, 1024, 384, torch.bfloat16), (300, 1024, 384, torch.float32),  # single CTAs
    (1030, 512, 5120, torch.bfloat16), (2048, 512, 2560, torch.bfloat16), (2048, 1024, 2560, torch.float32)])  # pairs
@pytest.mark.parametrize("stop_after", [0, 3])
def test_stalled_input_gradient(M, N, K, dtype, stop_after):
    """A weight producer that stops (in a pair the second CTA's): every role gives up, the error is
    reported, and the same workspace serves ordinary calls."""
    w, _ = packed(N, K, 128, 0.5, 7)
    dy = normal(rng(M), M, N, scale=0.01)
    want = aq.aq_linear_backward(w, dy, out_dtype=dtype)
    ws = torch.zeros(aq.aq_linear_backward_workspace_bytes(M, w), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    t0 = time.monotonic()
    aq.aq_debug_linear_backward_stalled(w, dy, ws, out_dtype=dtype, wait_ns=WAIT_NS, stop_after=stop_after)
    gave_up(ws, range(1, 8), t0)
    assert torch.equal(aq.aq_linear_backward(w, dy, out_dtype=dtype, ws=ws), want)
    assert aq.aq_workspace_status(ws) == (0, 0)


@pytest.mark.parametrize("kernel,codes", [(0, range(31, 37)), (1, range(41, 47)), (2, range(21, 27))])
@pytest.mark.parametrize("ranks", [[8, 24], [16, 40], [64]])
@pytest.mark.parametrize("checkpoint", [True, False])
@pytest.mark.parametrize("stop_after", [0, 2])
def test_stalled_adapters(kernel, codes, ranks, checkpoint, stop_after):
    M, N, K = 6000 if stop_after else 333, 1024, 1536
    c = LoraCase(M, N, K, ranks, mixed_ids(M, len(ranks), 3), seed=3)
    s = torch.empty(M, max(ranks), device="cuda")
    aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    x, sx = aq.aq_quant_act(c.x) if checkpoint else (c.x, None)
    want = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, x, sx=sx)
    ws = torch.zeros(aq.aq_lora_workspace_bytes(c.ad, M, True), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    t0 = time.monotonic()
    aq.aq_debug_lora_backward_stalled(c.ad, c.dy, c.ids, s, x, sx, kernel, ws, wait_ns=WAIT_NS, stop_after=stop_after)
    gave_up(ws, codes, t0)
    got = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, x, sx=sx, ws=ws)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert aq.aq_workspace_status(ws) == (0, 0)


def test_stalled_weight_gradients_of_few_tokens():
    c = LoraCase(30, 256, 512, [4, 7, 130], mixed_ids(30, 3, 3), seed=3)
    s = torch.zeros(30, 130, device="cuda")
    ws = torch.zeros(aq.aq_lora_workspace_bytes(c.ad, 30, True), dtype=torch.uint8, device="cuda")
    t0 = time.monotonic()
    aq.aq_debug_lora_backward_stalled(c.ad, c.dy, c.ids, s, c.x, None, 2, ws, wait_ns=WAIT_NS, stop_after=0)
    gave_up(ws, range(21, 27), t0)


# ------------------------------------------------------------------ workspaces

def test_workspaces_need_a_clear_header_only():
    """Whatever the rest of a workspace holds, the bits are the same."""
    c = LoraCase(333, 640, 1536, [5, 40, 64], mixed_ids(333, 3, 2), seed=2)
    few = LoraCase(40, 640, 1536, [5, 40, 200], mixed_ids(40, 3, 2), seed=2)
    w, _ = packed(640, 1536, 128, 0.5, 4)

    def filled(need, value):
        ws = torch.full((need,), value, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        return ws

    for case in (c, few):
        s = torch.empty(case.M, max(case.ranks), device="cuda")
        got = []
        for value in (0, 255, 127):
            out = aq.aq_lora_apply(case.ad, case.x, case.ids, s=s,
                                   ws=filled(aq.aq_lora_workspace_bytes(case.ad, case.M, False), value))
            got.append((out,) + aq.aq_lora_backward(case.ad, case.dy, case.ids, s, case.x,
                                                    ws=filled(aq.aq_lora_workspace_bytes(case.ad, case.M, True), value)))
            for dtype in (torch.bfloat16, torch.float32):
                ws = filled(aq.aq_linear_backward_workspace_bytes(case.M, w), value)
                got[-1] += (aq.aq_linear_backward(w, case.dy, ws=ws, out_dtype=dtype),)
        for other in got[1:]:
            assert all(torch.equal(p, q) for p, q in zip(got[0], other))


def test_a_replay_that_gives_up_is_reported():
    w, _ = packed(512, 2560, 128, 0.5, 7)
    dy = normal(rng(1), 300, 512, scale=0.01)
    c = LoraCase(333, 512, 640, [8, 24], mixed_ids(333, 2, 3), seed=3)
    s = torch.empty(333, 24, device="cuda")
    aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    want = aq.aq_linear_backward(w, dy)
    aq.check_all_workspaces()
    for stall in (lambda: aq.aq_debug_linear_backward_stalled(w, dy, wait_ns=WAIT_NS),
                  lambda: aq.aq_debug_lora_backward_stalled(c.ad, c.dy, c.ids, s, c.x, None, 0, wait_ns=WAIT_NS)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = aq.aq_linear_backward(w, dy)
            stall()
            again = aq.aq_linear_backward(w, dy)
        torch.cuda.synchronize()
        aq.check_all_workspaces()  # captured, not run
        for _ in range(2):  # each replay anew
            graph.replay()
            with pytest.raises(aq.AqError):
                aq.check_all_workspaces()
            aq.check_all_workspaces()  # and once
        assert torch.equal(got, want) and torch.equal(again, want)
        stall()  # not captured: the same
        with pytest.raises(aq.AqError):
            aq.check_all_workspaces()


def test_errors_outlive_a_grown_workspace_and_its_thread():
    import threading
    w, _ = packed(512, 2560, 128, 0.5, 7)
    small, large = normal(rng(1), 40, 512), normal(rng(2), 3000, 512)
    want = aq.aq_linear_backward(w, large, out_dtype=torch.float32)
    torch.cuda.synchronize()
    free, got = [], []

    def run():
        with torch.cuda.stream(torch.cuda.Stream()):
            aq.aq_debug_linear_backward_stalled(w, small, wait_ns=WAIT_NS, stop_after=0)
            got.append(aq.aq_linear_backward(w, large, out_dtype=torch.float32))  # a larger workspace takes its place
            free.append(torch.cuda.memory_allocated())
            torch.cuda.current_stream().synchronize()

    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    assert torch.equal(got[0], want)
    assert torch.cuda.memory_allocated() < free[0]  # the thread's workspaces went with it
    with pytest.raises(aq.AqError):
        aq.check_all_workspaces()
    aq.check_all_workspaces()


def test_a_captured_workspace_clears_its_header_only():
    w, _ = packed(256, 256, 128, 0.5, 1)  # (a header to report to)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ws = aq._new_ws(1 << 20, w.device)
    ws.fill_(9)
    graph.replay()
    torch.cuda.synchronize()
    assert bool((ws[256:] == 9).all()) and not ws[:16].any() and not ws[24:256].any()


# ------------------------------------------------------------------ products of adapters

@pytest.mark.parametrize("M", [8, 60, 150])
@pytest.mark.parametrize("rank", [2, 31, 48, 70])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products_keep_24_bits_whatever_the_output(M, rank, dtype):
    """S = (n, -p) with n a whole number of 24 bits and p its leading 16: the output n - p is what the last
    8 bits hold, in whole numbers, so every sum is exact."""
    L, K, N = 5, 128, 256
    g = torch.Generator().manual_seed(M + rank)
    n = torch.randint(2 ** 23, 2 ** 24, (L,), generator=g).double()
    hi = n.to(torch.bfloat16).double()
    p = hi + (n - hi).to(torch.bfloat16).double()
    assert (n != p).any()

    def row(v):  # 256 a + 16 b + c = v with 8-bit multiples of powers of two
        v, out = v.clone(), torch.zeros(L, K, dtype=torch.float64)
        for i, (x, step) in enumerate(((256, 65536), (16, 256), (1, 1))):
            digit = torch.trunc(v / step)
            out[:, i] = digit * step / x
            v -= digit * step
        assert not v.any()
        return out

    a = torch.zeros(L, rank, K, dtype=torch.float64)
    a[:, 0], a[:, 1] = row(n), -row(p)
    assert torch.equal(a.to(torch.bfloat16).double(), a)
    b = torch.zeros(L * rank, N, dtype=torch.bfloat16, device="cuda")
    b[0::rank], b[1::rank] = 1, 1
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = 256, 16, 1
    ids = torch.arange(M, dtype=torch.int32, device="cuda") % L
    want = (n - p).to(device="cuda")[ids.long()][:, None].expand(M, N).to(dtype)
    ad = aq.Adapters(a.reshape(L * rank, K).to(torch.bfloat16).cuda(), b, [rank] * L, [1.0] * L)
    assert torch.equal(aq.aq_lora_apply(ad, x, ids, out_dtype=dtype), want)
    # the same through the gradient of x, the tables' sides exchanged
    back = aq.Adapters(b, a.reshape(L * rank, K).to(torch.bfloat16).cuda(), [rank] * L, [1.0] * L)
    z = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dx = aq.aq_lora_backward(back, x, ids, torch.zeros(M, rank, device="cuda"), z, dx_dtype=dtype)[2]
    assert torch.equal(dx, want)


def test_exact_input_gradient_past_32_bit_offsets():
    """Several sums of 512 rows, each added where the last row lies more than 2^31 elements on."""
    M, N, K = 70, 1600, 256
    pitch = (1 << 31) // (M - 1) // 16 * 16 + 64
    w, _ = packed(N, K, 64, 0.5, 7)
    dy = normal(rng(8), M, N)
    want = aq.aq_linear_backward(w, dy, out_dtype=torch.float32)
    out = torch.empty(pitch * (M - 1) + K, device="cuda").as_strided((M, K), (pitch, 1))
    assert torch.equal(aq.aq_linear_backward(w, dy, out=out), want)


def test_exact_input_gradients_of_two_streams_and_a_graph():
    w, _ = packed(2560, 1280, 128, 0.5, 1)
    dy = [normal(rng(i), 700, 2560) for i in range(3)]
    want = [aq.aq_linear_backward(w, d, out_dtype=torch.float32) for d in dy]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = aq.aq_linear_backward(w, dy[0], out_dtype=torch.float32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        graph.replay()
        outs = []
        for s, d in zip(streams, dy[1:]):
            with torch.cuda.stream(s):
                outs.append(aq.aq_linear_backward(w, d, out_dtype=torch.float32))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip([got] + outs, want))
