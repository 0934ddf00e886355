"""Slots sorted by expert and rows moved there and back, against NumPy in 64 bits.

Tolerances, with u = eps / 2 of the output's type and v = 2^-24 (fp32):
* the sort and the plain row copies are exact;
* y and dx are a chain of at most K + 1 fp32 additions of (exact or once-rounded) products and one
  rounding: |err| <= (K + 2) v sum|terms| + u |ref| (1 + 2^-7) + the smallest subnormal;
* dys is one fp32 product and one rounding: |err| <= (u + 2 v) |ref| + the smallest subnormal;
* dweights is a sum of d fp32 products in some order: |err| <= (d + 2) v sum|terms|.
"""
import numpy as np
import pytest
import torch

from token_choice_routing_b200 import binding as B

pytestmark = pytest.mark.gpu

V = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def u_of(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


def f64(t):
    return t.detach().double().cpu().numpy()


def sort_ref(ids, N):
    """Rows of the stable (expert, slot) order, by the definition."""
    flat = np.asarray(ids, dtype=np.int64).reshape(-1)
    K = ids.shape[1]
    row = np.full(flat.size, -1, dtype=np.int64)
    has = (flat >= 0) & (flat < N)
    order = np.argsort(np.where(has, flat, N), kind="stable")
    R = int(has.sum())
    row[order[:R]] = np.arange(R)
    counts = np.bincount(flat[has], minlength=N)[:N] if R else np.zeros(N, dtype=np.int64)
    return counts, np.concatenate([[0], np.cumsum(counts)]), order[:R] // K, row.reshape(ids.shape)


def run_sort(ids, N, fill=-7):
    T, K = ids.shape
    o = dict(counts=torch.full((N,), fill, dtype=torch.int32, device="cuda"),
             offsets=torch.full((N + 1,), fill, dtype=torch.int32, device="cuda"),
             perm_tok=torch.full((T * K,), fill, dtype=torch.int32, device="cuda"),
             slot_row=torch.full((T, K), fill, dtype=torch.int32, device="cuda"))
    ws = torch.full((B.sort_workspace_bytes(T, K, N),), 255, dtype=torch.uint8, device="cuda")
    B.sort_slots(ids, N, o["counts"], o["offsets"], o["perm_tok"], o["slot_row"], ws)
    torch.cuda.synchronize()
    assert B.get_device_status(ws) == B.OK
    return o


def check_sort(ids, N, fill=-7):
    o = run_sort(ids, N, fill)
    counts, offsets, perm, row = sort_ref(ids.cpu().numpy(), N)
    assert np.array_equal(o["counts"].cpu().numpy(), counts)
    assert np.array_equal(o["offsets"].cpu().numpy(), offsets)
    assert np.array_equal(o["slot_row"].cpu().numpy(), row)
    R = int(offsets[-1])
    assert np.array_equal(o["perm_tok"][:R].cpu().numpy(), perm)
    assert bool((o["perm_tok"][R:] == fill).all())     # behind the last row: as it was


def draw_ids(rng, T, K, N, drop, dtype=np.int32):
    ids = rng.integers(0, N, size=(T, K))
    lost = rng.random((T, K)) < drop
    return torch.from_numpy(np.where(lost, rng.choice([-1, N, N + 5], size=(T, K)), ids).astype(dtype)).cuda()


@pytest.mark.parametrize("T,K,N,drop", [
    (1, 1, 1, 0.0), (1, 32, 1024, 0.3), (7, 3, 5, 0.5), (33, 1, 64, 0.2), (64, 4, 64, 0.5), (1000, 8, 60, 0.4),
    (1023, 16, 1000, 0.1), (4096, 1, 2, 0.0), (4097, 1, 33, 0.6), (5001, 7, 129, 0.3), (16384, 8, 64, 0.75),
    (131072, 8, 64, 0.4), (40000, 31, 1024, 0.2)])
@pytest.mark.parametrize("wide", [False, True])
def test_sort_is_the_stable_order(T, K, N, drop, wide):
    rng = np.random.default_rng(T * 31 + K * 7 + N)
    check_sort(draw_ids(rng, T, K, N, drop, np.int64 if wide else np.int32), N)


def test_sort_of_one_expert_every_expert_and_none():
    for T, K in ((5, 2), (9000, 8)):
        check_sort(torch.full((T, K), 3, dtype=torch.int32, device="cuda"), 9)      # the same index in every slot
        check_sort(torch.full((T, K), -1, dtype=torch.int32, device="cuda"), 9)     # no slot has an expert
        check_sort(torch.full((T, K), 9, dtype=torch.int64, device="cuda"), 9)


def test_sort_reads_wide_ids_in_full():
    """Ids that a 32-bit read would take for experts."""
    big = 1 << 32
    ids = torch.tensor([[0, big], [big + 3, 3], [-big + 2, 2], [1 << 62, 7]], dtype=torch.int64, device="cuda")
    check_sort(ids, 8)
    ids = torch.tensor([[2 ** 31 - 1, 0], [-2 ** 31, 1]], dtype=torch.int32, device="cuda")
    check_sort(ids, 2)


def test_sort_of_no_tokens_writes_zero_counts():
    o = run_sort(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 6)
    assert o["counts"].tolist() == [0] * 6 and o["offsets"].tolist() == [0] * 7


def test_sort_matches_the_layer_dispatch():
    """On the routing of the layer's own router, the layout that moe_dispatch gives."""
    from token_choice_routing_b200 import inputs as I
    from tests import gpu_helpers as H
    cfg = I.small_config("sort_dispatch", T=1500, d=128, N=24, F=64, F_shared=64, K=6, M=12, config_id=960)
    _, _, _, out = H.run_forward(I.make_inputs(cfg))
    o = run_sort(out["topk_idx"], cfg.N)
    for n in ("counts", "offsets", "slot_row"):
        assert torch.equal(o[n], out[n]), n
    R = int(out["offsets"][-1])
    assert torch.equal(o["perm_tok"][:R], out["perm_tok"][:R])


# --------------------------------------------------------------------------- row movement

SHAPES = [(1, 1, 1, 1), (1, 8, 64, 2048), (2, 4, 8, 8192), (3, 2, 4, 7), (33, 5, 9, 100), (70, 32, 50, 640), (64, 4, 16, 256), (130, 32, 40, 33),
          (257, 3, 7, 1001), (300, 8, 64, 1024), (2000, 6, 64, 72), (511, 16, 300, 520)]


def make(T, K, N, d, dt, seed, drop=0.4, pad=0, lead=0):
    """Row tensors with `pad` extra columns and `lead` leading elements, so that strides and
    alignment differ from the dense ones."""
    rng = np.random.default_rng(seed)
    ids = draw_ids(rng, T, K, N, drop)
    slot_row = run_sort(ids, N)["slot_row"]

    def rows(n, scale=1.0, fill=None):
        flat = torch.zeros(n * (d + pad) + lead, dtype=torch.float32)
        if fill is None:
            flat[:] = torch.from_numpy(rng.standard_normal(flat.numel()).astype(np.float32)) * scale
        else:
            flat[:] = fill
        return flat.to(dt).cuda()[lead:].view(n, d + pad)[:, :d]

    w = torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda()
    return rng, slot_row, rows, w


LAYOUTS = [(0, 0), (8, 0), (3, 0), (0, 1), (8, 8)]


@pytest.mark.parametrize("T,K,N,d", SHAPES)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_permute_copies_rows(T, K, N, d, dtype):
    dt = TYPES[dtype]
    for i, (pad, lead) in enumerate(LAYOUTS):
        _, sr, rows, _ = make(T, K, N, d, dt, 100 + i, pad=pad, lead=lead)
        x, xs = rows(T), rows(T * K, fill=5.0)
        B.permute(x, sr, xs)
        ref = torch.full((T * K, d), 5.0, dtype=dt, device="cuda")     # rows without a slot: as they were
        t, k = torch.nonzero(sr >= 0, as_tuple=True)
        ref[sr[t, k].long()] = x[t]
        assert torch.equal(xs, ref), (pad, lead)


def collect_ref(rows, sr, w, base):
    T, K = sr.shape
    acc, mag = (np.zeros((T, rows.shape[1])), 0.0) if base is None else (f64(base), np.abs(f64(base)))
    r, s = f64(rows), sr.cpu().numpy()
    mag = np.zeros_like(acc) + mag
    acc = acc.copy()
    for k in range(K):
        t = np.nonzero(s[:, k] >= 0)[0]
        term = r[s[t, k]] * (1.0 if w is None else f64(w)[t, k][:, None])
        acc[t] += term
        mag[t] += np.abs(term)
    return acc, mag


def check_collect(out, ref, mag, K):
    dt = out.dtype
    err = np.abs(f64(out) - ref)
    bound = (K + 2) * V * mag + u_of(dt) * np.abs(ref) * (1 + 2.0 ** -7) + tiny(dt)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("T,K,N,d", SHAPES)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_unpermute_and_permute_backward(T, K, N, d, dtype):
    dt = TYPES[dtype]
    for i, (pad, lead) in enumerate(LAYOUTS):
        _, sr, rows, w = make(T, K, N, d, dt, 200 + i, pad=pad, lead=lead)
        ys, base, y = rows(T * K), rows(T), rows(T, fill=9.0)
        # weights and rows that no slot with a row uses must not reach the result
        w = torch.where(sr >= 0, w, float("nan"))
        R = int((sr >= 0).sum())
        ys[R:] = float("nan")
        B.unpermute(ys, w, sr, y, base=base)
        check_collect(y, *collect_ref(ys, sr, w, base), K)
        B.unpermute(ys, w, sr, y)
        check_collect(y, *collect_ref(ys, sr, w, None), K)
        want = y.clone()
        y.copy_(base)
        B.unpermute(ys, w, sr, y, base=y)                             # in place
        B.unpermute(ys, w, sr, want, base=base)
        assert torch.equal(y, want)
        B.permute_backward(ys, sr, y, base=base)
        check_collect(y, *collect_ref(ys, sr, None, base), K)
        B.permute_backward(ys, sr, y)
        check_collect(y, *collect_ref(ys, sr, None, None), K)


@pytest.mark.parametrize("T,K,N,d", SHAPES)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_unpermute_backward(T, K, N, d, dtype):
    dt = TYPES[dtype]
    for i, (pad, lead) in enumerate(LAYOUTS):
        _, sr, rows, w = make(T, K, N, d, dt, 300 + i, pad=pad, lead=lead)
        dy, ys, dys = rows(T), rows(T * K), rows(T * K, fill=3.0)
        w = torch.where(sr >= 0, w, float("nan"))
        ys[int((sr >= 0).sum()):] = float("nan")
        dw = torch.full((T, K), 7.0, device="cuda")
        B.unpermute_backward(dy, ys, w, sr, dys, dw)
        check_spread(dy, f64(ys), w, sr, dys, dw, 3.0)
        dys2, dw2 = rows(T * K, fill=3.0), torch.full((T, K), 7.0, device="cuda")
        B.unpermute_backward(dy, None, w, sr, dys2, None)            # one output at a time
        B.unpermute_backward(dy, ys, w, sr, None, dw2)
        assert torch.equal(dys2, dys) and torch.equal(dw2, dw)


def check_spread(dy, ys, w, sr, dys, dw, fill):
    dt, (T, K), d = dy.dtype, sr.shape, dy.shape[1]
    s, g, wn = sr.cpu().numpy(), f64(dy), f64(w)
    ref = np.full((dys.shape[0], d), fill)
    dref, mag = np.zeros((T, K)), np.zeros((T, K))
    for k in range(K):
        t = np.nonzero(s[:, k] >= 0)[0]
        ref[s[t, k]] = g[t] * wn[t, k][:, None]
        dref[t, k] = (g[t] * ys[s[t, k]]).sum(1)
        mag[t, k] = np.abs(g[t] * ys[s[t, k]]).sum(1)
    err = np.abs(f64(dys) - ref)
    assert np.all(err <= (u_of(dt) + 2 * V) * np.abs(ref) + tiny(dt)), float(err.max())
    err = np.abs(f64(dw) - dref)
    assert np.all(err <= (d + 2) * V * mag), float((err / np.maximum(mag, 1e-300)).max())


@pytest.mark.parametrize("T,K,N,d", SHAPES)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_unpermute_backward_from_8_bit_rows(T, K, N, d, dtype):
    dt = TYPES[dtype]
    for i, (pad, lead) in enumerate(LAYOUTS[:4]):
        rng, sr, rows, w = make(T, K, N, d, dt, 400 + i, pad=pad, lead=lead)
        dy, dys = rows(T), rows(T * K, fill=3.0)
        codes = torch.from_numpy(rng.integers(-127, 128, size=(T * K, d)).astype(np.int8)).cuda()
        byte = rng.integers(110, 130, size=(T * K, (d + 31) // 32)).astype(np.uint8)
        scales = torch.from_numpy(byte).cuda()
        ys = f64(codes) * np.repeat(2.0 ** (byte.astype(np.float64) - 127), 32, axis=1)[:, :d]
        dw = torch.full((T, K), 7.0, device="cuda")
        B.unpermute_backward8(dy, codes, scales, w, sr, dys, dw)
        check_spread(dy, ys, w, sr, dys, dw, 3.0)
        dw2 = torch.full((T, K), 7.0, device="cuda")
        B.unpermute_backward8(dy, codes, scales, w, sr, None, dw2)
        assert torch.equal(dw2, dw)


def test_a_block_stored_as_nan_reaches_the_gate_gradient():
    dy = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.ones((2, 64), dtype=torch.int8, device="cuda")
    scales = torch.tensor([[127, 255], [127, 127]], dtype=torch.uint8, device="cuda")
    sr = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    dw = torch.zeros((2, 1), device="cuda")
    B.unpermute_backward8(dy, codes, scales, torch.ones((2, 1), device="cuda"), sr, None, dw)
    assert bool(torch.isnan(dw[0, 0])) and float(dw[1, 0]) == 64.0


def test_large_gradients_against_small_scales_stay_finite():
    """Products that are in range only with the block's scale applied first."""
    for d in (64, 33):
        dy = torch.full((2, d), 3e36, device="cuda")
        codes = torch.full((2, d), 100, dtype=torch.int8, device="cuda")
        scales = torch.full((2, (d + 31) // 32), 107, dtype=torch.uint8, device="cuda")      # 2^-20
        sr = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
        dw = torch.zeros((2, 1), device="cuda")
        B.unpermute_backward8(dy, codes, scales, torch.ones((2, 1), device="cuda"), sr, None, dw)
        ref = f64(dy)[0].sum() * 100 * 2.0 ** -20
        assert np.all(np.abs(f64(dw) - ref) <= (d + 2) * V * ref)


def test_non_finite_rows_go_where_their_slots_do():
    for dt in TYPES.values():
        ys = torch.ones((4, 40), dtype=dt, device="cuda")
        ys[1, 3], ys[2, 5] = float("inf"), float("nan")
        sr = torch.tensor([[0, 1], [2, -1], [3, -1]], dtype=torch.int32, device="cuda")
        w = torch.tensor([[1.0, -0.5], [2.0, float("inf")], [0.5, 0.0]], device="cuda")
        y = torch.zeros((3, 40), dtype=dt, device="cuda")
        B.unpermute(ys, w, sr, y)
        assert float(y[0, 3]) == -float("inf") and bool(torch.isnan(y[1, 5]))
        assert int(torch.isfinite(y).sum()) == 3 * 40 - 2


def test_gradients_agree_with_differences():
    """<y, dy> of unpermute(permute(x) * c) is linear in x and in the weights: its differences
    over any step are its derivatives, up to the fp32 sums' rounding."""
    T, K, N, d = 37, 4, 9, 48
    _, sr, rows, w = make(T, K, N, d, torch.float32, 500)
    x, dy = rows(T), rows(T)
    c = rows(T * K)

    def loss(x, w):
        xs, y = torch.zeros((T * K, d), device="cuda"), torch.zeros((T, d), device="cuda")
        B.permute(x, sr, xs)
        B.unpermute(xs * c, w, sr, y)
        return float((y.double() * dy.double()).sum())

    xs, dys, dx = torch.zeros((T * K, d), device="cuda"), torch.zeros((T * K, d), device="cuda"), torch.zeros_like(x)
    dw = torch.zeros((T, K), device="cuda")
    B.permute(x, sr, xs)
    B.unpermute_backward(dy, xs * c, w, sr, dys, dw)
    B.permute_backward(dys * c, sr, dx)
    rng = np.random.default_rng(501)
    size = float((dy.double().abs().sum(1)[:, None] * w.double()).sum())   # magnitude of the terms summed
    for _ in range(3):
        ex = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda()
        ew = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda()
        got = (loss(x + 0.5 * ex, w) - loss(x - 0.5 * ex, w), loss(x, w + 0.5 * ew) - loss(x, w - 0.5 * ew))
        want = (float((dx.double() * ex.double()).sum()),
                float((dw.double() * torch.where(sr >= 0, ew, 0.0).double()).sum()))
        # every quantity is O(1) normal: terms of at most 5^3 size each, K + 2 roundings of 2^-24
        for a, b in zip(got, want):
            assert abs(a - b) <= 125 * (K + 4) * V * size, (a, b)


def test_rows_past_the_buffer_are_skipped_and_recorded():
    T, K, d = 4, 2, 64
    for dt in TYPES.values():
        sr = torch.tensor([[0, 5], [1, -1], [2, 2 ** 31 - 1], [-2 ** 31, 3]], dtype=torch.int32, device="cuda")
        ok = torch.where(sr < 4, sr, -1)
        rng = np.random.default_rng(7)
        t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dt).cuda()
        x, ys, w = t(T, d), t(4, d), torch.rand((T, K), device="cuda")
        codes = torch.ones((4, d), dtype=torch.int8, device="cuda")
        scales = torch.full((4, 2), 127, dtype=torch.uint8, device="cuda")
        dw = torch.zeros((T, K), device="cuda")
        calls = [lambda s, o, ws: B.permute(x, s, o, ws), lambda s, o, ws: B.unpermute(ys, w, s, o, ws=ws),
                 lambda s, o, ws: B.permute_backward(ys, s, o, ws=ws),
                 lambda s, o, ws: B.unpermute_backward(x, ys, w, s, o, dw, ws),
                 lambda s, o, ws: B.unpermute_backward8(x, codes, scales, w, s, o, dw, ws)]
        for call in calls:
            ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
            a, b = torch.zeros((4, d), dtype=dt, device="cuda"), torch.zeros((4, d), dtype=dt, device="cuda")
            call(ok, b, ws)
            assert B.get_device_status(ws) == B.OK
            dwb = dw.clone()
            call(sr, a, ws)
            assert B.get_device_status(ws) == B.ERR_DEVICE_BOUNDS
            assert torch.equal(a, b) and torch.equal(dw, dwb)


def test_without_rows_only_the_token_side_is_written():
    """No slot has a row and the row buffers are empty, as on a rank that received nothing."""
    T, K, d = 5, 3, 96
    for dt in TYPES.values():
        none = torch.zeros((0, d), dtype=dt, device="cuda")
        sr = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
        x = torch.randn((T, d), device="cuda").to(dt)
        w, dw = torch.full((T, K), float("nan"), device="cuda"), torch.full((T, K), 7.0, device="cuda")
        y = torch.full_like(x, 9.0)
        B.permute(x, sr, none)
        B.unpermute(none, w, sr, y, base=x)
        assert torch.equal(y, x)
        B.permute_backward(none, sr, y)
        assert not bool(y.any())
        B.unpermute_backward(x, none, w, sr, none, dw)
        assert not bool(dw.any())
        codes, scales = none.to(torch.int8), torch.zeros((0, 3), dtype=torch.uint8, device="cuda")
        dw.fill_(7.0)
        B.unpermute_backward8(x, codes, scales, w, sr, None, dw)
        assert not bool(dw.any())
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        sr[2, 1] = 0                                       # a row that does not exist
        B.permute(x, sr, none, ws)
        assert B.get_device_status(ws) == B.ERR_DEVICE_BOUNDS


def test_a_stream_passed_to_the_call():
    T, K, N, d = 900, 4, 20, 128
    rng = np.random.default_rng(21)
    side = torch.cuda.Stream()
    ids = draw_ids(rng, T, K, N, 0.3)
    x = torch.randn((T, d), device="cuda").to(torch.bfloat16)
    w = torch.rand((T, K), device="cuda")
    o = run_sort(ids, N)
    want = torch.zeros((T * K, d), dtype=torch.bfloat16, device="cuda")
    y_want = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    B.permute(x, o["slot_row"], want)
    B.unpermute(want, w, o["slot_row"], y_want)
    ws = torch.empty(B.sort_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    got = {n: torch.empty_like(v) for n, v in o.items()}
    xs, y = torch.zeros_like(want), torch.zeros_like(y_want)
    torch.cuda.synchronize()
    B.sort_slots(ids, N, got["counts"], got["offsets"], got["perm_tok"], got["slot_row"], ws, side)
    B.permute(x, got["slot_row"], xs, ws, side)
    B.unpermute(xs, w, got["slot_row"], y, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(got["slot_row"], o["slot_row"]) and torch.equal(xs, want) and torch.equal(y, y_want)


@pytest.mark.parametrize("T,K,N", [(40, 4, 1024), (3000, 8, 1024), (20000, 8, 700)])
def test_captured_sorts_of_many_experts(T, K, N):
    """The sort's larger shared memory and its two launches under capture, on changing ids."""
    rng = np.random.default_rng(T)
    ids = draw_ids(rng, T, K, N, 0.2)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    o = dict(counts=z(N), offsets=z(N + 1), perm=z(T * K), row=z(T, K))
    ws = torch.empty(B.sort_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        B.sort_slots(ids, N, o["counts"], o["offsets"], o["perm"], o["row"], ws)
    for _ in range(4):
        ids.copy_(draw_ids(rng, T, K, N, 0.2))
        g.replay()
        counts, offsets, perm, row = sort_ref(ids.cpu().numpy(), N)
        assert np.array_equal(o["row"].cpu().numpy(), row) and np.array_equal(o["offsets"].cpu().numpy(), offsets)
        assert np.array_equal(o["perm"][:int(offsets[-1])].cpu().numpy(), perm)


def test_rows_beyond_32_bit_offsets():
    """Rows whose element offset passes 2^32 in a long buffer."""
    rows, d, T = 2 ** 21 + 40, 2080, 8
    buf = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((T, d), device="cuda").to(torch.bfloat16)
    at = torch.arange(T, device="cuda", dtype=torch.int32) * 5
    sr = torch.stack([at, rows - 1 - at], 1).contiguous()
    assert (rows - 40) * d > 2 ** 32
    B.permute(x, sr, buf)
    assert torch.equal(buf[sr[:, 1].long()], x) and torch.equal(buf[sr[:, 0].long()], x)
    y = torch.zeros_like(x)
    w = torch.tensor([[0.0, 1.0]], device="cuda").repeat(T, 1)
    B.unpermute(buf, w, sr, y)
    assert torch.equal(y, x)
    dw = torch.zeros((T, 2), device="cuda")
    B.unpermute_backward(x, buf, w, sr, None, dw)
    assert torch.equal(dw[:, 0], dw[:, 1])


def test_other_streams_captured_graphs_and_a_shared_workspace():
    """Sort, permute and unpermute on a side stream, then captured twice over one workspace and
    replayed in turn on new contents: each replay equals the eager calls on those contents."""
    T, K, N, d = 700, 4, 16, 192
    rng = np.random.default_rng(11)
    ws = torch.empty(B.sort_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")

    def state():
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
        return dict(ids=z(T, K), counts=z(N), offsets=z(N + 1), perm=z(T * K), sr=z(T, K),
                    x=z(T, d, dt=torch.bfloat16), xs=z(T * K, d, dt=torch.bfloat16), y=z(T, d, dt=torch.bfloat16),
                    w=z(T, K, dt=torch.float32))

    def step(s):
        B.sort_slots(s["ids"], N, s["counts"], s["offsets"], s["perm"], s["sr"], ws)
        B.permute(s["x"], s["sr"], s["xs"], ws)
        B.unpermute(s["xs"], s["w"], s["sr"], s["y"], ws=ws)

    def refill(s):
        s["ids"].copy_(draw_ids(rng, T, K, N, 0.5))
        s["x"].copy_(torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)))
        s["w"].copy_(torch.from_numpy(rng.random((T, K)).astype(np.float32)))

    a, b = state(), state()
    side = torch.cuda.Stream()
    refill(a)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
    torch.cuda.current_stream().wait_stream(side)
    on_side = a["y"].clone()
    step(a)
    assert torch.equal(on_side, a["y"])
    graphs = []
    for s in (a, b):
        refill(s)
        step(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    for _ in range(3):
        refill(a)
        refill(b)
        for g in graphs:
            g.replay()
        got = [s["y"].clone() for s in (a, b)]
        for s, y in zip((a, b), got):
            step(s)
            assert torch.equal(y, s["y"])
            check_collect(y, *collect_ref(s["xs"], s["sr"], s["w"], None), K)
    torch.cuda.synchronize()
    assert B.get_device_status(ws) == B.OK


# ------------------------------------------------------------- the layer on a given routing

from token_choice_routing_b200 import inputs as I  # noqa: E402

ROUTED = {
    "ragged": I.small_config("routed_ragged", T=300, d=256, N=12, F=192, F_shared=128, K=3, M=4, config_id=961),
    "wide": I.small_config("routed_wide", T=700, d=512, N=6, F=256, F_shared=384, K=2, M=2, config_id=962),
    "t1": I.small_config("routed_t1", T=1, d=128, N=8, F=64, F_shared=64, K=4, M=8, config_id=963),
}


@pytest.mark.parametrize("name", sorted(ROUTED))
@pytest.mark.parametrize("wide_ids", [False, True])
def test_replayed_routing_is_bitwise_the_layer_forward(name, wide_ids):
    from tests import gpu_helpers as H
    cfg = ROUTED[name]
    layer, x, _, out = H.run_forward(I.make_inputs(cfg))
    idx = out["topk_idx"].long() if wide_ids else out["topk_idx"]
    o = layer.forward_routed(x, idx, out["topk_gate"])
    torch.cuda.synchronize()
    assert B.get_device_status(o["workspace"]) == B.OK
    for n in ("offsets", "slot_row", "y"):
        assert torch.equal(o[n], out[n]), n


@pytest.mark.parametrize("name", sorted(ROUTED))
def test_routed_step_against_the_oracle(name):
    """Forward and backward on a routing that no router of the layer made: repeated experts,
    padding, gates that do not sum to one, another K than the layer's."""
    import oracle as O
    from tests import gpu_helpers as H
    cfg = ROUTED[name]
    inp = I.make_inputs(cfg)
    layer, x, _ = H.make_layer(inp)
    rng = np.random.default_rng(cfg.config_id)
    T, K, N = cfg.T, 5, cfg.N
    ids = draw_ids(rng, T, K, N, 0.4)
    gate = torch.from_numpy(rng.uniform(-1, 1, (T, K)).astype(np.float32)).cuda()
    dy = torch.from_numpy(rng.standard_normal((T, cfg.d)).astype(np.float32)).to(torch.bfloat16).cuda()
    out = layer.forward_routed(x, ids, gate)
    g = layer.backward_routed(x, gate, out, dy)
    torch.cuda.synchronize()
    assert B.get_device_status(out["workspace"]) == B.OK and B.get_device_status(g["workspace"]) == B.OK
    ex, sh = H.expert_weights(inp)
    xf, dyf, idn = H.f64(inp.x), f64(dy), ids.cpu().numpy()
    has = (idn >= 0) & (idn < N)
    gn = np.where(has, f64(gate), 0.0)
    y_ref = O.swiglu(xf, *sh)
    for k in range(K):     # slot by slot: the oracle's layer output takes a token's experts as distinct
        for e in range(N):
            t = np.nonzero(idn[:, k] == e)[0]
            if t.size:
                y_ref[t] += gn[t, k][:, None] * O.swiglu(xf[t], *(w[e] for w in ex))
    H.check_y(f64(out["y"]), y_ref)

    def ffn_backward(xr, wg, wu, wd, up):
        a, b = xr @ wg.T, xr @ wu.T
        s = 1 / (1 + np.exp(-a))
        dh = up @ wd
        da, db = dh * b * (s + a * s * (1 - s)), dh * a * s
        return da @ wg + db @ wu, da.T @ xr, db.T @ xr, up.T @ (a * s * b), (a * s * b) @ wd.T

    dx, dsg, dsu, dsd, _ = ffn_backward(xf, *sh, dyf)
    dgate, size = np.zeros((T, K)), np.zeros((T, K))
    dwg, dwu, dwd = (np.zeros_like(w) for w in ex)
    for t, k in zip(*np.nonzero(has)):
        e = idn[t, k]
        dxi, g0, g1, g2, o = ffn_backward(xf[t:t + 1], *(w[e] for w in ex), gn[t, k] * dyf[t:t + 1])
        dx[t] += dxi[0]
        dwg[e] += g0
        dwu[e] += g1
        dwd[e] += g2
        dgate[t, k] = dyf[t] @ o[0]
        size[t, k] = np.linalg.norm(dyf[t]) * np.linalg.norm(o[0])
    # the layer's backward tolerances: bf16 activations and weight gradients, fp32 sums
    for n, ref in (("dx", dx), ("dw_gate", dwg), ("dw_up", dwu), ("dw_down", dwd),
                   ("dws_gate", dsg), ("dws_up", dsu), ("dws_down", dsd)):
        err = np.linalg.norm(f64(g[n]) - ref)
        assert err <= 1e-2 * np.linalg.norm(ref), (n, err / np.linalg.norm(ref))
    # <dy, o> may cancel to any smaller value: with o off by at most 1e-2 in norm, as y is,
    # the product is off by at most 1e-2 |dy| |o| (Cauchy-Schwarz)
    assert np.all(np.abs(f64(g["dgate"]) - dgate) <= 1e-2 * size)


def test_routed_refusals_and_no_tokens():
    from tests import gpu_helpers as H
    cfg = ROUTED["ragged"]
    layer, x, _ = H.make_layer(I.make_inputs(cfg))
    T = cfg.T
    ids, gate = torch.zeros((T, 2), dtype=torch.int32, device="cuda"), torch.ones((T, 2), device="cuda")
    with pytest.raises(ValueError):
        layer.forward_routed(x[:-1], ids, gate)
    with pytest.raises(ValueError):
        layer.forward_routed(x.float(), ids, gate)
    with pytest.raises(ValueError):
        layer.forward_routed(x, ids, gate, layer.alloc_routed(T, 3))
    with pytest.raises(B.MoEError):
        layer.forward_routed(x, ids.repeat(1, 10), gate.repeat(1, 10))
    empty = layer.forward_routed(x[:0], ids[:0], gate[:0])
    torch.cuda.synchronize()
    assert int(empty["offsets"][-1]) == 0
    pp = I.small_config("routed_pp", T=8, d=128, N=4, F=64, F_shared=64, K=3, M=2, C=1, V=1, config_id=964)
    layer, x, _ = H.make_layer(I.make_inputs(pp))
    with pytest.raises(ValueError):
        layer.forward_routed(x, ids[:8], gate[:8])


def test_results_of_a_passed_stream_outlive_their_scratch():
    """Only y (and the gradients) of a call on a stream that has other work to do first are kept; the
    current stream then takes and overwrites memory of the sizes that were dropped. With zeros:
    a wrong index would be a valid one."""
    from tests import gpu_helpers as H
    cfg = ROUTED["wide"]
    layer, x, _ = H.make_layer(I.make_inputs(cfg))
    ids = draw_ids(np.random.default_rng(3), cfg.T, 3, cfg.N, 0.3)
    gate = torch.rand((cfg.T, 3), device="cuda")
    dy = torch.randn((cfg.T, cfg.d), device="cuda").to(torch.bfloat16)
    out = layer.forward_routed(x, ids, gate)
    want = dict(y=out["y"].clone(), own=layer.forward(x)["y"].clone())
    want.update((n, t.clone()) for n, t in layer.backward_routed(x, gate, out, dy).items() if n.startswith("dw"))
    busy = torch.ones((8192, 8192), device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()

    def crowd():
        for sizes in (layer.alloc_routed(cfg.T, 3), layer.alloc_routed_grads(cfg.T, 3), layer.alloc(cfg.T)):
            for t in sizes.values():
                if t is not None:
                    t.zero_()

    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(20):
                busy @ busy
        got = dict(y=layer.forward_routed(x, ids, gate, stream=side)["y"], own=layer.forward(x, stream=side)["y"])
        crowd()
        g = layer.backward_routed(x, gate, out, dy, stream=side)
        got.update((n, g[n]) for n in want if n.startswith("dw"))
        del g
        crowd()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for n, t in want.items():
            assert torch.equal(got[n], t), n


def test_a_routed_backward_without_tokens_gives_zero_gradients():
    """A rank without tokens adds zeros to the others' weight gradients, whatever the buffers held."""
    from tests import gpu_helpers as H
    cfg = ROUTED["ragged"]
    layer, x, _ = H.make_layer(I.make_inputs(cfg))
    gate = torch.ones((0, 2), device="cuda")
    out = layer.forward_routed(x[:0], torch.zeros((0, 2), dtype=torch.int32, device="cuda"), gate)
    grads = layer.alloc_routed_grads(0, 2)
    names = [n for n in B.GRAD_FIELDS if n in grads and n != "dx"]
    for stream in (None, torch.cuda.Stream()):
        for n in names:
            grads[n].fill_(float("nan"))
        torch.cuda.synchronize()
        g = layer.backward_routed(x[:0], gate, out, x[:0], grads, stream=stream)
        torch.cuda.synchronize()
        for n in names:
            assert int(torch.count_nonzero(g[n])) == 0, n
    assert sorted(names) == ["dw_down", "dw_gate", "dw_up", "dws_down", "dws_gate", "dws_up"]


def test_sorts_of_two_threads():
    """Two host threads, whose calls need different amounts of shared memory of the same kernel."""
    import threading
    T, K = 1024, 4
    failed = []

    def work(N):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                ids = draw_ids(np.random.default_rng(N), T, K, N, 0.2)
                counts, offsets, _, row = sort_ref(ids.cpu().numpy(), N)
                z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
                o = (z(N), z(N + 1), z(T * K), z(T, K))
                ws = torch.empty(B.sort_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
                for _ in range(8):
                    o[3].zero_()
                    for _ in range(1000):
                        B.sort_slots(ids, N, *o, ws)
                    assert np.array_equal(o[0].cpu().numpy(), counts) and np.array_equal(o[1].cpu().numpy(), offsets)
                    assert np.array_equal(o[3].cpu().numpy(), row)
        except Exception as e:  # noqa: BLE001  (the main thread reports it)
            failed.append((N, repr(e)))

    threads = [threading.Thread(target=work, args=(N,)) for N in (700, 1024)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_more_pieces_than_an_index_holds():
    """Narrow rows whose tokens times pieces pass 2^31: a piece is one element here."""
    d, T = 63, 2 ** 31 // 63 + 1000
    sr = torch.randperm(T, device="cuda").to(torch.int32).view(T, 1)
    sr[::3] = -1
    ys = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.rand((T, 1), device="cuda") + 0.5
    y = torch.full((T, d), 9.0, dtype=torch.bfloat16, device="cuda")

    def check(at, out, src, weight):      # one product and one rounding: the same in any order
        for a in range(0, T, 2 ** 22):
            s, o = at[a:a + 2 ** 22, 0].long(), out[a:a + 2 ** 22]
            has = (s >= 0)[:, None]
            ref = src[s.clamp(min=0)].float() * weight[a:a + 2 ** 22]
            assert torch.equal(o, torch.where(has, ref, 0.0).to(torch.bfloat16)), a

    B.unpermute(ys, w, sr, y)
    check(sr, y, ys, w)
    ones = torch.ones_like(w)
    B.permute_backward(ys, sr, y)
    check(sr, y, ys, ones)
    del y
    # the copies, 31 single elements a row
    d, T = 31, 2 ** 31 // 31 + 1000
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").normal_()
    sr = torch.randperm(T, device="cuda").to(torch.int32).view(T, 1)
    back = torch.empty_like(sr)
    back[sr[:, 0].long(), 0] = torch.arange(T, dtype=torch.int32, device="cuda")
    del ys
    xs = torch.zeros_like(x)
    w, ones = torch.rand((T, 1), device="cuda") + 0.5, torch.ones((T, 1), device="cuda")
    B.permute(x, sr, xs)
    check(back, xs, x, ones)
    B.unpermute_backward(x, None, w, sr, xs, None)
    check(back, xs, x, w[back[:, 0].long()])


@pytest.mark.parametrize("T,K,N", [(262500, 8, 64), (150001, 16, 700)])
def test_sort_of_several_passes_with_many_slots_in_the_last(T, K, N):
    """Chunks of more slots than a CTA holds at once, the last pass with several a thread."""
    check_sort(draw_ids(np.random.default_rng(T), T, K, N, 0.3), N)
