"""Activations stored in 8 bits and the backward passes that read them, against 64-bit forms.

Tolerances, with u = eps / 2 of the output's type: stored and restored values are exact.
swiglu_backward8 computes in fp32 from exact inputs: CUDA's expf is within 2 ulp, so
s = 1 / (1 + exp(-a)) is within 2^-21 relative (2 ulp of the exponential, two roundings) where
it does not underflow, and products of up to four factors add 2^-22. The bracket
1 + a (1 - s) has an absolute error of at most |a| 2^-24 (1 - s is rounded at 2^-24 of one, and
is exactly zero with s = 1 once exp(-a) < 2^-24, that is a > 17) + 2^-21 (1 + |a (1 - s)|): at
most 2^-19 + 2^-21 |a (1 - s)|. Then
  |da err| <= |dh b s| 2^-18 + |dh b s a (1 - s)| 2^-19 + u |da| + f,   |db err| <= (2^-20 + u) |db| + f
and h as db, with f = 2^-120 times the magnitudes plus the smallest subnormal for s below fp32's range.
"""
import numpy as np
import pytest
import torch

from token_choice_routing_b200 import binding as B
from token_choice_routing_b200 import inputs as I
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def tiny(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


def stored_ref(x):
    """Values and scale bytes of the blocks of x (float64, exact), by the definition."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    val, byte = np.empty_like(x), np.empty((rows, nb), dtype=np.int64)
    for j in range(nb):
        blk = x[:, 32 * j:32 * j + 32]
        m = np.abs(blk).max(axis=1)
        fin = np.isfinite(m)
        E = np.full(rows, -126, dtype=np.int64)
        pos = fin & (m > 0)
        E[pos] = np.maximum(np.floor(np.log2(m[pos])).astype(np.int64) - 6, -126)
        step = 2.0 ** E.astype(np.float64)
        with np.errstate(invalid="ignore"):
            q = np.clip(np.rint(blk / step[:, None]), -127, 127)
        val[:, 32 * j:32 * j + 32] = np.where(fin[:, None], q * step[:, None], np.nan)
        byte[:, j] = np.where(fin, E + 127, 255)
    return val, byte


def spaced(rng, rows, cols, dt, pad=0, lead=0, fill=None):
    flat = rng.standard_normal(rows * (cols + pad) + lead) if fill is None else np.full(rows * (cols + pad) + lead, fill)
    return torch.from_numpy(flat.astype(np.float32)).to(dt).cuda()[lead:].view(rows, cols + pad)[:, :cols]


SHAPES = [(1, 1), (1, 32), (3, 7), (5, 33), (64, 64), (17, 96), (33, 1001), (300, 1024), (128, 1536), (2, 8200)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_store_and_restore(rows, cols, dtype):
    dt = TYPES[dtype]
    for i, (pad, lead) in enumerate([(0, 0), (8, 0), (5, 0), (0, 1), (16, 16)]):
        rng = np.random.default_rng(rows * 1000 + cols + i)
        x = spaced(rng, rows, cols, dt, pad, lead)
        x *= torch.from_numpy(np.exp2(rng.integers(-9, 4, (rows, 1))).astype(np.float32)).to(dt).cuda()
        x[rng.integers(0, rows)] = 0.0
        codes = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
        scales = torch.full((rows, B.checkpoint8_scales(cols)), 77, dtype=torch.uint8, device="cuda")
        B.checkpoint8(x, codes, scales)
        val, byte = stored_ref(f64(x))
        assert np.array_equal(scales.cpu().numpy(), byte)
        got = f64(codes) * np.repeat(2.0 ** (byte - 127.0), 32, axis=1)[:, :cols]
        assert np.array_equal(got, val)
        back = spaced(rng, rows, cols, dt, pad, lead, fill=4.0)
        B.restore8(codes, scales, back)
        assert np.array_equal(f64(back), val)
        if lead or pad:                       # what lies between the rows stays as it was
            whole = back.as_strided((rows, cols + pad), (cols + pad, 1), back.storage_offset())
            assert bool((whole[:-1, cols:] == 4.0).all())


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("cols", [64, 45])
def test_extreme_values_and_borders(dtype, cols):
    """Zeros, the type's smallest and largest values, every mantissa around the clamp and the
    ties of rint, infinities and NaN."""
    dt = TYPES[dtype]
    fin = torch.finfo(dt)
    rng = np.random.default_rng(5)
    rows = []
    for top in (0.0, tiny(dt), fin.smallest_normal, fin.max, fin.max / 2, 1.0, 127.5, 2.0 - float(fin.eps)):
        r = rng.uniform(-1, 1, cols) * top
        r[3] = top
        rows.append(r)
    rows.append((np.arange(cols) - cols / 2 + 0.5) * (64.0 / cols))     # halves around a top of 32: ties
    ties = (np.arange(cols) % 64) + 0.5
    ties[0] = 127.5
    rows.append(ties)
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = rng.uniform(-1, 1, cols)
        r[cols - 1] = bad
        rows.append(r)
    x = torch.from_numpy(np.array(rows)).to(dt).cuda()
    codes = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    scales = torch.empty((len(rows), B.checkpoint8_scales(cols)), dtype=torch.uint8, device="cuda")
    back = torch.empty_like(x)
    B.checkpoint8(x, codes, scales)
    B.restore8(codes, scales, back)
    val, byte = stored_ref(f64(x))
    assert np.array_equal(scales.cpu().numpy(), byte)
    np.testing.assert_array_equal(f64(back), val)           # NaN where the definition says so
    assert int(codes.min()) >= -127
    fine = np.isfinite(val)
    step = np.repeat(2.0 ** (byte - 127.0), 32, axis=1)[:, :cols]
    lim = 0.5 if dt == torch.bfloat16 else 1.0
    assert np.all(np.abs(val - f64(x))[fine] <= lim * step[fine])


@pytest.mark.parametrize("cols", [45, 72, 96])
def test_rows_in_use(cols):
    rows = 40
    rng = np.random.default_rng(6)
    for dt in TYPES.values():
        x = spaced(rng, rows, cols, dt)
        x[30:] = float("nan")                                # not read
        for used in (0, 1, 30):
            n = torch.tensor([used], dtype=torch.int32, device="cuda")
            codes = torch.full((rows, cols), 5, dtype=torch.int8, device="cuda")
            nb = B.checkpoint8_scales(cols)
            scales = torch.full((rows, nb), 7, dtype=torch.uint8, device="cuda")
            ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
            B.checkpoint8(x, codes, scales, n, ws)
            val, byte = stored_ref(f64(x[:used])) if used else (np.empty((0, cols)), np.empty((0, nb)))
            assert np.array_equal(scales[:used].cpu().numpy(), byte)
            assert bool((codes[used:] == 5).all()) and bool((scales[used:] == 7).all())
            back = torch.full((rows, cols), 2.0, dtype=dt, device="cuda")
            B.restore8(codes, scales, back, n, ws)
            assert np.array_equal(f64(back[:used]), val) and bool((back[used:] == 2.0).all())
            assert B.get_device_status(ws) == B.OK


def test_restored_in_another_type_than_stored():
    """Values have at most 7 significant bits: exact in every type whose range they lie in."""
    rng = np.random.default_rng(9)
    for src in TYPES.values():
        for cols in (64, 40, 33):
            x = spaced(rng, 30, cols, src)
            codes = torch.empty((30, cols), dtype=torch.int8, device="cuda")
            scales = torch.empty((30, B.checkpoint8_scales(cols)), dtype=torch.uint8, device="cuda")
            B.checkpoint8(x, codes, scales)
            for dst in TYPES.values():
                back = torch.empty((30, cols), dtype=dst, device="cuda")
                B.restore8(codes, scales, back)
                assert np.array_equal(f64(back), stored_ref(f64(x))[0])


def test_rows_in_use_outside_the_buffer_are_clamped_and_recorded():
    rows, F = 6, 64
    x = torch.ones((rows, 2 * F), dtype=torch.bfloat16, device="cuda")
    for used, written in ((rows + 1, rows), (-1, 0), (2 ** 31 - 1, rows), (-2 ** 31, 0)):
        n = torch.tensor([used], dtype=torch.int32, device="cuda")
        codes = torch.zeros((rows, 2 * F), dtype=torch.int8, device="cuda")
        scales = torch.zeros((rows, 4), dtype=torch.uint8, device="cuda")
        back, dz = torch.zeros_like(x), torch.full_like(x, 3.0)
        h = torch.full((rows, F), 3.0, dtype=torch.bfloat16, device="cuda")
        for call in (lambda ws: B.checkpoint8(x, codes, scales, n, ws), lambda ws: B.restore8(codes, scales, back, n, ws),
                     lambda ws: B.swiglu_backward8(codes, scales, x[:, :F], dz, h, rows_used=n, ws=ws)):
            ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
            call(ws)
            assert B.get_device_status(ws) == B.ERR_DEVICE_BOUNDS
        assert int((back == 1.0).all(dim=1).sum()) == written and int((h != 3.0).all(dim=1).sum()) == written


def swiglu_ref(val, dh, packed):
    F = dh.shape[1]
    j = np.arange(F)
    ca = j // 64 * 128 + j % 64 if packed else j
    cb = ca + 64 if packed else j + F
    a, b = val[:, ca], val[:, cb]
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-a))
    q = 1 / (1 + np.exp(np.minimum(a, 700)))                  # 1 - s without cancellation
    da = dh * b * s * (1 + a * q)
    db = dh * a * s
    return ca, cb, a, b, s, q, da, db, a * s * b


def check_swiglu(codes, scales, dh, dz, h, packed):
    dt = dh.dtype
    u = torch.finfo(dt).eps / 2
    val = f64(codes) * np.repeat(2.0 ** (f64(scales) - 127.0), 32, axis=1)[:, :codes.shape[1]]
    g = f64(dh)
    ca, cb, a, b, s, q, da, db, href = swiglu_ref(val, g, packed)
    floor = 2.0 ** -120 * (1 + np.abs(a)) * (1 + np.abs(b)) * (1 + np.abs(g)) + tiny(dt)
    z = f64(dz)
    for got, ref, extra in ((z[:, ca], da, np.abs(g * b * s) * 2.0 ** -18 + np.abs(g * b * s * a * q) * 2.0 ** -19),
                            (z[:, cb], db, np.abs(db) * 2.0 ** -20), (f64(h), href, np.abs(href) * 2.0 ** -20)):
        top = np.abs(ref) >= float(torch.finfo(dt).max) * (1 - u)      # past the type: infinite either way
        err = np.abs(np.where(top, 0, got) - np.where(top, 0, ref))
        bound = extra + u * np.abs(ref) + floor
        assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("rows,F,packed", [(1, 64, True), (1, 1, False), (3, 37, False), (65, 128, True), (40, 512, False),
                                           (129, 768, True), (7, 1000, False), (513, 499, False), (300, 64, False),
                                           (20, 48, False)])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_swiglu_backward8(rows, F, packed, dtype):
    dt = TYPES[dtype]
    for i, (pad, lead) in enumerate([(0, 0), (8, 0), (3, 1)]):
        rng = np.random.default_rng(rows + 7 * F + i)
        codes = torch.from_numpy(rng.integers(-127, 128, size=(rows, 2 * F)).astype(np.int8)).cuda()
        # pre-activations from 2^-20 to about 100
        scales = torch.from_numpy(rng.integers(107, 128, size=(rows, (2 * F + 31) // 32)).astype(np.uint8)).cuda()
        dh = spaced(rng, rows, F, dt, pad, lead)
        dz, h = spaced(rng, rows, 2 * F, dt, pad, lead, fill=9.0), spaced(rng, rows, F, dt, pad, lead, fill=9.0)
        B.swiglu_backward8(codes, scales, dh, dz, h, packed=packed)
        check_swiglu(codes, scales, dh, dz, h, packed)
        dz2 = torch.empty((rows, 2 * F), dtype=dt, device="cuda")
        B.swiglu_backward8(codes, scales, dh, dz2, None, packed=packed)       # without h
        assert torch.equal(dz2, dz)
        used = rows // 2
        n = torch.tensor([used], dtype=torch.int32, device="cuda")
        dz3, h3 = spaced(rng, rows, 2 * F, dt, pad, lead, fill=9.0), spaced(rng, rows, F, dt, pad, lead, fill=9.0)
        B.swiglu_backward8(codes, scales, dh, dz3, h3, packed=packed, rows_used=n)
        assert torch.equal(dz3[:used], dz[:used]) and torch.equal(h3[:used], h[:used])
        assert bool((dz3[used:] == 9.0).all()) and bool((h3[used:] == 9.0).all())


def test_swiglu_backward8_extremes():
    """Saturated gates, zeros, and a block stored as NaN, which only its own columns see."""
    F = 64
    codes = torch.zeros((4, 2 * F), dtype=torch.int8, device="cuda")
    scales = torch.full((4, 4), 127, dtype=torch.uint8, device="cuda")
    codes[0, :F], codes[1, :F] = 127, -127                    # sigma(127) = 1, sigma(-127) ~ 7e-56
    codes[:, F:] = 3
    scales[2, 1] = 255                                        # gate columns 32..63 of row 2
    dh = torch.ones((4, F), dtype=torch.float32, device="cuda")
    dz, h = torch.empty((4, 2 * F), device="cuda"), torch.empty((4, F), device="cuda")
    B.swiglu_backward8(codes, scales, dh, dz, h)
    assert bool((dz[0, :F] == 3.0).all()) and bool((dz[0, F:] == 127.0).all()) and bool((h[0] == 381.0).all())
    assert float(dz[1].abs().max()) < 1e-30 and float(h[1].abs().max()) < 1e-30
    nan = torch.isnan(dz[2])
    assert bool(nan[32:64].all()) and bool(nan[96:].all()) and int(nan.sum()) == 64
    assert bool((dz[3, :F] == 1.5).all()) and bool((dz[3, F:] == 0.0).all())


@pytest.mark.parametrize("packed,F", [(True, 64), (False, 37)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_swiglu_backward8_large_products(dtype, packed, F):
    """dh b passes fp32's range while a closed gate keeps the gradient finite."""
    a = [-20, -60, -87, -100, -127, 0]
    codes = torch.empty((len(a), 2 * F), dtype=torch.int8, device="cuda")
    codes[:, :F] = torch.tensor(a, dtype=torch.int8, device="cuda")[:, None]
    codes[:, F:] = 100
    scales = torch.full((len(a), (2 * F + 31) // 32), 127, dtype=torch.uint8, device="cuda")
    # up: 100 x 2^60; with 37 gate columns the block they share with the up columns keeps scale 1
    scales[:, (F + 31) // 32:] = 187
    dh = torch.full((len(a), F), 1e20, dtype=TYPES[dtype], device="cuda")
    dh[-1] = 1.0
    dz, h = torch.empty((len(a), 2 * F), dtype=TYPES[dtype], device="cuda"), torch.empty_like(dh)
    B.swiglu_backward8(codes, scales, dh, dz, h, packed=packed)
    assert bool(torch.isfinite(dz).all()) and bool(torch.isfinite(h).all())
    check_swiglu(codes, scales, dh, dz, h, packed)


def test_swiglu_backward8_agrees_with_differences():
    """dz against central differences of sum(h dh), h = silu(a) b, in 64 bits at the stored values."""
    rows, F, eps = 9, 96, 1e-4
    rng = np.random.default_rng(8)
    codes = torch.from_numpy(rng.integers(-127, 128, size=(rows, 2 * F)).astype(np.int8)).cuda()
    scales = torch.full((rows, 6), 122, dtype=torch.uint8, device="cuda")
    dh = torch.randn((rows, F), device="cuda")
    dz, h = torch.empty((rows, 2 * F), device="cuda"), torch.empty((rows, F), device="cuda")
    B.swiglu_backward8(codes, scales, dh, dz, h, packed=False)
    z, g = f64(codes) * 2.0 ** -5, f64(dh)
    silu = lambda a: a / (1 + np.exp(-a))
    a, b = z[:, :F], z[:, F:]
    da = g * b * (silu(a + eps) - silu(a - eps)) / (2 * eps)     # error: eps^2 |silu'''| / 6 < 1e-8 |g b|
    db = g * silu(a)
    size = np.abs(g) * (1 + np.abs(a)) * (1 + np.abs(b))
    assert np.all(np.abs(f64(dz)[:, :F] - da) <= 1e-5 * size) and np.all(np.abs(f64(dz)[:, F:] - db) <= 1e-5 * size)


def test_elements_beyond_32_bit_offsets():
    rows, cols = 2 ** 21 + 3, 2080
    assert (rows - 3) * cols > 2 ** 32
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").fill_(1.0)
    x[-3:] = torch.randn((3, cols), device="cuda").to(torch.bfloat16)
    codes = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    scales = torch.empty((rows, 65), dtype=torch.uint8, device="cuda")
    B.checkpoint8(x, codes, scales)
    val, byte = stored_ref(f64(x[-3:]))
    x.zero_()
    B.restore8(codes, scales, x)
    assert np.array_equal(scales[-3:].cpu().numpy(), byte) and np.array_equal(f64(x[-3:]), val)
    assert bool((x[:-3] == 1.0).all())
    F = cols // 2
    dh = torch.ones((rows, F), dtype=torch.bfloat16, device="cuda")
    dz, h = x, torch.empty((rows, F), dtype=torch.bfloat16, device="cuda")
    B.swiglu_backward8(codes, scales, dh, dz, h, packed=False)
    check_swiglu(codes[-3:], scales[-3:], dh[-3:], dz[-3:], h[-3:], False)


# ------------------------------------------------------------------ the layer's training step

CASES = {
    "tiny": I.CONFIGS["tiny"],
    "ragged": I.small_config("ckpt_ragged", T=300, d=256, N=12, F=192, F_shared=128, K=3, M=4, config_id=970),
    "wide": I.small_config("ckpt_wide", T=700, d=512, N=6, F=256, F_shared=384, K=2, M=2, config_id=971),
    "t1": I.small_config("ckpt_t1", T=1, d=128, N=8, F=64, F_shared=64, K=4, M=8, config_id=972),
    "pp": I.small_config("ckpt_pp", T=300, d=256, N=8, F=128, F_shared=128, K=4, M=4, C=2, V=2, config_id=973),
}
ALPHA, BETA = 2e-2, 1e-3


def layer_step(cfg):
    from token_choice_routing_b200.layer import bf16_tensor
    inp = I.make_inputs(cfg)
    layer, x, tnb = H.make_layer(inp)
    dy = bf16_tensor(I.upstream_grad(cfg), "cuda")
    out = layer.alloc(cfg.T)
    ck = layer.alloc_checkpoint8(cfg.T)
    o = layer.forward_checkpoint8(x, tnb, out, ck)
    return layer, x, tnb, dy, out, ck, o


def rel(a, b):
    n = np.linalg.norm(b)
    return np.linalg.norm(a - b) / (n if n > 0 else 1.0)


@pytest.mark.parametrize("name", sorted(CASES))
def test_training_step_from_an_8_bit_checkpoint(name):
    """The backward from the checkpoint against moe_backward on the restored activations (the
    same formulas, so only bf16 roundings that fall the other way: 5e-3 in norm, a third of the
    layer's own tolerance), and against moe_backward on the exact ones. Storing rounds by at
    most m / 128 of a block's largest magnitude m (about 2.2 sigma over 32 normal values), that
    is by at most 2.2 / 64 / sqrt(12) = 1% of sigma in the mean square; the products of two
    stored factors and the derivative of silu take that at most twice, next to the layer's
    own 1e-2: 3e-2 in norm."""
    cfg = CASES[name]
    layer, x, tnb, dy, out, ck, o = layer_step(cfg)
    torch.cuda.synchronize()
    assert B.get_device_status(o["workspace"]) == B.OK
    plain = layer.forward(x, tnb, layer.alloc(cfg.T, save_preact=True))
    assert torch.equal(o["y"], plain["y"])
    exact = layer.backward(x, plain, dy, ALPHA, BETA)
    near = dict(plain)
    near["z"], near["z_shared"], near["ys"], near["h"], near["h_shared"] = (
        plain[n].clone() for n in ("z", "z_shared", "ys", "h", "h_shared"))
    B.restore8(ck["z_codes"], ck["z_scales"], near["z"], ck["offsets"][cfg.N:])
    B.restore8(ck["zs_codes"], ck["zs_scales"], near["z_shared"])
    B.restore8(ck["ys_codes"], ck["ys_scales"], near["ys"], ck["offsets"][cfg.N:])
    for z, h, F in ((near["z"], near["h"], cfg.F), (near["z_shared"], near["h_shared"], cfg.F_shared)):
        p = z.float().view(-1, F // 64, 2, 64)
        h.copy_((p[:, :, 0] * torch.sigmoid(p[:, :, 0]) * p[:, :, 1]).reshape(-1, F))
    want = layer.backward(x, near, dy, ALPHA, BETA)
    out["ys"].fill_(float("nan"))                      # scratch: another layer's forward has it now
    out["h_shared"].fill_(float("nan"))
    out["xs"].fill_(float("nan"))
    out["h"].fill_(float("nan"))
    got = layer.backward_checkpoint8(x, ck, dy, ALPHA, BETA)
    torch.cuda.synchronize()
    assert B.get_device_status(got["workspace"]) == B.OK
    for n in B.GRAD_FIELDS:
        if got.get(n) is None:
            continue
        g, w, e = f64(got[n]), f64(want[n]), f64(exact[n])
        assert np.isfinite(g).all(), n
        assert rel(g, w) <= 5e-3, (n, rel(g, w))
        assert rel(g, e) <= 3e-2, (n, rel(g, e))
    # statistics over two data-parallel ranks
    both = 2 * plain["counts_ext"]
    want = layer.backward(x, near, dy, ALPHA, BETA, counts_ext=both, t_total=3 * cfg.T)
    got = layer.backward_checkpoint8(x, ck, dy, ALPHA, BETA, counts_ext=both, t_total=3 * cfg.T)
    for n in ("dw_router", "dbias"):
        assert rel(f64(got[n]), f64(want[n])) <= 5e-3, n


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("combine,ffn", [("inplace", "single"), ("fused", "single"), ("separate", "pair")])
def test_forward_checkpoint_is_bitwise_the_stored_forward(name, combine, ffn):
    """The codes that the gate/up GEMM's epilogue writes are those of moe_checkpoint8 on the
    pre-activations that the training forward writes in bf16."""
    cfg = CASES[name]
    inp = I.make_inputs(cfg)
    layer, x, tnb = H.make_layer(inp, ffn=ffn)
    want = layer.forward(x, tnb, layer.alloc(cfg.T, save_preact=True, combine=combine))
    ck = layer.alloc_checkpoint8(cfg.T)
    for n in B.SAVED8_CODES:
        ck[n].fill_(99)
    got = layer.forward_checkpoint8(x, tnb, layer.alloc(cfg.T, combine=combine), ck)
    torch.cuda.synchronize()
    assert B.get_device_status(got["workspace"]) == B.OK
    for n in ("y", "logits", "topk_idx", "slot_row", "offsets", "losses"):
        assert torch.equal(got[n], want[n]), n
    R = int(want["offsets"][-1])
    for name, key, used in (("z", "z", R), ("zs", "z_shared", cfg.T), ("ys", "ys", R)):
        codes, scales = (torch.full_like(ck[f"{name}_{w}"], 99) for w in ("codes", "scales"))
        B.checkpoint8(want[key][:used], codes[:used], scales[:used])
        assert torch.equal(ck[name + "_codes"], codes) and torch.equal(ck[name + "_scales"], scales), name


def test_checkpointed_layers_share_their_scratch():
    """Two layers' forwards over one set of buffers, then their backwards in turn: each as if
    it had run alone."""
    cfg = CASES["ragged"]
    layer, x, tnb, dy, out, ck, _ = layer_step(cfg)
    alone = layer.backward_checkpoint8(x, ck, dy, ALPHA, BETA)
    alone = {n: alone[n].clone() for n in B.GRAD_FIELDS if alone.get(n) is not None}
    x2 = torch.flip(x, [0]).contiguous()
    ck2 = layer.alloc_checkpoint8(cfg.T)
    layer.forward_checkpoint8(x, tnb, out, ck)
    layer.forward_checkpoint8(x2, tnb, out, ck2)
    g = layer.alloc_grads(cfg.T, checkpoint8=True)
    layer.backward_checkpoint8(x2, ck2, dy, ALPHA, BETA, g)
    layer.backward_checkpoint8(x, ck, dy, ALPHA, BETA, g)
    torch.cuda.synchronize()
    for n, v in alone.items():
        assert torch.equal(g[n], v), n


def test_checkpointed_step_in_a_graph_and_on_fewer_tokens():
    cfg = CASES["wide"]
    layer, x, tnb, dy, out, ck, _ = layer_step(cfg)
    g = layer.alloc_grads(cfg.T, checkpoint8=True)
    layer.backward_checkpoint8(x, ck, dy, ALPHA, BETA, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward_checkpoint8(x, tnb, out, ck)
        layer.backward_checkpoint8(x, ck, dy, ALPHA, BETA, g)
    x.copy_(torch.flip(x, [0]))
    graph.replay()
    torch.cuda.synchronize()
    got = {n: g[n].clone() for n in B.GRAD_FIELDS if g.get(n) is not None}
    layer.forward_checkpoint8(x, tnb, out, ck)
    layer.backward_checkpoint8(x, ck, dy, ALPHA, BETA, g)
    for n, v in got.items():
        assert torch.equal(g[n], v), n
    T = 333                                            # fewer tokens in the same buffers
    few = layer.alloc_checkpoint8(T)
    layer.forward_checkpoint8(x[:T], tnb, out, few)
    a = layer.backward_checkpoint8(x[:T], few, dy[:T], ALPHA, BETA)
    layer.forward_checkpoint8(x[:T], tnb, out, ck)
    b = layer.backward_checkpoint8(x[:T], ck, dy[:T], ALPHA, BETA)
    torch.cuda.synchronize()
    for n in got:
        assert torch.equal(a[n], b[n]), n


def test_checkpoint_refusals():
    cfg = CASES["ragged"]
    layer, x, tnb, dy, out, ck, _ = layer_step(cfg)
    with pytest.raises(ValueError):
        layer.forward_checkpoint8(x, tnb, layer.alloc(cfg.T, xs=False), ck)
    with pytest.raises(ValueError):
        layer.forward_checkpoint8(x, tnb, layer.alloc(cfg.T - 1), ck)
    with pytest.raises(ValueError):
        layer.forward_checkpoint8(x, tnb, out, layer.alloc_checkpoint8(cfg.T - 1))
    with pytest.raises(ValueError):
        layer.backward_checkpoint8(x, layer.alloc_checkpoint8(cfg.T - 1), dy)
    with pytest.raises(ValueError):
        layer.backward_checkpoint8(x, ck, dy, grads=layer.alloc_grads(cfg.T))


@pytest.mark.parametrize("name", ["ragged", "pp"])
def test_a_checkpointed_backward_without_tokens_gives_zero_gradients(name):
    """A rank without tokens adds zeros to the others' weight gradients, whatever the buffers held;
    the gradients of the tokens, of which there are none, stay as they were."""
    cfg = CASES[name]
    layer, x, tnb = H.make_layer(I.make_inputs(cfg))
    x, tnb = x[:0], None if tnb is None else tnb[:0]
    ck, out = layer.alloc_checkpoint8(0), layer.alloc(0)
    grads = layer.alloc_grads(0, checkpoint8=True)
    for stream in (None, torch.cuda.Stream()):
        for n in B.GRAD_FIELDS:
            if grads[n] is not None:
                grads[n].fill_(float("nan"))
        torch.cuda.synchronize()
        layer.forward_checkpoint8(x, tnb, out, ck, stream)
        g = layer.backward_checkpoint8(x, ck, x, ALPHA, BETA, grads, torch.ones_like(ck["counts_ext"]), cfg.T, stream)
        torch.cuda.synchronize()
        for n in B.GRAD_FIELDS:
            if n in ("dx", "dtok_null_bias"):
                assert bool(torch.isnan(g[n]).all()), n
            elif g[n] is not None:
                assert int(torch.count_nonzero(g[n])) == 0, n


# --------------------------------------------- more items than the grid takes in one sweep


def power_of_two(e):
    """2^e in 64 bits from its exponent's bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def stored_on_gpu(x):
    """``stored_ref`` by blocks of all rows at once, in 64 bits on the GPU."""
    val, byte = torch.empty(x.shape, dtype=torch.float64, device="cuda"), []
    for c in range(0, x.shape[1], 32):
        blk = x[:, c:c + 32].double()
        m = blk.abs().amax(1)
        E = torch.where(m > 0, torch.frexp(m)[1].double() - 7, -126.0).clamp(min=-126)   # frexp: m = f 2^e, f < 1
        step = power_of_two(E)[:, None]
        val[:, c:c + 32] = torch.round(blk / step).clamp(-127, 127) * step
        byte.append((E + 127).to(torch.uint8))
    return val, torch.stack(byte, 1)


# (rows, columns, gap between the rows in elements). A sweep is 9472 items of eight blocks for single
# elements, 1.2M items of 16 columns (store) and 2.4M of 16 bytes (restore) for strided 16-byte pieces.
SWEEPS = [(20000, 1001, 0), (400003, 7, 0), (100001, 50, 1), (50001, 101, 0), (45001, 1000, 8), (45001, 1000, 0)]


@pytest.mark.parametrize("rows,cols,pad", SWEEPS)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_store_and_restore_in_many_sweeps(rows, cols, pad, dtype):
    dt = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn((rows, cols + pad), generator=g, device="cuda")
    x = (x * torch.exp2(torch.randint(-9, 4, (rows, 1), generator=g, device="cuda"))).to(dt)[:, :cols]
    for used in (rows, rows - 7):
        n = torch.tensor([used], dtype=torch.int32, device="cuda")
        codes = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
        scales = torch.full((rows, B.checkpoint8_scales(cols)), 77, dtype=torch.uint8, device="cuda")
        B.checkpoint8(x, codes, scales, n)
        val, byte = stored_on_gpu(x[:used])
        assert torch.equal(scales[:used], byte)
        step = power_of_two(byte.double() - 127).repeat_interleave(32, 1)[:, :cols]
        assert torch.equal(codes[:used].double() * step, val)
        assert bool((codes[used:] == 99).all()) and bool((scales[used:] == 77).all())
        whole = torch.full((rows, cols + pad), 4.0, dtype=dt, device="cuda")
        B.restore8(codes, scales, whole[:, :cols], n)
        assert torch.equal(whole[:used, :cols].double(), val)
        assert bool((whole[used:] == 4.0).all()) and bool((whole[:, cols:] == 4.0).all())


@pytest.mark.parametrize("rows,F,packed", [(30000, 499, False), (200001, 33, False), (30001, 800, False),
                                           (20001, 1024, True)])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_swiglu_backward8_in_many_sweeps(rows, F, packed, pad):
    """A sweep is 18944 items of 128 pairs for single elements and 9.7M pairs for 16-byte pieces."""
    rng = np.random.default_rng(rows + F)
    dt = torch.bfloat16
    codes = torch.from_numpy(rng.integers(-127, 128, size=(rows, 2 * F)).astype(np.int8)).cuda()
    scales = torch.from_numpy(rng.integers(107, 128, size=(rows, (2 * F + 31) // 32)).astype(np.uint8)).cuda()
    flat = torch.randn((rows, F + pad), generator=torch.Generator(device="cuda").manual_seed(F), device="cuda").to(dt)
    dh = flat[:, :F]
    dz = torch.full((rows, 2 * F + pad), 9.0, dtype=dt, device="cuda")
    h = torch.full((rows, F + pad), 9.0, dtype=dt, device="cuda")
    n = torch.tensor([rows - 3], dtype=torch.int32, device="cuda")
    B.swiglu_backward8(codes, scales, dh, dz[:, :2 * F], h[:, :F], packed=packed, rows_used=n)
    for a in range(0, rows - 3, 5000):
        r = slice(a, min(a + 5000, rows - 3))
        check_swiglu(codes[r], scales[r], dh[r], dz[r, :2 * F], h[r, :F], packed)
    for t, c in ((dz, 2 * F), (h, F)):
        assert bool((t[rows - 3:] == 9.0).all()) and bool((t[:, c:] == 9.0).all())
