"""Host-side refusals of the slot-sorting and 8-bit checkpoint entry points: the C ABI with
made-up addresses (nothing is enqueued) and the binding's checks of types and shapes."""
import ctypes as C

import pytest
import torch

from token_choice_routing_b200 import binding as B

P = C.c_void_p(4096)   # never dereferenced: every call below is refused on the host
NUL = None
INV, UNS = B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED


def test_sort_refusals():
    f = B.LIB.moe_sort_slots
    ok = [4, 2, 8, P, 4, P, P, P, P, P, NUL]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_0=-1) == INV and call(_1=0) == INV and call(_2=0) == INV
    assert call(_1=33) == UNS and call(_2=1025) == UNS and call(_0=1 << 30, _1=2) == UNS
    assert call(_4=2) == INV and call(_4=1) == INV
    for i in (3, 5, 6, 7, 8, 9):
        assert call(**{f"_{i}": NUL}) == INV, i
    assert B.sort_workspace_bytes(-1, 2, 8) == 0 and B.sort_workspace_bytes(4, 2, 1025) == 0
    small, big = B.sort_workspace_bytes(1, 1, 1), B.sort_workspace_bytes(131072, 8, 64)
    assert 256 < small <= big and small % 256 == 0 and big % 256 == 0
    assert B.sort_workspace_bytes(0, 8, 64) > 0


# argument positions: T, K, rows, d, dtype, then pointers and row strides
MOVES = {
    "moe_permute": [4, 2, 8, 64, 0, P, 64, P, P, 64, NUL, NUL],
    "moe_permute_backward": [4, 2, 8, 64, 0, P, 64, P, P, 64, P, 64, NUL, NUL],
    "moe_unpermute": [4, 2, 8, 64, 0, P, 64, P, P, P, 64, P, 64, NUL, NUL],
    "moe_unpermute_backward": [4, 2, 8, 64, 0, P, 64, P, 64, P, P, P, 64, P, NUL, NUL],
    "moe_unpermute_backward8": [4, 2, 8, 64, 0, P, 64, P, P, P, P, P, 64, P, NUL, NUL],
}
# positions of the pointers that may not be null
REQUIRED = {"moe_permute": (5, 7, 8), "moe_permute_backward": (5, 7, 10), "moe_unpermute": (5, 7, 8, 11),
            "moe_unpermute_backward": (5, 7, 9, 10, 13), "moe_unpermute_backward8": (5, 7, 8, 9, 10, 13)}


@pytest.mark.parametrize("name", sorted(MOVES))
def test_row_movement_refusals(name):
    f = getattr(B.LIB, name)

    def call(i, v):
        a = list(MOVES[name])
        a[i] = v
        return f(*a)

    assert call(0, -1) == INV and call(1, 0) == INV and call(2, -1) == INV and call(3, 0) == INV
    assert call(1, 33) == UNS and call(0, 1 << 30) == UNS and call(3, (1 << 30) + 1) == UNS
    assert call(4, 3) == INV and call(4, -1) == INV
    for i in REQUIRED[name]:
        assert call(i, NUL) == INV, i
    for i in range(5, len(MOVES[name])):
        if MOVES[name][i] == 64:  # a row stride below the width
            assert call(i, 63) == INV, i
    assert call(0, 0) == B.OK      # no tokens: nothing to do


def test_unpermute_backward_needs_an_output():
    a = list(MOVES["moe_unpermute_backward"])
    a[7] = a[11] = a[13] = NUL
    assert B.LIB.moe_unpermute_backward(*a) == INV


def test_checkpoint_refusals():
    L = B.LIB
    pack = [4, 64, 0, P, 64, NUL, P, P, NUL, NUL]
    restore = [4, 64, 0, P, P, NUL, P, 64, NUL, NUL]
    for f, a, ptrs, ld in ((L.moe_checkpoint8, pack, (3, 6, 7), 4), (L.moe_restore8, restore, (3, 4, 6), 7)):
        def call(i, v):
            b = list(a)
            b[i] = v
            return f(*b)
        assert call(0, -1) == INV and call(1, 0) == INV and call(2, 3) == INV and call(ld, 63) == INV
        assert call(1, (1 << 30) + 1) == UNS and call(0, 1 << 60) == UNS
        for i in ptrs:
            assert call(i, NUL) == INV, i
        assert call(0, 0) == B.OK
    assert [B.checkpoint8_scales(c) for c in (-1, 0, 1, 32, 33, 1001)] == [0, 0, 1, 1, 2, 32]


def test_swiglu_backward8_refusals():
    ok = [4, 64, 1, 0, P, P, P, 64, NUL, P, 128, P, 64, NUL, NUL]

    def call(i, v, **kw):
        a = list(ok)
        a[i] = v
        for j, u in kw.items():
            a[int(j[1:])] = u
        return B.LIB.moe_swiglu_backward8(*a)

    assert call(0, -1) == INV and call(1, 0) == INV and call(3, 7) == INV
    assert call(1, 32, _7=32, _10=64, _12=32) == INV            # packed needs whole panels
    assert call(1, (1 << 29) + 64) == UNS
    for i in (4, 5, 6, 9):
        assert call(i, NUL) == INV, i
    assert call(7, 63) == INV and call(10, 127) == INV and call(12, 63) == INV
    assert call(0, 0) == B.OK


def test_backward_checkpoint8_refusals():
    dm = B.dims(256, 128, 8, 8, 4, 64, 64)
    need = B.backward_checkpoint8_workspace_bytes(dm)
    assert need >= B.backward_workspace_bytes(dm) + 2 * 256 * 4 * (128 + 64) + 2 * 256 * 64
    pp = B.dims(256, 128, 8, 8, 4, 64, 64, C=1, V=1)
    assert B.backward_checkpoint8_workspace_bytes(pp) >= B.backward_workspace_bytes(pp) + 2 * 256 * 4 * (2 * 128 + 64)
    assert B.backward_checkpoint8_workspace_bytes(B.dims(-1, 128, 8, 8, 4, 64, 64)) == 0
    w = B.Weights(*[4096] * 8)
    g = B.Grads(*[4096] * 11)

    def call(field=None, value=None, weights=w, dims=dm):
        sv = B.Saved8()
        for n in B.SAVED8_FIELDS + B.SAVED8_CODES:
            setattr(sv, n, 4096)
        sv.t_total = 256
        if field:
            setattr(sv, field, value)
        return B.LIB.moe_backward_checkpoint8(C.byref(dims), C.byref(weights), C.byref(sv), P, 0.02, 0.001,
                                              C.byref(g), NUL, NUL)

    for n in B.SAVED8_FIELDS + B.SAVED8_CODES:
        assert call(n, None) == INV, n
    assert call("t_total", 255) == INV
    assert call() == INV  # no workspace
    assert call(dims=B.dims(256, 100, 8, 8, 4, 64, 64)) == UNS
    assert call(dims=B.dims(0, 128, 8, 8, 4, 64, 64)) == B.OK


def test_forward_checkpoint8_refusals():
    dm = B.dims(256, 128, 8, 8, 4, 64, 64)
    w = B.Weights(*[4096] * 8)

    def call(out=None, code=None, value=None, dims=dm, ws=P):
        o, q = B.Outputs(*[4096] * len(B.OUTPUT_FIELDS)), B.Codes8(*[4096] * 6)
        if out:
            setattr(o, out, value)
        if code:
            setattr(q, code, value)
        return B.LIB.moe_forward_checkpoint8(C.byref(dims), C.byref(w), P, NUL, C.byref(o), C.byref(q), ws, NUL)

    for n in ("xs", "logits", "topk_idx", "slot_row", "h", "ys", "y", "offsets", "losses"):
        assert call(out=n) == INV, n
    for n in B.SAVED8_CODES:
        assert call(code=n) == INV, n
        assert call(code=n, value=4096 + (8 if n.endswith("codes") else 2)) == INV, n   # alignment
    assert call(ws=NUL) == INV
    assert call(dims=B.dims(256, 100, 8, 8, 4, 64, 64)) == UNS
    assert call(dims=B.dims(0, 128, 8, 8, 4, 64, 64)) == B.OK


def test_saved8_layout_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [f for f, _ in B.Saved8._fields_]
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_null.h"', "int main(void) {"]
    src += [f'  printf("%zu\\n", offsetof(moe_saved8_t, {f}));' for f in fields]
    src += ['  printf("%zu\\n", sizeof(moe_saved8_t));']
    src += [f'  printf("%zu\\n", offsetof(moe_codes8_t, {f}));' for f, _ in B.Codes8._fields_]
    src += ["  return 0;", "}"]
    (tmp_path / "l.c").write_text("\n".join(src) + "\n")
    exe = str(tmp_path / "l")
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(tmp_path / "l.c"), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert got == ([getattr(B.Saved8, f).offset for f in fields] + [C.sizeof(B.Saved8)] +
                   [getattr(B.Codes8, f).offset for f, _ in B.Codes8._fields_])


# ---------------------------------------------------------------------- the binding's checks


@pytest.fixture
def cpu_as_device(monkeypatch):
    """The checks run before any pointer is used: with CPU tensors taken for the current
    device's, every call below must raise in the binding or be refused by the library."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(B, "_raw_stream", lambda stream, dev: None)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_checks_types_shapes_and_strides(cpu_as_device):
    i32, f32 = torch.int32, torch.float32
    x, sr, xs = z(4, 64), z(4, 2, dtype=i32), z(8, 64)
    bad = [
        lambda: B.permute(x, sr.long(), xs),
        lambda: B.permute(x, z(5, 2, dtype=i32), xs),
        lambda: B.permute(x, sr, z(8, 65)),
        lambda: B.permute(x, sr, z(8, 64, dtype=f32)),
        lambda: B.permute(x.double(), sr, xs.double()),
        lambda: B.permute(z(64, 4).t(), sr, xs),
        lambda: B.permute(z(1, 64).expand(4, 64), sr, xs),
        lambda: B.permute(x, z(2, 4, dtype=i32).t(), xs),
        lambda: B.permute(x[0], sr, xs),
        lambda: B.permute_backward(xs, sr, x, base=z(3, 64)),
        lambda: B.unpermute(xs, z(4, 2), sr, x),
        lambda: B.unpermute(xs, z(4, 3, dtype=f32), sr, x),
        lambda: B.unpermute_backward(x, xs, z(4, 2, dtype=f32), sr, z(9, 64), z(4, 2, dtype=f32)),
        lambda: B.unpermute_backward(x, xs, z(4, 2, dtype=f32), sr, xs, None),
        lambda: B.unpermute_backward(x, None, z(4, 2, dtype=f32), sr, None, None),
        lambda: B.unpermute_backward8(x, z(8, 64, dtype=torch.uint8), z(8, 2, dtype=torch.uint8), z(4, 2, dtype=f32),
                                      sr, xs, z(4, 2, dtype=f32)),
        lambda: B.unpermute_backward8(x, z(8, 64, dtype=torch.int8), z(8, 3, dtype=torch.uint8), z(4, 2, dtype=f32),
                                      sr, xs, z(4, 2, dtype=f32)),
        lambda: B.sort_slots(sr.short(), 8, z(8, dtype=i32), z(9, dtype=i32), z(8, dtype=i32), sr,
                             z(4096, dtype=torch.uint8)),
        lambda: B.sort_slots(sr, 8, z(8, dtype=i32), z(8, dtype=i32), z(8, dtype=i32), sr, z(4096, dtype=torch.uint8)),
        lambda: B.sort_slots(sr, 8, z(8, dtype=i32), z(9, dtype=i32), z(7, dtype=i32), sr, z(4096, dtype=torch.uint8)),
        lambda: B.sort_slots(sr, 8, z(8, dtype=i32), z(9, dtype=i32), z(8, dtype=i32), sr, z(16, dtype=torch.uint8)),
        lambda: B.sort_slots(sr, 8, z(8, dtype=i32), z(9, dtype=i32), z(8, dtype=i32), sr, None),
        lambda: B.checkpoint8(x, z(4, 64, dtype=torch.int8), z(4, 3, dtype=torch.uint8)),
        lambda: B.checkpoint8(x, z(4, 64, dtype=torch.int8), z(4, 2, dtype=torch.uint8), rows_used=z(2, dtype=i32)),
        lambda: B.checkpoint8(x, z(4, 64, dtype=torch.int8), z(4, 2, dtype=torch.uint8),
                              rows_used=z(1, dtype=torch.int64)),
        lambda: B.restore8(z(4, 64, dtype=torch.int8).t().contiguous().t(), z(4, 2, dtype=torch.uint8), x),
        lambda: B.swiglu_backward8(z(4, 128, dtype=torch.int8), z(4, 4, dtype=torch.uint8), x, z(4, 127), x),
        lambda: B.swiglu_backward8(z(4, 128, dtype=torch.int8), z(4, 4, dtype=torch.uint8), x, z(4, 128), z(4, 65)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")


def test_binding_passes_limits_on_to_the_library(cpu_as_device):
    with pytest.raises(B.MoEError):
        B.permute(z(1, 8), z(1, 33, dtype=torch.int32), z(33, 8))
    with pytest.raises(B.MoEError):
        B.swiglu_backward8(z(1, 64, dtype=torch.int8), z(1, 2, dtype=torch.uint8), z(1, 32), z(1, 64), None)


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # CPU tensors report -1
    with pytest.raises(ValueError, match="current device"):
        B.permute(z(4, 64), z(4, 2, dtype=torch.int32), z(8, 64))
    with pytest.raises(ValueError, match="current device"):
        B.checkpoint8(z(4, 64), z(4, 64, dtype=torch.int8), z(4, 2, dtype=torch.uint8))
