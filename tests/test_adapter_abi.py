"""Argument rules of the dropout and 8-bit entry points (no GPU: every call
here is refused before any CUDA call)."""
import ctypes

import pytest
import torch

ALIGNED = 0x7f0000001000      # never dereferenced: validation only
M, K, N, R_ = 128, 256, 512, 16
BIG = 1 << 40


def ptrs(n):
    return [ALIGNED + i * (1 << 32) for i in range(n)]


CALLS = {  # name: (pointer names, has flags, 8-bit)
    "lora_fwd_dropout": (("X", "W", "A", "B", "Y"), False, False),
    "lora_bwd_dropout": (("X", "W", "A", "B", "dY", "dX", "dA", "dB"), True, False),
    "lora_fwd_fp8": (("X", "Wq", "Ws", "A", "B", "Y"), False, True),
    "lora_bwd_fp8": (("X", "Wq", "Ws", "A", "B", "dY", "dX", "dA", "dB"), True, True),
}


def call(L, name, p=0.1, sizes=(M, K, N, R_), ws=ALIGNED + (1 << 37), ws_bytes=BIG, rng=ALIGNED + (1 << 38), flags=0,
         **over):
    names, has_flags, _ = CALLS[name]
    args = dict(zip(names, ptrs(len(names))))
    args.update(over)
    a = [ctypes.c_void_p(args[n]) if args[n] else None for n in names]
    a += [*sizes, 1.0, p, rng, ws, ws_bytes] + ([flags] if has_flags else []) + [None]
    return L.STATUS[getattr(L.lib(), name)(*a)]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_pointers(built_lib, name):
    for n in CALLS[name][0]:
        assert call(built_lib, name, **{n: 0}) == "LORA_ERR_NULL", n
        assert call(built_lib, name, **{n: ALIGNED + (1 << 36) + 8}) == "LORA_ERR_ALIGN", n


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("sizes,want", [
    ((-1, K, N, R_), "SHAPE"), ((M, 0, N, R_), "SHAPE"), ((M, K, -8, R_), "SHAPE"), ((M, K + 4, N, R_), "SHAPE"),
    ((M, K, N + 4, R_), "SHAPE"), ((M, K, N, 0), "RANK"), ((M, K, N, 12), "RANK"), ((M, K, N, 136), "RANK"),
    ((1 << 31, K, N, R_), "SHAPE"),
])
def test_sizes(built_lib, name, sizes, want):
    assert call(built_lib, name, sizes=sizes) == "LORA_ERR_" + want


def test_8_bit_rows_are_16_bytes(built_lib):
    L = built_lib
    for name in ("lora_fwd_fp8", "lora_bwd_fp8"):
        assert call(L, name, sizes=(M, K + 8, N, R_)) == "LORA_ERR_SHAPE"
        assert call(L, name, sizes=(M, K, N + 8, R_)) == "LORA_ERR_SHAPE"
    assert L.lora_fp8_workspace_size(M, K + 8, N, R_) == 0
    assert L.lora_fp8_workspace_size(0, K, N, R_) == 0
    so = L.lib()
    q = ptrs(3)
    for fn in (so.lora_quantize_fp8, so.lora_dequantize_fp8):
        assert L.STATUS[fn(*q, N, K + 8, None)] == "LORA_ERR_SHAPE"
        assert L.STATUS[fn(*q, 0, K, None)] == "LORA_ERR_SHAPE"
        for i in range(3):
            assert L.STATUS[fn(*[None if j == i else v for j, v in enumerate(q)], N, K, None)] == "LORA_ERR_NULL"
            assert L.STATUS[fn(*[v + 8 * (j == i) for j, v in enumerate(q)], N, K, None)] == "LORA_ERR_ALIGN"
        assert L.STATUS[fn(q[0], q[1], q[0] + 16, N, K, None)] == "LORA_ERR_ALIAS"


@pytest.mark.parametrize("name", sorted(CALLS))
def test_dropout_rules(built_lib, name):
    L = built_lib
    for p in (-0.1, 1.0, 1.5, float("nan"), float("inf"), 1.0 - 2.0 ** -18):
        assert call(L, name, p=p) == "LORA_ERR_DROPOUT", p
    assert call(L, name, rng=None) == "LORA_ERR_DROPOUT"
    assert call(L, name, rng=ALIGNED + 8) == "LORA_ERR_ALIGN"


@pytest.mark.parametrize("name", sorted(CALLS))
def test_workspace_rules(built_lib, name):
    L = built_lib
    size = L.lora_fp8_workspace_size if CALLS[name][2] else L.lora_bwd_workspace_size
    need = size(M, K, N, R_)
    assert need > 0
    assert call(L, name, ws=None) == "LORA_ERR_WORKSPACE"
    assert call(L, name, ws_bytes=need - 1) == "LORA_ERR_WORKSPACE"
    assert call(L, name, ws=ALIGNED + (1 << 37) + 128) == "LORA_ERR_ALIGN"
    for n in CALLS[name][0]:
        p = dict(zip(CALLS[name][0], ptrs(9)))[n]
        assert call(L, name, ws=p) == "LORA_ERR_ALIAS", n
    assert call(L, name, rng=ALIGNED + (1 << 37)) == "LORA_ERR_ALIAS"


@pytest.mark.parametrize("name", sorted(CALLS))
def test_outputs_overlap_nothing(built_lib, name):
    names = CALLS[name][0]
    where = dict(zip(names, ptrs(len(names))))
    for o in [n for n in names if n in ("Y", "dX", "dA", "dB")]:
        for other in names:
            if other != o:
                assert call(built_lib, name, **{o: where[other]}) == "LORA_ERR_ALIAS", (o, other)


def test_flags(built_lib):
    for name in ("lora_bwd_dropout", "lora_bwd_fp8"):
        assert call(built_lib, name, flags=4) == "LORA_ERR_FLAGS"


def test_workspace_holds_the_backwards(built_lib):
    L = built_lib
    for m, k, n, r in ((1, 16, 16, 8), (M, K, N, R_), (1000, 2560, 9728, 128)):
        codes = m * max(k, n)
        assert L.lora_fp8_workspace_size(m, k, n, r) >= L.lora_bwd_workspace_size(m, k, n, r) + codes


def test_binding_checks_tensors(built_lib):
    L = built_lib
    b = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    X, W, A, B, Y = b(M, K), b(N, K), b(R_, K), b(N, R_), b(M, N)
    rng = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        L.lora_fwd_dropout(X, W, A, B, Y, 1.0, 0.1, rng, ws)          # not CUDA tensors
    with pytest.raises(TypeError):
        L.lora_fwd_dropout(X.float(), W, A, B, Y, 1.0, 0.1, rng, ws)
    with pytest.raises(ValueError):
        L.lora_quantize_fp8(W, W.to(torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu))
    with pytest.raises(ValueError):
        L.lora_fwd_dropout(X[0], W, A, B, Y, 1.0, 0.1, rng, ws)
