"""The block-scaled 8-bit operators and the router's balance loss on a machine
without a GPU: what the entry points refuse, and with which code."""
import pytest

import tiled_tensor_core_persistent_gb300 as tcg
from tiled_tensor_core_persistent_gb300 import _build

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 5
P = 0x100000   # fake, aligned addresses: nothing is dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return tcg.lib()


def code(call):
    """The status of a call: 0, or the TcgError's code."""
    try:
        call()
        return 0
    except tcg.TcgError as e:
        return e.code


def no_gpu(call):
    """A request that passes every argument rule: accepted, or refused for the want of a GPU."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    return code(call) in (4, 6)


def op(data=P, ld=256, scales=P, scale_rows=1, rs=1, ks=300, gs=0):
    return tcg.block_operand(data, ld, scales, scale_rows, rs, ks, gs)


def gemm(M=300, N=200, K=256, A=None, B=None, beta=0.0, C=None, ldc=200, c="f32", D=P, ldd=200, d="bf16", ab="e4m3", **kw):
    return tcg.gemm_block128(M, N, K, A or op(), B or op(scale_rows=128), beta, C, ldc, c, D, ldd, d, ab_dtype=ab, **kw)


def test_gemm_refusals():
    assert no_gpu(lambda: gemm())
    assert no_gpu(lambda: gemm(ab="e5m2", B=op(scale_rows=1)))
    assert code(lambda: gemm(M=0, D=None)) == 0
    assert code(lambda: gemm(N=0, D=None)) == 0
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(ab="bf16"), dict(ab="mxe4m3"), dict(d="f16"), dict(D=None), dict(ldd=199),
                dict(A=op(scale_rows=2)), dict(B=op(scale_rows=64)), dict(A=op(data=None)), dict(B=op(scales=None)), dict(A=op(ld=255)),
                dict(A=op(ks=-1)), dict(beta=1.0), dict(beta=1.0, C=P, ldc=100), dict(beta=1.0, C=P, c="f16"), dict(act=7),
                dict(bias=P, bias_dtype="f16")):
        assert code(lambda: gemm(**bad)) == INVALID, bad
    for bad in (dict(A=op(scale_rows=128)), dict(A=op(data=P + 8)), dict(B=op(ld=264))):
        assert code(lambda: gemm(**bad)) == UNSUPPORTED, bad
    for bad in (dict(A=op(scales=P + 2)), dict(D=P + 1), dict(D=P + 2, d="f32"), dict(beta=1.0, C=P + 2), dict(bias=P + 1)):
        assert code(lambda: gemm(**bad)) == MISALIGNED, bad
    # K == 0 looks at neither operand
    assert no_gpu(lambda: gemm(K=0, A=op(data=None, scales=None), B=op(data=None, scales=None)))


def grouped(G=4, offsets=P, rows=100, N=200, K=256, A=None, B=None, D=P, ldd=200, d="bf16", ab="e4m3"):
    return tcg.gemm_block128_grouped(G, offsets, rows, N, K, A or op(), B or op(scale_rows=128), D, ldd, d, ab_dtype=ab)


def grouped_k(G=4, offsets=P, M=100, N=200, padded=256, A=None, B=None, beta=0.0, C=None, ldc=200, D=P, ldd=200, d="f32"):
    return tcg.gemm_block128_grouped_k(G, offsets, M, N, padded, A or op(), B or op(), beta, C, ldc, "f32", D, ldd, d)


def test_grouped_refusals():
    assert no_gpu(grouped)
    assert no_gpu(grouped_k)
    for call in (grouped, grouped_k):
        assert code(lambda: call(G=0)) == 0
        assert code(lambda: call(N=0)) == 0
        assert code(lambda: call(G=-1)) == INVALID
        assert code(lambda: call(offsets=None)) == INVALID
        assert code(lambda: call(D=None)) == INVALID
        assert code(lambda: call(offsets=P + 2)) == MISALIGNED
        assert code(lambda: call(G=1025)) == UNSUPPORTED
        assert code(lambda: call(A=op(scale_rows=128))) == UNSUPPORTED
    assert code(lambda: grouped(rows=0)) == 0
    assert code(lambda: grouped(G=1024, N=1 << 22, ldd=1 << 22)) == UNSUPPORTED
    assert code(lambda: grouped_k(M=0)) == 0
    assert code(lambda: grouped_k(padded=255)) == INVALID
    assert code(lambda: grouped_k(B=op(scale_rows=128))) == UNSUPPORTED
    assert code(lambda: grouped_k(beta=1.0)) == INVALID


def test_workspace_sizes():
    assert tcg.block128_workspace_size(0, 8192, 8192, 8192) >= 256
    assert tcg.block128_workspace_size(0, 1, 8192, 8192) > 256
    assert tcg.block128_workspace_size(16, 32, 4096, 4096) > 256
    assert tcg.block128_workspace_size(0, -1, 1, 1) == 0
    assert tcg.block128_workspace_size(-1, 1, 1, 1) == 0
    assert tcg.moe_balance_workspace_size() >= 256


def rows(r=10, c=200, x=P, ldx=200, xt="bf16", q=P, ldq=200, qt="e4m3", s=P, lds=10, **kw):
    return tcg.quantize_rows128(r, c, x, ldx, xt, q, ldq, qt, s, lds, **kw)


def cols(r=10, c=200, x=P, ldx=200, xt="bf16", q=P, ldq=128, qt="e4m3", s=P, lds=200, padded=128, **kw):
    return tcg.quantize_cols128(r, c, x, ldx, xt, q, ldq, qt, s, lds, padded_rows=padded, **kw)


def tiles(b=2, r=10, c=200, x=P, ldx=200, xt="bf16", q=P, ldq=200, qT=P, ldqt=10, qt="e4m3", s=P, **kw):
    return tcg.quantize_tiles128(b, r, c, x, ldx, xt, q, ldq, qT, ldqt, qt, s, **kw)


def test_quantize_refusals():
    for call in (rows, cols, tiles):
        assert no_gpu(call)
        for bad in (dict(r=-1), dict(c=-1), dict(xt="e4m3"), dict(qt="bf16"), dict(x=None), dict(ldx=199), dict(s=None)):
            assert code(lambda: call(**bad)) == INVALID, (call, bad)
        assert code(lambda: call(x=P + 1)) == MISALIGNED
        assert code(lambda: call(s=P + 2)) == MISALIGNED
        assert code(lambda: call(c=0)) == 0
    assert code(lambda: rows(r=0)) == 0
    assert code(lambda: rows(q=None)) == INVALID
    assert code(lambda: rows(ldq=199)) == INVALID
    assert code(lambda: rows(lds=9)) == INVALID
    assert code(lambda: rows(row_index=P + 1)) == MISALIGNED
    assert code(lambda: rows(source_rows=-1)) == INVALID
    assert code(lambda: cols(padded=127)) == INVALID
    assert code(lambda: cols(padded=0)) == 0
    assert code(lambda: cols(ldq=127)) == INVALID
    assert code(lambda: cols(lds=199)) == INVALID
    assert code(lambda: cols(r=200)) == INVALID                       # one group that does not fit
    assert code(lambda: cols(num_groups=2)) == INVALID                # groups without offsets
    assert code(lambda: cols(num_groups=1025, offsets=P)) == UNSUPPORTED
    assert code(lambda: cols(padded=65536 * 128, ldq=65536 * 128)) == UNSUPPORTED
    assert no_gpu(lambda: tiles(q=None))
    assert no_gpu(lambda: tiles(qT=None))
    assert code(lambda: tiles(q=None, qT=None)) == INVALID
    assert code(lambda: tiles(ldqt=9)) == INVALID
    assert code(lambda: tiles(b=-1)) == INVALID
    assert code(lambda: tiles(b=0)) == 0
    assert code(lambda: tiles(b=65536)) == UNSUPPORTED


def balance(t=10, e=8, k=2, x=P, ld=8, dt="bf16", topk=P, ldt=2, mask=None, counts=P, offsets=P, valid=P, loss=P):
    return tcg.moe_balance(t, e, k, x, ld, dt, topk, ldt, mask, 0.01, counts, offsets, valid, loss)


def balance_grad(t=10, e=8, k=2, x=P, ld=8, dt="bf16", counts=P, valid=P, grad=P, d=P, ldd=8, ddt="f32"):
    return tcg.moe_balance_backward(t, e, k, x, ld, dt, None, 0.01, counts, valid, grad, d, ldd, ddt)


def test_balance_refusals():
    assert no_gpu(balance)
    assert no_gpu(balance_grad)
    assert no_gpu(lambda: balance(offsets=None))
    for bad in (dict(t=-1), dict(e=0), dict(k=0), dict(x=None), dict(ld=7), dict(dt="e4m3")):
        assert code(lambda: balance(**bad)) == INVALID, bad
        assert code(lambda: balance_grad(**bad)) == INVALID, bad
    for bad in (dict(topk=None), dict(ldt=1), dict(counts=None), dict(valid=None), dict(loss=None)):
        assert code(lambda: balance(**bad)) == INVALID, bad
    for bad in (dict(counts=None), dict(valid=None), dict(grad=None), dict(d=None), dict(ldd=7), dict(ddt="e4m3")):
        assert code(lambda: balance_grad(**bad)) == INVALID, bad
    assert code(lambda: balance(e=1025, ld=1025)) == UNSUPPORTED
    assert code(lambda: balance(x=P + 1)) == MISALIGNED
    assert code(lambda: balance(topk=P + 2)) == MISALIGNED
    assert code(lambda: balance_grad(d=P + 2)) == MISALIGNED
    assert code(lambda: balance_grad(t=0, x=None)) == 0


def test_extents_past_the_index_range():
    """An index rounded up to a tile or a step has to fit an int: 2^31 - 4096 is taken, more is refused."""
    top = 2 ** 31 - 4096
    big = 2 ** 31 - 1
    for call in (rows, cols, tiles):
        assert code(lambda: call(c=top + 1, ldx=big, ldq=big, **({"lds": big} if call is cols else {}))) == UNSUPPORTED
    assert code(lambda: rows(r=top + 1, lds=big)) == UNSUPPORTED
    assert no_gpu(lambda: rows(r=top, lds=big))
    assert no_gpu(lambda: rows(c=top, ldx=big, ldq=big))
    for bad in (dict(M=top + 1), dict(N=top + 1, ldd=big), dict(K=top + 1, A=op(ld=big - 15), B=op(ld=big - 15))):
        assert code(lambda: gemm(**bad)) == UNSUPPORTED, bad
    assert code(lambda: grouped(rows=top + 1)) == UNSUPPORTED
    assert code(lambda: grouped(G=1, N=top + 1, ldd=big)) == UNSUPPORTED
    assert code(lambda: grouped(K=top + 1, A=op(ld=big - 15), B=op(ld=big - 15))) == UNSUPPORTED
    assert code(lambda: grouped_k(G=1, M=top + 1)) == UNSUPPORTED
    assert code(lambda: grouped_k(G=1, N=top + 1, ldd=big)) == UNSUPPORTED
    assert code(lambda: grouped_k(padded=2 ** 31 - 128, A=op(ld=big - 15), B=op(ld=big - 15))) == UNSUPPORTED
    assert code(lambda: balance(t=top + 1)) == UNSUPPORTED
    assert code(lambda: balance_grad(t=top + 1)) == UNSUPPORTED
    assert no_gpu(lambda: balance_grad(t=top))
