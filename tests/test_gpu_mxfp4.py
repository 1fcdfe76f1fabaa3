"""GPU parity of the MXFP4 variant against the oracle: the quantizer bit-exact
(codes, E8M0 scales, padding), the GEMM within the bound of an fp32 sum and
bit-exact where that sum is exact, in every tile shape and K split."""
import numpy as np
import pytest
import torch

import synth
from oracle import mxfp4_ref as X
from oracle import nvfp4_ref as N
from tests.gpu_helpers import assert_bytes_equal, assert_within_tol, f32, gpu_bytes, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


def _check_quant(F, x_bf16: torch.Tensor, what: str):
    q = F.quantize_mxfp4(x_bf16.cuda())
    torch.cuda.synchronize()
    codes, sf = X.quantize_mxfp4(f32(x_bf16))
    assert_bytes_equal(gpu_bytes(q.codes), codes, what + " codes")
    assert_bytes_equal(gpu_bytes(q.sf), X.swizzle_sf_mxfp4(sf), what + " scale buffer")  # zero padding included


@pytest.mark.parametrize("m,k", [(1, 64), (7, 192), (127, 320), (129, 64), (300, 4160), (256, 128), (9600, 2112)])
def test_quantize_ragged_shapes_including_padding(F, m, k):
    # the last shape takes the 256-row tiles, every stage of the ring reused
    _check_quant(F, synth.activations_with_outlier_channels(m, k, seed=m * 7 + k), f"{m}x{k}")


def test_quantize_tile_heights_are_both_covered(F):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert F.nvfp4_quantize_tile_rows(300, 4160, sms) == 128 and F.nvfp4_quantize_tile_rows(9600, 2112, sms) == 256


def test_quantize_every_bf16_value_inside_a_block(F):
    bits = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32)
    v = bits[np.isfinite(bits)]
    n_blk = (v.size + 30) // 31
    vals = np.zeros(n_blk * 31, np.float32)
    vals[:v.size] = v
    vals = np.clip(vals, -7.0, 7.0)
    for top in (4.0, 6.0, 7.75, 6.0 * 2.0 ** 20, 6.0 * 2.0 ** -30):
        scale = np.float32(2.0 ** (np.floor(np.log2(top)) - 2))
        blocks = np.concatenate([np.full((n_blk, 1), top, np.float32),
                                 np.clip(vals * scale, -top, top).reshape(n_blk, 31)], axis=1)
        rows = (n_blk + 1) // 2
        x = np.zeros((rows * 2, 32), np.float32)
        x[:n_blk] = blocks
        _check_quant(F, torch.from_numpy(x.reshape(rows, 64)).to(torch.bfloat16), f"all bf16 values, top {top}")


def test_quantize_every_bf16_maximum(F):
    # each finite bf16 magnitude as a block's maximum, subnormals and the largest included
    bits = (np.arange(0x7F80, dtype=np.uint32) << 16).view(np.float32)
    x = np.zeros((bits.size, 32), np.float32)
    x[:, 0] = bits
    x[:, 1] = -bits * np.float32(0.5)
    x[:, 2] = bits * np.float32(0.3)
    _check_quant(F, torch.from_numpy(x.reshape(-1, 64)).to(torch.bfloat16), "every maximum")


def test_quantize_writes_only_its_own_buffers_and_unaligned_codes(F):
    # a code buffer that is 16- but not 32-byte aligned takes two 16-byte stores a row
    x = synth.activations_with_outlier_channels(130, 192, seed=5).cuda()
    want = F.quantize_mxfp4(x)
    buf = torch.full((16 + want.codes.numel() + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    sfb = torch.full((want.sf.numel() + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    codes = buf[16:16 + want.codes.numel()]
    assert codes.data_ptr() % 32 == 16
    F.quantize_mxfp4(x, out=F.MXFP4Tensor(codes.view(130, 96), sfb[:want.sf.numel()], 130, 192))
    assert torch.equal(codes.view(130, 96), want.codes) and torch.equal(sfb[:want.sf.numel()], want.sf)
    assert bool((buf[:16] == 0xA5).all()) and bool((buf[16 + want.codes.numel():] == 0xA5).all())
    assert bool((sfb[want.sf.numel():] == 0xA5).all())


def _linear(F, m, n, k, bias=True, rows=None, cols=None, alpha=1.0):
    wl = synth.LinearWorkload(f"mxfp4_{m}x{n}x{k}", m, k, n, seed=m + n + k)
    x, w = wl.activations(), wl.weight()
    b = synth.normal_bf16((n,), 0.01, synth._gen(7)) if bias else None
    xq, wq = F.quantize_mxfp4(x.cuda()), F.quantize_mxfp4(w.cuda())
    y = F.gemm_mxfp4(xq, wq, bias=b.cuda() if bias else None, alpha=alpha)
    torch.cuda.synchronize()
    r = np.arange(m) if rows is None else rows
    c = np.arange(n) if cols is None else cols
    a_codes, a_sf = X.quantize_mxfp4(f32(x)[r])
    b_codes, b_sf = X.quantize_mxfp4(f32(w)[c])
    y_ref = X.gemm_ref_mxfp4(a_codes, a_sf, b_codes, b_sf, alpha, f32(b)[c] if bias else None)
    tol = X.gemm_tolerance_mxfp4(a_codes, a_sf, b_codes, b_sf, y_ref, alpha)
    assert_within_tol(y.float().cpu().numpy()[np.ix_(r, c)], y_ref, tol, wl.name)


@pytest.mark.parametrize("m,n,k", [(1, 8, 64), (1, 2048, 4096), (100, 200, 192), (128, 192, 64), (130, 264, 320),
                                   (257, 392, 4160), (512, 768, 2112), (1000, 1288, 448)])
def test_gemm_ragged(F, m, n, k):
    _linear(F, m, n, k)


def test_gemm_alpha_without_bias(F):
    _linear(F, 33, 264, 576, bias=False, alpha=-0.37)


@pytest.mark.parametrize("m,n,k", [(2341, 2056, 3136), (4608, 2568, 1088)])
def test_gemm_wide_tiles_ragged_sampled(F, m, n, k):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert F.nvfp4_gemm_tile_shape(m, n, sms) == (2, 256, 1)
    rng = np.random.default_rng(m + n)
    rows = np.unique(np.r_[rng.choice(m, 40, replace=False), m - 1, 127, 128, 255, 256])
    cols = np.unique(np.r_[rng.choice(n, 64, replace=False), n - 1, 127, 128, 255, 256])
    _linear(F, m, n, k, rows=rows, cols=cols)


# (tile shape, K split) of each: every launch variant the library picks from
@pytest.mark.parametrize("m,n,k,plan", [(1, 384, 4096, (1, 192, 2, 4)), (300, 512, 8192, (2, 128, 2, 2)),
                                        (300, 2048, 512, (2, 128, 2, 1)), (1536, 2048, 512, (2, 192, 2, 1)),
                                        (2560, 2048, 512, (2, 256, 1, 1))])
def test_gemm_bit_exact_when_accumulation_is_exact(F, m, n, k, plan):
    # codes of {0, +-0.5, +-1, +-1.5, +-2}, scales 2^-1 .. 2^1: every product is a multiple of 2^-4 below 2^4 and
    # every partial sum of up to 8192 of them fits fp32's 24 bits, so the result is the oracle's rounded to bf16
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 148:
        assert F.nvfp4_gemm_plan(m, n, k, sms) == plan
    rng = np.random.default_rng(m + n + k)
    a_codes = N.pack_codes(rng.choice(np.array([0, 1, 2, 3, 4, 9, 10, 11, 12], np.uint8), (m, k)))
    b_codes = N.pack_codes(rng.choice(np.array([0, 1, 2, 3, 4, 9, 10, 11, 12], np.uint8), (n, k)))
    a_sf = rng.choice(np.array([126, 127, 128], np.uint8), (m, k // 32))
    b_sf = rng.choice(np.array([126, 127, 128], np.uint8), (n, k // 32))
    a = F.MXFP4Tensor(torch.from_numpy(a_codes).cuda(), torch.from_numpy(X.swizzle_sf_mxfp4(a_sf)).cuda(), m, k)
    b = F.MXFP4Tensor(torch.from_numpy(b_codes).cuda(), torch.from_numpy(X.swizzle_sf_mxfp4(b_sf)).cuda(), n, k)
    y = F.gemm_mxfp4(a, b, alpha=0.25).float().cpu().numpy()
    want = N.round_to_bf16(X.gemm_ref_mxfp4(a_codes, a_sf, b_codes, b_sf, alpha=0.25))
    assert np.array_equal(y, want)


def test_every_scale_byte_reaches_its_block(F):
    # one scale of 2^1 among ones: a wrong byte selector, k-block or row group moves the doubled block
    m, n, k = 256, 192, 576
    a_codes = np.full((m, k // 2), 0x22, np.uint8)   # 1.0
    b_codes = np.full((n, k // 2), 0x22, np.uint8)
    for operand in ("a", "b"):
        for blk in range(k // 32):
            for row in (0, 37, 100, 130):
                a_sf = np.full((m, k // 32), 127, np.uint8)
                b_sf = np.full((n, k // 32), 127, np.uint8)
                (a_sf if operand == "a" else b_sf)[row, blk] = 128
                a = F.MXFP4Tensor(torch.from_numpy(a_codes).cuda(),
                                  torch.from_numpy(X.swizzle_sf_mxfp4(a_sf)).cuda(), m, k)
                b = F.MXFP4Tensor(torch.from_numpy(b_codes).cuda(),
                                  torch.from_numpy(X.swizzle_sf_mxfp4(b_sf)).cuda(), n, k)
                y = F.gemm_mxfp4(a, b).float().cpu().numpy()
                want = np.full((m, n), float(k))
                if operand == "a":
                    want[row] += 32
                else:
                    want[:, row] += 32
                assert np.array_equal(y, N.round_to_bf16(want)), (operand, blk, row)


def test_graph_replay_and_another_stream(F):
    x = synth.activations_with_outlier_channels(200, 448, seed=1).cuda()
    w = F.quantize_mxfp4(synth.normal_bf16((520, 448), 0.02, synth._gen(2)).cuda())
    xq, y = F.quantize_mxfp4(x), torch.empty(200, 520, dtype=torch.bfloat16, device="cuda")
    want = F.gemm_mxfp4(xq, w).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.quantize_mxfp4(x, out=xq)
        F.gemm_mxfp4(xq, w, y=y)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    x2 = (-2 * x).contiguous()
    want2 = F.gemm_mxfp4(F.quantize_mxfp4(x2), w)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want2) and torch.equal(y, -2 * want)  # powers of two scale exactly
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = F.gemm_mxfp4(F.quantize_mxfp4(x), w)
    side.synchronize()
    assert torch.equal(again, want2)


def test_no_kernel_reported_a_fault(F):
    torch.cuda.synchronize()
    F.nvfp4_check_fault()
