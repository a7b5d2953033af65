"""Host-side checks of the 8-bit products and the token log-probabilities (no GPU):
every refusal happens before any CUDA call, and the arithmetic that the kernels
rest on is checked with numpy."""
import ctypes

import numpy as np
import pytest

from decoder_only_transformer_sm_b200 import native

P = ctypes.c_void_p(64)      # never dereferenced: validation fails first
ODD = ctypes.c_void_p(65)


def _refused(fn, ok, changes):
    for change in changes:
        args = list(ok)
        for i, bad in change.items():
            args[i] = bad
        assert fn(*args) == -1, change


def test_quantize_rows_refusals():
    lib = native.load_library()
    ok = (1, P, 4, 8, 8, P, 8, P, None)
    _refused(lib.gpt2k_quantize_rows, ok,
             [{0: 2}, {2: 0}, {3: 0}, {4: 7}, {6: 7}, {1: None}, {5: None}, {7: None}, {1: ODD}, {7: ODD}, {2: (1 << 30) + 1},
              {3: (1 << 30) + 1, 4: 1 << 31, 6: 1 << 31}])


def test_matmul_i8_refusals():
    lib = native.load_library()
    #      0  1   2  3  4   5  6  7  8   9  10 11 12 13 14 15 16 17
    ok = (P, 16, P, P, 16, P, 4, 8, 16, 1, 1, P, 8, P, P, 8, P, None)
    _refused(lib.gpt2k_matmul_i8, ok,
             [{6: 0}, {7: 0}, {8: 0}, {1: 15}, {4: 15}, {12: 7}, {9: 4}, {9: 5}, {9: -1}, {10: 2},
              {1: 1 << 20, 4: 1 << 20, 8: 131072},                     # sums could pass 32 bits
              {6: (1 << 30) + 1}, {7: (1 << 30) + 1, 12: 1 << 31, 15: 1 << 31},
              {0: None}, {2: None}, {3: None}, {5: None}, {11: None}, {16: None},
              {13: None},                                              # bias wanted
              {9: 3},                                                  # bias_resid writes fp32
              {9: 3, 10: 0, 14: None}, {9: 3, 10: 0, 15: 7},
              {2: ODD}, {5: ODD}, {11: ODD}, {13: ODD}])


def test_token_logprobs_refusals():
    lib = native.load_library()
    #     0  1  2  3   4   5    6  7  8  9  10 11 12 13 14
    ok = (1, P, 3, 40, 40, 1.0, P, 5, P, P, P, P, P, P, None)
    _refused(lib.gpt2k_token_logprobs, ok,
             [{0: 2}, {2: 0}, {3: 0}, {4: 39}, {5: 0.0}, {5: -1.0}, {5: float("nan")}, {5: float("inf")}, {5: 1e-39},
              {2: (1 << 30) + 1}, {2: 1 << 20, 3: 1 << 22, 4: 1 << 22},
              {1: None}, {13: None}, {6: None}, {8: None}, {7: 33}, {7: -1}, {3: 4, 4: 4}, {11: None}, {12: None},
              {7: 0}, {6: None, 8: None, 9: None, 10: None, 7: 0, 11: None, 12: None}, {1: ODD}, {10: ODD}])


def test_token_logprobs_bwd_refusals():
    lib = native.load_library()
    Q = ctypes.c_void_p(4096)
    #     0  1  2  3   4   5    6  7  8  9  10 11 12  13 14
    ok = (1, P, 3, 40, 48, 1.0, P, P, P, P, P, Q, 48, P, None)
    _refused(lib.gpt2k_token_logprobs_bwd, ok,
             [{0: 2}, {2: 0}, {3: 0}, {4: 39}, {12: 39}, {5: 0.0}, {1: None}, {7: None}, {11: None}, {13: None},
              {8: None, 10: None, 6: None}, {6: None}, {8: None}, {9: None}, {11: P, 12: 40}, {11: ODD}, {7: ODD}])


def test_binding_refusals():
    """Shapes, types, strides and devices that the binding does not take."""
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 8))
    q, s = torch.zeros((4, 8), dtype=torch.int8), torch.zeros(4)
    for bad in [(x.double(), q, s), (x, q[:3], s), (x, q, s[:3]), (x, q.float(), s), (x[0], q, s),
                (x.t().contiguous().t(), q, s),
                (x, q, s)]:                                            # not on a GPU
        with pytest.raises(ValueError):
            native.quantize_rows(*bad)
    b, bs = torch.zeros((5, 8), dtype=torch.int8), torch.zeros(5)
    with pytest.raises(ValueError):
        native.matmul_i8(q, s, b[:, :7], bs, torch.zeros((4, 5)))
    with pytest.raises(ValueError):
        native.matmul_i8(q, s, b, bs, torch.zeros((4, 6)))
    with pytest.raises(ValueError):
        native.token_logprobs(x, 9, 1.0, lse=s)
    with pytest.raises(ValueError):
        native.token_logprobs(x, 8, 1.0, lse=s, top_ids=torch.zeros((4, 2), dtype=torch.int64),
                              top_logp=torch.zeros((4, 2)))
    with pytest.raises(ValueError):
        native.token_logprobs_bwd(x, 8, 1.0, s, x.bfloat16(), entropy=s, dentropy=s)


def test_fp32_quotient_is_within_its_bound():
    """For a > 1e-30 the kernel's first guess is the whole number nearest t = fl(x fl(127 / a)), read from the low bits
    of fl(t + 3 2^22); fp32 rows look again at a t within 1.7e-5 of a border. t has to be within 1.6e-5 of the quotient
    (two roundings of half a step each, 127 * 2 * 2^-24 = 1.5e-5), and a 64-bit quotient (smaller a) must not make or
    lose a tie."""
    rng = np.random.default_rng(0)
    for scale in (1.0, 1e-26, 3e37):
        a = (np.abs(rng.standard_normal(200000)) * scale + scale * 1e-3).astype(np.float32)
        x = (a * rng.uniform(-1, 1, a.size)).astype(np.float32)
        t = x * (np.float32(127.0) / a)
        exact = 127.0 * x.astype(np.float64) / a.astype(np.float64)
        assert np.max(np.abs(t.astype(np.float64) - exact)) < 1.6e-5
        whole = (t + np.float32(12582912.0)).view(np.uint32) & 0xff
        assert np.array_equal(whole.astype(np.uint8).view(np.int8), np.rint(t).astype(np.int8))
    # ties: a = 254 2^e, x = odd 2^e give quotients (2 k + 1) / 2; their fp32 neighbours do not
    for e in (-120, 0, 100):
        a = np.float32(254.0 * 2.0 ** e)
        odd = (np.arange(-253, 254, 2) * 2.0 ** e).astype(np.float32)
        twice = 2 * 127.0 * odd.astype(np.float64) / float(a)
        assert np.all(twice == np.rint(twice))
        for y in (np.nextafter(odd, np.float32(np.inf)), np.nextafter(odd, np.float32(-np.inf))):
            off = 2 * 127.0 * y.astype(np.float64) / float(a)
            assert np.all(off != np.rint(off))


def test_residual_in_place_with_another_stride_is_refused():
    """A tile's results would overwrite residuals that other tiles still read."""
    lib = native.load_library()
    #      0  1   2  3  4   5  6  7  8   9  10 11 12 13 14 15 16 17
    ok = (P, 16, P, P, 16, P, 4, 8, 16, 3, 0, P, 8, P, P, 8, ODD, None)   # (all but the status word, checked last)
    assert lib.gpt2k_matmul_i8(*ok) == -1 and b"aligned" in lib.gpt2_last_error()
    for ldo, ldr in ((8, 9), (16, 8)):
        args = list(ok)
        args[12], args[15] = ldo, ldr
        assert lib.gpt2k_matmul_i8(*args) == -1 and b"in place" in lib.gpt2_last_error()
    # one row has no stride
    args = list(ok)
    args[6], args[15] = 1, 9
    assert lib.gpt2k_matmul_i8(*args) == -1 and b"aligned" in lib.gpt2_last_error()


def test_temperatures_past_the_limit_are_refused():
    """Above 1e20 differences of logits no longer fit where the running sums need them (logits of -1e32 and 1e32 at
    temperature 1e32 lost a part of the entropy)."""
    lib = native.load_library()
    fwd = (1, P, 3, 40, 40, 1.0, P, 5, P, P, P, P, ODD, P, None)     # (all but one pointer, checked last)
    bwd = (1, P, 3, 40, 48, 1.0, P, P, P, P, P, ctypes.c_void_p(4097), 48, P, None)
    for fn, ok in ((lib.gpt2k_token_logprobs, fwd), (lib.gpt2k_token_logprobs_bwd, bwd)):
        for tau, said in ((1e20, b"aligned"), (1.0001e20, b"temperature"), (1e32, b"temperature"), (3e38, b"temperature")):
            args = list(ok)
            args[5] = tau
            assert fn(*args) == -1 and said in lib.gpt2_last_error(), (tau, lib.gpt2_last_error())


def test_binding_refuses_extents_that_32_bits_would_cut_off():
    """Sizes go to the library as 32-bit integers: 2^32 + 8 columns must not arrive as 8."""
    torch = pytest.importorskip("torch")
    big = (1 << 32) + 8

    def wide(rows, cols, dtype=torch.float32):
        return torch.empty(1, dtype=dtype).expand(rows, cols) if cols == 1 else torch.empty(
            (rows, cols), dtype=dtype, device="meta")

    s = torch.zeros(4)
    for x, q in ((wide(4, big), wide(4, big, torch.int8)), (wide(big, 8), wide(big, 8, torch.int8))):
        with pytest.raises(ValueError, match="2\\^31"):
            native.quantize_rows(x, q, s)
    q = torch.zeros((4, 8), dtype=torch.int8)
    with pytest.raises(ValueError, match="2\\^31"):
        native.matmul_i8(q, s, wide(big, 8, torch.int8), s, wide(4, big))
    with pytest.raises(ValueError, match="2\\^31"):
        native.matmul_i8(wide(4, big, torch.int8), s, wide(4, big, torch.int8), s, torch.zeros((4, 4)))
    # logits may have more columns than V; V itself, negative ones among them, is checked
    for V in (big, -(1 << 32) + 8):
        with pytest.raises(ValueError, match="V = "):
            native.token_logprobs(wide(4, 2 * big), V, 1.0, lse=s)
        with pytest.raises(ValueError, match="V = "):
            native.token_logprobs_bwd(wide(4, 2 * big), V, 1.0, s, wide(4, 2 * big), entropy=s, dentropy=s)
    with pytest.raises(ValueError, match="2\\^31"):
        native.token_logprobs(wide(big, 8), 8, 1.0, lse=wide(1, big)[0])
    with pytest.raises(ValueError, match="top_ids"):
        native.token_logprobs(wide(1, 8), 8, 1.0, top_ids=wide(1, big, torch.int32), top_logp=wide(1, big))
