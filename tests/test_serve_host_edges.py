"""Host side of the serving operators at the ends of their ranges (CPU)."""
import math

import pytest

import weight_quantized_gemm_amd as W


@pytest.mark.parametrize("rot,base,length,factor", [(128, 1e4, 131072, 8.0), (64, 1e4, 65536, 4.0), (128, 5e5, 8192, 8.0),
                                                    (128, 1e4, 4096, 16.0), (16, 100.0, 1 << 20, 2.0)])
def test_ramp_frequencies_blend_up_to_the_slow_end(rot, base, length, factor):
    """Also where even the lowest pair turns more than beta_slow times: the ramp's end lies past the last pair then,
    and that pair is blended like the others."""
    freq, _ = W.rope_frequencies(rot, base, scaling="ramp", factor=factor, original_length=length)
    plain, _ = W.rope_frequencies(rot, base)
    pairs = rot // 2
    # pair p turns length / (2 pi) * base^(-p / pairs) times
    place = lambda turns: pairs * math.log(length / (2 * math.pi * turns), base)
    lo, hi = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), rot - 1)
    for j in range(pairs):
        share = min(max((j - lo) / (hi - lo), 0.0), 1.0)
        want = float(plain[j]) * (1.0 - share + share / factor)
        assert abs(float(freq[j]) / want - 1) < 1e-6, j
        if length * float(plain[j]) / (2 * math.pi) > 1.0:  # turns more than beta_slow times
            assert float(freq[j]) > 1.000001 * float(plain[j]) / factor, j


def test_ramp_of_a_long_original_length():
    freq, _ = W.rope_frequencies(128, scaling="ramp", factor=8.0, original_length=131072)
    plain, _ = W.rope_frequencies(128)
    assert abs(float(freq[-1] / plain[-1]) - 0.370) < 5e-4


def test_tensors_and_workspaces_off_the_device_are_refused():
    """Their addresses would mean nothing to the kernels."""
    torch = pytest.importorskip("torch")
    gpu = torch.device("cuda:0")
    for given in (torch.empty(1 << 16, dtype=torch.uint8), torch.empty(1 << 16, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace is on"):
            W.serve._workspace(1 << 10, given, gpu)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        W.LoraMatmul(z(4, 64), z(2, 8, 64), z(2, 16, 8), i(4))
    with pytest.raises(ValueError, match="on a GPU"):
        W.Rope(z(4, 2, 64), None, None, i(4), torch.ones(32))
    with pytest.raises(ValueError, match="on a GPU"):
        W.TreeAttention(z(4, 2, 64), z(16, 2, 64), z(16, 2, 64), i(1, 1), i(1), i(2), page_size=16)


def test_tree_scale_whose_base_2_form_overflows_is_refused(wqlib):
    """The kernels take scale * log2(e): beyond 2^127 that may be infinite, and a score of 0 would become NaN."""
    import test_serve_host as host
    a = host.tree_args()
    t = [host.ref(x) for x in list(a.values())[:7]]
    call = lambda scale: wqlib.wq_tree_attention(*t, 16, scale, host.ref(a["output"]), None, 1 << 40, None)
    for scale in (2.4e38, -3.4e38, 2.0 ** 127 * (1 + 2.0 ** -20)):
        assert call(scale) == W.WQ_ERR_PARAM_INVALID, scale
    for scale in (2.0 ** 127, -2.0 ** 127, 0.0):  # (the missing workspace is found after the scale)
        assert call(scale) == W.WQ_ERR_PARAM_NULLPTR, scale
