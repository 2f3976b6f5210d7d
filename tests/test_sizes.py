"""Sizes that do not fit the 32 bits in which the library takes them are
refused, and not cut to their low bits: the convolution's, the scan's and the
verification's tensors can be that long (one channel, few tokens)."""
import pytest
import torch

import linear_attention_rnn_gdn_amd as gdn

LONG = (1 << 32) + 8   # its low bits: 8


@pytest.mark.parametrize("make", [
    lambda n: gdn.GdnConvShape(1, n, 1, 4, 0, 0, 1, gdn.BF16), lambda n: gdn.GdnConvShape(n, 1, 1, 4, 0, 0, 1, gdn.BF16),
    lambda n: gdn.GdnSsmShape(1, n, 1, 8, 1, 0, 1, 0, 0, 0, 0, 0, gdn.BF16, gdn.F32), lambda n: gdn.GdnSsmShape(1, 1, 1, 8, 1, n, 1, 0, 0, 0, 0, 0, gdn.BF16, gdn.F32),
    lambda n: gdn.GdnVerifyShape(1, 1, n), lambda n: gdn.GdnVerifyShape(n, 1, 1)])
def test_shapes(make):
    for n in (LONG, 1 << 31, -(1 << 31) - 1):
        with pytest.raises(gdn.GdnError) as error:
            make(n)
        assert error.value.status == -2
    make((1 << 31) - 1)
    make(8)


@pytest.mark.gpu
def test_calls():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w = torch.ones(1, 4, device="cuda")
    x = torch.empty(1, LONG, 1, device="cuda", dtype=torch.bfloat16)
    for call in (lambda: gdn.conv_fwd(x, w), lambda: gdn.conv_bwd(x, w, x), lambda: gdn.conv_fwd_varlen(x, w, [0, 8]),
                 lambda: gdn.conv_step(x[0], w, torch.zeros(8, 3, 1, device="cuda", dtype=torch.bfloat16))):
        with pytest.raises(gdn.GdnError):
            call()
    del x
    i = torch.zeros(1, 1, device="cuda", dtype=torch.int32)
    with pytest.raises(gdn.GdnError):
        gdn.tree_verify(i, i - 1, torch.empty(1, 2, LONG, device="cuda"), torch.zeros(1, 2, device="cuda"))
