"""GPU tests of the attention operators at the limits of what they are given, against the 64-bit implementations of attn_ref."""
import numpy as np
import pytest

from test_gpu_attention import _check_decode, _decode, lib  # noqa: F401

pytestmark = pytest.mark.gpu


# A block that no token has been appended to may hold any scale byte; 255 is NaN.
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hk,d,qn", [(4, 2, 64, 1), (8, 1, 128, 1), (16, 1, 128, 1), (6, 2, 96, 4)])
def test_decode_scales_of_blocks_that_nothing_wrote(page, hq, hk, d, qn):
    lens = [7, 16, 33, 48, 65, 100, 129, 300]

    def edit(table, codes, scales):
        for s in scales:
            written = np.zeros(s.shape, bool)
            for b, n in enumerate(lens):
                for p in range(0, n, 16):
                    written[table[b, p // page], :, p % page // 16] = True
            s[~written] = 255

    _, args, host, out, lse = _decode(lens, hq, hk, d, page, qn, 400 + page, edit)
    _check_decode(lens, hq, hk, d, page, qn, host, args[0], out, lse)
