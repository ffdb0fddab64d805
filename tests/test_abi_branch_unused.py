"""Arguments that a call of the gated branch does not look at do not refuse it: a pitch without its
tensor, rstd_branch without gamma_post, the pitches of an empty tensor. Host checks, without a GPU;
what the call refuses in the end (no workspace) is checked after them."""
import pytest

from test_abi_branch import ALIGN, NULL, SHAPE, WORKSPACE, _branch, _bwd, lib, pytestmark  # noqa: F401

CUDA = 5
FAR = 1 << 40                                          # beyond any pitch that is taken


@pytest.mark.parametrize("unused", [dict(dres=0, ld_dres=FAR),
                                    dict(h=0, ld_h=FAR, h_ckpt=(0x9000, 0x9100)),
                                    dict(branch=0, ld_branch=-1, branch_ckpt=(0x9200, 0x9300)),
                                    dict(branch=0, ld_branch=FAR, branch_ckpt=(0x9200, 0x9300)),
                                    dict(gamma_post=0, dgamma_post=0, rstd_branch=0xF002)])
def test_backward(lib, unused):                        # noqa: F811
    assert _bwd(lib, ws=None, **unused) == WORKSPACE


def test_backward_still_checks_what_it_reads(lib):     # noqa: F811
    for f in ("ld_dy", "ld_dres", "ld_h", "ld_branch"):
        assert _bwd(lib, ws=None, **{f: FAR}) == SHAPE
    assert _bwd(lib, ws=None, rstd_branch=0) == NULL


def test_forward(lib):                                 # noqa: F811
    for rstd_o in (0xC102, 0xC000):                    # misaligned, and rstd's own
        assert _branch(lib, rstd=0xC000, rstd_o=rstd_o) in (ALIGN, SHAPE)
        # nothing refused: there is no GPU to run it
        assert _branch(lib, rstd=0xC000, rstd_o=rstd_o, gamma_post=0) == CUDA
    none = dict(rows=0, wr=0, wc=0, y=0xE000)
    assert _branch(lib, ld_branch=FAR, ld_residual=FAR, **none) == 0       # nothing to read
