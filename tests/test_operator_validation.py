"""CPU checks of the C entry points of the block norm, the balance loss and the expert products: invalid arguments
are refused on the host before any HIP call, and calls with nothing to do return MOE_OK."""
import pytest

from moe_routing_fp8_amd import _native

INVALID, UNSUPPORTED, WS_SMALL = 1, 2, 3
FAKE = 0x10000  # a non-null, 256-byte aligned address never dereferenced on the host
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return _native.lib()


def _caller(fn, names, ok):
    def call(**kw):
        args = dict(zip(names, ok))
        args.update(kw)
        assert len(args) == len(names), set(args) - set(names)
        return fn(*args.values())
    return call


def test_block_norm(lib):
    names = ["r", "rs", "rd", "y", "ys", "ad", "T", "H", "pw", "gate", "mode", "scale", "nw", "eps", "out", "normed",
             "post", "pre", "stream"]
    call = _caller(lib.moe_block_norm, names, [FAKE, 64, 0, FAKE, 64, 0, 4, 64, FAKE, FAKE, 1, 1.0, FAKE, 1e-6, FAKE,
                                               FAKE, FAKE, FAKE, None])
    assert call(T=-1) == INVALID and call(H=0) == INVALID
    assert call(rd=2) == INVALID and call(ad=-1) == INVALID
    assert call(mode=3) == INVALID and call(mode=0) == INVALID and call(gate=None) == INVALID
    assert call(eps=-1e-9) == INVALID and call(eps=NAN) == INVALID and call(scale=NAN) == INVALID
    assert call(rs=63) == INVALID and call(ys=63) == INVALID
    assert call(r=None) == INVALID and call(out=None) == INVALID and call(y=None) == INVALID
    assert call(normed=None) == INVALID and call(nw=None) == INVALID
    assert call(normed=None, nw=None) == INVALID                       # pre_rstd without its norm
    assert call(pw=None) == INVALID                                    # post_rstd without its norm
    assert call(r=FAKE + 1) == INVALID and call(rd=1, r=FAKE + 2) == INVALID and call(nw=FAKE + 2) == INVALID
    assert call(y=FAKE + 1) == INVALID and call(post=FAKE + 1) == INVALID
    # without a block: only the norm before the next one
    only = dict(y=None, out=None, pw=None, post=None, gate=None, mode=0)
    assert call(**only, scale=0.5) == INVALID and call(**{**only, "pw": FAKE}) == INVALID
    assert call(**only, normed=None, nw=None, pre=None) == INVALID     # nothing to compute
    assert call(H=16385, rs=20000, ys=20000) == UNSUPPORTED and call(T=(1 << 22) + 1) == UNSUPPORTED
    assert call(T=0, r=None, y=None, out=None, normed=None) == 0


def test_block_norm_backward(lib):
    need = lib.moe_block_norm_backward_workspace_bytes(4, 64)
    assert need > 0 and need % 256 == 0
    assert lib.moe_block_norm_backward_workspace_bytes(-1, 64) == 0
    assert lib.moe_block_norm_backward_workspace_bytes(4, 0) == 0
    assert lib.moe_block_norm_backward_workspace_bytes(4, 16385) == 0
    names = ["dr", "dn", "out", "outs", "rd", "y", "ys", "ad", "T", "H", "pw", "gate", "mode", "scale", "nw", "post",
             "pre", "gr", "gy", "gpw", "gg", "gnw", "ws", "wsb", "stream"]
    call = _caller(lib.moe_block_norm_backward, names,
                   [FAKE, FAKE, FAKE, 64, 0, FAKE, 64, 0, 4, 64, FAKE, FAKE, 1, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                    FAKE, FAKE, FAKE, need, None])
    assert call(T=-1) == INVALID and call(H=0) == INVALID and call(rd=2) == INVALID and call(ad=3) == INVALID
    assert call(mode=0) == INVALID and call(gg=None) == INVALID and call(gpw=None) == INVALID
    assert call(gnw=None) == INVALID and call(scale=NAN) == INVALID
    assert call(outs=63) == INVALID and call(ys=63) == INVALID
    for k in ("dn", "out", "y", "post", "pre", "gr", "gy"):
        assert call(**{k: None}) == INVALID, k
    assert call(nw=None, gnw=None) == INVALID                          # grad_normed without its weight
    assert call(nw=None, gnw=None, dn=None, pre=None, dr=None) == INVALID  # no gradient at all
    assert call(y=None, gy=None) == INVALID                            # a gate without a block
    assert call(dr=FAKE + 1) == INVALID and call(gy=FAKE + 1) == INVALID and call(pre=FAKE + 2) == INVALID
    assert call(ws=None) == INVALID and call(ws=FAKE + 64) == INVALID
    assert call(wsb=need - 1) == WS_SMALL
    assert call(H=16385, outs=20000, ys=20000) == UNSUPPORTED and call(T=(1 << 22) + 1) == UNSUPPORTED
    nothing = dict(T=0, pw=None, gpw=None, gate=None, gg=None, mode=0, nw=None, gnw=None, dn=None)
    assert call(**nothing) == 0


def test_balance_loss(lib):
    f = lib.moe_balance_loss_workspace_bytes
    need = f(100, 16, 3)
    assert need > 0 and need % 256 == 0 and f(0, 16, 1) > 0
    assert f(-1, 16, 1) == 0 and f(10, 0, 1) == 0 and f(10, 1025, 1) == 0 and f(10, 16, 0) == 0
    assert f(10, 16, 65537) == 0 and f(1 << 28, 16, 1) == 0
    names = ["z", "zd", "zs", "T", "E", "score", "idx", "K", "mask", "off", "S", "loss", "counts", "n", "mean", "ws",
             "wsb", "stream"]
    call = _caller(lib.moe_balance_loss, names, [FAKE, 1, 16, 100, 16, 0, FAKE, 2, None, FAKE, 3, FAKE, FAKE, FAKE, FAKE,
                                                 FAKE, need, None])
    assert call(T=-1) == INVALID and call(E=0) == INVALID and call(E=1025, zs=1025) == INVALID
    assert call(K=0) == INVALID and call(K=17) == INVALID and call(T=1 << 28) == INVALID
    assert call(S=0) == INVALID and call(S=65537) == INVALID and call(off=None) == INVALID
    assert call(zd=2) == INVALID and call(score=2) == INVALID and call(zs=15) == INVALID
    for k in ("z", "idx", "loss", "counts", "n", "ws"):
        assert call(**{k: None}) == INVALID, k
    for k in ("z", "idx", "loss", "counts", "n", "mean", "off"):
        assert call(**{k: FAKE + 2}) == INVALID, k
    assert call(ws=FAKE + 64) == INVALID and call(wsb=need - 1) == WS_SMALL
    names = ["dl", "z", "zd", "zs", "T", "E", "score", "K", "mask", "off", "S", "counts", "n", "grad", "stream"]
    call = _caller(lib.moe_balance_loss_backward, names,
                   [FAKE, FAKE, 1, 16, 100, 16, 0, 2, None, FAKE, 3, FAKE, FAKE, FAKE, None])
    assert call(T=-1) == INVALID and call(E=0) == INVALID and call(K=17) == INVALID and call(off=None) == INVALID
    for k in ("dl", "z", "counts", "n", "grad"):
        assert call(**{k: None}) == INVALID and call(**{k: FAKE + 2}) == INVALID, k
    assert call(T=0, dl=None, z=None, counts=None, n=None, grad=None) == 0


def test_expert_matvec(lib):
    names = ["x", "xd", "xsf", "X", "tok", "R", "K", "N", "E", "off", "w", "sf", "g", "ue8m0", "out", "stream"]
    call = _caller(lib.moe_expert_matvec, names, [FAKE, 0, None, 5, None, 5, 256, 20, 2, FAKE, FAKE, FAKE, 32, 1, FAKE,
                                                  None])
    assert call(R=-1) == INVALID and call(X=-1) == INVALID and call(R=1 << 31) == INVALID
    assert call(X=4) == INVALID                                         # no row_token: one x row for each row
    assert call(xd=1) == INVALID and call(xd=3) == INVALID
    assert call(E=0) == INVALID and call(E=1025) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID
    assert call(ue8m0=2) == INVALID and call(off=None) == INVALID
    assert call(g=16) == UNSUPPORTED and call(g=64) == UNSUPPORTED
    assert call(K=240) == INVALID and call(K=160, g=128) == INVALID
    assert call(K=160, xd=2, xsf=FAKE) == INVALID                       # e4m3 rows: scales of 128
    assert call(xd=2) == INVALID and call(xsf=FAKE) == INVALID          # x_sf goes with e4m3 rows
    assert call(N=(1 << 20) + 1) == UNSUPPORTED and call(K=(1 << 20) + 128) == UNSUPPORTED
    for k in ("x", "w", "sf", "out"):
        assert call(**{k: None}) == INVALID, k
    assert call(x=FAKE + 8) == INVALID and call(w=FAKE + 8) == INVALID and call(out=FAKE + 1) == INVALID
    assert call(sf=FAKE + 2, ue8m0=0) == INVALID and call(off=FAKE + 2) == INVALID and call(tok=FAKE + 1) == INVALID
    assert call(R=0, X=0, x=None, w=None, sf=None, out=None, off=FAKE) == 0


def test_no_rows_by_token(lib):
    """An empty row_token has no address: no rows, though x has some."""
    names = ["x", "xd", "xsf", "X", "tok", "R", "K", "N", "E", "off", "w", "sf", "g", "ue8m0", "out", "stream"]
    call = _caller(lib.moe_expert_matvec, names, [FAKE, 0, None, 5, None, 0, 256, 20, 2, FAKE, FAKE, FAKE, 32, 1, None,
                                                  None])
    assert call() == 0 and call(tok=FAKE) == 0
    assert call(xd=2, xsf=FAKE) == 0
    assert call(g=16) == UNSUPPORTED and call(K=240) == INVALID and call(off=None) == INVALID


def test_no_tokens_with_a_token_gate(lib):
    """A gate per token of a batch without tokens has no address."""
    names = ["r", "rs", "rd", "y", "ys", "ad", "T", "H", "pw", "gate", "mode", "scale", "nw", "eps", "out", "normed",
             "post", "pre", "stream"]
    call = _caller(lib.moe_block_norm, names, [None, 64, 0, None, 64, 0, 0, 64, FAKE, None, 2, 1.0, FAKE, 1e-6, None,
                                               None, None, None, None])
    assert call() == 0 and call(gate=FAKE) == 0 and call(pw=None) == 0
    assert call(mode=1) == INVALID and call(mode=0, gate=FAKE) == INVALID and call(T=4) == INVALID
    names = ["dr", "dn", "out", "outs", "rd", "y", "ys", "ad", "T", "H", "pw", "gate", "mode", "scale", "nw", "post",
             "pre", "gr", "gy", "gpw", "gg", "gnw", "ws", "wsb", "stream"]
    call = _caller(lib.moe_block_norm_backward, names,
                   [None, None, None, 64, 0, None, 64, 0, 0, 64, None, None, 2, 1.0, None, None, None, None, None, None,
                    None, None, None, 0, None])
    assert call() == 0 and call(gate=FAKE, gg=FAKE) == 0
    assert call(mode=1) == INVALID and call(mode=1, gate=FAKE) == INVALID and call(mode=0, gate=FAKE) == INVALID
    assert call(T=4) == INVALID
