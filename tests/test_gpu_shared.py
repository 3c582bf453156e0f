"""GPU shared-prefix decode vs the fp64 oracle on identical cache bytes: the
decode's bound (max-abs 2e-3, mean-abs 2e-4), since both phases carry the
decode's operand precision."""
import numpy as np
import pytest
import torch

import oracle
from kvq_cases import ALL_FORMATS, assert_decode_close, decode_case
from quantized_paged_kv_reshape_gb300 import _abi, ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def shared_case(fmt, plens, sizes, lens, nq, nkv, hd, bs=16, seed=0, tail=0):
    """decode_case whose first len(plens) rows are the prefixes; `sizes` members
    per group, `tail` sequences behind the last group."""
    assert sum(sizes) + tail == len(lens)
    c = decode_case(fmt, list(plens) + list(lens), nq, nkv, hd, bs=bs, seed=seed)
    g = len(plens)
    c["cu"] = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    w = lambda t, n: np.ascontiguousarray(t[:, :max(1, max([-(-int(x) // bs) for x in n] or [1]))])
    c["ptab"], c["plens"] = w(c["tables"][:g], c["lens"][:g]), c["lens"][:g]
    c["stab"], c["slens"] = w(c["tables"][g:], c["lens"][g:]), c["lens"][g:]
    c["q"] = c["q"][g:]
    return c


def dev(c):
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return dict(kp=t(c["kc"].reshape(c["num_blocks"], c["kst"])), vp=t(c["vc"].reshape(c["num_blocks"], c["vst"])),
                ptab=t(c["ptab"]), plens=t(c["plens"]), cu=t(c["cu"]), stab=t(c["stab"]), slens=t(c["slens"]), q=t(c["q"]))


def run(c, d, **kw):
    return ops.paged_decode_shared(kw.pop("q", d["q"]), d["kp"], d["vp"], d["ptab"], d["plens"], d["cu"], d["stab"],
                                   d["slens"], c["fmt"], c["nkv"], c["bs"], k_scale=c["k_scale"],
                                   v_scale=c["v_scale"], **kw)


def ref(c, window=0, q=None):
    return oracle.paged_decode_shared(c["q"] if q is None else q, c["kc"], c["vc"], c["ptab"], c["plens"], c["cu"],
                                      c["stab"], c["slens"], c["nkv"], c["hd"], c["bs"], c["kst"], c["vst"], c["fmt"],
                                      k_scale=c["k_scale"], v_scale=c["v_scale"], window=window)


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("hd,nq,nkv", [(64, 4, 2), (128, 8, 2), (256, 4, 2), (128, 8, 1)])
def test_shared_parity(fmt, hd, nq, nkv):
    c = shared_case(fmt, [100, 37], [3, 2], [5, 0, 33, 1, 70], nq, nkv, hd, seed=hd + nq)
    assert_decode_close(host(run(c, dev(c))), ref(c))


@pytest.mark.parametrize("plens,sizes,lens,tail", [
    ([0], [3], [4, 5, 6], 0),                       # an empty prefix
    ([50, 0, 7], [2, 0, 1], [0, 9, 3], 0),          # an empty group
    ([33], [1], [0], 0),                            # prefix only
    ([0], [2], [0, 5], 0),                          # a row with nothing to attend
    ([40], [2], [3, 4, 5, 0], 2),                   # sequences in no group
    ([1], [40], [1] * 40, 0),                       # one position, several tiles of members
    ([700, 5, 64], [35, 1, 33], [3] * 69, 0),       # groups over tile edges
    ([20] * 40, [1] * 40, [2] * 40, 0)])            # more groups than one look holds
def test_shared_shapes(plens, sizes, lens, tail):
    for fmt in ("bf16", "turbo4"):
        c = shared_case(fmt, plens, sizes, lens, 8, 2, 128, seed=len(lens), tail=tail)
        assert_decode_close(host(run(c, dev(c))), ref(c))


@pytest.mark.parametrize("nq,nkv", [(2, 2), (3, 1), (6, 2), (5, 1), (8, 1)])
def test_shared_gqa(nq, nkv):
    c = shared_case("fp8", [130, 60], [20, 3], list(range(23)), nq, nkv, 128, seed=nq)
    assert_decode_close(host(run(c, dev(c))), ref(c))


@pytest.mark.parametrize("fmt", ["bf16", "fp8k_turbo2v", "turbo4k_turbo3v", "turbo8"])
@pytest.mark.parametrize("window", [1, 4, 30, 90, 500])
def test_shared_window(fmt, window):
    """Windows that end in the own positions, cut the prefix, or cover all."""
    c = shared_case(fmt, [100, 70], [3, 2], [5, 0, 33, 1, 64], 8, 2, 128, seed=window)
    assert_decode_close(host(run(c, dev(c), sliding_window=window)), ref(c, window))


@pytest.mark.parametrize("bs", [8, 32])
@pytest.mark.parametrize("hd", [64, 256])
def test_shared_block_sizes(bs, hd):
    c = shared_case("bf16k_turbo4v", [99], [4], [1, 17, 40, 8], 4, 2, hd, bs=bs, seed=bs)
    assert_decode_close(host(run(c, dev(c))), ref(c))


def test_shared_equals_unshared_decode():
    """Whole-page prefixes: the plain decode over joined tables agrees."""
    c = shared_case("turbo4", [512], [5], [40, 1, 300, 16, 77], 32, 8, 128, seed=8)
    d = dev(c)
    got = run(c, d)
    joined = torch.cat([d["ptab"].expand(5, -1), d["stab"]], 1).contiguous()
    plain = ops.paged_decode(d["q"], d["kp"], d["vp"], joined, d["slens"] + 512, "turbo4", 8, 16)
    assert (got - plain).abs().max() <= 2e-3


def test_shared_bf16_io():
    c = shared_case("fp8", [200], [6], [3, 9, 0, 64, 1, 5], 8, 2, 128, seed=12)
    d = dev(c)
    qb = d["q"].to(torch.bfloat16)
    got = host(run(c, d, q=qb, out_dtype=torch.bfloat16))
    want = ref(c, q=host(qb.float()))
    assert (np.abs(got - want) <= 2e-3 + 2.0 ** -8 * np.abs(want)).all()


def test_shared_masked_rows_of_pages_never_enter():
    """NaN bytes behind the prefix's end, behind the own end, and before a
    window's start do not reach the rows that do not attend to them."""
    c = shared_case("bf16", [100], [2], [20, 90], 4, 2, 128, seed=13)
    d = dev(c)
    want, wantw = run(c, d), run(c, d, sliding_window=60)
    rows = lambda p, blk, off: p.view(torch.bfloat16).view(-1, 16, 2, 128)[blk, off]
    for p in (d["kp"], d["vp"]):
        rows(p, int(c["ptab"][0, 6]), slice(4, 16)).fill_(float("nan"))      # positions 100 .. 111
        rows(p, int(c["stab"][0, 1]), slice(4, 16)).fill_(float("nan"))      # own positions 20 .. 31
    assert torch.equal(run(c, d), want)
    assert torch.equal(run(c, d, sliding_window=60), wantw)
    for p in (d["kp"], d["vp"]):
        rows(p, int(c["ptab"][0, 3]), slice(0, 16)).fill_(float("inf"))      # positions 48 .. 63
    got = run(c, d, sliding_window=60)    # sequence 0 attends from 60 on, sequence 1 to no prefix position
    assert torch.equal(got[1], wantw[1])
    assert not torch.isfinite(got[0]).all()
    got = run(c, d, sliding_window=50)    # 70 on
    assert torch.isfinite(got).all()


def test_shared_window_edge_with_nonfinite_values():
    """Members of one tile whose windows start at different prefix positions:
    an infinite value one attends to stays out of the others' rows."""
    c = shared_case("bf16", [64], [3], [1, 10, 30], 4, 2, 128, seed=14)
    d = dev(c)
    want = run(c, d, sliding_window=50)   # starts 15, 24, 44
    for p in (d["kp"], d["vp"]):
        p.view(torch.bfloat16).view(-1, 16, 2, 128)[int(c["ptab"][0, 1]), 4].fill_(float("nan"))   # position 20
    got = run(c, d, sliding_window=50)
    # the step that holds the value is added in another order: each of the two
    # sums over n = 94 positions at most rounds by (n + 2) u sum p|v| <= (n + 2) u max|v|
    # relative to the unit sum of p, u = 2^-24
    assert (got[1:] - want[1:]).abs().max() <= 2 * 96 * 2.0 ** -24 * np.abs(c["v"]).max()
    assert not torch.isfinite(got[0]).any()


def test_shared_bad_pages_are_flagged():
    c = shared_case("turbo4", [60], [3], [20, 5, 9], 8, 2, 128, seed=15)
    for tab, row, col, val in (("ptab", 0, 1, -1), ("ptab", 0, 2, 9999), ("stab", 1, 0, 9999)):
        d = dev(c)
        d[tab][row, col] = val
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = run(c, d, error_flag=err)
        torch.cuda.synchronize()
        assert err.item() & _abi.KVQ_DEVERR_BLOCK
        assert torch.isfinite(out).all()


def test_shared_workspace_any_content_and_reuse():
    """The workspace may hold anything; one serves calls of other shapes."""
    a = shared_case("turbo4", [300, 90], [9, 8], [1 + 7 * i for i in range(17)], 8, 2, 128, seed=16)
    b = shared_case("bf16", [40], [3], [3, 2, 100], 4, 4, 64, seed=17)
    size = max(ops.shared_workspace_bytes(17, 2, 8, 2, 128, 16, a["ptab"].shape[1], a["stab"].shape[1], 0, "turbo4"),
               ops.shared_workspace_bytes(3, 1, 4, 4, 64, 16, b["ptab"].shape[1], b["stab"].shape[1], 0, "bf16"))
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)
    for c in (a, b, a):
        d = dev(c)
        assert_decode_close(host(run(c, d, workspace=ws)), ref(c))


def test_shared_streams_and_graphs():
    c = shared_case("turbo4", [333], [6], [3, 9, 0, 64, 1, 5], 8, 2, 128, seed=18)
    d = dev(c)
    want = run(c, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on = run(c, d, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(on, want)
    out = torch.empty_like(want)
    ws = ops.alloc_shared_workspace(6, 1, 8, 2, 128, 16, d["ptab"].shape[1], d["stab"].shape[1], 0, "turbo4")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c, d, out=out, workspace=ws)
    q2 = torch.randn_like(d["q"])
    want2 = run(c, d, q=q2)
    for q, w in ((q2, want2), (torch.from_numpy(c["q"]).to(DEV), want)):
        d["q"].copy_(q)
        g.replay()
        assert torch.equal(out, w)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("hd,nq,nkv", [(64, 6, 2), (128, 8, 1), (256, 4, 2)])
def test_shared_window_edge_with_nonfinite_values_of_many_members(fmt, hd, nq, nkv):
    """Members of a tile whose windows start on either side of a position with
    a NaN value: their rows differ in what they add, lane by lane."""
    own = [1 + 3 * i for i in range(11)]
    c = shared_case(fmt, [130], [11], own, nq, nkv, hd, seed=hd)
    d = dev(c)
    window = 100                          # starts 130 + own - 100: 31, 34, ..., 61
    want = run(c, d, sliding_window=window)
    pos, bs = 45, 16
    row = d["vp"][int(c["ptab"][0, pos // bs])]
    size = nkv * hd * (2 if fmt == "bf16" else 1)
    bad = torch.tensor([0xFF, 0x7F], dtype=torch.uint8, device=DEV) if fmt == "bf16" else \
        torch.tensor([0x7F], dtype=torch.uint8, device=DEV)
    row[pos % bs * size:(pos % bs + 1) * size] = bad.repeat(size // bad.numel())
    got = run(c, d, sliding_window=window)
    sees = torch.tensor([30 + n <= pos for n in own], device=DEV)
    assert torch.isnan(got[sees]).all()
    # the step with the value is added in another order, and from weights in two
    # 16-bit parts (2^-16 of a weight at most) as the products': sums of n terms
    # each, (n + 2) 2^-24 max|v|
    n = 130 + max(own)
    assert (got[~sees] - want[~sees]).abs().max() <= 2 * (n + 2) * 2.0 ** -24 * np.abs(c["v"]).max()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bs", [8, 16])
def test_shared_pages_freed_before_the_window(hd, bs):
    """Pages that lie wholly before every member's window may be gone from the
    table: no flag, no difference.  One inside it is flagged."""
    c = shared_case("bf16k_turbo4v", [100], [2], [20, 28], 8, 2, hd, bs=bs, seed=19)
    d = dev(c)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = run(c, d, sliding_window=60, error_flag=err)   # from positions 60 and 68 on
    d["ptab"][0, :60 // bs] = -1
    got = run(c, d, sliding_window=60, error_flag=err)
    assert err.item() == 0
    assert torch.equal(got, want)
    d["ptab"][0, 60 // bs] = -1
    run(c, d, sliding_window=60, error_flag=err)
    assert err.item() == _abi.KVQ_DEVERR_BLOCK


@pytest.mark.parametrize("cu,like", [([0, 4, 2, 6], None), ([2, 1, 6, 6], None), ([0, 6, 5, 4], None),
                                     ([-3, 2, 4, 6], [0, 2, 4, 6]), ([0, 2, 4, 99], [0, 2, 4, 6])])
def test_shared_bad_groups_are_flagged(cu, like):
    """Offsets outside the batch are cut; a decreasing one leaves the prefixes
    out: the result is that of the sequences' own positions."""
    c = shared_case("fp8", [300, 64, 200], [2, 2, 2], [5, 0, 33, 1, 70, 9], 8, 2, 128, seed=20)
    d = dev(c)
    d["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full((ops.shared_workspace_bytes(6, 3, 8, 2, 128, 16, d["ptab"].shape[1], d["stab"].shape[1], 0, "fp8"),),
                    0x7E, dtype=torch.uint8, device=DEV)
    got = run(c, d, workspace=ws, error_flag=err)
    assert err.item() == _abi.KVQ_DEVERR_RANGE
    if like is None:
        want = ops.paged_decode(d["q"], d["kp"], d["vp"], d["stab"], d["slens"], "fp8", 2, 16, k_scale=c["k_scale"],
                                v_scale=c["v_scale"])
    else:
        d["cu"].copy_(torch.tensor(like, dtype=torch.int32))
        err.zero_()
        want = run(c, d, error_flag=err)
        assert err.item() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4", "fp8k_turbo2v"])
@pytest.mark.parametrize("factor", [2.0 ** 17, 2.0 ** -20])
def test_shared_query_magnitudes(fmt, factor):
    """BF16 queries past the range of fp16, above and below, with a score scale
    that brings the scores back: the same scores, the same result."""
    c = shared_case(fmt, [300, 37], [3, 2], [5, 0, 33, 1, 70], 8, 2, 128, seed=21)
    q = torch.from_numpy(c["q"]).to(torch.bfloat16)
    scale = 128 ** -0.5
    want = oracle.paged_decode_shared(host(q), c["kc"], c["vc"], c["ptab"], c["plens"], c["cu"], c["stab"], c["slens"],
                                      2, 128, 16, c["kst"], c["vst"], fmt, k_scale=c["k_scale"], v_scale=c["v_scale"],
                                      sm_scale=scale)
    got = run(c, dev(c), q=(q.float() * factor).to(torch.bfloat16).to(DEV), sm_scale=scale / factor)
    assert_decode_close(host(got), want)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("hd,nq,nkv", [(64, 4, 2), (128, 8, 2), (256, 4, 2)])
def test_shared_bf16_io_formats(fmt, hd, nq, nkv):
    """BF16 queries and outputs (other operand forms than fp32 ones), several
    ranges of the prefix: the decode's bound and half a step of the output."""
    c = shared_case(fmt, [700, 90], [3, 2], [5, 0, 33, 1, 70], nq, nkv, hd, seed=hd + 1)
    d = dev(c)
    qb = d["q"].to(torch.bfloat16)
    want = ref(c, q=host(qb))
    got = host(run(c, d, q=qb, out_dtype=torch.bfloat16))
    assert (np.abs(got - want) <= 2e-3 + 2.0 ** -8 * np.abs(want)).all()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", [True, False])
def test_shared_small_weights_add_up(out_dtype, first):
    """One position with nearly all of the weight and a zero value, 4095 with
    2^-26 of it each and a value of 256: all of the output comes from the small
    ones.  K and V are exact in FP8 and the scores exact in fp32.

    A weight is held in fp16 parts, 2^7 above its size beside the row's maximum:
    half a step of a subnormal is 2^-25, hence off by at most 2^-32, or 2^-12 of
    itself in two parts of 11 bits; 2^-18 covers exp2 and the sums, 2^-8 of the
    result a BF16 output."""
    n, groups, nq, nkv, hd, bs = 4096, 8, 8, 8, 64, 16
    k = torch.zeros(n, nkv, hd, device=DEV)
    v = torch.full((n, nkv, hd), 256.0, device=DEV)
    one = 0 if first else n - 1
    k[one, :, 0], v[one] = 1.0, 0.0
    kp, vp = (ops.alloc_pool(n // bs + 1, "fp8", side, bs, nkv, hd) for side in (0, 1))
    ops.cache_write(k, v, kp, vp, torch.arange(n, device=DEV), "fp8", nkv, hd, bs)
    q = torch.zeros(groups, nq, hd, device=DEV, dtype=torch.bfloat16)
    q[:, :, 0] = 26.0
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    tab = torch.arange(n // bs, dtype=torch.int32, device=DEV).expand(groups, -1).contiguous()
    out = ops.paged_decode_shared(q, kp, vp, tab, i(*[n] * groups), i(*range(groups + 1)), i(*[0] * groups)[:, None].contiguous(),
                                  i(*[0] * groups), "fp8", nkv, bs, out_dtype=out_dtype, sm_scale=float(np.log(2.0)))
    w = 2.0 ** -26 * (n - 1)
    want = 256.0 * w / (1 + w)
    tol = 256.0 * n * 2.0 ** -32 + want * (2.0 ** -12 + 2.0 ** -18 + (2.0 ** -8 if out_dtype == torch.bfloat16 else 0))
    assert np.abs(host(out) - want).max() <= tol


@pytest.mark.parametrize("fmt", ["fp8", "turbo4", "nvfp4", "bf16"])
def test_shared_bf16_outputs_are_the_fp32_ones_rounded(fmt):
    """The type of the output changes its own rounding alone."""
    c = shared_case(fmt, [700, 90], [3, 2], [5, 0, 33, 1, 70], 8, 2, 128, seed=23)
    d = dev(c)
    for q in (d["q"], d["q"].to(torch.bfloat16)):
        assert torch.equal(run(c, d, q=q, out_dtype=torch.bfloat16), run(c, d, q=q).to(torch.bfloat16))
