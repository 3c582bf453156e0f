"""GPU attention mass, selection and compaction vs the oracle.

Mass bound: with u = 2^-24, q and K carry at least 21 bits (a relative 2^-20
for both) and a dot product of hd terms adds (hd + 2) u, so a base-2 score is
off by d = scale2 max sum|q k| (2^-20 + (hd + 4) u); a weight and its row's
sum each by a relative 2 d + 2^-20 (exp2 and the sums' joins), and a position
adds up `rows` weights: |err| <= w (4 d + 2^-18) + u (|mass_in| + w) (rows + 2)
with w the oracle's weight.  Selection and compaction are exact."""
import math

import numpy as np
import pytest
import torch

import oracle
from kvq_cases import ALL_FORMATS, decode_case
from quantized_paged_kv_reshape_gb300 import _abi, ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
K_FORMATS = ["bf16", "fp8", "nvfp4", "turbo4", "turbo3", "turbo2", "turbo8"]


def t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def host(x):
    return x.double().cpu().numpy()


def pools(c):
    return t(c["kc"].reshape(c["num_blocks"], c["kst"])), t(c["vc"].reshape(c["num_blocks"], c["vst"]))


def check_mass(fmt, lens, chunks, nq, nkv, hd, bs=16, window=0, seed=0, q_dtype=torch.float32, scale=0.0):
    c = decode_case(fmt, lens, nq, nkv, hd, bs=bs, seed=seed)
    rng = np.random.default_rng(seed + 7)
    cu = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    q = t(rng.standard_normal((int(cu[-1]), nq, hd)).astype(np.float32)).to(q_dtype)
    width = max(max(lens), 1)
    prev = t(rng.random((len(lens), nkv, width)).astype(np.float32))
    out = torch.full_like(prev, 5.0)
    kp, _ = pools(c)
    ops.attention_mass(q, t(cu), max(max(chunks), 1), kp, t(c["tables"]), t(c["lens"]), fmt, nkv, bs, mass_in=prev,
                       mass_out=out, k_scale=c["k_scale"], sliding_window=window, sm_scale=scale)
    w = oracle.attention_mass(host(q), cu, c["kc"], c["tables"], c["lens"], nkv, hd, bs, c["kst"], fmt, width,
                              k_scale=c["k_scale"], window=window, sm_scale=scale)
    rows = max(chunks) * nq // nkv
    qk = 0.0
    for s, n in enumerate(lens):
        if n and cu[s + 1] > cu[s]:
            k = oracle.gather_side(c["kc"], oracle.kv_pair(fmt)[0], c["tables"][s, np.arange(n) // bs], np.arange(n) % bs,
                                   nkv, hd, bs, c["kst"], c["k_scale"], to_original_basis=False)
            qs = host(q)[cu[s]:cu[s + 1]]
            if oracle.is_wht_rotated(oracle.kv_pair(fmt)[0]):
                qs = oracle.wht_f64(qs)
            for j in range(nq):
                qk = max(qk, (np.abs(qs[:, j]) @ np.abs(k[:, j // (nq // nkv)]).T).max())
    u = 2.0 ** -24
    d = (abs(scale) or 1 / math.sqrt(hd)) * math.log2(math.e) * qk * (2.0 ** -20 + (hd + 4) * u)
    tol = w * (4 * d + 2.0 ** -18) + u * (host(prev) + w) * (rows + 2)
    for s, n in enumerate(lens):
        assert (np.abs(host(out)[s, :, :n] - (host(prev) + w)[s, :, :n]) <= tol[s, :, :n]).all()
        assert (out[s, :, n:] == 5.0).all()      # behind the sequence's end nothing is written


LENS, CHUNKS = [37, 50, 1, 300, 129, 16, 3], [5, 50, 1, 64, 129, 0, 5]


@pytest.mark.parametrize("fmt", K_FORMATS)
@pytest.mark.parametrize("hd,nq,nkv", [(64, 4, 2), (128, 8, 2), (256, 4, 2), (128, 8, 1)])
def test_mass_chunks(fmt, hd, nq, nkv):
    check_mass(fmt, LENS, CHUNKS, nq, nkv, hd, seed=hd + nq)


@pytest.mark.parametrize("fmt", K_FORMATS)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (4, 1), (8, 1), (6, 2)])
def test_mass_single_queries(fmt, hd, nq, nkv):
    lens = [1, 2, 127, 128, 129, 500, 0, 17]
    check_mass(fmt, lens, [1, 1, 1, 1, 1, 1, 0, 1], nq, nkv, hd, seed=hd + nq, q_dtype=torch.bfloat16)


@pytest.mark.parametrize("fmt", ["bf16", "turbo4"])
@pytest.mark.parametrize("window", [1, 5, 64, 130, 1000])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_mass_window(fmt, window, bs):
    check_mass(fmt, [300, 64, 7], [40, 64, 1], 8, 2, 128, bs=bs, window=window, seed=window)
    check_mass(fmt, [300, 64, 7], [1, 1, 1], 8, 2, 64, bs=bs, window=window, seed=window + 1)


def test_mass_long_rows_and_scale():
    check_mass("turbo4", [5000, 3], [2, 1], 8, 2, 128, seed=2)
    check_mass("bf16", [9001], [1], 4, 1, 128, seed=3, q_dtype=torch.bfloat16)
    check_mass("fp8", [700], [3], 4, 2, 64, seed=4, scale=0.3)
    for scale in (0.3, -0.2):                          # few and many score rows
        check_mass("turbo4", [300, 17], [1, 1], 8, 2, 128, seed=5, scale=scale)
        check_mass("bf16", [300, 170], [40, 9], 8, 2, 128, seed=6, scale=scale)


def test_mass_many_sequences():
    """More (sequence, kv head) rows than CTAs fit at once; row blocks of 128."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 200, 90)]
    check_mass("fp8", lens, [min(n, 5) for n in lens], 16, 4, 64, seed=7)
    check_mass("turbo3", [260, 40], [260, 40], 8, 1, 128, seed=8)


def test_mass_adds_up_and_defaults():
    """In place, without a start, and over a decode's steps: rows sum to the heads."""
    c = decode_case("turbo4", [200, 77], 8, 2, 128, seed=5)
    kp, _ = pools(c)
    q = t(c["q"])
    cu = t(np.array([0, 1, 2], np.int32))
    args = (q, cu, 1, kp, t(c["tables"]), t(c["lens"]), "turbo4", 2, 16)
    m = ops.attention_mass(*args)
    assert m.shape == (2, 2, c["tables"].shape[1] * 16)
    assert (m.sum(-1) - 4.0).abs().max() <= 1e-4        # 4 heads per kv head, weights sum to 1
    assert (m[1, :, 77:] == 0).all()
    twice = ops.attention_mass(*args, mass_in=m.clone(), mass_out=None)
    ip = m.clone()
    assert ops.attention_mass(*args, mass_in=ip, mass_out=ip) is ip
    assert torch.equal(ip, twice)
    assert (ip - 2 * m).abs().max() <= 1e-6


def test_mass_nonfinite_rows_stay_their_own():
    """A NaN key makes only the rows that attend to it NaN; masked ones do not matter."""
    c = decode_case("bf16", [200], 4, 2, 128, seed=6)
    kp, _ = pools(c)
    q = torch.randn(3, 4, 128, device=DEV)
    cu = t(np.array([0, 3], np.int32))
    args = lambda w: dict(q=q, cu_q=cu, max_chunk=3, k_cache=kp, block_tables=t(c["tables"]), seq_lens=t(c["lens"]),
                          fmt="bf16", num_kv_heads=2, block_size=16, sliding_window=w)
    want = ops.attention_mass(**args(50))
    kp.view(torch.bfloat16).view(-1, 16, 2, 128)[int(c["tables"][0, 0])].fill_(float("nan"))   # positions 0 .. 15
    assert torch.equal(ops.attention_mass(**args(50)), want)
    assert torch.isnan(ops.attention_mass(**args(0))).any()


def test_mass_flags():
    c = decode_case("turbo4", [100, 40], 4, 2, 64, seed=7)
    kp, _ = pools(c)
    q = torch.randn(6, 4, 64, device=DEV)
    tab, lens = t(c["tables"]), t(c["lens"])

    def flags(cu, mx, tab=tab, lens=lens, out=None):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        r = ops.attention_mass(q, t(np.array(cu, np.int32)), mx, kp, tab, lens, "turbo4", 2, 16, error_flag=err,
                               mass_out=out)
        assert torch.isfinite(r).all()
        return err.item()

    assert flags([0, 3, 6], 3) == 0
    assert flags([0, 3, 9], 6) == _abi.KVQ_DEVERR_RANGE
    assert flags([-2, 3, 6], 6) == _abi.KVQ_DEVERR_RANGE
    assert flags([0, 3, 6], 2) == _abi.KVQ_DEVERR_RANGE
    assert flags([0, 3, 6], 3, out=torch.zeros(2, 2, 50, device=DEV)) == _abi.KVQ_DEVERR_RANGE
    bad = tab.clone()
    bad[0, 2] = 9999
    assert flags([0, 3, 6], 3, tab=bad) == _abi.KVQ_DEVERR_BLOCK
    assert flags([0, 3, 6], 3, lens=lens + 1000) & _abi.KVQ_DEVERR_BLOCK


# ------------------------------------------------------------------ selection

def check_select(mass, lens, keep, sink=0, recent=0):
    kept, new = ops.evict_select(t(mass), t(np.array(lens, np.int32)), keep, sink=sink, recent=recent)
    rk, rn = oracle.evict_select(mass, lens, keep, sink, recent)
    assert np.array_equal(new.cpu().numpy(), rn)
    assert np.array_equal(kept.cpu().numpy(), rk)


@pytest.mark.parametrize("width,keep", [(1, 1), (5, 3), (64, 64), (64, 1), (1000, 999), (1000, 37), (4097, 512),
                                        (20000, 3001), (70001, 70000)])
def test_select_sizes(width, keep):
    rng = np.random.default_rng(width)
    mass = rng.random((3, 2, width)).astype(np.float32)
    check_select(mass, [width, max(0, width - 1), width // 2], keep)


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "signs", "nonfinite", "tiny", "close"])
def test_select_values(kind):
    rng = np.random.default_rng(1)
    n = 3001
    m = {"equal": lambda: np.full((2, 2, n), 0.25), "zeros": lambda: np.where(rng.random((2, 2, n)) < .5, 0.0, -0.0),
         "few": lambda: rng.integers(0, 5, (2, 2, n)) / 4, "signs": lambda: rng.standard_normal((2, 2, n)),
         "nonfinite": lambda: rng.choice([np.nan, np.inf, -np.inf, 0.0, 1.0], (2, 2, n)),
         "tiny": lambda: rng.random((2, 2, n)) * 1e-42,
         "close": lambda: 1 + rng.integers(0, 3, (2, 2, n)) * 2.0 ** -23}[kind]().astype(np.float32)
    for keep in (1, 100, 1500, 3000):
        check_select(m, [n, 2000], keep)
        check_select(m, [n, 2000], keep, sink=keep // 2, recent=keep - keep // 2)
        check_select(m, [n, 17], keep, sink=min(keep, 4))


def test_select_many_short_rows_and_one_long():
    rng = np.random.default_rng(2)
    check_select(rng.random((70, 8, 40)).astype(np.float32), list(rng.integers(0, 41, 70)), 20, 2, 5)
    check_select(rng.random((1, 1, 450001)).astype(np.float32), [450001], 1000, 4, 10)   # past the shared-memory cache


def test_select_flags_and_negative_lengths():
    m = np.random.default_rng(3).random((2, 1, 50)).astype(np.float32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept, new = ops.evict_select(t(m), t(np.array([60, -3], np.int32)), 10, error_flag=err)
    assert err.item() == _abi.KVQ_DEVERR_RANGE and new.tolist() == [10, 0]
    rk, _ = oracle.evict_select(m, [50, 0], 10)
    assert np.array_equal(kept.cpu().numpy(), rk)


# ------------------------------------------------------------------ compaction

def compact_case(fmt, lens, keep, nkv, hd, bs=16, seed=0):
    c = decode_case(fmt, lens, nkv, nkv, hd, bs=bs, seed=seed, spare=sum(-(-min(n, keep) // bs) for n in lens) + 2)
    rng = np.random.default_rng(seed + 3)
    kept = np.full((len(lens), nkv, keep), -1, np.int32)
    for s, n in enumerate(lens):
        k = min(n, keep)
        for h in range(nkv):
            kept[s, h, :k] = np.sort(rng.choice(n, k, replace=False)) if k else []
    free = np.setdiff1d(np.arange(c["num_blocks"]), c["tables"][c["tables"] >= 0])
    dst = np.full((len(lens), max(1, -(-keep // bs))), -1, np.int32)
    cur = 0
    for s, n in enumerate(lens):
        b = -(-min(n, keep) // bs)
        dst[s, :b] = free[cur:cur + b]
        cur += b
    c.update(kept=kept, dst=dst)
    return c


def check_compact(c, inplace):
    kp, vp = pools(c)
    width = c["tables"].shape[1] * c["bs"]
    mass = torch.rand(len(c["lens"]), c["nkv"], width, device=DEV)
    old = mass.cpu().numpy()
    out = mass if inplace else torch.full((len(c["lens"]), c["nkv"], c["kept"].shape[2]), 9.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.cache_compact(kp, vp, t(c["tables"]), t(c["lens"]), t(c["kept"]), c["fmt"], c["nkv"], c["hd"], c["bs"],
                      dst_tables=None if inplace else t(c["dst"]), mass=mass, mass_out=out, error_flag=err)
    rk, rv = oracle.cache_compact(c["fmt"], c["kc"], c["vc"], c["tables"], None if inplace else c["dst"], c["kept"],
                                  c["nkv"], c["hd"], c["bs"], c["kst"], c["vst"])
    assert err.item() == 0
    assert np.array_equal(kp.cpu().numpy().reshape(-1), rk)
    assert np.array_equal(vp.cpu().numpy().reshape(-1), rv)
    want = out.cpu().numpy().copy()
    for s in range(len(c["lens"])):
        for h in range(c["nkv"]):
            k = c["kept"][s, h][c["kept"][s, h] >= 0]
            want[s, h, :k.size] = old[s, h, k]
    assert np.array_equal(out.cpu().numpy(), want)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_compact_formats(fmt, hd, inplace):
    check_compact(compact_case(fmt, [90, 33, 0, 1, 16], 25, 3, hd, seed=hd), inplace)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("bs", [8, 32])
@pytest.mark.parametrize("keep", [1, 16, 200, 700])
def test_compact_sizes(bs, keep, inplace):
    check_compact(compact_case("turbo4k_turbo3v", [900, 640, 250], keep, 2, 128, bs=bs, seed=keep), inplace)


def test_compact_many_heads():
    check_compact(compact_case("turbo2", [40], 20, 150, 64, seed=1), False)
    check_compact(compact_case("turbo2", [40], 20, 150, 64, seed=1), True)


def test_compact_identity_and_holes():
    c = compact_case("fp8", [64, 64], 64, 2, 64, seed=2)      # everything kept
    check_compact(c, True)
    c = compact_case("fp8", [64, 64], 30, 2, 64, seed=3)
    c["kept"][0, 1, 5] = -1                                   # an entry that moves nothing
    kp, vp = pools(c)
    ops.cache_compact(kp, vp, t(c["tables"]), t(c["lens"]), t(c["kept"]), "fp8", 2, 64, 16, dst_tables=t(c["dst"]))
    rk, _ = oracle.cache_compact("fp8", c["kc"], c["vc"], c["tables"], c["dst"], c["kept"], 2, 64, 16, c["kst"], c["vst"])
    assert np.array_equal(kp.cpu().numpy().reshape(-1), rk)


@pytest.mark.parametrize("inplace", [False, True])
def test_compact_same_row_twice(inplace):
    """An entry may repeat: each copy holds the row."""
    c = compact_case("turbo4", [64], 6, 2, 64, seed=6)
    c["kept"][0, 0] = [3, 3, 9, 40, 40, 63]
    c["kept"][0, 1] = [0, 1, 2, 3, 63, 63]
    check_compact(c, inplace)


def test_pools_past_32_bits():
    """Blocks whose byte offset needs more than 32 bits: the same rows at low
    and at high block ids give the same results, moved and attended."""
    bs, nkv, hd, nq, n = 16, 8, 128, 32, 600
    nblk = 140000                                     # 32 KB a block: 4.6 GB a side
    need = -(-n // bs)
    kp = torch.zeros(nblk, bs * nkv * hd * 2, dtype=torch.uint8, device=DEV)
    vp = torch.zeros_like(kp)
    k = torch.randn(n, nkv, hd, device=DEV).bfloat16()
    v = torch.randn(n, nkv, hd, device=DEV).bfloat16()
    q = torch.randn(1, nq, hd, device=DEV).bfloat16()
    low = torch.arange(need, dtype=torch.int32, device=DEV)[None] + 1
    high = nblk - 1 - low
    lens = t(np.array([n], np.int32))
    got = []
    for tab, dst in ((low, low + need), (high, high - need)):
        slots = tab[0].long()[torch.arange(n, device=DEV) // bs] * bs + torch.arange(n, device=DEV) % bs
        ops.cache_write(k, v, kp, vp, slots, "bf16", nkv, hd, bs)
        tab, dst = tab.contiguous(), dst.contiguous()
        cu = t(np.array([0, 1], np.int32))
        m1 = ops.attention_mass(q, cu, 1, kp, tab, lens, "bf16", nkv, bs)
        m8 = ops.attention_mass(q.expand(8, -1, -1).contiguous(), t(np.array([0, 8], np.int32)), 8, kp, tab, lens, "bf16", nkv, bs)
        sh = ops.paged_decode_shared(q, kp, vp, tab, lens, cu, tab, t(np.array([20], np.int32)), "bf16", nkv, bs)
        kept, new = ops.evict_select(m1, lens, 100)
        ops.cache_compact(kp, vp, tab, lens, kept, "bf16", nkv, hd, bs, dst_tables=dst)
        out = ops.paged_decode(q, kp, vp, dst, new, "bf16", nkv, bs)
        ops.cache_compact(kp, vp, tab, lens, kept, "bf16", nkv, hd, bs)
        again = ops.paged_decode(q, kp, vp, tab, new, "bf16", nkv, bs)
        assert torch.equal(out, again)
        got.append((m1, m8, sh, kept, out))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert (got[0][0].sum(-1) - 4).abs().max() <= 1e-4


def test_two_calls_at_once():
    """Independent calls on two streams, each with its own workspace."""
    c = decode_case("turbo4", [700, 300], 8, 2, 128, seed=9)
    kp, vp = pools(c)
    tab, lens = t(c["tables"]), t(c["lens"])
    qs = [torch.randn(2, 8, 128, device=DEV) for _ in range(2)]
    cu = t(np.array([0, 1, 2], np.int32))
    run = lambda q, st=None: (ops.attention_mass(q, cu, 1, kp, tab, lens, "turbo4", 2, 16, stream=st),
                              ops.paged_decode_shared(q, kp, vp, tab[:1], lens[:1], cu[[0, 2]].contiguous(), tab, lens,
                                                      "turbo4", 2, 16, stream=st))
    want = [run(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [run(q, s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_compact_flags():
    c = compact_case("bf16", [64], 20, 2, 64, seed=4)

    def flags(kept=None, dst=None, tab=None, inplace=False):
        kp, vp = pools(c)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ops.cache_compact(kp, vp, t(c["tables"] if tab is None else tab), t(c["lens"]),
                          t(c["kept"] if kept is None else kept), "bf16", 2, 64, 16,
                          dst_tables=None if inplace else t(c["dst"] if dst is None else dst), error_flag=err)
        return err.item()

    bad = c["kept"].copy()
    bad[0, 0, 3] = 64
    assert flags(kept=bad) == _abi.KVQ_DEVERR_RANGE
    bad[0, 0, 3] = -7
    assert flags(kept=bad) == _abi.KVQ_DEVERR_RANGE
    bad[0, 0, 3] = 2                                          # below its own index: only other pages can take it
    assert flags(kept=bad, inplace=True) == _abi.KVQ_DEVERR_RANGE
    assert flags(kept=bad) == 0
    dst = c["dst"].copy()
    dst[0, 0] = 10 ** 6
    assert flags(dst=dst) == _abi.KVQ_DEVERR_BLOCK
    tab = c["tables"].copy()
    tab[0, 1] = -1
    assert flags(tab=tab) == _abi.KVQ_DEVERR_BLOCK


@pytest.mark.parametrize("inplace", [False, True])
def test_compact_short_weight_rows(inplace):
    """Rows of weights shorter than the sequence: positions past their end are
    skipped and flagged, and nothing is read there."""
    c = compact_case("bf16", [64, 50], 20, 2, 64, seed=5)
    rows = 40
    kept = np.full((2, 2, 20), -1, dtype=np.int32)
    kept[..., :3] = [7, rows - 1, rows]
    kp, vp = pools(c)
    ref = kp.clone()
    mass, out = t(np.arange(4 * rows, dtype=np.float32).reshape(2, 2, rows)), torch.full((2, 2, 20), -1.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tab, lens, kept, dst = t(c["tables"]), t(c["lens"]), t(kept), t(c["dst"])
    _abi.kvq_cache_compact(
        kp.data_ptr(), vp.data_ptr(), tab.data_ptr(), tab.shape[1], lens.data_ptr(), kept.data_ptr(), 20,
        None if inplace else dst.data_ptr(), 0 if inplace else dst.shape[1], 2, kp.shape[0], 2, 64, 16, kp.stride(0),
        vp.stride(0), mass.data_ptr(), rows, out.data_ptr(), 20, ops.fmt_id("bf16"), err.data_ptr(),
        torch.cuda.current_stream().cuda_stream)
    assert err.item() == _abi.KVQ_DEVERR_RANGE
    assert torch.equal(out[..., :2], mass[..., [7, rows - 1]])
    assert (out[..., 2:] == -1).all()
    rowb = 2 * 64 * 2                                         # bytes of a position: 2 heads of 64 bf16
    first = (tab if inplace else dst)[:, 0].long()
    page = kp[first].reshape(2, -1)
    assert torch.equal(page[:, 2 * rowb:3 * rowb], ref[first].reshape(2, -1)[:, 2 * rowb:3 * rowb])
    assert torch.equal(page[:, :rowb], ref[tab[:, 0].long()].reshape(2, -1)[:, 7 * rowb:8 * rowb])


def test_sizes_from_two_threads():
    """Calls of different sizes from two host threads: neither's launch limits
    touch the other's."""
    import threading
    c = compact_case("turbo4", [300], 200, 2, 64, seed=6)
    d = compact_case("bf16", [300], 200, 2, 256, seed=7)
    big = torch.rand(1, 1, 300_000, device=DEV)
    small = torch.rand(3, 2, 100, device=DEV)
    want = [ops.evict_select(m, torch.full((m.shape[0],), m.shape[2], dtype=torch.int32, device=DEV), k)[0]
            for m, k in ((big, 1000), (small, 9))]
    failures = []

    def work(m, keep, ref, case, hd, fmt):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                lens = torch.full((m.shape[0],), m.shape[2], dtype=torch.int32, device=DEV)
                kp, vp = pools(case)
                tab, clens, kept = t(case["tables"]), t(case["lens"]), t(case["kept"])
                for _ in range(300):
                    got = ops.evict_select(m, lens, keep)[0]
                    ops.cache_compact(kp, vp, tab, clens, kept, fmt, 2, hd, 16)
                if not torch.equal(got, ref):
                    failures.append("wrong positions")
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            failures.append(repr(e))

    threads = [threading.Thread(target=work, args=x) for x in
               ((big, 1000, want[0], c, 64, "turbo4"), (small, 9, want[1], d, 256, "bf16"))]
    torch.cuda.synchronize()
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not failures


# ------------------------------------------------------------------ as used together

def test_prompt_write_evict_decode():
    """Prompt attention, cache write, weights of the last queries, selection,
    compaction in place, a decode over the kept rows: the decode equals the
    attention over exactly those rows."""
    lens, nq, nkv, hd, keep = [400, 150, 60], 8, 2, 128, 96
    torch.manual_seed(0)
    total = sum(lens)
    q = torch.randn(total, nq, hd, device=DEV).bfloat16()
    k = torch.randn(total, nkv, hd, device=DEV).bfloat16()
    v = torch.randn(total, nkv, hd, device=DEV).bfloat16()
    cu = t(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    ops.prompt_attention(q, k, v, cu, 400, out_dtype=torch.bfloat16)
    need = [-(-n // 16) for n in lens]
    tab = torch.full((3, max(need)), -1, dtype=torch.int32)
    perm = torch.randperm(sum(need)).int()
    for s in range(3):
        tab[s, :need[s]] = perm[sum(need[:s]):sum(need[:s + 1])]
    tab = tab.to(DEV)
    kp = ops.alloc_pool(sum(need), "bf16", 0, 16, nkv, hd)
    vp = ops.alloc_pool(sum(need), "bf16", 1, 16, nkv, hd)
    slots = torch.cat([tab[s].long()[torch.arange(n, device=DEV) // 16] * 16 + torch.arange(n, device=DEV) % 16
                       for s, n in enumerate(lens)])
    ops.cache_write(k, v, kp, vp, slots, "bf16", nkv, hd, 16)
    sl = t(np.array(lens, np.int32))
    last = torch.cat([q[int(cu[s + 1]) - 8:int(cu[s + 1])] for s in range(3)])
    cq = t(np.array([0, 8, 16, 24], np.int32))
    mass = ops.attention_mass(last, cq, 8, kp, tab, sl, "bf16", nkv, 16)
    kept, new = ops.evict_select(mass, sl, keep, sink=4, recent=16)
    ops.cache_compact(kp, vp, tab, sl, kept, "bf16", nkv, hd, 16, mass=mass)
    assert new.tolist() == [96, 96, 60]
    qd = torch.randn(3, nq, hd, device=DEV)
    got = host(ops.paged_decode(qd, kp, vp, tab, new, "bf16", nkv, 16))
    kh, vh, kk = host(k), host(v), kept.cpu().numpy()
    for s in range(3):
        a, n = int(cu[s]), int(new[s])
        for h in range(nkv):
            rows = a + kk[s, h, :n]
            ref = oracle.attend(host(qd)[s, 4 * h:4 * h + 4], kh[rows][:, h:h + 1], vh[rows][:, h:h + 1])
            assert np.abs(got[s, 4 * h:4 * h + 4] - ref).max() <= 2e-3
    # a second round: the moved weights go on adding up, and select again
    mass2 = ops.attention_mass(qd, t(np.array([0, 1, 2, 3], np.int32)), 1, kp, tab, new, "bf16", nkv, 16, mass_in=mass,
                               mass_out=mass)
    kept2, new2 = ops.evict_select(mass2, new, 64, sink=4, recent=16)
    assert new2.tolist() == [64, 64, 60] and (kept2[:, :, :4].cpu() == torch.arange(4)).all()


def test_evict_streams_and_graphs():
    c = compact_case("turbo4", [300, 120], 64, 2, 128, seed=9)
    kp, vp = pools(c)
    kp0, vp0 = kp.clone(), vp.clone()
    q = torch.randn(2, 8, 128, device=DEV)
    cu, tab, lens = t(np.array([0, 1, 2], np.int32)), t(c["tables"]), t(c["lens"])
    mass = torch.zeros(2, 2, tab.shape[1] * 16, device=DEV)
    ws = ops.alloc_mass_workspace(2, 2, 1, 8, 2, 16, tab.shape[1])
    kept = torch.zeros(2, 2, 64, dtype=torch.int32, device=DEV)
    new = torch.zeros(2, dtype=torch.int32, device=DEV)

    def chain(stream=None):
        ops.attention_mass(q, cu, 1, kp, tab, lens, "turbo4", 2, 16, mass_out=mass, workspace=ws, stream=stream)
        ops.evict_select(mass, lens, 64, 2, 8, kept=kept, new_lens=new, stream=stream)
        ops.cache_compact(kp, vp, tab, lens, kept, "turbo4", 2, 128, 16, mass=mass, stream=stream)

    def reset(q2):
        kp.copy_(kp0); vp.copy_(vp0); mass.zero_(); q.copy_(q2)

    qs = [torch.randn(2, 8, 128, device=DEV) for _ in range(2)]
    want = []
    for x in qs:
        reset(x)
        chain()
        want.append([y.clone() for y in (kp, vp, mass, kept, new)])
    s = torch.cuda.Stream()
    reset(qs[0])
    s.wait_stream(torch.cuda.current_stream())
    chain(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip((kp, vp, mass, kept, new), want[0]))
    reset(qs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for x, w in zip(qs, want):
        reset(x)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip((kp, vp, mass, kept, new), w))


def mass_error_bound(c, q, cu, w, scale=None):
    """The bound of this file's head for totals that start from zero."""
    lens, nkv, nq, bs, hd = c["lens"], c["nkv"], c["nq"], c["bs"], c["hd"]
    side = oracle.kv_pair(c["fmt"])[0]
    qk, q = 0.0, host(q)
    for s, n in enumerate(int(x) for x in lens):
        pos = np.arange(n)
        k = np.abs(oracle.gather_side(c["kc"], side, c["tables"][s, pos // bs], pos % bs, nkv, hd, bs, c["kst"],
                                      c["k_scale"], to_original_basis=False))
        qs = q[cu[s]:cu[s + 1]]
        qs = np.abs(oracle.wht_f64(qs) if oracle.is_wht_rotated(side) else qs)
        qk = max([qk] + [(qs[:, j] @ k[:, j * nkv // nq].T).max() for j in range(nq)])
    u = 2.0 ** -24
    d = (scale or 1 / math.sqrt(hd)) * math.log2(math.e) * qk * (2.0 ** -20 + (hd + 4) * u)
    rows = max(np.diff(cu)) * nq // nkv
    return w * (4 * d + 2.0 ** -18) + u * w * (rows + 2)


@pytest.mark.parametrize("fmt", ["bf16", "turbo4"])
def test_mass_workspace_of_a_larger_chunk(fmt):
    """A workspace sized for chunks of 32 queries serves every smaller chunk of
    the same batch, single queries among them."""
    lens, nq, nkv, bs = [300, 2000, 17], 8, 2, 16
    c = decode_case(fmt, lens, nq, nkv, 128, seed=9)
    kp, _ = pools(c)
    size = ops.mass_workspace_bytes(3 * 32, 3, 32, nq, nkv, bs, c["tables"].shape[1])
    for chunk in (32, 3, 2, 1):
        cu = np.concatenate([[0], np.cumsum([min(chunk, n) for n in lens])]).astype(np.int32)
        q = t(np.random.default_rng(chunk).standard_normal((int(cu[-1]), nq, 128)).astype(np.float32))
        out = ops.attention_mass(q, t(cu), chunk, kp, t(c["tables"]), t(c["lens"]), fmt, nkv, bs,
                                 workspace=torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV))
        w = oracle.attention_mass(host(q), cu, c["kc"], c["tables"], c["lens"], nkv, 128, bs, c["kst"], fmt, out.shape[2])
        assert (np.abs(host(out) - w) <= mass_error_bound(c, q, cu, w)).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4", "turbo4", "turbo8"])
@pytest.mark.parametrize("factor", [2.0 ** 17, 2.0 ** -20])
@pytest.mark.parametrize("chunk", [1, 20])
def test_mass_query_magnitudes(fmt, factor, chunk):
    """Queries past the range of fp16, above and below, with a score scale that
    brings the scores back: the weights of the same queries at size one."""
    c = decode_case(fmt, [200, 33], 8, 2, 128, seed=10)
    kp, _ = pools(c)
    cu = np.array([0, chunk, 2 * chunk], np.int32)
    q = t(np.random.default_rng(11).standard_normal((2 * chunk, 8, 128)).astype(np.float32))
    scale = 128 ** -0.5
    out = ops.attention_mass(q * factor, t(cu), chunk, kp, t(c["tables"]), t(c["lens"]), fmt, 2, 16,
                             sm_scale=scale / factor, k_scale=c["k_scale"])
    w = oracle.attention_mass(host(q), cu, c["kc"], c["tables"], c["lens"], 2, 128, 16, c["kst"], fmt, out.shape[2],
                              k_scale=c["k_scale"], sm_scale=scale)
    assert (np.abs(host(out) - w) <= mass_error_bound(c, q, cu, w, scale)).all()
